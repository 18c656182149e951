"""Latent attention against plain 64-bit formulas: append with norm and rotation,
gather, the expanded and the absorbed attention, and a serving run of all four.

Tolerances, from the inputs and in FP64 (u = half a step of the 16-bit type):
* rows: rotation, norm and weight are a few FP32 operations (2^-24 each; rsqrtf
  2^-22.4 relative, the sum of 512 squares 2^-20 at most) rounded once: u + 2^-19
  relative of the terms' magnitudes, |x cos| + |y sin| for a rotated value.
* attention: a score is off by at most ds = K 2^-23 scale sum|q k| (K products
  accumulated with truncation, at most 2^-23 each) plus 2^-22 of its size (the FP32
  scaling); its weight by 2 ds relative (ds < 0.1) plus ex2.approx's 2^-22; the
  weight is rounded to 16 bits (u) for the product with the values, which
  accumulates n of them (n 2^-23), and the output is rounded once (u |o|):
  |do| <= u |o| + (u + 4 ds + (n + 16) 2^-22) sum p|v|,
  |dlse| <= 2 ds + (n + 16) 2^-22 + 2^-22 |lse|.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
C, R, NOPE, V = 512, 64, 128, 128
ROW = C + R
SCALE = 1.0 / math.sqrt(NOPE + R)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gqa_softmax_attention_gb300 import build
    build.build()
    import gqa_softmax_attention_gb300 as m
    yield m
    m.gqa_device_error()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def sums(x):
    out = [0]
    for n in x:
        out.append(out[-1] + n)
    return out


def unit(dt):
    return torch.finfo(dt).eps / 2


def attend(q, k, v, at, scale):
    """o, lse and the tolerances of both for queries q [n, d] at key positions `at`, in 64 bits."""
    q, k, v = q.double(), k.double(), v.double()
    n = k.shape[0]
    z = q @ k.t() * scale
    seen = torch.arange(n, device=q.device) <= at[:, None]
    z = z.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(z, 1) if n else torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.exp(z - lse.nan_to_num(neginf=0.0)[:, None])
    mag = (q.abs() @ k.abs().t() * abs(scale)).masked_fill(~seen, 0.0)
    ds = (q.shape[1] * 2.0 ** -23 * mag.amax(1) if n else torch.zeros_like(lse)) + 2.0 ** -22 * \
        (z.masked_fill(~seen, 0.0).abs().amax(1) if n else torch.zeros_like(lse))
    acc = (n + 16) * 2.0 ** -22
    return p @ v, lse, p @ v.abs(), ds, acc


def check(o, lse, ref, label):
    ro, rl, mag, ds, acc = ref
    u = unit(o.dtype)
    o, lse = o.double(), lse.double()
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty), label + ": other rows are empty"
    assert bool((o[empty] == 0).all()), label + ": an empty row is not zero"
    tol = u * ro.abs() + (u + 4 * ds + acc)[:, None] * mag + 2.0 ** -25
    bad = ((o - ro).abs() - tol).max().item() if o.numel() else -1
    assert bad <= 0, "%s: o off by %.3e more than allowed (max diff %.3e)" % (label, bad, (o - ro).abs().max().item())
    ok = ~empty
    d = (lse - rl)[ok].abs() - (2 * ds + acc + 2.0 ** -22 * rl.abs())[ok]
    assert not d.numel() or d.max().item() <= 0, "%s: lse off by %.3e too much" % (label, d.max().item())


# ---------------------------------------------------------------- absorbed, paged

def paged_case(gen, nq, lens, H, ps, dt, spare=3, scale=1.0):
    pages = [-(-n // ps) for n in lens]
    num_pages = sum(pages) + spare
    perm = torch.randperm(num_pages, generator=gen).tolist()
    table = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32)
    k = 0
    for b, n in enumerate(pages):
        for p in range(n):
            table[b, p] = perm[k]
            k += 1
    cache = (scale * torch.randn(num_pages, ps, ROW, generator=gen)).to(dt)
    used = torch.zeros(num_pages, ps, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[table[b, t // ps], t % ps] = True
    cache[~used] = math.nan                                    # no slot past a request's end may matter
    q = torch.randn(sum(nq), H, ROW, generator=gen).to(dt)
    return dict(q=q.cuda(), cache=cache.cuda(), cu=i32(sums(nq)), lens=i32(lens), table=table.cuda(), nq=nq, L=lens, H=H,
                ps=ps)


def paged_refs(c, causal=True, scale=SCALE):
    cu = sums(c["nq"])
    for b, (n, L) in enumerate(zip(c["nq"], c["L"])):
        t = torch.arange(L, device="cuda")
        rows = c["cache"].flatten(0, 1)[c["table"][b].long()[t // c["ps"]] * c["ps"] + t % c["ps"]] if L else \
            c["cache"].flatten(0, 1)[:0]
        at = torch.arange(n, device="cuda") + (L - n) if causal else torch.full((n,), L, device="cuda")
        yield b, slice(cu[b], cu[b + 1]), attend(c["q"][cu[b]:cu[b + 1]].flatten(0, 1), rows, rows[:, :C],
                                                 at.repeat_interleave(c["H"]), scale)


def paged_check(g, c, causal=True, scale=SCALE, **kw):
    o, lse = g.attn_fwd_latent_paged(c["q"], c["cache"], c["cu"], c["lens"], c["table"], scale, causal=causal, **kw)
    torch.cuda.synchronize()
    g.gqa_device_error()
    for b, rows, ref in paged_refs(c, causal, scale):
        check(o[rows].flatten(0, 1), lse[rows].flatten(), ref, "request %d" % b)
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,ps", [(16, 64), (128, 64), (40, 16), (1, 8), (20, 24), (64, 128), (8, 1), (16, 5)])
def test_absorbed_decode(g, H, ps, dtype):
    lens = [1, 127, 128, 129, 700, 5, 64, 0, 2049]
    paged_check(g, paged_case(torch.Generator().manual_seed(H + ps), [1] * len(lens), lens, H, ps, DT[dtype]))


@pytest.mark.parametrize("H,ps", [(16, 64), (128, 16), (20, 24), (3, 1)])
def test_absorbed_ragged_queries(g, H, ps):
    nq = [4, 0, 1, 37, 2, 130, 5, 1]
    lens = [300, 50, 1, 37, 1000, 400, 3, 0]                   # the last but one has fewer keys than queries
    c = paged_case(torch.Generator().manual_seed(H), nq, lens, H, ps, torch.bfloat16)
    paged_check(g, c)
    paged_check(g, c, causal=False)


def test_absorbed_one_long_request(g):
    """Cut into as many pieces as there are teams, and two requests of it."""
    gen = torch.Generator().manual_seed(5)
    for H, nq, lens in ((16, [1], [40001]), (128, [2], [20011]), (5, [3, 1], [30000, 12345])):
        paged_check(g, paged_case(gen, nq, lens, H, 64, torch.bfloat16, spare=0))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_absorbed_growing_scores(g, dtype):
    """Scores that rise along the keys move the reference maximum in every tile."""
    gen = torch.Generator().manual_seed(7)
    c = paged_case(gen, [1, 3], [1500, 900], 16, 64, DT[dtype])
    c["q"][..., C:] = 0
    c["q"][..., C] = 4.0
    t = torch.arange(1500, device="cuda")
    for b, L in enumerate(c["L"]):
        rows = c["table"][b].long()[t[:L] // 64] * 64 + t[:L] % 64
        c["cache"].view(-1, ROW)[rows, C] = (t[:L] / 8.0).to(DT[dtype])
    paged_check(g, c)
    paged_check(g, c, scale=-SCALE)
    paged_check(g, c, scale=0.0)


def test_absorbed_page_ids_outside_the_pool_read_as_zeros(g):
    c = paged_case(torch.Generator().manual_seed(9), [1, 2], [300, 200], 16, 16, torch.bfloat16)
    c["table"][0, 3] = -1
    c["table"][1, 0] = c["cache"].shape[0]
    o, lse = g.attn_fwd_latent_paged(c["q"], c["cache"], c["cu"], c["lens"], c["table"], SCALE)
    cu = sums(c["nq"])
    for b, (n, L) in enumerate(zip(c["nq"], c["L"])):
        t = torch.arange(L, device="cuda")
        page = c["table"][b].long()[t // 16]
        ok = (page >= 0) & (page < c["cache"].shape[0])
        rows = torch.where(ok[:, None], c["cache"].flatten(0, 1)[torch.where(ok, page * 16 + t % 16, 0)], 0.0)
        at = (torch.arange(n, device="cuda") + (L - n)).repeat_interleave(16)
        check(o[cu[b]:cu[b + 1]].flatten(0, 1), lse[cu[b]:cu[b + 1]].flatten(),
              attend(c["q"][cu[b]:cu[b + 1]].flatten(0, 1), rows, rows[:, :C], at, SCALE), "request %d" % b)


def test_absorbed_query_that_is_no_number(g):
    """Its own row is NaN, every other one as it was."""
    c = paged_case(torch.Generator().manual_seed(10), [1, 1, 1], [3000, 100, 700], 16, 64, torch.bfloat16)
    o, lse = g.attn_fwd_latent_paged(c["q"], c["cache"], c["cu"], c["lens"], c["table"], SCALE)
    c["q"][0, 3, 100] = math.nan
    c["q"][2, 5, 570] = math.inf
    o2, lse2 = g.attn_fwd_latent_paged(c["q"], c["cache"], c["cu"], c["lens"], c["table"], SCALE)
    for r, h in ((0, 3), (2, 5)):
        assert bool(o2[r, h].isnan().all()) and bool(lse2[r, h].isnan())
        o2[r, h], lse2[r, h] = o[r, h], lse[r, h]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_absorbed_padding_rows_stay(g):
    c = paged_case(torch.Generator().manual_seed(11), [1, 2], [100, 200], 16, 64, torch.bfloat16)
    q = torch.cat([c["q"], c["q"][:2]])
    out = torch.full((5, 16, C), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 16), 7.0, device="cuda")
    g.attn_fwd_latent_paged(q, c["cache"], c["cu"], c["lens"], c["table"], SCALE, out=out, lse=lse)
    assert bool((out[3:] == 7).all()) and bool((lse[3:] == 7).all())
    for b, rows, ref in paged_refs(c):
        check(out[rows].flatten(0, 1), lse[rows].flatten(), ref, "request %d" % b)


def test_absorbed_runs_alike_and_in_graphs(g):
    """Bitwise equal runs; a captured call follows new lengths, tables and queries; another stream."""
    gen = torch.Generator().manual_seed(12)
    c = paged_case(gen, [1] * 6, [3000, 1, 900, 128, 0, 4000], 16, 64, torch.bfloat16)
    args = (c["q"], c["cache"], c["cu"], c["lens"], c["table"], SCALE)
    o, lse = g.attn_fwd_latent_paged(*args)
    o1, lse1 = g.attn_fwd_latent_paged(*args)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2 = g.attn_fwd_latent_paged(*args)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = g.attn_fwd_latent_paged(*args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, og) and torch.equal(lse, lg)
    c["L"] = [5, 2000, 0, 129, 700, 64]
    pool = torch.randperm(c["cache"].shape[0], generator=gen).int().cuda()
    c["cache"].nan_to_num_(0.5)
    width = c["table"].shape[1]
    c["table"].copy_(pool[:6 * width].view(6, width) if pool.numel() >= 6 * width else
                     pool[torch.arange(6 * width, device="cuda") % pool.numel()].view(6, width))
    c["lens"].copy_(i32(c["L"]))
    c["q"].copy_(randn(gen, 6, 16, ROW))
    graph.replay()
    torch.cuda.synchronize()
    for b, rows, ref in paged_refs(c):
        check(og[rows].flatten(0, 1), lg[rows].flatten(), ref, "replayed, request %d" % b)


def test_absorbed_far_rows(g):
    """Cache rows past 2^31 elements and 4 GiB."""
    dev, ps = "cuda", 64
    pages = (5 << 30) // (ps * ROW * 2)
    cache = torch.empty(pages, ps, ROW, dtype=torch.bfloat16, device=dev)
    gen = torch.Generator().manual_seed(13)
    lens = [200, 130]
    table = i32([[pages - 1, 0, pages - 3, pages // 2], [pages - 2, pages - 4, 7, -1]])
    for p in table.flatten().tolist():
        if p >= 0:
            cache[p] = randn(gen, ps, ROW)
    c = dict(q=randn(gen, 3, 16, ROW), cache=cache, cu=i32([0, 1, 3]), lens=i32(lens), table=table, nq=[1, 2], L=lens, H=16,
             ps=ps)
    paged_check(g, c)


# ---------------------------------------------------------------- expanded

def varlen_case(gen, nq, lens, H, dt):
    kv = torch.randn(sum(lens), H, NOPE + V, generator=gen).to(dt).cuda()
    rows = torch.randn(sum(lens), ROW, generator=gen).to(dt).cuda()
    return dict(q=torch.randn(sum(nq), H, NOPE + R, generator=gen).to(dt).cuda(), k=kv[..., :NOPE], v=kv[..., NOPE:],
                pe=rows[:, C:], cq=i32(sums(nq)), ck=i32(sums(lens)), nq=nq, L=lens, H=H)


def varlen_refs(c, causal=True, scale=SCALE):
    cq, ck = sums(c["nq"]), sums(c["L"])
    for b, (n, L) in enumerate(zip(c["nq"], c["L"])):
        at = torch.arange(n, device="cuda") + (L - n) if causal else torch.full((n,), L, device="cuda")
        for h in range(c["H"]):
            k = torch.cat([c["k"][ck[b]:ck[b + 1], h], c["pe"][ck[b]:ck[b + 1]]], 1)
            yield b, h, slice(cq[b], cq[b + 1]), attend(c["q"][cq[b]:cq[b + 1], h], k, c["v"][ck[b]:ck[b + 1], h], at,
                                                       scale)


def varlen_check(g, c, causal=True, scale=None):
    o, lse = g.attn_fwd_latent_varlen(c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"], causal=causal, scale=scale)
    torch.cuda.synchronize()
    g.gqa_device_error()
    for b, h, rows, ref in varlen_refs(c, causal, SCALE if scale is None else scale):
        check(o[rows, h], lse[rows, h], ref, "request %d head %d" % (b, h))
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nq,lens,H", [
    ([1], [1], 1),
    ([128], [128], 2),
    ([129, 1, 300], [129, 1, 300], 3),
    ([256, 257, 63], [256, 700, 1000], 2),
    ([5, 0, 1, 40], [2000, 10, 900, 40], 4),
    ([300, 20], [100, 0], 2),                                 # rows without a key, a request without any
])
def test_expanded(g, nq, lens, H, dtype):
    c = varlen_case(torch.Generator().manual_seed(sum(nq) + H), nq, lens, H, DT[dtype])
    varlen_check(g, c)
    varlen_check(g, c, causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nq,lens,H", [
    ([300], [5000], 3),                                       # six items, ten parts each
    ([1], [9001], 1),                                         # one row
    ([700, 3, 129], [3000, 2500, 1100], 20),                  # a tail behind whole rounds, shorter requests in it
    ([200, 50], [100, 2000], 5),                              # rows without a key among cut items
    ([2048, 1], [2048, 4000], 19),
])
def test_expanded_cut_along_the_keys(g, nq, lens, H, dtype):
    c = varlen_case(torch.Generator().manual_seed(sum(lens) + H), nq, lens, H, DT[dtype])
    o, lse = varlen_check(g, c)
    varlen_check(g, c, causal=False)
    # the least workspace: nothing is cut
    ws = torch.empty(g.attn_varlen_workspace_size(len(nq), sum(nq), H, H), dtype=torch.uint8, device="cuda")
    o2, lse2 = g.attn_fwd_latent_varlen(c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"], workspace=ws)
    for b, h, rows, ref in varlen_refs(c):
        check(o2[rows, h], lse2[rows, h], ref, "uncut, request %d head %d" % (b, h))
    o3, lse3 = g.attn_fwd_latent_varlen(c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"])
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


def test_expanded_in_a_graph(g):
    """A captured call follows new offsets, lengths and values, cut or not."""
    gen = torch.Generator().manual_seed(23)
    c = varlen_case(gen, [200, 56], [3000, 1000], 4, torch.bfloat16)
    args = (c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"])
    g.attn_fwd_latent_varlen(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = g.attn_fwd_latent_varlen(*args)
    for nq, lens in (([200, 56], [3000, 1000]), ([1, 255], [60, 3940]), ([256, 0], [500, 3500])):
        c["nq"], c["L"] = nq, lens
        c["cq"].copy_(i32(sums(nq)))
        c["ck"].copy_(i32(sums(lens)))
        c["q"].copy_(randn(gen, 256, 4, 192))
        graph.replay()
        torch.cuda.synchronize()
        for b, h, rows, ref in varlen_refs(c):
            check(o[rows, h], lse[rows, h], ref, "request %d head %d" % (b, h))
    g.gqa_device_error()


def test_expanded_many_items(g):
    """More items than CTAs, requests of every length."""
    nq = [1, 513, 130, 7, 255, 384, 2, 900]
    varlen_check(g, varlen_case(torch.Generator().manual_seed(3), nq, [n + 11 * i for i, n in enumerate(nq)], 40,
                                torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_expanded_growing_scores(g, dtype):
    c = varlen_case(torch.Generator().manual_seed(4), [700], [1000], 2, DT[dtype])
    c["q"][..., NOPE] = 4.0
    c["pe"][:, 0] = torch.arange(1000, device="cuda") / 8.0
    varlen_check(g, c)
    varlen_check(g, c, scale=-SCALE)
    varlen_check(g, c, scale=0.0)


def test_expanded_neighbours_that_are_no_numbers(g):
    """What lies behind a request's rows does not matter to it."""
    c = varlen_case(torch.Generator().manual_seed(5), [100, 50, 30], [200, 90, 30], 2, torch.bfloat16)
    c["k"][200:290], c["v"][200:290], c["pe"][200:290] = math.nan, math.inf, math.nan
    o, lse = g.attn_fwd_latent_varlen(c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"])
    for b, h, rows, ref in varlen_refs(c):
        if b != 1:
            check(o[rows, h], lse[rows, h], ref, "request %d head %d" % (b, h))


def test_expanded_layouts(g):
    """Dense, sliced, head-major and unaligned k, v and k_pe give one result; padding rows stay."""
    c = varlen_case(torch.Generator().manual_seed(6), [60, 140], [100, 140], 4, torch.bfloat16)
    o, lse = varlen_check(g, c)
    odd = torch.zeros(240, 4 * 128 + 1, dtype=torch.bfloat16, device="cuda")[:, 1:].unflatten(1, (4, 128))
    odd.copy_(c["v"])
    for k, v, pe in ((c["k"].contiguous(), c["v"].contiguous(), c["pe"].contiguous()),
                     (c["k"].transpose(0, 1).contiguous().transpose(0, 1), odd, c["pe"])):
        o2, lse2 = g.attn_fwd_latent_varlen(c["q"], k, v, pe, c["cq"], c["ck"])
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    shared = c["k"][:, :1].expand(240, 4, 128)                # one head's keys for all
    o3, lse3 = g.attn_fwd_latent_varlen(c["q"], shared, c["v"], c["pe"], c["cq"], c["ck"])
    o4, lse4 = g.attn_fwd_latent_varlen(c["q"], shared.contiguous(), c["v"], c["pe"], c["cq"], c["ck"])
    assert torch.equal(o3, o4) and torch.equal(lse3, lse4)
    out = torch.full((203, 4, V), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((203, 4), 7.0, device="cuda")
    q = torch.cat([c["q"], c["q"][:3]])
    g.attn_fwd_latent_varlen(q, c["k"], c["v"], c["pe"], c["cq"], c["ck"], out=out, lse=lse)
    assert bool((out[200:] == 7).all()) and bool((lse[200:] == 7).all()) and torch.equal(out[:200], o)


# ---------------------------------------------------------------- rows

def turned(x, cos_sin, pos, interleaved):
    """R(p) x in 64 bits and the magnitude of its terms, x [T, ..., 64]."""
    h = R // 2
    t = cos_sin.double()[pos.long()].view(x.shape[0], *[1] * (x.dim() - 2), R)
    co, si = t[..., :h], t[..., h:]
    x = x.double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    pairs = (a * co - b * si, b * co + a * si), ((a * co).abs() + (b * si).abs(), (b * co).abs() + (a * si).abs())
    return tuple(torch.stack(p, -1).flatten(-2) if interleaved else torch.cat(p, -1) for p in pairs)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,H,interleaved,weight", [(1, 1, True, "same"), (5, 128, False, "f32"), (300, 20, True, None),
                                                    (1000, 33, False, "same")])
def test_append(g, T, H, interleaved, weight, dtype):
    dt, gen, ps, pages = DT[dtype], torch.Generator().manual_seed(T + H), 24, T // 24 + 5
    q = torch.randn(T, H, NOPE + R, generator=gen).to(dt).cuda()
    kv = (3 * torch.randn(T, ROW + 8, generator=gen)).to(dt).cuda()[:, :ROW]
    w = None
    if weight:
        w = (1 + 0.3 * torch.randn(C, generator=gen)).cuda()
        w = w if weight == "f32" else w.to(dt)
    pos = torch.randint(0, 500, (T,), generator=gen).int().cuda()
    slots = torch.randperm(pages * ps, generator=gen)[:T].int().cuda()
    if T > 2:
        slots[1], slots[2] = -1, pages * ps                    # padding
    real = (slots >= 0) & (slots < pages * ps)
    cs = g.rope_table(500, R)
    cache = torch.full((pages, ps, ROW), 7.0, dtype=dt, device="cuda")
    q_abs = torch.full((T, H, ROW), 7.0, dtype=dt, device="cuda")
    packed = torch.full((T, ROW), 7.0, dtype=dt, device="cuda")
    out = g.attn_latent_norm_rope_paged(q[..., NOPE:], kv, cs, pos, slots, cache, kv_weight=w, interleaved=interleaved,
                                        out=q_abs[..., C:], kv_out=packed)
    torch.cuda.synchronize()
    assert out.data_ptr() == q_abs[..., C:].data_ptr()
    assert bool((q_abs[..., :C] == 7).all()) and bool((q_abs[~real] == 7).all()) and bool((packed[~real] == 7).all())
    u = unit(dt) + 2.0 ** -19
    want, mag = turned(q[..., NOPE:], cs, pos, interleaved)
    assert bool(((q_abs[..., C:].double() - want).abs() <= u * mag + 2.0 ** -25)[real].all())
    c = kv[:, :C].double()
    if w is not None:
        c = c / (c.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    pe, pe_mag = turned(kv[:, C:], cs, pos, interleaved)
    rows, mag = torch.cat([c, pe], 1), torch.cat([c.abs(), pe_mag], 1)
    assert bool(((packed.double() - rows).abs() <= u * mag + 2.0 ** -25)[real].all())
    flat = cache.view(-1, ROW)
    assert torch.equal(flat[slots[real].long()], packed[real])
    rest = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    rest[slots[real].long()] = False
    assert bool((flat[rest] == 7).all())
    # in place, and from one fused projection
    fused = torch.cat([q.flatten(1), kv, torch.zeros(T, 8, dtype=dt, device="cuda")], 1)
    q2, kv2 = fused[:, :H * (NOPE + R)].unflatten(1, (H, NOPE + R))[..., NOPE:], fused[:, H * (NOPE + R):][:, :ROW]
    cache2 = torch.full_like(cache, 7.0)
    g.attn_latent_norm_rope_paged(q2, kv2, cs, pos, slots, cache2, kv_weight=w, interleaved=interleaved, out=q2)
    assert torch.equal(cache2, cache) and torch.equal(q2[real], q_abs[..., C:][real])
    dense = kv.contiguous()
    g.attn_latent_norm_rope_paged(q[..., NOPE:], dense, cs, pos, slots, torch.empty_like(cache), kv_weight=w,
                                  interleaved=interleaved, kv_out=dense)
    assert torch.equal(dense[real], packed[real]) and torch.equal(dense[~real], kv[~real])


@pytest.mark.parametrize("ps,lens", [(16, [0, 1, 33, 0, 200, 64]), (1, [5, 3]), (64, [1000] * 40), (24, [0])])
def test_gather(g, ps, lens):
    gen = torch.Generator().manual_seed(ps)
    c = paged_case(gen, [1] * len(lens), lens, 1, ps, torch.float16)
    c["cache"].nan_to_num_(9.0)
    cu, total = sums(lens), sum(lens) + 5
    if sum(lens) > 150:
        c["table"][lens.index(max(lens)), 1] = -1
    out = torch.full((total, ROW), 7.0, dtype=torch.float16, device="cuda")
    got = g.attn_latent_gather(c["cache"], i32(cu), c["table"], total, out=out)
    assert got is out and bool((out[sum(lens):] == 7).all())
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        page = c["table"][b].long()[t // ps]
        want = torch.where((page >= 0)[:, None], c["cache"].flatten(0, 1)[page.clamp(min=0) * ps + t % ps], 0.0)
        assert torch.equal(out[cu[b]:cu[b + 1]], want)
    assert torch.equal(g.attn_latent_gather(c["cache"], i32(cu), c["table"], cu[-1]), out[:cu[-1]])


# ---------------------------------------------------------------- together

def test_serving_run(g):
    """A prompt in its expanded form, a second chunk over gathered rows, then decode
    steps in the absorbed form: one causal attention over the whole sequences."""
    gen, H, ps, dt = torch.Generator().manual_seed(20), 20, 16, torch.bfloat16
    B, max_pages = 3, 40
    w_k = (torch.randn(H, NOPE, C, generator=gen) / math.sqrt(C)).to(dt).cuda()
    w_v = (torch.randn(H, V, C, generator=gen) / math.sqrt(C)).to(dt).cuda()
    weight = (1 + 0.2 * torch.randn(C, generator=gen)).to(dt).cuda()
    cs = g.rope_table(max_pages * ps, R)
    cache = torch.zeros(B * max_pages, ps, ROW, dtype=dt, device="cuda")
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(B * max_pages, generator=gen).int().cuda()
    start, past = torch.zeros(1, dtype=torch.int32, device="cuda"), [0] * B
    rows_all, steps = [[] for _ in range(B)], [[100, 33, 260], [57, 1, 140], [1, 1, 1], [2, 0, 1], [1, 1, 1]]
    for n, new in enumerate(steps):
        T = sum(new)
        cu, lens, slots, pos, req, counts = g.attn_paged_slots(i32(past), i32(new), table, free, ps, B * max_pages, T,
                                                               free_start=start)
        start = counts[2:].clone()
        q = torch.randn(T, H, NOPE + R, generator=gen).to(dt).cuda()
        kv = torch.randn(T, ROW, generator=gen).to(dt).cuda()
        past = [p + x for p, x in zip(past, new)]
        packed = torch.empty_like(kv)
        if n < 2:
            g.attn_latent_norm_rope_paged(q[..., NOPE:], kv, cs, pos, slots, cache, kv_weight=weight, out=q[..., NOPE:],
                                          kv_out=packed)
            ck = i32(sums(past))
            rows = packed if n == 0 else g.attn_latent_gather(cache, ck, table, sum(past))
            k = torch.einsum("tc,hdc->thd", rows[:, :C], w_k)
            v = torch.einsum("tc,hdc->thd", rows[:, :C], w_v)
            o, lse = g.attn_fwd_latent_varlen(q, k, v, rows[:, C:], cu, ck)
        else:
            q_abs = torch.empty(T, H, ROW, dtype=dt, device="cuda")
            q_abs[..., :C] = torch.einsum("thd,hdc->thc", q[..., :NOPE], w_k)
            g.attn_latent_norm_rope_paged(q[..., NOPE:], kv, cs, pos, slots, cache, kv_weight=weight, out=q_abs[..., C:],
                                          kv_out=packed)
            o, lse = g.attn_fwd_latent_paged(q_abs, cache, cu, lens, table, SCALE)
        torch.cuda.synchronize()
        at = sums(new)
        for b in range(B):
            rows_all[b].append(packed[at[b]:at[b + 1]])
            rows, nq = torch.cat(rows_all[b]).double(), new[b]
            if nq == 0:
                continue
            t = torch.arange(past[b], device="cuda")
            assert torch.equal(cache.view(-1, ROW)[table[b].long()[t // ps] * ps + t % ps], rows.to(dt))
            seen = torch.arange(nq, device="cuda") + past[b] - nq
            if n < 2:
                # the products' 16-bit keys and values are the attention's inputs
                for h in range(H):
                    kb = torch.cat([k[sums(past)[b]:sums(past)[b + 1], h], rows[:, C:].to(dt)], 1)
                    check(o[at[b]:at[b + 1], h], lse[at[b]:at[b + 1], h],
                          attend(q[at[b]:at[b + 1], h], kb, v[sums(past)[b]:sums(past)[b + 1], h], seen, SCALE),
                          "step %d request %d head %d" % (n, b, h))
            else:
                check(o[at[b]:at[b + 1]].flatten(0, 1), lse[at[b]:at[b + 1]].flatten(),
                      attend(q_abs[at[b]:at[b + 1]].flatten(0, 1), rows, rows[:, :C], seen.repeat_interleave(H), SCALE),
                      "step %d request %d" % (n, b))
    g.gqa_device_error()


def test_both_forms_agree(g):
    """The absorbed output times the value projection is the expanded one: in 64-bit
    projections of FP32 inputs they are one function, so what differs is the rounding of
    q W_k, k and v to 16 bits (u relative of sqrt(C) terms each, about 4 u on values
    of size one, and scores moved by about 6 u): 16 u is left of it."""
    gen, H, n = torch.Generator().manual_seed(21), 8, 200
    dt = torch.float16
    rows = torch.randn(n, ROW, generator=gen).to(dt).cuda()
    w_k, w_v = ((torch.randn(H, NOPE, C, generator=gen) / math.sqrt(C)).cuda() for _ in range(2))
    q = torch.randn(n, H, NOPE + R, generator=gen).to(dt).cuda()
    k = torch.einsum("tc,hdc->thd", rows[:, :C].double(), w_k.double()).to(dt)
    v = torch.einsum("tc,hdc->thd", rows[:, :C].double(), w_v.double()).to(dt)
    o1, lse1 = g.attn_fwd_latent_varlen(q, k, v, rows[:, C:], i32([0, n]), i32([0, n]))
    q_abs = torch.cat([torch.einsum("thd,hdc->thc", q[..., :NOPE].double(), w_k.double()).to(dt), q[..., NOPE:]], 2)
    cache = torch.zeros(4, 64, ROW, dtype=dt, device="cuda")
    cache.view(-1, ROW)[:n] = rows
    o2, lse2 = g.attn_fwd_latent_paged(q_abs, cache, i32([0, n]), i32([n]), i32([[0, 1, 2, 3]]), SCALE)
    o2 = torch.einsum("thc,hdc->thd", o2.double(), w_v.double())
    d = (o1.double() - o2).abs()
    assert d.max().item() <= 16 * unit(dt) * 4 and d.mean().item() <= 16 * unit(dt), (d.max().item(), d.mean().item())
    assert (lse1 - lse2).abs().max().item() <= 32 * unit(dt)


def test_expanded_blocks_without_a_partner(g):
    """Many requests of one row block each, and some without a key: items of which one
    or both query tiles take no part, among others that do; no wait may give up."""
    gen = torch.Generator().manual_seed(22)
    nq = [int(x) for x in torch.randint(1, 129, (150,), generator=gen)]
    nq[::7] = [300] * len(nq[::7])
    lens = [n + 5 * (i % 3) for i, n in enumerate(nq)]
    lens[3::10] = [0] * len(lens[3::10])
    c = varlen_case(gen, nq, lens, 4, torch.bfloat16)
    args = (c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"])
    o, lse = g.attn_fwd_latent_varlen(*args)
    for _ in range(300):
        o2, lse2 = g.attn_fwd_latent_varlen(*args)
    torch.cuda.synchronize()
    g.gqa_device_error()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for b, h, rows, ref in varlen_refs(c):
        check(o[rows, h], lse[rows, h], ref, "request %d head %d" % (b, h))


# ---------------------------------------------------------------- odd calls

@pytest.mark.parametrize("H", [8, 40])
def test_absorbed_most_requests(g, H):
    """16384 requests of one key: its latent, whatever the query.  One more is refused."""
    gen = torch.Generator().manual_seed(29)
    B, ps = 16384, 8
    cache, q = randn(gen, 100, ps, ROW), randn(gen, 64, H, ROW).repeat(B // 64, 1, 1)
    table = torch.randint(0, 100, (B, 1), generator=gen).int().cuda()
    cu, lens = torch.arange(B + 1).int().cuda(), torch.ones(B, dtype=torch.int32, device="cuda")
    o, _ = g.attn_fwd_latent_paged(q, cache, cu, lens, table, SCALE)
    assert torch.equal(o, cache[table[:, 0].long(), 0, :C][:, None].expand(B, H, C))
    with pytest.raises((ValueError, RuntimeError), match="unsupported"):
        g.attn_fwd_latent_paged(q, cache, torch.arange(B + 2).int().cuda(), torch.ones(B + 1).int().cuda(),
                                torch.zeros(B + 1, 1).int().cuda(), SCALE)


def test_absorbed_many_requests(g):
    """More requests than threads of a CTA, most of them short or without queries."""
    gen = torch.Generator().manual_seed(30)
    lens = [int(x) for x in torch.randint(0, 40, (900,), generator=gen)]
    lens[17], lens[500] = 3000, 777
    nq = [int(x) for x in torch.randint(0, 3, (900,), generator=gen)]
    paged_check(g, paged_case(gen, nq, lens, 6, 16, torch.bfloat16))


@pytest.mark.parametrize("H,ps", [(200, 256), (7, 1000), (64, 40), (33, 64)])
def test_absorbed_head_counts_and_page_sizes(g, H, ps):
    gen = torch.Generator().manual_seed(H)
    paged_check(g, paged_case(gen, [1, 3, 2], [1500, 77, 640], H, ps, torch.float16))


def test_absorbed_malformed_metadata(g):
    """Lengths past the table's capacity are cut to it, negative ones count as none,
    offsets are clamped into the packed rows: wrong input, but no access out of range."""
    gen = torch.Generator().manual_seed(31)
    c = paged_case(gen, [1, 1, 1], [256, 128, 64], 16, 64, torch.bfloat16)
    c["cache"].nan_to_num_(0.25)
    c["table"].clamp_(min=0)
    c["lens"].copy_(i32([1 << 29, -5, 64]))
    c["L"] = [256, 0, 64]
    paged_check(g, c)
    for cu in ([0, -3, 1 << 30, 2], [2, 1, 0, 3], [5, 6, 7, 8]):
        g.attn_fwd_latent_paged(c["q"], c["cache"], i32(cu), c["lens"], c["table"], SCALE)
        g.attn_fwd_latent_varlen(c["q"][..., :192].contiguous(), c["q"][..., :128], c["q"][..., 128:256],
                                 c["q"][:, 0, 256:320], i32(cu), i32(cu[::-1]))
        g.attn_latent_gather(c["cache"], i32(cu), c["table"], 50)
    torch.cuda.synchronize()
    g.gqa_device_error()


def test_sliced_queries_and_two_streams_at_once(g):
    """Queries that are a slice are copied; calls side by side on two streams do not meet."""
    gen = torch.Generator().manual_seed(32)
    c = paged_case(gen, [1] * 40, [int(x) for x in torch.randint(1, 5000, (40,), generator=gen)], 16, 64, torch.bfloat16)
    e = varlen_case(gen, [300, 411], [300, 900], 8, torch.bfloat16)
    wide = torch.cat([c["q"], c["q"]], 2)[..., 100:676]
    args = (c["cache"], c["cu"], c["lens"], c["table"], SCALE)
    o, lse = g.attn_fwd_latent_paged(c["q"], *args)
    o2, lse2 = g.attn_fwd_latent_paged(wide, *args)
    assert torch.equal(*(g.attn_fwd_latent_paged(x, *args)[0] for x in (wide, wide.contiguous()))) and o2.shape == o.shape
    oe, le = g.attn_fwd_latent_varlen(e["q"], e["k"], e["v"], e["pe"], e["cq"], e["ck"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for n in range(20):
        with torch.cuda.stream(streams[n % 2]):
            got.append(g.attn_fwd_latent_paged(c["q"], *args) if n % 4 < 2 else
                       g.attn_fwd_latent_varlen(e["q"], e["k"], e["v"], e["pe"], e["cq"], e["ck"]))
    torch.cuda.synchronize()
    for n, (x, y) in enumerate(got):
        assert torch.equal(x, o if n % 4 < 2 else oe) and torch.equal(y, lse if n % 4 < 2 else le), n
    g.gqa_device_error()


def test_one_workspace_for_calls_in_turn(g):
    """A caller's workspace, larger than needed and full of NaN, used call after call."""
    gen = torch.Generator().manual_seed(33)
    cases = [paged_case(gen, [1] * 5, [3000, 10, 500, 1, 64], 16, 64, torch.bfloat16),
             paged_case(gen, [4, 1], [700, 2000], 64, 16, torch.bfloat16)]
    size = max(g.attn_latent_paged_workspace_size(len(c["nq"]), sum(c["nq"]), c["H"]) for c in cases)
    ws = torch.full((size // 4 + 64,), math.nan, device="cuda")
    for c in cases * 2:
        paged_check(g, c, workspace=ws)


# A weight 2^-26 of the strongest keeps its share: n of them before one strong key.  P is 2^-20 (six binades of
# room), which float16 has exactly.
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_many_weak_keys_behind_a_strong_one(g, form, dtype):
    dt, scale = DT[dtype], 26 * math.log(2.0) / 256
    if form == "absorbed":
        B, L, H, ps = 160, 16384, 16, 64                    # all requests read the same pages
        rows = torch.zeros(L, ROW, dtype=dt, device="cuda")
        rows[1:, :C] = 1.0
        rows[0, C] = 16.0
        q = torch.zeros(B, H, ROW, dtype=dt, device="cuda")
        q[..., C] = 16.0
        table = torch.arange(L // ps, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
        o, lse = g.attn_fwd_latent_paged(q, rows.view(L // ps, ps, ROW), i32(list(range(B + 1))), i32([L] * B), table,
                                         scale)
        q, k, v = q[0], rows, rows[:, :C]
    else:
        B, L, H = 1, 16384, 2
        kk = torch.zeros(L, H, NOPE, dtype=dt, device="cuda")
        vv = torch.ones(L, H, V, dtype=dt, device="cuda")
        pe = torch.zeros(L, R, dtype=dt, device="cuda")
        pe[0, 0], vv[0] = 16.0, 0.0
        q = torch.zeros(1, H, NOPE + R, dtype=dt, device="cuda")
        q[..., NOPE] = 16.0
        ws = torch.empty(g.attn_varlen_workspace_size(1, 1, H, H), dtype=torch.uint8, device="cuda")   # keys uncut
        o, lse = g.attn_fwd_latent_varlen(q, kk, vv, pe, i32([0, 1]), i32([0, L]), scale=scale, workspace=ws)
        q, k, v = q[0], torch.cat([kk[:, 0], pe], 1), vv[:, 0]
    torch.cuda.synchronize()
    ref = attend(q, k, v, torch.full((H,), L, device="cuda"), scale)
    for b in range(B):
        check(o[b], lse[b], ref, "request %d" % b)


# Rotated dims of -inf hide a key from queries that are positive there, whole tiles of keys too.
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_absorbed_keys_hidden_by_infinity(g, dtype):
    gen = torch.Generator().manual_seed(31)
    dt = DT[dtype]
    lens, hidden, ps, H = [200, 64, 130, 20000], [70, 63, 129, 19000], 8, 40
    c = paged_case(gen, [1] * 4, lens, H, ps, dt)
    c["q"][..., C] = c["q"][..., C].abs() + 0.5
    flat = c["cache"].flatten(0, 1)
    places = []
    for b, (n, x) in enumerate(zip(lens, hidden)):
        t = torch.arange(n, device="cuda")
        at = c["table"][b].long()[t // ps] * ps + t % ps
        flat[at[:x], C] = -math.inf
        places.append(at[x:])
    o, lse = g.attn_fwd_latent_paged(c["q"], c["cache"], c["cu"], c["lens"], c["table"], SCALE)
    torch.cuda.synchronize()
    for b, at in enumerate(places):
        rows = flat[at]
        check(o[b], lse[b], attend(c["q"][b], rows, rows[:, :C], torch.full((H,), lens[b], device="cuda"), SCALE),
              "request %d" % b)


def test_expanded_keys_hidden_by_infinity(g):
    gen = torch.Generator().manual_seed(32)
    n, L, H, x = 20, 300, 3, 200
    q = randn(gen, n, H, NOPE + R)
    q[..., NOPE] = q[..., NOPE].abs() + 0.5
    k, v, pe = randn(gen, L, H, NOPE), randn(gen, L, H, V), randn(gen, L, R)
    pe[:x, 0] = -math.inf
    o, lse = g.attn_fwd_latent_varlen(q, k, v, pe, i32([0, n]), i32([0, L]))
    torch.cuda.synchronize()
    at = torch.arange(n, device="cuda") + (L - n) - x
    for h in range(H):
        check(o[:, h], lse[:, h], attend(q[:, h], torch.cat([k[x:, h], pe[x:]], 1), v[x:, h], at, SCALE), "head %d" % h)


def test_empty_calls(g):
    """No query, no key, no token: shapes come back, nothing runs."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")
    o, lse = g.attn_fwd_latent_paged(z(0, 16, ROW), z(4, 16, ROW), i32([0, 0]), i32([20]), i32([[0, 1]]), SCALE)
    assert o.shape == (0, 16, C) and lse.shape == (0, 16)
    o, lse = g.attn_fwd_latent_varlen(z(0, 4, 192), z(0, 4, 128), z(0, 4, 128), z(0, 64), i32([0, 0]), i32([0, 0]))
    assert o.shape == (0, 4, V) and lse.shape == (0, 4)
    o, lse = g.attn_fwd_latent_varlen(z(3, 4, 192), z(0, 4, 128), z(0, 4, 128), z(0, 64), i32([0, 3]), i32([0, 0]))
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    assert g.attn_latent_gather(z(4, 16, ROW), i32([0, 0]), i32([[0]]), 0).shape == (0, ROW)
    out = g.attn_latent_norm_rope_paged(z(0, 4, 64), z(0, ROW), g.rope_table(8, 64), i32([]), i32([]), z(4, 16, ROW))
    assert out.shape == (0, 4, 64)


def test_refusals(g):
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")
    cs = g.rope_table(8, 64)
    paged = dict(q=z(1, 4, ROW), kv_cache=z(4, 16, ROW), cu_seqlens_q=i32([0, 1]), cache_seqlens=i32([20]),
                 block_table=i32([[0, 1]]), scale=SCALE)
    for bad in (dict(q=z(1, 4, 512)), dict(q=z(1, 4, ROW, d=torch.float32)), dict(kv_cache=z(4, 16, ROW, d=torch.float16)),
                dict(kv_cache=z(4, 16, 640)), dict(kv_cache=z(4, 32, ROW)[:, ::2]), dict(cu_seqlens_q=i32([0])),
                dict(cache_seqlens=i32([20]).long()), dict(block_table=i32([0, 1])), dict(block_table=i32([[0, 1], [0, 1]])),
                dict(scale=math.inf), dict(out=z(1, 4, ROW)), dict(lse=z(1, 4)), dict(workspace=z(16, d=torch.uint8))):
        with pytest.raises(ValueError):
            g.attn_fwd_latent_paged(**{**paged, **bad})
    var = dict(q=z(2, 4, 192), k=z(3, 4, 128), v=z(3, 4, 128), k_pe=z(3, 64), cu_seqlens_q=i32([0, 2]),
               cu_seqlens_kv=i32([0, 3]))
    for bad in (dict(q=z(2, 4, 128)), dict(k=z(3, 2, 128)), dict(v=z(4, 4, 128)), dict(k_pe=z(3, 32)), dict(k_pe=z(3, 4, 64)),
                dict(v=z(3, 4, 128, d=torch.float16)), dict(cu_seqlens_kv=i32([0, 1, 3])), dict(cu_seqlens_q=i32([0])),
                dict(out=z(2, 4, 192)), dict(workspace=z(8, d=torch.uint8))):
        with pytest.raises(ValueError):
            g.attn_fwd_latent_varlen(**{**var, **bad})
    app = dict(q_pe=z(2, 4, 64), kv=z(2, ROW), cos_sin=cs, positions=i32([0, 1]), slots=i32([0, 1]), kv_cache=z(4, 16, ROW))
    for bad in (dict(q_pe=z(2, 4, 32)), dict(kv=z(3, ROW)), dict(kv=z(2, 512)), dict(cos_sin=g.rope_table(8, 32)),
                dict(positions=i32([0])), dict(slots=i32([0, 1]).long()), dict(kv_cache=z(4, 16, ROW, d=torch.float16)),
                dict(kv_weight=z(64)), dict(kv_weight=z(512, d=torch.float16)), dict(eps=-1.0),
                dict(out=z(2, 4, 65)[..., 1:]), dict(out=z(2, 4, 64, d=torch.float16)), dict(kv_out=z(2, 640)[:, :ROW])):
        with pytest.raises(ValueError):
            g.attn_latent_norm_rope_paged(**{**app, **bad})
    for bad in (dict(kv_cache=z(4, 16, 512)), dict(cu_seqlens_kv=i32([0])), dict(total_kv=-1), dict(total_kv=1 << 30),
                dict(out=z(19, ROW))):
        with pytest.raises(ValueError):
            g.attn_latent_gather(**{**dict(kv_cache=z(4, 16, ROW), cu_seqlens_kv=i32([0, 20]), block_table=i32([[0, 1]]),
                                          total_kv=20), **bad})
