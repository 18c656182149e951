"""Packed queries over a float8_e4m3fn paged cache on the GPU (chunks and decode
steps in one call) against the FP64 oracle, request by request; unread slots
hold the NaN code.

Every output is held to what its roundings allow: half a step of the output
type (eps / 2 of the value), and half a step of a float16 weight, 2^-11 of each
p, so at most 2^-11 max|v| of the weighted mean; the FP32 scores and
exponentials add less than 2^-13 max|v| (128 to 256 products of 2^-24 each on
scores of a few units, and 2^-22 of an exponential).  The absolute 2e-2 of
parity.compare does not fit here: a row that sees one key returns its value, up
to 5.5 x 2 with scales up to 2, and half a bfloat16 step between 8 and 16 is
2^-5 = 3.1e-2.  The LSE limit (1e-3) and the empty rows are those of compare.
"""
import math

import pytest
import torch

import oracle
from gqa_softmax_attention_gb300 import workloads as W

from parity import TOL_LSE

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gqa_softmax_attention_gb300 import build
    build.build()
    import gqa_softmax_attention_gb300 as m
    yield m
    m.gqa_device_error()          # no kernel wait may have timed out


def inputs(ql, L, Hq, Hkv, D, ps, seed=0, dtype=torch.bfloat16, scale_range=(0.25, 1.0)):
    """varlen_paged_inputs with e4m3 caches and scales; slots no request owns hold NaN codes."""
    p = W.varlen_paged_inputs(ql, L, Hq, Hkv, D, ps, seed=seed)
    p["q"] = p["q"].to(dtype)
    gen = torch.Generator().manual_seed(seed + 77)
    lo, hi = scale_range
    p["k_scale"], p["v_scale"] = (lo + (hi - lo) * torch.rand(len(ql), Hkv, generator=gen) for _ in range(2))
    owned = torch.zeros(p["num_pages"] * ps, dtype=torch.bool)
    for b, n in enumerate(L):
        t = torch.arange(n)
        owned[p["block_table"][b].long()[t // ps] * ps + t % ps] = True
    for n in ("k_cache", "v_cache"):
        c = p[n].float().to(torch.float8_e4m3fn).view(torch.uint8)
        c.view(-1, Hkv, D)[~owned] = 0x7F
        p[n] = c.view(torch.float8_e4m3fn)
    return p


NAMES = ("q", "k_cache", "v_cache", "k_scale", "v_scale", "cu_seqlens_q", "cache_seqlens", "block_table")


def run(g, p, **kw):
    o, lse = g.attn_fwd_paged_fp8kv(*[p[n].cuda() for n in NAMES], **kw)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu()


def check(p, o, lse, label="", requests=None, **kw):
    cu, D = p["cu_seqlens_q"].tolist(), p["q"].shape[2]
    for b in range(len(cu) - 1) if requests is None else requests:
        a, z = cu[b], cu[b + 1]
        if a == z:
            continue
        one = slice(b, b + 1)
        ro, rl = oracle.attn_paged_fp8kv(p["q"][None, a:z], p["k_cache"], p["v_cache"], p["k_scale"][one],
                                         p["v_scale"][one], p["cache_seqlens"][one], p["block_table"][one], **kw)
        ro, rl, go, gl = ro[0], rl[0], o[a:z], lse[a:z]
        top = torch.isposinf(rl)                       # heads with a +inf sink
        assert bool(torch.isposinf(gl[top]).all()) and bool((go.float()[top] == 0).all()), label
        ro, rl, go, gl = ro[~top], rl[~top], go[~top], gl[~top]
        empty = torch.isneginf(rl)
        assert torch.equal(torch.isneginf(gl), empty) and bool((go.float()[empty] == 0).all()), label
        assert bool(((gl.double() - rl)[~empty].abs() <= TOL_LSE).all()), "%s request %d: LSE" % (label, b)
        vmax = 5.5 * float(p["v_scale"][b].max())          # N(0, 1) draws of this size stay below 5.5
        tol = torch.finfo(o.dtype).eps / 2 * ro.abs() + (2.0 ** -11 + 2.0 ** -13) * vmax
        off = (go.double() - ro).abs()
        assert bool((off <= tol).all()), "%s request %d: %.3g of its tolerance" % (label, b, float((off / tol).max()))


CASES = [
    # q lengths, cache lengths (query tokens included), Hq, Hkv, D, page_size
    ([2], [2], 4, 2, 128, 16), ([1], [1], 4, 2, 128, 16), ([7], [300], 4, 4, 256, 8),
    ([1, 300, 0, 4, 1, 129], [1000, 800, 50, 333, 1, 129], 8, 2, 128, 16),
    ([1, 1, 1, 1, 2, 200], [17, 4000, 129, 640, 2, 200], 32, 8, 128, 64),
    ([4, 4, 1, 64], [3000, 17, 700, 64], 24, 2, 256, 16),
    ([3, 100, 1], [77, 100, 1000], 4, 2, 128, 8),
    ([1, 40, 2], [500, 300, 2], 8, 2, 128, 24),
    ([5, 1, 130], [900, 600, 130], 16, 2, 256, 256),
    ([1, 1, 20, 1], [0, 700, 40, 1], 8, 2, 128, 16),                       # a decode step with an empty cache
    ([1, 37, 3], [300, 200, 3], 8, 2, 128, 1),
    ([2, 1, 150], [41, 500, 400], 8, 2, 128, 3),
    ([1, 129, 4], [777, 129, 260], 24, 2, 256, 5),
    ([200, 1, 1], [1000, 13, 1200], 32, 8, 128, 12),
    ([20, 1, 6], [20, 300, 1111], 33, 1, 128, 16),                         # g = 33: decode steps stay packed
    ([9, 1], [2000, 130], 128, 1, 128, 64), ([40, 3], [500, 260], 12, 12, 128, 64),   # g = 128, g = 1
    ([128, 127, 129, 256], [128, 255, 257, 512], 8, 8, 128, 128),          # whole tiles and their neighbours
]


@pytest.mark.parametrize("split_decode", [True, False], ids=["split_decode", "packed_only"])
@pytest.mark.parametrize("case", CASES, ids=[str(c[:2]) + "/%d/%d/D%d/ps%d" % c[2:] for c in CASES])
def test_matches_oracle(g, case, split_decode):
    p = inputs(*case, seed=sum(case[1]) % 97)
    check(p, *run(g, p, split_decode=split_decode))


SPLIT = [
    # few rows over long caches: the keys are cut into parts for the idle SMs
    ([3], [5000], 8, 2, 128, 16), ([2, 5], [9000, 300], 4, 1, 128, 64), ([7], [6001], 24, 2, 256, 16),
    ([4, 1, 2, 1], [4097, 3000, 513, 7], 8, 2, 128, 24), ([33], [1025], 16, 1, 256, 5), ([5], [2], 8, 2, 128, 16),
    ([9, 2], [8200, 8191], 32, 8, 128, 128), ([2], [513], 4, 4, 256, 8),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", SPLIT, ids=[str(c[:2]) + "/%d/%d/D%d/ps%d" % c[2:] for c in SPLIT])
def test_keys_in_parts(g, case, dtype):
    p = inputs(*case, seed=sum(case[1]) % 89, dtype=dtype)
    Hq, L = case[2], max(case[1])
    sinks = torch.randn(Hq, generator=torch.Generator().manual_seed(2))
    sinks[0], sinks[-1] = INF, -INF
    for kw in (dict(), dict(sinks=sinks), dict(window_left=L // 3), dict(window_left=200, softcap=9.0, sinks=sinks),
               dict(causal=False, window_left=L // 2, window_right=3)):
        check(p, *run(g, p, **kw), label=str(kw), **kw)


def test_keys_in_parts_of_a_replayed_call(g):
    """The number of parts follows the lengths on the device; each call fills the same workspace."""
    p = inputs([6, 3], [7000, 900], 8, 2, 128, 64, seed=2)
    for n in ("k_cache", "v_cache"):
        c = p[n].view(torch.uint8)
        p[n] = torch.where(c == 0x7F, torch.zeros_like(c), c).view(torch.float8_e4m3fn)
    dev = {n: p[n].cuda() for n in NAMES}
    size = g.attn_paged_fp8kv_workspace_size(2, 9, 8, 2, 128, 64, p["block_table"].shape[1])
    assert size > g.attn_paged_workspace_size(2, 9, 8, 2, 128, 64, p["block_table"].shape[1])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(dev["q"]), torch.empty((9, 8), device="cuda")
    call = lambda: g.attn_fwd_paged_fp8kv(*[dev[n] for n in NAMES], out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, cu in (([7000, 900], [0, 6, 9]), ([130, 40], [0, 6, 9]), ([3000, 899], [0, 8, 9]), ([2, 0], [0, 6, 9])):
        p["cache_seqlens"], p["cu_seqlens_q"] = (torch.tensor(x, dtype=torch.int32) for x in (lens, cu))
        dev["cache_seqlens"].copy_(p["cache_seqlens"])
        dev["cu_seqlens_q"].copy_(p["cu_seqlens_q"])
        graph.replay()
        torch.cuda.synchronize()
        check(p, out.cpu(), lse.cpu(), "replay %s" % lens)


@pytest.mark.parametrize("split_decode", [True, False], ids=["split_decode", "packed_only"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("geometry", [(24, 2, 256, 32), (32, 8, 128, 64)], ids=str)
def test_options(g, geometry, dtype, split_decode):
    Hq = geometry[0]
    p = inputs([1, 200, 4, 1, 300], [2000, 450, 40, 90, 1500], *geometry, seed=5, dtype=dtype, scale_range=(0.05, 2.0))
    sinks = torch.randn(Hq, generator=torch.Generator().manual_seed(9)) * 2
    sinks[0], sinks[-1] = -INF, INF
    for kw in (dict(window_left=300, softcap=20.0, sinks=sinks), dict(window_left=0), dict(softcap=5.0),
               dict(window_left=129, window_right=0, scale=0.03), dict(scale=-0.1), dict(scale=0.0),
               dict(scale=-0.1, softcap=4.0), dict(scale=0.0, softcap=4.0), dict(scale=2.0, softcap=1.5)):
        check(p, *run(g, p, split_decode=split_decode, **kw), label=str(kw), **kw)


def test_noncausal_and_two_sided_window(g):
    p = inputs([60, 200, 1, 5], [300, 200, 77, 90], 6, 3, 128, 16, seed=12)
    check(p, *run(g, p, causal=False), causal=False)
    kw = dict(causal=False, window_left=40, window_right=17)
    check(p, *run(g, p, **kw), **kw)


def test_rows_without_a_key(g):
    """More queries than cached tokens (leading rows see nothing) and no cache at all: zeros and -inf."""
    p = inputs([5, 130, 1, 40], [2, 100, 0, 0], 8, 2, 128, 16, seed=3)
    p["block_table"] = p["block_table"].contiguous()
    o, lse = run(g, p)
    check(p, o, lse)
    assert bool(torch.isneginf(lse[:3]).all()) and bool((o[:3].float() == 0).all())
    assert bool(torch.isneginf(lse[-41:]).all()) and bool((o[-41:].float() == 0).all())


def test_every_code(g):
    """Every finite e4m3 code among keys and values, subnormals included: one
    visible key gives its value exactly (scales are powers of two)."""
    D, Hkv, T = 128, 2, 4
    codes = torch.arange(256, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    cache = codes.repeat(4)[:T * Hkv * D].view(1, T, Hkv, D)
    q = torch.zeros(2 * T, 2 * Hkv, D, dtype=torch.float16)
    cu = torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32)
    lens = torch.ones(T, dtype=torch.int32)
    pool = cache.view(T, 1, Hkv, D).contiguous()
    table = torch.arange(T, dtype=torch.int32)[:, None].contiguous()
    vs = torch.full((T, Hkv), 0.5)
    o, lse = g.attn_fwd_paged_fp8kv(q.cuda(), pool.cuda(), pool.cuda(), None, vs.cuda(), cu.cuda(), lens.cuda(),
                                    table.cuda())
    want = (oracle.e4m3_decode(pool)[:, 0] * 0.5).repeat_interleave(2, dim=1)
    assert torch.equal(o[1::2].double().cpu(), want)               # row 1 of each request sees its one key
    assert bool((lse[1::2] == 0).all()) and bool(torch.isneginf(lse[0::2]).all())


def test_unit_scales_equal_the_16bit_call(g):
    """Codes are float16 values: with unit scales the 16-bit call on the widened cache has the same inputs."""
    p = inputs([100, 1, 30], [900, 400, 30], 8, 2, 128, 16, seed=6, dtype=torch.float16)
    kc, vc = (p[n].float().nan_to_num(0).half().cuda() for n in ("k_cache", "v_cache"))
    o, lse = g.attn_fwd_paged_fp8kv(p["q"].cuda(), p["k_cache"].cuda(), p["v_cache"].view(torch.uint8).cuda(), None,
                                    None, *[p[n].cuda() for n in NAMES[5:]])
    o2, lse2 = g.attn_fwd_paged(p["q"].cuda(), kc, vc, *[p[n].cuda() for n in NAMES[5:]])
    tol = (2.0 ** -11 * o2.float().abs() + 2 * (2.0 ** -11 + 2.0 ** -13) * 5.5)
    assert bool(((o.float() - o2.float()).abs() <= tol).all())
    assert bool(((lse - lse2).abs() <= 1e-4).all())


def test_bad_page_ids_read_as_zeros_and_stay_in_the_pool(g):
    p = inputs([150, 20], [400, 100], 8, 2, 128, 16, seed=8)
    p["block_table"][0, 3] = 2**31 - 1
    p["block_table"][0, 5] = -9
    p["block_table"][1, 0] = p["num_pages"]
    o, lse = run(g, p)
    assert bool(o.isfinite().all()) and bool(lse.isfinite().all())
    # the same call with those pages zeroed
    z = dict(p, block_table=p["block_table"].clone())
    spare = sorted(set(range(p["num_pages"])) - set(p["block_table"].flatten().tolist()))[:1]
    for b, j in ((0, 3), (0, 5), (1, 0)):
        z["block_table"][b, j] = spare[0]
    for n in ("k_cache", "v_cache"):
        z[n] = p[n].view(torch.uint8).clone()
        z[n][spare[0]] = 0
        z[n] = z[n].view(torch.float8_e4m3fn)
    o2, lse2 = run(g, z)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [128, 256])
def test_pages_left_of_every_window_may_hold_anything(g, D):
    """Slots that no query's window reaches any more: freed pages (NaN codes here, or no page at all)."""
    p = inputs([40, 3, 200], [1000, 700, 900], 8, 2, D, 16, seed=14)
    wl = 100
    want = run(g, p, window_left=wl)
    check(p, *want, window_left=wl)
    z = dict(p, block_table=p["block_table"].clone())
    kc, vc = (p[n].view(torch.uint8).clone() for n in ("k_cache", "v_cache"))
    for b, (n, L) in enumerate(zip([40, 3, 200], [1000, 700, 900])):
        dead = L - n - wl                                  # keys below it are left of the first query's window
        for t in range(dead):
            kc[p["block_table"][b, t // 16], t % 16] = 0x7F
            vc[p["block_table"][b, t // 16], t % 16] = 0x7F
        z["block_table"][b, :dead // 16] = -1
    z["k_cache"], z["v_cache"] = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    for case in (z, dict(z, block_table=p["block_table"])):
        got = run(g, case, window_left=wl, split_decode=False)
        check(p, *got, window_left=wl)


@pytest.mark.parametrize("D,Hkv,ps", [(128, 8, 64), (256, 2, 24)])
def test_pages_past_4_gib_of_a_cache(g, D, Hkv, ps):
    """Chunks, drafted tokens and decode steps whose pages lie behind byte 2^32."""
    p = inputs([1, 200, 4], [500, 700, 3000], 4 * Hkv, Hkv, D, ps, seed=31)
    first = (1 << 32) // (ps * Hkv * D) + 1                    # first page wholly past it
    far = dict(p, block_table=torch.where(p["block_table"] >= 0, p["block_table"] + first, p["block_table"]))
    dev = {n: far[n].cuda() for n in NAMES if n not in ("k_cache", "v_cache")}
    for n in ("k_cache", "v_cache"):
        pool = torch.full((first + p["num_pages"], ps, Hkv, D), 0x7F, dtype=torch.uint8, device="cuda")
        pool[first:] = p[n].view(torch.uint8).cuda()
        dev[n] = pool.view(torch.float8_e4m3fn)
    for split in (True, False):
        o, lse = g.attn_fwd_paged_fp8kv(*[dev[n] for n in NAMES], split_decode=split)
        torch.cuda.synchronize()
        check(p, o.cpu(), lse.cpu(), "split_decode %s" % split)


def test_rows_outside_the_requests_stay(g):
    p = inputs([3, 140, 1], [50, 300, 70], 8, 2, 128, 16, seed=4)
    q = torch.cat([p["q"], torch.full((9, 8, 128), float("nan"), dtype=p["q"].dtype)])
    out = torch.full_like(q, 3.0).cuda()
    lse = torch.full((q.shape[0], 8), 5.0, device="cuda")
    g.attn_fwd_paged_fp8kv(q.cuda(), *[p[n].cuda() for n in NAMES[1:]], out=out, lse=lse)
    check(p, out[:144].cpu(), lse[:144].cpu())
    assert bool((out[144:] == 3).all()) and bool((lse[144:] == 5).all())


def test_many_requests(g):
    gen = torch.Generator().manual_seed(21)
    B = 1200
    ql = torch.randint(0, 3, (B,), generator=gen).tolist()
    L = [max(n, int(x)) for n, x in zip(ql, torch.randint(1, 200, (B,), generator=gen))]
    p = inputs(ql, L, 4, 2, 128, 8, seed=3)
    check(p, *run(g, p), requests=range(0, B, 37))


def test_long_cache_and_mixed_batch(g):
    """A serving-sized mix: 30 decode steps and two chunks over long caches, sampled."""
    gen = torch.Generator().manual_seed(4)
    L = [int(x) for x in torch.randint(1024, 9000, (32,), generator=gen)]
    ql = [1] * 32
    ql[5], ql[20] = 700, 1024
    p = inputs(ql, L, 32, 8, 128, 64, seed=11)
    o, lse = run(g, p)
    assert bool(o.isfinite().all()) and bool(lse.isfinite().all())
    check(p, o, lse, requests=(0, 17, 31))
    for b in (5, 20):
        a, n = int(p["cu_seqlens_q"][b]), ql[b]
        for i in (0, 1, 31, 32, 511, n - 1):
            r = dict(p, q=p["q"][a + i:a + i + 1], cu_seqlens_q=torch.tensor([0, 1], dtype=torch.int32),
                     cache_seqlens=p["cache_seqlens"][b:b + 1] - n + i + 1, block_table=p["block_table"][b:b + 1],
                     k_scale=p["k_scale"][b:b + 1], v_scale=p["v_scale"][b:b + 1])
            check(r, o[a + i:a + i + 1], lse[a + i:a + i + 1], "request %d row %d" % (b, i))


def test_graph_replay_with_new_lengths_and_scales(g):
    p = inputs([1, 300, 1, 4], [1500, 700, 50, 1000], 32, 8, 128, 64, seed=9)
    for n, c in zip(("k_cache", "v_cache"), (p["k_cache"], p["v_cache"])):      # any slot may be read below
        p[n] = torch.where(c.view(torch.uint8) == 0x7F, 0, c.view(torch.uint8)).to(torch.uint8).view(torch.float8_e4m3fn)
    dev = {n: p[n].cuda() for n in NAMES}
    out = torch.empty_like(dev["q"])
    lse = torch.empty((p["q"].shape[0], 32), device="cuda")
    call = lambda: g.attn_fwd_paged_fp8kv(*[dev[n] for n in NAMES], out=out, lse=lse)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, cu in (([900, 301, 20, 700], [0, 1, 301, 302, 306]), ([1500, 305, 30, 10], [0, 0, 300, 302, 306])):
        p["cache_seqlens"], p["cu_seqlens_q"] = (torch.tensor(x, dtype=torch.int32) for x in (lens, cu))
        p["k_scale"], p["v_scale"] = p["v_scale"].flip(0), p["k_scale"].flip(0)
        for n in ("cache_seqlens", "cu_seqlens_q", "k_scale", "v_scale"):
            dev[n].copy_(p[n])
        graph.replay()
        torch.cuda.synchronize()
        check(p, out.cpu(), lse.cpu(), "replay %s" % lens)


def test_other_stream_and_repeat(g):
    p = inputs([1, 600, 1, 300], [3000, 1800, 40, 700], 32, 8, 128, 64, seed=6)
    dev = [p[n].cuda() for n in NAMES]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    copies = []
    with torch.cuda.stream(st):
        for _ in range(3):
            o, lse = g.attn_fwd_paged_fp8kv(*dev)
            copies.append((o.clone(), lse.clone()))          # queued behind the call
    torch.cuda.synchronize()
    check(p, copies[0][0].cpu(), copies[0][1].cpu())
    for o, lse in copies[1:]:
        assert torch.equal(o, copies[0][0]) and torch.equal(lse, copies[0][1])


def test_two_calls_at_once(g):
    """Two streams, neither waiting for the other, each with its own tensors."""
    ps = [inputs([1, 400, 1, 5], [2500, 900, 40, 3000], 32, 8, 128, 64, seed=21),
          inputs([3, 1, 250], [2000, 700, 600], 24, 2, 256, 16, seed=22)]
    streams = [torch.cuda.Stream() for _ in ps]
    devs = [[p[n].cuda() for n in NAMES] for p in ps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(g.attn_fwd_paged_fp8kv(*devs[i]))
    torch.cuda.synchronize()
    for p, runs in zip(ps, got):
        check(p, runs[0][0].cpu(), runs[0][1].cpu())
        for o, lse in runs[1:]:
            assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])


def test_two_graphs_share_a_workspace(g):
    """Captured calls of other sizes (one with its keys in parts) replayed in
    turn over one workspace: nothing in it is taken over from a call."""
    ps = [inputs([4, 2], [3000, 2500], 32, 8, 128, 64, seed=23),
          inputs([1, 300, 1], [900, 800, 1200], 32, 8, 128, 16, seed=24)]
    size = max(g.attn_paged_fp8kv_workspace_size(len(p["cache_seqlens"]), p["q"].shape[0], 32, 8, 128, pg,
                                                 p["block_table"].shape[1]) for p, pg in zip(ps, (64, 16)))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for p in ps:
        dev = [p[n].cuda() for n in NAMES]
        out, lse = torch.empty_like(dev[0]), torch.empty(p["q"].shape[0], 32, device="cuda")
        call = lambda: g.attn_fwd_paged_fp8kv(*dev, out=out, lse=lse, workspace=ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, dev))
        outs.append((out, lse))
    for i in (0, 1, 0, 0, 1, 1, 0):
        for t in outs[i]:
            t.fill_(float("nan"))
        graphs[i][0].replay()
        torch.cuda.synchronize()
        check(ps[i], outs[i][0].cpu(), outs[i][1].cpu(), "graph %d" % i)


def test_refusals(g):
    p = inputs([2, 3], [20, 30], 8, 2, 128, 16)
    d = {n: p[n].cuda() for n in NAMES}
    for bad in (dict(q=d["q"].float()), dict(q=d["q"][..., :64]), dict(k_cache=d["k_cache"].half()),
                dict(k_cache=d["k_cache"][:, ::2]), dict(v_cache=d["v_cache"][1:]), dict(k_scale=d["k_scale"][:1]),
                dict(v_scale=d["v_scale"].double()), dict(cu_seqlens_q=d["cu_seqlens_q"].long()),
                dict(cu_seqlens_q=d["cu_seqlens_q"][:2]), dict(cache_seqlens=d["cache_seqlens"].cpu()),
                dict(block_table=d["block_table"][:1]), dict(block_table=d["block_table"].t().contiguous().t()),
                dict(q=d["q"][:, :7]), dict(window_left=-2), dict(softcap=-1.0), dict(softcap=float("nan")),
                dict(scale=float("inf")), dict(sinks=torch.zeros(3)), dict(out=torch.empty(5, 8, 128, device="cuda")),
                dict(lse=torch.empty(5, 9, device="cuda")),
                dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            g.attn_fwd_paged_fp8kv(**{**d, **bad})
    d64 = {n: p[n].cuda() for n in NAMES}
    d64["q"], d64["k_cache"], d64["v_cache"] = (d64[n][..., :64].contiguous() for n in ("q", "k_cache", "v_cache"))
    with pytest.raises(ValueError):
        g.attn_fwd_paged_fp8kv(**d64)                                     # D = 64


def one_part(g, p):
    """A workspace without room for key parts: the same call with the keys of every block in one part."""
    (T, Hq, D), (_, ps, Hkv, _) = p["q"].shape, p["k_cache"].shape
    size = g.attn_paged_workspace_size(len(p["cache_seqlens"]), T, Hq, Hkv, D, ps, p["block_table"].shape[1])
    return torch.empty(size, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("value", [float("nan"), INF, -INF, 1e5], ids=str)
@pytest.mark.parametrize("geometry", [(8, 2, 128, 64), (24, 2, 256, 16)], ids=str)
def test_queries_that_are_no_numbers_show(g, geometry, value):
    """A NaN or infinite value in one head of one query (in bfloat16 also one past
    float16's range, which becomes infinite): that row is NaN, O and LSE, with its keys
    in one part and in several, with a sink and without; every other row is as it was.
    Infinite scores of both signs among 5000 keys make every such row inf - inf."""
    p = inputs([4], [5000], *geometry, seed=41)
    Hq, D = geometry[0], geometry[2]
    bad = dict(p, q=p["q"].clone())
    bad["q"][1, 2, 5] = value
    bad["q"][3, Hq - 1, D - 1] = value
    hit = torch.zeros(4, Hq, dtype=torch.bool)
    hit[1, 2] = hit[3, Hq - 1] = True
    sinks = torch.randn(Hq, generator=torch.Generator().manual_seed(3))
    sinks[-1] = INF
    for kw in (dict(), dict(sinks=sinks), dict(window_left=3000)):
        for ws in (None, one_part(g, p)):
            o, lse = run(g, bad, workspace=ws, **kw)
            assert bool(o[hit].isnan().all()) and bool(lse[hit].isnan().all()), str(kw)
            clean, cl = run(g, p, workspace=ws, **kw)
            o[hit], lse[hit] = clean[hit], cl[hit]
            check(p, o, lse, label=str(kw), **kw)


def test_a_query_without_a_key_is_empty_whatever_it_holds(g):
    """NaN in a row whose mask leaves nothing: zeros and -inf, as for any row without a key."""
    p = inputs([600, 3], [40, 5000], 8, 2, 128, 64, seed=43)
    p["q"][:560] = float("nan")
    o, lse = run(g, p)
    assert bool(torch.isneginf(lse[:560]).all()) and bool((o[:560].float() == 0).all())
    check(p, o, lse)


@pytest.mark.parametrize("value", [float("nan"), INF, -INF, 1e5], ids=str)
@pytest.mark.parametrize("geometry", [(32, 8, 128, 64), (24, 2, 256, 16), (12, 1, 128, 24), (36, 2, 128, 64),
                                      (64, 2, 256, 64), (64, 2, 128, 5)], ids=str)
def test_single_queries_that_are_no_numbers_show(g, geometry, value):
    """The same in single-token requests, on the split decode kernels (rows of up to 8, 16
    and 32 per KV head, the tensor-core form, pages that do not fit its boxes)."""
    p = inputs([1, 1, 1], [3000, 200, 1], *geometry, seed=47)
    Hq, D = geometry[0], geometry[2]
    bad = dict(p, q=p["q"].clone())
    bad["q"][0, Hq - 1, 5] = value
    bad["q"][1, 0, D - 1] = value
    hit = torch.zeros(3, Hq, dtype=torch.bool)
    hit[0, Hq - 1] = hit[1, 0] = True
    sinks = torch.randn(Hq, generator=torch.Generator().manual_seed(3))
    sinks[0] = INF
    for kw in (dict(), dict(sinks=sinks), dict(window_left=150)):
        o, lse = run(g, bad, **kw)
        assert bool(o[hit].isnan().all()) and bool(lse[hit].isnan().all()), str(kw)
        clean, cl = run(g, p, **kw)
        o[hit], lse[hit] = clean[hit], cl[hit]
        check(p, o, lse, label=str(kw), **kw)


@pytest.mark.parametrize("parts", [False, True], ids=["one_part", "in_parts"])
@pytest.mark.parametrize("cap", [None, 20.0], ids=["plain", "softcap"])
@pytest.mark.parametrize("geometry", [(4, 1, 128, 64), (12, 1, 256, 16)], ids=str)
@pytest.mark.parametrize("bits", [12.0, 20.6, 25.05, 27.5])
def test_one_strong_key_and_a_long_flat_tail(g, bits, geometry, cap, parts):
    """Key 0 leads every other of 131072 keys by `bits` binades and has the value
    zero, so the result is what the tail's small weights carry:
    n w / (1 + n w), w = 2^-bits, n keys behind the first.

    Tolerance: half a step of the output; a weight above float16's normal range keeps
    2^-11 of itself, one below it is off by half a float16 subnormal step, 2^-25, in
    units of 2^-6 of the leading weight: n 2^-31 in all; scores of at most 20 log2
    units carry 2^-13 of each weight (2^-23 relative of 38, and the softcap's 1e-7 of
    20 / ln 2 log2 units)."""
    Hq, Hkv, D, ps = geometry
    L, nq = 131072, 3
    lead = bits * math.log(2.0)                              # the leading score in nats
    z = lead if cap is None else cap * math.atanh(lead / cap)
    kc = torch.zeros(L // ps, ps, Hkv, D, dtype=torch.uint8)
    kc[0, 0] = 0x38                                          # 1.0
    vc = torch.full_like(kc, 0x38)
    vc[0, 0] = 0
    p = dict(q=torch.ones(nq, Hq, D, dtype=torch.float16), k_cache=kc.view(torch.float8_e4m3fn),
             v_cache=vc.view(torch.float8_e4m3fn), k_scale=torch.ones(1, Hkv), v_scale=torch.ones(1, Hkv),
             cu_seqlens_q=torch.tensor([0, nq], dtype=torch.int32), cache_seqlens=torch.tensor([L], dtype=torch.int32),
             block_table=torch.arange(L // ps, dtype=torch.int32)[None].contiguous())
    o, lse = run(g, p, scale=z / D, softcap=cap, workspace=None if parts else one_part(g, p))
    n = (L - nq + torch.arange(nq, dtype=torch.float64))[:, None, None]
    nw = n * 2.0 ** -bits
    want = (nw / (1 + nw)).expand(nq, Hq, D)
    tol = torch.finfo(o.dtype).eps / 2 * want + (2.0 ** -11 + 2.0 ** -13) * want + n * 2.0 ** -31
    off = (o.double() - want).abs()
    assert bool((off <= tol).all()), "%.3g of its tolerance" % float((off / tol).max())
    ref = lead + torch.log1p(nw[..., 0])
    assert bool(((lse.double() - ref).abs() <= 2.0 ** -13).all())


def test_outputs_over_inputs_are_refused_and_next_to_them_are_not(g):
    p = inputs([3, 40], [700, 90], 8, 2, 128, 16, seed=51)
    d = {n: p[n].cuda() for n in NAMES}
    T, n = 43, 43 * 8 * 128
    size = g.attn_paged_fp8kv_workspace_size(2, T, 8, 2, 128, 16, p["block_table"].shape[1])
    # q, o, lse and the workspace one behind the other in one buffer
    buf = torch.zeros(4 * n + T * 8 * 4 + 256 + size, dtype=torch.uint8, device="cuda")
    q, o = (buf[i * 2 * n:(i + 1) * 2 * n].view(torch.bfloat16).view(T, 8, 128) for i in range(2))
    lse = buf[4 * n:4 * n + T * 8 * 4].view(torch.float32).view(T, 8)
    at = (4 * n + T * 8 * 4 + 255) // 256 * 256
    ws = buf[at:at + size]
    q.copy_(d["q"])
    d["q"] = q
    g.attn_fwd_paged_fp8kv(**d, out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    check(p, o.cpu(), lse.cpu())
    kb = d["k_cache"].view(torch.uint8).flatten()
    for bad in (dict(out=q), dict(lse=buf[:T * 8 * 4].view(torch.float32).view(T, 8)),
                dict(out=kb[:2 * n].view(torch.bfloat16).view(T, 8, 128)), dict(workspace=buf),
                dict(workspace=kb), dict(out=o, lse=o.view(torch.float32).flatten()[:T * 8].view(T, 8))):
        with pytest.raises(ValueError):
            g.attn_fwd_paged_fp8kv(**d, **bad)


def test_a_workspace_that_is_no_tensor_is_refused(g):
    p = inputs([2, 3], [20, 30], 8, 2, 128, 16)
    d = {n: p[n].cuda() for n in NAMES}
    for bad in (1 << 20, b"0" * 4096, [0] * 4096, torch.empty(1 << 20, dtype=torch.uint8),
                torch.empty(1 << 20, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError):
            g.attn_fwd_paged_fp8kv(**d, workspace=bad)


@pytest.mark.parametrize("lens,kw,parts", [
    # 8 KV heads, one block each: the tiles visited by the longest block decide, four of them to a part
    ([100000], dict(window_left=200), (1, 1)), ([9000, 300], dict(window_left=400), (1, 1)),
    ([100000], dict(window_left=4095), (2, 9)), ([1100], dict(window_left=300), (1, 1)), ([1100], dict(), (2, 2)),
    ([1100] * 9, dict(), (1, 1)),
    ([8192, 300, 3], dict(), (2, 6)), ([20000], dict(causal=False, window_left=300, window_right=10), (1, 1)),
], ids=str)
def test_parts_follow_the_visited_tiles(g, lens, kw, parts):
    """The plan leaves the number of parts in the fourth word of the workspace (where the
    window alone already rules parts out, it is not asked)."""
    p = inputs([4] + [2] * (len(lens) - 1), lens, 16, 8, 128, 64, seed=53)
    T, B = p["q"].shape[0], len(lens)
    size = g.attn_paged_fp8kv_workspace_size(B, T, 16, 8, 128, 64, p["block_table"].shape[1])
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    ws[:16].view(torch.int32)[3] = 1
    o, lse = run(g, p, workspace=ws, **kw)
    check(p, o, lse, label=str(kw), **kw)
    got = int(ws[:16].view(torch.int32)[3])
    assert parts[0] <= got <= parts[1], got
