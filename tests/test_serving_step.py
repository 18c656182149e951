"""Serving steps end to end on the GPU: page tables and slots from the lengths,
norm + rotation into the paged cache, attention over that cache; prompt chunks
first, then decode steps, against one plain causal attention over the whole
sequences in 64 bits.

Tolerance.  Beside the attention's own roundings (the parity limits), a stored
16-bit key or query is off by 2^-9 relative in bfloat16, which moves a score of
|scale * q.k| <= sqrt(D) * rms^2 units by less than 2^-8 * sqrt(D) ~ 0.05 at
the extreme and 2^-8 typically; the 64-bit side therefore starts from the values
that the cache and q_out hold, so that only the attention's roundings remain,
and the stored values are checked against the formula on their own.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gqa_softmax_attention_gb300 import build
    build.build()
    import gqa_softmax_attention_gb300 as m
    yield m
    m.gqa_device_error()


def norm_rope(x, w, table, pos):
    n = x.double() / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6) * w.double()
    half = table.shape[1] // 2
    co, si = table.double()[pos, :half][:, None], table.double()[pos, half:][:, None]
    a, b = n[..., :half], n[..., half:]
    return torch.cat([a * co - b * si, b * co + a * si], -1)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_chunks_then_decode(g, e4m3, graph):
    dev, B, Hq, Hkv, D, ps, max_pages = "cuda", 5, 8, 2, 128, 16, 32
    gen = torch.Generator().manual_seed(1)
    num_pages, pad = B * max_pages, 7
    cdtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc = torch.zeros(num_pages, ps, Hkv, D, device=dev).to(cdtype)
    vc = torch.zeros(num_pages, ps, Hkv, D, device=dev).to(cdtype)
    ks = (0.01 + 0.02 * torch.rand(B, Hkv, generator=gen)).to(dev) if e4m3 else None
    vs = (0.01 + 0.02 * torch.rand(B, Hkv, generator=gen)).to(dev) if e4m3 else None
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(num_pages, generator=gen).int().to(dev)
    start = torch.zeros(1, dtype=torch.int32, device=dev)
    past = torch.zeros(B, dtype=torch.int32, device=dev)
    cos_sin = g.rope_table(max_pages * ps, D, base=1e6, device=dev)
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=gen)).bfloat16().to(dev) for _ in range(2))
    steps = [[100, 1, 0, 260, 33], [57, 3, 9, 1, 40]] + [[1, 1, 1, 1, 1]] * 4 + [[1, 0, 4, 1, 2]]
    hist = [dict(x=[], q=[], o=[], lse=[]) for _ in range(B)]
    T = max(sum(s) for s in steps) + pad
    new = torch.zeros(B, dtype=torch.int32, device=dev)
    qkv = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device=dev)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    qo = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
    o, lse = torch.zeros_like(qo), torch.zeros(T, Hq, device=dev)
    state = {}

    def step():
        state["m"] = g.attn_paged_slots(past, new, table, free, ps, num_pages, T, free_start=start,
                                        out=state.get("m"))
        cu, lens, slots, pos, req, counts = state["m"]
        g.attn_qk_norm_rope_paged(q, k, v, cos_sin, pos, slots, kc, vc, qw, kw, k_scale=ks, v_scale=vs,
                                  requests=req if e4m3 else None, out=qo)
        if e4m3:
            g.attn_fwd_paged_fp8kv(qo, kc, vc, ks, vs, cu, lens, table, out=o, lse=lse)
        else:
            g.attn_fwd_paged(qo, kc, vc, cu, lens, table, out=o, lse=lse)

    recorded = None
    for s in steps:
        rows = [torch.randn(n, (Hq + 2 * Hkv) * D, generator=gen).bfloat16() for n in s]
        flat = torch.cat(rows).to(dev)
        qkv.fill_(float("nan"))
        qkv[:sum(s)] = flat
        new.copy_(torch.tensor(s, dtype=torch.int32))
        if graph and recorded is None:
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                step()                                       # buffers and kernels, before the capture
            torch.cuda.current_stream().wait_stream(stream)
            recorded = torch.cuda.CUDAGraph()
            with torch.cuda.graph(recorded, stream=stream):
                step()
        if graph:
            recorded.replay()
        else:
            step()
        torch.cuda.synchronize()
        cu = state["m"][0].tolist()
        for b, n in enumerate(s):
            hist[b]["x"].append(rows[b])
            hist[b]["q"].append(qo[cu[b]:cu[b + 1]].cpu())
            hist[b]["o"].append(o[cu[b]:cu[b + 1]].cpu())
            hist[b]["lse"].append(lse[cu[b]:cu[b + 1]].cpu())
        past.copy_(state["m"][1])
        start.copy_(state["m"][5][2:])

    totals = [sum(s[b] for s in steps) for b in range(B)]
    assert past.tolist() == totals
    assert int(start) == sum(-(-n // ps) for n in totals)
    used = [p for row in table.tolist() for p in row if p >= 0]
    assert len(used) == len(set(used)) == int(start)
    for b in range(B):
        n, x = totals[b], torch.cat(hist[b]["x"])
        xq, xk, xv = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        pos = torch.arange(n)
        t = torch.arange(n, device=dev)
        at = table[b].long()[t // ps] * ps + t % ps
        raw = [c.view(torch.uint8 if e4m3 else torch.bfloat16).view(-1, Hkv, D)[at].view(cdtype) for c in (kc, vc)]
        sk = ks[b].double().cpu()[:, None] if e4m3 else 1.0
        sv = vs[b].double().cpu()[:, None] if e4m3 else 1.0
        k64, v64 = raw[0].float().cpu().double() * sk, raw[1].float().cpu().double() * sv
        # what was stored, against the formula: half a step of the stored type and FP32 slop
        want = norm_rope(xk, kw.cpu(), cos_sin.cpu(), pos)
        step_of = 2.0 ** -4 if e4m3 else 2.0 ** -8
        floor = 2.0 ** -10 * sk if e4m3 else 0.0
        assert bool(((k64 - want).abs() <= step_of * want.abs() * 1.001 + floor + 1e-4 * step_of).all())
        assert bool(((v64 - xv.double()).abs() <= (step_of * xv.double().abs() * 1.001 + floor if e4m3 else 0)).all())
        q64 = torch.cat(hist[b]["q"]).double()
        wq = norm_rope(xq, qw.cpu(), cos_sin.cpu(), pos)
        assert bool(((q64 - wq).abs() <= 2.0 ** -8 * wq.abs() * 1.001 + 2.0 ** -12 * 1e-4 + 1e-4 * 2.0 ** -8).all())
        rep = Hq // Hkv
        z = torch.einsum("ihd,jhd->hij", q64, k64.repeat_interleave(rep, 1)) / math.sqrt(D)
        z.masked_fill_(torch.arange(n)[None] > torch.arange(n)[:, None], -math.inf)
        ref = torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), v64.repeat_interleave(rep, 1))
        got, gl = torch.cat(hist[b]["o"]).double(), torch.cat(hist[b]["lse"]).double()
        assert float((got - ref).abs().max()) <= 2e-2 and float((got - ref).abs().mean()) <= 2e-3
        assert float((gl - torch.logsumexp(z, -1).t()).abs().max()) <= 1e-3


@pytest.mark.parametrize("over", ["capacity", "rows"])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_a_request_that_does_not_fit(g, e4m3, over):
    """One request past the table's capacity, or a batch cut by its rows: the other
    requests are as ever, the tokens with a slot are stored, the cut shows where the
    documentation says, and the step repeated with the lengths cut is right throughout."""
    dev, Hq, Hkv, D, ps, max_pages = "cuda", 8, 2, 128, 16, 6
    cap, B = ps * max_pages, 3
    gen = torch.Generator().manual_seed(5)
    held = [40, cap - 2, 20] if over == "capacity" else [40, 30, 20]
    asked = [3, 5, 2] if over == "capacity" else [3, 2, 6]
    fits = [3, 2, 2]
    T = 12 if over == "capacity" else 7
    num_pages = B * max_pages + 4
    cdtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    raw = torch.uint8 if e4m3 else torch.bfloat16
    kc, vc = (torch.randn(num_pages, ps, Hkv, D, generator=gen).to(cdtype).to(dev) for _ in range(2))
    sc = torch.full((B, Hkv), 0.02, device=dev) if e4m3 else None
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    ids = torch.randperm(num_pages, generator=gen).int()
    table, at = torch.full((B, max_pages), -1, dtype=torch.int32), 0
    for b, n in enumerate(held):
        m = -(-n // ps)
        table[b, :m] = ids[at:at + m]
        at += m
    table, free = table.to(dev), ids[at:].contiguous().to(dev)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=gen).bfloat16().to(dev)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cos_sin, w = g.rope_table(cap + 8, D, device=dev), torch.ones(D, dtype=torch.bfloat16, device=dev)

    def step(new, x):
        m = g.attn_paged_slots(i32(held), i32(new), table, free, ps, num_pages, T)
        a = (x[0], x[1], x[2], cos_sin, m[3], m[2], kc, vc, w, w)
        qo = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
        if e4m3:
            g.attn_qk_norm_rope_paged(*a, k_scale=sc, v_scale=sc, requests=m[4], out=qo)
            o, lse = g.attn_fwd_paged_fp8kv(qo, kc, vc, sc, sc, m[0], m[1], table)
        else:
            g.attn_qk_norm_rope_paged(*a, out=qo)
            o, lse = g.attn_fwd_paged(qo, kc, vc, m[0], m[1], table)
        torch.cuda.synchronize()
        return m, qo, o, lse

    def right(b, m, qo, o, lse, n):
        """Request b's n queries, at positions held + i, against 64 bits."""
        a, L = int(m[0][b]), held[b] + n
        t = torch.arange(L, device=dev)
        rows = table[b].long()[t // ps] * ps + t % ps
        f = 0.02 if e4m3 else 1.0
        k64, v64 = ((c.view(raw).view(-1, Hkv, D)[rows].view(cdtype).float().cpu().double() * f)
                    .repeat_interleave(Hq // Hkv, 1) for c in (kc, vc))
        z = torch.einsum("ihd,jhd->hij", qo[a:a + n].cpu().double(), k64) / math.sqrt(D)
        z.masked_fill_(torch.arange(L)[None] > (held[b] + torch.arange(n))[:, None], -math.inf)
        ref = torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), v64)
        assert float((o[a:a + n].cpu().double() - ref).abs().max()) <= 2e-2
        assert float((lse[a:a + n].cpu().double() - torch.logsumexp(z, -1).t()).abs().max()) <= 1e-3

    m, qo, o, lse = step(asked, (q, k, v))
    cut = 1 if over == "capacity" else 2
    for b in range(B):
        if b != cut:
            right(b, m, qo, o, lse, asked[b])
    slots, pos, req, counts = (x.tolist() for x in m[2:])
    a = int(m[0][cut])
    for i in range(min(asked[cut], T - a)):
        p = held[cut] + i
        assert req[a + i] == cut and pos[a + i] == p
        assert slots[a + i] == (int(table[cut, p // ps]) * ps + p % ps if p < cap else -1)
    stored = g.attn_qk_norm_rope(q, k, cos_sin, m[3], w, w)[1]
    if not e4m3:
        for i in range(fits[cut]):
            assert torch.equal(kc.view(-1, Hkv, D)[slots[a + i]], stored[a + i])
            assert torch.equal(vc.view(-1, Hkv, D)[slots[a + i]], v[a + i])
    short = [L < h + n for L, h, n in zip(m[1].tolist(), held, asked)]
    assert short == [False, over == "capacity", False]
    assert (counts[0] > T) == (over == "rows") and counts[0] == sum(asked)
    # the step again, with what fits (the tokens that are left out closed up)
    keep = [int(m[0][b]) + i for b in range(B) for i in range(fits[b])]
    keep += [t for t in range(T) if t not in keep]
    m, qo, o, lse = step(fits, (q[keep], k[keep], v[keep]))
    assert m[5].tolist()[0] == sum(fits)
    for b in range(B):
        right(b, m, qo, o, lse, fits[b])
