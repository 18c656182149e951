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
