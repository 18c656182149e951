"""Cases of the serving-step operators around the paged attention calls.

Four operators, in the order one serving step uses them:

* ``slots``: block tables, slot map and packed offsets from request lengths
  (``attn_paged_slots``).  Whole numbers only.
* ``rope``: per-head RMS norm of queries and keys and the position rotation in
  one pass (``attn_qk_norm_rope``).
* ``rope_paged``: the same, with keys and values written into a paged cache
  through the slot map, 16-bit or float8_e4m3fn (``attn_qk_norm_rope_paged``).
* ``attn``: packed queries (chunks and single-token steps) over a
  float8_e4m3fn paged cache (``attn_fwd_paged_fp8kv``).

``run`` computes them with elementary torch operations, or, with ``own`` set,
through the package's entry points.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
E4M3_MAX = 448.0


def listed():
    return [
        # the table update of a decode batch: one new token per request, every step of a serving loop
        dict(name="slots_decode", op="slots", B=64, lo=1, hi=1, ctx=16384, page_size=64),
        # admission of a large batch of prompt chunks with small pages; some requests bring no token
        dict(name="slots_chunks", op="slots", B=768, lo=0, hi=331, ctx=4096, page_size=16),
        # a few tokens of a small model: launch latency
        dict(name="rope_few", op="rope", T=5, Hq=4, Hkv=2, D=64, rot=64, dtype="fp16", pairs="half", axes="one",
             norm=True, max_pos=4096),
        # image or video patches: three position axes taking turns over the pairs, an odd number of tokens
        dict(name="rope_patches", op="rope", T=4099, Hq=16, Hkv=16, D=64, rot=64, dtype="bf16", pairs="half",
             axes="cycle", norm=False, max_pos=1024),
        # a long prompt at the 32/8/128 geometry, q and k being columns of one fused projection
        dict(name="rope_prompt", op="rope", T=16384, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16", pairs="half",
             axes="one", norm=True, max_pos=32768),
        # a decode batch padded to 64 rows, e4m3 caches: launch latency
        dict(name="cache_decode", op="rope_paged", T=64, real=61, B=64, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16",
             pairs="half", axes="one", norm=True, max_pos=32768, page_size=64, e4m3=True),
        # ragged chunks at the 24/2/256 geometry: partial rotation of neighbouring pairs, sectioned axes, 16-bit caches
        dict(name="cache_chunk", op="rope_paged", T=3001, real=3001, B=7, Hq=24, Hkv=2, D=256, rot=64, dtype="fp16",
             pairs="next", axes="sections", norm=True, max_pos=8192, page_size=16, e4m3=False),
        # a full prefill step into e4m3 caches at the 64/8/128 geometry
        dict(name="cache_prefill", op="rope_paged", T=16384, real=16384, B=16, Hq=64, Hkv=8, D=128, rot=128,
             dtype="bf16", pairs="half", axes="one", norm=True, max_pos=32768, page_size=64, e4m3=True),
        # short requests, a few new tokens each (drafts to verify), odd pages: latency
        dict(name="attn_short", op="attn", Hq=32, Hkv=8, D=128, dtype="bf16", page_size=24, steps=2, step_lo=1,
             step_hi=300, chunks=3, q_lo=2, q_hi=9, ctx_lo=0, ctx_hi=500, window=-1, softcap=0.0, sinks=False),
        # one serving step: 60 decode steps and four 1024-token chunks at the 32/8/128 geometry
        dict(name="attn_mixed", op="attn", Hq=32, Hkv=8, D=128, dtype="bf16", page_size=64, steps=60, step_lo=1024,
             step_hi=16384, chunks=4, q_lo=1024, q_hi=1024, ctx_lo=0, ctx_hi=8192, window=-1, softcap=0.0,
             sinks=False),
        # ragged chunks at the 24/2/256 geometry with a window, capped scores and sinks, float16
        dict(name="attn_wide", op="attn", Hq=24, Hkv=2, D=256, dtype="fp16", page_size=16, steps=3, step_lo=1,
             step_hi=4096, chunks=5, q_lo=300, q_hi=1100, ctx_lo=0, ctx_hi=6000, window=4095, softcap=30.0,
             sinks=True),
        # a 2048-token chunk at the end of a 32768-token cache, 64/8/128
        dict(name="attn_long", op="attn", Hq=64, Hkv=8, D=128, dtype="bf16", page_size=64, steps=0, step_lo=1,
             step_hi=1, chunks=1, q_lo=2048, q_hi=2048, ctx_lo=30720, ctx_hi=30720, window=-1, softcap=0.0,
             sinks=False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["slots", "rope", "rope_paged", "attn", "attn"])
    if op == "slots":
        B = _log(rng, 1, 768)
        hi = rng.choice([1, 1, _log(rng, 2, 331)])
        return dict(op=op, B=B, lo=min(hi, rng.choice([0, 1])), hi=hi, ctx=_log(rng, 64, 16384),
                    page_size=rng.choice([1, 8, 16, 24, 64, 128]))
    if op == "attn":
        Hq, Hkv, D = rng.choice([(32, 8, 128), (16, 2, 128), (24, 2, 256), (8, 8, 128)])
        q_hi = _log(rng, 2, 1200)
        return dict(op=op, Hq=Hq, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "fp16"]),
                    page_size=rng.choice([8, 16, 24, 64, 128]), steps=rng.randrange(0, 17), step_lo=1,
                    step_hi=_log(rng, 16, 8192), chunks=rng.randrange(1, 5), q_lo=max(2, q_hi // 3), q_hi=q_hi,
                    ctx_lo=0, ctx_hi=_log(rng, 16, 6000), window=rng.choice([-1, -1, _log(rng, 1, 4096)]),
                    softcap=rng.choice([0.0, 0.0, 20.0]), sinks=rng.random() < 0.3)
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    rot = D if rng.random() < 0.6 else 16 * rng.randrange(1, D // 16 + 1)
    c = dict(op=op, T=_log(rng, 1, 12000), Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, D=D, rot=rot,
             dtype=rng.choice(["bf16", "fp16"]), pairs=rng.choice(["half", "next"]),
             axes=rng.choice(["one", "one", "sections", "cycle"]), norm=rng.random() < 0.8,
             max_pos=_log(rng, 512, 32768))
    if op == "rope_paged":
        c.update(real=c["T"] - rng.choice([0, 0, c["T"] // 9]), B=_log(rng, 1, 64),
                 page_size=rng.choice([1, 8, 16, 24, 64, 128]), e4m3=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed, k=0):
    return torch.Generator(device="cuda").manual_seed(seed * 16 + k)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_slots(c, seed):
    rng = random.Random(seed)
    B, ps = c["B"], c["page_size"]
    past = [rng.randint(0, c["ctx"]) for _ in range(B)]
    new = [rng.randint(c["lo"], c["hi"]) for _ in range(B)]
    max_pages = -(-(c["ctx"] + c["hi"]) // ps)
    held = [-(-n // ps) for n in past]
    used = sum(held)
    taken = sum(-(-(p + n) // ps) for p, n in zip(past, new)) - used
    spare = taken + 8
    perm = torch.randperm(used + spare, generator=_gen(seed), device="cuda").to(torch.int32)
    first = torch.tensor([0] + held[:-1], device="cuda").cumsum(0)
    p = torch.arange(max_pages, device="cuda")[None, :]
    h = torch.tensor(held, device="cuda")[:, None]
    at = (first[:, None] + p).clamp(max=max(used - 1, 0))
    table = torch.where(p < h, perm[at], torch.full_like(perm[at], -1)).contiguous()
    return dict(past=_ints(past), new=_ints(new), table=table, free=perm[used:].contiguous(), page_size=ps,
                num_pages=used + spare, tokens=B * c["hi"], out=None)


def _axes(c):
    """Position axis of each of the rot / 2 pairs, or None for one axis."""
    n = c["rot"] // 2
    if c["axes"] == "one":
        return None
    if c["axes"] == "cycle":
        return [j % 3 for j in range(n)]
    first, second = n // 4, n // 4 + (n - n // 4) // 2
    return [0 if j < first else (1 if j < second else 2) for j in range(n)]


def _prepare_rope(c, seed):
    T, Hq, Hkv, D, rot = (c[k] for k in ("T", "Hq", "Hkv", "D", "rot"))
    dt, g = DT[c["dtype"]], _gen(seed)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(dt)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    s = dict(q=q, k=k, v=v, qw=None, kw=None, half=c["pairs"] == "half", axes=_axes(c), rot=rot, dtype=dt)
    if c["norm"]:
        s["qw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        s["kw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
    freq = 1e6 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2))
    angle = torch.arange(c["max_pos"], device="cuda", dtype=torch.float64)[:, None] * freq
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["pair_axis"] = None if s["axes"] is None else torch.tensor(s["axes"], device="cuda")
    B = c.get("B", 1)
    request = torch.randint(0, B, (T,), generator=g, device="cuda").sort().values
    counts = torch.zeros(B, dtype=torch.int64, device="cuda").index_add_(0, request, torch.ones_like(request))
    within = torch.arange(T, device="cuda") - (counts.cumsum(0) - counts)[request]
    if s["axes"] is None:
        past = torch.randint(0, max(1, c["max_pos"] // 2), (B,), generator=g, device="cuda")
        s["positions"] = ((past[request] + within) % c["max_pos"]).int()
    else:
        s["positions"] = torch.randint(0, c["max_pos"], (3, T), generator=g, device="cuda").int()
    s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
    s["k_out"] = torch.zeros(T, Hkv, D, dtype=dt, device="cuda")
    if c["op"] == "rope_paged":
        ps, n = c["page_size"], c["real"]
        pages = (counts + ps - 1) // ps
        num_pages = -(-T // ps) + B + 1          # at least the pages that any split over B requests takes
        perm = torch.randperm(num_pages, generator=g, device="cuda")
        slot = perm[(pages.cumsum(0) - pages)[request] + within // ps] * ps + within % ps
        real = torch.arange(T, device="cuda") < n
        s.update(n=n, slots=torch.where(real, slot, -1).int(), requests=torch.where(real, request, -1).int(),
                 k_scale=None, v_scale=None, page_size=ps)
        ct = torch.float8_e4m3fn if c["e4m3"] else dt
        s["kc"] = torch.zeros(num_pages, ps, Hkv, D, device="cuda").to(ct)
        s["vc"] = torch.zeros(num_pages, ps, Hkv, D, device="cuda").to(ct)
        if c["e4m3"]:
            s["k_scale"] = 0.004 + 0.012 * torch.rand(B, Hkv, generator=g, device="cuda")
            s["v_scale"] = 0.004 + 0.012 * torch.rand(B, Hkv, generator=g, device="cuda")
    return s


def _lengths(c, seed):
    """(query counts, cache lengths), the single-token steps first.  The query
    counts belong to the case, so that every seed gives outputs of one shape."""
    mix, rng = random.Random(c["q_hi"] * 8 + c["chunks"]), random.Random(seed)
    nq = [1] * c["steps"] + [mix.randint(c["q_lo"], c["q_hi"]) for _ in range(c["chunks"])]
    past = [rng.randint(c["step_lo"], c["step_hi"]) - 1 for _ in range(c["steps"])]
    past += [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["chunks"])]
    return nq, [p + n for p, n in zip(past, nq)]


def _prepare_attn(c, seed):
    Hq, Hkv, D, ps, dt, g = c["Hq"], c["Hkv"], c["D"], c["page_size"], DT[c["dtype"]], _gen(seed)
    nq, L = _lengths(c, seed)
    B, pages = len(nq), [-(-n // ps) for n in L]
    used = sum(pages)
    num_pages = used + used // 10 + 1
    perm = torch.randperm(num_pages, generator=g, device="cuda").int()
    max_pages = max(pages)
    first = torch.tensor([0] + pages[:-1], device="cuda").cumsum(0)
    p = torch.arange(max_pages, device="cuda")[None, :]
    at = (first[:, None] + p).clamp(max=num_pages - 1)
    table = torch.where(p < torch.tensor(pages, device="cuda")[:, None], perm[at], -1).int().contiguous()
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    s = dict(c=c, q=torch.randn(cu[-1], Hq, D, generator=g, device="cuda").to(dt), cu=_ints(cu), L=_ints(L),
             table=table, page_size=ps, nq=nq, lens=L, sinks=None, window=c["window"], softcap=c["softcap"],
             scale=1.0 / math.sqrt(D))
    s["kc"] = torch.randn(num_pages, ps, Hkv, D, generator=g, device="cuda").to(torch.float8_e4m3fn)
    s["vc"] = torch.randn(num_pages, ps, Hkv, D, generator=g, device="cuda").to(torch.float8_e4m3fn)
    s["k_scale"] = 0.25 + 0.75 * torch.rand(B, Hkv, generator=g, device="cuda")
    s["v_scale"] = 0.25 + 0.75 * torch.rand(B, Hkv, generator=g, device="cuda")
    if c["sinks"]:
        s["sinks"] = torch.randn(Hq, generator=g, device="cuda")
    return s


def prepare(case, seed):
    op = case["op"]
    s = (_prepare_slots if op == "slots" else _prepare_attn if op == "attn" else _prepare_rope)(case, seed)
    s["op"] = op
    return s


# ---------------------------------------------------------------- the plain forms

def _slots_plain(s):
    ps, T, table, free = s["page_size"], s["tokens"], s["table"], s["free"]
    B, max_pages = table.shape
    cap = max_pages * ps
    past, new = s["past"].long().clamp(0, cap), s["new"].long().clamp(min=0)
    end = past + new
    total = new.cumsum(0)
    n0 = (past + ps - 1) // ps
    n1 = torch.maximum(n0, ((end + ps - 1) // ps).clamp(max=max_pages))
    need = (n1 - n0).cumsum(0)
    p = torch.arange(max_pages, device=table.device)[None, :]
    at = (need - (n1 - n0) - n0)[:, None] + p
    ids = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where((p >= n0[:, None]) & (p < n1[:, None]), ids, table))
    t = torch.arange(T, device=table.device)
    first = total - new
    begins = torch.zeros(T + 1, dtype=torch.int64, device=table.device)
    begins.index_add_(0, first.clamp(max=T), torch.ones_like(first))
    real = t < total[-1]
    b = (begins[:T].cumsum(0) - 1).clamp(0, B - 1)
    pos = past[b] + t - first[b]
    page = table[b, (pos // ps).clamp(max=max_pages - 1)].long()
    ok = real & (pos < cap) & (page >= 0) & (page < s["num_pages"])
    cu = torch.cat([torch.zeros_like(total[:1]), total]).clamp(max=T)
    counts = torch.stack([total[-1], need[-1], need[-1]])
    return (cu.int(), end.clamp(max=cap).int(), torch.where(ok, page * ps + pos % ps, -1).int(),
            torch.where(real, pos, 0).int(), torch.where(real, b, -1).int(), counts.int(), table)


def _rope_plain(s, x, w):
    """The normed and rotated heads [T, H, D] in 32 bits."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    rot, n = s["rot"], s["rot"] // 2
    pos = s["positions"].long()
    if s["axes"] is None:
        cos, sin = s["table"][pos].split(n, 1)
    else:
        p, j = pos[s["pair_axis"]].t(), torch.arange(n, device=x.device)
        cos, sin = s["table"][p, j], s["table"][p, j + n]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., :n], x[..., n:rot]) if s["half"] else (x[..., 0:rot:2], x[..., 1:rot:2])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([ya, yb], -1) if s["half"] else torch.stack([ya, yb], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _store_plain(s, cache, x, scale):
    rows, at = cache.view(-1, *cache.shape[2:]), s["slots"][:s["n"]].long()
    if scale is None:
        rows[at] = x.to(cache.dtype)
    else:
        x = (x / scale[s["requests"][:s["n"]].long()][..., None]).clamp(-E4M3_MAX, E4M3_MAX)
        rows.view(torch.uint8)[at] = x.to(cache.dtype).view(torch.uint8)


def _attn_plain_group(s, b0, b1, t0, o, lse):
    """Requests b0 .. b1 - 1 (queries from row t0), padded to their longest."""
    c, ps = s["c"], s["page_size"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    n, nb, dev = Hq // Hkv, b1 - b0, o.device
    S, M = max(s["nq"][b0:b1]), max(s["lens"][b0:b1])
    cu, L = s["cu"][b0:b1 + 1].long(), s["L"][b0:b1].long()
    nq = cu[1:] - cu[:-1]
    i, j = torch.arange(S, device=dev), torch.arange(M, device=dev)
    page = s["table"][b0:b1, :-(-M // ps)].long().clamp(min=0)
    row = (page[:, :, None] * ps + torch.arange(ps, device=dev)).flatten(1)[:, :M]
    k = s["kc"].view(torch.uint8).view(-1, Hkv, D)[row].view(torch.float8_e4m3fn).float()
    v = s["vc"].view(torch.uint8).view(-1, Hkv, D)[row].view(torch.float8_e4m3fn).float()
    k = (k * s["k_scale"][b0:b1, None, :, None]).permute(0, 2, 3, 1)                      # [nb, Hkv, D, M]
    v = torch.where((j < L[:, None])[:, :, None, None], v * s["v_scale"][b0:b1, None, :, None], 0.0).transpose(1, 2)
    qi = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][qi].float().view(nb, S, Hkv, n, D).permute(0, 2, 1, 3, 4).reshape(nb, Hkv, S * n, D)
    z = torch.matmul(q, k).mul_(s["scale"]).view(nb, Hkv, S, n, M)
    if s["softcap"]:
        z = torch.tanh(z / s["softcap"]) * s["softcap"]
    at = i + (L - nq)[:, None]                                                            # key position of query i
    seen = (j <= at[:, :, None]) & (j < L[:, None, None])
    if s["window"] >= 0:
        seen &= j >= at[:, :, None] - s["window"]
    z = z.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(Hkv, 1, n, 1)
        top = torch.maximum(top, sink)
    w = z.sub_(top).exp_()
    den = w.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        den = den + (sink - top).exp()
    y = torch.matmul(w.view(nb, Hkv, S * n, M), v).view(nb, Hkv, S, n, D) / den
    real = (i < nq[:, None]).flatten()
    rows = torch.where(real, qi.flatten(), o.shape[0] - 1)     # the padding goes to a spare last row
    o[rows] = y.permute(0, 2, 1, 3, 4).reshape(nb * S, Hq, D).to(o.dtype)
    lse[rows] = (top + den.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(nb * S, Hq)


def _attn_plain(s):
    c, T = s["c"], s["q"].shape[0]
    o = torch.empty(T + 1, c["Hq"], c["D"], dtype=s["q"].dtype, device=s["q"].device)
    lse = torch.empty(T + 1, c["Hq"], device=s["q"].device)
    if c["steps"]:
        _attn_plain_group(s, 0, c["steps"], 0, o, lse)
    if c["chunks"]:
        _attn_plain_group(s, c["steps"], c["steps"] + c["chunks"], c["steps"], o, lse)
    return o[:T], lse[:T]


def _run_plain(s):
    if s["op"] == "slots":
        return _slots_plain(s)
    if s["op"] == "attn":
        return _attn_plain(s)
    if s["op"] == "rope":
        return _rope_plain(s, s["q"], s["qw"]).to(s["dtype"]), _rope_plain(s, s["k"], s["kw"]).to(s["dtype"])
    n = s["n"]
    s["q_out"][:n] = _rope_plain(s, s["q"], s["qw"])[:n].to(s["dtype"])
    _store_plain(s, s["kc"], _rope_plain(s, s["k"], s["kw"])[:n], s["k_scale"])
    _store_plain(s, s["vc"], s["v"][:n].float(), s["v_scale"])
    return s["q_out"], s["kc"], s["vc"]


# ---------------------------------------------------------------- the package's operators

def _run_own(s):
    import gqa_softmax_attention_gb300 as gqa
    if s["op"] == "slots":
        s["out"] = gqa.attn_paged_slots(s["past"], s["new"], s["table"], s["free"], s["page_size"], s["num_pages"],
                                        s["tokens"], out=s["out"])
        return s["out"] + (s["table"],)
    if s["op"] == "rope":
        return gqa.attn_qk_norm_rope(s["q"], s["k"], s["table"], s["positions"], q_weight=s["qw"], k_weight=s["kw"],
                                     eps=EPS, interleaved=not s["half"], axes=s["axes"], out=(s["q_out"], s["k_out"]))
    if s["op"] == "rope_paged":
        q = gqa.attn_qk_norm_rope_paged(s["q"], s["k"], s["v"], s["table"], s["positions"], s["slots"], s["kc"],
                                        s["vc"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                        interleaved=not s["half"], axes=s["axes"], k_scale=s["k_scale"],
                                        v_scale=s["v_scale"],
                                        requests=s["requests"] if s["k_scale"] is not None else None, out=s["q_out"])
        return q, s["kc"], s["vc"]
    return gqa.attn_fwd_paged_fp8kv(s["q"], s["kc"], s["vc"], s["k_scale"], s["v_scale"], s["cu"], s["L"], s["table"],
                                    scale=s["scale"], window_left=s["window"], softcap=s["softcap"] or None,
                                    sinks=s["sinks"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work and exact values

def work(case):
    op = case["op"]
    if op == "slots":
        B, T, mean = case["B"], case["B"] * case["hi"], (case["lo"] + case["hi"]) / 2
        pages = B * mean / case["page_size"]
        return {"bytes": 16.0 * B + 12.0 * T + 8.0 * pages, "flops": 0.0}
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if op == "attn":
        nq, L = _lengths(case, 1)
        w, pairs, read = case["window"], 0.0, 0.0
        for n, m in zip(nq, L):
            if w < 0:
                pairs += n * (m - n) + n * (n + 1) / 2
                read += m
            else:
                pairs += sum(min(w + 1, m - n + i + 1) for i in range(n))
                read += min(m, n + w)
        return {"bytes": 4.0 * sum(nq) * Hq * (D + 1) + 2.0 * read * Hkv * D, "flops": 4.0 * D * Hq * pairs}
    n = case.get("real", case["T"])
    table = 4.0 * case["rot"] * min(n, case["max_pos"])
    if op == "rope":
        return {"bytes": 4.0 * n * (Hq + Hkv) * D + table, "flops": 6.0 * n * (Hq + Hkv) * D}
    out = 1.0 if case["e4m3"] else 2.0
    return {"bytes": n * D * (4.0 * Hq + 2 * Hkv * (2.0 + out)) + table, "flops": 6.0 * n * (Hq + 2 * Hkv) * D}


def _exact_slots(case, seed):
    s = _prepare_slots(case, seed)
    past, new, table, free = (s[k].cpu().tolist() for k in ("past", "new", "table", "free"))
    ps, T, cap = s["page_size"], s["tokens"], len(table[0]) * s["page_size"]
    cu, lens, slots, positions, requests, taken = [0], [], [], [], [], 0
    for b, (p, n) in enumerate(zip(past, new)):
        for page in range(-(-p // ps), min(-(-(p + n) // ps), len(table[b]))):
            table[b][page] = free[taken] if taken < len(free) else -1
            taken += 1
        for x in range(p, p + n):
            page = table[b][x // ps] if x < cap else -1
            slots.append(page * ps + x % ps if 0 <= page < s["num_pages"] else -1)
            positions.append(x)
            requests.append(b)
        lens.append(min(p + n, cap))
        cu.append(min(T, cu[-1] + n))
    pad = T - len(slots)
    return tuple(_ints(x) for x in (cu, lens, slots + [-1] * pad, positions + [0] * pad, requests + [-1] * pad,
                                    [sum(new), taken, taken], table))


def _exact_heads(s, x, w):
    """Pair by pair: complex numbers times e^(i angle), in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    n = s["rot"] // 2
    lead = torch.arange(n, device=x.device) * (1 if s["half"] else 2)
    mate = lead + (n if s["half"] else 1)
    axis = torch.zeros(n, dtype=torch.int64, device=x.device) if s["axes"] is None else s["pair_axis"]
    pos = s["positions"].long().view(-1, x.shape[0])
    turn = torch.stack([torch.complex(s["table"][pos[axis[j]], j].double(), s["table"][pos[axis[j]], j + n].double())
                        for j in range(n)], 1)
    z = torch.complex(x[..., lead], x[..., mate]) * turn[:, None]
    y = x.clone()
    y[..., lead], y[..., mate] = z.real, z.imag
    return y


def _exact_rope(case, seed):
    s = _prepare_rope(case, seed)
    q, k = _exact_heads(s, s["q"], s["qw"]), _exact_heads(s, s["k"], s["kw"])
    if case["op"] == "rope":
        return q, k
    n, at = s["n"], s["slots"][:s["n"]].long()
    q[n:] = 0
    out = [q]
    for cache, x, scale in ((s["kc"], k[:n], s["k_scale"]), (s["vc"], s["v"][:n].double(), s["v_scale"])):
        full = torch.zeros(cache.shape, dtype=torch.float64, device=x.device)
        if scale is not None:
            x = (x / scale.double()[s["requests"][:n].long()][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        full.flatten(0, 1)[at] = x
        out.append(full)
    return tuple(out)


def _exact_attn(case, seed):
    s = _prepare_attn(case, seed)
    Hq, Hkv, D, ps = case["Hq"], case["Hkv"], case["D"], case["page_size"]
    n, q0 = Hq // Hkv, 0
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, (nq, L) in enumerate(zip(s["nq"], s["lens"])):
        t = torch.arange(L, device="cuda")
        row = s["table"][b].long()[t // ps] * ps + t % ps
        at = torch.arange(nq, device="cuda")[:, None] + (L - nq)
        hidden = t > at
        if s["window"] >= 0:
            hidden |= t < at - s["window"]
        for h in range(Hkv):
            k = s["kc"].flatten(0, 1)[:, h].view(torch.uint8)[row].view(torch.float8_e4m3fn).double() * s["k_scale"][b, h].double()
            v = s["vc"].flatten(0, 1)[:, h].view(torch.uint8)[row].view(torch.float8_e4m3fn).double() * s["v_scale"][b, h].double()
            for r in range(h * n, h * n + n):
                z = s["q"][q0:q0 + nq, r].double() @ k.t() * s["scale"]
                if s["softcap"]:
                    z = s["softcap"] * torch.tanh(z / s["softcap"])
                z[hidden] = -math.inf
                if s["sinks"] is not None:
                    z = torch.cat([z, s["sinks"][r].double().expand(nq, 1)], 1)
                l = torch.logsumexp(z, 1)
                o[q0:q0 + nq, r] = torch.exp(z[:, :L] - l[:, None]) @ v
                lse[q0:q0 + nq, r] = l
        q0 += nq
    return o, lse


def exact(case, seed):
    op = case["op"]
    return (_exact_slots if op == "slots" else _exact_attn if op == "attn" else _exact_rope)(case, seed)
