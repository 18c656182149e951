"""Cases of latent attention: keys and values held as one shared latent vector a token.

A token's cache row is 576 numbers: a normed latent of 512, from which every
head's keys (128 dims) and values (128 dims) are projected, and 64 rotated dims
that all heads share.  Four operators, in the order a serving step uses them:

* ``append``: RMS norm of the latents and rotation of the shared dims, written
  into a paged cache, with the queries' rotated dims put beside their absorbed
  part (``attn_latent_norm_rope_paged``).
* ``gather``: the cache rows of requests, packed, for the projection that expands
  them (``attn_latent_gather``).
* ``expanded``: prompts and chunks over the projected keys and values of each
  head and the shared dims (``attn_fwd_latent_varlen``).
* ``absorbed``: packed queries already projected into the latent space, over the
  paged cache itself (``attn_fwd_latent_paged``).

``run`` computes them with elementary torch operations, or, with ``own`` set,
through the package's entry points.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
LATENT, SHARED, NOPE, VDIM = 512, 64, 128, 128
ROW = LATENT + SHARED
SCALE = 1.0 / math.sqrt(NOPE + SHARED)


def listed():
    return [
        # the next tokens of one or two short conversations: latency
        dict(name="absorbed_few", op="absorbed", H=16, dtype="bf16", page_size=64, steps=2, step_lo=300, step_hi=700,
             chunks=0, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=0),
        # a decode batch of a model whose 128 heads are shared out over eight GPUs
        dict(name="absorbed_decode", op="absorbed", H=16, dtype="bf16", page_size=64, steps=64, step_lo=1024,
             step_hi=16384, chunks=0, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=0),
        # drafted tokens to verify beside plain decode steps, small pages, ragged, float16
        dict(name="absorbed_drafts", op="absorbed", H=40, dtype="fp16", page_size=16, steps=9, step_lo=1,
             step_hi=5000, chunks=23, q_lo=2, q_hi=5, ctx_lo=0, ctx_hi=7000),
        # a decode batch with all 128 heads on one GPU
        dict(name="absorbed_wide", op="absorbed", H=128, dtype="bf16", page_size=64, steps=64, step_lo=1024,
             step_hi=16384, chunks=0, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=0),
        # a few short prompts of a small model, float16: latency
        dict(name="expanded_few", op="expanded", H=8, dtype="fp16", chunks=3, q_lo=7, q_hi=411, ctx_lo=0, ctx_hi=0),
        # a prefill batch of ragged prompts
        dict(name="expanded_prompts", op="expanded", H=32, dtype="bf16", chunks=8, q_lo=300, q_hi=4001, ctx_lo=0,
             ctx_hi=0),
        # the last 2048-token chunk of a 16384-token prompt
        dict(name="expanded_chunk", op="expanded", H=64, dtype="bf16", chunks=1, q_lo=2048, q_hi=2048, ctx_lo=14336,
             ctx_hi=14336),
        # a decode batch padded to 64 rows: latency
        dict(name="append_decode", op="append", T=64, real=61, B=64, H=128, dtype="bf16", pairs="next",
             max_pos=32768, page_size=64, packed=False),
        # chunks of a prompt, whose packed latents go on to the projection as well
        dict(name="append_prompt", op="append", T=16384, real=16384, B=4, H=32, dtype="bf16", pairs="next",
             max_pos=32768, page_size=64, packed=True),
        # odd chunks, small pages, rotation of halves, float16
        dict(name="append_ragged", op="append", T=1237, real=1201, B=7, H=20, dtype="fp16", pairs="half",
             max_pos=8192, page_size=24, packed=False),
        # the cached prefixes of two requests, small pages
        dict(name="gather_few", op="gather", B=2, lo=200, hi=1500, dtype="bf16", page_size=16),
        # the cached prefixes of a prefill batch
        dict(name="gather_long", op="gather", B=16, lo=1024, hi=16384, dtype="bf16", page_size=64),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["absorbed", "absorbed", "expanded", "append", "gather"])
    dtype = rng.choice(["bf16", "fp16"])
    ps = rng.choice([1, 8, 16, 24, 64, 128])
    if op == "gather":
        hi = _log(rng, 4, 16384)
        return dict(op=op, B=_log(rng, 1, 16), lo=rng.choice([0, 1, hi // 2]), hi=hi, dtype=dtype, page_size=ps)
    if op == "append":
        T = _log(rng, 1, 12000)
        return dict(op=op, T=T, real=T - rng.choice([0, 0, T // 9]), B=_log(rng, 1, 64),
                    H=rng.choice([1, 4, 8, 20, 32]), dtype=dtype, pairs=rng.choice(["next", "half"]),
                    max_pos=_log(rng, 512, 32768), page_size=ps, packed=rng.random() < 0.4)
    if op == "expanded":
        q_hi = _log(rng, 2, 1800)
        return dict(op=op, H=rng.choice([1, 4, 8, 12, 20, 32]), dtype=dtype, chunks=rng.randrange(1, 7),
                    q_lo=max(1, q_hi // 3), q_hi=q_hi, ctx_lo=0, ctx_hi=rng.choice([0, 0, _log(rng, 16, 4000)]))
    q_hi = _log(rng, 2, 60)
    steps = rng.choice([0, _log(rng, 1, 48), _log(rng, 1, 48)])
    return dict(op=op, H=rng.choice([1, 8, 16, 20, 32, 64, 128]), dtype=dtype, page_size=ps, steps=steps, step_lo=1,
                step_hi=_log(rng, 16, 12000), chunks=rng.randrange(1, 5) if steps == 0 else rng.randrange(0, 3),
                q_lo=max(1, q_hi // 3), q_hi=q_hi, ctx_lo=0, ctx_hi=_log(rng, 16, 6000))


# ---------------------------------------------------------------- inputs

def _gen(seed, k=0):
    return torch.Generator(device="cuda").manual_seed(seed * 16 + k)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _sums(x):
    out = [0]
    for n in x:
        out.append(out[-1] + n)
    return out


def _lengths(c, seed):
    """(query counts, key counts), the single-token steps first.  The query
    counts belong to the case, so that every seed gives outputs of one shape."""
    steps = c.get("steps", 0)
    mix, rng = random.Random(c["q_hi"] * 8 + c["chunks"]), random.Random(seed)
    nq = [1] * steps + [mix.randint(c["q_lo"], c["q_hi"]) for _ in range(c["chunks"])]
    past = [rng.randint(c["step_lo"], c["step_hi"]) - 1 for _ in range(steps)]
    past += [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["chunks"])]
    return nq, [p + n for p, n in zip(past, nq)]


def _pages(lens, ps, g):
    """Block table of requests of these lengths over shuffled pages, and the number of pages of the pool."""
    pages = [-(-n // ps) for n in lens]
    used, most = sum(pages), max(1, max(pages))
    num_pages = used + used // 10 + 1
    perm = torch.randperm(num_pages, generator=g, device="cuda").int()
    first = torch.tensor(_sums(pages)[:-1], device="cuda")
    p = torch.arange(most, device="cuda")[None, :]
    at = (first[:, None] + p).clamp(max=num_pages - 1)
    return torch.where(p < torch.tensor(pages, device="cuda")[:, None], perm[at], -1).int().contiguous(), num_pages


def _cache(num_pages, ps, dt, g):
    return torch.randn(num_pages, ps, ROW, generator=g, device="cuda").to(dt)


def _prepare_absorbed(c, seed):
    dt, g, ps = DT[c["dtype"]], _gen(seed), c["page_size"]
    nq, L = _lengths(c, seed)
    table, num_pages = _pages(L, ps, g)
    cu = _sums(nq)
    return dict(c=c, nq=nq, lens=L, table=table, page_size=ps, cu=_ints(cu), L=_ints(L),
                q=torch.randn(cu[-1], c["H"], ROW, generator=g, device="cuda").to(dt),
                cache=_cache(num_pages, ps, dt, g))


def _prepare_expanded(c, seed):
    dt, g, H = DT[c["dtype"]], _gen(seed), c["H"]
    nq, L = _lengths(c, seed)
    cq, ck = _sums(nq), _sums(L)
    kv = torch.randn(ck[-1], H, NOPE + VDIM, generator=g, device="cuda").to(dt)    # one projection of the latents
    rows = torch.randn(ck[-1], ROW, generator=g, device="cuda").to(dt)             # whose last dims are the shared ones
    return dict(c=c, nq=nq, lens=L, cq=_ints(cq), ck=_ints(ck), k=kv[..., :NOPE], v=kv[..., NOPE:],
                k_pe=rows[:, LATENT:], q=torch.randn(cq[-1], H, NOPE + SHARED, generator=g, device="cuda").to(dt))


def _prepare_append(c, seed):
    T, H, B, ps, n = c["T"], c["H"], c["B"], c["page_size"], c["real"]
    dt, g = DT[c["dtype"]], _gen(seed)
    q = torch.randn(T, H, NOPE + SHARED, generator=g, device="cuda").to(dt)
    freq = 1e4 ** (-torch.arange(SHARED // 2, device="cuda", dtype=torch.float64) / (SHARED // 2))
    angle = torch.arange(c["max_pos"], device="cuda", dtype=torch.float64)[:, None] * freq
    request = torch.randint(0, B, (T,), generator=g, device="cuda").sort().values
    counts = torch.zeros(B, dtype=torch.int64, device="cuda").index_add_(0, request, torch.ones_like(request))
    within = torch.arange(T, device="cuda") - (counts.cumsum(0) - counts)[request]
    past = torch.randint(0, max(1, c["max_pos"] // 2), (B,), generator=g, device="cuda")
    pages = (counts + ps - 1) // ps
    num_pages = -(-T // ps) + B + 1              # at least the pages that any split over B requests takes
    perm = torch.randperm(num_pages, generator=g, device="cuda")
    slot = perm[(pages.cumsum(0) - pages)[request] + within // ps] * ps + within % ps
    return dict(c=c, n=n, q_pe=q[..., NOPE:], kv=torch.randn(T, ROW, generator=g, device="cuda").to(dt),
                weight=(1 + 0.2 * torch.randn(LATENT, generator=g, device="cuda")).to(dt),
                table=torch.cat([angle.cos(), angle.sin()], 1).float(), half=c["pairs"] == "half",
                positions=((past[request] + within) % c["max_pos"]).int(),
                slots=torch.where(torch.arange(T, device="cuda") < n, slot, -1).int(),
                cache=torch.zeros(num_pages, ps, ROW, dtype=dt, device="cuda"),
                q_out=torch.zeros(T, H, ROW, dtype=dt, device="cuda")[..., LATENT:],
                packed=torch.zeros(T, ROW, dtype=dt, device="cuda") if c["packed"] else None)


def _prepare_gather(c, seed):
    g, ps = _gen(seed), c["page_size"]
    mix = random.Random(c["hi"] * 8 + c["B"])                # of the case: the output has one shape
    lens = [mix.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    table, num_pages = _pages(lens, ps, g)
    return dict(c=c, lens=lens, cu=_ints(_sums(lens)), table=table, page_size=ps,
                cache=_cache(num_pages, ps, DT[c["dtype"]], g))


def prepare(case, seed):
    return {"absorbed": _prepare_absorbed, "expanded": _prepare_expanded, "append": _prepare_append,
            "gather": _prepare_gather}[case["op"]](case, seed)


# ---------------------------------------------------------------- the plain forms

def _softmax_parts(z, hidden):
    """(weights, their sums, log of the sums of the exponentials) of scores over
    their last axis; a row with nothing to see has weights and sums of zero."""
    z.masked_fill_(hidden, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = z.sub_(top).exp_()
    den = w.sum(-1, keepdim=True)
    return w, den, (top + den.log()).squeeze(-1)


def _absorbed_group(s, b0, b1, o, lse):
    """Requests b0 .. b1 - 1, padded to their longest."""
    ps, H, nb, dev = s["page_size"], s["c"]["H"], b1 - b0, o.device
    S, M = max(s["nq"][b0:b1]), max(s["lens"][b0:b1])
    cu, L = s["cu"][b0:b1 + 1].long(), s["L"][b0:b1].long()
    nq = cu[1:] - cu[:-1]
    i, j = torch.arange(S, device=dev), torch.arange(M, device=dev)
    row = (s["table"][b0:b1].long().clamp(min=0)[:, j // ps] * ps + j % ps)
    k = s["cache"].view(-1, ROW)[row].float().masked_fill_((j >= L[:, None])[..., None], 0.0)        # [nb, M, ROW]
    qi = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][qi].float().view(nb, S * H, ROW)
    z = torch.matmul(q, k.transpose(1, 2)).mul_(SCALE).view(nb, S, H, M)
    hidden = (j > (i + (L - nq)[:, None])[..., None]) | (j >= L[:, None, None])
    w, den, l = _softmax_parts(z, hidden[:, :, None, :])
    y = torch.matmul(w.view(nb, S * H, M), k[..., :LATENT]).view(nb, S, H, LATENT) / den.clamp(min=1e-38)
    rows = torch.where((i < nq[:, None]).flatten(), qi.flatten(), o.shape[0] - 1)   # the padding goes to a spare row
    o[rows] = y.view(nb * S, H, LATENT).to(o.dtype)
    lse[rows] = l.reshape(nb * S, H)


def _absorbed_plain(s):
    T, H, steps, B = s["q"].shape[0], s["c"]["H"], s["c"]["steps"], len(s["nq"])
    o = torch.empty(T + 1, H, LATENT, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(T + 1, H, device="cuda")
    if steps:
        _absorbed_group(s, 0, steps, o, lse)
    if B > steps:
        _absorbed_group(s, steps, B, o, lse)
    return o[:T], lse[:T]


def _expanded_plain(s):
    T, H, dev = s["q"].shape[0], s["c"]["H"], s["q"].device
    B, S, M = len(s["nq"]), max(s["nq"]), max(s["lens"])
    cq, ck = s["cq"].long(), s["ck"].long()
    nq, L = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    i, j = torch.arange(S, device=dev), torch.arange(M, device=dev)
    qi = (cq[:-1, None] + i).clamp(max=T - 1)
    kj = (ck[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"][qi].float().transpose(1, 2)                                          # [B, H, S, 192]
    z = torch.matmul(q[..., :NOPE], s["k"][kj].float().permute(0, 2, 3, 1))
    z += torch.matmul(q[..., NOPE:], s["k_pe"][kj].float().transpose(1, 2)[:, None])
    hidden = (j > (i + (L - nq)[:, None])[..., None]) | (j >= L[:, None, None])
    w, den, l = _softmax_parts(z.mul_(SCALE), hidden[:, None])
    v = s["v"][kj].float().masked_fill_((j >= L[:, None])[..., None, None], 0.0).transpose(1, 2)
    y = torch.matmul(w, v) / den.clamp(min=1e-38)
    real = i < nq[:, None]
    return y.transpose(1, 2)[real].to(s["q"].dtype), l.transpose(1, 2)[real]


def _turned_plain(s, x, n):
    """The first n rows of x [T, ..., 64], rotated by position."""
    cos, sin = s["table"][s["positions"][:n].long()].view(n, *[1] * (x.dim() - 2), SHARED).chunk(2, -1)
    x, h = x[:n].float(), SHARED // 2
    a, b = (x[..., :h], x[..., h:]) if s["half"] else (x[..., 0::2], x[..., 1::2])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    return torch.cat([ya, yb], -1) if s["half"] else torch.stack([ya, yb], -1).flatten(-2)


def _append_plain(s):
    n, dt = s["n"], s["kv"].dtype
    s["q_out"][:n] = _turned_plain(s, s["q_pe"], n).to(dt)
    c = s["kv"][:n, :LATENT].float()
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    rows = torch.cat([c, _turned_plain(s, s["kv"][:, LATENT:], n)], 1).to(dt)
    s["cache"].view(-1, ROW)[s["slots"][:n].long()] = rows
    if s["packed"] is None:
        return s["q_out"], s["cache"]
    s["packed"][:n] = rows
    return s["q_out"], s["cache"], s["packed"]


def _gather_plain(s):
    cu, ps = s["cu"].long(), s["page_size"]
    j = torch.arange(sum(s["lens"]), device="cuda")
    b = torch.searchsorted(cu, j, right=True) - 1
    t = j - cu[b]
    return s["cache"].view(-1, ROW)[s["table"][b, t // ps].long() * ps + t % ps]


# ---------------------------------------------------------------- the package's operators

def _run_own(s):
    import gqa_softmax_attention_gb300 as gqa
    op = s["c"]["op"]
    if op == "absorbed":
        return gqa.attn_fwd_latent_paged(s["q"], s["cache"], s["cu"], s["L"], s["table"], SCALE)
    if op == "expanded":
        return gqa.attn_fwd_latent_varlen(s["q"], s["k"], s["v"], s["k_pe"], s["cq"], s["ck"])
    if op == "gather":
        return gqa.attn_latent_gather(s["cache"], s["cu"], s["table"], sum(s["lens"]))
    q = gqa.attn_latent_norm_rope_paged(s["q_pe"], s["kv"], s["table"], s["positions"], s["slots"], s["cache"],
                                        kv_weight=s["weight"], eps=EPS, interleaved=not s["half"], out=s["q_out"],
                                        kv_out=s["packed"])
    return (q, s["cache"]) if s["packed"] is None else (q, s["cache"], s["packed"])


def run(state):
    if own:
        return _run_own(state)
    return {"absorbed": _absorbed_plain, "expanded": _expanded_plain, "append": _append_plain,
            "gather": _gather_plain}[state["c"]["op"]](state)


# ---------------------------------------------------------------- work and exact values

def work(case):
    op = case["op"]
    if op == "gather":
        mix = random.Random(case["hi"] * 8 + case["B"])
        return {"bytes": 4.0 * ROW * sum(mix.randint(case["lo"], case["hi"]) for _ in range(case["B"])), "flops": 0.0}
    if op == "append":
        n = case["real"]
        rows = 2.0 * ROW * n * (3 if case["packed"] else 2)
        return {"bytes": rows + 4.0 * n * case["H"] * SHARED + 4.0 * SHARED * min(n, case["max_pos"]),
                "flops": 4.0 * n * LATENT + 3.0 * n * SHARED * (case["H"] + 1)}
    nq, L = _lengths(case, 1)
    H = case["H"]
    pairs = sum(n * (m - n) + n * (n + 1) / 2 for n, m in zip(nq, L))
    if op == "absorbed":
        return {"bytes": 2.0 * ROW * sum(L) + sum(nq) * H * (2.0 * (ROW + LATENT) + 4),
                "flops": 2.0 * (ROW + LATENT) * H * pairs}
    return {"bytes": 2.0 * sum(L) * (H * (NOPE + VDIM) + SHARED) + sum(nq) * H * (2.0 * (NOPE + SHARED + VDIM) + 4),
            "flops": 2.0 * (NOPE + SHARED + VDIM) * H * pairs}


def _exact_rows(q, k, v, at, o, lse):
    """One request's attention of one head, in 64 bits: queries q [n, .] at key positions `at`."""
    z = q @ k.t() * SCALE
    z[torch.arange(k.shape[0], device=q.device) > at[:, None]] = -math.inf
    l = torch.logsumexp(z, 1)
    o.copy_(torch.where((l > -math.inf)[:, None], torch.exp(z - l.nan_to_num(neginf=0.0)[:, None]) @ v, 0.0))
    lse.copy_(l)


def _exact_attention(case, seed):
    absorbed = case["op"] == "absorbed"
    s = prepare(case, seed)
    T, H = s["q"].shape[:2]
    o = torch.empty(T, H, LATENT if absorbed else VDIM, dtype=torch.float64, device="cuda")
    lse = torch.empty(T, H, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for b, (n, m) in enumerate(zip(s["nq"], s["lens"])):
        q1, t = q0 + n, torch.arange(m, device="cuda")
        at = torch.arange(n, device="cuda") + (m - n)
        if absorbed:
            rows = s["cache"].flatten(0, 1)[s["table"][b].long()[t // s["page_size"]] * s["page_size"]
                                            + t % s["page_size"]].double()
            # the heads of a query see the same keys: one product over all of them
            _exact_rows(s["q"][q0:q1].double().flatten(0, 1), rows, rows[:, :LATENT], at.repeat_interleave(H),
                        o[q0:q1].view(n * H, LATENT), lse[q0:q1].view(n * H))
        else:
            for h in range(H):
                k = torch.cat([s["k"][k0:k0 + m, h], s["k_pe"][k0:k0 + m]], 1).double()
                _exact_rows(s["q"][q0:q1, h].double(), k, s["v"][k0:k0 + m, h].double(), at, o[q0:q1, h], lse[q0:q1, h])
        q0, k0 = q1, k0 + m
    return o, lse


def _exact_turn(s, x, n):
    """Pair by pair: complex numbers times e^(i angle), in 64 bits."""
    y, h = x.double().clone(), SHARED // 2
    y[n:] = 0
    pos = s["positions"][:n].long()
    for j in range(h):
        a, b = (j, j + h) if s["half"] else (2 * j, 2 * j + 1)
        turn = torch.complex(s["table"][pos, j].double(), s["table"][pos, j + h].double())
        z = torch.complex(x[:n, ..., a].double(), x[:n, ..., b].double()) * turn.view(n, *[1] * (x.dim() - 2))
        y[:n, ..., a], y[:n, ..., b] = z.real, z.imag
    return y


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    n = s["n"]
    c = s["kv"][:, :LATENT].double()
    c = c / (c.pow(2).sum(1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].double()
    rows = torch.cat([c, _exact_turn(s, s["kv"][:, LATENT:], n)], 1)
    rows[n:] = 0
    cache = torch.zeros(s["cache"].shape, dtype=torch.float64, device="cuda")
    cache.flatten(0, 1)[s["slots"][:n].long()] = rows[:n]
    q = _exact_turn(s, s["q_pe"], n)
    return (q, cache, rows) if case["packed"] else (q, cache)


def _exact_gather(case, seed):
    s = _prepare_gather(case, seed)
    out = []
    for b, n in enumerate(s["lens"]):
        pages = s["table"][b, :-(-n // s["page_size"])].long()
        out.append(s["cache"][pages].flatten(0, 1)[:n].double())
    return torch.cat(out)


def exact(case, seed):
    op = case["op"]
    return (_exact_append if op == "append" else _exact_gather if op == "gather" else _exact_attention)(case, seed)
