"""Per-head norm and rotation on the GPU, dense and into paged caches, against
the formula in 64 bits.

Tolerance.  A 16-bit result is the rounding of an FP32 value: half a step of
the type, eps / 2 relative (2^-8 bfloat16, 2^-11 float16), or half the smallest
subnormal.  The FP32 value itself: the mean square of D <= 256 values is off by
at most 8 + 5 + 2 roundings of 2^-24 relative, the root and its use by 4 more,
the weight times cosine, the products and the sum by 4 more, the mate's terms
likewise, so at most 32 roundings of 2^-24 of the magnitudes summed,
|n_d| + |n_mate|: DELTA = 2^-19.  An e4m3 code of y: half a step, 2^-4 relative
or 2^-10 absolute (steps of 2^-9 below 2^-6), after the same DELTA.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DELTA = 2.0 ** -19


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gqa_softmax_attention_gb300 import build
    build.build()
    import gqa_softmax_attention_gb300 as m
    yield m
    m.gqa_device_error()


def reference(x, w, table, pos, interleaved=False, axes=None, eps=1e-6):
    """(y, magnitude): x [T, H, D] normed and rotated in 64 bits, and |n_d| + |n_mate|."""
    x = x.double().cpu()
    n = x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double().cpu()
    y, mag = n.clone(), n.abs()
    if table is not None:
        table, pos, half = table.double().cpu(), pos.long().cpu(), table.shape[1] // 2
        for j in range(half):
            p = (pos if axes is None else pos[axes[j]]).reshape(-1)
            p = p.clamp(0, table.shape[0] - 1)
            co, si = table[p, j][:, None], table[p, half + j][:, None]
            d0, d1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            y[..., d0] = n[..., d0] * co - n[..., d1] * si
            y[..., d1] = n[..., d1] * co + n[..., d0] * si
            mag[..., d0] = mag[..., d1] = n[..., d0].abs() + n[..., d1].abs()
    return y, mag


def close16(got, ref, mag, label=""):
    dt = got.dtype
    d = DELTA * mag
    tol = torch.finfo(dt).eps / 2 * (ref.abs() + d) + d + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    off = (got.double().cpu() - ref).abs()
    assert bool((off <= tol).all()), "%s: worst %.3g of its tolerance" % (label, float((off / tol).max()))


def close8(codes, ref, mag, label=""):
    d = DELTA * mag
    want = ref.clamp(-448, 448)
    tol = torch.maximum(2.0 ** -4 * (want.abs() + d), torch.tensor(2.0 ** -10, dtype=torch.float64)) + d
    off = (codes.view(torch.float8_e4m3fn).float().cpu().double() - want).abs()
    assert bool((off <= tol).all()), "%s: worst %.3g of its tolerance" % (label, float((off / tol).max()))


def inputs(T, Hq, Hkv, D, dtype=torch.bfloat16, rot=None, max_pos=500, n_axes=1, seed=0, wdtype=None, fused=True):
    gen = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen).to(dtype).cuda()
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    rot = D if rot is None else rot
    angle = torch.rand(max_pos, rot // 2, generator=gen, dtype=torch.float64) * 20 - 10
    table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    shape = (T,) if n_axes == 1 else (n_axes, T)
    pos = torch.randint(0, max_pos, shape, generator=gen).int().cuda()
    w = [(1 + 0.3 * torch.randn(D, generator=gen)).to(wdtype or dtype).cuda() for _ in range(2)]
    return q, k, v, table, pos, w[0], w[1]


SHAPES = [
    # T, Hq, Hkv, D, rot
    (1, 1, 1, 64, 64), (5, 4, 2, 64, 64), (3, 3, 1, 128, 128), (17, 32, 8, 128, 128), (33, 24, 2, 256, 256),
    (7, 40, 40, 64, 32), (65, 5, 5, 128, 16), (9, 24, 2, 256, 192), (13, 6, 3, 128, 112), (2, 64, 8, 128, 96),
    (700, 13, 1, 64, 48), (1000, 32, 8, 128, 128),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "next"])
def test_dense(g, shape, dtype, interleaved):
    T, Hq, Hkv, D, rot = shape
    q, k, v, table, pos, qw, kw = inputs(T, Hq, Hkv, D, dtype, rot)
    oq, ok = g.attn_qk_norm_rope(q, k, table, pos, qw, kw, interleaved=interleaved)
    for o, x, w in ((oq, q, qw), (ok, k, kw)):
        assert o.shape == x.shape and o.dtype == dtype and o.is_contiguous()
        close16(o, *reference(x, w, table, pos, interleaved))


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "next"])
@pytest.mark.parametrize("n_axes", [2, 3, 4])
@pytest.mark.parametrize("pattern", ["cycle", "sections"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 96), (256, 256)])
def test_axes(g, interleaved, n_axes, pattern, D, rot):
    q, k, v, table, pos, qw, kw = inputs(21, 6, 2, D, rot=rot, n_axes=n_axes)
    n = rot // 2
    axes = [j % n_axes for j in range(n)] if pattern == "cycle" else [min(j * n_axes // n, n_axes - 1) for j in range(n)]
    oq, ok = g.attn_qk_norm_rope(q, k, table, pos, qw, kw, interleaved=interleaved, axes=axes)
    close16(oq, *reference(q, qw, table, pos, interleaved, axes))
    close16(ok, *reference(k, kw, table, pos, interleaved, axes))


def test_norm_or_rotation_alone_and_float32_weights(g):
    q, k, v, table, pos, qw, kw = inputs(19, 8, 2, 128, wdtype=torch.float32)
    oq, ok = g.attn_qk_norm_rope(q, k, table, pos, qw, kw, eps=0.25)
    close16(oq, *reference(q, qw, table, pos, eps=0.25))
    close16(ok, *reference(k, kw, table, pos, eps=0.25))
    oq, ok = g.attn_qk_norm_rope(q, k, None, None, qw, None)                 # norm of q only, no rotation
    close16(oq, *reference(q, qw, None, None))
    assert torch.equal(ok, k)
    oq, ok = g.attn_qk_norm_rope(q, k, table, pos, None, kw)                 # rotation, norm of k only
    close16(oq, *reference(q, None, table, pos))
    close16(ok, *reference(k, kw, table, pos))


def test_layouts_and_in_place(g):
    T, D = 24, 128
    q, k, v, table, pos, qw, kw = inputs(T, 8, 2, D)
    want = g.attn_qk_norm_rope(q, k, table, pos, qw, kw)
    assert torch.equal(g.attn_qk_norm_rope(q.contiguous(), k.contiguous(), table, pos, qw, kw)[0], want[0])
    # [B, S, H, D], heads outermost, odd strides (copied), a broadcast row
    four = g.attn_qk_norm_rope(q.view(4, 6, 8, D), k.view(4, 6, 2, D), table, pos.view(4, 6), qw, kw)
    assert four[0].shape == (4, 6, 8, D) and torch.equal(four[0].view(T, 8, D), want[0])
    assert torch.equal(four[1].view(T, 2, D), want[1])
    outer = q.transpose(0, 1).contiguous().transpose(0, 1)
    odd = torch.zeros(T, 8, D + 4, dtype=q.dtype, device="cuda")[..., :D].copy_(q)
    unaligned = torch.zeros(T * 8 * D + 1, dtype=q.dtype, device="cuda")[1:].view(T, 8, D).copy_(q)
    for x in (outer, odd, unaligned):
        assert torch.equal(g.attn_qk_norm_rope(x, k, table, pos, qw, kw)[0], want[0])
    one = q[:1].expand(T, 8, D)
    close16(g.attn_qk_norm_rope(one, k, table, pos, qw, kw)[0], *reference(one, qw, table, pos))
    step = torch.randn(3, 1, 8, D, device="cuda").bfloat16()[:, ::1]
    sk = step[:, :, :2]
    o = g.attn_qk_norm_rope(step, sk, table, pos[:3].view(3, 1), qw, kw)
    close16(o[0].view(3, 8, D), *reference(step.reshape(3, 8, D), qw, table, pos[:3]))
    close16(o[1].view(3, 2, D), *reference(sk.reshape(3, 2, D), kw, table, pos[:3]))
    # in place, and into given buffers
    a, b = q.contiguous(), k.contiguous()
    got = g.attn_qk_norm_rope(a, b, table, pos, qw, kw, out=(a, b))
    assert got[0].data_ptr() == a.data_ptr() and torch.equal(a, want[0]) and torch.equal(b, want[1])
    empty = g.attn_qk_norm_rope(q[:0], k[:0], table, pos[:0], qw, kw)
    assert empty[0].shape == (0, 8, D)


def test_positions_out_of_range_read_the_nearest_row(g):
    q, k, v, table, pos, qw, kw = inputs(6, 4, 4, 64)
    pos = torch.tensor([-1, 0, 499, 500, 2**31 - 1, -2**31], dtype=torch.int32, device="cuda")
    oq, _ = g.attn_qk_norm_rope(q, k, table, pos, qw, kw)
    close16(oq, *reference(q, qw, table, pos))


def test_special_values_stay_in_their_row(g):
    """Zeros, huge and tiny rows; infinities and NaN in one head leave the others alone."""
    q, k, v, table, pos, qw, kw = inputs(8, 4, 2, 128, rot=64)
    q = q.contiguous()
    q[0, 0] = 0
    q[1, 0] = 1e18
    q[2, 0] = 1e-18
    oq, _ = g.attn_qk_norm_rope(q, k, table, pos, qw, kw)
    close16(oq, *reference(q, qw, table, pos))
    bad = q.clone()
    bad[3, 1, 5] = float("nan")
    bad[4, 2, 100] = float("inf")
    ob, _ = g.attn_qk_norm_rope(bad, k, table, pos, qw, kw)
    assert bool(ob[3, 1].isnan().all())
    ob[3, 1], ob[4, 2] = oq[3, 1], oq[4, 2]
    assert torch.equal(ob, oq)
    ob, _ = g.attn_qk_norm_rope(bad, k, table, pos, None, None)          # no norm: a value meets its mate only
    assert ob[4, 2, 100] == float("inf") and int((~ob[4, 2].isfinite()).sum()) == 1
    assert int(ob[3, 1].isnan().sum()) == 2 and bool(ob[3, 1, 5].isnan()) and bool(ob[3, 1, 37].isnan())


# ---------------------------------------------------------------- into paged caches

def slot_map(T, num_pages, ps, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randperm(num_pages * ps, generator=gen)[:T].int().cuda()


PAGED = [
    # T, Hq, Hkv, D, page_size, num_pages
    (1, 4, 1, 64, 1, 1), (6, 32, 8, 128, 64, 3), (61, 32, 8, 128, 24, 4), (40, 24, 2, 256, 16, 9), (333, 6, 3, 64, 7, 60),
    (900, 32, 8, 128, 16, 70),
]


@pytest.mark.parametrize("shape", PAGED, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_paged_16bit(g, shape, dtype):
    T, Hq, Hkv, D, ps, pages = shape
    q, k, v, table, pos, qw, kw = inputs(T, Hq, Hkv, D, dtype)
    slots = slot_map(T, pages, ps)
    kc = torch.full((pages, ps, Hkv, D), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    oq = g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, kc, vc, qw, kw)
    dq, dk = g.attn_qk_norm_rope(q, k, table, pos, qw, kw)
    at = slots.long()
    assert torch.equal(oq, dq)
    assert torch.equal(kc.view(-1, Hkv, D)[at], dk) and torch.equal(vc.view(-1, Hkv, D)[at], v)
    rest = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool(kc.view(-1, Hkv, D)[rest].isnan().all()) and bool(vc.view(-1, Hkv, D)[rest].isnan().all())


@pytest.mark.parametrize("shape", PAGED, ids=str)
@pytest.mark.parametrize("as_bytes", [False, True], ids=["fp8", "bytes"])
def test_paged_e4m3(g, shape, as_bytes):
    T, Hq, Hkv, D, ps, pages = shape
    q, k, v, table, pos, qw, kw = inputs(T, Hq, Hkv, D)
    gen = torch.Generator().manual_seed(3)
    B = 5
    ks = (0.001 + 0.05 * torch.rand(B, Hkv, generator=gen)).cuda()       # from saturating to coarse
    vs = (0.001 + 0.05 * torch.rand(B, Hkv, generator=gen)).cuda()
    req = torch.randint(0, B, (T,), generator=gen).int().cuda()
    slots = slot_map(T, pages, ps)
    kc = torch.full((pages, ps, Hkv, D), 0x5A, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    c = (lambda t: t) if as_bytes else (lambda t: t.view(torch.float8_e4m3fn))
    oq = g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, c(kc), c(vc), qw, kw, k_scale=ks, v_scale=vs,
                                   requests=req)
    assert torch.equal(oq, g.attn_qk_norm_rope(q, k, table, pos, qw, kw)[0])
    at, r = slots.long(), req.long()
    y, mag = reference(k, kw, table, pos)
    s = ks[r].double().cpu()[..., None]
    close8(kc.view(-1, Hkv, D)[at], y / s, mag / s)
    want = (v.float().cpu() / vs[r].cpu()[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)     # one fp32 division
    assert torch.equal(vc.view(-1, Hkv, D)[at].cpu(), want.view(torch.uint8))
    rest = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((kc.view(-1, Hkv, D)[rest] == 0x5A).all()) and bool((vc.view(-1, Hkv, D)[rest] == 0x5A).all())
    # unit scales, one side only
    g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, c(kc), c(vc), qw, kw, v_scale=vs, requests=req)
    close8(kc.view(-1, Hkv, D)[at], y, mag)
    g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, c(kc), c(vc), qw, kw)
    assert torch.equal(vc.view(-1, Hkv, D)[at].cpu(), v.float().cpu().to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_rows_past_4_gib_of_a_cache(g, e4m3):
    """Slots whose rows lie behind byte 2^32 of the caches; the same results as in a small pool."""
    T, Hq, Hkv, D, ps, pages = 37, 8, 8, 128, 16, 5
    q, k, v, table, pos, qw, kw = inputs(T, Hq, Hkv, D)
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    first = (1 << 32) // (ps * Hkv * D * dt.itemsize) + 1      # first page wholly past it
    slots = slot_map(T, pages, ps)
    small = [torch.zeros(pages, ps, Hkv, D, dtype=dt, device="cuda") for _ in range(2)]
    large = [torch.zeros(first + pages, ps, Hkv, D, dtype=dt, device="cuda") for _ in range(2)]
    a = g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, *small, qw, kw)
    b = g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots + first * ps, *large, qw, kw)
    assert torch.equal(a, b)
    for s, l in zip(small, large):
        assert torch.equal(l[first:].view(torch.uint8), s.view(torch.uint8))
        assert not bool(l[:first].view(torch.int32).any())


def test_every_e4m3_rounding(g):
    """All float16 values: nearest even, saturation, subnormals, NaN."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16)
    v = bits.view(128, 8, 64).cuda()
    T, Hkv, D = v.shape
    z = torch.zeros_like(v)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kc = torch.zeros(2, 64, Hkv, D, dtype=torch.float8_e4m3fn, device="cuda")
    vc = kc.clone()
    g.attn_qk_norm_rope_paged(z, z, v, None, None, slots, kc, vc)
    got = vc.view(-1).float().cpu()
    x = bits.float()
    assert torch.equal(got.isnan(), x.isnan())
    fine = ~x.isnan()
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert torch.equal(got[fine], want[fine])


def test_padding_rows_are_left_alone(g):
    T, Hq, Hkv, D, ps, pages = 70, 8, 2, 128, 16, 4
    q, k, v, table, pos, qw, kw = inputs(T, Hq, Hkv, D)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[:50] = slot_map(50, pages, ps)
    slots[50:53] = torch.tensor([pages * ps, 2**31 - 1, -2**31], dtype=torch.int32)
    pos[50:] = -12345
    for x in (q, k, v):
        x[50:] = float("nan")
    out = torch.full_like(q, 7.0)
    kc = torch.zeros(pages, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    got = g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, kc, vc, qw, kw, out=out)
    assert got.data_ptr() == out.data_ptr() and bool((out[50:] == 7).all())
    close16(out[:50], *reference(q[:50], qw, table, pos[:50]))
    assert bool(kc.isfinite().all()) and bool(vc.isfinite().all())
    # a request id outside the scales is padding too
    req = torch.zeros(T, dtype=torch.int32, device="cuda")
    req[:3] = torch.tensor([-1, 2, 2**31 - 1], dtype=torch.int32)
    s = torch.ones(2, Hkv, device="cuda")
    k8 = torch.zeros(pages, ps, Hkv, D, dtype=torch.float8_e4m3fn, device="cuda")
    out.fill_(7.0)
    g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, k8, k8.clone(), qw, kw, k_scale=s, requests=req, out=out)
    assert bool((out[:3] == 7).all()) and bool((out[50:] == 7).all()) and not bool((out[3:50] == 7).all())
    assert bool((k8.view(-1, Hkv, D)[slots[:3].long()].float() == 0).all())


def test_other_stream_and_graph_replay(g):
    T, Hq, Hkv, D, ps, pages = 48, 8, 2, 128, 16, 6
    q, k, v, table, pos, qw, kw = inputs(T, Hq, Hkv, D)
    slots = slot_map(T, pages, ps)
    kc = torch.zeros(pages, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc, out = kc.clone(), torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call = lambda: g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, kc, vc, qw, kw, out=out)  # noqa: E731
    with torch.cuda.stream(stream):
        call()
    torch.cuda.current_stream().wait_stream(stream)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    pos.copy_((pos + 17) % 500)
    slots.copy_(slot_map(T, pages, ps, seed=9))
    kc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(first, out)
    close16(out, *reference(q, qw, table, pos))
    close16(kc.view(-1, Hkv, D)[slots.long()], *reference(k, kw, table, pos))


def test_refusals(g):
    T, D = 6, 128
    q, k, v, table, pos, qw, kw = inputs(T, 8, 2, D)
    kc = torch.zeros(2, 16, 2, D, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    slots = slot_map(T, 2, 16)
    s = torch.ones(1, 2, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k=k[:3]), dict(k=k.half()), dict(q=q[..., :96], k=k[..., :96]),
                dict(cos_sin=table.half()), dict(cos_sin=table[:, :24]), dict(cos_sin=None), dict(positions=None),
                dict(positions=pos.long()), dict(positions=pos[:3]), dict(q_weight=qw[:64]), dict(k_weight=kw.half()),
                dict(q_weight=qw.float()), dict(eps=-1.0), dict(axes=[0] * 63), dict(axes=[0] * 64),
                dict(axes=[1] * 64, positions=pos[None]), dict(axes=[4] * 64, positions=pos[None].repeat(5, 1)),
                dict(out=(torch.empty_like(k), torch.empty_like(k))),
                dict(out=(torch.empty(T, 8, 2 * D, dtype=q.dtype, device="cuda")[..., :D], torch.empty_like(k)))):
        with pytest.raises(ValueError):
            g.attn_qk_norm_rope(**{**dict(q=q, k=k, cos_sin=table, positions=pos, q_weight=qw, k_weight=kw), **bad})
    qc, kk = q.contiguous(), k.contiguous()
    for bad in (dict(q=qc, out=(qc[:1].expand(T, 8, D), torch.empty_like(kk))), dict(k=kk, out=(torch.empty_like(qc), qc[:, :2])),
                dict(q=kk, k=kk, out=(kk, torch.empty_like(kk)))):
        with pytest.raises(ValueError):
            g.attn_qk_norm_rope(**{**dict(q=q, k=k, cos_sin=table, positions=pos, q_weight=qw, k_weight=kw), **bad})
    for bad in (dict(v=v[:3]), dict(v=v[:, :1]), dict(slots=slots.long()), dict(slots=slots[:3]),
                dict(k_cache=kc.half()), dict(k_cache=kc[:, ::2]), dict(v_cache=vc[:1]), dict(k_scale=s),
                dict(requests=slots), dict(k_cache=kc.cpu()),
                dict(k_cache=torch.zeros(2, 16, 2, D, dtype=torch.uint8, device="cuda")),
                dict(out=torch.empty(T, 8, D, device="cuda"))):
        with pytest.raises(ValueError):
            g.attn_qk_norm_rope_paged(**{**dict(q=q, k=k, v=v, cos_sin=table, positions=pos, slots=slots, k_cache=kc,
                                                v_cache=vc, q_weight=qw, k_weight=kw), **bad})
    k8 = torch.zeros(2, 16, 2, D, dtype=torch.float8_e4m3fn, device="cuda")
    for bad in (dict(k_scale=s), dict(k_scale=s.double(), requests=slots), dict(k_scale=s[:, :1], requests=slots),
                dict(k_scale=s, v_scale=torch.ones(2, 2, device="cuda"), requests=slots)):
        with pytest.raises(ValueError):
            g.attn_qk_norm_rope_paged(q, k, v, table, pos, slots, k8, k8.clone(), qw, kw, **bad)


def test_extreme_scales(g):
    """Scales at the ends of the normal and subnormal range divide like any other."""
    T, Hkv, D = 4, 1, 64
    v = torch.tensor([0.0, 1.0, -3.5, 1e-30, 3e38, -1e20, 7e-39, 240.0], dtype=torch.bfloat16).repeat(T * Hkv * D // 8)
    v = v.view(T, Hkv, D).cuda()
    z = torch.zeros_like(v)
    vs = torch.tensor([[1e-45], [2.0 ** -126], [2.0 ** 127], [1e30]], device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kc = torch.zeros(1, T, Hkv, D, dtype=torch.float8_e4m3fn, device="cuda")
    vc = kc.clone()
    g.attn_qk_norm_rope_paged(z, z, v, None, None, slots, kc, vc, v_scale=vs, requests=slots)
    want = (v.float().cpu() / vs.cpu()[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(vc.view(T, Hkv, D).cpu().float(), want.float())


@pytest.mark.parametrize("n_axes", [2, 3])
def test_axes_of_every_integer_type(g, n_axes):
    """axes as a list, a tuple, bytes, a NumPy array of any integer type, a tensor: the same result."""
    np = pytest.importorskip("numpy")
    q, k, v, table, pos, qw, kw = inputs(9, 6, 2, 128, n_axes=n_axes)
    axes = [(j * j + 1) % n_axes for j in range(64)]
    want = g.attn_qk_norm_rope(q, k, table, pos, qw, kw, axes=axes)
    close16(want[0], *reference(q, qw, table, pos, axes=axes))
    forms = [tuple(axes), bytes(axes), torch.tensor(axes), torch.tensor(axes, dtype=torch.int32).cuda()]
    forms += [np.array(axes, dtype=t) for t in ("int8", "uint8", "int16", "int32", "uint32", "int64", ">i4")]
    forms += [np.array([axes, axes], dtype="int64").T[:, 0], [np.int64(a) for a in axes]]
    for form in forms:
        for o, w in zip(g.attn_qk_norm_rope(q, k, table, pos, qw, kw, axes=form), want):
            assert torch.equal(o, w), type(form)
    for bad in ([0.0] * 64, np.zeros(64), np.zeros((64, 2), dtype="int64"), torch.zeros(64), ["0"] * 64, [-1] * 64,
                [n_axes] * 64, [256] * 64, np.full(64, 256), [0] * 63, 7):
        with pytest.raises(ValueError):
            g.attn_qk_norm_rope(q, k, table, pos, qw, kw, axes=bad)
