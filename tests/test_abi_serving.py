"""Host-side argument checks of the serving-step entry points (slot maps, norm
and rotation, packed queries over e4m3 caches), on the CPU: every refusal comes
back before anything reaches a GPU."""
import ctypes

import pytest
import torch

from gqa_softmax_attention_gb300 import _lib, api, build, rope_table

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
P = ctypes.c_void_p
A16, A16b, A16c = P(1 << 20), P(2 << 20), P(3 << 20)   # aligned stand-in pointers; never dereferenced
MIS = P((1 << 20) + 2)                                  # aligned for no type here


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def at(k):
    return P((4 << 20) + (k << 12))                     # stand-in buffers of 4 KB


def slots(lib, past=at(0), new=at(1), table=at(2), free=at(3), start=None, B=2, max_pages=4, ps=16, pages=10, n_free=3,
          T=8, cu=at(4), lens=at(5), slot=at(6), pos=at(7), req=at(8), counts=at(9)):
    return lib.attn_paged_slots(past, new, table, free, start, B, max_pages, ps, pages, n_free, T, cu, lens, slot, pos,
                                req, counts, None)


def test_paged_slots_argument_checks(lib):
    for bad in (dict(B=0), dict(B=-1), dict(max_pages=0), dict(ps=0), dict(pages=-1), dict(n_free=-1), dict(T=-1),
                dict(past=None), dict(new=None), dict(table=None), dict(free=None), dict(cu=None), dict(lens=None),
                dict(slot=None), dict(pos=None), dict(req=None), dict(counts=None), dict(max_pages=1 << 26),
                dict(T=1 << 30), dict(start=at(9)), dict(start=P(at(9).value + 8)), dict(lens=at(0)), dict(counts=at(1)),
                dict(cu=P(at(1).value + 4)), dict(slot=at(3)), dict(req=P(at(2).value + 28)), dict(past=at(2))):
        assert slots(lib, **bad) == INVALID, bad
    assert slots(lib, pages=1 << 27) == UNSUPPORTED
    for name in ("past", "new", "table", "free", "start", "cu", "lens", "slot", "pos", "req", "counts"):
        assert slots(lib, **{name: MIS}) == MISALIGNED, name


def test_paged_slots_refuses_outputs_over_each_other(lib):
    outs = dict(cu=at(4), lens=at(5), slot=at(6), pos=at(7), req=at(8), counts=at(9))      # B = 2, T = 8
    for a in outs:
        for b in outs:
            if a != b:
                assert slots(lib, **{a: outs[b]}) == INVALID, (a, b)
    assert slots(lib, pos=P(at(6).value + 28)) == INVALID          # the last of the eight slots
    assert slots(lib, lens=P(at(4).value + 8)) == INVALID          # the last of the three offsets


def rows(data=A16, token=1024, head=128):
    return _lib.HeadRows(data, token, head)


def rope(cos=A16, pos=A16, max_pos=100, rot=64, inter=0, n_axes=1, axis=None):
    return _lib.Rope(cos, pos, max_pos, rot, inter, n_axes, axis)


def dense(lib, q=None, k=None, qw=None, kw=None, eps=1e-6, r=None, qo=A16b, ko=A16c, T=4, Hq=8, Hkv=2, D=128, dtype=0):
    q, k, r = q or rows(), k or rows(), r or rope()
    return lib.attn_qk_norm_rope(ctypes.byref(q), ctypes.byref(k), qw, kw, 0, eps, ctypes.byref(r), qo, ko, T, Hq, Hkv,
                                 D, dtype, None)


def paged(lib, q=None, k=None, v=None, r=None, qo=A16b, slot=A16, kc=A16b, vc=A16c, e4m3=0, ks=None, vs=None, req=None,
          B=0, T=4, Hq=8, Hkv=2, D=128, pages=10, ps=16, dtype=0):
    q, k, v, r = q or rows(), k or rows(), v or rows(), r or rope()
    return lib.attn_qk_norm_rope_paged(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), None, None, 0, 1e-6,
                                       ctypes.byref(r), qo, slot, kc, vc, e4m3, ks, vs, req, B, T, Hq, Hkv, D, pages,
                                       ps, dtype, None)


@pytest.mark.parametrize("call", [dense, paged])
def test_qk_norm_rope_argument_checks(lib, call):
    for bad in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(dtype=2), dict(qo=None), dict(q=rows(data=None)),
                dict(k=rows(data=None)), dict(q=rows(token=-8)), dict(k=rows(head=-8)), dict(r=rope(rot=-16)),
                dict(r=rope(rot=144)), dict(r=rope(max_pos=0)), dict(r=rope(n_axes=0)), dict(r=rope(n_axes=5)),
                dict(r=rope(cos=None)), dict(r=rope(pos=None)), dict(r=rope(n_axes=2)),
                dict(r=rope(n_axes=2, axis=bytes([0] * 31 + [2])))):
        assert call(lib, **bad) == INVALID, bad
    for bad in (dict(D=96), dict(D=512), dict(r=rope(rot=24)), dict(T=(1 << 30) - 1)):
        assert call(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=rows(data=MIS)), dict(k=rows(token=1028)), dict(q=rows(head=4)), dict(qo=MIS),
                dict(r=rope(cos=MIS)), dict(r=rope(pos=MIS))):
        assert call(lib, **bad) == MISALIGNED, bad
    assert call(lib, T=0, q=rows(data=None), k=rows(data=None), qo=None) == OK


def test_qk_norm_rope_refuses_overlaps(lib):
    """Outputs may be the very input rows; nothing else may overlap (T = 4: 8 KB of q, 2 KB of k)."""
    q, k, v = rows(at(0)), rows(at(8), 256), rows(at(16), 256)
    far, far2 = at(64), at(128)
    for bad in (dict(q=q, k=k, qo=P(at(0).value + 16)), dict(q=q, k=k, qo=at(8)), dict(q=q, k=k, ko=at(0)),
                dict(q=q, k=k, qo=far, ko=far), dict(q=rows(at(0), 1280), k=k, qo=at(0))):
        assert dense(lib, **{**dict(ko=far2), **bad}) == INVALID, bad
    for bad in (dict(qo=at(16)), dict(kc=at(16)), dict(vc=at(0)), dict(kc=at(200), vc=at(200)), dict(kc=at(64))):
        assert paged(lib, **{**dict(q=q, k=k, v=v, qo=far, kc=at(200), vc=at(400)), **bad}) == INVALID, bad


def test_qk_norm_rope_own_checks(lib):
    assert dense(lib, eps=-1.0) == INVALID
    assert dense(lib, eps=float("nan")) == INVALID
    assert dense(lib, ko=None) == INVALID
    assert dense(lib, ko=MIS) == MISALIGNED
    assert dense(lib, qw=MIS) == MISALIGNED
    assert dense(lib, kw=MIS) == MISALIGNED
    assert paged(lib, ps=0) == INVALID
    assert paged(lib, pages=-1) == INVALID
    assert paged(lib, pages=1 << 27) == UNSUPPORTED
    assert paged(lib, slot=None) == INVALID
    assert paged(lib, kc=None) == INVALID
    assert paged(lib, ks=A16, req=A16, B=1) == INVALID               # scales without e4m3 caches
    assert paged(lib, ks=A16, e4m3=1, req=A16, B=0) == INVALID
    assert paged(lib, vs=A16, e4m3=1, req=None, B=2) == INVALID
    assert paged(lib, v=rows(data=MIS)) == MISALIGNED
    assert paged(lib, v=rows(token=12)) == MISALIGNED
    assert paged(lib, v=rows(head=-8)) == INVALID
    for name in ("slot", "kc", "vc"):
        assert paged(lib, **{name: MIS}) == MISALIGNED, name
    assert paged(lib, e4m3=1, ks=MIS, req=A16, B=1) == MISALIGNED
    assert paged(lib, e4m3=1, ks=A16, req=MIS, B=1) == MISALIGNED


def packed(lib, q=A16, kc=A16, ks=None, vs=None, cu=A16, lens=A16, B=2, total_q=8, Hq=8, Hkv=2, D=128, ps=16, pages=4,
           max_pages=2, ws=A16, ws_bytes=1 << 20):
    return lib.attn_fwd_paged_fp8kv(q, kc, A16, ks, vs, cu, lens, A16, ps, A16b, None, B, total_q, Hq, Hkv, D, pages,
                                    max_pages, 1, 0.125, None, ws, ws_bytes, None)


def test_fwd_paged_fp8kv_argument_checks(lib):
    for bad in (dict(B=0), dict(total_q=-1), dict(Hq=6, Hkv=4), dict(ps=0), dict(pages=0), dict(max_pages=0),
                dict(kc=None), dict(cu=None), dict(lens=None), dict(q=None)):
        assert packed(lib, **bad) == INVALID, bad
    for bad in (dict(D=64), dict(D=96), dict(Hq=512, Hkv=2), dict(pages=1 << 27)):
        assert packed(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(kc=MIS), dict(ks=MIS), dict(vs=MIS), dict(cu=MIS), dict(lens=MIS)):
        assert packed(lib, **bad) == MISALIGNED, bad
    assert packed(lib, ws=None) == WORKSPACE
    assert packed(lib, ws_bytes=16) == WORKSPACE
    assert packed(lib, total_q=0) == OK


def test_python_refuses_cpu_tensors():
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    t = i.view(2, 2)
    with pytest.raises(ValueError):
        api.attn_paged_slots(i, i, t, i, 16, 4, 8)
    with pytest.raises(ValueError):
        api.attn_qk_norm_rope(x, x, None, None)
    with pytest.raises(ValueError):
        api.attn_qk_norm_rope_paged(x, x, x, None, None, i, x, x)
    c = torch.zeros(2, 16, 8, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        api.attn_fwd_paged_fp8kv(x, c, c, None, None, i, i[:3], t)


def test_rope_table_matches_its_formula():
    t = rope_table(1000, 48, base=1e4, device="cpu").double()
    p, j = 999, 7
    angle = torch.tensor(p, dtype=torch.float64) * 1e4 ** (-2 * j / 48)
    # one rounding to float32
    assert abs(t[p, j] - angle.cos()) <= 2.0 ** -24
    assert abs(t[p, 24 + j] - angle.sin()) <= 2.0 ** -24
    assert t.shape == (1000, 48)
    with pytest.raises(ValueError):
        rope_table(10, 7)


def test_fp8kv_workspace_size_of_invalid_sizes(lib):
    size = lambda **k: lib.attn_paged_fp8kv_workspace_size(*{**dict(B=2, total_q=8, Hq=8, Hkv=2, D=128, page_size=16,  # noqa: E731
                                                                    max_pages=400), **k}.values())
    assert size() >= lib.attn_paged_workspace_size(2, 8, 8, 2, 128, 16, 400) > 0      # and room for key parts, on a GPU
    assert size(D=256) > 0 and size(max_pages=2) > 0
    for bad in (dict(D=64), dict(D=96), dict(D=0), dict(D=-1), dict(D=-1000), dict(D=512), dict(page_size=0),
                dict(page_size=-16), dict(max_pages=0), dict(max_pages=-3), dict(page_size=-16, max_pages=-400),
                dict(max_pages=1 << 26), dict(total_q=-1), dict(total_q=1 << 30), dict(B=0), dict(Hq=0), dict(Hkv=0),
                dict(Hq=6, Hkv=4), dict(Hq=258, Hkv=2)):
        assert size(**bad) == 0, bad


def test_fwd_paged_fp8kv_refuses_overlaps(lib):
    """Nothing written (o, lse, the workspace) may overlap what is read or another of them."""
    MB = 1 << 20
    place = {n: (16 + 16 * i) * MB for i, n in enumerate(("q", "kc", "vc", "ks", "vs", "cu", "lens", "table", "o", "lse",
                                                          "ws", "sinks"))}
    B, T, Hq, Hkv, D, ps, pages, max_pages = 3, 40, 8, 2, 128, 16, 50, 20
    size = lib.attn_paged_fp8kv_workspace_size(B, T, Hq, Hkv, D, ps, max_pages)
    bytes_of = dict(q=T * Hq * D * 2, kc=pages * ps * Hkv * D, vc=pages * ps * Hkv * D, ks=B * Hkv * 4, vs=B * Hkv * 4,
                    cu=(B + 1) * 4, lens=B * 4, table=B * max_pages * 4, sinks=Hq * 4, o=T * Hq * D * 2, lse=T * Hq * 4,
                    ws=size)

    def call(**moved):
        p = {n: P(a) for n, a in {**place, **moved}.items()}
        opt = _lib.Options(-1, -1, 0.0, p["sinks"], 0)
        return lib.attn_fwd_paged_fp8kv(p["q"], p["kc"], p["vc"], p["ks"], p["vs"], p["cu"], p["lens"], p["table"], ps,
                                        p["o"], p["lse"], B, T, Hq, Hkv, D, pages, max_pages, 1, 0.125,
                                        ctypes.byref(opt), p["ws"], size + (1 << 30), None)

    for w in ("o", "lse", "ws"):
        for r in bytes_of:
            if r == w:
                continue
            up = 256 * ((bytes_of[r] - 1) // 256)                      # the last 256 bytes of the other
            assert call(**{w: place[r]}) == INVALID, (w, r)
            assert call(**{w: place[r] + up}) == INVALID, (w, r)
            down = 256 * ((bytes_of[w] - 1) // 256)
            assert call(**{w: place[r] - down}) == INVALID, (w, r)
