"""Host-side argument checks of the latent attention entry points, on the CPU:
every refusal comes back before anything reaches a GPU."""
import ctypes

import pytest
import torch

from gqa_softmax_attention_gb300 import _lib, api, build

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def at(k):
    return P((4 << 20) + (k << 20))                     # stand-in buffers of 1 MB, never dereferenced


def off(p, n):
    return P(p.value + n)


def rows(data, token, head=0):
    return _lib.HeadRows(data, token, head)


def rope(cos=at(1), pos=at(2), max_pos=100, rot=64, inter=0, n_axes=1):
    return _lib.Rope(cos, pos, max_pos, rot, inter, n_axes, None)


# T = 4 tokens of 8 heads: q_pe a slice of [4, 8, 192], out one of [4, 8, 576]
def append(lib, q=rows(at(3), 1536, 192), kv=rows(at(4), 576), w=at(5), wf=0, eps=1e-6, r=rope(),
           out=rows(at(6), 4608, 576), kv_out=at(7), slots=at(8), cache=at(9), T=4, H=8, pages=10, ps=16, dtype=0):
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return lib.attn_latent_norm_rope_paged(ref(q), ref(kv), w, wf, eps, ref(r), ref(out), kv_out, slots, cache, T, H, pages,
                                           ps, dtype, None)


def test_append_argument_checks(lib):
    for bad in (dict(T=-1), dict(T=1 << 30), dict(H=0), dict(q=None), dict(kv=None), dict(r=None), dict(out=None),
                dict(pages=-1), dict(ps=0), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")), dict(r=rope(max_pos=0)),
                dict(r=rope(n_axes=2)), dict(r=rope(cos=None)), dict(r=rope(pos=None)), dict(slots=None), dict(cache=None),
                dict(q=rows(None, 1536, 192)), dict(kv=rows(None, 576)), dict(out=rows(None, 4608, 576)),
                dict(q=rows(at(3), -8, 192)), dict(kv=rows(at(4), -8)), dict(out=rows(at(6), 4608, -8)),
                dict(out=rows(at(6), 0, 576)), dict(out=rows(at(6), 4608, 56)), dict(out=rows(at(6), 64, 64))):
        assert append(lib, **bad) == INVALID, bad
    for bad in (dict(r=rope(rot=32)), dict(r=rope(rot=128)), dict(pages=1 << 27), dict(T=(1 << 30) - 1, H=8)):
        assert append(lib, **bad) == UNSUPPORTED, bad
    mis = off(at(3), 8)
    for bad in (dict(q=rows(mis, 1536, 192)), dict(kv=rows(off(at(4), 2), 576)), dict(w=off(at(5), 4)),
                dict(kv_out=off(at(7), 8)), dict(cache=off(at(9), 8)), dict(slots=off(at(8), 2)),
                dict(out=rows(off(at(6), 8), 4608, 576)), dict(q=rows(at(3), 1540, 192)), dict(q=rows(at(3), 1536, 196)),
                dict(out=rows(at(6), 4612, 576)), dict(kv=rows(at(4), 580)), dict(r=rope(cos=off(at(1), 4))),
                dict(r=rope(pos=off(at(2), 2)))):
        assert append(lib, **bad) == MISALIGNED, bad
    assert append(lib, T=0, q=rows(None, 0, 0), kv=rows(None, 0), out=rows(None, 0, 0), kv_out=None, slots=None) == 0


def test_append_refuses_overlaps(lib):
    q, kv, out = rows(at(3), 1536, 192), rows(at(4), 576), rows(at(6), 4608, 576)
    inside = lambda r, n: off(P(r.data), n)
    for bad in (dict(out=rows(inside(q, 64), 1536, 192)), dict(out=rows(inside(q, 0), 1536, 64)),
                dict(out=rows(inside(kv, 0), 4608, 576)), dict(kv_out=inside(q, 1536)), dict(kv_out=inside(out, 1024)),
                dict(kv_out=inside(kv, 16)), dict(cache=inside(q, 0)), dict(cache=inside(kv, 16)),
                dict(cache=inside(out, 0)), dict(cache=off(at(7), 16)), dict(slots=off(at(9), 64)), dict(slots=off(at(7), 64)),
                dict(r=rope(pos=inside(out, 128))), dict(w=off(at(9), 1024)), dict(r=rope(cos=off(at(7), 0))),
                # rows of one buffer that touch: 8 heads of 64 dims behind one another, and the latents from dim 448 on
                dict(q=rows(at(3), 2048, 192), out=rows(off(at(3), 1200 * 2), 2048, 64), kv=rows(off(at(3), 1648 * 2), 2048)),
                dict(kv=rows(at(4), 584), kv_out=at(4))):
        assert append(lib, **bad) == INVALID, bad


# requests: 2; 5 cached rows of 3 pages of 16
def gather(lib, cache=at(1), cu=at(2), table=at(3), ps=16, out=at(4), B=2, total=40, pages=10, max_pages=3):
    return lib.attn_latent_gather(cache, cu, table, ps, out, B, total, pages, max_pages, None)


def test_gather_argument_checks(lib):
    for bad in (dict(B=0), dict(total=-1), dict(total=1 << 30), dict(ps=0), dict(pages=-1), dict(max_pages=0), dict(cache=None),
                dict(cu=None), dict(table=None), dict(out=None), dict(max_pages=1 << 26), dict(out=off(at(1), 1152)),
                dict(cu=off(at(4), 64)), dict(table=off(at(4), 64))):
        assert gather(lib, **bad) == INVALID, bad
    assert gather(lib, pages=1 << 27) == UNSUPPORTED
    for bad in (dict(cache=off(at(1), 8)), dict(out=off(at(4), 8)), dict(cu=off(at(2), 2)), dict(table=off(at(3), 2))):
        assert gather(lib, **bad) == MISALIGNED, bad
    assert gather(lib, total=0) == 0 and gather(lib, total=0, out=None, cache=None) == 0


# 2 requests, 10 queries and 40 keys of 4 heads
def varlen(lib, q=at(1), k=rows(at(2), 1024, 256), v=rows(off(at(2), 256), 1024, 256), pe=rows(at(3), 576), cq=at(4),
           ck=at(5), o=at(6), lse=at(7), B=2, tq=10, tk=40, H=4, scale=0.07, dtype=0, ws=at(8), n=1 << 20):
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return lib.attn_fwd_latent_varlen(q, ref(k), ref(v), ref(pe), cq, ck, o, lse, B, tq, tk, H, 1, scale, dtype, ws, n, None)


def test_varlen_argument_checks(lib):
    for bad in (dict(B=0), dict(tq=-1), dict(tk=-1), dict(tk=1 << 30), dict(tq=1 << 30), dict(H=0), dict(scale=float("inf")),
                dict(dtype=2), dict(q=None), dict(k=None), dict(v=None), dict(pe=None), dict(cq=None), dict(ck=None),
                dict(o=None), dict(k=rows(None, 1024, 256)), dict(k=rows(at(2), -1024, 256)), dict(k=rows(at(2), 0, 256)),
                dict(v=rows(at(2), 1024, 0)), dict(pe=rows(at(3), 0)), dict(o=off(at(1), 64)), dict(o=off(at(2), 1024)),
                dict(lse=off(at(3), 64)), dict(ws=off(at(6), 256)), dict(lse=off(at(6), 4)), dict(ws=off(at(5), 0)),
                dict(o=off(at(8), 16))):
        assert varlen(lib, **bad) == INVALID, bad
    for bad in (dict(q=off(at(1), 8)), dict(o=off(at(6), 8)), dict(lse=off(at(7), 2)), dict(cq=off(at(4), 2)),
                dict(ck=off(at(5), 2)), dict(k=rows(off(at(2), 8), 1024, 256)), dict(v=rows(at(2), 1028, 256)),
                dict(pe=rows(at(3), 580)), dict(ws=off(at(8), 8))):
        assert varlen(lib, **bad) == MISALIGNED, bad
    need = lib.attn_varlen_workspace_size(2, 10, 4, 4)      # the least; the rest is for cut items
    assert 0 < need < lib.attn_latent_varlen_workspace_size(2, 10, 4)
    assert lib.attn_latent_varlen_workspace_size(2, 1 << 20, 128) < 1 << 20      # many rounds: nothing is cut
    assert varlen(lib, n=need - 1) == WORKSPACE and varlen(lib, ws=None) == WORKSPACE
    assert varlen(lib, tq=(1 << 30) - 1, H=400, n=1 << 40) == UNSUPPORTED
    assert varlen(lib, tq=0) == 0 and varlen(lib, tq=0, q=None, o=None, lse=None, ws=None, n=0) == 0
    for sizes in ((0, 10, 4), (2, -1, 4), (2, 10, 0), (2, 1 << 30, 4)):
        assert lib.attn_latent_varlen_workspace_size(*sizes) == 0, sizes


def paged(lib, q=at(1), cache=at(2), cq=at(3), lens=at(4), table=at(5), ps=16, o=at(6), lse=at(7), B=2, tq=10, H=4, pages=10,
          max_pages=5, scale=0.07, dtype=0, ws=at(8), n=1 << 30):
    return lib.attn_fwd_latent_paged(q, cache, cq, lens, table, ps, o, lse, B, tq, H, pages, max_pages, 1, scale, dtype, ws, n,
                                     None)


def test_paged_argument_checks(lib):
    for bad in (dict(B=0), dict(tq=-1), dict(tq=1 << 30), dict(H=0), dict(ps=0), dict(pages=0), dict(max_pages=0),
                dict(max_pages=1 << 26), dict(scale=float("nan")), dict(dtype=-1), dict(q=None), dict(cache=None), dict(cq=None),
                dict(lens=None), dict(table=None), dict(o=None)):
        assert paged(lib, **bad) == INVALID, bad
    for bad in (dict(B=16385), dict(pages=1 << 27), dict(tq=1 << 25, H=64), dict(tq=(1 << 24) - 1, H=128)):
        assert paged(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=off(at(1), 8)), dict(cache=off(at(2), 8)), dict(o=off(at(6), 8)), dict(lse=off(at(7), 2)),
                dict(cq=off(at(3), 2)), dict(lens=off(at(4), 2)), dict(table=off(at(5), 2))):
        assert paged(lib, **bad) == MISALIGNED, bad
    need = lib.attn_latent_paged_workspace_size(2, 10, 4)
    assert need > 0 and need % 256 == 0
    assert paged(lib, n=need - 1) == WORKSPACE and paged(lib, ws=None) == WORKSPACE
    assert paged(lib, ws=off(at(8), 16)) == MISALIGNED
    for bad in (dict(o=off(at(1), 64)), dict(o=off(at(2), 64)), dict(lse=off(at(5), 4)), dict(ws=at(0)), dict(lse=off(at(6), 4)),
                dict(o=off(at(8), 256)), dict(lse=off(at(3), 8)), dict(lse=at(4))):
        assert paged(lib, n=need, **bad) == INVALID, bad
    assert paged(lib, tq=0) == 0 and paged(lib, tq=0, q=None, o=None, lse=None, ws=None, n=0) == 0
    for sizes in ((0, 10, 4), (16385, 10, 4), (2, -1, 4), (2, 10, 0), (2, 1 << 25, 64), (2, 1 << 30, 1)):
        assert lib.attn_latent_paged_workspace_size(*sizes) == 0, sizes


def test_python_refusals():
    """What is not a CUDA tensor of the right kind never reaches the library."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for call in (lambda: api.attn_fwd_latent_paged(z(1, 4, 576), z(2, 16, 576), i(2), i(1), i(1, 2), 0.1),
                 lambda: api.attn_fwd_latent_varlen(z(1, 4, 192), z(1, 4, 128), z(1, 4, 128), z(1, 64), i(2), i(2)),
                 lambda: api.attn_latent_gather(z(2, 16, 576), i(2), i(1, 2), 4),
                 lambda: api.attn_latent_norm_rope_paged(z(1, 4, 64), z(1, 576), z(8, 64, d=torch.float32), i(1), i(1),
                                                         z(2, 16, 576))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
