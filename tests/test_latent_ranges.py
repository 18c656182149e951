"""Latent calls at the ends of their ranges: cache rows past 4 GiB in append and gather,
many requests in the gather, no LSE, workspaces between the plan's size and the full one."""
import ctypes

import pytest
import torch

from test_latent import C, R, ROW, SCALE, check, i32, paged_case, paged_refs, randn, sums, varlen_case, varlen_refs

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


def test_append_and_gather_far_rows(g):
    """Rows on both sides of 2^31 elements and of 4 GiB, and the pool's last one: written by the
    append, brought back by the gather."""
    gen, ps, T, H = torch.Generator().manual_seed(1), 64, 200, 3
    pages = (5 << 30) // (ps * ROW * 2)
    cache = torch.empty(pages, ps, ROW, dtype=torch.bfloat16, device="cuda")
    table = i32([[pages - 1, (1 << 31) // (ps * ROW), 0, (1 << 32) // (2 * ps * ROW) - 1, (1 << 32) // (2 * ps * ROW)]])
    t = torch.arange(T, device="cuda")
    slots = (table[0].long()[t // ps] * ps + t % ps).int()
    q, kv, packed = randn(gen, T, H, R), randn(gen, T, ROW), torch.zeros(T, ROW, dtype=torch.bfloat16, device="cuda")
    w = randn(gen, C)
    g.attn_latent_norm_rope_paged(q, kv, g.rope_table(T, R), t.int(), slots, cache, kv_weight=w, kv_out=packed)
    assert torch.equal(cache.view(-1, ROW)[slots.long()], packed) and bool(packed.any())
    assert torch.equal(g.attn_latent_gather(cache, i32([0, T]), table, T), packed)


@pytest.mark.parametrize("B", [33, 1000, 5000])
def test_gather_many_requests(g, B):
    """Requests of no row, of a few, and one that spans blocks, among thousands; the rows before the first."""
    gen, ps = torch.Generator().manual_seed(B), 16
    lens = torch.randint(0, 9, (B,), generator=gen).tolist()
    lens[B // 3], lens[B - 2] = 100, 70
    lens[B // 2:B // 2 + 12] = [0] * 12
    c = paged_case(gen, [1] * B, lens, 1, ps, torch.bfloat16)
    c["cache"].nan_to_num_(3.0)
    cu = [x + 5 for x in sums(lens)]
    out = torch.full((cu[-1] + 3, ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    g.attn_latent_gather(c["cache"], i32(cu), c["table"], cu[-1] + 3, out=out)
    b = torch.arange(B, device="cuda").repeat_interleave(i32(lens))
    t = torch.arange(sum(lens), device="cuda") - torch.tensor(sums(lens)[:-1], device="cuda")[b]
    want = c["cache"].view(-1, ROW)[c["table"].long()[b, t // ps] * ps + t % ps]
    assert torch.equal(out[5:cu[-1]], want)
    assert bool((out[:5] == 7).all()) and bool((out[cu[-1]:] == 7).all())


def test_no_lse(g):
    """lse NULL at the C entries: the same output, written and joined alike."""
    from gqa_softmax_attention_gb300 import _lib
    lib, gen = _lib.load(), torch.Generator().manual_seed(2)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    c = paged_case(gen, [1, 3], [3000, 40], 16, 64, torch.bfloat16)
    o, _ = g.attn_fwd_latent_paged(c["q"], c["cache"], c["cu"], c["lens"], c["table"], SCALE)
    o2 = torch.zeros_like(o)
    ws = torch.empty(g.attn_latent_paged_workspace_size(2, 4, 16), dtype=torch.uint8, device="cuda")
    st = lib.attn_fwd_latent_paged(c["q"].data_ptr(), c["cache"].data_ptr(), c["cu"].data_ptr(), c["lens"].data_ptr(),
                                   c["table"].data_ptr(), 64, o2.data_ptr(), None, 2, 4, 16, c["cache"].shape[0],
                                   c["table"].shape[1], 1, SCALE, 0, ws.data_ptr(), ws.numel(), stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(o, o2)
    e = varlen_case(gen, [300, 2], [5000, 900], 3, torch.bfloat16)
    rows = [_lib.HeadRows(x.data_ptr(), x.stride(0), x.stride(1) if x.dim() == 3 else 8) for x in (e["k"], e["v"], e["pe"])]
    for size in (g.attn_latent_varlen_workspace_size(2, 302, 3), g.attn_varlen_workspace_size(2, 302, 3, 3)):
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        o, _ = g.attn_fwd_latent_varlen(e["q"], e["k"], e["v"], e["pe"], e["cq"], e["ck"], workspace=ws)
        o2 = torch.zeros_like(o)
        st = lib.attn_fwd_latent_varlen(e["q"].data_ptr(), *(ctypes.byref(r) for r in rows), e["cq"].data_ptr(),
                                        e["ck"].data_ptr(), o2.data_ptr(), None, 2, 302, 5900, 3, 1, SCALE, 0,
                                        ws.data_ptr(), ws.numel(), stream)
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(o, o2)
    g.gqa_device_error()


def test_workspaces_between_the_least_and_the_full_size(g):
    """Too small for the parts: nothing is cut, and nothing is written past the plan."""
    c = varlen_case(torch.Generator().manual_seed(3), [300, 2], [5000, 900], 3, torch.bfloat16)
    least, full = g.attn_varlen_workspace_size(2, 302, 3, 3), g.attn_latent_varlen_workspace_size(2, 302, 3)
    got = {}
    for size in (least, least + 16, (least + full) // 2, full - 1, full, full + 4096):
        ws = torch.full((size + 256,), 90, dtype=torch.uint8, device="cuda")
        o, lse = g.attn_fwd_latent_varlen(c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"], workspace=ws[:size])
        torch.cuda.synchronize()
        assert bool((ws[least if size < full else full:] == 90).all())
        for b, h, rows, ref in varlen_refs(c):
            check(o[rows, h], lse[rows, h], ref, "%d bytes, request %d head %d" % (size, b, h))
        first = got.setdefault(size >= full, (o, lse))
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    with pytest.raises((ValueError, RuntimeError)):
        g.attn_fwd_latent_varlen(c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"],
                                 workspace=torch.empty(least - 1, dtype=torch.uint8, device="cuda"))
    p = paged_case(torch.Generator().manual_seed(4), [1, 1], [3000, 40], 16, 64, torch.bfloat16)
    size = g.attn_latent_paged_workspace_size(2, 2, 16)
    ws = torch.full((size + 256,), 90, dtype=torch.uint8, device="cuda")
    o, lse = g.attn_fwd_latent_paged(p["q"], p["cache"], p["cu"], p["lens"], p["table"], SCALE, workspace=ws[:size])
    torch.cuda.synchronize()
    assert bool((ws[size:] == 90).all())
    for b, rows, ref in paged_refs(p):
        check(o[rows].flatten(0, 1), lse[rows].flatten(), ref, "request %d" % b)
    with pytest.raises((ValueError, RuntimeError)):
        g.attn_fwd_latent_paged(p["q"], p["cache"], p["cu"], p["lens"], p["table"], SCALE, workspace=ws[:size - 1])
