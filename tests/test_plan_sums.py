"""Packed calls whose plan's sums pass 32 bits: the cost of one request of very many
queries, and the blocks of malformed offsets that list the same rows again and
again (cut to the list, as wrong input, with no access out of range)."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_cost_of_one_request(g):
    """140 million queries over 2^17 keys, each seeing the key at its own position: 2047 cost units
    for every 128 queries, 2.2e9 in all.  The last 2^17 queries have a position, and
    copy its value."""
    T, L = 140_000_000, 1 << 17
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    gen = torch.Generator().manual_seed(1)
    q = torch.zeros(T, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(L, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.randn(L, 1, 64, generator=gen).bfloat16().cuda()
    o, lse = g.varlen(q, k, v, i32([0, T]), i32([0, L]), causal=False, window_left=0, window_right=0)
    torch.cuda.synchronize()
    g.gqa_device_error()
    assert torch.equal(o[T - L:], v) and bool((lse[T - L:] == 0).all())
    for i in range(0, T - L, 20_000_000):
        part = slice(i, min(T - L, i + 20_000_000))
        assert not bool(o[part].any()) and bool(torch.isneginf(lse[part]).all())


def test_blocks_of_malformed_offsets(g):
    """32768 times the same 17 million rows: 2^31 blocks and more in all, of which the list
    takes what it has room for."""
    T, B = 17_000_000, 65536
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    q = torch.zeros(T, 1, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    o, lse = g.varlen(q, kv, kv, cu, torch.zeros_like(cu), causal=True)
    torch.cuda.synchronize()
    g.gqa_device_error()
    assert not bool(o[:1 << 20].any()) and bool(torch.isneginf(lse[:1 << 20]).all())
