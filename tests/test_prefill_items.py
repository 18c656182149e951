"""Items of the two-tile prefill kernel whose query tiles see no key, alone and
among others (packed and dense calls): no wait may give up, results as ever."""
import pytest
import torch

import oracle
from gqa_softmax_attention_gb300 import workloads as W

from parity import compare

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


def again(run, times=100):
    """The result of run(), which it repeats bit by bit."""
    o, lse = run()
    for _ in range(times):
        o2, lse2 = run()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    return o.cpu(), lse.cpu()


@pytest.mark.parametrize("D", [64, 128])
def test_packed_requests_without_a_key(g, D):
    """Several items of no key in a row for every CTA, behind items that have some; pairs of
    row blocks of which either one has no key or no row."""
    ql, kl = [], []
    for i in range(400):
        ql.append((1, 33, 64, 65, 300, 7, 129)[i % 7])
        kl.append(0 if i % 3 else (40, 300, 1, 90)[i % 4])          # 300 queries over 40 or 90 keys among them
    d = W.varlen_inputs(ql, kl, 8, 4, D, seed=D)
    dev = [d[n].cuda() for n in ("q", "k", "v", "cu_seqlens_q", "cu_seqlens_kv")]
    for causal in (True, False):
        o, lse = again(lambda: g.varlen(*dev, causal=causal))
        g.gqa_device_error()
        ro, rl = oracle.attn_varlen(d["q"], d["k"], d["v"], d["cu_seqlens_q"], d["cu_seqlens_kv"], causal=causal)
        compare(o, lse, ro, rl, "causal %s" % causal)


def test_packed_call_without_any_key(g):
    ql = [5, 200, 1, 130] * 200
    d = W.varlen_inputs(ql, [0] * len(ql), 8, 4, 128, seed=1)
    dev = [d[n].cuda() for n in ("q", "k", "v", "cu_seqlens_q", "cu_seqlens_kv")]
    o, lse = again(lambda: g.varlen(*dev, causal=True))
    g.gqa_device_error()
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("D", [64, 128])
def test_dense_batches_without_a_key(g, D):
    """Half the batches padded away whole, and first row blocks before the first key."""
    B, Hq, Hkv, Sq, Skv = 6, 16, 4, 700, 300
    d = W.dense_inputs(B, Hq, Hkv, Sq, Skv, D, seed=D + 1)
    mask = torch.ones(B, Skv, dtype=torch.bool)
    mask[1::2] = False
    mask[4, 100:] = False
    q, k, v, m = (x.cuda() for x in (d["q"], d["k"], d["v"], mask))
    for causal in (True, False):
        o, lse = again(lambda: g.attention(q, k, v, causal=causal, key_padding_mask=m))
        g.gqa_device_error()
        ro, rl = oracle.attn_dense(d["q"], d["k"], d["v"], causal=causal, key_padding_mask=mask)
        compare(o, lse, ro, rl, "causal %s" % causal)
