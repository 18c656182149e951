"""float16 prefill with scores that rise far past a row's standing reference
maximum, up to 32 binades from one key tile to the next: a weight formed
against the old reference (2^16 and more) is no float16, so the row has to
take a new one.  Against the FP64 oracle, in the usual tolerances."""
import math

import pytest
import torch

import oracle

from parity import compare

pytestmark = pytest.mark.gpu
LN2 = math.log(2.0)


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gqa_softmax_attention_gb300 import build
    build.build()
    import gqa_softmax_attention_gb300 as m
    yield m
    m.gqa_device_error()


def rising(Sq, Skv, Hq, Hkv, D, seed):
    """q, k, v of one request: in query head h the scores (log2 units, scale ln 2)
    rise by 9 + 3 h at every 128th key, next to noise of about 2 (products of small
    integers and halves, exact in float16)."""
    gen = torch.Generator().manual_seed(seed)
    q = torch.randint(-2, 3, (Sq, Hq, D), generator=gen).float() / 4
    k = torch.randint(-2, 3, (Skv, Hkv, D), generator=gen).float() / 4
    q[..., 0] = (9 + 3 * torch.arange(Hq)).float()
    k[..., 0] = (torch.arange(Skv) // 128)[:, None].float()
    return q.half(), k.half(), torch.randn(Skv, Hkv, D, generator=gen).half()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_dense(g, D, causal):
    q, k, v = (x[None] for x in rising(200, 900, 8, 2, D, D))
    o, lse = g.attention(q.cuda(), k.cuda(), v.cuda(), causal=causal, scale=LN2)
    torch.cuda.synchronize()
    ro, rl = oracle.attn_dense(q, k, v, causal=causal, scale=LN2)
    compare(o, lse, ro, rl, "dense")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_packed(g, D, causal):
    parts = [rising(n, L, 8, 2, D, n) for n, L in ((150, 700), (3, 1000), (64, 300))]
    q, k, v = (torch.cat(x) for x in zip(*parts))
    cq = torch.tensor([0, 150, 153, 217], dtype=torch.int32)
    ck = torch.tensor([0, 700, 1700, 2000], dtype=torch.int32)
    o, lse = g.varlen(q.cuda(), k.cuda(), v.cuda(), cq.cuda(), ck.cuda(), causal=causal, scale=LN2)
    torch.cuda.synchronize()
    ro, rl = oracle.attn_varlen(q, k, v, cq, ck, causal=causal, scale=LN2)
    compare(o, lse, ro, rl, "packed")
