"""Expanded latent calls whose last items are cut along the keys: results repeat bit
by bit however alike the requests are, and the rule cuts where long items come
last.  The plan's header in the workspace is [items' entries, counter, tiles of
a part, parts of a cut item]."""
import pytest
import torch

from test_latent import DT, check, i32, sums, varlen_case, varlen_refs

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


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def call(g, c, causal=True):
    """o, lse and the parts that the call's cut items went in."""
    ws = torch.zeros(g.attn_latent_varlen_workspace_size(len(c["nq"]), sum(c["nq"]), c["H"]), dtype=torch.uint8, device="cuda")
    o, lse = g.attn_fwd_latent_varlen(c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"], causal=causal, workspace=ws)
    return o, lse, int(ws[:16].view(torch.int32)[3])


def repeats(g, c, times):
    o, lse, parts = call(g, c)
    for n in range(times):
        o2, lse2, _ = call(g, c)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), "call %d differs" % n
    g.gqa_device_error()
    return o, lse, parts


def test_equal_prompts_repeat(g):
    """Three prompts of one length: their entries lie in different warps of the plan."""
    c = varlen_case(torch.Generator().manual_seed(1), [4096] * 3, [4096] * 3, 20, torch.bfloat16)
    repeats(g, c, 100)


@pytest.mark.parametrize("tail", [1, 5, 20])
def test_equal_chunks_repeat(g, tail):
    """One item a request, all of one cost, the last `tail` of them cut."""
    B = sms() + tail
    c = varlen_case(torch.Generator().manual_seed(tail), [16] * B, [1500] * B, 1, torch.bfloat16)
    o, lse, parts = repeats(g, c, 100)
    assert parts > 1
    for b, h, rows, ref in varlen_refs(c):
        if b % 7 == 0 or b > B - 30:
            check(o[rows, h], lse[rows, h], ref, "request %d" % b)


@pytest.mark.parametrize("B", [1, 33, 700, 3000])
def test_requests_of_one_cost_keep_their_order(g, B):
    """The plan's entries {request, first query, ...}: requests by cost (buckets of 16 units: two
    for each key tile of a row block, three where the block has fewer than 64 rows), those of one bucket as
    they come, each one's blocks from the last to the first."""
    gen = torch.Generator().manual_seed(B)
    kinds = [(1, 1), (300, 900), (0, 50), (40, 2000), (700, 700), (1, 0), (5, 1600)]
    pick = torch.randint(0, len(kinds), (B,), generator=gen).tolist()
    pick[B // 2:] = [pick[B // 2]] * len(pick[B // 2:])                       # half of them alike
    nq, lens = [kinds[i][0] for i in pick], [kinds[i][1] for i in pick]
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(g.attn_latent_varlen_workspace_size(B, sum(nq), 1), dtype=torch.uint8, device="cuda")
    g.attn_fwd_latent_varlen(z(sum(nq), 1, 192), z(sum(lens), 1, 128), z(sum(lens), 1, 128), z(sum(lens), 64),
                             i32(sums(nq)), i32(sums(lens)), workspace=ws)

    def cost(n, L):
        return sum(-(-max(0, min(L, q0 + rows + L - n)) // 128) * (2 if rows >= 64 else 3)
                   for q0 in range(0, n, 128) for rows in [min(128, n - q0)])
    order = sorted(range(B), key=lambda b: -min(2047, cost(nq[b], lens[b]) // 16))     # stable
    want = [[b, q0] for b in order for q0 in reversed(range(0, nq[b], 256))]
    head = ws[:16].view(torch.int32).tolist()
    assert head[0] == len(want)
    assert ws[16:16 + 32 * len(want)].view(torch.int32).view(-1, 8)[:, :2].tolist() == want


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nq,lens,last", [
    ([4096, 1], [4096, 8192], 1),              # a prompt, and one query at the end of a long context
    ([2048, 1], [2048, 4000], 1),
    ([1500, 1500, 16], [1500, 1500, 12000], 1),
])
def test_long_items_that_come_last_are_cut(g, nq, lens, last, dtype):
    """A chunk of few queries over many keys weighs less than a prompt as a whole and comes
    after it, the longest items of the call last.  As many heads as leave the tail those items and some
    short ones before them."""
    entries = sum(-(-n // 256) for n in nq)
    group = (64 << 20) // (512 * sum(lens))                   # heads whose items follow one another
    heads = [H for H in range(2, group + 1) if entries * H > sms() and last * H < entries * H % sms() <= sms() // 2]
    H = heads[0] if heads else next(H for H in range(group, 1, -1) if last * H < entries * H % sms() <= sms() // 2)
    c = varlen_case(torch.Generator().manual_seed(sum(lens)), nq, lens, H, DT[dtype])
    o, lse, parts = call(g, c)
    assert parts > 1
    for b, h, rows, ref in varlen_refs(c):
        if h in (0, H - 1):
            check(o[rows, h], lse[rows, h], ref, "request %d head %d" % (b, h))
    o2, lse2, _ = call(g, c)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("nq,lens,H,least", [([1], [9000], 1, 12), ([300], [5000], 3, 8), ([2, 1], [4000, 6000], 2, 8)])
def test_few_items_are_cut_for_idle_sms(g, nq, lens, H, least):
    """A call of fewer items than SMs takes more CTAs than it has items: as many parts as
    pay, not as many as the items' own CTAs could hold."""
    c = varlen_case(torch.Generator().manual_seed(sum(lens)), nq, lens, H, torch.bfloat16)
    o, lse, parts = repeats(g, c, 5)
    assert parts >= least
    for b, h, rows, ref in varlen_refs(c):
        check(o[rows, h], lse[rows, h], ref, "request %d head %d" % (b, h))


def test_short_items_of_a_tail_stay_whole(g):
    """Nothing is cut where every item is short."""
    c = varlen_case(torch.Generator().manual_seed(4), [100] * 20, [100] * 20, 3, torch.bfloat16)
    o, lse, parts = call(g, c)
    assert parts <= 1
    for b, h, rows, ref in varlen_refs(c):
        check(o[rows, h], lse[rows, h], ref, "request %d head %d" % (b, h))


def test_offsets_of_one_call_to_the_next(g):
    """One workspace for calls that cut into other numbers of parts, or nothing."""
    cases = [varlen_case(torch.Generator().manual_seed(n), nq, lens, H, torch.bfloat16)
             for n, (nq, lens, H) in enumerate((([1], [9000], 1), ([300, 2], [2000, 5000], 3), ([60] * 9, [60] * 8 + [900], 2)))]
    size = max(g.attn_latent_varlen_workspace_size(len(c["nq"]), sum(c["nq"]), c["H"]) for c in cases)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for c in cases * 2:
        o, lse = g.attn_fwd_latent_varlen(c["q"], c["k"], c["v"], c["pe"], c["cq"], c["ck"], workspace=ws)
        for b, h, rows, ref in varlen_refs(c):
            check(o[rows, h], lse[rows, h], ref, "request %d head %d" % (b, h))
