"""Block tables, offsets and slot map built on the GPU against a plain Python
construction, token by token.  Whole numbers: every comparison is exact."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
I32_MAX = 2**31 - 1


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gqa_softmax_attention_gb300 import build
    build.build()
    import gqa_softmax_attention_gb300 as m
    yield m
    m.gqa_device_error()


def plain(past, new, table, free, ps, num_pages, T, start=0):
    table = [row[:] for row in table]
    max_pages = len(table[0])
    cap = max_pages * ps
    cu, lens, slots, positions, requests, taken = [0], [], [], [], [], max(start, 0)
    total = 0
    for b, (p, n) in enumerate(zip(past, new)):
        p, n = min(max(p, 0), cap), max(n, 0)
        first = taken
        n0, n1 = -(-p // ps), min(-(-(p + n) // ps), max_pages)
        taken += max(0, n1 - n0)
        for x in range(p, p + min(n, max(0, T - len(slots)))):
            page = -1
            if x < cap:
                if x // ps >= n0:
                    f = first + x // ps - n0
                    page = free[f] if f < len(free) else -1
                    table[b][x // ps] = page
                else:
                    page = table[b][x // ps]
            slots.append(page * ps + x % ps if 0 <= page < num_pages else -1)
            positions.append(x)
            requests.append(b)
        lens.append(min(p + n, cap))
        total += n
        cu.append(min(total, T))
    pad = T - len(slots)
    counts = [min(total, I32_MAX), taken - max(start, 0), taken]
    return cu, lens, slots + [-1] * pad, positions + [0] * pad, requests + [-1] * pad, counts, table


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


NAMES = ("cu_seqlens_q", "cache_seqlens", "slots", "positions", "requests", "counts")


def check(g, past, new, table, free, ps, num_pages, T, start=None, out=None):
    dt = i32(table)
    got = g.attn_paged_slots(i32(past), i32(new), dt, i32(free), ps, num_pages, T,
                             free_start=None if start is None else i32([start]), out=out)
    want = plain(past, new, table, free, ps, num_pages, T, start or 0)
    for n, x, y in zip(NAMES, got, want):
        assert x.tolist() == y, n
    assert dt.tolist() == want[6], "block_table"
    return got


def draw(seed, B, lo, hi, ctx, ps, extra_pages=0):
    r = random.Random(seed)
    past = [r.randint(0, ctx) for _ in range(B)]
    new = [r.randint(lo, hi) for _ in range(B)]
    max_pages = max(1, -(-(ctx + hi) // ps)) + extra_pages
    need = sum(-(-(p + n) // ps) for p, n in zip(past, new))
    ids = list(range(need + 5))
    r.shuffle(ids)
    table, at = [], 0
    for p in past:
        held = -(-p // ps)
        table.append(ids[at:at + held] + [-1] * (max_pages - held))
        at += held
    return past, new, table, ids[at:], ps, need + 5


CASES = [
    # B, lo, hi, ctx, page_size
    (1, 1, 1, 0, 1), (1, 0, 0, 10, 16), (3, 1, 1, 100, 16), (64, 1, 1, 300, 64), (33, 0, 9, 40, 8), (7, 5, 200, 64, 24),
    (511, 0, 3, 20, 16), (512, 0, 3, 20, 16), (513, 0, 3, 20, 16), (1300, 0, 2, 9, 5), (5, 400, 1000, 30, 128),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("pad", [0, 37])
def test_matches_plain(g, case, pad):
    past, new, table, free, ps, num_pages = draw(1, *case)
    check(g, past, new, table, free, ps, num_pages, sum(new) + pad)


def test_many_tokens_over_many_blocks(g):
    past, new, table, free, ps, num_pages = draw(2, 900, 0, 350, 60, 16)
    check(g, past, new, table, free, ps, num_pages, sum(new) + 1000)


def test_free_start_and_chained_calls(g):
    past, new, table, free, ps, num_pages = draw(3, 20, 0, 30, 50, 8)
    lead = [10**6] * 4
    first = check(g, past, new, table, lead + free, ps, num_pages, sum(new), start=4)
    # the next step: what was written becomes the past, the table and the free list go on
    dt = i32(table)
    a = g.attn_paged_slots(i32(past), i32(new), dt, i32(free + [777] * 50), ps, num_pages, sum(new))
    t1 = dt.tolist()
    b = g.attn_paged_slots(a[1], i32([1] * 20), dt, i32(free + [777] * 50), ps, num_pages, 20, free_start=a[5][2:])
    want = plain(a[1].tolist(), [1] * 20, t1, free + [777] * 50, ps, num_pages, 20, start=a[5][2].item())
    for n, x, y in zip(NAMES, b, want):
        assert x.tolist() == y, n
    assert dt.tolist() == want[6]
    assert first[5].tolist()[1] == a[5].tolist()[1]


def test_repeats_and_writes_the_given_buffers(g):
    past, new, table, free, ps, num_pages = draw(4, 30, 0, 40, 50, 16)
    first = check(g, past, new, table, free, ps, num_pages, sum(new) + 3)
    kept = [t.clone() for t in first]
    again = check(g, past, new, plain(past, new, table, free, ps, num_pages, sum(new))[6], free, ps, num_pages,
                  sum(new) + 3, out=first)
    for x, y, z in zip(first, again, kept):
        assert x.data_ptr() == y.data_ptr() and torch.equal(x, z)


def test_rows_pages_and_capacity_run_out(g):
    past, new, table, free, ps, num_pages = draw(5, 12, 5, 40, 30, 8)
    check(g, past, new, table, free, ps, num_pages, sum(new) // 2)              # fewer rows than tokens
    check(g, past, new, table, free, ps, num_pages, 0)                          # none at all
    check(g, past, new, table, free[:3], ps, num_pages, sum(new))               # the free list ends
    check(g, past, new, table, [], ps, num_pages, sum(new))
    check(g, past, new, table, free, ps, num_pages, sum(new), start=len(free) + 9)
    narrow = [row[:4] for row in table]                                         # 32 tokens of capacity
    check(g, past, new, narrow, free, ps, num_pages, sum(new))


def test_lengths_and_ids_out_of_range(g):
    past, new, table, free, ps, num_pages = draw(6, 10, 0, 20, 30, 8)
    past[3], new[4], past[5] = -7, -3, 10**9
    check(g, past, new, table, free, ps, num_pages, sum(max(n, 0) for n in new) + 5, start=-4)
    check(g, past, new, table, [x + num_pages if i % 2 else -x - 1 for i, x in enumerate(free)], ps, num_pages, 200)
    check(g, past, new, table, free, ps, 0, 200)                                # an empty pool: no slot at all
    big = [2**31 - 1] * 10                                                      # sums past 32 bits
    check(g, past, big, table, free, ps, num_pages, 100)


def test_replay_in_a_graph_with_new_lengths(g):
    past, new, table, free, ps, num_pages = draw(7, 40, 0, 25, 60, 16)
    dp, dn, dt, df = i32(past), i32(new), i32(table), i32(free)
    T = 40 * 25
    out = g.attn_paged_slots(dp, dn, dt, df, ps, num_pages, T)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        g.attn_paged_slots(dp, dn, dt, df, ps, num_pages, T, out=out)
    new2 = [(n * 7 + i) % 25 for i, n in enumerate(new)]
    dn.copy_(i32(new2))
    dt.copy_(i32(table))
    df.copy_(i32((free * 50)[:len(free)]))
    graph.replay()
    torch.cuda.synchronize()
    want = plain(past, new2, table, free, ps, num_pages, T)
    for n, x, y in zip(NAMES, out, want):
        assert x.tolist() == y, n
    assert dt.tolist() == want[6]


def test_refusals(g):
    past, new, table, free, ps, num_pages = draw(8, 4, 1, 3, 10, 8)
    args = lambda **k: {**dict(past_lens=i32(past), new_lens=i32(new), block_table=i32(table), free_pages=i32(free),  # noqa: E731
                               page_size=ps, num_pages=num_pages, max_tokens=12), **k}
    counts = g.attn_paged_slots(**args())
    for bad in (dict(past_lens=i32(past).long()), dict(new_lens=i32(new[:3])), dict(block_table=i32(table)[:, ::2]),
                dict(block_table=i32(table).cpu()), dict(free_pages=i32([free])), dict(page_size=0),
                dict(max_tokens=-1), dict(num_pages=-1), dict(free_start=i32([0, 0])), dict(out=counts[:5]),
                dict(out=counts, free_start=counts[5][1:2]), dict(out=counts, past_lens=counts[1]), dict(max_tokens=13, out=counts),
                dict(past_lens=i32([]), new_lens=i32([]), block_table=torch.empty(0, 4, dtype=torch.int32,
                                                                                  device="cuda"))):
        with pytest.raises(ValueError):
            g.attn_paged_slots(**args(**bad))


def test_sizes_past_32_bits_are_refused(g):
    """A size whose low 32 bits would pass for a good one."""
    past, new, table, free, ps, num_pages = draw(9, 4, 1, 3, 10, 8)
    for bad in (dict(page_size=(1 << 32) + ps), dict(num_pages=(1 << 32) + num_pages), dict(max_tokens=(1 << 32) + 12),
                dict(max_tokens=1 << 30), dict(page_size=1 << 31), dict(page_size=ps - (1 << 32)),
                dict(num_pages=num_pages - (1 << 32)), dict(max_tokens=12 - (1 << 32))):
        with pytest.raises(ValueError):
            g.attn_paged_slots(**{**dict(past_lens=i32(past), new_lens=i32(new), block_table=i32(table),
                                         free_pages=i32(free), page_size=ps, num_pages=num_pages, max_tokens=12), **bad})
