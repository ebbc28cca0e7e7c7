"""The plan of a step over the paged cache: pages, stack and row maps equal those of a plan
made sequence by sequence with lists."""

import random

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from tests import prefill_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(table, lens, free, count, keep, next_pos, n_rows, page, n_pages, status=0):
    k = torch.zeros(n_pages, page, 1, 8, dtype=torch.bfloat16, device="cuda")
    cache = qb.PagedCache(k, torch.zeros_like(k), i32(table), i32(lens))
    stack = free + [99] * (n_pages - len(free))
    pool = qb.PagePool(i32(stack), i32([len(free)]))
    got = qb.paged_plan(cache, pool, i32(count), keep=None if keep is None else i32(keep),
                        next_pos=None if next_pos is None else i32(next_pos), n_rows=n_rows)
    torch.cuda.synchronize()
    assert qb.query_status() == status
    table, lens, left, *maps = ref.plan(table, lens, free, count, keep, next_pos, n_rows, page, n_pages)
    assert cache.table.tolist() == table
    assert cache.lens.tolist() == lens
    assert int(pool.n_free) == len(left) and pool.free[:len(left)].tolist() == left
    assert pool.free[max(len(left), len(free)):].tolist() == stack[max(len(left), len(free)):]
    for a, b in zip(got, maps):
        assert a.tolist() == b
    return got


def scene(seed, seqs, width, page, most, spare, keep_all=False):
    rng = random.Random(seed)
    lens = [rng.choice([0, rng.randint(0, width * page), page * rng.randint(0, width)]) for _ in range(seqs)]
    owned = [min(width, -(-n // page) + rng.choice([0, 0, 1, 3])) for n in lens]
    n_pages = sum(owned) + spare
    pages = list(range(n_pages))
    rng.shuffle(pages)
    table, at = [], 0
    for o in owned:
        table.append(pages[at:at + o] + [-1] * (width - o))
        at += o
    free = pages[at:]
    count = [rng.choice([0, 1, 1, rng.randint(0, most), -3]) for _ in range(seqs)]
    keep = [rng.choice([-1, 0, n, n, max(0, n - 5), n + 10, rng.randint(0, n)]) for n in lens]
    return table, lens, free, count, keep if keep_all or rng.random() < 0.8 else None, [rng.randint(0, 10 ** 6) for _ in lens], max(1, n_pages)


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("seqs,width,page,most,spare", [(1, 4, 16, 40, 3), (7, 6, 8, 30, 10), (33, 40, 8, 200, 150), (40, 3, 64, 5, 1)])
def test_random_scenes(seed, seqs, width, page, most, spare):
    table, lens, free, count, keep, nxt, n_pages = scene(seed, seqs, width, page, most, spare)
    asked = sum(max(c, 0) for c in count)
    n_rows = max(0, asked + random.Random(seed).choice([0, 5, 5, -4]))
    check(table, lens, free, count, keep, nxt if seed % 2 else None, n_rows, page, n_pages)


@pytest.mark.parametrize("seqs", [1024, 1025, 2500])
def test_more_sequences_than_threads(seqs):
    table, lens, free, count, keep, nxt, n_pages = scene(5, seqs, 5, 8, 20, 400, keep_all=True)
    check(table, lens, free, count, keep, nxt, sum(max(c, 0) for c in count) + 3, 8, n_pages)


@pytest.mark.parametrize("n_rows", [1023, 1024, 1025, 1026, 40000])
def test_long_rows(n_rows):
    """One prompt over many pages, on both sides of the single launch's rows."""
    check([[-1] * 3000, [0] + [-1] * 2999], [0, 5], list(range(1, 2700)), [n_rows - 2, 2], None, [7, 9], n_rows, 16, 2700)


def test_first_pages_in_order():
    cache = qb.PagedCache.empty(2, 256, 2, 64, page=64, n_pages=6)
    pool = qb.PagePool.full(cache)
    first, granted, seq, slot, pos = qb.paged_plan(cache, pool, i32([65, 3]), n_rows=70)
    assert cache.table.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]] and int(pool.n_free) == 3
    assert first.tolist() == [0, 65] and granted.tolist() == [65, 3]
    assert slot.tolist() == list(range(65)) + [0, 1, 2, -1, -1] and pos[68:].tolist() == [0, 0]
    # nothing was appended: the same plan again takes no page
    qb.paged_plan(cache, pool, i32([65, 3]), n_rows=70)
    assert int(pool.n_free) == 3
    # both are given up
    qb.paged_plan(cache, pool, i32([0, 0]), keep=i32([0, 0]), n_rows=0)
    assert int(pool.n_free) == 6 and cache.table.tolist() == [[-1] * 4] * 2
    assert sorted(pool.free.tolist()) == list(range(6))


def test_a_starved_pool_serves_in_order():
    """Sequence 1 asks for more than there is: it and those behind it that need pages get none, one that needs none does."""
    table = [[-1, -1, -1], [-1, -1, -1], [3, -1, -1], [-1, -1, -1]]
    got = check(table, [0, 0, 4, 0], [0, 1, 2], [8, 24, 4, 1], None, None, 40, 8, 4)
    assert got[1].tolist() == [8, 0, 4, 0]


def test_too_long_for_the_table_or_the_rows():
    got = check([[0, -1], [1, -1], [-1, -1]], [8, 3, 0], [2, 3, 4], [9, 14, 6], None, None, 25, 8, 5)
    assert got[1].tolist() == [0, 0, 0]
    got = check([[0, -1], [1, -1], [-1, -1]], [8, 3, 0], [2, 3, 4], [9, 13, 2], None, None, 25, 8, 5)
    assert got[1].tolist() == [0, 13, 2]


@pytest.mark.parametrize("free,n_free", [([0, 1, 2], -1), ([0, 1, 2], 9), ([0, 77, 2], 3)])
def test_bad_pools_are_reported(free, n_free):
    cache = qb.PagedCache.empty(1, 24, 1, 8, page=8, n_pages=3)
    pool = qb.PagePool(i32(free), i32([n_free]))
    qb.paged_plan(cache, pool, i32([24]), n_rows=24)
    torch.cuda.synchronize()
    assert qb.query_status() == -8
    assert 0 <= int(pool.n_free) <= 3 and all(-1 <= p < 3 for p in cache.table[0].tolist())


def test_pages_that_come_back_twice_are_reported():
    cache = qb.PagedCache.empty(3, 16, 1, 8, page=8, n_pages=3)
    cache.table[:] = i32([[0, 1], [0, 1], [0, 1]])
    cache.lens[:] = 16
    pool = qb.PagePool(i32([0, 0, 0]), i32([0]))
    qb.paged_plan(cache, pool, i32([0, 0, 0]), keep=i32([0, 0, 0]), n_rows=0)
    torch.cuda.synchronize()
    assert qb.query_status() == -8 and int(pool.n_free) == 3 and cache.table.tolist() == [[-1, -1]] * 3


def test_the_lengths_as_keep_and_positions():
    """keep = lens returns the pages that hold nothing; positions that are slots."""
    table, lens = [[5, 2, 7, -1], [0, 1, -1, -1], [-1] * 4], [9, 0, 0]
    k = torch.zeros(9, 8, 1, 8, dtype=torch.bfloat16, device="cuda")
    cache = qb.PagedCache(k, torch.zeros_like(k), i32(table), i32(lens))
    pool = qb.PagePool(i32([3, 4, 6, 8, 99, 99, 99, 99, 99]), i32([4]))
    got = qb.paged_plan(cache, pool, i32([2, 0, 3]), keep=cache.lens, next_pos=cache.lens, n_rows=6)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    want, kept, left, *maps = ref.plan(table, lens, [3, 4, 6, 8], [2, 0, 3], lens, lens, 6, 8, 9)
    assert cache.table.tolist() == want and cache.lens.tolist() == kept == lens
    assert pool.free[:len(left)].tolist() == left and int(pool.n_free) == len(left)
    assert [t.tolist() for t in got] == maps


def test_a_bad_number_on_the_stack_ends_what_is_handed_out():
    """A sequence that asks for it gets none of its pages, nor do those behind it that need pages: no page is
    lost and no sequence's table has a hole. It is reported where it is asked for."""
    k = torch.zeros(5, 8, 1, 8, dtype=torch.bfloat16, device="cuda")
    cache = qb.PagedCache(k, torch.zeros_like(k), i32([[-1] * 3, [-1] * 3, [4, -1, -1], [-1] * 3]), i32([0, 0, 5, 0]))
    pool = qb.PagePool(i32([0, 77, 2, 3, 99]), i32([4]))
    _, granted, _, slot, _ = qb.paged_plan(cache, pool, i32([8, 16, 3, 1]), n_rows=28)
    torch.cuda.synchronize()
    assert qb.query_status() == -8
    assert granted.tolist() == [8, 0, 3, 0] and slot.tolist() == list(range(8)) + [-1] * 16 + [5, 6, 7, -1]
    assert cache.table.tolist() == [[3, -1, -1], [-1] * 3, [4, -1, -1], [-1] * 3]
    assert int(pool.n_free) == 3 and pool.free[:3].tolist() == [0, 77, 2]
    # all are given up, and one asks for pages that came back and the one above the bad number
    cache.lens[0] = 8
    _, granted, *_ = qb.paged_plan(cache, pool, i32([0, 24, 0, 0]), keep=i32([0, 0, 0, 0]), n_rows=24)
    torch.cuda.synchronize()
    assert qb.query_status() == 0 and granted.tolist() == [0, 24, 0, 0]
    assert cache.table.tolist() == [[-1] * 3, [4, 3, 2], [-1] * 3, [-1] * 3]
    assert int(pool.n_free) == 2 and pool.free[:2].tolist() == [0, 77]


@pytest.mark.parametrize("n_rows", [8 * 2000, 8])
def test_a_bad_number_deep_in_a_long_stack(n_rows):
    """2500 free pages, more than a CTA has threads; the numbers 1100 and 1700 from the top are none."""
    n, width = 2600, 2000
    k = torch.zeros(n, 8, 1, 8, dtype=torch.bfloat16, device="cuda")
    cache = qb.PagedCache(k, torch.zeros_like(k), torch.full((3, width), -1, dtype=torch.int32, device="cuda"), i32([0, 0, 0]))
    free = torch.arange(n, dtype=torch.int32, device="cuda")
    free[2500 - 1 - 1100], free[2500 - 1 - 1700] = -5, n
    pool = qb.PagePool(free.clone(), i32([2500]))
    _, granted, *_ = qb.paged_plan(cache, pool, i32([8 * 1100, 8, 8 * 600]), n_rows=8 * 1100 + n_rows)
    torch.cuda.synchronize()
    assert qb.query_status() == -8 and granted.tolist() == [8 * 1100, 0, 0]
    assert cache.table[0, :1100].tolist() == list(range(2499, 1399, -1)) and bool((cache.table[1:] == -1).all())
    assert int(pool.n_free) == 1400 and torch.equal(pool.free, free)
    # what is not asked for is not looked at
    _, granted, *_ = qb.paged_plan(cache, qb.PagePool(free.clone(), i32([2500])), i32([0, 8 * 1100, 0]), n_rows=8 * 1100)
    torch.cuda.synchronize()
    assert qb.query_status() == 0 and granted.tolist() == [0, 8 * 1100, 0]
