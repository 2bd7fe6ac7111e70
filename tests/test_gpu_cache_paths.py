"""The paged cache's calls where they take other ways than small ones do: forks by three launches,
lists of more than 1024 sequences, rows of many heads. Against the model on the host, bit for bit."""

import random

import pytest
import torch

from tests.test_gpu_cache import Model, ints, make, new_rows, same, starts_of, state
from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


def filled(seed, lengths, pages, page, slot_pages, heads=1, dh=64, layers=1):
    """A cache whose slots hold `lengths` tokens, in an order of their own, and its model."""
    slots = len(lengths)
    c, m = make(layers, pages, page, heads, dh, slots, slot_pages, seed=seed)
    assert isinstance(m, Model)
    rng = random.Random(seed)
    order = rng.sample(range(slots), slots)
    counts = [lengths[s] for s in order]
    st = ints(starts_of(counts))
    k, v = new_rows(rng, layers, sum(counts), heads, dh)
    c.extend(ints(order), st)
    m.extend(order, counts)
    c.write(k.cuda(), v.cuda(), ints(order), st)
    m.write(order, counts, k, v)
    return c, m, rng


def test_fork_of_many_entries():
    # rows of 600 pages: sources read and targets written by launches of their own
    slots, slot_pages, page = 40, 600, 4
    rng = random.Random(7)
    lengths = [rng.choice([0, 1, page, rng.randint(1, 900), slot_pages * page]) for _ in range(slots)]
    c, m, rng = filled(1, lengths, 40 * 600, page, slot_pages)
    m.check(c)
    for n in (28, 40, 40, 35):
        dst = rng.sample(range(slots), n)
        src = [rng.randrange(slots) for _ in dst]  # targets among them, some more than once
        c.fork(ints(src), ints(dst))
        m.fork(src, dst)
        m.check(c)
        some = rng.sample(range(slots), 12)  # some grow or are cut in between
        counts = [rng.randint(0, 9) if m.length[s] + 9 <= slot_pages * page else 0 for s in some]
        st = ints(starts_of(counts))
        k, v = new_rows(rng, 1, sum(counts), 1, 64)
        c.extend(ints(some), st)
        m.extend(some, counts)
        c.write(k.cuda(), v.cuda(), ints(some), st)
        m.write(some, counts, k, v)
        cut = rng.sample(range(slots), 5)
        to = [rng.randint(0, 500) for _ in cut]
        c.truncate(ints(cut), ints(to))
        m.truncate(cut, to)
        m.check(c)
    # a rotation, and every slot onto itself
    for src, dst in ([list(range(1, 40)) + [0], list(range(40))], [list(range(40))] * 2):
        c.fork(ints(src), ints(dst))
        m.fork(src, dst)
        m.check(c)


@pytest.mark.parametrize("n,slot_pages", [(64, 128), (64, 129), (63, 128), (65, 64), (65, 65), (128, 64),
                                          (128, 65), (129, 8), (129, 64), (1, 128), (1, 129)])
def test_forks_by_one_launch_and_by_three(n, slot_pages):
    page = 4
    rng = random.Random(n)
    lengths = [rng.choice([0, rng.randint(1, slot_pages * page), slot_pages * page])
               for _ in range(n + 1)]
    c, m, rng = filled(n, lengths, (n + 1) * slot_pages, page, slot_pages)
    for _ in range(3):
        dst = rng.sample(range(n + 1), n)
        src = [rng.randrange(n + 1) for _ in dst]
        c.fork(ints(src), ints(dst))
        m.fork(src, dst)
        m.check(c)
    before = state(c)
    c.fork(ints(src), ints(dst[:-1] + [n + 1]))
    assert c.fault() == pb.PB_ERR_CACHE + 256 * 3
    assert same(before, state(c))


def test_faulty_forks_of_many_entries_change_nothing():
    slots, slot_pages, page = 40, 600, 4
    c, m, rng = filled(2, [50 + 3 * i for i in range(slots)], 3000, page, slot_pages)
    good = list(range(slots))

    def fork(src, dst):
        before = state(c)
        c.fork(ints(src), ints(dst))
        fault = c.fault()
        c.status.zero_()
        assert same(before, state(c))
        return fault

    twice, outside = good[:39] + [3], good[:39] + [slots]
    assert fork(good, twice) == pb.PB_ERR_CACHE + 256 * 3
    assert fork(good, outside) == pb.PB_ERR_CACHE + 256 * 3
    assert fork(outside, good) == pb.PB_ERR_CACHE + 256 * 3
    old = int(c.table[37, 5])
    for bad in (-1, 3000):
        c.table[37, 5] = bad
        assert fork([37] + good[1:], good) == pb.PB_ERR_CACHE + 256 * 5
        assert fork([0] * slots, good) == pb.PB_ERR_CACHE + 256 * 5  # what slot 37 held is released
    c.table[37, 5] = old
    c.fork(ints(good[::-1]), ints(good))
    m.fork(good[::-1], good)
    m.check(c)


@pytest.mark.parametrize("slot_pages", [8, 12])
def test_lists_of_more_than_1024(slot_pages):
    slots, page = 1500, 4
    rng = random.Random(slot_pages)
    c, m, rng = filled(slot_pages, [rng.randint(0, 14) for _ in range(slots)], 9000, page, slot_pages)
    order = rng.sample(range(slots), slots)
    # drafts, of which some are kept
    counts = [rng.randint(0, 7) for _ in order]
    st = ints(starts_of(counts))
    k, v = new_rows(rng, 1, sum(counts), 1, 64)
    c.extend(ints(order), st)
    m.extend(order, counts)
    c.write(k.cuda(), v.cuda(), ints(order), st)
    m.write(order, counts, k, v)
    paths = [sorted(rng.sample(range(n), rng.randint(0, n))) for n in counts]
    path = sum([p + [-1] * (n - len(p)) for p, n in zip(paths, counts)], [])
    c.keep(ints(order), st, ints(path), ints([len(p) for p in paths]))
    m.keep(order, counts, paths)
    m.check(c)
    src = [rng.randrange(slots) for _ in order]
    c.fork(ints(src), ints(order))
    m.fork(src, order)
    m.check(c)
    to = [rng.randint(-2, 16) for _ in order]
    c.truncate(ints(order), ints(to))
    m.truncate(order, to)
    m.check(c)


@pytest.mark.parametrize("slot_pages", [8, 12])
def test_faults_behind_the_first_1024_change_nothing(slot_pages):
    slots = 1500
    c, m, rng = filled(3, [5] * slots, 6000, 4, slot_pages)
    good = list(range(slots))
    twice = good[:1400] + [2] + good[1401:]
    one = starts_of([1] * slots)
    fall = one[:1301] + [one[1300] - 1] + one[1302:]
    kept = [1] * slots
    long = kept[:1200] + [2] + kept[1201:]
    for why, call in (
            (3, lambda: c.extend(ints(twice), ints(one))), (4, lambda: c.extend(ints(good), ints(fall))),
            (3, lambda: c.truncate(ints(twice), ints([0] * slots))),
            (3, lambda: c.fork(ints(good), ints(twice))),
            (3, lambda: c.fork(ints(good[:1499] + [-1]), ints(good))),
            (3, lambda: c.keep(ints(twice), ints(one), ints([0] * slots), ints(kept))),
            (4, lambda: c.keep(ints(good), ints(fall), ints([0] * slots), ints([0] * slots))),
            (6, lambda: c.keep(ints(good), ints(one), ints([0] * slots), ints(long)))):
        before = state(c)
        call()
        assert c.fault() == pb.PB_ERR_CACHE + 256 * why
        c.status.zero_()
        assert same(before, state(c))
    m.check(c)


@pytest.mark.parametrize("heads,dh", [(9, 128), (16, 128), (32, 128), (17, 64), (40, 64)])
def test_rows_of_many_heads(heads, dh):
    rng = random.Random(heads)
    c, m = make(2, 40, 7, heads, dh, 5, 9)
    counts = [10, 0, 33, 1]
    some = [4, 2, 0, 1]
    st = ints(starts_of(counts))
    k, v = new_rows(rng, 2, sum(counts) + 3, heads, dh)
    c.extend(ints(some), st)
    m.extend(some, counts)
    c.write(k.cuda(), v.cuda(), ints(some), st)
    m.write(some, counts, k, v)
    m.check(c)
    # heads with gaps between them, tokens in another order in memory
    wide = torch.randn(2, heads, 50, dh + 8, device="cuda").to(torch.bfloat16).permute(0, 2, 1, 3)
    x = wide[:, ::2, :, :dh]
    c.extend(ints([3]), ints([0, 25]))
    m.extend([3], [25])
    c.write(x, x, ints([3]), ints([0, 25]))
    m.write([3], [25], x.cpu(), x.cpu())
    path = [0, 1, 5, 6, 7, 20, 24]
    c.keep(ints([3]), ints([0, 25]), ints(path + [0] * 18), ints([7]))
    m.keep([3], [25], [path])
    c.fork(ints([3]), ints([2]))
    m.fork([3], [2])
    c.extend(ints([2, 3]), ints([0, 1, 2]))
    m.extend([2, 3], [1, 1])
    m.check(c)
