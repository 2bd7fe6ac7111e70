"""The paged cache against a plain model of it on the host: tables, lengths, counts of users and the
rows themselves are equal, bit for bit, after random runs of every call; calls at fault change
nothing and say why."""

import random

import pytest
import torch

from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """What the calls are documented to do, on the host."""

    def __init__(self, cache):
        self.page = cache.k.shape[3]
        self.pages, self.slots = cache.refs.numel(), cache.slots
        self.rows = [[] for _ in range(self.slots)]  # page numbers
        self.length = [0] * self.slots
        self.refs = [0] * self.pages
        self.k, self.v = cache.k.cpu().clone(), cache.v.cpu().clone()

    def _drop(self, slot, n):
        keep = -(-n // self.page)
        for p in self.rows[slot][keep:]:
            self.refs[p] -= 1
        self.rows[slot] = self.rows[slot][:keep]
        self.length[slot] = n

    def extend(self, slots, counts):
        free = [p for p in range(self.pages) if self.refs[p] == 0]
        shared = [c > 0 and self.length[s] % self.page != 0 and self.refs[self.rows[s][-1]] > 1
                  for s, c in zip(slots, counts)]
        for s, c, copy in zip(slots, counts, shared):
            n = self.length[s]
            if copy:
                old, new = self.rows[s][-1], free.pop(0)
                for pool in (self.k, self.v):
                    pool[:, new, :, :n % self.page] = pool[:, old, :, :n % self.page]
                self.rows[s][-1] = new
                self.refs[old] -= 1
                self.refs[new] = 1
            while len(self.rows[s]) * self.page < n + c:
                new = free.pop(0)
                self.refs[new] = 1
                self.rows[s].append(new)
            self.length[s] = n + c

    def place(self, slot, t):
        return self.rows[slot][t // self.page], t % self.page

    def write(self, slots, counts, k, v, layer=0):
        t = 0
        for s, c in zip(slots, counts):
            for j in range(c):
                p, r = self.place(s, self.length[s] - c + j)
                self.k[layer:layer + k.shape[0], p, :, r] = k[:, t]
                self.v[layer:layer + v.shape[0], p, :, r] = v[:, t]
                t += 1

    def keep(self, slots, counts, paths):
        for s, c, path in zip(slots, counts, paths):
            base = self.length[s] - c
            for j, at in enumerate(path):
                (p, r), (q, u) = self.place(s, base + at), self.place(s, base + j)
                for pool in (self.k, self.v):
                    pool[:, q, :, u] = pool[:, p, :, r].clone()
            self._drop(s, base + len(path))

    def fork(self, src, dst):
        old = [(list(self.rows[s]), self.length[s]) for s in src]
        for rows, _ in old:
            for p in rows:
                self.refs[p] += 1
        for d in dst:
            self._drop(d, 0)
        for d, (rows, n) in zip(dst, old):
            self.rows[d], self.length[d] = list(rows), n

    def truncate(self, slots, lengths):
        for s, n in zip(slots, lengths):
            self._drop(s, min(self.length[s], max(0, n)))

    def check(self, cache):
        assert cache.fault() == 0
        assert cache.lengths.tolist() == self.length
        assert cache.refs.tolist() == self.refs
        table = cache.table.tolist()
        for s in range(self.slots):
            assert table[s][:len(self.rows[s])] == self.rows[s], s
        for got, want in ((cache.k.cpu(), self.k), (cache.v.cpu(), self.v)):
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        users = [0] * self.pages
        for rows in self.rows:
            for p in rows:
                users[p] += 1
        assert users == self.refs


def make(layers=2, pages=60, page=16, heads=3, dh=64, slots=8, slot_pages=12, seed=0):
    c = pb.Cache.empty(layers, pages, page, heads, dh, slots, slot_pages)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    c.table.fill_(-7)
    c.scratch.fill_(255)
    return c, Model(c)


def starts_of(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


def new_rows(rng, layers, tokens, heads, dh):
    g = torch.Generator()
    g.manual_seed(rng.randrange(1 << 30))
    return [torch.randn(layers, tokens, heads, dh, generator=g).to(torch.bfloat16)
            for _ in range(2)]


def fits(m, slots, counts, slot_pages):
    need = 0
    for s, c in zip(slots, counts):
        if m.length[s] + c > slot_pages * m.page:
            return False
        need += -(-(m.length[s] + c) // m.page) - len(m.rows[s])
        need += c > 0 and m.length[s] % m.page != 0 and m.refs[m.rows[s][-1]] > 1
    return need <= sum(r == 0 for r in m.refs)


@pytest.mark.parametrize("page,dh,heads,layers", [(16, 64, 3, 2), (1, 64, 1, 1), (7, 128, 2, 3),
                                                  (64, 128, 1, 1), (5, 64, 9, 1), (100, 64, 2, 2)])
def test_random_runs(page, dh, heads, layers):
    rng = random.Random(page)
    slots, slot_pages = 8, 12
    c, m = make(layers, 60, page, heads, dh, slots, slot_pages)
    for step in range(60):
        some = rng.sample(range(slots), rng.randint(1, slots))
        op = rng.choice(["new", "new", "draft", "fork", "cut"])
        if op in ("new", "draft"):
            counts = [rng.choice([0, 1, 1, rng.randint(1, 2 * page), rng.randint(1, 9)])
                      for _ in some]
            if not fits(m, some, counts, slot_pages):
                op = "cut"
        if op in ("new", "draft"):
            st = ints(starts_of(counts))
            k, v = new_rows(rng, layers, sum(counts) + 2, heads, dh)
            c.extend(ints(some), st)
            m.extend(some, counts)
            c.write(k.cuda(), v.cuda(), ints(some), st)
            m.write(some, counts, k, v)
            if op == "draft":
                paths = [sorted(rng.sample(range(n), rng.randint(0, n))) for n in counts]
                path = []
                for p, n in zip(paths, counts):
                    path += p + [9999] * (n - len(p))
                c.keep(ints(some), st, ints(path + [5]), ints([len(p) for p in paths]))
                m.keep(some, counts, paths)
        elif op == "fork":
            src = [rng.randrange(slots) for _ in some]
            c.fork(ints(src), ints(some))
            m.fork(src, some)
        else:
            to = [rng.choice([0, rng.randint(-3, 5 * page), 10 ** 6]) for _ in some]
            c.truncate(ints(some), ints(to))
            m.truncate(some, to)
        if step % 6 == 5:
            m.check(c)
    m.check(c)


def test_many_slots_and_pages():
    # more sequences than a block has threads, more pages than one scan takes
    slots = 1500
    c, m = make(1, 9000, 4, 1, 64, slots, 8)
    rng = random.Random(3)
    order = rng.sample(range(slots), slots)
    counts = [rng.randint(0, 20) for _ in order]
    st = ints(starts_of(counts))
    k, v = new_rows(rng, 1, sum(counts), 1, 64)
    c.extend(ints(order), st)
    m.extend(order, counts)
    c.write(k.cuda(), v.cuda(), ints(order), st)
    m.write(order, counts, k, v)
    m.check(c)
    c.truncate(ints(order[:700]), ints([0] * 700))
    m.truncate(order[:700], [0] * 700)
    src = [order[700 + i % 800] for i in range(700)]
    c.fork(ints(src), ints(order[:700]))
    m.fork(src, order[:700])
    one = [1] * slots
    c.extend(ints(order), ints(starts_of(one)))
    m.extend(order, one)
    m.check(c)


def test_fork_onto_its_own_sources():
    # beams change places: every source is read as it was before the call
    c, m = make()
    counts = [5, 20, 33, 0, 16, 1, 40, 7]
    st = ints(starts_of(counts))
    k, v = new_rows(random.Random(1), 2, sum(counts), 3, 64)
    c.extend(ints(range(8)), st)
    m.extend(range(8), counts)
    c.write(k.cuda(), v.cuda(), ints(range(8)), st)
    m.write(range(8), counts, k, v)
    for src, dst in (([1, 2, 0, 3], [0, 1, 2, 3]), ([4, 4, 4], [4, 5, 6]), ([7, 0], [0, 7])):
        c.fork(ints(src), ints(dst))
        m.fork(src, dst)
        m.check(c)


def test_keep_beside_a_shared_page():
    # pages of 16: tokens 20 to 31 share a page with the fork and stay where they are, those behind move
    c, m = make()
    counts = [45]
    st = ints(starts_of(counts))
    k, v = (torch.randn(2, 45, 3, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    c.extend(ints([0]), st)
    m.extend([0], counts)
    c.write(k, v, ints([0]), st)
    m.write([0], counts, k.cpu(), v.cpu())
    c.fork(ints([0]), ints([1]))
    m.fork([0], [1])
    c.truncate(ints([1]), ints([32]))
    m.truncate([1], [32])
    path = list(range(12)) + [13, 17, 24]
    c.keep(ints([0]), ints([0, 25]), ints(path + [0] * 10), ints([15]))
    m.keep([0], [25], [path])
    m.check(c)


def test_layers_apart_and_views():
    c, m = make(layers=3, heads=4)
    counts = [17, 3]
    st = ints(starts_of(counts))
    c.extend(ints([2, 5]), st)
    m.extend([2, 5], counts)
    buf = torch.randn(20, 3, 12, 64, device="cuda").to(torch.bfloat16)  # [tokens, layers, q|k|v]
    k, v = buf[:, :, 4:8].transpose(0, 1), buf[:, :, 8:].transpose(0, 1)
    c.write(k[1:], v[1:], ints([2, 5]), st, layer=1)
    m.write([2, 5], counts, k[1:].cpu(), v[1:].cpu(), layer=1)
    c.write(buf[:, 0, :4], buf[:, 0, 8:], ints([2, 5]), st)
    m.write([2, 5], counts, buf[:, 0, :4].cpu()[None], buf[:, 0, 8:].cpu()[None])
    m.check(c)


def state(c):
    return [t.clone() for t in (c.lengths, c.refs, c.table, c.k, c.v)]


def same(a, b):
    return all(bool((x.view(torch.int16) == y.view(torch.int16)).all()) if x.dtype is torch.bfloat16
               else bool((x == y).all()) for x, y in zip(a, b))


def filled():
    c, m = make()
    c.extend(ints([0, 1, 2]), ints([0, 20, 50, 60]))
    c.fork(ints([0]), ints([3]))
    assert c.fault() == 0
    return c


def zeros(tokens):
    return torch.zeros(2, tokens, 3, 64, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("why,call", [
    (1, lambda c: c.extend(ints([4, 5, 6, 7, 0]), ints([0, 192, 384, 576, 768, 900]))),
    (2, lambda c: c.extend(ints([0]), ints([0, 173]))),
    (2, lambda c: c.extend(ints([0]), ints([-2 ** 31, 2 ** 31 - 1]))),
    (3, lambda c: c.extend(ints([0, 1, 0]), ints([0, 1, 2, 3]))),
    (3, lambda c: c.extend(ints([0, 8]), ints([0, 1, 2]))),
    (3, lambda c: c.extend(ints([-1]), ints([0, 1]))),
    (4, lambda c: c.extend(ints([0, 1]), ints([0, 5, 3]))),
    (3, lambda c: c.truncate(ints([2, 2]), ints([0, 0]))),
    (3, lambda c: c.fork(ints([0, 1]), ints([4, 4]))),
    (3, lambda c: c.fork(ints([8]), ints([4]))),
    (4, lambda c: c.keep(ints([0, 1]), ints([0, 3, 60]), ints([0] * 70), ints([0, 0]))),
    (4, lambda c: c.keep(ints([1]), ints([0, 3]), ints([0, 1]), ints([0]))),
    (4, lambda c: c.keep(ints([1]), ints([-1, 2]), ints([0, 1]), ints([0]))),
    (6, lambda c: c.keep(ints([1]), ints([0, 3]), ints([0, 1, 2]), ints([4]))),
    (6, lambda c: c.keep(ints([1]), ints([0, 3]), ints([0, 1, 2]), ints([-1]))),
    (6, lambda c: c.keep(ints([1]), ints([0, 3]), ints([1, 1, 2]), ints([2]))),
    (6, lambda c: c.keep(ints([1]), ints([0, 3]), ints([0, 3, 2]), ints([2]))),
    (6, lambda c: c.keep(ints([1]), ints([0, 3]), ints([-1, 1, 2]), ints([2]))),
    (7, lambda c: c.keep(ints([0]), ints([0, 3]), ints([0, 2, 2]), ints([2]))),
    (3, lambda c: c.write(zeros(2), zeros(2), ints([9]), ints([0, 2]))),
    (4, lambda c: c.write(zeros(60), zeros(60), ints([0]), ints([0, 60]))),
    (4, lambda c: c.write(zeros(3), zeros(3), ints([0]), ints([0, 4]))),
    (4, lambda c: c.write(zeros(3), zeros(3), ints([0]), ints([-1, 3]))),
])
def test_faults_change_nothing(why, call):
    c = filled()
    before = state(c)
    call(c)
    assert c.fault() == pb.PB_ERR_CACHE + 256 * why
    assert same(before, state(c))
    # and the cache stands still until the word is cleared
    c.extend(ints([5]), ints([0, 4]))
    c.truncate(ints([0]), ints([0]))
    c.fork(ints([1]), ints([5]))
    c.keep(ints([1]), ints([0, 3]), ints([0, 1, 2]), ints([1]))
    c.write(zeros(1), zeros(1), ints([1]), ints([0, 1]))
    assert same(before, state(c))
    c.status.zero_()
    c.extend(ints([5]), ints([0, 4]))
    assert c.fault() == 0 and c.lengths[5].item() == 4


def test_tables_at_fault():
    # pages that are none are refused, not followed
    for bad in (-1, 60, 2 ** 31 - 1, -2 ** 31):
        for at, call in ((1, lambda c: c.extend(ints([0]), ints([0, 1]))),
                         (1, lambda c: c.truncate(ints([0]), ints([3]))),
                         (0, lambda c: c.fork(ints([0]), ints([5]))),
                         (0, lambda c: c.fork(ints([1]), ints([0]))),
                         (1, lambda c: c.keep(ints([0]), ints([0, 6]), ints([0] * 6), ints([1]))),
                         (1, lambda c: c.write(zeros(1), zeros(1), ints([0]), ints([0, 1])))):
            c = filled()
            c.table[0, at] = bad
            before = state(c)
            call(c)
            assert c.fault() == pb.PB_ERR_CACHE + 256 * 5
            assert same(before, state(c))
    for bad in (-1, 12 * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        for call in (lambda c: c.extend(ints([0]), ints([0, 1])),
                     lambda c: c.truncate(ints([0]), ints([3])),
                     lambda c: c.fork(ints([0]), ints([5])), lambda c: c.fork(ints([1]), ints([0])),
                     lambda c: c.keep(ints([0]), ints([0, 6]), ints([0] * 6), ints([1])),
                     lambda c: c.write(zeros(1), zeros(1), ints([0]), ints([0, 1]))):
            c = filled()
            c.lengths[0] = bad
            before = state(c)
            call(c)
            assert c.fault() == pb.PB_ERR_CACHE + 256 * 5
            assert same(before, state(c))


def test_a_captured_loop():
    # a step of extend, write and keep as a graph: the numbers come from the device each time
    c, m = make(layers=2, pages=80, slots=6)
    slots, counts = [4, 0, 2], [3, 3, 3]
    st, path, kept = ints(starts_of(counts)), ints([0] * 9), ints([0] * 3)
    k, v = (torch.zeros(2, 9, 3, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sl = ints(slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.extend(sl, st)
        c.write(k, v, sl, st)
        c.keep(sl, st, path, kept)
    rng = random.Random(5)
    for _ in range(12):
        kk, vv = new_rows(rng, 2, 9, 3, 64)
        paths = [sorted(rng.sample(range(3), rng.randint(0, 3))) for _ in slots]
        k.copy_(kk)
        v.copy_(vv)
        path.copy_(torch.tensor(sum([p + [0] * (3 - len(p)) for p in paths], []), dtype=torch.int32))
        kept.copy_(torch.tensor([len(p) for p in paths], dtype=torch.int32))
        graph.replay()
        m.extend(slots, counts)
        m.write(slots, counts, kk, vv)
        m.keep(slots, counts, paths)
    m.check(c)


def test_offsets_past_32_bits():
    # a pool of more than 2^31 values in k: rows of its last pages and layer
    pages, page, heads, dh, layers = 40000, 64, 4, 128, 2
    c = pb.Cache.empty(layers, pages, page, heads, dh, 3, 20)
    assert c.k.numel() > 2 ** 31
    c.refs[:pages - 30] = 1  # all but the last pages are taken
    counts = [200, 0, 150]
    st = ints(starts_of(counts))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k, v = (torch.randn(layers, 350, heads, dh, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    sl = ints([2, 1, 0])
    c.extend(sl, st)
    c.write(k, v, sl, st)
    c.fork(ints([2]), ints([1]))
    c.extend(ints([1]), ints([0, 2]))
    c.keep(ints([2]), ints([0, 10]), ints([1, 3, 4, 9] + [0] * 6), ints([4]))
    assert c.fault() == 7 * 256 + 8  # tokens would move in a page that the fork uses too
    c.status.zero_()
    assert c.lengths.tolist() == [150, 202, 200]
    t = c.table.tolist()
    assert t[2][:4] == [pages - 30, pages - 29, pages - 28, pages - 27]

    def rows(pool, slot, n):
        return torch.stack([pool[:, t[slot][i // page], :, i % page] for i in range(n)], 1)

    assert torch.equal(rows(c.k, 2, 200), k[:, :200]) and torch.equal(rows(c.v, 0, 150), v[:, 200:])
    assert torch.equal(rows(c.k, 1, 200), k[:, :200])
