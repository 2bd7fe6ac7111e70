"""The serving operators at their borders: lists of items made by blocks and by a launch of their own,
writes outside results and scratch, offsets past 32 bits, several streams and host threads, graphs,
many sequences in one call. The formulas and tolerances are those of the operators' own tests."""

import random
import threading

import pytest
import torch

from tests import test_gpu_cache_attention as ca
from tests import test_gpu_prompt_attention as pa
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


@pytest.mark.parametrize("n", [127, 128, 129])
def test_prompts_listed_by_blocks_and_by_a_launch(n):
    pa.run([(i * 29) % 70 for i in range(n)], 6, 2, 64, tail=5, at=3)


def test_prompts_with_more_items_than_blocks_list():
    # one sequence, 160 key heads of their own: pairs x heads is beyond 64 items an SM
    t, w = 16000, 40
    q, k, v = (pa.randn(i, t, 160, 64) for i in range(3))
    out = pb.prompt_attention(q, k, v, window=w)
    for c in range(0, t, 1000):  # a piece and the keys before it that it sees
        a = max(0, c - w)
        want, size = pa.reference(q, k, v, a, c + 1000 - a, w, 0.125)
        bar = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -11) * size
        err = (out[a:c + 1000].double() - want).abs()
        assert bool((err <= bar)[c - a:].all()), c


@pytest.mark.parametrize("n", [8, 200])
def test_falling_starts_stay_inside(n):
    # sequences that overlap: rows have no defined value, but nothing outside out is written, and the
    # status word says so where they are more than the tokens allow
    t = 300
    q, k, v = pa.randn(1, t, 4, 64), pa.randn(2, t, 2, 64), pa.randn(3, t, 2, 64)
    st = ints([0 if i % 2 == 0 else t for i in range(n + 1)])
    big = torch.zeros(3 * t, 4, 64, dtype=torch.bfloat16, device="cuda")
    nbytes = pb.prompt_attention_scratch_bytes(t, n)
    scratch = torch.full((nbytes + 8192,), 77, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pb.prompt_attention(q, k, v, st, out=big[t:2 * t], scratch=scratch[:nbytes], status=status)
    assert status.item() in (0, 1)
    assert not big[:t].any() and not big[2 * t:].any()
    assert bool((scratch[nbytes:] == 77).all())


@pytest.mark.parametrize("n,t,group", [(128, 300, 2), (2 ** 20, 8192, 128)])
def test_falling_starts_do_nothing(n, t, group):
    # the second: more than 2^31 pairs of tiles, were they taken one by one
    q, k, v = pa.randn(1, t, group, 64), pa.randn(2, t, 1, 64), pa.randn(3, t, 1, 64)
    st = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    st[1::2] = t
    out = torch.full_like(q, 3.0)
    nbytes = pb.prompt_attention_scratch_bytes(t, n)
    scratch = torch.full((4096 + nbytes + 4096,), 77, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pb.prompt_attention(q, k, v, st, out=out, scratch=scratch[4096:-4096], status=status)
    assert status.item() == 1
    assert bool((out == 3).all())
    assert bool((scratch[:4096] == 77).all()) and bool((scratch[-4096:] == 77).all())
    # and the same scratch serves a sound call
    st[:] = t
    st[0] = 0
    pb.prompt_attention(q[:300], k[:300], v[:300], st[:2].clamp(max=300), out=out[:300],
                        scratch=scratch[4096:-4096])
    pa.check(out[:300], q[:300], k[:300], v[:300], [0, 300])


@pytest.mark.parametrize("n", [8, 40])
def test_faults_while_blocks_begin(n):
    # a fault is recorded while blocks of the same call look at the status word: each goes on as a whole
    # or not at all, so rows are right or as they were
    lengths = [300 + 37 * i for i in range(n)]
    c, data = ca.fill(lengths, 2, 64, 16)
    counts = [1 + i % 3 for i in range(n)]
    starts = pa.starts_of(counts)
    q = ca.randn(5, starts[-1], 4, 64)
    slots = list(range(n))
    good = c.attention(q, ints(slots), ints(starts))
    assert c.fault() == 0
    ca.check(good, q, data, slots, starts, None, None, 0.125, good)
    before = torch.full_like(q, 7.0)
    outs = []
    bad = ints(slots[:n // 2] + [n + 5] + slots[n // 2 + 1:])
    for _ in range(200):
        out = before.clone()
        c.attention(q, bad, ints(starts), out=out)
        c.status.zero_()
        outs.append(out)
    a, z = starts[n // 2], starts[n // 2 + 1]
    all_ = torch.stack(outs)
    assert bool((all_[:, a:z] == 7).all())
    rest = torch.ones(starts[-1], dtype=torch.bool, device="cuda")
    rest[a:z] = False
    as_was = (all_[:, rest] == 7).all(-1)
    # pieces are cut elsewhere without the sequence left out: twice the operator's bar, 2^-8 |out| +
    # 0.0063 sum p |v|, of which the sum over 300 keys and more stays below 1.2
    near = ((all_[:, rest].float() - good[rest].float()).abs()
            <= 2.0 ** -7 * good[rest].float().abs() + 2.0 ** -6).all(-1)
    assert bool((as_was | near).all())


def test_nothing_behind_scratch_or_out():
    lengths = [(i * 53) % 90 for i in range(150)]
    s = pa.starts_of(lengths)
    q, k, v = pa.randn(1, s[-1], 4, 64), pa.randn(2, s[-1], 2, 64), pa.randn(3, s[-1], 2, 64)
    nbytes = pb.prompt_attention_scratch_bytes(s[-1], 150)
    scratch = torch.full((nbytes + 4096,), 77, dtype=torch.uint8, device="cuda")
    big = torch.full((s[-1] + 200, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = big[100:-100]
    pb.prompt_attention(q, k, v, ints(s), out=out, scratch=scratch[:nbytes])
    pa.check(out, q, k, v, s)
    assert bool((big[:100] == 3).all()) and bool((big[-100:] == 3).all())
    assert bool((scratch[nbytes:] == 77).all())
    for hq, counts in ((8, [1, 1, 1]), (8, [7, 3, 6]), (16, [16, 9, 12])):
        c, data = ca.fill([700, 90, 300], 2, 128, 24)
        t = sum(counts)
        q = ca.randn(5, t, hq, 128)
        scratch = torch.full((c.attention_scratch_bytes + 4096,), 77, dtype=torch.uint8, device="cuda")
        big = torch.full((t + 20, hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        st = pa.starts_of(counts)
        c.attention(q, ints([0, 1, 2]), ints(st), out=big[10:-10],
                    scratch=scratch[:c.attention_scratch_bytes])
        ca.check(big[10:-10], q, data, [0, 1, 2], st, None, None, 128 ** -0.5, big[10:-10])
        assert bool((big[:10] == 3).all()) and bool((big[-10:] == 3).all())
        assert bool((scratch[c.attention_scratch_bytes:] == 77).all())


def test_nothing_beside_the_caches_words():
    # every buffer of the cache lies inside a larger one
    page, pages, slots, row = 16, 40, 6, 7

    def inside(n, fill, dtype=torch.int32):
        big = torch.full((n + 2048,), fill, dtype=dtype, device="cuda")
        return big, big[1024:1024 + n]

    bk, k = inside(2 * pages * 3 * page * 64, 5.0, torch.bfloat16)
    bv, v = inside(2 * pages * 3 * page * 64, 6.0, torch.bfloat16)
    bt, table = inside(slots * row, -5)
    bl, lengths = inside(slots, -6)
    br, refs = inside(pages, -7)
    bs, status = inside(1, -8)
    for t in (lengths, refs, status):
        t.zero_()
    c = pb.Cache(k.view(2, pages, 3, page, 64), v.view(2, pages, 3, page, 64),
                 table.view(slots, row), lengths, refs, status)
    scratch = torch.full((c.scratch_bytes + 4096,), 77, dtype=torch.uint8, device="cuda")
    c.scratch, c._scratch = scratch, scratch.data_ptr()
    rng = random.Random(1)
    for _ in range(20):
        some = rng.sample(range(slots), 3)
        counts = [rng.randint(0, 20) for _ in some]
        st = ints(pa.starts_of(counts))
        x = torch.randn(2, sum(counts), 3, 64, device="cuda").to(torch.bfloat16)
        c.truncate(ints(some), ints([rng.randint(0, 60) for _ in some]))
        c.extend(ints(some), st)
        c.write(x, x, ints(some), st)
        c.keep(ints(some), st, ints([j for n in counts for j in range(n)] + [0]),
               ints([n // 2 for n in counts]))
        c.fork(ints(some[:1]), ints([rng.randrange(slots)]))
        if c.fault():  # more than fits: that too has to stay inside
            c.status.zero_()
            c.truncate(ints(list(range(slots))), ints([0] * slots))
    for big, n, fill in ((bk, k.numel(), 5.0), (bv, v.numel(), 6.0), (bt, table.numel(), -5),
                         (bl, slots, -6), (br, pages, -7), (bs, 1, -8)):
        assert bool((big[:1024] == fill).all()) and bool((big[1024 + n:] == fill).all())
    assert bool((scratch[c.scratch_bytes:] == 77).all())


def test_prompt_offsets_past_32_bits():
    # rows 2^20 values apart: the last ones lie beyond 2^32 values
    t, row = 5000, 1 << 20
    big = torch.empty(t * row + 4096, dtype=torch.bfloat16, device="cuda")

    def view(at, heads):
        return big.as_strided((t, heads, 128), (row, 128, 1), at)

    q, k, v, out = view(0, 4), view(8192, 2), view(16384, 2), view(32768, 4)
    for x, seed in ((q, 1), (k, 2), (v, 3)):
        x.copy_(pa.randn(seed, *x.shape))
    s = [0, 900, 4990]
    out.fill_(2.0)
    before = out.clone()
    pb.prompt_attention(q, k, v, ints(s), out=out)
    pa.check(out.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), s, before=before)
    x = q.contiguous()
    rows, _ = pa.reference(x, k.contiguous(), v.contiguous(), 900, 4090, None, 128 ** -0.5)
    assert float((out[900:4990].double() - rows).abs().max()) < 0.1


def test_thousands_of_sequences():
    # more than a block has threads, in the lists, the shares and the bookkeeping
    rng = random.Random(4)
    lengths = [rng.randint(1, 40) for _ in range(2500)]
    ca.run(lengths, [1] * 2500, 2, 1, 64, 8)
    pa.run([rng.randint(0, 9) for _ in range(5000)], 4, 2, 64)


def test_several_host_threads():
    # distinct caches and scratch are independent, on streams of their own
    def work(i, errors):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for step in range(4):
                    ca.run([300 + 10 * i, 40, 999], [3, 1, 9], 8, 2, 64, 16, tree=True, seed=i)
                    pa.run([257, 30 + i, 400], 8, 2, 128, seed=i, tail=2)
        except BaseException as e:  # reported by the test
            errors.append(e)

    errors = []
    threads = [threading.Thread(target=work, args=(i, errors)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_host_threads_on_one_stream():
    # two launches a call: those of two threads may come in any order on the stream
    c, data = ca.fill([9000, 70, 4555], 4, 128, 32)
    sl, st = ints([0, 1, 2]), ints([0, 1, 2, 3])
    qs = [ca.randn(i, 3, 16, 128) for i in range(4)]
    want = [c.attention(q, sl, st).clone() for q in qs]
    torch.cuda.synchronize()
    wrong, done = [], []

    def work(i):
        torch.cuda.set_device(0)
        for _ in range(20):
            outs = [c.attention(qs[i], sl, st) for _ in range(50)]
            wrong.extend(i for o in outs if not torch.equal(o, want[i]))
        done.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(1, 4)]
    for t in threads:
        t.start()
    work(0)
    for t in threads:
        t.join()
    assert not wrong and len(done) == 4
    assert c.fault() == 0


def test_first_calls_inside_a_capture_and_two_graphs():
    # every kind of call captured; two graphs of one cache's attention replayed at once
    c, data = ca.fill([3000, 70, 555], 4, 128, 32)
    q = ca.randn(1, 3, 16, 128)
    sl, st = ints([0, 1, 2]), ints([0, 1, 2, 3])
    graphs, outs = [], []
    for _ in range(2):
        g, out = torch.cuda.CUDAGraph(), torch.zeros_like(q)
        with torch.cuda.graph(g):
            c.attention(q, sl, st, out=out)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        c.attention(q, sl, st)  # and an eager one meanwhile
        torch.cuda.synchronize()
        for out in outs:
            ca.check(out, q, data, [0, 1, 2], [0, 1, 2, 3], None, None, 128 ** -0.5, out)


def test_runs_without_a_pause():
    # steps in a row, each launch beginning during the one before, equal the same steps with a pause
    def steps(pause):
        c = pb.Cache.empty(2, 200, 16, 2, 64, 6, 30)
        c.k.zero_()
        c.v.zero_()
        got = []
        sl = ints([3, 0, 5, 1])
        st = ints([0, 5, 6, 9, 16])
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        for step in range(12):
            x = torch.randn(2, 16, 8, 64, generator=g, device="cuda").to(torch.bfloat16)
            q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
            calls = [lambda: c.extend(sl, st), lambda: c.write(k, v, sl, st),
                     lambda: got.append(c.attention(q[0], sl, st, layer=0)),
                     lambda: got.append(c.attention(q[1], sl, st, layer=1)),
                     lambda: got.append(pb.prompt_attention(q[1], k[1], v[1], st)),
                     lambda: c.keep(sl, st, ints([0, 2, 4, 0, 0, 0, 1, 2, 0, 0, 1, 2, 3, 6, 0, 0]),
                                    ints([3, 1, 2, 4])),
                     lambda: c.fork(ints([3, 0]), ints([2, 4])),
                     lambda: c.truncate(ints([2, 4]), ints([0, 7]))]
            for call in calls:
                call()
                if pause:
                    torch.cuda.synchronize()
        assert c.fault() == 0
        return got + [c.k, c.v, c.lengths, c.refs]

    for a, b in zip(steps(True), steps(False)):
        assert torch.equal(a, b)
