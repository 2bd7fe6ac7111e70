"""GPU parity of the attention of new tokens over a paged cache against the formula in 64 bits: one
token, lines and trees of drafted ones, head sizes, groups, page sizes, windows, lengths from the
tokens alone to long ones; what the pool holds elsewhere is NaN.

Tolerance, as for packed prompts: the softmax's weights are rounded to bf16 once (2^-8 of each; their
sum is of the unrounded ones) and the result once (2^-8). In fp32 a score is a sum of dh <= 128
products, off by dh 2^-23 sum |q_d k_d| at most, and sum |q_d k_d| / sqrt(dh) stays below 40 for values
below 6, so a weight is off by less than 2^-10 of itself; exp2, the sums and the joining of pieces add
less than 2^-12. With A = sum_j p_j |v_j|: |err| <= 2^-8 |out| + (2^-8 + 2 (2^-10 + 2^-12)) A."""

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


def randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").clamp(-5.9, 5.9).to(torch.bfloat16)


def fill(lengths, hk, dh, page, layers=1, spare=3, seed=0):
    """A cache whose slots hold `lengths` tokens in pages of any order, in its last layer; all else
    is NaN, and the table's rest is no page. Returns it and the sequences' (k, v), [n, hk, dh]."""
    used = [-(-n // page) for n in lengths]
    c = pb.Cache.empty(layers, sum(used) + spare, page, hk, dh, len(lengths), max(used + [1]) + 1)
    c.k.fill_(float("nan"))
    c.v.fill_(float("inf"))
    c.table.fill_(2 ** 31 - 1)
    order = list(range(sum(used) + spare))
    random.Random(seed).shuffle(order)
    data, at = [], 0
    for i, (n, u) in enumerate(zip(lengths, used)):
        mine = ints(order[at:at + u])
        at += u
        c.lengths[i] = n
        c.table[i, :u] = mine
        c.refs[mine.long()] = 1
        kv = [randn(seed * 1000 + 2 * i + j, n, hk, dh) for j in range(2)]
        for pool, x in zip((c.k, c.v), kv):
            pad = torch.full((u * page, hk, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
            pad[:n] = x
            pool[layers - 1, mine.long()] = pad.view(u, page, hk, dh).transpose(1, 2)
        data.append(kv)
    return c, data


def visible(n, count, parents, window):
    """[count, n]: what each new token sees."""
    base = n - count
    seen = torch.zeros(count, n, dtype=torch.bool)
    for t in range(count):
        path, u = [], t
        while True:
            path.append(u)
            up = u - 1 if parents is None else parents[u]
            if up < 0 or up >= u:
                break
            u = up
        d = len(path) - 1
        w = window or n + 1
        seen[t, max(0, base + d - w + 1):base] = True
        for steps, u in enumerate(path):
            seen[t, base + u] = steps < w
    return seen.cuda()


def reference(q, k, v, seen, scale):
    """q [count, hq, dh], k and v [n, hk, dh], seen [count, n]: (out, A) in 64 bits."""
    g = q.shape[1] // k.shape[1]
    qd = q.double().transpose(0, 1)
    kd, vd = (t.double().transpose(0, 1).repeat_interleave(g, 0) for t in (k, v))
    s = (qd @ kd.transpose(1, 2) * scale).masked_fill(~seen, float("-inf"))
    p = torch.softmax(s, -1)
    return (p @ vd).transpose(0, 1), (p @ vd.abs()).transpose(0, 1)


def check(out, q, data, slots, starts, parents, window, scale, before):
    left = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    for slot, a, z in zip(slots, starts, starts[1:]):
        if z == a:
            continue
        left[a:z] = False
        k, v = data[slot]
        seen = visible(len(k), z - a, None if parents is None else parents[a:z], window)
        want, size = reference(q[a:z], k, v, seen, scale)
        bar = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -11) * size
        err = (out[a:z].double() - want).abs()
        assert bool((err <= bar).all()), (slot, a, z, float((err - bar).max()))
    assert torch.equal(out[left].view(torch.int16), before[left].view(torch.int16))


def run(lengths, counts, hq, hk, dh, page, tree=False, window=None, scale=None, at=0, tail=0, seed=0,
        layers=1):
    """`counts` of `lengths`, slot by slot; the call lists the slots in another order."""
    c, data = fill(lengths, hk, dh, page, layers=layers, seed=seed)
    slots = list(range(len(lengths)))
    rng = random.Random(seed)
    rng.shuffle(slots)
    counts = [counts[s] for s in slots]
    starts = [at]
    for n in counts:
        starts.append(starts[-1] + n)
    t = starts[-1] + tail
    parents = None
    if tree:
        parents = [99] * t  # rows in no sequence: anything
        for a, n in zip(starts, counts):
            for j in range(n):
                parents[a + j] = rng.choice([j - 1, rng.randint(-1, j - 1) if j else -1])
    q, out = randn(seed + 7, t, hq, dh), randn(seed + 8, t, hq, dh)
    q[:at] = float("nan")
    q[starts[-1]:] = float("nan")
    before = out.clone()
    got = c.attention(q, ints(slots), ints(starts), parents=None if parents is None else ints(parents),
                      layer=layers - 1, window=window, scale=scale, out=out)
    assert got is out and c.fault() == 0
    check(out, q, data, slots, starts, parents, window, dh ** -0.5 if scale is None else scale, before)


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000])
def test_one_token(dh, n):
    run([n], [1], 4, 2, dh, 16, tail=2)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 128, 1000])
def test_page_sizes(page):
    run([300, 1, 77, 513], [1, 1, 1, 1], 6, 2, 64, page)
    run([300, 40], [1, 5], 8, 1, 128, page, tree=True, seed=1)


@pytest.mark.parametrize("dh,hq,hk", [(128, 1, 1), (64, 20, 5), (128, 6, 2), (64, 7, 1), (128, 40, 8),
                                      (64, 96, 1), (128, 130, 1), (128, 17, 1), (64, 33, 1),
                                      (128, 65, 1)])
@pytest.mark.parametrize("counts", [(1, 1, 1), (7, 2, 0), (64, 33, 5)])
def test_groups_and_counts(dh, hq, hk, counts):
    run([300, 301, 500], list(counts), hq, hk, dh, 24, tree=True, at=3, tail=9)
    run([300, 301, 500], list(counts), hq, hk, dh, 24, at=3, tail=9, seed=1)


@pytest.mark.parametrize("window", [1, 2, 5, 63, 64, 65, 200, 100000, 2 ** 31 - 1])
@pytest.mark.parametrize("tree", [False, True])
def test_windows(window, tree):
    run([700, 1000, 70], [16, 16, 16], 8, 2, 64, 16, tree=tree, window=window)
    run([700, 64, 300], [1, 20, 60], 4, 1, 128, 40, tree=tree, window=window, seed=1)


def test_new_tokens_alone():
    # nothing cached before them: whole prompts through the cache
    run([1, 64, 5], [1, 64, 5], 4, 2, 64, 16)
    run([64, 64, 3], [64, 64, 3], 4, 2, 64, 16, tree=True)
    run([200, 130, 200], [200, 130, 200], 4, 2, 128, 16)


def test_pieces_of_prompts():
    run([900, 900], [513, 700], 8, 2, 128, 64)
    run([900, 900], [513, 700], 6, 6, 64, 20, window=100)


def test_batches():
    rng = random.Random(2)
    lengths = [rng.randint(40, 900) for _ in range(200)]
    run(lengths, [1] * 200, 8, 2, 128, 16, layers=2)
    run(lengths, [rng.randint(0, 20) for _ in range(200)], 8, 4, 64, 32, tree=True)


def test_one_long_sequence():
    # pieces of one item in every block
    run([40000], [1], 4, 1, 128, 64)
    run([50000], [16], 4, 2, 64, 128, tree=True)
    run([30011, 5, 20000], [3, 3, 3], 16, 4, 128, 48)


def test_scale_and_views():
    run([300, 40], [1, 7], 8, 2, 64, 16, scale=0.3)
    c, data = fill([100, 200], 2, 64, 16)
    buf = randn(3, 12, 10, 64)
    q = buf[::2, 1:7]                                    # every other row, some of the heads
    out = torch.zeros(6, 6, 72, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[:, :, :64]
    c.attention(q, ints([1, 0]), ints([0, 2, 6]), out=out)
    check(out, q, data, [1, 0], [0, 2, 6], None, None, 0.125, out)


def test_same_bits_again_and_any_scratch():
    c, data = fill([5000, 333, 20], 4, 128, 32)
    q = randn(1, 24, 16, 128)
    args = (q, ints([2, 0, 1]), ints([0, 8, 16, 24]))
    first = c.attention(*args)
    for byte in (255, 0, 127):
        scratch = torch.full((c.attention_scratch_bytes,), byte, dtype=torch.uint8, device="cuda")
        assert torch.equal(c.attention(*args, scratch=scratch), first)


def test_streams_and_graph():
    c, data = fill([3000, 333, 20], 4, 64, 32)
    q = randn(1, 3, 16, 64)
    sl, st = ints([0, 1, 2]), ints([0, 1, 2, 3])
    want = c.attention(q, sl, st)
    sides = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in sides:  # calls that only read may overlap, each with its scratch
        s.wait_stream(torch.cuda.current_stream())
        got.append(c.attention(q, sl, st, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attention(q, sl, st, out=out)
    for lengths in ([3000, 333, 20], [1, 333, 20], [2999, 64, 1]):
        c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        out.zero_()
        graph.replay()
        cut = [(k[:n], v[:n]) for (k, v), n in zip(data, lengths)]
        check(out, q, cut, [0, 1, 2], [0, 1, 2, 3], None, None, 0.125, out)


@pytest.mark.parametrize("why,slots,starts,parents", [
    (3, [0, 2], [0, 1, 2], None), (3, [-1, 0], [0, 1, 2], None), (4, [0, 1], [0, 2, 1], None),
    (4, [0, 1], [-1, 1, 2], None), (4, [0, 1], [0, 1, 200], None), (4, [1, 0], [0, 31, 32], None),
    (4, [0, 1], [0, 65, 66], True),
])
def test_faults(why, slots, starts, parents):
    c, data = fill([100, 30], 2, 64, 16)
    q = randn(1, 70, 4, 64)
    big = torch.zeros(210, 4, 64, dtype=torch.bfloat16, device="cuda")
    c.attention(q, ints(slots), ints(starts), out=big[70:140],
                parents=None if parents is None else ints([-1] * 70))
    assert c.fault() == pb.PB_ERR_CACHE + 256 * why
    assert not big[:70].any() and not big[140:].any()
    # nothing more happens until the word is cleared
    out = torch.full_like(q, 3.0)
    c.attention(q, ints([0]), ints([0, 1]), out=out)
    assert bool((out == 3).all())
    c.status.zero_()
    c.attention(q, ints([0]), ints([0, 1]), out=out)
    check(out, q, data, [0], [0, 1], None, None, 0.125, torch.full_like(q, 3.0))


def test_pages_and_lengths_at_fault():
    for bad in (-1, 8, 2 ** 31 - 1, -2 ** 31):
        c, data = fill([100], 2, 64, 16, spare=1)
        assert c.refs.numel() == 8
        c.table[0, 3] = bad
        c.attention(randn(1, 1, 4, 64), ints([0]), ints([0, 1]))
        assert c.fault() == pb.PB_ERR_CACHE + 256 * 5
    for bad in (-1, 2 ** 31 - 1, -2 ** 31, 8 * 16 + 1):
        c, data = fill([100], 2, 64, 16, spare=1)
        c.lengths[0] = bad
        c.attention(randn(1, 1, 4, 64), ints([0]), ints([0, 1]))
        assert c.fault() == pb.PB_ERR_CACHE + 256 * 5


def test_strange_parents():
    # a parent that is none, or does not come before its token, is the last token before the new ones
    c, data = fill([50], 1, 64, 16)
    q = randn(1, 6, 2, 64)
    given = [5, -9, 2, 2 ** 31 - 1, -2 ** 31, 4]
    meant = [-1, -1, -1, -1, -1, 4]
    out = c.attention(q, ints([0]), ints([0, 6]), parents=ints(given))
    check(out, q, data, [0], [0, 6], meant, None, 0.125, out)


def test_offsets_past_32_bits():
    # the sequence's pages lie at the end of layers of more than 2^32 values
    hk, dh, page, pages = 8, 128, 64, 70000
    c = pb.Cache.empty(2, pages, page, hk, dh, 1, 10)
    assert c.k[0].numel() > 2 ** 32
    n = 500
    mine = [pages - 1 - 3 * i for i in range(8)]
    c.table[0, :8] = ints(mine)
    c.lengths[0] = n
    kv = [randn(5 + j, n, hk, dh) for j in range(2)]
    for pool, x in zip((c.k, c.v), kv):
        pad = torch.full((8 * page, hk, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
        pad[:n] = x
        for i, at in enumerate(mine):
            pool[1, at] = pad[i * page:(i + 1) * page].transpose(0, 1)
    q = randn(1, 2, 16, dh)
    out = c.attention(q, ints([0]), ints([0, 2]), layer=1)
    assert c.fault() == 0
    check(out, q, [kv], [0], [0, 2], None, None, dh ** -0.5, out)


def test_prompt_then_decoding():
    # the operators together, as a serving loop has them: prompts with rotation, the cache filled,
    # trees of drafts verified and kept, step after step; against the sequences in 64 bits
    hq, hk, dh, page = 8, 2, 128, 16
    rope = pb.Rope(dh)
    lengths = [37, 64, 5]
    starts = [0, 37, 101, 106]
    c = pb.Cache.empty(1, 60, page, hk, dh, 3, 12)
    sl, st = ints([2, 0, 1]), ints(starts)
    x = randn(1, 106, hq + 2 * hk, dh)
    pos = ints([i for n in lengths for i in range(n)]).view(1, 1, -1)
    q, k = pb.qk_norm_rope(rope, x[None, :, :hq], x[None, :, hq:hq + hk], pos)
    q, k, v = q[0], k[0], x[:, hq + hk:]
    out = pb.prompt_attention(q, k, v, st)
    c.extend(sl, st)
    c.write(k, v, sl, st)
    assert c.fault() == 0
    # the prompts' attention is what the cache gives for them
    again = c.attention(q, sl, st)
    rows = [(k[a:z], v[a:z]) for a, z in zip(starts, starts[1:])]
    for o in (out, again):
        check(o, q, rows, [0, 1, 2], starts, None, None, dh ** -0.5, o)
    rng = random.Random(3)
    hist = [[t.clone() for t in kv] for kv in rows]
    for step in range(4):
        counts = [rng.randint(1, 6) for _ in range(3)]
        s = [0]
        for n in counts:
            s.append(s[-1] + n)
        dst = ints(s)
        parents, depth = [], []
        for a, n in zip(s, counts):
            for j in range(n):
                up = rng.randint(-1, j - 1) if j else -1
                depth.append(0 if up < 0 else depth[a + up] + 1)
                parents.append(up)
        y = randn(50 + step, s[-1], hq + 2 * hk, dh)
        base = [len(h[0]) for h in hist]
        pos = ints([base[i] + depth[a] for i in range(3) for a in range(s[i], s[i + 1])])
        q, k = pb.qk_norm_rope(rope, y[None, :, :hq], y[None, :, hq:hq + hk], pos.view(1, 1, -1))
        q, k, v = q[0], k[0], y[:, hq + hk:]
        c.extend(sl, dst)
        c.write(k, v, sl, dst)
        out = c.attention(q, sl, dst, parents=ints(parents))
        full = [(torch.cat([h[0], k[a:z]]), torch.cat([h[1], v[a:z]]))
                for h, a, z in zip(hist, s, s[1:])]
        check(out, q, full, [0, 1, 2], s, parents, None, dh ** -0.5, out)
        # a path from the root down is accepted
        path, kept = [0] * s[-1], []
        for i, (a, n) in enumerate(zip(s, counts)):
            chain, u = [], rng.randint(-1, n - 1)
            while u >= 0:
                chain.append(u)
                u = parents[a + u]
            chain.reverse()
            path[a:a + len(chain)] = chain
            kept.append(len(chain))
            hist[i] = [torch.cat([h, new[a:a + n][chain]]) for h, new in zip(hist[i], (k, v))]
        c.keep(sl, dst, ints(path), ints(kept))
    assert c.fault() == 0
    assert c.lengths.tolist() == [len(hist[1][0]), len(hist[2][0]), len(hist[0][0])]
