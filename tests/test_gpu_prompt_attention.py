"""GPU parity of the attention of packed prompts against the formula in 64 bits, over head sizes,
groups, ragged lengths, windows, layouts and buffers with rows in no sequence.

Tolerance. out_i = sum_j p_j v_j with the softmax's weights p. The kernel rounds each weight to bf16
(half a step, 2^-8 of it; the sum that divides is of the unrounded ones) and the result once (2^-8 of
it). In fp32: a score is a sum of dh products, off by dh 2^-23 sum |q_d k_d| at most (the tensor core
cuts sums off, a unit in the last place each), times the scale: with the values used, |q|, |k| < 6 and
dh = 128, sum |q_d k_d| / sqrt(dh) stays below 40, so a weight is off by 128 x 2^-23 x 40 < 2^-10 of
itself in the worst case; exp2, the sums of weights and of products add less than 2^-12 each. With
A_i = sum_j p_j |v_j|: |err| <= 2^-8 |out_i| + (2^-8 + 2 (2^-10 + 2^-12)) A_i (a weight's error
counts in the sum above and below the line), and a value below bf16's normal range cannot matter."""

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


def randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").clamp(-5.9, 5.9).to(torch.bfloat16)


def reference(q, k, v, first, n, window, scale):
    """(out, A) in 64 bits of the sequence of n tokens from `first` on."""
    rows = slice(first, first + n)
    g = q.shape[1] // k.shape[1]
    qd = q[rows].double().transpose(0, 1)
    kd, vd = (t[rows].double().transpose(0, 1).repeat_interleave(g, 0) for t in (k, v))
    i = torch.arange(n, device="cuda")
    gap = i.view(-1, 1) - i
    s = (qd @ kd.transpose(1, 2)) * scale
    s = s.masked_fill((gap < 0) | (gap >= (window or n)), float("-inf"))
    p = torch.softmax(s, -1)
    return (p @ vd).transpose(0, 1), (p @ vd.abs()).transpose(0, 1)


def check(out, q, k, v, starts, window=None, scale=None, before=None):
    """`starts`: a list. Rows in no sequence must be `before`'s, bit for bit."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    left = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    for a, z in zip(starts, starts[1:]):
        if z > a:
            left[a:z] = False
            want, size = reference(q, k, v, a, z - a, window, scale)
            got = out[a:z].double()
            bar = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -11) * size
            assert bool(((got - want).abs() <= bar).all()), (a, z, float(
                ((got - want).abs() - bar).max()))
    if before is not None:
        assert torch.equal(out[left].view(torch.int16), before[left].view(torch.int16))


def starts_of(lengths, at=0):
    s = [at]
    for n in lengths:
        s.append(s[-1] + n)
    return s


def run(lengths, hq, hk, dh, window=None, scale=None, head_pad=0, tail=0, at=0, seed=0, packed=True,
        nan=True):
    s = starts_of(lengths, at)
    t = s[-1] + tail
    if packed:
        buf = randn(seed, t, hq + 2 * hk, dh)
        q, k, v = buf[:, :hq], buf[:, hq:hq + hk], buf[:, hq + hk:]
    else:
        q, k, v = randn(seed, t, hq, dh), randn(seed + 1, t, hk, dh), randn(seed + 2, t, hk, dh)
    if nan:  # rows in no sequence hold anything
        for x in (q, k, v):
            x[:at] = float("nan")
            x[s[-1]:] = float("inf")
    out = randn(seed + 3, t, hq, dh)
    before = out.clone()
    got = pb.prompt_attention(q, k, v, torch.tensor(s, dtype=torch.int32, device="cuda"),
                              window=window, scale=scale, out=out)
    assert got is out
    check(out, q, k, v, s, window, scale, before)


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 127, 128, 129, 255, 256, 257, 511, 640])
def test_one_sequence(dh, n):
    run([n], 2, 2, dh, tail=3)


@pytest.mark.parametrize("dh,hq,hk", [(128, 8, 2), (64, 20, 5), (128, 6, 2), (64, 7, 1), (128, 8, 1),
                                      (64, 32, 1), (64, 96, 1), (64, 128, 1), (128, 33, 3),
                                      (64, 65, 1), (128, 3, 3)])
def test_groups(dh, hq, hk):
    run([1, 77, 0, 300, 128, 5], hq, hk, dh, tail=40, at=9)


@pytest.mark.parametrize("window", [1, 2, 16, 127, 128, 129, 300, 2 ** 31 - 1])
@pytest.mark.parametrize("hq,hk", [(2, 2), (8, 2)])
def test_windows(window, hq, hk):
    run([513, 1, 200, 0, 0, 64, 700], hq, hk, 64, window=window)
    run([260, 900], hq, hk, 128, window=window, packed=False)


def test_many_sequences():
    # more than a round of items for every SM, lengths of all kinds
    lengths = [(i * 37) % 190 for i in range(300)]
    run(lengths, 8, 4, 64, tail=11)


def test_long_sequences():
    run([4096, 1], 4, 1, 128)
    run([3000, 2500], 4, 4, 128, window=1000)


def test_scale():
    run([300, 20], 4, 2, 64, scale=0.3)
    run([300, 20], 4, 2, 128, scale=1e-3)


def test_layouts():
    # [heads, tokens, dh] storage, rows with gaps, a single head, out as a view
    t, hq, hk, dh = 333, 6, 3, 64
    s = [0, 100, 333]
    st = torch.tensor(s, dtype=torch.int32, device="cuda")
    q = randn(1, hq, t, dh).transpose(0, 1)
    k = randn(2, t, hk, 2 * dh)[:, :, dh:]
    v = randn(3, 2 * t, hk, dh)[::2]
    out = torch.zeros(hq, t, dh + 8, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[:, :, :dh]
    check(pb.prompt_attention(q, k, v, st, out=out), q, k, v, s)
    q1, k1 = randn(4, t, 1, dh), randn(5, t, 1, dh)
    check(pb.prompt_attention(q1, k1, k1), q1, k1, k1, [0, t])


def test_other_sequences_reach_nothing():
    # whatever one sequence holds, its neighbours' results keep their bits
    hq, hk, dh = 8, 2, 128
    s = [0, 130, 200, 460]
    st = torch.tensor(s, dtype=torch.int32, device="cuda")
    q, k, v = randn(1, 460, hq, dh), randn(2, 460, hk, dh), randn(3, 460, hk, dh)
    want = pb.prompt_attention(q, k, v, st)
    for bad in (float("nan"), float("inf"), -3e38):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for x in (q2, k2, v2):
            x[130:200] = bad
        got = pb.prompt_attention(q2, k2, v2, st)
        assert torch.equal(got[:130], want[:130]) and torch.equal(got[200:], want[200:])


def test_large_scores():
    # weights of one key: rows whose maximum moves by far more than the rescaling step
    t, dh = 600, 128
    q, k, v = randn(1, t, 2, dh), randn(2, t, 2, dh), randn(3, t, 2, dh)
    q, k = (q.float() * 8).to(torch.bfloat16), (k.float() * 4).to(torch.bfloat16)
    out = pb.prompt_attention(q, k, v)
    # sum |q_d k_d| scale is 32 times larger here: a weight is off by 2^-5 of itself at most
    want, size = reference(q, k, v, 0, t, None, dh ** -0.5)
    bar = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -4) * size
    assert bool(((out.double() - want).abs() <= bar).all())
    # and equal scores: the mean of the values seen
    z = torch.zeros_like(q)
    out = pb.prompt_attention(z, k, v).double()
    mean = v.double().cumsum(0) / torch.arange(1, t + 1, device="cuda").view(-1, 1, 1)
    size = v.double().abs().cumsum(0) / torch.arange(1, t + 1, device="cuda").view(-1, 1, 1)
    # a weight is exactly 1: only the sum and the result's rounding
    assert bool(((out - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -12 * size).all())


def test_starts_outside_and_falling():
    # starts outside [0, tokens] are moved there; falling ones write nothing outside
    q, k, v = randn(1, 200, 4, 64), randn(2, 200, 2, 64), randn(3, 200, 2, 64)
    st = torch.tensor([-50, 100, 100000], dtype=torch.int32, device="cuda")
    check(pb.prompt_attention(q, k, v, st), q, k, v, [0, 100, 200])
    guard = torch.zeros(600, 4, 64, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = torch.tensor([0, 200, 0, 200, 0, 200, 0, 200], dtype=torch.int32, device="cuda")
    pb.prompt_attention(q, k, v, st, out=guard[200:400], status=status)
    torch.cuda.synchronize()
    assert not guard[:200].any() and not guard[400:].any()


def test_stream_and_graph():
    q, k, v = randn(1, 700, 8, 128), randn(2, 700, 2, 128), randn(3, 700, 2, 128)
    s = [0, 300, 301, 700]
    st = torch.tensor(s, dtype=torch.int32, device="cuda")
    want = pb.prompt_attention(q, k, v, st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pb.prompt_attention(q, k, v, st, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pb.prompt_attention(q, k, v, st, out=out)
    # the lengths are read when the graph runs
    for s in ([0, 300, 301, 700], [0, 0, 699, 700], [5, 10, 200, 600]):
        st.copy_(torch.tensor(s, dtype=torch.int32))
        out.fill_(7.0)
        before = out.clone()
        graph.replay()
        check(out, q, k, v, s, before=before)


def test_scratch_contents_and_repeat():
    # scratch holds anything before the call, and the same call gives the same bits
    lengths = [(i * 53) % 400 for i in range(40)]
    s = starts_of(lengths)
    q, k, v = randn(1, s[-1], 8, 64), randn(2, s[-1], 4, 64), randn(3, s[-1], 4, 64)
    st = torch.tensor(s, dtype=torch.int32, device="cuda")
    scratch = torch.full((pb.prompt_attention_scratch_bytes(s[-1], 40),), 255, dtype=torch.uint8,
                         device="cuda")
    first = pb.prompt_attention(q, k, v, st, scratch=scratch)
    for _ in range(3):
        assert torch.equal(pb.prompt_attention(q, k, v, st, scratch=scratch), first)


def test_nothing_to_do():
    q = randn(1, 5, 4, 64)
    out = torch.full_like(q, 3.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")  # no sequences
    assert bool((pb.prompt_attention(q, q, q, st, out=out) == 3).all())
    st = torch.tensor([5, 5, 5], dtype=torch.int32, device="cuda")  # empty ones
    assert bool((pb.prompt_attention(q, q, q, st, out=out) == 3).all())
    assert pb.prompt_attention(q[:0], q[:0], q[:0]).shape == (0, 4, 64)
