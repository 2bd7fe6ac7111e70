"""GPU parity of the query/key norm and rotation and its backward pass against the formulas in
64 bits, over head sizes, partial rotations, axes, pairings, layouts and odd token counts.

Tolerances. A result y (or gradient) is computed in fp32 and rounded once to bf16: half a step,
2^-8 |y|. The fp32 part: a pair's rotation adds at most |a| + |b| <= 2 max of the head's
values, each with a few roundings and the sine's error (2^-33 of a turn, its fp32 rounding
2^-25 turn = 2e-7 rad, sincospi 2 units): 2^-20 of the head's largest value covers it. The
norm's mean adds dh roundings of 2^-24, halved by the square root: dh 2^-24 <= 2^-16 relative
at dh = 256. So |err| <= 2^-8 |y| + 2^-15 max|head|. dgamma is a sum of fp32 products: 2^-24
per addition of partial sums no larger than the sum of magnitudes A; the longest chain (a
lane's tokens, shuffles, partial sums of blocks) stays below 512 additions and each term has
the head's relative 2^-15: |err| <= 2^-14 A."""

import math

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


def angles(dh, rot, sections, ladder, pos, theta=10000.0, inv_freq=None):
    """float64 [batch, seq, rot / 2]."""
    f, axis = [], []
    for a, n in enumerate(sections):
        for j in range(n):
            i = len(f)
            e = i / (rot // 2) if ladder == "shared" else j / n
            f.append(theta ** -e if inv_freq is None else inv_freq[i])
            axis.append(a)
    p = pos.double()
    if not f:
        return p.new_zeros(p.shape[1:] + (0,))
    return torch.stack([p[a] * w for a, w in zip(axis, f)], -1)


def rotate(y, ang, rot, pairing, back=False):
    out = y.clone()
    c, s = torch.cos(ang).unsqueeze(2), torch.sin(ang).unsqueeze(2)
    if back:
        s = -s
    ia = slice(0, rot // 2) if pairing == "halves" else slice(0, rot, 2)
    ib = slice(rot // 2, rot) if pairing == "halves" else slice(1, rot, 2)
    a, b = y[..., ia], y[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = a * s + b * c
    return out


def forward64(x, gamma, eps, ang, rot, pairing):
    y = x.double()
    if gamma is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * gamma.double()
    return rotate(y, ang, rot, pairing)


def backward64(x, gamma, eps, dy, ang, rot, pairing):
    d = rotate(dy.double(), ang, rot, pairing, back=True)
    if gamma is None:
        return d, None, None
    xd = x.double()
    rstd = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + eps)
    n = xd * rstd
    g = d * gamma.double()
    dx = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    return dx, (d * n).sum((0, 1, 2)), (d * n).abs().sum((0, 1, 2))


def close(got, ref, what, scale=None):
    top = (ref if scale is None else scale).abs().amax(-1, keepdim=True)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.float()).all(), what
    bad = err > 2.0 ** -8 * ref.abs() + 2.0 ** -15 * top + 1e-30
    assert not bad.any(), (what, int(bad.sum()), float(err.max()))


def tensors(b, s, nq, nk, dh, layout, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def new(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    if layout == "packed":  # q, k of one [q | k | v] buffer
        buf = new(b, s, nq + 2 * nk, dh)
        return buf[:, :, :nq], buf[:, :, nq:nq + nk], buf
    if layout == "heads_first":  # [batch, heads, seq, dh]
        return new(b, nq, s, dh).transpose(1, 2), new(b, nk, s, dh).transpose(1, 2), None
    return new(b, s, nq, dh), new(b, s, nk, dh), None


CASES = [
    # b, s, nq, nk, dh, rot, pairing, sections, ladder, layout
    (1, 1, 1, 1, 64, 64, "halves", (32,), "shared", "apart"),
    (3, 1, 32, 8, 128, 128, "halves", (64,), "shared", "packed"),
    (2, 33, 5, 1, 128, 128, "adjacent", (16, 24, 24), "per_axis", "packed"),
    (2, 130, 4, 2, 64, 32, "halves", (4, 6, 6), "shared", "heads_first"),
    (1, 257, 3, 3, 128, 64, "adjacent", (32,), "shared", "apart"),
    (1, 7, 2, 1, 96, 96, "halves", (10, 38), "per_axis", "apart"),
    (1, 19, 2, 2, 80, 48, "adjacent", (24,), "shared", "packed"),
    (2, 5, 3, 1, 256, 256, "halves", (32, 32, 32, 32), "shared", "apart"),
    (1, 9, 2, 1, 16, 16, "adjacent", (8,), "shared", "apart"),
    (1, 9, 70, 1, 32, 0, "halves", (0,), "shared", "apart"),
    (5, 1000, 2, 1, 64, 64, "halves", (32,), "shared", "packed"),
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_forward_and_backward(case, norm):
    b, s, nq, nk, dh, rot, pairing, sections, ladder, layout = case
    q, k, buf = tensors(b, s, nq, nk, dh, layout, 1)
    dq, dk, _ = tensors(b, s, nq, nk, dh, layout, 2, 1e-3)
    g = torch.Generator(device="cuda").manual_seed(3)
    gq, gk = [(1 + 0.3 * torch.randn(dh, generator=g, device="cuda")).to(torch.bfloat16)
              if norm else None for _ in range(2)]
    pos = torch.randint(-50, 200000, (len(sections), b, s), generator=g, device="cuda",
                        dtype=torch.int32)
    rope = pb.Rope(dh, rot_dim=rot, pairing=pairing, sections=list(sections), ladder=ladder)
    before = None if buf is None else buf.clone()
    yq, yk = pb.qk_norm_rope(rope, q, k, pos, gq, gk, eps=1e-5)
    ang = angles(dh, rot, sections, ladder, pos)
    for got, x, gam in ((yq, q, gq), (yk, k, gk)):
        close(got, forward64(x, gam, 1e-5, ang, rot, pairing), "forward")
    oq, ok, dgq, dgk = pb.qk_norm_rope_backward(rope, q, k, pos, dq, dk, gq, gk, eps=1e-5)
    for got, x, gam, dy, dg in ((oq, q, gq, dq, dgq), (ok, k, gk, dk, dgk)):
        ref, dref, size = backward64(x, gam, 1e-5, dy, ang, rot, pairing)
        # the terms of dx before they cancel: rstd times the turned gradient
        scale = ref
        if norm:
            rstd = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-5)
            scale = rstd * rotate(dy.double(), ang, rot, pairing, True) * gam.double() + 0 * ref
            scale = scale.abs() + ref.abs()
        close(got, ref, "backward", scale)
        if norm:
            assert ((dg.double() - dref).abs() <= 2.0 ** -14 * size + 1e-30).all()
        else:
            assert dg is None
    if buf is not None:
        assert torch.equal(buf, before)


def test_in_place_leaves_the_rest_of_the_buffer():
    q, k, buf = tensors(2, 65, 6, 2, 128, "packed", 5)
    rope = pb.Rope(128)
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    want = pb.qk_norm_rope(rope, q, k, None, gamma, gamma)
    v = buf[:, :, 8:].clone()
    got = pb.qk_norm_rope(rope, q, k, None, gamma, gamma, out_q=q, out_k=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, :, 8:], v)
    # the backward in place of the incoming gradient, and in place of the forward's input
    x, xk, _ = tensors(2, 65, 6, 2, 128, "packed", 6)
    d, dk, _ = tensors(2, 65, 6, 2, 128, "packed", 7, 1e-3)
    ref = pb.qk_norm_rope_backward(rope, x, xk, None, d, dk, gamma, gamma)
    d2, x2 = d.clone(), x.clone()
    a = pb.qk_norm_rope_backward(rope, x, None, None, d2, None, gamma, out_dq=d2)
    assert torch.equal(a[0], ref[0]) and torch.equal(a[2], ref[2]) and a[1] is None
    a = pb.qk_norm_rope_backward(rope, x2, None, None, d, None, gamma, out_dq=x2)
    assert torch.equal(x2, ref[0])


def test_one_tensor_only_and_own_frequencies():
    _, k, _ = tensors(2, 17, 1, 3, 64, "apart", 8)
    freq = [0.5 / (1 + i) for i in range(32)]
    rope = pb.Rope(64, inv_freq=freq)
    none, yk = pb.qk_norm_rope(rope, None, k)
    assert none is None
    pos = torch.arange(17, device="cuda", dtype=torch.int32).expand(1, 2, 17)
    ang = angles(64, 64, (32,), "shared", pos, inv_freq=freq)
    close(yk, forward64(k, None, 0, ang, 64, "halves"), "own frequencies")
    # frequencies of whole turns more, and of the other sign, turn alike
    more = pb.Rope(64, inv_freq=[f + 2 * math.pi * 3 for f in freq])
    assert torch.equal(pb.qk_norm_rope(more, None, k)[1], yk) or \
        (pb.qk_norm_rope(more, None, k)[1].float() - yk.float()).abs().max() <= 2.0 ** -7 * 4


def test_far_positions():
    # the ends of the int32 range, against angles reduced in exact arithmetic
    from fractions import Fraction
    q, _, _ = tensors(1, 6, 2, 1, 128, "apart", 9)
    at = [2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, -1, 0, 123456789]
    pos = torch.tensor(at, device="cuda", dtype=torch.int32).view(1, 1, 6)
    y, _ = pb.qk_norm_rope(pb.Rope(128), q, None, pos)
    ang = torch.empty(1, 6, 64, dtype=torch.float64)
    two_pi = 2 * math.pi
    for i in range(64):
        turn = Fraction((10000.0 ** -(i / 64)) / two_pi)
        for j, p in enumerate(at):
            ang[0, j, i] = float((turn * p) % 1) * two_pi
    close(y, forward64(q, None, 0, ang.cuda(), 128, "halves"), "far positions")


def test_zero_rows_and_non_finite_heads_stay_apart():
    q, _, _ = tensors(1, 4, 3, 1, 64, "apart", 10)
    q[0, 1, 1] = 0
    q[0, 2, 0, 5] = float("nan")
    q[0, 3, 2, 7] = float("inf")
    gamma = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, _ = pb.qk_norm_rope(pb.Rope(64), q, None, None, gamma)
    assert torch.equal(y[0, 1, 1], torch.zeros_like(y[0, 1, 1]))
    assert y[0, 2, 0].isnan().all()
    fine = torch.ones(4, 3, dtype=torch.bool)
    fine[2, 0] = fine[3, 2] = False
    assert torch.isfinite(y[0][fine.cuda()].float()).all()


def test_accumulate_repeat_and_no_tokens():
    rope = pb.Rope(128)
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    q, k, _ = tensors(2, 300, 8, 2, 128, "packed", 11)
    dq, dk, _ = tensors(2, 300, 8, 2, 128, "packed", 12)
    a = pb.qk_norm_rope_backward(rope, q, k, None, dq, dk, gamma, gamma)
    b = pb.qk_norm_rope_backward(rope, q, k, None, dq, dk, gamma, gamma)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    acc = [x.clone() for x in a[2:]]
    pb.qk_norm_rope_backward(rope, q, k, None, dq, dk, gamma, gamma, dgamma_q=acc[0],
                             dgamma_k=acc[1], accumulate=True)
    for x, y in zip(acc, a[2:]):
        assert ((x - 2 * y).abs() <= 1e-5 * y.abs().max()).all()
    e = torch.empty(0, 5, 4, 128, dtype=torch.bfloat16, device="cuda")
    out = pb.qk_norm_rope_backward(rope, e, None, None, e, None, gamma,
                                   dgamma_q=acc[0])
    assert out[0].numel() == 0 and (acc[0] == 0).all()
    assert pb.qk_norm_rope(rope, e, None, None, gamma)[0].numel() == 0


def test_gradient_against_differences():
    # sum(dy * y(x)) along a direction, by central differences of the formula in 64 bits
    g = torch.Generator(device="cuda").manual_seed(13)
    q, _, _ = tensors(1, 3, 2, 1, 64, "apart", 14)
    dy, _, _ = tensors(1, 3, 2, 1, 64, "apart", 15)
    gamma = (1 + 0.2 * torch.randn(64, generator=g, device="cuda")).to(torch.bfloat16)
    pos = torch.tensor([[[3, 700, 41]]], dtype=torch.int32, device="cuda")
    dq, _, dg, _ = pb.qk_norm_rope_backward(pb.Rope(64), q, None, pos, dy, None, gamma)
    ang = angles(64, 64, (32,), "shared", pos)
    for _ in range(4):
        u = torch.randn(q.shape, generator=g, device="cuda", dtype=torch.float64)
        w = torch.randn(64, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4

        def f(t):
            return (dy.double() * forward64(q.double() + t * u, gamma.double() + t * w, 1e-6, ang,
                                            64, "halves")).sum()

        want = (f(h) - f(-h)) / (2 * h)
        got = (dq.double() * u).sum() + (dg.double() * w).sum()
        # 384 gradient values off by 2^-8 of themselves at most
        room = 2.0 ** -8 * (dq.double() * u).abs().sum() + 1e-4 * (dg.double() * w).abs().sum()
        assert abs(want - got) <= room + 1e-5 * abs(want)


def test_graph_and_side_stream():
    rope = pb.Rope(128)
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    q, k, _ = tensors(8, 1, 16, 4, 128, "packed", 16)
    pos = torch.arange(8, device="cuda", dtype=torch.int32).view(1, 8, 1).contiguous()
    oq, ok = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(
        k.shape, dtype=k.dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pb.qk_norm_rope(rope, q, k, pos, gamma, gamma, out_q=oq, out_k=ok)
    for step in range(3):
        pos += 1000
        graph.replay()
        want = pb.qk_norm_rope(rope, q, k, pos, gamma, gamma)
        torch.cuda.synchronize()
        assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])


def test_refused_calls():
    rope = pb.Rope(64)
    q, k, buf = tensors(2, 8, 4, 2, 64, "packed", 17)
    gamma = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pb.PbError, match="overlap"):
        pb.qk_norm_rope(rope, q, k, out_q=buf[:, :, 1:5], out_k=k)
    with pytest.raises(pb.PbError, match="overlap"):
        pb.qk_norm_rope(rope, q, k, out_q=buf[:, :, 4:8])  # k's columns
    with pytest.raises(pb.PbError, match="overlap"):
        out = torch.empty(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda").expand(2, 8, 4, 64)
        pb.qk_norm_rope(rope, q, None, out_q=out)
    with pytest.raises(ValueError):
        pb.qk_norm_rope(rope, q.float(), k)
    with pytest.raises(ValueError):
        pb.qk_norm_rope(rope, q, k, gamma_q=gamma.float())
    with pytest.raises(ValueError):
        pb.qk_norm_rope(rope, q.cpu(), k)
    with pytest.raises(ValueError):
        pb.qk_norm_rope(rope, q, k, positions=torch.zeros(1, 2, 7, dtype=torch.int32,
                                                          device="cuda"))
    with pytest.raises(pb.PbError, match="eps"):
        pb.qk_norm_rope(rope, q, k, gamma_q=gamma, eps=0.0)
    with pytest.raises(pb.PbError, match="NULL"):
        pb.qk_norm_rope_backward(rope, None, None, None, q, None, gamma)
