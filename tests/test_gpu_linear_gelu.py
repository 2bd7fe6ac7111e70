"""GELU in the linear layer's epilogue is as exact as its result's type, for few tokens and many.

x = 0, so that the pre-activation is the bias, exactly, and GELU(z) = z Phi(z) is held against its
value in 64 bits relative to its size, in the left tail too, where a Phi with an absolute error
(of 1e-7, say) would be off by 5e-5 at z = -3. Units of 2^-24 of Phi(-a), a = |z|: the exponent of
exp(-a^2 / 2) is off by 2.5 of itself (the rounded square, the product, half for the constant),
which is 2.5 a^2 / 2 = 1.25 a^2 of the exponential; the other factor t P(t) with t = 1 / (1 + a / 4) changes by at most 3.2 times as much
as t, which is off by 3 (a rounded sum, the reciprocal's 2): 10; eight steps of P and its fit:
4; the exponential 4; products and the difference z - z Phi(-z): 4. Together (1.25 a^2 + 22) 2^-24.
The form for few tokens (erfc, 4 units of its last place, an argument rounded 1.5 times, which
counts a^2 + 1 times) is within (1.5 (a^2 + 1) + 10) 2^-24. Bar: (1.5 a^2 + 24) 2^-24, and the
rounding of a 16-bit result. GELU'(z) = Phi(z) + z phi(z): the same share of |Phi| + |z| phi, whose
terms cancel near z = -0.75, and fp16's half step."""

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


def share(z):
    return (1.5 * z * z + 24) * 2.0 ** -24


def every(dt, lo, hi):
    """All values of a 16-bit type from lo to hi."""
    v = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(dt)
    return v[(v.float() >= lo) & (v.float() <= hi)]


# one launch of the few-token kernel, the GEMM, and (k long, tiles few) its split form
@pytest.mark.parametrize("m,k", [(1, 64), (32, 64), (33, 64), (300, 64), (33, 8192)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("wide", [True, False], ids=["fp32 result", "own type"])
def test_gelu_on_both_sides(m, k, dt, wide):
    z = torch.cat([every(dt, -5, -2.0 ** -10), every(dt, 2.0 ** -10, 6)])
    if k > 64:
        z = z[::max(1, z.numel() // 1000)][:1000].contiguous()
    n = z.numel()
    x = torch.zeros(m, k, dtype=dt, device="cuda")
    w = torch.zeros(k, n + -n % 8, dtype=dt, device="cuda")[:, :n]
    scratch = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device="cuda")
    y = pb.linear(x, w, z, activation="gelu", out_dtype=torch.float32 if wide else dt,
                  scratch=scratch)
    zd = z.double()
    ref = zd * torch.special.ndtr(zd)
    half = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[y.dtype]
    room = ref.abs() * (share(zd) + half * (1 + 2.0 ** -6))
    if y.dtype is torch.float16:
        room = room.clamp(min=2.0 ** -25 * (1 + 2.0 ** -6))
    err = (y.double() - ref).abs()
    bad = (err > room).any(0)
    worst = (err / ref.abs()).max(0).values
    assert not bad.any(), (int(bad.sum()), [(float(a), float(b)) for a, b in
                                            zip(zd[bad][:5], worst[bad][:5])])


@pytest.mark.parametrize("m", [32, 33, 300])
def test_gelu_derivative_fp16(m):
    # dy w^T = 1: one output feature, both ones
    z = every(torch.float16, -6, 6)
    k = z.numel()
    dy = torch.zeros(m, 8, dtype=torch.float16, device="cuda")
    dy[:, 0] = 1
    w = torch.zeros(k, 8, dtype=torch.float16, device="cuda")
    w[:, 0] = 1
    pre = torch.empty(m, k + -k % 8, dtype=torch.float16, device="cuda")[:, :k]
    pre.copy_(z.expand(m, k))
    dx, _, _ = pb.linear_backward(dy, None, w, pre=pre, activation="gelu", need_dw=False)
    zd = z.double()
    phi = torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    cdf = torch.special.ndtr(zd)
    ref = cdf + zd * phi
    room = share(zd) * (cdf + zd.abs() * phi) + 2.0 ** -11 * (1 + 2.0 ** -6) * ref.abs()
    room = room.clamp(min=2.0 ** -25 * (1 + 2.0 ** -6))
    err = (dx.double() - ref).abs()
    bad = (err > room).any(0)
    assert not bad.any(), (int(bad.sum()), zd[bad][:5], err.max(0).values[bad][:5])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m", [1, 32, 33, 300])
def test_sigmoid_forms_relative_to_their_size(m, act):
    # z sigmoid(s), s = z or 2 sqrt(2 / pi) (z + 0.044715 z^3). Units of 2^-24 of the value: the
    # exponential's argument -s log2(e) is off by 1.5 of itself for SiLU, where s is exact, and by 8 for
    # the tanh form (six products and sums, four rounded constants at half): times |s|, from the exponent
    # on; the exponential's 4, the sum's 1, the reciprocal's 2, the last product's 1.
    z = torch.cat([every(torch.bfloat16, -20 if act == "silu" else -5, -2.0 ** -10),
                   every(torch.bfloat16, 2.0 ** -10, 20)])
    n = z.numel()
    x = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, n + -n % 8, dtype=torch.bfloat16, device="cuda")[:, :n]
    y = pb.linear(x, w, z, activation=act, out_dtype=torch.float32)
    zd = z.double()
    s = zd if act == "silu" else math.sqrt(8 / math.pi) * (zd + 0.044715 * zd ** 3)
    ref = zd * torch.sigmoid(s)
    room = ((1.5 if act == "silu" else 8) * s.abs() + 9) * 2.0 ** -24 * ref.abs()
    room = torch.where(zd > 0, 9 * 2.0 ** -24 * ref.abs() + room * torch.exp(-s.abs()), room)
    err = (y.double() - ref).abs()
    bad = (err > room).any(0)
    assert not bad.any(), (int(bad.sum()), zd[bad][:5], (err / ref.abs()).max(0).values[bad][:5])
