"""Sums over long contractions keep to the result's type: the tensor core cuts partial sums off
towards zero, so a chain of them shrinks the result, by 1.05e-9 of it for each k (measured: 8.6e-6
of the norm at 8192), before its rounding, which does not lean to either side. The lean is what is
measured: <y - ref, ref> / <ref, ref>, in which N roundings of at most u (fp16 2^-11, bf16 2^-8)
average to u / sqrt(N) at most (one standard deviation, and they are not all in step).

An accumulator's chain ends after 7,168 k for an fp16 result and 57,344 for a bf16 one, where the
lean is u / 64; the segments are then added in rounded fp32 additions. Allowed: twice that,
and three standard deviations of the roundings. One chain over all of k leans by 1.4e-4 at 131,072
(fp16: 3e-5 is allowed) and by 5.5e-4 at 524,288 (bf16: 1.8e-4)."""

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
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt,k,u", [(torch.float16, 131072, 2.0 ** -11),
                                    (torch.bfloat16, 524288, 2.0 ** -8)], ids=["fp16", "bf16"])
@pytest.mark.parametrize("split", [False, True])
def test_long_contraction_does_not_lean(dt, k, u, split):
    m, n = 96, 512
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(m, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).to(dt)
    ref = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for c in range(0, k, 65536):
        ref += x[:, c:c + 65536].double() @ w[:, c:c + 65536].double().t()
    scratch = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device="cuda") if split \
        else None
    y = pb.linear(x, w, layout=pb.PB_WEIGHT_OUT_IN, scratch=scratch)
    # dx = dy w^T contracts over w's other side
    back, _, _ = pb.linear_backward(x, None, w, layout=pb.PB_WEIGHT_IN_OUT, need_dw=False,
                                    scratch=scratch)
    for got in (y, back):
        lean = float(((got.double() - ref) * ref).sum() / (ref * ref).sum())
        assert abs(lean) <= 2 * u / 64 + 3 * u * (m * n) ** -0.5, lean


@pytest.mark.parametrize("scratch", [False, True])
def test_segments_with_an_epilogue(scratch):
    # Bias, pre-activation, GELU and residual behind a sum of several segments. A chain cuts off at
    # most 2^-22 S an instruction of 16 k (S = sum |x| |w| + |b|), at most 7,168 k of them; the
    # segments' and split parts' additions: 100 more. GELU changes by at most 1.13 a unit.
    m, n, k = 96, 264, 20000
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(m, k, generator=g, device="cuda").half()
    w = (torch.randn(k, n, generator=g, device="cuda") * k ** -0.5).half()
    b = torch.randn(n, generator=g, device="cuda").half()
    r = torch.randn(m, n, generator=g, device="cuda").half()
    pre = torch.empty(m, n, dtype=torch.float16, device="cuda")
    work = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device="cuda") if scratch \
        else None
    y = pb.linear(x, w, b, residual=r, activation="gelu", pre=pre, scratch=work)
    z = x.double() @ w.double() + b.double()
    room = (7168 / 16 + 100) * 2.0 ** -22 * (x.double().abs() @ w.double().abs() + b.double().abs())
    half = 2.0 ** -11 * (1 + 2.0 ** -6)
    assert ((pre.double() - z).abs() <= room + half * z.abs() + 2.0 ** -25).all()
    ref = z * torch.special.ndtr(z) + r.double()
    room = 1.13 * room + 2.0 ** -19 * (1 + z.abs())
    assert ((y.double() - ref).abs() <= room + half * ref.abs() + 2.0 ** -25).all()
