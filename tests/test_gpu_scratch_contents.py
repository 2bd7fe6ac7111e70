"""No result depends on what scratch memory or a result's buffer held before the call.

Every byte of both is set to 0xFF, which reads as NaN in every type used, against the same call
on zeroed memory: values that a kernel reads without having written them (rows behind the last
query of a tile, sums that are multiplied by a zero probability) turn up as NaN. Results are
equal bit for bit, except where dq enters: it is summed by atomic additions whose order varies.
fp32 sums of a few dozen terms in another order are off by 1e-6 of the largest, so a bf16 value
that lies near a rounding border may move by one step, 2^-8 of itself: 1e-2 of the largest."""

import pytest
import torch

from transformer_block_gb300 import inputs, pb
from transformer_block_gb300.configs import Workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


def filled(n, byte):
    return torch.full((n,), byte, dtype=torch.uint8, device="cuda")


SHAPES = [(1, 1, 256, 2, 128, 512, 4), (2, 65, 256, 2, 128, 512, 64),
          (3, 33, 128, 2, 64, 256, 5), (2, 130, 256, 4, 64, 512, 100)]


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("variant", [0, 1])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"b{s[0]}s{s[1]}dh{s[4]}")
def test_block_training_ignores_scratch_contents(shape, variant, rotated):
    wl = Workload("scratch", *shape, 1, 0.02, variant=variant)
    x, params = inputs.make_layer(wl, 0, seed=1, device="cuda", biases=True)
    block = pb.ParallelBlock(pb.make_dims(wl), params)
    if rotated:
        gamma = torch.linspace(0.5, 1.5, wl.head_dim, device="cuda").to(torch.bfloat16)
        block.set_qk_norm_rope(pb.Rope(wl.head_dim), gamma, gamma, 1e-5, training=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    dy = torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16)
    runs = []
    for byte in (0, 0xFF):
        scratch = filled(pb.train_scratch_bytes(block.dims), byte)
        y = block.forward_train(x, scratch).clone()
        grads = dict(block.backward(x, dy, scratch))
        if rotated:
            grads.update({k: v.clone() for k, v in block.rope_grads.items()})
        runs.append((y, grads))
    (y0, g0), (y1, g1) = runs
    assert torch.equal(y0, y1)
    for name, want in g0.items():
        assert torch.isfinite(g1[name].float()).all(), name
        gap = (g1[name].double() - want.double()).abs().max()
        assert float(gap) <= 1e-2 * float(want.double().abs().max()), name
    assert block.status() == 0


@pytest.mark.parametrize("m,K", [(1, 1032), (7, 4104), (40, 1032), (333, 4104), (777, 264)])
@pytest.mark.parametrize("layout", [pb.PB_WEIGHT_IN_OUT, pb.PB_WEIGHT_OUT_IN])
def test_linear_ignores_scratch_contents(m, K, layout):
    N = 264
    g = torch.Generator(device="cuda").manual_seed(m)

    def t(*s):
        return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    x, dy, b = t(m, K), t(m, N), t(N)
    w = t(K, N) if layout == pb.PB_WEIGHT_IN_OUT else t(N, K)
    runs = []
    for byte in (0, 0xFF):
        scratch = filled(pb.linear_scratch_bytes(), byte)
        y = filled(2 * m * N, byte).view(torch.bfloat16).view(m, N)
        pre = filled(2 * m * N, byte).view(torch.bfloat16).view(m, N)
        pb.linear(x, w, b, activation="gelu", layout=layout, out=y, pre=pre, scratch=scratch)
        dw = filled(4 * K * N, byte).view(torch.float32).view(w.shape)
        dx = filled(2 * m * K, byte).view(torch.bfloat16).view(m, K)
        db = filled(4 * N, byte).view(torch.float32)
        pb.linear_backward(dy, x, w, layout=layout, bias=True, dx=dx, dw=dw, db=db,
                           scratch=scratch)
        runs.append([y, pre, dx, dw, db])
    for a, b_ in zip(*runs):
        assert torch.equal(a, b_)


def test_norm_and_rotation_gradients_ignore_scratch_contents():
    g = torch.Generator(device="cuda").manual_seed(9)

    def t(heads):
        return torch.randn(2, 33, heads, 80, generator=g, device="cuda").to(torch.bfloat16)
    q, k, dq, dk = t(3), t(1), t(3), t(1)
    gamma = torch.ones(80, dtype=torch.bfloat16, device="cuda")
    runs = []
    for byte in (0, 0xFF):
        out = pb.qk_norm_rope_backward(pb.Rope(80), q, k, None, dq, dk, gamma, gamma,
                                       scratch=filled(pb.qk_norm_rope_scratch_bytes(), byte))
        runs.append([v for v in out if v is not None])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_grad_norm_ignores_scratch_contents():
    g = torch.Generator(device="cuda").manual_seed(11)
    tensors = []
    for n in (1, 777, 70001):
        p = torch.randn(n, generator=g, device="cuda")
        tensors.append({"param": p, "grad": torch.randn(n, generator=g, device="cuda"),
                        **pb.adamw_states(p)})
    opt = pb.AdamW(tensors)
    first = opt.grad_norm(1.0, scratch=filled(opt.scratch_bytes, 0)).clone()
    assert torch.equal(first, opt.grad_norm(1.0, scratch=filled(opt.scratch_bytes, 0xFF)))
