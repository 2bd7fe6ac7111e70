"""Heads of zeros, and a norm's eps at the end of what its backward pass takes."""

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


@pytest.mark.parametrize("eps", [2.0 ** -80, 1e-12, 1e-6])
@pytest.mark.parametrize("dh", [64, 80, 128])
def test_heads_of_zeros(eps, dh):
    # x = 0: n = 0, dgamma = 0, dx = rstd dy gamma with rstd = eps^(-1/2) (2^-20.5 for the fast
    # functions of the angle at most, and the roundings of a product of three: 2^-19), bf16
    g = torch.Generator(device="cuda").manual_seed(dh)
    x = torch.zeros(2, 9, 3, dh, dtype=torch.bfloat16, device="cuda")
    x[:, 4:] = torch.randn(2, 5, 3, dh, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(2, 9, 3, dh, generator=g, device="cuda").to(torch.bfloat16)
    gamma = (1 + torch.rand(dh, generator=g, device="cuda")).to(torch.bfloat16)
    pos = torch.zeros(1, 2, 9, dtype=torch.int32, device="cuda")
    rope = pb.Rope(dh)
    y, _ = pb.qk_norm_rope(rope, x, None, pos, gamma, eps=eps)
    assert (y[:, :4] == 0).all() and torch.isfinite(y.float()).all()
    dx, _, dgamma, _ = pb.qk_norm_rope_backward(rope, x, None, pos, dy, None, gamma, eps=eps)
    want = dy.double() * gamma.double() * eps ** -0.5
    room = (2.0 ** -8 + 2.0 ** -18) * want.abs()
    assert ((dx.double() - want).abs() <= room)[:, :4].all()
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dgamma).all()
    alone = pb.qk_norm_rope_backward(rope, x[:, :4], None, pos[:, :, :4].contiguous(),
                                     dy[:, :4], None, gamma, eps=eps)[2]
    assert (alone == 0).all()


def test_training_with_a_vanishing_eps_is_refused_before_it_begins():
    wl = Workload("eps", 1, 33, 256, 2, 128, 512, 16, 1, 0.02)
    x, params = inputs.make_layer(wl, 0, seed=1, device="cuda", biases=True)
    block = pb.ParallelBlock(pb.make_dims(wl), params)
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    scratch = pb.new_train_scratch(block.dims)
    block.set_qk_norm_rope(pb.Rope(128), gamma, gamma, 1e-30, training=True)
    with pytest.raises(pb.PbError, match="2\\^-80"):
        block.forward_train(x, scratch)
    assert torch.isfinite(block.forward(x).float()).all()  # the forward pass takes any eps
    block.set_qk_norm_rope(pb.Rope(128), gamma, gamma, 2.0 ** -80, training=True)
    block.forward_train(x, scratch)
    grads = block.backward(x, x.clone(), scratch)
    assert all(torch.isfinite(v.float()).all() for v in grads.values())
