"""Buffers of the block's norm that overlap what the same pass reads or writes are refused before
anything runs (the tensors are real, the refused calls enqueue nothing)."""

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


@pytest.fixture(scope="module")
def setup():
    wl = Workload("apart", 2, 40, 256, 2, 128, 512, 16, 1, 0.02)
    x, params = inputs.make_layer(wl, 0, seed=1, device="cuda", biases=True)
    return wl, x, pb.ParallelBlock(pb.make_dims(wl), params)


def set_raw(block, gq, gk, pos, saved, n, dgq, dgk):
    r = pb.pb_block_rope(pb.Rope(128).plan, gq, gk, 1e-6, pos, saved, n, dgq, dgk)
    pb._check("pb_set_qk_norm_rope",
              pb.lib().pb_set_qk_norm_rope(block.handle, pb.ctypes.byref(r)))


def test_set_refuses_buffers_that_share_bytes(setup):
    wl, _, block = setup
    n = wl.batch * wl.seq * wl.hidden * 4
    saved = torch.zeros(n, dtype=torch.uint8, device="cuda")
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(wl.batch * wl.seq, dtype=torch.int32, device="cuda")
    grads = torch.zeros(256, device="cuda")
    at, g, p, d = saved.data_ptr(), gamma.data_ptr(), pos.data_ptr(), grads.data_ptr()
    good = dict(gq=g, gk=g, pos=p, saved=at, n=n, dgq=d, dgk=d + 512)
    for kw in (dict(gq=at), dict(gk=at + n - 256), dict(pos=at), dict(pos=at + n - 16),
               dict(dgq=g), dict(dgk=g + 252), dict(dgq=p), dict(dgk=p + 300)):
        with pytest.raises(pb.PbError, match="apart"):
            set_raw(block, **(good | kw))
    set_raw(block, **good)
    set_raw(block, **(good | dict(gk=g + 256)))


def test_backward_refuses_gradients_inside_its_arguments(setup):
    wl, x, block = setup
    n = wl.batch * wl.seq * wl.hidden * 4
    saved = torch.zeros(n, dtype=torch.uint8, device="cuda")
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    spare = torch.zeros(128, device="cuda")
    scratch = pb.new_train_scratch(block.dims)
    dy, dx = x.clone(), torch.zeros_like(x)
    x = x.clone()
    before = [t.clone() for t in (x, dy)]
    for t in (x, dy, dx, scratch):
        for at in (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size() - 512):
            for pair in ((at, spare.data_ptr()), (spare.data_ptr(), at)):
                set_raw(block, gamma.data_ptr(), gamma.data_ptr(), None, saved.data_ptr(), n, *pair)
                block.forward_train(x, scratch)
                with pytest.raises(pb.PbError, match="dgamma"):
                    block.backward(x, dy, scratch, grads={"dx": dx})
    assert all(torch.equal(a, b) for a, b in zip((x, dy), before))
    assert (dx == 0).all()
