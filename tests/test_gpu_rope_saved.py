"""What the norm's backward pass inside the block reads: the q and k that pb_block_rope.saved keeps
belong to one forward pass, whatever is set on the handle between it and its backward pass.

Gradients of two runs are equal but for dq, which is summed by atomic additions whose order
varies: fp32 sums in another order move a bf16 value near a rounding border by one step, 2^-8 of
itself, so 1e-2 of the largest is allowed; with other q and k they are off by the whole value."""

import pytest
import torch

from transformer_block_gb300 import inputs, pb
from transformer_block_gb300.configs import Workload

pytestmark = pytest.mark.gpu

WL = Workload("saved", 2, 130, 256, 2, 128, 512, 64, 1, 0.02)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


class Setup:
    def __init__(self, seed=0):
        self.x, params = inputs.make_layer(WL, 0, seed=seed, device="cuda", biases=True)
        self.block = pb.ParallelBlock(pb.make_dims(WL), params)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.gq, self.gk = [(1 + 0.2 * torch.randn(128, generator=g, device="cuda")).to(
            torch.bfloat16) for _ in range(2)]
        self.x2 = torch.randn(self.x.shape, generator=g, device="cuda").to(torch.bfloat16)
        self.dy = torch.randn(self.x.shape, generator=g, device="cuda").to(torch.bfloat16)
        self.bytes = WL.batch * WL.seq * WL.hidden * 4

    def set(self, **kw):
        self.block.set_qk_norm_rope(pb.Rope(128), self.gq, self.gk, 1e-5, training=True, **kw)

    def scratch(self):
        return pb.new_train_scratch(self.block.dims)

    def back(self, x, scratch):
        g = dict(self.block.backward(x, self.dy, scratch))
        g.update({k: v.clone() for k, v in self.block.rope_grads.items()})
        return g


def same(got, want):
    for name, w in want.items():
        assert torch.isfinite(got[name].float()).all(), name
        gap = float((got[name].double() - w.double()).abs().max())
        assert gap <= 1e-2 * float(w.double().abs().max()), name


def test_set_between_forward_and_backward():
    s = Setup()
    scratch = s.scratch()
    s.set()
    s.block.forward_train(s.x, scratch)
    want = s.back(s.x, scratch)
    s.block.forward_train(s.x, scratch)
    # what is allocated next holds NaN
    del_me = torch.full((s.bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    del del_me
    s.set()
    same(s.back(s.x, scratch), want)
    assert s.block.status() == 0


def test_backward_without_a_forward_is_refused():
    s = Setup(1)
    s.set()
    with pytest.raises(pb.PbError, match="no forward"):
        s.back(s.x, s.scratch())
    scratch = s.scratch()
    s.block.forward_train(s.x, scratch)
    s.back(s.x, scratch)
    # a buffer of the caller's that no forward has filled
    s.set(saved=torch.empty(s.bytes, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pb.PbError, match="no forward"):
        s.back(s.x, scratch)


def test_two_forwards_in_flight():
    s = Setup(2)
    one, two = s.scratch(), s.scratch()
    a, b = (torch.empty(s.bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    want = []
    for x in (s.x, s.x2):
        s.set()
        s.block.forward_train(x, one)
        want.append(s.back(x, one))
    s.set(saved=a)
    s.block.forward_train(s.x, one)
    s.set(saved=b)
    s.block.forward_train(s.x2, two)
    with pytest.raises(pb.PbError, match="another scratch"):
        s.back(s.x, one)
    s.set(saved=a)
    with pytest.raises(pb.PbError, match="another scratch"):
        s.back(s.x2, two)
    same(s.back(s.x, one), want[0])
    s.set(saved=b)
    same(s.back(s.x2, two), want[1])
    # the scratch belongs to a later forward that kept its q and k elsewhere
    s.block.forward_train(s.x2, one)
    s.set(saved=a)
    with pytest.raises(pb.PbError, match="no forward"):
        s.back(s.x, one)
    # ... or that kept none
    s.block.forward_train(s.x, one)
    s.block.set_qk_norm_rope(pb.Rope(128), training=True)
    s.block.forward_train(s.x2, one)
    s.set(saved=a)
    with pytest.raises(pb.PbError, match="no forward"):
        s.back(s.x, one)
    assert s.block.status() == 0


def test_part_of_a_saved_buffer_written_by_another_forward():
    s = Setup(3)
    one, two = s.scratch(), s.scratch()
    both = torch.empty(s.bytes + 4096, dtype=torch.uint8, device="cuda")
    s.set(saved=both[:s.bytes])
    s.block.forward_train(s.x, one)
    s.set(saved=both[4096:])
    s.block.forward_train(s.x2, two)
    s.back(s.x2, two)
    s.set(saved=both[:s.bytes])
    with pytest.raises(pb.PbError, match="no forward"):
        s.back(s.x, one)


def test_buffers_that_do_not_fit_are_refused():
    s = Setup(4)
    for bad in (torch.empty(s.bytes - 1, dtype=torch.uint8, device="cuda"),
                torch.empty(s.bytes, dtype=torch.uint8),
                torch.empty(s.bytes, dtype=torch.float32, device="cuda"),
                torch.empty(s.bytes * 2, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            s.set(saved=bad)
    with pytest.raises(pb.PbError, match="256-byte"):
        s.set(saved=torch.empty(s.bytes + 16, dtype=torch.uint8, device="cuda")[16:])
    with pytest.raises(ValueError, match="training"):
        s.block.set_qk_norm_rope(pb.Rope(128), s.gq, s.gk,
                                 saved=torch.empty(s.bytes, dtype=torch.uint8, device="cuda"))
