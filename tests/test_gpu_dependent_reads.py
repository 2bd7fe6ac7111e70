"""A launch that begins while the one before it still runs reads what that one writes: the norm's
gamma, updated by the AdamW step directly in front of the rotation, and that step's gradient and
clip factor, written by the calls before it. Every result equals, bit for bit, that of the same run with a wait after every call."""

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


def run(tokens, wait, copy, steps=60):
    """Rotations with a gamma that changes in between: forward, update, forward, backward, update."""
    g = torch.Generator(device="cuda").manual_seed(tokens)

    def t(*s, dt=torch.bfloat16):
        return torch.randn(*s, generator=g, device="cuda").to(dt)

    rope = pb.Rope(128)
    q, dq = t(1, tokens, 8, 128), t(1, tokens, 8, 128)
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    grad = t(128, dt=torch.float32)
    if copy:  # gamma is the bf16 copy of fp32 parameters
        param = gamma.float()
        opt = pb.AdamW([dict(param=param, copy=gamma, grad=grad, **pb.adamw_states(param))])
    else:
        opt = pb.AdamW([dict(param=gamma, grad=grad, **pb.adamw_states(gamma))])
    norm = torch.empty(2, device="cuda")
    partials = torch.empty(opt.scratch_bytes, dtype=torch.uint8, device="cuda")
    sums = torch.empty(pb.qk_norm_rope_scratch_bytes(), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(1, tokens, 8, 128, dtype=torch.bfloat16, device="cuda")
            for _ in range(2 * steps)]
    dgammas = torch.empty(steps, 128, device="cuda")
    gammas = torch.empty(steps, 128, dtype=torch.bfloat16, device="cuda")

    def pause():
        if wait:
            torch.cuda.synchronize()

    torch.cuda.synchronize()
    for i in range(steps):
        pb.qk_norm_rope(rope, q, None, None, gamma, out_q=outs[2 * i])
        pause()
        opt.grad_norm(1.0, out=norm, scratch=partials)
        pause()
        opt.step(lr=0.05, step=i + 1, grad_scale=norm[1:])
        pause()
        # gamma's gradient is what the next update reads
        pb.qk_norm_rope_backward(rope, q, None, None, dq, None, gamma, out_dq=outs[2 * i + 1],
                                 dgamma_q=grad, scratch=sums)
        pause()
        dgammas[i].copy_(grad)
        gammas[i].copy_(gamma)
        pause()
    torch.cuda.synchronize()
    return outs + [dgammas, gammas]


@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("tokens", [1, 300, 4000])
def test_gamma_written_by_the_launch_before(tokens, copy):
    want = run(tokens, True, copy)
    got = run(tokens, False, copy)
    assert not torch.equal(want[-1][0], want[-1][-1])
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i
