"""Packed prompts whose starts fall: the call does nothing and says so, wherever the fall is and
whoever lists the items (blocks by themselves, or a launch of its own)."""

import pytest
import torch

from tests import test_gpu_prompt_attention as pa
from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


def alternating(n, t):
    return [0 if i % 2 == 0 else t for i in range(n + 1)]


def one_fall(n, at, t):
    s = [min(t, i * t // n) for i in range(n + 1)]
    s[at] = s[at - 1] - 1
    return s


@pytest.mark.parametrize("t,starts", [
    (200, alternating(7, 200)), (300, alternating(8, 300)), (300, alternating(200, 300)),
    (300, [0, 100, 200, 150]), (300, [1, 0, 300]), (300, [0, 200, 199, 300]),
    (300, [0, 500, 400]), (300, [-5, -10, 300]), (300, [2 ** 31 - 1, -2 ** 31]),  # outside, and fall
    (300, one_fall(128, 128, 300)), (300, one_fall(128, 1, 300)), (300, one_fall(129, 129, 300)),
    (5000, one_fall(2500, 2049, 5000)), (5000, one_fall(2500, 1, 5000)),
])
def test_nothing_happens(t, starts):
    n = len(starts) - 1
    q, k, v = pa.randn(1, t, 4, 64), pa.randn(2, t, 2, 64), pa.randn(3, t, 2, 64)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    big = torch.full((3 * t, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pb.prompt_attention(q, k, v, st, out=big[t:2 * t], status=status)
    assert status.item() == 1  # PB_ERR_INVALID_ARG
    assert bool((big == 3).all())
    # without a word to record it in
    pb.prompt_attention(q, k, v, st, out=big[t:2 * t])
    assert bool((big == 3).all())
    # the word keeps the first fault, and a sound call is not held up by it
    sound = torch.tensor([0] * n + [t], dtype=torch.int32, device="cuda")
    got = pb.prompt_attention(q, k, v, sound, status=status)
    assert status.item() == 1
    assert torch.equal(got, pb.prompt_attention(q, k, v))
