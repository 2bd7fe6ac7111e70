"""Runs of the rotation, linear and AdamW calls over the same buffers, one after the other without
a pause: their launches begin while the one before still runs, so each result is compared, bit for
bit, with the same run that waits after every call. Without waiting: on two streams at once (each
with buffers of its own) and from a captured graph. Every call sums in a fixed order."""

import random

import pytest
import torch

from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu

RESULTS = ("x", "y", "w", "dw", "db", "pre", "dx", "few", "q", "dq", "dgamma", "w32", "m", "v",
           "norm")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


def buffers(m, n, k):
    g = torch.Generator(device="cuda").manual_seed(5)

    def t(*s, dt=torch.bfloat16):
        return torch.randn(*s, generator=g, device="cuda").to(dt)

    def raw(size):
        return torch.zeros(size, dtype=torch.uint8, device="cuda")

    b = dict(x=t(m, k), y=t(m, n), dw=t(k, n, dt=torch.float32), bias=t(n), pre=t(m, n),
             db=t(n, dt=torch.float32), dx=t(m, k), few=t(8, n), q=t(1, m, 4, 64),
             dq=t(1, m, 4, 64), gamma=t(64), dgamma=t(64, dt=torch.float32),
             w32=t(k, n, dt=torch.float32) / k ** 0.5, norm=t(2, dt=torch.float32),
             scratch=raw(pb.linear_scratch_bytes()), sums=raw(pb.qk_norm_rope_scratch_bytes()))
    b["w"] = b["w32"].to(torch.bfloat16)
    b.update(pb.adamw_states(b["w32"]))
    b["opt"] = pb.AdamW([dict(param=b["w32"], copy=b["w"], grad=b["dw"], m=b["m"], v=b["v"])])
    b["partials"] = raw(b["opt"].scratch_bytes)
    return b


def run(calls, b, wait):
    rope = pb.Rope(64)
    for what, act, number in calls:
        if what == "linear":
            pb.linear(b["x"], b["w"], b["bias"], activation=act, out=b["y"], pre=b["pre"],
                      scratch=b["scratch"])
        elif what == "backward":
            pb.linear_backward(b["y"], b["x"], b["w"], bias=True, dx=b["dx"], dw=b["dw"],
                               db=b["db"], scratch=b["scratch"])
        elif what == "few":
            pb.linear(b["x"][:8], b["w"], out=b["few"], scratch=b["scratch"])
        elif what == "rotate":
            pb.qk_norm_rope(rope, b["q"], None, None, b["gamma"], out_q=b["q"])
        elif what == "rotate backward":
            pb.qk_norm_rope_backward(rope, b["q"], None, None, b["dq"], None, b["gamma"],
                                     out_dq=b["dq"], dgamma_q=b["dgamma"], scratch=b["sums"])
        elif what == "update":
            b["opt"].grad_norm(1.0, out=b["norm"], scratch=b["partials"])
            b["opt"].step(lr=1e-3, step=number, grad_scale=b["norm"][1:])
        else:  # results become inputs
            b["x"].copy_(b["dx"]).clamp_(-3, 3)
            b["y"][:8].copy_(b["few"]).clamp_(-3, 3)
        if wait:
            torch.cuda.synchronize()


@pytest.mark.parametrize("m,n,k", [(40, 72, 1032), (100, 2056, 264), (333, 264, 2056),
                                   (777, 520, 1032)])
def test_runs_without_a_pause(m, n, k):
    rng = random.Random(m)
    kinds = ["linear", "backward", "few", "rotate", "rotate backward", "update", "copy"]
    calls = [(rng.choice(kinds), rng.choice(["none", "gelu", "silu"]), rng.randint(1, 100))
             for _ in range(60)]
    want = buffers(m, n, k)
    run(calls, want, True)
    both = [buffers(m, n, k) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for b, st in zip(both, streams):
        with torch.cuda.stream(st):
            run(calls, b, False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(calls, both[2], False)
    graph.replay()
    torch.cuda.synchronize()
    for where, b in zip(("stream 1", "stream 2", "graph"), both):
        for name in RESULTS:
            assert torch.isfinite(b[name].float()).all(), (where, name)
            assert torch.equal(b[name], want[name]), (where, name)
