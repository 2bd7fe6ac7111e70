"""The rotation, linear and AdamW calls at their largest offsets and on other streams: tensors of
more than 2^31 values (element offsets past 32 bits), results allocated for a side stream, calls
from several host threads at once."""

import threading

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


def test_linear_result_beyond_32_bit_offsets():
    m, n, k = 66000, 32776, 64  # 2.16e9 values
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(k, n, generator=g, device="cuda").to(torch.bfloat16)
    y = pb.linear(x, w, activation="relu")
    rows = torch.tensor([0, 1, 65537, m - 1], device="cuda")
    ref = (x[rows].double() @ w.double()).clamp(min=0)
    room = 2.0 ** -8 * ref + 2.0 ** -17 * (x[rows].double().abs() @ w.double().abs())
    assert ((y[rows].double() - ref).abs() <= room).all()
    # backward: dw contracts over the rows; one column of dy is not zero
    y.zero_()
    y[:, n - 1] = 1.0
    dx, dw, db = pb.linear_backward(y, x, w, bias=True)
    assert torch.equal(dx, w[:, n - 1].expand(m, k))
    assert float(db[n - 1]) == m and float(db[:n - 1].abs().max()) == 0
    want = x.double().sum(0)
    assert ((dw[:, n - 1].double() - want).abs() <= 2.0 ** -14 * x.double().abs().sum(0)).all()
    assert float(dw[:, :n - 1].abs().max()) == 0


def test_rotation_beyond_32_bit_offsets():
    s, h, d = 66000, 257, 128  # 2.17e9 values
    q = torch.empty(1, s, h, d, dtype=torch.bfloat16, device="cuda")
    q.fill_(1.0)
    q[0, s - 1, h - 1] = 2.0
    pos = torch.zeros(1, 1, s, dtype=torch.int32, device="cuda")
    gamma = torch.full((d,), 3.0, dtype=torch.bfloat16, device="cuda")
    # position 0 does not turn: the norm makes every value gamma
    pb.qk_norm_rope(pb.Rope(d), q, None, pos, gamma, out_q=q)
    assert float(q[0, ::4000].float().min()) == 3.0 and float(q[0, ::4000].float().max()) == 3.0
    assert float(q[0, s - 1, h - 1].float().min()) == 3.0
    dq, _, dg, _ = pb.qk_norm_rope_backward(pb.Rope(d), q, None, pos, q, None, gamma, out_dq=q)
    # dy = x, all values equal: the norm's backward leaves nothing, dgamma sums 3 x 1
    assert float(q[0, s - 1].float().abs().max()) <= 2.0 ** -15 * 9
    assert ((dg.double() - 3.0 * s * h).abs() <= 2.0 ** -14 * 3.0 * s * h).all()


def test_adamw_beyond_32_bit_offsets():
    n = 2 ** 31 + 12345
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    grad = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    st = pb.adamw_states(p, 8)
    opt = pb.AdamW([dict(param=p, grad=grad, **st)])
    norm = opt.grad_norm(max_norm=1e9)
    assert abs(float(norm[0]) - n ** 0.5) <= 2.0 ** -17 * n ** 0.5
    opt.step(lr=0.25, step=1)  # a first step moves every parameter by lr
    for part in (slice(0, 4096), slice(2 ** 31 - 4096, 2 ** 31 + 4096), slice(n - 4096, n)):
        assert (p[part] == 0.75).all()
        assert (st["m"][part].float() == 448).all() and (st["v"][part].float() == 448).all()


def test_results_belong_to_the_stream_of_the_call():
    # while a side stream works, its temporaries and results are not handed to the current one
    side = torch.cuda.Stream()
    rope = pb.Rope(128)
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(4, 512, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(512, 2048, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(2048, 512, generator=g, device="cuda").to(torch.bfloat16)
    want = pb.qk_norm_rope_backward(rope, q, None, None, q, None, gamma)
    ref = pb.linear(x, w)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = []
        for _ in range(20):
            got.append(pb.qk_norm_rope_backward(rope, q, None, None, q, None, gamma, stream=stream))
            got.append(pb.linear(x, w, stream=stream))
            torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")  # takes what is free
        torch.cuda.synchronize()
        for a in got[::2]:
            assert torch.equal(a[0], want[0]) and torch.equal(a[2], want[2])
        assert all(torch.equal(a, ref) for a in got[1::2])


def test_several_host_threads_at_once():
    rope = pb.Rope(64)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(2, 100, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(200, 1024, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(1024, 640, generator=g, device="cuda").to(torch.bfloat16)
    one = x[:1]
    want = (pb.qk_norm_rope(rope, q, None)[0], pb.linear(x, w), pb.linear(one, w))
    torch.cuda.synchronize()
    wrong = []

    def work():
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            scratch = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device="cuda")
            for _ in range(50):
                got = (pb.qk_norm_rope(rope, q, None)[0], pb.linear(x, w),
                       pb.linear(one, w, scratch=scratch))
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                    wrong.append(got)
            try:
                pb.linear(x, w[:5])
                wrong.append("not refused")
            except ValueError:
                pass

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# Every call for the first time in a process while a graph is captured, behind a copy and a
# join of two streams; then the graph twice against the same calls without one.
FIRST_IN_CAPTURE = """
import torch
from transformer_block_gb300 import pb
torch.manual_seed(0)
dev = "cuda"
bf = torch.bfloat16
x = torch.randn(333, 1032, device=dev).to(bf); w = torch.randn(1032, 264, device=dev).to(bf)
src = torch.randn_like(x); one = x[:3]
q = torch.randn(2, 65, 4, 64, device=dev).to(bf); gamma = torch.rand(64, device=dev).to(bf)
n = 70001
p = torch.randn(n, device=dev); grad = torch.randn(n, device=dev)
opt = pb.AdamW([dict(param=p, grad=grad, **pb.adamw_states(p))])
rope = pb.Rope(64)
scratch = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device=dev)
d_step = torch.ones(1, dtype=torch.int32, device=dev)
start = p.clone()

def calls():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x.copy_(src)
    with torch.cuda.stream(side):
        k = pb.qk_norm_rope(rope, q, q, None, gamma, gamma)[1]
    torch.cuda.current_stream().wait_stream(side)
    back = pb.qk_norm_rope_backward(rope, q, None, None, k, None, gamma)
    y = pb.linear(x, w, activation="gelu", scratch=scratch)
    z = pb.linear(one, w)
    g = pb.linear_backward(y, x, w, bias=True, scratch=scratch)
    a = pb.activation_backward(y, y, "silu")
    norm = opt.grad_norm(1.0)
    opt.step(lr=1e-3, d_step=d_step, grad_scale=norm[1:])
    return [k, back[0], back[2], y, z, *g, a, norm]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = calls()
for _ in range(2):
    for t in out:
        t.fill_(float("nan"))
    x.zero_()
    graph.replay()
torch.cuda.synchronize()
got, stepped = [t.clone() for t in out], p.clone()
p.copy_(start); opt.tensors[0]["m"].zero_(); opt.tensors[0]["v"].zero_()
for _ in range(2):
    want = calls()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert torch.equal(stepped, p)
print("equal")
"""


def test_first_calls_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-3000:]


def test_two_graphs_on_two_streams_with_scratches_of_their_own():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(333, 4104, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(4104, 520, generator=g, device="cuda").to(torch.bfloat16)
    few = x[:20]
    graphs, outs, streams = [], [], []
    for _ in range(2):
        scratch = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device="cuda")
        want = [pb.linear(x, w, scratch=scratch), pb.linear(few, w, scratch=scratch),
                pb.linear_backward(want_dy(333, 520), x, w, scratch=scratch)[1]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [pb.linear(x, w, scratch=scratch), pb.linear(few, w, scratch=scratch),
                   pb.linear_backward(want_dy(333, 520), x, w, scratch=scratch)[1]]
        graphs.append((graph, scratch))
        outs.append(out)
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(20):
        for (graph, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def want_dy(m, n):
    i = torch.arange(m * n, device="cuda", dtype=torch.float32)
    return torch.sin(i).view(m, n).to(torch.bfloat16)
