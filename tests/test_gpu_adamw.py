"""GPU parity of the AdamW step and the gradient norm against the formulas in 64 bits: many
tensors at once, odd sizes, both state widths, parameter and gradient types, device scalars.

Tolerances. m and v are each one fused or separate multiply-add of fp32 values: 3 roundings of
the larger term, 2^-22. The step's quotient adds fewer than ten roundings (2^-20 relative) to
lr |up|, the parameter's own two subtractions 2^-22 |p|; a bf16 parameter or copy half a step,
2^-8. An 8-bit state is the E4M3 code of a value that is itself within 2^-17 (the scale, its
reciprocal and their products among it): the code is the
exact one's, or where that lies within 2^-17 of a border between two codes, its neighbour,
a step of 2^-3 relative at most (2^-9 below 2^-6)."""

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


def e4m3(x):
    """Nearest E4M3 value (ties to even) of |x| <= 448, in float64."""
    unit = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / unit) * unit


def blocks_of(x):
    n = x.numel()
    return torch.cat([x, x.new_zeros(-n % 256)]).view(-1, 256)


def spread(scale, n):
    return scale.double().repeat_interleave(256)[:n]


def make(sizes, param, grad, bits, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        p = torch.randn(n, generator=g, device="cuda") * 0.05
        t = dict(param=p.to(torch.bfloat16) if param == "bf16" else p,
                 copy=p.to(torch.bfloat16) if param == "fp32+bf16" else None,
                 grad=(torch.randn(n, generator=g, device="cuda") * 10.0 ** (i % 5 - 4)).to(
                     torch.bfloat16 if grad == "bf16" else torch.float32),
                 weight_decay=0.1 * (i % 3))
        t.update(pb.adamw_states(p, bits))
        out.append(t)
    return out


def state64(t, n, bits):
    if bits == 32:
        return t["m"].double(), t["v"].double()
    m = t["m"].float().double() * spread(t["m_scale"], n)
    return m, (t["v"].float().double() * spread(t["v_scale"], n)) ** 2


def check(t, old, bits, coef, lr, step, b1=0.9, b2=0.95, eps=1e-8):
    n = old["param"].numel()
    g = old["grad"].double() * coef
    m, v = state64(old, n, bits)
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    size = b1 * m.abs() + (1 - b1) * g.abs()
    up = m2 / (1 - b1 ** step) / (torch.sqrt(v2 / (1 - b2 ** step)) + eps)
    top = size / (1 - b1 ** step) / (torch.sqrt(v2 / (1 - b2 ** step)) + eps)
    p = old["param"].double()
    p2 = p - lr * old["weight_decay"] * p - lr * up
    room = 2.0 ** -20 * lr * top + 2.0 ** -22 * p.abs() + 1e-30
    if t["param"].dtype == torch.bfloat16:
        room = room + 2.0 ** -8 * p2.abs()
    assert ((t["param"].double() - p2).abs() <= room).all()
    if t.get("copy") is not None:
        assert torch.equal(t["copy"], t["param"].to(torch.bfloat16))
    if bits == 32:
        assert ((t["m"].double() - m2).abs() <= 2.0 ** -22 * size + 1e-40).all()
        assert ((t["v"].double() - v2).abs() <= 2.0 ** -22 * v2 + 1e-40).all()
        return
    for name, x, second in (("m", m2, False), ("v", torch.sqrt(v2), True)):
        amax = blocks_of(x.abs()).amax(1)
        scale = t[name + "_scale"].double()
        assert ((scale - amax / 448).abs() <= 2.0 ** -19 * amax / 448).all()
        code = torch.where(spread(scale, n) > 0, x / spread(scale, n), torch.zeros_like(x))
        got = t[name].float().double()
        if second:
            assert (got[x > 0] > 0).all()
            code = torch.where((x > 0) & (code < 2.0 ** -9), 2.0 ** -9 + 0 * code, code)
        # the value is the nearest code to something within the room of the exact one
        slack = 2.0 ** -17 * (size / spread(scale, n).clamp(min=1e-300) if not second else code)
        lo, hi = e4m3(code - slack), e4m3(code + slack)
        ok = (got >= lo) & (got <= hi)
        if second:
            ok |= (x > 0) & (got == 2.0 ** -9) & (lo <= 2.0 ** -9)
        assert ok.all(), (name, int((~ok).sum()))


SIZES = [1, 7, 8, 9, 255, 256, 257, 2047, 2048, 2049, 5000, 100003, 16]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("param", ["fp32+bf16", "fp32", "bf16"])
def test_steps_match_the_formula(param, grad, bits):
    ts = make(SIZES, param, grad, bits, 1)
    opt = pb.AdamW(ts, beta1=0.9, beta2=0.95, eps=1e-8)
    for step in (1, 2, 3):
        for t in ts:
            t["grad"].mul_(0.7).add_(0.01 * t["grad"].abs().mean())
        old = [{k: v.clone() if torch.is_tensor(v) else v for k, v in t.items()} for t in ts]
        norm = opt.grad_norm(max_norm=0.5)
        opt.step(lr=1e-2, step=step, grad_scale=norm[1:])
        want = math.sqrt(sum(float(t["grad"].double().square().sum()) for t in old))
        # squares of fp32 values, summed in chains of some hundred: 2^-17 relative at most
        assert abs(float(norm[0]) - want) <= 2.0 ** -17 * want
        assert abs(float(norm[1]) - min(1.0, 0.5 / (want + 1e-6))) <= 2.0 ** -16
        for t, o in zip(ts, old):
            check(t, o, bits, float(norm[1]), 1e-2, step)


def test_more_tensors_than_one_launch_holds():
    sizes = [(i * 37) % 700 for i in range(900)]  # some of no values
    ts = make(sizes, "fp32", "fp32", 8, 2)
    opt = pb.AdamW(ts, beta1=0.9, beta2=0.95)
    old = [{k: v.clone() if torch.is_tensor(v) else v for k, v in t.items()} for t in ts]
    norm = opt.grad_norm(max_norm=1.0)
    opt.step(lr=1e-3, step=5, grad_scale=norm[1:])
    want = math.sqrt(sum(float(t["grad"].double().square().sum()) for t in old))
    assert abs(float(norm[0]) - want) <= 2.0 ** -17 * want
    for t, o in zip(ts, old):
        if t["param"].numel():
            check(t, o, 8, float(norm[1]), 1e-3, 5)


@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_behind_a_tensor_is_written(bits):
    n = 1000  # ends inside a thread's 8 values' warp
    flat = {k: torch.full((1280,), 7.0, device="cuda") for k in ("param", "grad")}
    flat["copy"] = torch.full((1280,), 7.0, device="cuda", dtype=torch.bfloat16)
    st = pb.adamw_states(torch.empty(1280, device="cuda"), bits)
    t = {k: v[:n] for k, v in {**flat, "m": st["m"], "v": st["v"]}.items()}
    if bits == 8:
        t["m_scale"], t["v_scale"] = st["m_scale"][:4], st["v_scale"][:4]
    pb.AdamW([t]).step(lr=0.1, step=1)
    for k in ("param", "copy"):
        assert (flat[k][n:] == 7).all() and (flat[k][:n] != 7).all()
    assert (st["m"].float()[n:] == 0).all() and (st["v"].float()[n:] == 0).all()
    if bits == 8:
        assert (st["m_scale"][4:] == 0).all() and (st["m_scale"][:4] > 0).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_scale_that_is_not_finite_leaves_the_step_out(bits):
    ts = make([300, 5], "fp32+bf16", "fp32", bits, 3)
    opt = pb.AdamW(ts)
    opt.step(lr=1e-2, step=1)
    old = [{k: v.clone() if torch.is_tensor(v) else v for k, v in t.items()} for t in ts]
    for value in (float("inf"), float("nan"), 1e25):  # 1e25: its square overflows
        ts[1]["grad"][3] = value
        norm = opt.grad_norm(max_norm=1.0)
        assert not math.isfinite(float(norm[0])) and math.isnan(float(norm[1]))
        opt.step(lr=1e-2, step=2, grad_scale=norm[1:])
        for t, o in zip(ts, old):
            for k in ("param", "copy", "m", "v"):
                assert torch.equal(t[k].float(), o[k].float())


def test_eight_bits_blocks_of_zeros_and_a_wide_range():
    n = 768
    p = torch.zeros(n, device="cuda")
    t = dict(param=p, grad=torch.zeros(n, device="cuda"), **pb.adamw_states(p, 8))
    # block 0: no gradient; block 1: 2^-60 next to 1; block 2: all far below the fp32 normal range
    t["grad"][256] = 1.0
    t["grad"][257:512] = 2.0 ** -60
    t["grad"][512:] = 2.0 ** -130
    opt = pb.AdamW([t], eps=1e-30)
    for step in range(1, 4):
        opt.step(lr=1.0, step=step)
    assert torch.isfinite(t["param"]).all()
    assert (t["param"][:256] == 0).all() and (t["v"].float()[:256] == 0).all()
    assert (t["v"].float()[256:512] > 0).all()
    # what became zero in v or rose to the least code never makes a step beyond the first's
    assert (t["param"][256:512].abs() <= 3.5).all()


def test_device_scalars_in_a_graph():
    ts = make([1000, 33], "fp32", "fp32", 32, 4)
    twin = [{k: v.clone() if torch.is_tensor(v) else v for k, v in t.items()} for t in ts]
    opt, other = pb.AdamW(ts, beta2=0.999), pb.AdamW(twin, beta2=0.999)
    lr = torch.zeros(1, device="cuda")
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    norm = torch.empty(2, device="cuda")
    scratch = torch.empty(opt.scratch_bytes, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        opt.grad_norm(max_norm=1.0, out=norm, scratch=scratch)
        opt.step(lr=0.0, d_lr=lr, d_step=step, grad_scale=norm[1:])
    for k in range(1, 4):
        lr.fill_(1e-2 / k)
        step.fill_(k)
        for t, o in zip(ts, twin):
            t["grad"].mul_(1.5)
            o["grad"].mul_(1.5)
        graph.replay()
        n2 = other.grad_norm(max_norm=1.0)
        other.step(lr=float(lr), step=k, grad_scale=n2[1:])
        assert torch.equal(norm, n2)
    for t, o in zip(ts, twin):
        assert torch.equal(t["m"], o["m"]) and torch.equal(t["v"], o["v"])
        # the corrections differ by some units: expm1 of a product in fp32, against double
        d = (t["param"] - o["param"]).abs()
        assert (d <= 2.0 ** -18 * 3e-2 + 2.0 ** -22 * o["param"].abs()).all()


def test_repeats_give_the_same_bits():
    runs = []
    for _ in range(2):
        ts = make([70001, 300], "fp32+bf16", "bf16", 8, 5)
        opt = pb.AdamW(ts)
        for step in (1, 2):
            norm = opt.grad_norm(max_norm=0.1)
            opt.step(lr=1e-3, step=step, grad_scale=norm[1:])
        runs.append([norm] + [t[k].float() for t in ts for k in ("param", "copy", "m", "v")])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_refused_calls():
    ts = make([300, 40], "fp32", "fp32", 32, 6)
    with pytest.raises(pb.PbError, match="overlaps"):
        pb.AdamW([ts[0], ts[0]]).step(lr=1e-3, step=1)
    with pytest.raises(pb.PbError, match="overlaps"):
        pb.AdamW([dict(ts[0], grad=ts[0]["m"])]).step(lr=1e-3, step=1)
    opt = pb.AdamW(ts)
    with pytest.raises(pb.PbError, match="step"):
        opt.step(lr=1e-3, step=0)
    with pytest.raises(pb.PbError, match="lr"):
        opt.step(lr=float("nan"), step=1)
    with pytest.raises(pb.PbError, match="max_norm"):
        opt.grad_norm(max_norm=0.0)
    with pytest.raises(pb.PbError, match="aligned"):
        big = torch.zeros(64, device="cuda")
        pb.AdamW([dict(ts[1], param=big[1:41])]).step(lr=1e-3, step=1)
    with pytest.raises(ValueError):
        pb.AdamW([ts[0], dict(ts[1], param=ts[1]["param"].to(torch.bfloat16))])
    with pytest.raises(ValueError):
        pb.AdamW([dict(ts[0], m=ts[0]["m"][:10])])
