"""GPU parity of the linear layer (bias, activation, residual in the epilogue; from one token to
thousands), its backward pass and the activation's, against the formulas in 64 bits.

Tolerances. Let S = sum |x| |w| + |bias| bound every partial sum of pre = x w + bias. The
tensor core adds 16 products at a time and cuts off: at most 2^-22 S an instruction (an fp32
step of a partial sum, doubled for the alignment of the addends), K / 16 instructions in one
chain, or for fp32 results chains of 1024 / 16 and one rounded addition for each; a split
product adds up to 96 partial sums. So |err(pre)| <= (K / 16 + 100) 2^-22 S. The activations
and their derivatives change by at most 1.2 a unit (1.2 and 0.8 x the incoming gradient's
error) and are computed to 2^-19 (1 + |z|); the residual's addition rounds at 2^-24. The
result is rounded once: half a step of its type."""

import math

import pytest
import torch

from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
FEW = 32  # tokens of the few-token kernel


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


@pytest.fixture(scope="module")
def scratch():
    # never prepared: the counters in it may hold anything
    g = torch.Generator(device="cuda").manual_seed(99)
    return torch.randint(0, 256, (pb.linear_scratch_bytes(),), dtype=torch.uint8, device="cuda",
                         generator=g)


def act64(name, z):
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z.clamp(min=0) if name == "relu" else z


def act_grad64(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    y = z.clone().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(act64(name, y).sum(), y)[0]


def strided(g, rows, cols, dt, pad, scale=1.0):
    """[rows, cols] inside a buffer with `pad` more columns (NaN) in every row."""
    ld = cols + pad
    ld += -ld % 8
    buf = torch.full((rows, ld), float("nan"), dtype=dt, device="cuda")
    buf[:, :cols] = (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(dt)
    return buf[:, :cols]


def room_of(x, w, b, K):
    s = x.double().abs() @ w.double().abs()
    if b is not None:
        s = s + b.double().abs()
    return (K / 16 + 100) * 2.0 ** -22 * s


def check(got, ref, room, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.float()).all(), what
    bad = err > HALF[got.dtype] * ref.abs() * (1 + 2.0 ** -6) + room + 1e-30
    if got.dtype == torch.float16:  # steps of fp16's smallest values
        bad &= err > 2.0 ** -25 + room
    assert not bad.any(), (what, int(bad.sum()), float(err.max()))


# m, n, k, pad: one token to several tiles; rows, columns and k that end inside a tile, a vector
# or a step; products that split along k; n and k of one
SHAPES = [
    (1, 64, 32, 0), (1, 8, 8, 0), (1, 1, 1, 0), (1, 200, 1000, 0), (2, 513, 77, 8), (5, 70, 4096, 0),
    (8, 1024, 2048, 0), (9, 129, 264, 0), (16, 4100, 520, 0), (17, 72, 640, 16), (24, 65, 33, 0),
    (31, 1000, 520, 8), (32, 96, 1032, 0), (33, 1000, 520, 8), (64, 256, 4096, 0),
    (100, 13, 129, 0), (129, 257, 65, 0), (256, 512, 2048, 0), (300, 2504, 1000, 8),
    (513, 1032, 264, 0), (1000, 7, 4104, 0), (2100, 2600, 520, 0),
]


@pytest.mark.parametrize("layout", [pb.PB_WEIGHT_IN_OUT, pb.PB_WEIGHT_OUT_IN],
                         ids=["in_out", "out_in"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, dt, layout, scratch):
    m, n, k, pad = shape
    g = torch.Generator(device="cuda").manual_seed(m * 31 + n * 7 + k)
    x = strided(g, m, k, dt, pad)
    w = strided(g, k, n, dt, pad, 0.05) if layout == pb.PB_WEIGHT_IN_OUT else \
        strided(g, n, k, dt, pad, 0.05)
    w64 = w.double() if layout == pb.PB_WEIGHT_IN_OUT else w.double().t()
    b = (torch.randn(n, generator=g, device="cuda") * 0.1).to(dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    z = x.double() @ w64
    acc, accb = room_of(x, w64, None, k), room_of(x, w64, b, k)
    # plain, into rows with other columns behind them, with and without scratch
    out = strided(g, m, n, dt, 8)
    behind = out.as_strided((m, out.stride(0) - n), out.stride(), out.storage_offset() + n).clone()
    pb.linear(x, w, out=out, layout=layout, scratch=scratch, status=status)
    check(out, z, acc, "plain")
    after = out.as_strided((m, out.stride(0) - n), out.stride(), out.storage_offset() + n)
    assert torch.equal(after.view(torch.int16), behind.view(torch.int16))
    check(pb.linear(x, w, out=strided(g, m, n, torch.float32, 4), layout=layout, status=status), z,
          acc, "fp32, no scratch")
    zb = z + b.double()
    for act in ("gelu", "gelu_tanh", "silu", "relu"):
        pre = strided(g, m, n, dt, 0)
        res = strided(g, m, n, torch.float32 if act == "silu" else dt, 8)
        od = torch.float32 if act in ("gelu_tanh", "relu") else dt
        y = pb.linear(x, w, b, residual=res, activation=act, layout=layout, pre=pre,
                      out=strided(g, m, n, od, 8), scratch=scratch, status=status)
        check(pre, zb, accb, act + " pre")
        ref = act64(act, zb) + res.double()
        check(y, ref, 1.2 * accb + 2.0 ** -19 * (1 + zb.abs()) + 2.0 ** -23 * res.double().abs(),
              act)
    assert int(status.item()) == 0


def test_residual_in_place_and_repeats(scratch):
    for m, n, k in ((3, 264, 512), (200, 1032, 4096), (700, 2056, 520)):
        g = torch.Generator(device="cuda").manual_seed(m)
        x = strided(g, m, k, torch.bfloat16, 0)
        w = strided(g, k, n, torch.bfloat16, 0, 0.05)
        for dt in (torch.bfloat16, torch.float32):
            r = strided(g, m, n, dt, 8)
            want = pb.linear(x, w, residual=r, activation="silu", out_dtype=dt, scratch=scratch)
            again = pb.linear(x, w, residual=r, activation="silu", out_dtype=dt, scratch=scratch)
            assert torch.equal(want, again)  # whichever pair arrives last
            got = pb.linear(x, w, residual=r, activation="silu", out=r, scratch=scratch)
            assert got is r and torch.equal(r, want)


def test_activations_at_their_ends(scratch):
    # pre is set through the bias: x = 0
    z = [0.0, -0.0, 1e-30, 5.5, -5.5, 13.0, -13.0, 79.0, -79.0, 81.0, -81.0, 1e4, -1e4, 6e4, -6e4,
         3e38, -3e38, float("inf")]
    n = 24
    for m in (1, 40):
        for dt in (torch.bfloat16, torch.float16):
            b = torch.zeros(n, dtype=dt, device="cuda")
            v = torch.tensor(z, device="cuda").clamp(-3.38e38, None).to(dt)
            b[:len(z)] = v
            x = torch.zeros(m, 8, dtype=dt, device="cuda")
            w = torch.zeros(8, n, dtype=dt, device="cuda")
            for act in ("gelu", "gelu_tanh", "silu", "relu"):
                y = pb.linear(x, w, b, activation=act, out_dtype=torch.float32, scratch=scratch)
                zd = b.double()
                ref = torch.where(zd > 80, zd, act64(act, zd.clamp(max=80)))
                ref = torch.where(zd < -80, torch.zeros_like(zd), ref)
                err = (y.double() - ref).abs()
                ok = (err <= 2.0 ** -18 * (1 + ref.abs())) | (y.double() == ref)
                assert ok.all(), (act, m, dt, y[0], ref)
                bad = b.clone()
                bad[3] = float("nan")
                y = pb.linear(x, w, bad, activation=act, out_dtype=torch.float32)
                assert y[:, 3].isnan().all() and not y[:, :3].isnan().any()


BWD_SHAPES = [
    (1, 64, 128, 0), (3, 77, 40, 8), (17, 520, 264, 0), (32, 1000, 72, 0), (33, 264, 1032, 8),
    (129, 13, 257, 0), (300, 1000, 520, 0), (777, 520, 2056, 8), (2000, 264, 136, 0), (5, 1, 1, 0),
]


@pytest.mark.parametrize("layout", [pb.PB_WEIGHT_IN_OUT, pb.PB_WEIGHT_OUT_IN],
                         ids=["in_out", "out_in"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", BWD_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, dt, layout, scratch):
    m, n, k, pad = shape
    g = torch.Generator(device="cuda").manual_seed(m * 31 + n * 7 + k)
    in_out = layout == pb.PB_WEIGHT_IN_OUT
    dy = strided(g, m, n, dt, pad, 0.1)
    w = strided(g, k, n, dt, pad, 0.2) if in_out else strided(g, n, k, dt, pad, 0.2)
    w64 = w.double() if in_out else w.double().t()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for act in ("none", "gelu", "gelu_tanh", "silu", "relu"):
        pre = strided(g, m, k, dt, 8) if act != "none" else None
        x = strided(g, m, k, dt, 0)
        dx, dw, db = pb.linear_backward(dy, x, w, pre=pre, activation=act, layout=layout,
                                        bias=True, dx=strided(g, m, k, dt, 8),
                                        dw=strided(g, *w.shape, torch.float32, 4),
                                        scratch=scratch, status=status)
        d = dy.double() @ w64.t()
        acc = room_of(dy, w64.t(), None, n)
        fac = act_grad64(act, pre.double()) if pre is not None else torch.ones_like(d)
        check(dx, d * fac, 1.2 * acc + 2.0 ** -18 * d.abs(), act + " dx")
        ref = x.double().t() @ dy.double()
        acc = room_of(x.t(), dy, None, m)
        check(dw, ref if in_out else ref.t(), acc if in_out else acc.t(), act + " dw")
        # chains of rows / 512 + 8 + 64 fp32 additions
        room = (m / 512 + 80) * 2.0 ** -24 * dy.double().abs().sum(0)
        check(db, dy.double().sum(0), room, act + " db")
        # added to, and each alone
        dw2, db2 = strided(g, *w.shape, torch.float32, 4).copy_(dw), db.clone()
        only = pb.linear_backward(dy, x, None, layout=layout, need_dx=False, dw=dw2, db=db2,
                                  accumulate=True, scratch=scratch, status=status)
        assert only[0] is None
        assert torch.equal(dw2, dw + dw) and torch.equal(db2, db + db)
        alone = pb.linear_backward(dy, None, w, pre=pre, activation=act, layout=layout,
                                   need_dw=False, scratch=scratch)
        assert alone[1] is None and torch.equal(alone[0], dx)
        a = pb.activation_backward(x, pre, act) if pre is not None else None
        if a is not None:
            f = act_grad64(act, pre.double())
            check(a, x.double() * f, 2.0 ** -18 * x.double().abs(), act + " backward")
            assert torch.equal(pb.activation_backward(x, pre, act, out=x), a)
    assert int(status.item()) == 0


def test_no_tokens(scratch):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, 40, dtype=torch.bfloat16, device="cuda")
    assert pb.linear(e, w, scratch=scratch).shape == (0, 40)
    dy = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((64, 48), 3.0, device="cuda")
    db = torch.full((40,), 3.0, device="cuda")
    pb.linear_backward(dy, e, w, dw=dw[:, :40], db=db, accumulate=True, scratch=scratch)
    assert (dw == 3).all() and (db == 3).all()
    pb.linear_backward(dy, e, w, dw=dw[:, :40], db=db, scratch=scratch)
    assert (dw[:, :40] == 0).all() and (dw[:, 40:] == 3).all() and (db == 0).all()


def test_long_k_keeps_fp32_sums(scratch):
    # A chain of K / 16 sums that are cut off loses 8.6e-6 at K = 8192 (norm of the error over
    # the result's); segments of 1024 stay at that length's 1.0e-6, with room for a factor 2.
    for m, n, k in ((40, 300, 8192), (300, 520, 16384)):
        g = torch.Generator(device="cuda").manual_seed(k)
        x = strided(g, m, k, torch.bfloat16, 0)
        w = strided(g, n, k, torch.bfloat16, 0)
        ref = x.double() @ w.double().t()
        y = pb.linear(x, w, layout=pb.PB_WEIGHT_OUT_IN, out_dtype=torch.float32)
        assert float((y.double() - ref).norm() / ref.norm()) <= 2e-6


def test_gradients_against_differences(scratch):
    g = torch.Generator(device="cuda").manual_seed(21)
    m, n, k = 37, 72, 48
    pre = strided(g, m, k, torch.bfloat16, 0)
    w = strided(g, k, n, torch.bfloat16, 0, 0.2)
    dy = strided(g, m, n, torch.bfloat16, 0)
    for act in ("gelu", "gelu_tanh", "silu"):
        x = act64(act, pre.double()).to(torch.bfloat16)
        dx, dw, _ = pb.linear_backward(dy, x, w, pre=pre, activation=act, scratch=scratch)
        u = torch.randn(m, k, generator=g, device="cuda", dtype=torch.float64)
        v = torch.randn(k, n, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4

        def f(s, t):
            return (dy.double() * (act64(act, pre.double() + s * u) @ (w.double() + t * v))).sum()

        want = (f(h, 0) - f(-h, 0)) / (2 * h)
        assert abs(want - (dx.double() * u).sum()) <= 2.0 ** -8 * (dx.double() * u).abs().sum()
        want = (f(0, h) - f(0, -h)) / (2 * h)  # x was rounded to bf16
        room = 2.0 ** -8 * ((x.double().abs().t() @ dy.double().abs()) * v.abs()).sum()
        assert abs(want - (dw.double() * v).sum()) <= room


def test_two_streams_and_a_replayed_graph(scratch):
    # split products at once on two streams, each with a scratch of its own
    g = torch.Generator(device="cuda").manual_seed(22)
    x = strided(g, 200, 4096, torch.bfloat16, 0)
    w = strided(g, 4096, 1536, torch.bfloat16, 0, 0.05)
    want = pb.linear(x, w, scratch=scratch)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [torch.empty_like(scratch) for _ in range(2)]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(pb.linear(x, w, scratch=work[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for part in outs for o in part)
    # two graphs that share one scratch, replayed in turn; the counters are clear each time
    y1, y2 = torch.empty_like(want), torch.empty(200, 1536, device="cuda")
    graphs = []
    for out in (y1, y2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pb.linear(x, w, out=out, scratch=scratch)
        graphs.append(graph)
    for _ in range(3):
        x.mul_(0.5)
        for graph in graphs:
            graph.replay()
        assert torch.equal(y1, pb.linear(x, w, scratch=work[0]))
        assert torch.equal(y2, pb.linear(x, w, out_dtype=torch.float32, scratch=work[0]))


def test_refused_calls(scratch):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        pb.linear(x, w.half())
    with pytest.raises(ValueError):
        pb.linear(x, w[:60])
    with pytest.raises(ValueError):
        pb.linear(x, w, bias=torch.zeros(31, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        pb.linear(x, w.cpu())
    with pytest.raises(ValueError):
        pb.linear(x, w, out=torch.zeros(4, 32, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        pb.linear(x, w, layout=pb.PB_WEIGHT_OUT_IN)
    with pytest.raises(pb.PbError, match="multiple"):
        odd = torch.zeros(4, 61, dtype=torch.bfloat16, device="cuda")
        pb.linear(odd, torch.zeros(61, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(pb.PbError, match="overlap"):
        sq = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
        pb.linear(sq, sq, out=sq)
    with pytest.raises(pb.PbError, match="overlap"):
        r = torch.zeros(5, 32, dtype=torch.bfloat16, device="cuda")
        pb.linear(x, w, residual=r[:4], out=r[1:])
    with pytest.raises(pb.PbError, match="scratch"):
        pb.linear(x, w, scratch=scratch[:1000])
    with pytest.raises(ValueError):
        pb.linear_backward(x, x, torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda"),
                           activation="gelu")
