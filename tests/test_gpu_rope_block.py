"""The rotation inside the block, and the new steps run together as a user would run them.

* Forward: a handle with pb_set_qk_norm_rope gives, bit for bit, what the single steps give on
  the projection of the same block without it (scratch qk -> pb_qk_norm_rope ->
  pb_swa_attention), for every operand precision, the serial block and a stack.
* Backward: every gradient of the block with norm and rotation against torch autograd through a
  restatement in float64. Bars as for the block's backward: a mean of 6e-3 for what reads dS,
  and in quadrature what the norm adds. One bf16 rounding has a mean error of 1.4e-3 (rms
  1.7e-3). dq and dk are rounded once more on their way back: 1.4e-3. q and k are rounded twice
  each, so a score's terms are 2 x 1.7e-3 off, and normed heads make scores of standard
  deviation 1 (the projection alone makes 0.1, where this vanishes), so P is off by 3.3e-3 rms,
  2.6e-3 in the mean: sqrt(6^2 + 1.4^2 + 2.6^2) = 6.7e-3. dWo reads the attention's output and
  with it P's error: sqrt(4^2 + 2.6^2) = 4.8e-3 where the others that read no dS have 4e-3. The
  gammas' gradients are 64 or 128 values: magnitudes of normal values spread by 0.76 of their
  mean, so the ratio of two means of 64 spreads by 0.76 sqrt(2 / 64) = 13 %; three times that
  is allowed, 1.4 x 6.7e-3.
* A layer of single steps (projection, norm and rotation, attention, output projection with its
  residual), and a training step of an MLP (linear forward, backward, clip, AdamW), against
  float64."""

import math

import pytest
import torch

from tests.parity import assert_parity, host
from transformer_block_gb300 import inputs, pb
from transformer_block_gb300.configs import Workload

pytestmark = pytest.mark.gpu

DS_MEAN_TOL = 6.7e-3
COMPOUND_MEAN_TOL = 4e-3
WO_MEAN_TOL = 4.8e-3


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


def workload(B, S, H, nh, dh, F, w, variant=0):
    return Workload("rope", B, S, H, nh, dh, F, w, 1, 0.02, variant=variant)


def make(wl, seed=0, **kw):
    x, params = inputs.make_layer(wl, 0, seed=seed, device="cuda", biases=True)
    return x, params, pb.ParallelBlock(pb.make_dims(wl), params, **kw)


def plan_of(wl, kind):
    if kind == "axes":
        n = wl.head_dim // 2
        return pb.Rope(wl.head_dim, pairing="adjacent", sections=[n // 2, n // 4, n - n // 2 - n // 4],
                       ladder="per_axis")
    return pb.Rope(wl.head_dim, rot_dim=wl.head_dim // 2 if kind == "half" else None)


def extras(wl, rope, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gammas = [(1 + 0.2 * torch.randn(wl.head_dim, generator=g, device="cuda")).to(torch.bfloat16)
              for _ in range(2)]
    pos = torch.randint(0, 5000, (rope.axes, wl.batch, wl.seq), generator=g, device="cuda",
                        dtype=torch.int32)
    return gammas, pos


CASES = [
    (workload(2, 130, 256, 2, 128, 512, 64), "full"),
    (workload(1, 257, 192, 3, 64, 384, 300), "half"),
    (workload(2, 33, 256, 4, 64, 512, 8), "axes"),
    (workload(1, 1, 256, 2, 128, 512, 4), "full"),
    (workload(2, 65, 256, 2, 128, 512, 64, variant=1), "axes"),
]


@pytest.mark.parametrize("wl,kind", CASES, ids=lambda c: c if isinstance(c, str) else
                         f"b{c.batch}s{c.seq}dh{c.head_dim}v{c.variant}")
@pytest.mark.parametrize("precision", [pb.PB_OPERANDS_BF16, pb.PB_OPERANDS_FP16,
                                       pb.PB_OPERANDS_FP8])
def test_block_forward_is_the_single_steps(wl, kind, precision):
    if precision == pb.PB_OPERANDS_FP8 and (wl.hidden % 128 or (wl.hidden + wl.ffn) % 128):
        pytest.skip("FP8 needs multiples of 128")
    x, _, block = make(wl, operand_precision=precision)
    d, H, nh = block.dims, wl.hidden, wl.heads
    rope = plan_of(wl, kind)
    (gq, gk), pos = extras(wl, rope, 1)
    scratch = pb.new_scratch(d)
    plain = block.forward(x, scratch=scratch)
    qk = pb.scratch_view(scratch, d, "qk").clone().view(wl.batch, wl.seq, 2 * nh, wl.head_dim)
    vt = pb.scratch_view(scratch, d, "vt").clone()
    block.set_qk_norm_rope(rope, gq, gk, 1e-5, pos)
    y = block.forward(x, scratch=scratch)
    q, k = pb.qk_norm_rope(rope, qk[:, :, :nh], qk[:, :, nh:], pos, gq, gk, eps=1e-5)
    want = torch.cat([q, k], 2).view(-1, 2 * H).contiguous()
    got = pb.scratch_view(scratch, d, "qk")
    assert torch.equal(got, want)
    if precision == pb.PB_OPERANDS_BF16:
        act = torch.zeros(d.batch * d.seq, H, dtype=torch.bfloat16, device="cuda")
        pb.swa_attention(d, want, vt, act)
        assert torch.equal(act, pb.scratch_view(scratch, d, "act")[:, :H])
    # one key has all of the softmax's weight, however it and the query are turned
    assert torch.equal(y, plain) == (wl.seq == 1)
    # in place, a stack of it, and through the host: the same block
    assert torch.equal(pb.forward_stack([block], x), y)
    z = x.clone()
    assert torch.equal(block.forward(z, y=z), y)
    if precision != pb.PB_OPERANDS_FP8:
        serial = block.forward_serial(x, scratch=scratch)
        assert torch.equal(pb.scratch_view(scratch, d, "qk"), want)
    block.set_qk_norm_rope(None)
    assert torch.equal(block.forward(x, scratch=scratch), plain)
    if precision != pb.PB_OPERANDS_FP8:
        assert torch.equal(block.forward_serial(x, scratch=scratch), serial) == (wl.seq == 1)
    assert block.status() == 0


def rotated64(x, gamma, pos, wl, kind, eps):
    """Norm and rotation in float64, differentiable."""
    d = wl.head_dim
    rot = d // 2 if kind == "half" else d
    n = rot // 2
    parts = [d // 4, d // 8, d // 2 - d // 4 - d // 8] if kind == "axes" else [n]
    e = torch.cat([torch.arange(p).double() / p for p in parts]) if kind == "axes" else \
        torch.arange(n).double() / n
    axis = torch.repeat_interleave(torch.arange(len(parts)), torch.tensor(parts))
    ang = (pos.double()[axis.cuda()].permute(1, 2, 0) * (10000.0 ** -e).cuda()).unsqueeze(2)
    y = x
    if gamma is not None:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma
    c, s = torch.cos(ang), torch.sin(ang)
    if kind == "axes":
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = y[..., :n], y[..., n:rot]
    return torch.cat([a * c - b * s, a * s + b * c, y[..., rot:]], -1)


def block64(p, x, gq, gk, pos, wl, kind, eps):
    """The block with norm and rotation, restated in float64."""
    B, S, H, nh, d = wl.batch, wl.seq, wl.hidden, wl.heads, wl.head_dim
    if wl.variant == 1:
        xn = x / torch.sqrt((x * x).mean(-1, keepdim=True) + wl.ln_eps) * p["ln_gamma"]
    else:
        xn = torch.nn.functional.layer_norm(x, (H,), p["ln_gamma"], p["ln_beta"], wl.ln_eps)
    qkv = (xn @ p["wqkv"] + p["b_qkv"]).view(B, S, 3, nh, d)
    q = rotated64(qkv[:, :, 0], gq, pos, wl, kind, eps).transpose(1, 2)
    k = rotated64(qkv[:, :, 1], gk, pos, wl, kind, eps).transpose(1, 2)
    v = qkv[:, :, 2].transpose(1, 2)
    i = torch.arange(S, device="cuda")
    gap = i[:, None] - i[None, :]
    mask = (gap < 0) | (gap >= wl.window)
    s = (q @ k.transpose(-1, -2) / math.sqrt(d)).masked_fill(mask, -math.inf)
    attn = (torch.softmax(s, -1) @ v).transpose(1, 2).reshape(B * S, H)
    h = xn @ p["w1"] + p["b1"]
    if wl.variant == 1:
        mlp = torch.nn.functional.silu(h[:, :wl.ffn]) * h[:, wl.ffn:]
    else:
        mlp = torch.nn.functional.gelu(h)
    return x + attn @ p["wo"] + p["b_o"] + mlp @ p["w2"] + p["b2"]


@pytest.mark.parametrize("wl,kind", [c for c in CASES if c[0].seq > 1], ids=lambda c: c if
                         isinstance(c, str) else f"b{c.batch}s{c.seq}dh{c.head_dim}v{c.variant}")
def test_block_backward_matches_autograd(wl, kind):
    x, params, block = make(wl, seed=3)
    rope = plan_of(wl, kind)
    (gq, gk), pos = extras(wl, rope, 4)
    block.set_qk_norm_rope(rope, gq, gk, 1e-5, pos, training=True)
    scratch = pb.new_train_scratch(block.dims)
    g = torch.Generator(device="cuda").manual_seed(5)
    dy = torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16)
    y = block.forward_train(x, scratch)
    grads = block.backward(x, dy, scratch)
    p = {k: v.double().requires_grad_(True) for k, v in params.items()}
    xd = x.double().requires_grad_(True)
    gqd, gkd = gq.double().requires_grad_(True), gk.double().requires_grad_(True)
    ref = block64(p, xd, gqd, gkd, pos, wl, kind, 1e-5)
    assert_parity(host(y), ref.detach().cpu().numpy(), "y")
    ref.backward(dy.double())
    names = {"dwqkv": "wqkv", "dw1": "w1", "dwo": "wo", "dw2": "w2", "dgamma": "ln_gamma",
             "db_qkv": "b_qkv", "db1": "b1", "db_o": "b_o", "db2": "b2"}
    for name, key in names.items():
        tol = DS_MEAN_TOL if name in ("dwqkv", "dgamma", "db_qkv") else \
            WO_MEAN_TOL if name == "dwo" else COMPOUND_MEAN_TOL
        got, want = grads[name], p[key].grad
        if name in ("dwqkv", "db_qkv"):  # its q, k and v parts apart: they differ in size
            H = wl.hidden
            for i, part in enumerate(("q", "k", "v")):
                if part == "k" and name == "db_qkv":
                    continue  # a shift of every key: nearly zero, a difference of roundings
                assert_parity(host(got[..., i * H:(i + 1) * H]),
                              want[..., i * H:(i + 1) * H].cpu().numpy(), name + part,
                              mean_tol=DS_MEAN_TOL)
        else:
            assert_parity(host(got), want.cpu().numpy(), name, mean_tol=tol)
    assert_parity(host(grads["dx"]), xd.grad.cpu().numpy(), "dx", mean_tol=DS_MEAN_TOL)
    for name, want in (("dgamma_q", gqd.grad), ("dgamma_k", gkd.grad)):
        assert_parity(host(block.rope_grads[name]), want.cpu().numpy(), name,
                      mean_tol=1.4 * DS_MEAN_TOL)
    # accumulated: dq sums in an order that varies, so nearly twice
    once = {k: v.clone() for k, v in block.rope_grads.items()}
    block.forward_train(x, scratch)
    block.backward(x, dy, scratch, grads={k: v for k, v in grads.items()}, accumulate=True)
    for k, v in once.items():
        assert float((block.rope_grads[k] - 2 * v).abs().max()) <= 1e-2 * float(v.abs().max())
    assert block.status() == 0


def test_block_rotation_without_norm_trains_without_saved():
    wl, kind = CASES[0]
    x, params, block = make(wl, seed=6)
    rope = plan_of(wl, kind)
    _, pos = extras(wl, rope, 7)
    block.set_qk_norm_rope(rope, positions=pos, training=True)
    scratch = pb.new_train_scratch(block.dims)
    g = torch.Generator(device="cuda").manual_seed(8)
    dy = torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16)
    block.forward_train(x, scratch)
    grads = block.backward(x, dy, scratch)
    p = {k: v.double().requires_grad_(True) for k, v in params.items()}
    xd = x.double().requires_grad_(True)
    block64(p, xd, None, None, pos, wl, kind, 1e-5).backward(dy.double())
    assert_parity(host(grads["dx"]), xd.grad.cpu().numpy(), "dx", mean_tol=DS_MEAN_TOL)
    assert_parity(host(grads["dwqkv"]), p["wqkv"].grad.cpu().numpy(), "dwqkv",
                  mean_tol=DS_MEAN_TOL)


def test_block_rotation_refusals():
    wl, _ = CASES[0]
    x, _, block = make(wl)
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pb.PbError, match="head_dim"):
        block.set_qk_norm_rope(pb.Rope(64))
    with pytest.raises(ValueError):
        block.set_qk_norm_rope(pb.Rope(128), gamma[:64])
    with pytest.raises(pb.PbError, match="eps"):
        block.set_qk_norm_rope(pb.Rope(128), gamma, gamma, eps=0.0)
    with pytest.raises(pb.PbError, match="positions"):
        block.set_qk_norm_rope(pb.Rope(128, sections=[32, 32]))
    block.set_qk_norm_rope(pb.Rope(128), gamma, gamma)  # not for training
    with pytest.raises(pb.PbError, match="saved"):
        block.forward_train(x, pb.new_train_scratch(block.dims))
    block.set_qk_norm_rope(pb.Rope(128), gamma, gamma, training=True)
    block.forward_train(x, pb.new_train_scratch(block.dims))


@pytest.mark.parametrize("B,S", [(1, 1), (2, 130), (1, 300)])
def test_attention_layer_of_single_steps(B, S):
    wl = workload(B, S, 256, 2, 128, 512, 64)
    H, nh, d, T = 256, 2, 128, B * S
    x, params = inputs.make_layer(wl, 0, seed=9, device="cuda", biases=True)
    rope = plan_of(wl, "full")
    (gq, gk), pos = extras(wl, rope, 10)
    dims = pb.make_dims(wl)
    scratch = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device="cuda")
    xn = pb.layernorm(x, params["ln_gamma"], params["ln_beta"])
    qkv = pb.linear(xn, params["wqkv"], params["b_qkv"], scratch=scratch)
    v4 = qkv.view(B, S, 3 * nh, d)
    qk = torch.empty(B, S, 2 * nh, d, dtype=torch.bfloat16, device="cuda")
    pb.qk_norm_rope(rope, v4[:, :, :nh], v4[:, :, nh:2 * nh], pos, gq, gk, eps=1e-5,
                    out_q=qk[:, :, :nh], out_k=qk[:, :, nh:])
    pad = (S + 7) // 8 * 8
    vt = torch.zeros(B, nh, d, pad, dtype=torch.bfloat16, device="cuda")
    vt[..., :S] = v4[:, :, 2 * nh:].permute(0, 2, 3, 1)
    attn = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    pb.swa_attention(dims, qk, vt, attn)
    y = pb.linear(attn, params["wo"], params["b_o"], residual=x, scratch=scratch)
    p = {k: t.double() for k, t in params.items()}
    xd = x.double()
    ln = torch.nn.functional.layer_norm(xd, (H,), p["ln_gamma"], p["ln_beta"], 1e-5)
    w = (ln @ p["wqkv"] + p["b_qkv"]).view(B, S, 3, nh, d)
    q = rotated64(w[:, :, 0], gq.double(), pos, wl, "full", 1e-5).transpose(1, 2)
    k = rotated64(w[:, :, 1], gk.double(), pos, wl, "full", 1e-5).transpose(1, 2)
    i = torch.arange(S, device="cuda")
    gap = i[:, None] - i[None, :]
    s = (q @ k.transpose(-1, -2) / math.sqrt(d)).masked_fill((gap < 0) | (gap >= 64), -math.inf)
    a = (torch.softmax(s, -1) @ w[:, :, 2].transpose(1, 2)).transpose(1, 2).reshape(T, H)
    assert_parity(host(y), (xd + a @ p["wo"] + p["b_o"]).cpu().numpy(), "layer")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("tokens", [7, 300])
def test_training_step_of_an_mlp(tokens, bits):
    # y = x + gelu(x W1 + b1) W2 + b2: forward, backward, clip, step; parameters against float64.
    # A first step moves a parameter by lr g / (|g| + eps') whatever g's size, so where |g| is
    # below its own error (2^-6 of the typical gradient covers the bf16 roundings of x's
    # activation and of the incoming gradient) either sign is right; elsewhere the step is lr
    # within 1 %.
    g = torch.Generator(device="cuda").manual_seed(11)
    H, F = 136, 520

    def new(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    x = new(tokens, H).to(torch.bfloat16)
    master = {"w1": new(H, F, scale=0.05), "b1": new(F, scale=0.05), "w2": new(F, H, scale=0.05),
              "b2": new(H, scale=0.05)}
    work = {k: v.to(torch.bfloat16) for k, v in master.items()}
    old = {k: v.clone() for k, v in master.items()}
    dy = new(tokens, H).to(torch.bfloat16)
    scratch = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device="cuda")
    pre = torch.empty(tokens, F, dtype=torch.bfloat16, device="cuda")
    h = pb.linear(x, work["w1"], work["b1"], activation="gelu", pre=pre, scratch=scratch)
    y = pb.linear(h, work["w2"], work["b2"], residual=x, scratch=scratch)
    dpre, dw2, db2 = pb.linear_backward(dy, h, work["w2"], pre=pre, activation="gelu", bias=True,
                                        scratch=scratch)
    dx, dw1, db1 = pb.linear_backward(dpre, x, work["w1"], bias=True, scratch=scratch)
    grads = {"w1": dw1, "b1": db1, "w2": dw2, "b2": db2}
    opt = pb.AdamW([dict(param=master[k], copy=work[k], grad=grads[k], weight_decay=0.0,
                         **pb.adamw_states(master[k], bits)) for k in master])
    norm = opt.grad_norm(max_norm=1.0)
    p = {k: v.to(torch.bfloat16).double().requires_grad_(True) for k, v in old.items()}
    xd = x.double().requires_grad_(True)
    ref = xd + torch.nn.functional.gelu(xd @ p["w1"] + p["b1"]) @ p["w2"] + p["b2"]
    assert_parity(host(y), ref.detach().cpu().numpy(), "y")
    ref.backward(dy.double())
    assert_parity(host(dx) + host(dy), xd.grad.cpu().numpy(), "dx", mean_tol=COMPOUND_MEAN_TOL)
    for k, v in grads.items():
        assert_parity(host(v), p[k].grad.cpu().numpy(), "d" + k, mean_tol=COMPOUND_MEAN_TOL)
    total = math.sqrt(sum(float(v.grad.square().sum()) for v in p.values()))
    assert abs(float(norm[0]) - total) <= 4e-3 * total
    opt.step(lr=1e-2, step=1, grad_scale=norm[1:])
    for k in master:
        gr = p[k].grad
        clear = gr.abs() > 2.0 ** -6 * gr.abs().mean()
        want = old[k].double() - 1e-2 * torch.sign(gr)
        assert ((master[k].double() - want).abs()[clear] <= 1e-4).all(), k
        assert ((master[k].double() - old[k].double()).abs() <= 1.01e-2).all(), k
        assert torch.equal(work[k], master[k].to(torch.bfloat16))


def test_guarded_buffers():
    """Nothing is written outside results and scratch: canaries around every buffer."""
    G, C = 4096, 0xA5

    def guarded(nbytes):
        buf = torch.full((nbytes + 2 * G,), C, dtype=torch.uint8, device="cuda")
        return buf, buf[G:G + nbytes]

    bufs = []

    def out(dtype, *shape):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        buf, t = guarded(n)
        bufs.append(buf)
        return t.view(dtype).view(*shape)

    g = torch.Generator(device="cuda").manual_seed(12)
    scratch = out(torch.uint8, pb.linear_scratch_bytes())
    for m, n, k in ((1, 72, 2056), (13, 4104, 264), (33, 264, 4104), (130, 520, 2056),
                    (300, 2504, 5120), (777, 264, 520)):
        x = torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)
        for layout in (0, 1):
            shape = (k, n) if layout == 0 else (n, k)
            w = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
            dy = torch.randn(m, n, generator=g, device="cuda").to(torch.bfloat16)
            for od in (torch.bfloat16, torch.float32):
                pb.linear(x, w, activation="silu", out=out(od, m, n),
                          pre=out(torch.bfloat16, m, n), scratch=scratch, layout=layout)
            pb.linear_backward(dy, x, w, pre=x, activation="gelu", dx=out(torch.bfloat16, m, k),
                               dw=out(torch.float32, *shape), db=out(torch.float32, n),
                               scratch=scratch, layout=layout)
        pb.activation_backward(x, x, "relu", out=out(torch.bfloat16, m, k))
    for b, s, nq, nk, d in ((1, 1, 1, 1, 64), (3, 37, 5, 1, 96), (2, 300, 8, 2, 128)):
        gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
        q = torch.randn(b, s, nq, d, generator=g, device="cuda").to(torch.bfloat16)
        k = torch.randn(b, s, nk, d, generator=g, device="cuda").to(torch.bfloat16)
        rope = pb.Rope(d, rot_dim=d // 32 * 16)
        pb.qk_norm_rope(rope, q, k, None, gamma, gamma, out_q=out(torch.bfloat16, b, s, nq, d),
                        out_k=out(torch.bfloat16, b, s, nk, d))
        pb.qk_norm_rope_backward(rope, q, k, None, q, k, gamma, gamma,
                                 out_dq=out(torch.bfloat16, b, s, nq, d),
                                 out_dk=out(torch.bfloat16, b, s, nk, d),
                                 dgamma_q=out(torch.float32, d), dgamma_k=out(torch.float32, d),
                                 scratch=out(torch.uint8, pb.qk_norm_rope_scratch_bytes()))
    for bits in (32, 8):
        for n in (1, 255, 2049, 70001):
            st = pb.adamw_states(torch.empty(n, device="cuda"), bits)
            t = {k: out(torch.uint8 if v.dtype == torch.float8_e4m3fn else v.dtype, *v.shape)
                 for k, v in st.items()}
            t = {k: v.zero_().view(st[k].dtype) for k, v in t.items()}
            t["param"] = out(torch.float32, n).zero_()
            t["copy"] = out(torch.bfloat16, n)
            t["grad"] = torch.randn(n, generator=g, device="cuda")
            opt = pb.AdamW([t])
            norm = opt.grad_norm(1.0, out=out(torch.float32, 2),
                                 scratch=out(torch.uint8, opt.scratch_bytes))
            opt.step(1e-3, 1, grad_scale=norm[1:])
    torch.cuda.synchronize()
    for i, buf in enumerate(bufs):
        assert (buf[:G] == C).all() and (buf[-G:] == C).all(), i


def test_block_rotation_gradients_apart():
    wl, _ = CASES[0]
    _, _, block = make(wl)
    d = block.dims
    n = d.batch * d.seq * d.hidden * 4
    gamma = torch.ones(d.head_dim, dtype=torch.bfloat16, device="cuda")
    grads = torch.zeros(2 * d.head_dim, dtype=torch.float32, device="cuda")
    saved = torch.empty(n, dtype=torch.uint8, device="cuda")
    at, g = grads.data_ptr(), gamma.data_ptr()

    def refused(dgq, dgk):
        r = pb.pb_block_rope(pb.Rope(d.head_dim).plan, g, g, 1e-6, None, saved.data_ptr(), n, dgq,
                             dgk)
        with pytest.raises(pb.PbError, match="apart"):
            pb._check("pb_set_qk_norm_rope",
                      pb.lib().pb_set_qk_norm_rope(block.handle, pb.ctypes.byref(r)))

    refused(at, at)
    refused(at, at + 4 * d.head_dim - 4)
    refused(saved.data_ptr() + n - 4, at)
    refused(at, saved.data_ptr())


def test_block_rotation_saves_one_forward():
    # what the norm's backward reads is the last forward's: an earlier one's scratch is refused
    wl, kind = CASES[0]
    x, _, block = make(wl, seed=12)
    rope = plan_of(wl, kind)
    (gq, gk), pos = extras(wl, rope, 13)
    block.set_qk_norm_rope(rope, gq, gk, 1e-5, pos, training=True)
    one, two = pb.new_train_scratch(block.dims), pb.new_train_scratch(block.dims)
    block.forward_train(x, one)
    block.forward_train(x, two)
    with pytest.raises(pb.PbError, match="another scratch"):
        block.backward(x, x.clone(), one)
    last = block.backward(x, x.clone(), two)["dw1"]
    block.forward_train(x, one)
    assert torch.equal(block.backward(x, x.clone(), one)["dw1"], last)
    # without a norm nothing is kept, and forwards may be in flight together
    block.set_qk_norm_rope(rope, positions=pos, training=True)
    block.forward_train(x, one)
    block.forward_train(x, two)
    block.backward(x, x.clone(), one)
    assert block.status() == 0
