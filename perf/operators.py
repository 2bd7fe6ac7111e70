"""Cases, plain forms and 64-bit definitions of the operators around the block's GEMMs and
attention, for timing and comparison:

* ``qk``         norm of every query and key head and its rotation by the token's position
* ``qk_bwd``     its backward pass
* ``linear``     y = residual + act(x W + b), from one token to thousands
* ``linear_bwd`` dx = (dy W^T) act'(pre), dW = x^T dy, db = sum of dy
* ``adamw``      one AdamW step over many tensors, with its clip by the global gradient norm

``run`` computes them by elementary torch operations in 32 bits, or with ``own`` through the
library's binding.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 256      # elements of an 8-bit state that share a scale
E4M3_MAX = 448.0  # largest E4M3 value
E4M3_MIN = 2.0 ** -9


# ------------------------------------------------------------------------------- cases

def _block_sizes(hidden, ffn, layers=1):
    """Parameters of `layers` blocks in pb_weights order: gamma, beta, wqkv, w1, wo, w2."""
    one = [hidden, hidden, hidden * 3 * hidden, hidden * ffn, hidden * hidden, ffn * hidden]
    return ",".join(str(n) for n in one * layers)


def listed():
    return [
        # one decoding step of a batch of 64 sequences with shared key heads, far positions
        dict(name="qk decode 64x1", op="qk", batch=64, seq=1, q_heads=32, k_heads=8, head_dim=128,
             rot=128, pairing="halves", axes=1, sections="64", ladder="shared", norm=True,
             far=131072, packed=True),
        # a video latent of 21 x 30 x 52 positions, q and k columns of one [q | k | v] buffer
        dict(name="qk video 32760", op="qk", batch=1, seq=32760, q_heads=32, k_heads=32,
             head_dim=128, rot=128, pairing="adjacent", axes=3, sections="16,24,24",
             ladder="per_axis", norm=True, far=0, packed=True),
        # the training step of the hidden-2048 block: 16 heads, four sequences
        dict(name="qk backward 4x2048", op="qk_bwd", batch=4, seq=2048, q_heads=16, k_heads=16,
             head_dim=128, rot=128, pairing="halves", axes=1, sections="64", ladder="shared",
             norm=True, far=0, packed=True),
        # odd lengths, half of each head rotated, an image's three axes, shared key heads
        dict(name="qk backward odd 3x777", op="qk_bwd", batch=3, seq=777, q_heads=20, k_heads=5,
             head_dim=64, rot=32, pairing="halves", axes=3, sections="4,6,6", ladder="shared",
             norm=True, far=4096, packed=False),
        # one token through the first MLP linear of the hidden-2048 block
        dict(name="linear 1 token", op="linear", m=1, n=8192, k=2048, w="in_out", act="gelu",
             bias=True, residual="none", pre=False, dtype="bf16", out="bf16"),
        # a decoding batch through the output projection of the 175B-shaped layer
        dict(name="linear 24 tokens", op="linear", m=24, n=12288, k=12288, w="in_out", act="none",
             bias=True, residual="bf16", pre=False, dtype="bf16", out="bf16"),
        # a ragged batch of prompts, fp16 weights stored [out, in], fp32 result
        dict(name="linear ragged 333", op="linear", m=333, n=2504, k=5120, w="out_in", act="silu",
             bias=True, residual="none", pre=False, dtype="fp16", out="fp32"),
        # the first MLP linear of the hidden-5120 stack in training: pre-activation kept
        dict(name="linear 8192x20480x5120", op="linear", m=8192, n=20480, k=5120, w="in_out",
             act="gelu", bias=True, residual="none", pre=True, dtype="bf16", out="bf16"),
        # backward of a ragged batch through a linear without activation
        dict(name="linear backward ragged 777", op="linear_bwd", m=777, n=4104, k=2056,
             w="out_in", act="none", bias=True, dtype="bf16"),
        # backward of the hidden-2048 block's second MLP linear, through the GeLU before it
        dict(name="linear backward 8192x2048x8192", op="linear_bwd", m=8192, n=2048, k=8192,
             w="in_out", act="gelu", bias=True, dtype="bf16"),
        # the hidden-2048 block's parameters after its backward pass: fp32 masters and states
        dict(name="adamw 32-bit 50M", op="adamw", sizes=_block_sizes(2048, 8192), param="fp32+bf16",
             grad="fp32", bits=32, clip=True, step=1000),
        # one layer of the hidden-5120 stack with 8-bit states and bf16 gradients
        dict(name="adamw 8-bit 315M", op="adamw", sizes=_block_sizes(5120, 20480),
             param="fp32+bf16", grad="bf16", bits=8, clip=True, step=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "qk", "qk_bwd", "linear", "linear", "linear", "linear_bwd", "adamw"])
    if op in ("qk", "qk_bwd"):
        dh = rng.choice([64, 128])
        axes = rng.choice([1, 1, 2, 3])
        rot = rng.choice([dh, dh, dh // 2])
        k_heads = _log(rng, 1, 32)
        q_heads = k_heads * rng.choice([1, 1, 2, 4, 8])
        most = 32760 * 64 * 128 // ((q_heads + k_heads) * dh * (1 if op == "qk" else 2))
        tokens = _log(rng, 1, max(1, min(65536, most)))
        seq = rng.choice([1, tokens, max(1, tokens // rng.randint(1, 8)), _log(rng, 1, tokens)])
        half, parts = rot // 2, []
        for a in range(axes - 1):
            parts.append(rng.randint(1, half - sum(parts) - (axes - 1 - a)))
        parts.append(half - sum(parts))
        return dict(op=op, batch=max(1, tokens // seq), seq=seq, q_heads=q_heads, k_heads=k_heads,
                    head_dim=dh, rot=rot, pairing=rng.choice(["halves", "adjacent"]), axes=axes,
                    sections=",".join(map(str, parts)),
                    ladder=rng.choice(["shared", "per_axis"]) if axes > 1 else "shared",
                    norm=rng.random() < 0.8, far=rng.choice([0, 4096, 131072]),
                    packed=rng.random() < 0.5)
    if op in ("linear", "linear_bwd"):
        n, k = 8 * _log(rng, 8, 2560), 8 * _log(rng, 8, 2048)
        most = 8.5e11 / (2.0 * n * k) / (1 if op == "linear" else 2)
        m = _log(rng, 1, max(1, min(8192, int(most))))
        case = dict(op=op, m=m, n=n, k=k, w=rng.choice(["in_out", "out_in"]),
                    act=rng.choice(["none", "gelu", "gelu_tanh", "silu", "relu"]),
                    bias=rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "fp16"]))
        if op == "linear":
            case.update(residual=rng.choice(["none", "none", case["dtype"], "fp32"]),
                        pre=rng.random() < 0.3, out=rng.choice([case["dtype"], "fp32"]))
        return case
    sizes, left = [], 150_000_000
    for _ in range(_log(rng, 1, 200)):
        if left < 1:
            break
        n = _log(rng, 1, max(1, min(40_000_000, left)))
        sizes.append(n)
        left -= n
    return dict(op="adamw", sizes=",".join(map(str, sizes)),
                param=rng.choice(["fp32+bf16", "fp32", "bf16"]), grad=rng.choice(["fp32", "bf16"]),
                bits=rng.choice([32, 8]), clip=rng.random() < 0.7, step=_log(rng, 1, 100000))


DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


def work(case):
    if case["op"] in ("qk", "qk_bwd"):
        el = case["batch"] * case["seq"] * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
        pos = 4 * case["batch"] * case["seq"] * case["axes"]
        gam = 4 * case["head_dim"] if case["norm"] else 0
        if case["op"] == "qk":  # read and write every head once
            return dict(bytes=2 * 2 * el + pos + gam, flops=6 * el)
        # read the incoming gradient, and the heads where there is a norm; write the gradient
        return dict(bytes=(3 if case["norm"] else 2) * 2 * el + pos + 3 * gam, flops=14 * el)
    if case["op"] == "linear":
        m, n, k, e = case["m"], case["n"], case["k"], 2
        out = m * n * (4 if case["out"] == "fp32" else 2) + (m * n * e if case["pre"] else 0)
        if case["residual"] != "none":
            out += m * n * (4 if case["residual"] == "fp32" else 2)
        return dict(bytes=e * (m * k + k * n) + (e * n if case["bias"] else 0) + out,
                    flops=2 * m * n * k)
    if case["op"] == "linear_bwd":
        m, n, k, e = case["m"], case["n"], case["k"], 2
        acts = 2 if case["act"] == "none" else 3  # x, dx, and the pre-activation
        return dict(bytes=e * (m * n + acts * m * k + k * n) + 4 * k * n + 4 * n * case["bias"],
                    flops=4 * m * n * k)
    n = sum(_sizes(case))
    p = {"fp32+bf16": 4 + 4 + 2, "fp32": 8, "bf16": 4}[case["param"]]
    s = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return dict(bytes=n * (p + s + (4 if case["grad"] == "fp32" else 2)),
                flops=n * (15 + 2 * case["clip"]))


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _positions(case, g):
    """int32 [axes, batch, seq]: places in a sequence from `far` on, or on a grid."""
    b, s, axes = case["batch"], case["seq"], case["axes"]
    first = torch.randint(0, case["far"] + 1, (b, 1), generator=g, device="cuda")
    i = torch.arange(s, device="cuda").view(1, s)
    if axes == 1:
        at = [first + i]
    elif axes == 2:  # rows of an image
        w = max(1, math.isqrt(s))
        at = [first + i // w, first + i % w]
    else:            # frames of rows
        h, w = (30, 52) if s >= 1560 else (3, 5)
        at = [first + i // (h * w), first + i // w % h, first + i % w]
    return torch.stack(at).to(torch.int32).contiguous()


def _heads(case, g, scale):
    """q and k, [batch, seq, heads, head_dim]: views of one [q | k | v] buffer, or apart."""
    b, s, d, nq, nk = (case[n] for n in ("batch", "seq", "head_dim", "q_heads", "k_heads"))
    if case["packed"]:
        buf = _randn(g, (b, s, nq + 2 * nk, d), scale, torch.bfloat16)
        return buf[:, :, :nq], buf[:, :, nq:nq + nk]
    return (_randn(g, (b, s, nq, d), scale, torch.bfloat16),
            _randn(g, (b, s, nk, d), scale, torch.bfloat16))


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] in ("qk", "qk_bwd"):
        st["pos"] = _positions(case, g)
        st["q"], st["k"] = _heads(case, g, 1.7)
        for n in ("gq", "gk"):
            st[n] = (1.0 + 0.1 * torch.randn(case["head_dim"], generator=g, device="cuda")).to(
                torch.bfloat16) if case["norm"] else None
        if case["op"] == "qk_bwd":
            st["dq"], st["dk"] = _heads(case, g, 1e-3)
    elif case["op"] in ("linear", "linear_bwd"):
        m, n, k, dt = case["m"], case["n"], case["k"], DT[case["dtype"]]
        shape = (k, n) if case["w"] == "in_out" else (n, k)
        st["w"] = _randn(g, shape, 0.02, dt)
        st["x"] = _randn(g, (m, k), 1.0, dt)
        st["b"] = _randn(g, (n,), 0.02, dt) if case["bias"] else None
        if case["op"] == "linear":
            r = case["residual"]
            st["r"] = None if r == "none" else _randn(g, (m, n), 1.0, DT[r])
        else:
            st["dy"] = _randn(g, (m, n), 1e-2, dt)
            st["pre"] = None
            if case["act"] != "none":  # x is the activation of pre
                st["pre"] = _randn(g, (m, k), 1.0, dt)
                st["x"] = _act(case["act"], st["pre"].float()).to(dt)
    else:
        # the tensors lie in flat buffers, each from a whole block on; zeros between them
        sizes = _sizes(case)
        blocks = torch.tensor([-(-n // BLOCK) for n in sizes])
        st["first"] = (torch.cumsum(blocks, 0) - blocks).tolist()
        total = int(blocks.sum())
        live = torch.repeat_interleave(torch.tensor(sizes).cuda(), blocks.cuda()).view(-1, 1)
        start = torch.repeat_interleave(torch.tensor(st["first"]).cuda(), blocks.cuda())
        at = (torch.arange(total, device="cuda") - start).view(-1, 1) * BLOCK
        live = (at + torch.arange(BLOCK, device="cuda") < live).float()
        rows = torch.exp(_randn(g, (total, 1)))  # parts of a weight differ in gradient scale
        p = live * _randn(g, (total, BLOCK), 0.02)
        st["grad"] = (1e-3 * rows * live * _randn(g, (total, BLOCK))).to(
            DT[case["grad"]]).view(-1)
        m = 3e-4 * rows * live * _randn(g, (total, BLOCK))
        v = (1e-3 * rows) ** 2 * live * torch.exp(_randn(g, (total, BLOCK), 0.5))
        if case["step"] == 1:
            m, v = torch.zeros_like(m), torch.zeros_like(v)
        st["param"] = (p.to(torch.bfloat16) if case["param"] == "bf16" else p).view(-1)
        st["copy"] = p.to(torch.bfloat16).view(-1) if case["param"] == "fp32+bf16" else None
        if case["bits"] == 8:
            st["m"], st["m_scale"] = _pack(m)
            st["v"], st["v_scale"] = _pack(v.sqrt(), v > 0)
        else:
            st["m"], st["v"], st["m_scale"], st["v_scale"] = m.view(-1), v.view(-1), None, None
        # no weight decay for norms and biases
        st["decays"] = [0.1 if n >= 65536 else 0.0 for n in sizes]
        st["decay"] = torch.repeat_interleave(torch.tensor(st["decays"]).cuda(),
                                              blocks.cuda()).view(-1, 1)
    return st


# ------------------------------------------------------------------------- plain forms

def _act(name, z):
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    return z


def _act_grad(name, z):
    if name == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _frequencies(case):
    """(angle per position of every rotated pair, the axis it follows), as float64 / int64."""
    parts = [int(p) for p in case["sections"].split(",")]
    half = case["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(len(parts)), torch.tensor(parts))
    if case["ladder"] == "shared":
        e = torch.arange(half, dtype=torch.float64) / half
    else:
        e = torch.cat([torch.arange(p, dtype=torch.float64) / p for p in parts])
    return 10000.0 ** -e, axis


def _angles(case, pos):
    f, axis = _frequencies(case)
    return pos.to(torch.float64)[axis.to(pos.device)].permute(1, 2, 0) * f.to(pos.device)


def _split(case, x):
    """The two members of each rotated pair of the last dimension, and what stays."""
    r = case["rot"]
    if case["pairing"] == "halves":
        return x[..., :r // 2], x[..., r // 2:r], x[..., r:]
    return x[..., :r:2], x[..., 1:r:2], x[..., r:]


def _join(case, a, b, rest):
    if case["pairing"] == "halves":
        return torch.cat([a, b, rest], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _qk_plain(case, x, gamma, cos, sin):
    y = x.float()
    if gamma is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * gamma.float()
    a, b, rest = _split(case, y)
    return _join(case, a * cos - b * sin, a * sin + b * cos, rest).to(x.dtype)


def _qk_bwd_plain(case, x, gamma, dy, cos, sin):
    a, b, rest = _split(case, dy.float())
    d = _join(case, a * cos + b * sin, b * cos - a * sin, rest)
    if gamma is None:
        return d.to(dy.dtype), None
    xf = x.float()
    rstd = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
    xhat = xf * rstd
    dgamma = (d * xhat).sum((0, 1, 2))
    g = d * gamma.float()
    return (rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))).to(dy.dtype), dgamma


def _pack(y, keep=None):
    """E4M3 codes of [blocks, BLOCK] values and a scale for each block; where `keep` says so
    no code is zero."""
    amax = y.abs().amax(1, keepdim=True)
    inv = torch.where(amax > 0, E4M3_MAX / amax, torch.zeros_like(amax))
    c = (y * inv).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float()
    if keep is not None:
        c = torch.where(keep & (c < E4M3_MIN), torch.full_like(c, E4M3_MIN), c)
    return c.to(torch.float8_e4m3fn).view(-1), (amax / E4M3_MAX).view(-1)


def _adamw_plain(st):
    case = st["case"]
    b1, b2, lr, eps, step = 0.9, 0.95, 3e-4, 1e-8, case["step"]
    g, p, m, v = (st[n].float().view(-1, BLOCK) for n in ("grad", "param", "m", "v"))
    norm = None
    if case["clip"]:
        norm = g.square().sum(1).sum().sqrt()
        g = g * torch.clamp(1.0 / (norm + 1e-6), max=1.0)
    if case["bits"] == 8:
        m, v = m * st["m_scale"].view(-1, 1), (v * st["v_scale"].view(-1, 1)).square()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    up = (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + eps)
    p = p - lr * st["decay"] * p - lr * up
    st["param"].copy_(p.view(-1))
    if st["copy"] is not None:
        st["copy"].copy_(p.view(-1))
    if case["bits"] == 8:
        for name, x, keep in (("m", m, None), ("v", v.sqrt(), v > 0)):
            code, scale = _pack(x, keep)
            st[name].copy_(code)
            st[name + "_scale"].copy_(scale)
    else:
        st["m"].copy_(m.view(-1))
        st["v"].copy_(v.view(-1))
    return _adamw_out(st, norm)


def _adamw_out(st, norm):
    names = ("param", "copy", "m", "v", "m_scale", "v_scale")
    out = {n: st[n] for n in names if st[n] is not None}
    return out if norm is None else dict(out, norm=norm)


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if case["op"] in ("qk", "qk_bwd"):
        ang = _angles(case, st["pos"])
        cos, sin = ang.cos().float().unsqueeze(2), ang.sin().float().unsqueeze(2)
        if case["op"] == "qk":
            return (_qk_plain(case, st["q"], st["gq"], cos, sin),
                    _qk_plain(case, st["k"], st["gk"], cos, sin))
        dq, dgq = _qk_bwd_plain(case, st["q"], st["gq"], st["dq"], cos, sin)
        dk, dgk = _qk_bwd_plain(case, st["k"], st["gk"], st["dk"], cos, sin)
        return [t for t in (dq, dk, dgq, dgk) if t is not None]
    if case["op"] == "linear":
        w = st["w"].float()
        z = torch.matmul(st["x"].float(), w if case["w"] == "in_out" else w.t())
        if st["b"] is not None:
            z = z + st["b"].float()
        y = _act(case["act"], z)
        if st["r"] is not None:
            y = y + st["r"].float()
        y = y.to(DT[case["out"]])
        return (y, z.to(DT[case["dtype"]])) if case["pre"] else y
    if case["op"] == "linear_bwd":
        w, dy, x = st["w"].float(), st["dy"].float(), st["x"].float()
        dx = torch.matmul(dy, w.t() if case["w"] == "in_out" else w)
        if st["pre"] is not None:
            dx = dx * _act_grad(case["act"], st["pre"].float())
        dw = torch.matmul(x.t(), dy) if case["w"] == "in_out" else torch.matmul(dy.t(), x)
        out = [dx.to(st["dy"].dtype), dw]
        return out + [dy.sum(0)] if case["bias"] else out
    return _adamw_plain(st)


# ------------------------------------------------------------------- the library's calls

def _run_own(st):
    from transformer_block_gb300 import pb
    case = st["case"]
    if case["op"] in ("qk", "qk_bwd"):
        if "rope" not in st:
            st["rope"] = pb.Rope(case["head_dim"], rot_dim=case["rot"], theta=10000.0,
                                 pairing=case["pairing"], ladder=case["ladder"],
                                 sections=[int(p) for p in case["sections"].split(",")])
        if case["op"] == "qk":
            return pb.qk_norm_rope(st["rope"], st["q"], st["k"], st["pos"], gamma_q=st["gq"],
                                   gamma_k=st["gk"], eps=1e-6)
        out = pb.qk_norm_rope_backward(st["rope"], st["q"], st["k"], st["pos"], st["dq"],
                                       st["dk"], gamma_q=st["gq"], gamma_k=st["gk"], eps=1e-6)
        return [t for t in out if t is not None]
    if case["op"] in ("linear", "linear_bwd"):
        if "scratch" not in st:
            st["scratch"] = torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8,
                                        device="cuda")
        layout = pb.PB_WEIGHT_IN_OUT if case["w"] == "in_out" else pb.PB_WEIGHT_OUT_IN
        if case["op"] == "linear":
            pre = torch.empty(case["m"], case["n"], dtype=st["x"].dtype,
                              device="cuda") if case["pre"] else None
            y = pb.linear(st["x"], st["w"], st["b"], residual=st["r"], activation=case["act"],
                          layout=layout, out_dtype=DT[case["out"]], pre=pre,
                          scratch=st["scratch"])
            return (y, pre) if case["pre"] else y
        dx, dw, db = pb.linear_backward(st["dy"], st["x"], st["w"], pre=st["pre"],
                                        activation=case["act"], layout=layout,
                                        bias=case["bias"], scratch=st["scratch"])
        return [dx, dw, db] if case["bias"] else [dx, dw]
    if "adamw" not in st:
        def part(name, i, n, unit=1):
            at = st["first"][i] * BLOCK // unit
            return None if st[name] is None else st[name][at:at + -(-n // unit)]

        st["adamw"] = pb.AdamW(
            [dict(param=part("param", i, n), copy=part("copy", i, n), grad=part("grad", i, n),
                  m=part("m", i, n), v=part("v", i, n), m_scale=part("m_scale", i, n, BLOCK),
                  v_scale=part("v_scale", i, n, BLOCK), weight_decay=st["decays"][i])
             for i, n in enumerate(_sizes(case))], beta1=0.9, beta2=0.95, eps=1e-8)
    norm = st["adamw"].grad_norm(max_norm=1.0) if case["clip"] else None
    st["adamw"].step(lr=3e-4, step=case["step"], grad_scale=None if norm is None else norm[1:])
    return _adamw_out(st, None if norm is None else norm[0])


# ----------------------------------------------------------------- the definition in 64 bits

def _exact_qk(case, x, gamma, turn, dy=None):
    """Pairs as complex numbers: a rotation is a product with exp(i angle)."""
    r = case["rot"]
    xd = x.double()
    rstd = 1 / torch.sqrt(xd.pow(2).sum(-1, keepdim=True) / xd.shape[-1] + 1e-6)

    def rotated(y, by):
        pair = y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) \
            if case["pairing"] == "halves" else y[..., :r].unflatten(-1, (r // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * by.unsqueeze(2))
        z = (z.transpose(-1, -2) if case["pairing"] == "halves" else z).flatten(-2)
        return torch.cat([z, y[..., r:]], -1)

    if dy is None:
        return rotated(xd * rstd * gamma.double() if gamma is not None else xd, turn), None
    d = rotated(dy.double(), turn.conj())
    if gamma is None:
        return d, None
    n = xd * rstd
    dot = torch.einsum("bshd,bshd,d->bsh", d, n, gamma.double()).unsqueeze(-1) / xd.shape[-1]
    return rstd * (d * gamma.double() - n * dot), torch.einsum("bshd,bshd->d", d, n)


def _exact_act(name, z):
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z.clamp(min=0) if name == "relu" else z


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("qk", "qk_bwd"):
        f, axis = _frequencies(case)
        pos = st["pos"].double().cpu().numpy()
        ang = np.stack([pos[a] * w for a, w in zip(axis.tolist(), f.tolist())], -1)
        turn = torch.polar(torch.ones(ang.shape, dtype=torch.float64), torch.from_numpy(ang)).cuda()
        if case["op"] == "qk":
            return (_exact_qk(case, st["q"], st["gq"], turn)[0],
                    _exact_qk(case, st["k"], st["gk"], turn)[0])
        dq, dgq = _exact_qk(case, st["q"], st["gq"], turn, st["dq"])
        dk, dgk = _exact_qk(case, st["k"], st["gk"], turn, st["dk"])
        return [t for t in (dq, dk, dgq, dgk) if t is not None]
    if case["op"] == "linear":
        z = torch.einsum("mk,kn->mn" if case["w"] == "in_out" else "mk,nk->mn",
                         st["x"].double(), st["w"].double())
        z = z if st["b"] is None else z + st["b"].double()
        y = _exact_act(case["act"], z)
        y = y if st["r"] is None else y + st["r"].double()
        return (y, z) if case["pre"] else y
    if case["op"] == "linear_bwd":
        dy, x = st["dy"].double(), st["x"].double()
        dx = torch.einsum("mn,kn->mk" if case["w"] == "in_out" else "mn,nk->mk", dy,
                          st["w"].double())
        if st["pre"] is not None:
            z = st["pre"].double().requires_grad_(True)
            with torch.enable_grad():
                dx = torch.autograd.grad(_exact_act(case["act"], z), z, dx)[0]
        dw = torch.einsum("mk,mn->kn" if case["w"] == "in_out" else "mk,mn->nk", x, dy)
        return [dx, dw, dy.sum(0)] if case["bias"] else [dx, dw]
    b1, b2, n = 0.9, 0.95, case["step"]
    g, p, m, v = (st[x].double() for x in ("grad", "param", "m", "v"))
    norm = torch.linalg.vector_norm(g) if case["clip"] else None
    if norm is not None:
        g = g * min(1.0, 1.0 / (float(norm) + 1e-6))
    at = torch.arange(g.numel(), device="cuda") // BLOCK
    if case["bits"] == 8:
        m, v = m * st["m_scale"].double()[at], (v * st["v_scale"].double()[at]) ** 2
    m, v = m + (1 - b1) * (g - m), v + (1 - b2) * (g * g - v)
    down = m / -math.expm1(n * math.log(b1)) / (
        torch.sqrt(v / -math.expm1(n * math.log(b2))) + 1e-8)
    decay = torch.tensor(st["decays"], dtype=torch.float64, device="cuda")
    each = torch.tensor([-(-x // BLOCK) * BLOCK for x in _sizes(case)], device="cuda")
    st["param"] = p * (1 - 3e-4 * decay.repeat_interleave(each)) - 3e-4 * down
    st["copy"] = None if st["copy"] is None else st["param"]
    if case["bits"] == 32:
        st["m"], st["v"] = m, v
        return _adamw_out(st, norm)
    for name, x in (("m", m), ("v", v.sqrt())):
        scale = x.abs().view(-1, BLOCK).max(1).values / E4M3_MAX
        code = torch.where(scale[at] > 0, x / scale[at], torch.zeros_like(x))
        # nearest E4M3 value: steps of 2^-3 of the power of two below, 2^-9 at least
        unit = torch.exp2(torch.floor(torch.log2(code.abs().clamp(min=2.0 ** -6))) - 3)
        code = torch.round(code / unit) * unit
        if name == "v":
            code = torch.where((v > 0) & (code < E4M3_MIN), E4M3_MIN, code)
        st[name], st[name + "_scale"] = code, scale
    return _adamw_out(st, norm)
