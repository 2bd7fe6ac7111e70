"""Python binding of the C ABI in ``include/pb.h`` (argument marshalling only).

Every step of the forward pass runs in ``libpb.so``'s kernels; PyTorch only supplies
device memory and the current CUDA stream. There is no fallback: if the library has not
been built, or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

from . import build as _build
from .configs import Workload

PB_OK = 0
PB_ERR_DEVICE_TIMEOUT = 5
PB_ERR_RANGE = 7
STATUS_NAMES = {0: "PB_OK", 1: "PB_ERR_INVALID_ARG", 2: "PB_ERR_UNSUPPORTED",
                3: "PB_ERR_WORKSPACE", 4: "PB_ERR_CUDA", 5: "PB_ERR_DEVICE_TIMEOUT",
                6: "PB_ERR_BAD_HANDLE", 7: "PB_ERR_RANGE"}
PB_OPERANDS_BF16, PB_OPERANDS_FP16, PB_OPERANDS_FP8 = 0, 1, 2
PB_DTYPE_BF16, PB_DTYPE_FP16, PB_DTYPE_FP32 = 0, 1, 2
PB_WEIGHT_IN_OUT, PB_WEIGHT_OUT_IN = 0, 1
PB_ADAMW_BLOCK = 256
PB_ROPE_MAX_AXES = 4
ACTIVATIONS = {"none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3, "relu": 4}
ROPE_PAIRINGS = {"halves": 0, "adjacent": 1}
ROPE_LADDERS = {"shared": 0, "per_axis": 1}
_DTYPES = {torch.bfloat16: PB_DTYPE_BF16, torch.float16: PB_DTYPE_FP16,
           torch.float32: PB_DTYPE_FP32}


class PbError(RuntimeError):
    def __init__(self, func: str, status: int, message: str):
        super().__init__(f"{func}: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class pb_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seq", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("window", ctypes.c_int32), ("ln_eps", ctypes.c_float),
                ("variant", ctypes.c_int32)]


WEIGHT_FIELDS = ["ln_gamma", "ln_beta", "wqkv", "w1", "wo", "w2", "b_qkv", "b1", "b_o", "b2"]


class pb_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_FIELDS]


class pb_scratch_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("xn", "qk", "vt", "act", "io", "io2", "res0", "res1", "sk", "q8", "qscale", "seq_pad",
                 "total", "hpre", "lse", "d_attn", "delta", "dq_acc", "dz", "dxn", "stats",
                 "partials", "train_total")]


GRAD_FIELDS = ("dx", "dgamma", "dbeta", "dwqkv", "dw1", "dwo", "dw2", "db_qkv", "db1", "db_o",
               "db2")


class pb_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in GRAD_FIELDS]


class pb_options(ctypes.Structure):
    _fields_ = [("operand_precision", ctypes.c_int32), ("wait_limit_ns", ctypes.c_uint64)]


class pb_rope(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("head_dim", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("pairing", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("section_end", ctypes.c_int32 * PB_ROPE_MAX_AXES),
                ("turns", ctypes.c_uint64 * 128)]


class pb_heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("batch_stride", ctypes.c_int64), ("seq_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class pb_block_rope(ctypes.Structure):
    _fields_ = [("rope", pb_rope), ("gamma_q", ctypes.c_void_p), ("gamma_k", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("positions", ctypes.c_void_p),
                ("saved", ctypes.c_void_p), ("saved_bytes", ctypes.c_size_t),
                ("dgamma_q", ctypes.c_void_p), ("dgamma_k", ctypes.c_void_p)]


class pb_linear_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("m", "n", "k", "dtype", "w_layout", "activation")] + [
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p),
        ("ldw", ctypes.c_int64), ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
        ("ldr", ctypes.c_int64), ("residual_dtype", ctypes.c_int32), ("pre", ctypes.c_void_p),
        ("ldp", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
        ("y_dtype", ctypes.c_int32)]


class pb_linear_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("m", "n", "k", "dtype", "w_layout", "activation", "accumulate")] + [
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("x", ctypes.c_void_p),
        ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64),
        ("pre", ctypes.c_void_p), ("ldp", ctypes.c_int64), ("dx", ctypes.c_void_p),
        ("lddx", ctypes.c_int64), ("dw", ctypes.c_void_p), ("lddw", ctypes.c_int64),
        ("db", ctypes.c_void_p)]


class pb_adamw_tensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64)] + [
        (n, ctypes.c_void_p) for n in ("param", "param_copy", "grad", "m", "v", "m_scale",
                                       "v_scale")] + [("weight_decay", ctypes.c_float)]


class pb_adamw_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps")] + [
        ("step", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32),
        ("d_lr", ctypes.c_void_p), ("d_step", ctypes.c_void_p),
        ("d_grad_scale", ctypes.c_void_p)]


# name -> (restype, argtypes); every function of include/pb.h
_P, _S, _I32, _I64, _U64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, \
    ctypes.c_uint64
_DP = ctypes.POINTER(pb_dims)
SIGNATURES = {
    "pb_weight_workspace_bytes": (ctypes.c_int, [_DP, ctypes.POINTER(_S)]),
    "pb_scratch_bytes": (ctypes.c_int, [_DP, ctypes.POINTER(_S)]),
    "pb_get_scratch_layout": (ctypes.c_int, [_DP, ctypes.POINTER(pb_scratch_layout)]),
    "pb_create": (ctypes.c_int, [_DP, ctypes.POINTER(pb_weights), _P, _S, _P,
                                 ctypes.POINTER(_P)]),
    "pb_create_ex": (ctypes.c_int, [_DP, ctypes.POINTER(pb_weights),
                                    ctypes.POINTER(pb_options), _P, _S, _P, ctypes.POINTER(_P)]),
    "pb_forward": (ctypes.c_int, [_P, _P, _P, _P, _S, _P]),
    "pb_forward_serial": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _S, _P]),
    "pb_forward_stack": (ctypes.c_int, [ctypes.POINTER(_P), _I32, _P, _P, _P, _S, _P]),
    "pb_forward_stack_host": (ctypes.c_int, [ctypes.POINTER(_P), _I32, _P, _P, _P, _S, _P]),
    "pb_forward_stack_f32": (ctypes.c_int, [ctypes.POINTER(_P), _I32, _P, _P, _P, _S, _P]),
    "pb_get_status": (ctypes.c_int, [_P]),
    "pb_clear_status": (ctypes.c_int, [_P, _P]),
    "pb_set_wait_limit_ns": (ctypes.c_int, [_P, _U64]),
    "pb_trace_enable": (ctypes.c_int, [_P, _I32]),
    "pb_trace_read": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(_I32)]),
    "pb_destroy": (ctypes.c_int, [_P]),
    "pb_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pb_last_error_message": (ctypes.c_char_p, []),
    "pb_layernorm": (ctypes.c_int, [_I64, _I32, _P, _P, _P, ctypes.c_float, _P, _P]),
    "pb_quantize_rows_e4m3": (ctypes.c_int, [_I64, _I32, _P, _P, _P, _P]),
    "pb_train_scratch_bytes": (ctypes.c_int, [_P, _P]),
    "pb_forward_train": (ctypes.c_int, [_P, _P, _P, _P, _S, _P]),
    "pb_forward_stack_host_steps": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P, _S, _P]),
    "pb_backward": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _S, _P]),
    "pb_gemm_scratch_bytes": (ctypes.c_int, [ctypes.POINTER(_S)]),
    "pb_gemm_bf16": (ctypes.c_int, [_I32, _I32, _I32, _P, _P, _P, _P, _S, _P, _P]),
    "pb_gemm_bf16_layout": (ctypes.c_int, [_I32, _I32, _I32, _P, _I32, _P, _I32, _P, _P, _S, _P,
                                           _P]),
    "pb_swa_attention": (ctypes.c_int, [_DP, _P, _P, _P, _I64, _P, _P]),
    "pb_wait_probe": (ctypes.c_int, [_U64, _P, _P]),
    "pb_gemm_bf16_static": (ctypes.c_int, [_I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "pb_set_guard_bytes": (ctypes.c_int, [_S]),
    "pb_get_guard_bytes": (ctypes.c_int, [ctypes.POINTER(_S)]),
    "pb_rope_init": (ctypes.c_int, [_I32, _I32, _I32, _I32, _P, _I32, ctypes.c_double, _P, _P]),
    "pb_qk_norm_rope": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P,
                                       _P]),
    "pb_set_qk_norm_rope": (ctypes.c_int, [_P, _P]),
    "pb_qk_norm_rope_scratch_bytes": (ctypes.c_int, [ctypes.POINTER(_S)]),
    "pb_qk_norm_rope_backward": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P, _P, ctypes.c_float,
                                                _P, _P, _P, _P, _P, _P, _P, _I32, _P, _S, _P]),
    "pb_linear_scratch_bytes": (ctypes.c_int, [ctypes.POINTER(_S)]),
    "pb_linear": (ctypes.c_int, [_P, _P, _S, _P, _P]),
    "pb_linear_backward": (ctypes.c_int, [_P, _P, _S, _P, _P]),
    "pb_activation_backward": (ctypes.c_int, [_I64, _I64, _I32, _I32, _P, _I64, _P, _I64, _P,
                                              _I64, _P]),
    "pb_adamw": (ctypes.c_int, [_P, _I32, _P, _P]),
    "pb_grad_norm_scratch_bytes": (ctypes.c_int, [_I32, ctypes.POINTER(_S)]),
    "pb_grad_norm": (ctypes.c_int, [_I32, _P, _I32, ctypes.c_float, _P, _P, _S, _P]),
}

_lib = None


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded ``libpb.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with transformer_block_gb300.build."
                               "build(); the forward pass has no other implementation")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(func: str, status: int):
    if status != PB_OK:
        msg = lib().pb_last_error_message()
        raise PbError(func, status, msg.decode() if msg else "")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:  # the raw handle: no Stream object for every call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_dims(wl: Workload | None = None, **kw) -> pb_dims:
    src = dict(wl.__dict__) if wl is not None else {}
    src.update(kw)
    return pb_dims(src["batch"], src["seq"], src["hidden"], src["heads"], src["head_dim"],
                   src["ffn"], src["window"], float(src.get("ln_eps", 1e-5)),
                   int(src.get("variant", 0)))


def weight_workspace_bytes(dims: pb_dims) -> int:
    n = ctypes.c_size_t()
    _check("pb_weight_workspace_bytes", lib().pb_weight_workspace_bytes(ctypes.byref(dims),
                                                                        ctypes.byref(n)))
    return n.value


def scratch_bytes(dims: pb_dims) -> int:
    n = ctypes.c_size_t()
    _check("pb_scratch_bytes", lib().pb_scratch_bytes(ctypes.byref(dims), ctypes.byref(n)))
    return n.value


def train_scratch_bytes(dims: pb_dims) -> int:
    n = ctypes.c_size_t()
    _check("pb_train_scratch_bytes", lib().pb_train_scratch_bytes(ctypes.byref(dims),
                                                                  ctypes.byref(n)))
    return n.value


def new_train_scratch(dims: pb_dims, device="cuda") -> torch.Tensor:
    return torch.empty(train_scratch_bytes(dims), dtype=torch.uint8, device=device)


def scratch_layout(dims: pb_dims) -> pb_scratch_layout:
    L = pb_scratch_layout()
    _check("pb_get_scratch_layout", lib().pb_get_scratch_layout(ctypes.byref(dims),
                                                                ctypes.byref(L)))
    return L


def new_scratch(dims: pb_dims, device="cuda") -> torch.Tensor:
    return torch.empty(scratch_bytes(dims), dtype=torch.uint8, device=device)


def scratch_view(scratch: torch.Tensor, dims: pb_dims, name: str,
                 dtype=torch.bfloat16) -> torch.Tensor:
    """A view of one intermediate in the scratch (``xn, qk, vt, act, io, res0, res1, q8,
    qscale``); ``dtype`` is the element type it holds (fp16 for ``xn``/``act`` with fp16
    operands, uint8 E4M3 codes for ``xn`` with FP8 operands; ``res0``/``res1``/``qscale``
    are always fp32 and ``q8`` uint8)."""
    L = scratch_layout(dims)
    T, H, F = dims.batch * dims.seq, dims.hidden, dims.ffn
    shapes = {"xn": (T, H), "qk": (T, 2 * H), "act": (T, H + F), "io": (T, H),
              "res0": (T, H), "res1": (T, H),
              "vt": (dims.batch, dims.heads, dims.head_dim, L.seq_pad),
              "q8": (T, H + F), "qscale": (2 * T,)}
    Fp = 2 * F if dims.variant == 1 else F
    nrow = dims.batch * dims.heads * ((dims.seq + 63) // 64 * 64)
    shapes.update({"hpre": (T, Fp), "lse": (nrow,), "d_attn": (T, H), "delta": (nrow,),
                   "dq_acc": (T, H), "dz": (T, 3 * H + Fp), "dxn": (T, H)})
    if name in ("res0", "res1", "qscale", "lse", "delta", "dq_acc", "dxn"):
        dtype = torch.float32
    elif name == "q8":
        dtype = torch.uint8
    shape = shapes[name]
    n = 1
    for s in shape:
        n *= s
    off = getattr(L, name)
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    return scratch[off:off + nbytes].view(dtype).view(*shape)


class ParallelBlock:
    """One parallel transformer block: a ``pb_handle`` plus the workspace it owns."""

    def __init__(self, dims: pb_dims, params: dict, stream=None,
                 operand_precision: int = PB_OPERANDS_BF16, wait_limit_ns: int = 0,
                 workspace: torch.Tensor | None = None):
        """``workspace``: a caller-provided uint8 CUDA tensor of at least
        ``weight_workspace_bytes(dims)`` (256-byte aligned), else one is allocated."""
        self.dims = dims
        self.operand_precision = operand_precision
        self._lib = lib()
        dev = params["wqkv"].device
        if workspace is None:
            workspace = torch.empty(weight_workspace_bytes(dims), dtype=torch.uint8, device=dev)
        self.workspace = workspace
        w = pb_weights(*[_ptr(params.get(n)) for n in WEIGHT_FIELDS])
        opt = pb_options(operand_precision, wait_limit_ns)
        h = ctypes.c_void_p()
        _check("pb_create_ex", self._lib.pb_create_ex(ctypes.byref(dims), ctypes.byref(w),
                                                      ctypes.byref(opt), _ptr(self.workspace),
                                                      self.workspace.numel(), _stream(stream),
                                                      ctypes.byref(h)))
        self.handle = h
        self._rope, self._rope_saved, self.rope_grads = None, None, {}

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None,
                scratch: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if y is None:
            y = torch.empty_like(x)
        if scratch is None:
            scratch = new_scratch(self.dims, x.device)
        _check("pb_forward", self._lib.pb_forward(self.handle, _ptr(x), _ptr(y), _ptr(scratch),
                                                  scratch.numel(), _stream(stream)))
        return y

    __call__ = forward

    def forward_serial(self, x: torch.Tensor, y: torch.Tensor | None = None,
                       ln2_gamma: torch.Tensor | None = None, ln2_beta: torch.Tensor | None = None,
                       scratch: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The serial block of eq. (3) on the same weights (``pb_forward_serial``)."""
        if y is None:
            y = torch.empty_like(x)
        if scratch is None:
            scratch = new_scratch(self.dims, x.device)
        _check("pb_forward_serial",
               self._lib.pb_forward_serial(self.handle, _ptr(x), _ptr(y), _ptr(ln2_gamma),
                                           _ptr(ln2_beta), _ptr(scratch), scratch.numel(),
                                           _stream(stream)))
        return y

    def forward_train(self, x: torch.Tensor, scratch: torch.Tensor, y: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
        """``pb_forward_train``: the forward pass, keeping in ``scratch`` (a training
        scratch, ``new_train_scratch``) what ``backward`` reads."""
        if y is None:
            y = torch.empty_like(x)
        _check("pb_forward_train",
               self._lib.pb_forward_train(self.handle, _ptr(x), _ptr(y), _ptr(scratch),
                                          scratch.numel(), _stream(stream)))
        return y

    def backward(self, x: torch.Tensor, dy: torch.Tensor, scratch: torch.Tensor,
                 grads: dict | None = None, accumulate: bool = False, biases: bool = True,
                 stream=None) -> dict:
        """``pb_backward`` after ``forward_train(x, scratch)``: returns the gradients (``dx``
        bf16, the parameter gradients fp32 in their ``pb_weights`` layout, keyed like
        ``GRAD_FIELDS``). ``grads`` may hold preallocated buffers (needed for
        ``accumulate``)."""
        d = self.dims
        H, F, T = d.hidden, d.ffn, d.batch * d.seq
        Fp = 2 * F if d.variant == 1 else F
        shapes = {"dx": (T, H), "dgamma": (H,), "dbeta": (H,), "dwqkv": (H, 3 * H),
                  "dw1": (H, Fp), "dwo": (H, H), "dw2": (F, H), "db_qkv": (3 * H,),
                  "db1": (Fp,), "db_o": (H,), "db2": (H,)}
        g = dict(grads or {})
        for n, shp in shapes.items():
            if n in g:
                continue
            if n in ("db_qkv", "db1", "db_o", "db2") and not biases:
                continue
            if n == "dbeta" and d.variant == 1:
                continue
            dt = torch.bfloat16 if n == "dx" else torch.float32
            g[n] = torch.zeros(shp, dtype=dt, device=x.device)
        gs = pb_grads(*[_ptr(g.get(n)) for n in GRAD_FIELDS])
        _check("pb_backward",
               self._lib.pb_backward(self.handle, _ptr(x), _ptr(dy), ctypes.byref(gs),
                                     int(accumulate), _ptr(scratch), scratch.numel(),
                                     _stream(stream)))
        return g

    def set_qk_norm_rope(self, rope: "Rope | None", gamma_q=None, gamma_k=None,
                         eps: float = 1e-6, positions=None, training: bool = False, saved=None):
        """``pb_set_qk_norm_rope``: q and k are normed (where there is a gamma) and rotated at
        ``positions`` (int32 [axes, batch, seq], or None) before the attention, in every call
        from now on; ``rope=None`` takes that out. The tensors are kept and read by each call.
        ``training`` makes the gradients ``self.rope_grads`` (``dgamma_q``, ``dgamma_k``: fp32,
        written by ``backward``). What ``forward_train`` keeps of its last call is in a buffer of
        the block's, the same for every such call; for several forwards in flight give each a
        ``saved`` of its own (a uint8 CUDA tensor of batch * seq * hidden * 4 bytes), set before
        it and again before its ``backward``. Between the two, gammas, positions and eps are the
        caller's to keep the same; a ``backward`` whose q and k are no longer kept is refused."""
        if rope is None:
            _check("pb_set_qk_norm_rope", self._lib.pb_set_qk_norm_rope(self.handle, None))
            self._rope, self.rope_grads = None, {}
            return
        d = self.dims
        _here(gamma_q, gamma_k, positions, saved, self.workspace)
        n, grads = d.batch * d.seq * d.hidden * 4, {}
        if saved is not None:
            _is(training, "saved goes with training")
            _is(saved.dtype is torch.uint8 and saved.is_contiguous() and saved.numel() >= n,
                f"saved must be {n} contiguous bytes (uint8)")
        if training and (gamma_q is not None or gamma_k is not None):
            if saved is None:
                if self._rope_saved is None:
                    self._rope_saved = torch.empty(n, dtype=torch.uint8,
                                                   device=self.workspace.device)
                saved = self._rope_saved
            for name, g in (("dgamma_q", gamma_q), ("dgamma_k", gamma_k)):
                if g is not None:
                    grads[name] = torch.zeros(d.head_dim, dtype=torch.float32, device=g.device)
        r = pb_block_rope(rope.plan, _flat(gamma_q, d.head_dim, torch.bfloat16, "gamma_q"),
                          _flat(gamma_k, d.head_dim, torch.bfloat16, "gamma_k"), eps,
                          _positions(rope, positions, d.batch, d.seq), _ptr(saved),
                          0 if saved is None else saved.numel(), _ptr(grads.get("dgamma_q")),
                          _ptr(grads.get("dgamma_k")))
        _check("pb_set_qk_norm_rope",
               self._lib.pb_set_qk_norm_rope(self.handle, ctypes.byref(r)))
        self._rope, self.rope_grads = (gamma_q, gamma_k, positions, saved), grads

    def status(self) -> int:
        return self._lib.pb_get_status(self.handle)

    def clear_status(self, stream=None):
        _check("pb_clear_status", self._lib.pb_clear_status(self.handle, _stream(stream)))

    def set_wait_limit_ns(self, ns: int):
        _check("pb_set_wait_limit_ns", self._lib.pb_set_wait_limit_ns(self.handle, int(ns)))

    def trace_enable(self, n_calls: int):
        _check("pb_trace_enable", self._lib.pb_trace_enable(self.handle, int(n_calls)))

    def trace_read(self):
        """Summed ms of [LayerNorm, first GEMM, attention, second GEMM] and the call count."""
        ms = (ctypes.c_float * 4)()
        n = ctypes.c_int32()
        _check("pb_trace_read", self._lib.pb_trace_read(self.handle, ms, ctypes.byref(n)))
        return list(ms), n.value

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _check("pb_destroy", self._lib.pb_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _handles(blocks):
    arr = (ctypes.c_void_p * len(blocks))(*[b.handle.value for b in blocks])
    return arr


def forward_stack(blocks, x, y=None, scratch=None, stream=None):
    if y is None:
        y = torch.empty_like(x)
    if scratch is None:
        scratch = new_scratch(blocks[0].dims, x.device)
    _check("pb_forward_stack", lib().pb_forward_stack(_handles(blocks), len(blocks), _ptr(x),
                                                      _ptr(y), _ptr(scratch), scratch.numel(),
                                                      _stream(stream)))
    return y


def forward_stack_f32(blocks, x, y=None, scratch=None, stream=None):
    """``forward_stack`` returning the fp32 residual stream (float32 [T, H]) instead of its
    bf16 rounding (``pb_forward_stack_f32``)."""
    if y is None:
        y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    if scratch is None:
        scratch = new_scratch(blocks[0].dims, x.device)
    _check("pb_forward_stack_f32", lib().pb_forward_stack_f32(_handles(blocks), len(blocks),
                                                              _ptr(x), _ptr(y), _ptr(scratch),
                                                              scratch.numel(), _stream(stream)))
    return y


def forward_stack_host(blocks, x_host, y_host, scratch, stream=None):
    """Host (pinned) x -> device -> stack -> host y, enqueued on ``stream``."""
    _check("pb_forward_stack_host",
           lib().pb_forward_stack_host(_handles(blocks), len(blocks), _ptr(x_host), _ptr(y_host),
                                       _ptr(scratch), scratch.numel(), _stream(stream)))
    return y_host


def forward_stack_host_steps(blocks, x_hosts, y_hosts, scratch, stream=None):
    """Host (pinned) x_hosts[s] -> stack -> y_hosts[s] for every step s, the copies of
    neighbouring steps overlapping each step's compute (``pb_forward_stack_host_steps``)."""
    n = len(x_hosts)
    assert len(y_hosts) == n
    xs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in x_hosts])
    ys = (ctypes.c_void_p * n)(*[t.data_ptr() for t in y_hosts])
    _check("pb_forward_stack_host_steps",
           lib().pb_forward_stack_host_steps(_handles(blocks), len(blocks), n, xs, ys,
                                             _ptr(scratch), scratch.numel(), _stream(stream)))
    return y_hosts


def layernorm(x, gamma, beta, eps=1e-5, out=None, stream=None):
    if out is None:
        out = torch.empty_like(x)
    _check("pb_layernorm", lib().pb_layernorm(x.shape[0], x.shape[1], _ptr(x), _ptr(gamma),
                                              _ptr(beta), float(eps), _ptr(out),
                                              _stream(stream)))
    return out


def set_guard_bytes(n: int):
    """Unused bytes after every workspace and scratch region of the layouts computed from
    now on (``pb_set_guard_bytes``; process-wide, a debugging aid)."""
    _check("pb_set_guard_bytes", lib().pb_set_guard_bytes(int(n)))


def guard_bytes() -> int:
    n = ctypes.c_size_t()
    _check("pb_get_guard_bytes", lib().pb_get_guard_bytes(ctypes.byref(n)))
    return n.value


def gemm_scratch_bytes() -> int:
    n = ctypes.c_size_t()
    _check("pb_gemm_scratch_bytes", lib().pb_gemm_scratch_bytes(ctypes.byref(n)))
    return n.value


def gemm(a, b, out=None, scratch=None, status=None, stream=None):
    """``a [M, K] @ b[N, K]^T`` -> bf16 ``[M, N]`` on the tensor cores; ``scratch`` (a uint8
    CUDA tensor of ``gemm_scratch_bytes()``) enables stream-K for the last waves."""
    M, K = a.shape
    N = b.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    nbytes = 0 if scratch is None else scratch.numel()
    _check("pb_gemm_bf16", lib().pb_gemm_bf16(M, N, K, _ptr(a), _ptr(b), _ptr(out), _ptr(scratch),
                                              nbytes, _ptr(status), _stream(stream)))
    return out


def gemm_layout(a, b, a_mn=False, b_mn=False, out=None, scratch=None, status=None,
                stream=None):
    """``C[m, n] = sum_k A(m, k) B(n, k)`` -> bf16 ``[M, N]`` with ``a`` stored ``[M, K]``
    (or ``[K, M]`` when ``a_mn``) and ``b`` stored ``[N, K]`` (or ``[K, N]`` when ``b_mn``)."""
    M, K = (a.shape[1], a.shape[0]) if a_mn else a.shape
    N = b.shape[1] if b_mn else b.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    nbytes = 0 if scratch is None else scratch.numel()
    _check("pb_gemm_bf16_layout",
           lib().pb_gemm_bf16_layout(M, N, K, _ptr(a), int(a_mn), _ptr(b), int(b_mn), _ptr(out),
                                     _ptr(scratch), nbytes, _ptr(status), _stream(stream)))
    return out


def gemm_static(a, b, out=None, status=None, stream=None):
    """``gemm`` without caller scratch: the stream-K partial tiles live in the library's
    own fixed device array (for callers that cannot allocate; calls must not overlap)."""
    M, K = a.shape
    N = b.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _check("pb_gemm_bf16_static", lib().pb_gemm_bf16_static(M, N, K, _ptr(a), _ptr(b), _ptr(out),
                                                            _ptr(status), _stream(stream)))
    return out


def quantize_rows_e4m3(x: torch.Tensor, stream=None):
    """Per-row current scaling of a bf16 [rows, cols] CUDA tensor to FP8 E4M3 codes
    (``pb_quantize_rows_e4m3``): returns ``(codes uint8 [rows, cols], scales fp32 [rows])``."""
    rows, cols = x.shape
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check("pb_quantize_rows_e4m3", lib().pb_quantize_rows_e4m3(rows, cols, _ptr(x), _ptr(codes),
                                                                _ptr(scales), _stream(stream)))
    return codes, scales


def swa_attention(dims: pb_dims, qk, vt, act, status=None, stream=None):
    _check("pb_swa_attention", lib().pb_swa_attention(ctypes.byref(dims), _ptr(qk), _ptr(vt),
                                                      _ptr(act), act.shape[1], _ptr(status),
                                                      _stream(stream)))
    return act


def wait_probe(limit_ns: int, status: torch.Tensor, stream=None):
    """Runs the bounded-wait self-test kernel; ``status`` is a 1-element int32 CUDA tensor."""
    _check("pb_wait_probe", lib().pb_wait_probe(int(limit_ns), _ptr(status), _stream(stream)))


# ------------------------------------------------------------------- arguments of the steps
# below: the library sees pointers and strides only, so what a tensor knows is checked here.

def _here(*tensors):
    """Every given tensor is a CUDA tensor on the current device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")


def _run_on(stream, call, *args):
    """``call`` with ``stream`` (a torch.cuda.Stream or a raw handle) as the current stream, so
    that what it allocates belongs to that stream and is not handed out again before its work
    on it is done."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return call(*args)


def _is(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


def _rows(t: torch.Tensor, rows: int, cols: int, dtype, what: str) -> int:
    """A [rows, cols] tensor with contiguous rows; returns its row stride."""
    if t.dtype is not dtype or t.dim() != 2 or t.size(0) != rows or t.size(1) != cols:
        raise ValueError(f"{what} must be [{rows}, {cols}] {dtype}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{what}: the values of a row must be contiguous")
    return s0 if rows > 1 else cols + (-cols) % 8


def _new_rows(rows: int, cols: int, dtype, device, zero: bool = False) -> torch.Tensor:
    """A new [rows, cols] tensor whose rows start on 16-byte boundaries."""
    new = torch.zeros if zero else torch.empty
    return new((rows, cols + (-cols) % 8), dtype=dtype, device=device)[:, :cols] if cols % 8 else \
        new((rows, cols), dtype=dtype, device=device)


def _flat(t, n: int, dtype, what: str):
    """A contiguous tensor of n values, or None; returns its address."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be {n} contiguous values of {dtype}")
    return t.data_ptr()


# ------------------------------------------------------------------- query/key norm, rotation

class Rope:
    """The plan of a rotation (``pb_rope_init``): ``sections`` are the pairs of each axis
    (their sum is ``rot_dim / 2``; default one axis), ``inv_freq`` radians a position of every
    pair instead of ``theta``'s ladder. Host memory only; may be shared."""

    def __init__(self, head_dim: int, rot_dim: int | None = None, theta: float = 10000.0,
                 pairing: str = "halves", sections=None, ladder: str = "shared", inv_freq=None):
        rot_dim = head_dim if rot_dim is None else rot_dim
        n = 1 if sections is None else len(sections)
        sec = None if sections is None else (ctypes.c_int32 * n)(*sections)
        freq = None
        if inv_freq is not None:
            _is(len(inv_freq) == rot_dim // 2, "inv_freq must have rot_dim / 2 values")
            freq = (ctypes.c_double * max(1, len(inv_freq)))(*[float(f) for f in inv_freq])
        self.plan = pb_rope()
        self.head_dim, self.axes = head_dim, n
        _check("pb_rope_init", lib().pb_rope_init(
            head_dim, rot_dim, ROPE_PAIRINGS[pairing], n, sec, ROPE_LADDERS[ladder],
            float(theta), freq, ctypes.byref(self.plan)))


# pb_heads as bytes: cheaper to make for every call than a ctypes structure
_pack_heads = struct.Struct("@Piqqq").pack
assert struct.calcsize("@Piqqq") == ctypes.sizeof(pb_heads)


def _heads(t, head_dim: int, b: int, s: int, what: str):
    """``pb_heads`` of a [batch, seq, heads, head_dim] bf16 view."""
    if t is None:
        return None
    if t.dtype is not torch.bfloat16 or t.dim() != 4:
        raise ValueError(f"{what} must be a bfloat16 [batch, seq, heads, head_dim]")
    n0, n1, h, d = t.shape
    s0, s1, s2, s3 = t.stride()
    if n0 != b or n1 != s or d != head_dim or s3 != 1:
        raise ValueError(f"{what} must be [{b}, {s}, heads, {head_dim}], a head's values "
                         "contiguous")
    return _pack_heads(t.data_ptr(), h, s0 if b > 1 else 0, s1 if s > 1 else 0,
                       s2 if h > 1 else 0)


def _positions(rope, positions, b: int, s: int):
    if positions is None:
        return None
    # the same values in another order have as many: an order shows in the lengths beyond 1
    if positions.dim() > 1 and [n for n in positions.shape if n != 1] != \
            [n for n in (rope.axes, b, s) if n != 1]:
        raise ValueError(f"positions must be [{rope.axes}, {b}, {s}] (axes, batch, seq)")
    return _flat(positions, rope.axes * b * s, torch.int32, "positions ([axes, batch, seq])")


def qk_norm_rope(rope: Rope, q, k, positions=None, gamma_q=None, gamma_k=None, eps: float = 1e-6,
                 out_q=None, out_k=None, stream=None):
    """``pb_qk_norm_rope``: norm (where there is a gamma) and rotation of ``q`` and ``k``
    ([batch, seq, heads, head_dim] bf16 views, either may be None) at ``positions`` (int32
    [axes, batch, seq]; None: 0, 1, ... in each sequence). ``out_q=q`` works in place."""
    if stream is not None:
        return _run_on(stream, qk_norm_rope, rope, q, k, positions, gamma_q, gamma_k, eps, out_q,
                       out_k)
    first = q if q is not None else k
    _is(first is not None, "q and k are both None")
    b, s = first.size(0), first.size(1)
    if q is not None and out_q is None:
        out_q = torch.empty_like(q, memory_format=torch.contiguous_format)
    if k is not None and out_k is None:
        out_k = torch.empty_like(k, memory_format=torch.contiguous_format)
    _here(q, k, positions, gamma_q, gamma_k, out_q, out_k)
    d = rope.head_dim
    _check("pb_qk_norm_rope", lib().pb_qk_norm_rope(
        ctypes.addressof(rope.plan), b, s, _heads(q, d, b, s, "q"), _heads(k, d, b, s, "k"),
        _flat(gamma_q, d, torch.bfloat16, "gamma_q"),
        _flat(gamma_k, d, torch.bfloat16, "gamma_k"), eps, _positions(rope, positions, b, s),
        _heads(out_q, d, b, s, "out_q"), _heads(out_k, d, b, s, "out_k"), _stream(stream)))
    return out_q, out_k


@functools.cache
def qk_norm_rope_scratch_bytes() -> int:
    n = ctypes.c_size_t()
    _check("pb_qk_norm_rope_scratch_bytes", lib().pb_qk_norm_rope_scratch_bytes(ctypes.byref(n)))
    return n.value


def qk_norm_rope_backward(rope: Rope, q, k, positions, dq, dk, gamma_q=None, gamma_k=None,
                          eps: float = 1e-6, out_dq=None, out_dk=None, dgamma_q=None,
                          dgamma_k=None, accumulate: bool = False, scratch=None, stream=None):
    """``pb_qk_norm_rope_backward``: ``(dq, dk, dgamma_q, dgamma_k)`` of the forward call's
    inputs, from the gradients ``dq``, ``dk`` of its results. ``q`` and ``k`` are the forward's
    inputs (None where there is no gamma); a gamma's gradient is fp32 [head_dim], None without
    that gamma, and added to with ``accumulate`` (give the buffer)."""
    if stream is not None:
        return _run_on(stream, qk_norm_rope_backward, rope, q, k, positions, dq, dk, gamma_q,
                       gamma_k, eps, out_dq, out_dk, dgamma_q, dgamma_k, accumulate, scratch)
    first = dq if dq is not None else dk
    _is(first is not None, "dq and dk are both None")
    b, s = first.size(0), first.size(1)
    d, dev = rope.head_dim, first.device
    if dq is not None and out_dq is None:
        out_dq = torch.empty_like(dq, memory_format=torch.contiguous_format)
    if dk is not None and out_dk is None:
        out_dk = torch.empty_like(dk, memory_format=torch.contiguous_format)
    new = torch.zeros if accumulate else torch.empty
    if gamma_q is not None and dq is not None and dgamma_q is None:
        dgamma_q = new(d, dtype=torch.float32, device=dev)
    if gamma_k is not None and dk is not None and dgamma_k is None:
        dgamma_k = new(d, dtype=torch.float32, device=dev)
    if scratch is None and (gamma_q is not None or gamma_k is not None):
        scratch = torch.empty(qk_norm_rope_scratch_bytes(), dtype=torch.uint8, device=dev)
    _here(q, k, positions, dq, dk, gamma_q, gamma_k, out_dq, out_dk, dgamma_q, dgamma_k, scratch)
    _check("pb_qk_norm_rope_backward", lib().pb_qk_norm_rope_backward(
        ctypes.addressof(rope.plan), b, s, _heads(q, d, b, s, "q"), _heads(k, d, b, s, "k"),
        _flat(gamma_q, d, torch.bfloat16, "gamma_q"),
        _flat(gamma_k, d, torch.bfloat16, "gamma_k"), eps, _positions(rope, positions, b, s),
        _heads(dq, d, b, s, "dq"), _heads(dk, d, b, s, "dk"), _heads(out_dq, d, b, s, "out_dq"),
        _heads(out_dk, d, b, s, "out_dk"),
        _flat(dgamma_q, d, torch.float32, "dgamma_q"),
        _flat(dgamma_k, d, torch.float32, "dgamma_k"), int(accumulate), _ptr(scratch),
        0 if scratch is None else scratch.numel(), _stream(stream)))
    return out_dq, out_dk, dgamma_q, dgamma_k


# ------------------------------------------------------------------- linear

def linear_scratch_bytes() -> int:
    n = ctypes.c_size_t()
    _check("pb_linear_scratch_bytes", lib().pb_linear_scratch_bytes(ctypes.byref(n)))
    return n.value


# pb_linear_args as bytes
_LINEAR_FORMAT = "@6iPqPqPPqiPqPqi0q"
_pack_linear = struct.Struct(_LINEAR_FORMAT).pack
assert struct.calcsize(_LINEAR_FORMAT) == ctypes.sizeof(pb_linear_args)


def linear(x, w, bias=None, residual=None, activation: str = "none",
           layout: int = PB_WEIGHT_IN_OUT, out=None, out_dtype=None, pre=None, scratch=None,
           status=None, stream=None):
    """``pb_linear``: ``activation(x @ w + bias) + residual`` for ``x`` [m, k] and ``w`` [k, n]
    (or [n, k], ``PB_WEIGHT_OUT_IN``), bf16 or fp16; ``out_dtype`` (or ``out``'s) is theirs or
    fp32, and a new one's rows start on 16-byte boundaries (a view where n is odd). ``pre`` (a
    [m, n] tensor of their type) receives ``x @ w + bias``. ``scratch`` (a
    uint8 CUDA tensor of ``linear_scratch_bytes()``) lets the product be split along k."""
    if stream is not None:
        return _run_on(stream, linear, x, w, bias, residual, activation, layout, out, out_dtype,
                       pre, scratch, status)
    m, k = x.shape
    in_out = layout == PB_WEIGHT_IN_OUT
    n = w.size(1 if in_out else 0)
    dt = x.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError("x must be torch.bfloat16 or torch.float16")
    if out is None:
        out = _new_rows(m, n, out_dtype or dt, x.device)
    od, rd = out.dtype, None if residual is None else residual.dtype
    if (od is not dt and od is not torch.float32) or (out_dtype is not None and od != out_dtype):
        raise ValueError(f"out must be {dt} or torch.float32, and out_dtype")
    if rd is not None and rd is not dt and rd is not torch.float32:
        raise ValueError(f"residual must be {dt} or torch.float32")
    _here(x, w, bias, residual, out, pre, scratch, status)
    args = _pack_linear(
        m, n, k, _DTYPES[dt], layout, ACTIVATIONS[activation], x.data_ptr(),
        _rows(x, m, k, dt, "x"), w.data_ptr(),
        _rows(w, k, n, dt, "w") if in_out else _rows(w, n, k, dt, "w"),
        _flat(bias, n, dt, "bias") or 0, 0 if residual is None else residual.data_ptr(),
        0 if residual is None else _rows(residual, m, n, rd, "residual"),
        0 if residual is None else _DTYPES[rd], 0 if pre is None else pre.data_ptr(),
        0 if pre is None else _rows(pre, m, n, dt, "pre"), out.data_ptr(),
        _rows(out, m, n, od, "out"), _DTYPES[od])
    _check("pb_linear", lib().pb_linear(args, _ptr(scratch),
                                        0 if scratch is None else scratch.numel(), _ptr(status),
                                        _stream(stream)))
    return out


def linear_backward(dy, x, w, pre=None, activation: str = "none", layout: int = PB_WEIGHT_IN_OUT,
                    need_dx: bool = True, need_dw: bool = True, bias: bool = False, dx=None,
                    dw=None, db=None, accumulate: bool = False, scratch=None, status=None,
                    stream=None):
    """``pb_linear_backward``: ``(dx, dw, db)`` of ``x @ w + bias`` for ``dy`` [m, n]; dx in the
    operands' type, dw (``w``'s layout) and db fp32, None where not wanted (``x`` is read for dw and
    ``w`` for dx: None without those). ``pre`` and ``activation``: ``x`` is ``activation(pre)``,
    and dx is the gradient of ``pre``. ``accumulate`` adds to the given ``dw`` and ``db``."""
    if stream is not None:
        return _run_on(stream, linear_backward, dy, x, w, pre, activation, layout, need_dx, need_dw,
                       bias, dx, dw, db, accumulate, scratch, status)
    m, n = dy.shape
    in_out = layout == PB_WEIGHT_IN_OUT
    if x is None and w is None:
        _is(not need_dx and dx is None, "dx needs w")
        _is(not need_dw and dw is None, "dw needs x")
        k = 1  # nothing of it is read
    else:
        k = (x if x is not None else w).shape[1 if x is not None or not in_out else 0]
    dt, dev = dy.dtype, dy.device
    _is(dt in (torch.bfloat16, torch.float16), "dy must be torch.bfloat16 or torch.float16")
    w_shape = (k, n) if in_out else (n, k)
    need_dx, need_dw = need_dx or dx is not None, need_dw or dw is not None
    if need_dx and dx is None:
        dx = _new_rows(m, k, dt, dev)
    if need_dw and dw is None:
        dw = _new_rows(*w_shape, torch.float32, dev, zero=accumulate)
    if bias and db is None:
        db = (torch.zeros if accumulate else torch.empty)(n, dtype=torch.float32, device=dev)
    _here(dy, x, w, pre, dx, dw, db, scratch, status)
    _is((pre is not None) == (ACTIVATIONS[activation] != 0), "pre goes with an activation")
    a = pb_linear_grads(m, n, k, _DTYPES[dt], layout, ACTIVATIONS[activation], int(accumulate),
                        dy.data_ptr(), _rows(dy, m, n, dt, "dy"))
    if need_dw:
        _is(x is not None, "dw needs x")
        a.x, a.ldx = x.data_ptr(), _rows(x, m, k, dt, "x")
        a.dw, a.lddw = dw.data_ptr(), _rows(dw, *w_shape, torch.float32, "dw")
    if need_dx:
        _is(w is not None, "dx needs w")
        a.w, a.ldw = w.data_ptr(), _rows(w, *w_shape, dt, "w")
        a.dx, a.lddx = dx.data_ptr(), _rows(dx, m, k, dt, "dx")
        if pre is not None:
            a.pre, a.ldp = pre.data_ptr(), _rows(pre, m, k, dt, "pre")
    a.db = _flat(db, n, torch.float32, "db")
    _check("pb_linear_backward", lib().pb_linear_backward(
        ctypes.byref(a), _ptr(scratch), 0 if scratch is None else scratch.numel(), _ptr(status),
        _stream(stream)))
    return dx if need_dx else None, dw if need_dw else None, db


def activation_backward(dy, pre, activation: str, out=None, stream=None):
    """``pb_activation_backward``: ``dy * activation'(pre)``, [rows, cols] bf16 or fp16."""
    if stream is not None:
        return _run_on(stream, activation_backward, dy, pre, activation, out)
    rows, cols = dy.shape
    _is(dy.dtype in (torch.bfloat16, torch.float16), "dy must be torch.bfloat16 or torch.float16")
    if out is None:
        out = _new_rows(rows, cols, dy.dtype, dy.device)
    _here(dy, pre, out)
    _check("pb_activation_backward", lib().pb_activation_backward(
        rows, cols, _DTYPES[dy.dtype], ACTIVATIONS[activation], _ptr(dy),
        _rows(dy, rows, cols, dy.dtype, "dy"), _ptr(pre),
        _rows(pre, rows, cols, dy.dtype, "pre"), _ptr(out),
        _rows(out, rows, cols, dy.dtype, "out"), _stream(stream)))
    return out


# ------------------------------------------------------------------- AdamW

class AdamW:
    """The tensors of an AdamW step (``pb_adamw``). Each is a dict: ``param`` (fp32 or bf16,
    updated in place), ``copy`` (a bf16 copy of fp32 parameters, or None), ``grad`` (fp32 or
    bf16), the states ``m`` and ``v`` (fp32, or ``torch.float8_e4m3fn`` with fp32 ``m_scale``
    and ``v_scale``, one per 256 values), ``weight_decay`` (default 0). States start at zero:
    ``adamw_states`` makes them. Types are the same for all tensors of a step."""

    def __init__(self, tensors, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8):
        self.tensors = [dict(t) for t in tensors]
        self.beta1, self.beta2, self.eps = float(beta1), float(beta2), float(eps)
        n = len(self.tensors)
        _is(n > 0, "no tensors")
        t0 = self.tensors[0]
        self.device = t0["param"].device
        ptype, gtype, eight = t0["param"].dtype, t0["grad"].dtype, t0.get("m_scale") is not None
        _is(ptype in (torch.float32, torch.bfloat16), "param must be fp32 or bf16")
        _is(gtype in (torch.float32, torch.bfloat16), "grad must be fp32 or bf16")
        self.param_dtype, self.grad_dtype = _DTYPES[ptype], _DTYPES[gtype]
        self.state_bits = 8 if eight else 32
        stype = torch.float8_e4m3fn if eight else torch.float32
        self.array = (pb_adamw_tensor * n)()
        for i, t in enumerate(self.tensors):
            size = t["param"].numel()
            blocks = -(-size // PB_ADAMW_BLOCK)
            for name in ("param", "copy", "grad", "m", "v", "m_scale", "v_scale"):
                x = t.get(name)
                _is(x is None or x.device == self.device, f"tensor {i}: {name} is elsewhere")
            _is((t.get("m_scale") is not None) == eight == (t.get("v_scale") is not None),
                f"tensor {i}: m_scale and v_scale go with 8-bit states, for all tensors")
            a = self.array[i]
            a.n = size
            a.param = _flat(t["param"], size, ptype, f"tensor {i}: param")
            a.param_copy = _flat(t.get("copy"), size, torch.bfloat16, f"tensor {i}: copy")
            a.grad = _flat(t["grad"], size, gtype, f"tensor {i}: grad")
            a.m = _flat(t["m"], size, stype, f"tensor {i}: m")
            a.v = _flat(t["v"], size, stype, f"tensor {i}: v")
            a.m_scale = _flat(t.get("m_scale"), blocks, torch.float32, f"tensor {i}: m_scale")
            a.v_scale = _flat(t.get("v_scale"), blocks, torch.float32, f"tensor {i}: v_scale")
            a.weight_decay = float(t.get("weight_decay", 0.0))
        b = ctypes.c_size_t()
        _check("pb_grad_norm_scratch_bytes", lib().pb_grad_norm_scratch_bytes(n, ctypes.byref(b)))
        self.scratch_bytes = b.value

    def grad_norm(self, max_norm: float, out=None, scratch=None, stream=None) -> torch.Tensor:
        """``pb_grad_norm``: fp32 [2], the norm of all gradients and the factor that clips them
        to ``max_norm`` (``step(grad_scale=out[1:])``)."""
        if stream is not None:
            return _run_on(stream, self.grad_norm, max_norm, out, scratch)
        if out is None:
            out = torch.empty(2, dtype=torch.float32, device=self.device)
        if scratch is None:
            scratch = torch.empty(self.scratch_bytes, dtype=torch.uint8, device=self.device)
        _here(out, scratch, self.tensors[0]["param"])
        _check("pb_grad_norm", lib().pb_grad_norm(
            len(self.tensors), self.array, self.grad_dtype, max_norm,
            _flat(out, 2, torch.float32, "out"), _ptr(scratch), scratch.numel(),
            _stream(stream)))
        return out

    def step(self, lr: float, step: int = 0, grad_scale=None, d_lr=None, d_step=None,
             stream=None):
        """``pb_adamw``, in place: step number ``step`` (from 1 on). ``d_lr`` (fp32), ``d_step``
        (int32) and ``grad_scale`` (fp32): one-element CUDA tensors read when the step runs."""
        _here(grad_scale, d_lr, d_step, self.tensors[0]["param"])
        a = pb_adamw_args(lr, self.beta1, self.beta2, self.eps, step, self.param_dtype,
                          self.grad_dtype, self.state_bits,
                          _flat(d_lr, 1, torch.float32, "d_lr"),
                          _flat(d_step, 1, torch.int32, "d_step"),
                          _flat(grad_scale, 1, torch.float32, "grad_scale"))
        _check("pb_adamw", lib().pb_adamw(ctypes.byref(a), len(self.tensors), self.array,
                                          _stream(stream)))


def adamw_states(param: torch.Tensor, bits: int = 32) -> dict:
    """The states of one tensor before its first step: ``m`` and ``v``, with ``bits=8`` their
    scales too."""
    _is(bits in (8, 32), "bits must be 8 or 32")
    n = param.numel()
    if bits == 32:
        return {k: torch.zeros(n, dtype=torch.float32, device=param.device) for k in ("m", "v")}
    st = {k: torch.zeros(n, dtype=torch.uint8, device=param.device).view(torch.float8_e4m3fn)
          for k in ("m", "v")}
    for k in ("m_scale", "v_scale"):
        st[k] = torch.zeros(-(-n // PB_ADAMW_BLOCK), dtype=torch.float32, device=param.device)
    return st
