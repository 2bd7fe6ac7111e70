"""The rotation, linear and AdamW entry points refuse bad arguments on the host, before anything
is enqueued (CPU only; the pointers are made up and never read)."""

import ctypes
import math

import pytest

from transformer_block_gb300 import build, pb

P = 0x10000000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pb.lib()


def message(lib):
    return lib.pb_last_error_message().decode()


# --------------------------------------------------------------------------- rotation

def init(lib, dh=128, rot=128, pairing=0, axes=1, sections=None, ladder=0, theta=1e4, freq=None):
    plan = pb.pb_rope()
    sec = None if sections is None else (ctypes.c_int32 * len(sections))(*sections)
    frq = None if freq is None else (ctypes.c_double * len(freq))(*freq)
    return lib.pb_rope_init(dh, rot, pairing, axes, sec, ladder, theta, frq,
                            ctypes.byref(plan)), plan


@pytest.mark.parametrize("kw,code", [
    (dict(dh=0), 2), (dict(dh=24, rot=16), 2), (dict(dh=272), 2), (dict(rot=144), 1),
    (dict(rot=-16), 1), (dict(rot=24), 2), (dict(pairing=2), 1), (dict(ladder=-1), 1),
    (dict(axes=0), 1), (dict(axes=5, sections=[16] * 5), 1), (dict(axes=2), 1),
    (dict(axes=2, sections=[32, 31]), 1), (dict(axes=2, sections=[32, 33]), 1),
    (dict(axes=2, sections=[-1, 65]), 1), (dict(theta=0.0), 1), (dict(theta=math.inf), 1),
    (dict(freq=[0.1] * 63 + [math.nan]), 1),
])
def test_rope_plans_refused(lib, kw, code):
    got, plan = init(lib, **kw)
    assert got == code and message(lib)
    assert plan.magic == 0  # such a plan is refused by the calls


def test_rope_plan_turns(lib):
    # frequencies as fractions of a turn, modulo one: position x turns wraps as the angle does
    ok, plan = init(lib)
    assert ok == 0 and list(plan.section_end) == [64] * 4
    for i in (0, 1, 17, 63):
        want = 1e4 ** (-i / 64) / (2 * math.pi)
        assert abs(plan.turns[i] / 2 ** 64 - want) <= 2.0 ** -52 * want + 2.0 ** -64
    ok, plan = init(lib, axes=3, sections=[16, 24, 24], ladder=1)
    assert ok == 0 and list(plan.section_end) == [16, 40, 64, 64]
    assert plan.turns[0] == plan.turns[16] == plan.turns[40]
    ok, plan = init(lib, freq=[-0.5] * 64)
    assert ok == 0 and abs(plan.turns[0] / 2 ** 64 - (1 - 0.5 / (2 * math.pi))) <= 2.0 ** -52
    ok, plan = init(lib, axes=2, sections=[0, 64])  # an axis without pairs
    assert ok == 0 and list(plan.section_end) == [0, 64, 64, 64]
    assert init(lib, rot=0)[0] == 0
    assert lib.pb_rope_init(128, 128, 0, 1, None, 0, 1e4, None, None) == 1


def heads(ptr=P, n=4, b=8 * 512, s=512, h=128):
    return ctypes.byref(pb.pb_heads(ptr, n, b, s, h))


def rope_call(lib, plan, b=2, s=8, q=None, k=None, gq=None, gk=None, eps=1e-6, pos=None, qo=None,
              ko=None):
    return lib.pb_qk_norm_rope(ctypes.byref(plan) if plan is not None else None, b, s, q, k, gq,
                               gk, eps, pos, qo, ko, None)


def test_rotation_refused(lib):
    plan = init(lib)[1]
    far = P + 0x1000000
    assert rope_call(lib, None, q=heads(), qo=heads(far)) == 1
    assert rope_call(lib, pb.pb_rope(), q=heads(), qo=heads(far)) == 1
    assert rope_call(lib, plan) == 1                                       # neither q nor k
    assert rope_call(lib, plan, q=heads()) == 1                            # no result
    assert rope_call(lib, plan, b=-1, q=heads(), qo=heads(far)) == 1
    assert rope_call(lib, plan, b=65536, s=65536, q=heads(), qo=heads(far)) == 2
    assert rope_call(lib, plan, q=heads(None), qo=heads(far)) == 1
    assert rope_call(lib, plan, q=heads(P + 8), qo=heads(far)) == 1        # alignment
    assert rope_call(lib, plan, q=heads(s=516), qo=heads(far)) == 1        # stride % 8
    assert rope_call(lib, plan, q=heads(s=-512), qo=heads(far)) == 1
    assert rope_call(lib, plan, q=heads(n=0), qo=heads(far)) == 1
    assert rope_call(lib, plan, q=heads(), qo=heads(far, n=3)) == 1
    assert rope_call(lib, plan, q=heads(), qo=heads(far), gq=P + 4) == 1   # gamma alignment
    assert rope_call(lib, plan, q=heads(), qo=heads(far), gq=P, eps=0.0) == 1
    assert rope_call(lib, plan, q=heads(), qo=heads(far), gq=P, eps=math.nan) == 1
    assert rope_call(lib, plan, q=heads(), qo=heads(far), pos=P + 2) == 1
    assert rope_call(lib, plan, q=heads(), qo=heads(far, h=64)) == 1       # heads of it overlap
    assert rope_call(lib, plan, q=heads(), qo=heads(far, s=0)) == 1
    assert rope_call(lib, plan, q=heads(), qo=heads(P + 256)) == 1         # shifted by a head
    assert "overlap" in message(lib)
    assert rope_call(lib, plan, q=heads(), k=heads(far), qo=heads(far), ko=heads(far)) == 1
    two = init(lib, axes=2, sections=[32, 32])[1]
    assert rope_call(lib, two, q=heads(), qo=heads(far)) == 1              # positions needed
    # nothing to do: no tokens
    assert rope_call(lib, plan, b=0, q=heads(), qo=heads(far)) == 0
    assert rope_call(lib, plan, s=0, q=heads(None), qo=heads(None)) == 0


def rope_back(lib, plan, x=None, g=None, dy=None, out=None, dg=None, scratch=None, n=0, b=2, s=8):
    return lib.pb_qk_norm_rope_backward(ctypes.byref(plan), b, s, x, None, g, None, 1e-6, None, dy,
                                        None, out, None, dg, None, 0, scratch, n, None)


def test_rotation_backward_refused(lib):
    plan = init(lib)[1]
    n = pb.qk_norm_rope_scratch_bytes()
    a, b, c, w = P, P + 0x1000000, P + 0x2000000, P + 0x3000000
    assert rope_back(lib, plan) == 1
    assert rope_back(lib, plan, dy=heads(a)) == 1
    assert rope_back(lib, plan, dy=heads(a), out=heads(b), dg=c) == 1          # no gamma
    assert rope_back(lib, plan, dy=heads(a), out=heads(b), g=w, dg=c, scratch=w, n=n) == 1  # no x
    assert rope_back(lib, plan, x=heads(c), g=a, dy=heads(a), out=heads(b)) == 1            # no scratch
    assert rope_back(lib, plan, x=heads(c), g=a, dy=heads(a), out=heads(b), scratch=w + 16,
                     n=n) == 1
    assert rope_back(lib, plan, x=heads(c), g=a, dy=heads(a), out=heads(b), scratch=w,
                     n=n - 1) == 3
    assert rope_back(lib, plan, x=heads(c, n=3), g=a, dy=heads(a), out=heads(b), scratch=w,
                     n=n) == 1
    assert rope_back(lib, plan, x=heads(c), g=a, dy=heads(a), out=heads(c + 256), scratch=w,
                     n=n) == 1
    assert rope_back(lib, plan, x=heads(c), g=a, dy=heads(a), out=heads(b), dg=w + 2, scratch=w,
                     n=n) == 1
    assert rope_back(lib, plan, dy=heads(a), out=heads(b), b=0) == 0


# --------------------------------------------------------------------------- linear

def linear(lib, scratch=None, nbytes=0, **kw):
    a = pb.pb_linear_args(40, 64, 128, 0, 0, 0, P, 128, P + (1 << 24), 64, None, None, 0, 0, None,
                          0, P + (2 << 24), 64, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.pb_linear(ctypes.byref(a), scratch, nbytes, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(dtype=2), 2), (dict(dtype=9), 2),
    (dict(w_layout=2), 1), (dict(activation=5), 1), (dict(activation=-1), 1),
    (dict(y_dtype=1), 2), (dict(x=None), 1), (dict(x=P + 8), 1), (dict(ldx=120), 1),
    (dict(ldx=132), 1), (dict(ldw=56), 1), (dict(w_layout=1, ldw=64), 1), (dict(ldy=60), 1),
    (dict(y=None), 1), (dict(y_dtype=2, ldy=66), 1), (dict(ldx=1 << 36), 2),
    (dict(bias=P + 4), 1), (dict(residual=P + (3 << 24), ldr=60), 1),
    (dict(residual=P + (3 << 24), ldr=64, residual_dtype=1), 2),
    (dict(pre=P + (3 << 24), ldp=0), 1),
    (dict(y=P), 1), (dict(y=P + (1 << 24) + 1024), 1),                     # overlaps x, w
    (dict(pre=P + (2 << 24), ldp=64), 1),                                  # pre is y
    (dict(residual=P + (2 << 24) + 16, ldr=64), 1),                        # part of y
    (dict(residual=P + (2 << 24), ldr=72), 1),
    (dict(residual=P + (2 << 24), ldr=64, residual_dtype=2), 1),           # y's place, other type
    (dict(m=1 << 30, n=1 << 20), 2),
])
def test_linear_refused(lib, kw, code):
    assert linear(lib, **kw) == code and message(lib)


def test_linear_scratch_and_no_tokens(lib):
    n = pb.linear_scratch_bytes()
    assert linear(lib, scratch=P + (4 << 24), nbytes=n - 1) == 3
    assert linear(lib, scratch=P + (4 << 24) + 16, nbytes=n) == 3
    assert linear(lib, scratch=P + (2 << 24), nbytes=n) == 1               # overlaps y
    assert lib.pb_linear(None, None, 0, None, None) == 1
    assert linear(lib, m=0, x=None, y=None) == 0
    assert lib.pb_linear_scratch_bytes(None) == 1


def linear_back(lib, scratch=None, nbytes=0, **kw):
    a = pb.pb_linear_grads(40, 64, 128, 0, 0, 0, 0, P, 64, P + (1 << 24), 128, P + (2 << 24), 64,
                           None, 0, P + (3 << 24), 128, P + (4 << 24), 64, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.pb_linear_backward(ctypes.byref(a), scratch, nbytes, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), 1), (dict(dtype=2), 2), (dict(activation=7), 1), (dict(dy=None), 1),
    (dict(lddy=62), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(activation=1), 1),  # no pre
    (dict(dx=P), 1), (dict(dw=P + (2 << 24)), 1), (dict(db=P + (4 << 24)), 1),
    (dict(db=P + 2), 1), (dict(lddw=60), 1), (dict(lddx=124), 1),
    (dict(dx=P + (4 << 24)), 1),
])
def test_linear_backward_refused(lib, kw, code):
    assert linear_back(lib, **kw) == code and message(lib)


def test_activation_backward_refused(lib):
    def call(rows=4, cols=64, dtype=0, act=1, dy=P, ld=64, pre=P + 4096, out=P + 8192):
        return lib.pb_activation_backward(rows, cols, dtype, act, dy, ld, pre, 64, out, 64, None)

    assert call(rows=-1) == 1 and call(cols=0) == 1 and call(dtype=2) == 2 and call(act=9) == 1
    assert call(dy=None) == 1 and call(ld=60) == 1 and call(out=P + 64) == 1
    assert call(ld=72, out=P) == 1  # in place with another stride
    assert call(rows=0, dy=None) == 0


# --------------------------------------------------------------------------- AdamW

def adamw(lib, tensors=None, **kw):
    a = pb.pb_adamw_args(1e-3, 0.9, 0.95, 1e-8, 1, 2, 2, 32, None, None, None)
    for k, v in kw.items():
        setattr(a, k, v)
    ts = [tensor()] if tensors is None else tensors
    arr = (pb.pb_adamw_tensor * max(1, len(ts)))(*ts)
    return lib.pb_adamw(ctypes.byref(a), len(ts), arr, None)


def tensor(at=P, n=1000, **kw):
    t = pb.pb_adamw_tensor(n, at, None, at + 0x10000, at + 0x20000, at + 0x30000, None, None, 0.0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def test_adamw_refused(lib):
    assert lib.pb_adamw(None, 0, None, None) == 1
    assert adamw(lib, []) == 0                                  # nothing to do
    assert adamw(lib, [tensor(n=0, param=None)]) == 0
    for kw, code in ((dict(param_dtype=1), 2), (dict(grad_dtype=1), 2), (dict(state_bits=16), 2),
                     (dict(beta1=1.0), 1), (dict(beta2=-0.1), 1), (dict(eps=0.0), 1),
                     (dict(eps=1e-42), 1), (dict(eps=math.nan), 1), (dict(lr=math.inf), 1),
                     (dict(step=0), 1), (dict(d_lr=P + 2), 1), (dict(state_bits=8), 1),
                     (dict(beta1=math.nan), 1)):
        assert adamw(lib, **kw) == code, kw
        assert message(lib)
    for kw in (dict(n=-1), dict(n=1 << 41), dict(param=None), dict(param=P + 4), dict(grad=None),
               dict(m=None), dict(v=P + 0x30004), dict(m_scale=P), dict(param_copy=P + 0x40008),
               dict(weight_decay=math.nan), dict(v=P + 0x20000), dict(grad=P),
               dict(param_copy=P + 0x10000)):
        assert adamw(lib, [tensor(**kw)]) == 1, kw
    assert adamw(lib, [tensor(), tensor(P + 0x100000), tensor()]) == 1     # listed twice
    assert "overlap" in message(lib)
    assert adamw(lib, [tensor(param_copy=P + 0x40000)], param_dtype=0) == 1
    # gradients may be shared: they are only read (refused here for another reason)
    two = [tensor(), tensor(P + 0x100000, grad=P + 0x10000, m=None)]
    assert adamw(lib, two) == 1 and "16-byte" in message(lib)


def test_grad_norm_refused(lib):
    n = ctypes.c_size_t()
    assert lib.pb_grad_norm_scratch_bytes(1, ctypes.byref(n)) == 0 and n.value > 0
    arr = (pb.pb_adamw_tensor * 1)(tensor())

    def call(count=1, dtype=2, max_norm=1.0, out=P, scratch=P + 0x1000000, nbytes=n.value):
        return lib.pb_grad_norm(count, arr, dtype, max_norm, out, scratch, nbytes, None)

    assert call(count=-1) == 1 and call(dtype=1) == 2 and call(max_norm=0.0) == 1
    assert call(max_norm=math.inf) == 1 and call(out=None) == 1 and call(out=P + 2) == 1
    assert call(scratch=None) == 1 and call(scratch=P + 16) == 1 and call(nbytes=8) == 3
    assert lib.pb_grad_norm_scratch_bytes(-1, ctypes.byref(n)) == 1
    assert lib.pb_grad_norm_scratch_bytes(1, None) == 1


def test_block_rotation_needs_a_handle(lib):
    assert lib.pb_set_qk_norm_rope(None, None) == 6


# --------------------------------------------------------------------------- overlaps, extremes

def rope_back2(lib, plan, gq, gk, dgq, dgk, scratch, pos=None, out=P + 0x2000000, accumulate=1):
    """The backward pass of q and k (its views lie between P and P + 0x4000000)."""
    return lib.pb_qk_norm_rope_backward(
        ctypes.byref(plan), 2, 8, heads(P), heads(P + 0x800000), gq, gk, 1e-6, pos,
        heads(P + 0x1000000), heads(P + 0x1800000), heads(out), heads(out + 0x800000), dgq, dgk,
        accumulate, scratch, pb.qk_norm_rope_scratch_bytes(), None)


def test_rotation_gradients_of_gammas_apart(lib):
    plan = init(lib)[1]
    g, d, w = P + 0x4000000, P + 0x5000000, P + 0x6000000
    for kw in (dict(dgk=d),                                 # one buffer for both sums
               dict(dgk=d + 508), dict(dgk=w + 4096),       # part of it, in scratch
               dict(dgk=g), dict(dgk=P), dict(dgk=P + 0x1000000), dict(dgk=P + 0x2800000),
               dict(scratch=P), dict(scratch=P + 0x1800000), dict(scratch=P + 0x2000000),
               dict(scratch=g), dict(pos=d + 64), dict(pos=w), dict(pos=P + 0x2000000),
               dict(gq=P + 0x2000000), dict(gk=P + 0x2800000 + 256)):
        args = dict(gq=g, gk=g, dgq=d, dgk=d + 512, scratch=w) | kw
        assert rope_back2(lib, plan, **args) == 1, kw
        assert "overlaps" in message(lib), kw
    # the forward call
    for kw in (dict(gq=P + 0x1000000), dict(gk=P + 0x1000000 + 64, k=heads(P + 0x100000),
                                            ko=heads(P + 0x2000000)), dict(pos=P + 0x1000040)):
        assert rope_call(lib, plan, q=heads(), qo=heads(P + 0x1000000), **kw) == 1, kw
        assert "overlaps" in message(lib), kw


def test_linear_extremes_refused(lib):
    top = 2 ** 31 - 1
    for kw in (dict(n=top, ldw=2 ** 31, ldy=2 ** 31), dict(m=top), dict(k=top, ldx=2 ** 31),
               dict(k=2 ** 31 - 1024, ldx=2 ** 31)):
        assert linear(lib, **kw) == 2, kw
        assert "2^31" in message(lib)
    assert linear_back(lib, n=top, lddy=2 ** 31, ldw=2 ** 31, lddw=2 ** 31) == 2
    # a stride and a number of rows whose product passes 64 bits in bytes
    assert linear(lib, m=1 << 30, ldx=1 << 33) == 2 and "2^48" in message(lib)
    assert lib.pb_activation_backward((1 << 40) - 1, 64, 0, 1, P, 1 << 34, P, 1 << 34, P,
                                      1 << 34, None) == 2


def test_adamw_scalars_and_norm_apart(lib):
    for name in ("d_lr", "d_step", "d_grad_scale"):
        for at in (P, P + 0x20000 + 396, P + 0x30000):       # param, m, v
            assert adamw(lib, **{name: at}) == 1 and "overlaps" in message(lib)
    arr = (pb.pb_adamw_tensor * 2)(tensor(n=0), tensor())
    n = ctypes.c_size_t()
    lib.pb_grad_norm_scratch_bytes(2, ctypes.byref(n))
    far = P + 0x1000000
    for out, scratch in ((P + 0x10000 + 3996, far), (P, P + 0x10000), (far, far),
                         (far + n.value - 4, far), (P, P + 0x10000 - 256)):
        assert lib.pb_grad_norm(2, arr, 2, 1.0, out, scratch, n.value, None) == 1
        assert "overlaps" in message(lib)


def test_positions_in_another_order_refused():
    import torch
    three = pb.Rope(64, sections=[16, 8, 8])
    one = pb.Rope(64)

    def pos(*shape):
        return torch.zeros(*shape, dtype=torch.int32)

    for rope, good, bad in ((three, [(3, 2, 5), (30,)], [(2, 3, 5), (2, 5, 3), (3, 5, 2), (3, 10)]),
                            (one, [(1, 2, 5), (2, 5), (10,), (2, 5, 1)], [(5, 2), (1, 5, 2)])):
        for shape in good:
            assert pb._positions(rope, pos(*shape), 2, 5) is not None
        for shape in bad:
            with pytest.raises(ValueError, match="positions"):
                pb._positions(rope, pos(*shape), 2, 5)
    assert pb._positions(three, pos(3, 5), 1, 5) is not None      # one sequence
    assert pb._positions(three, pos(3, 2), 2, 1) is not None      # one token each
    for p in (pos(3, 2, 4), pos(31), pos(3, 2, 5).long()):
        with pytest.raises(ValueError):
            pb._positions(three, p, 2, 5)
