"""More arguments of the operators around the block that are refused on the host, before anything
is enqueued (CPU only; the pointers are made up and never read)."""

import ctypes

import pytest

from transformer_block_gb300 import build, pb

P = 0x10000000
W = P + (8 << 24)  # scratch


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pb.lib()


def message(lib):
    return lib.pb_last_error_message().decode()


def linear(lib, **kw):
    a = pb.pb_linear_args(40, 64, 128, 0, 0, 0, P, 128, P + (1 << 24), 64, None, None, 0, 0, None,
                          0, P + (2 << 24), 64, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.pb_linear(ctypes.byref(a), W, pb.linear_scratch_bytes(), None, None)


def linear_back(lib, **kw):
    a = pb.pb_linear_grads(40, 64, 128, 0, 0, 0, 0, P, 64, P + (1 << 24), 128, P + (2 << 24), 64,
                           None, 0, P + (3 << 24), 128, P + (4 << 24), 64, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.pb_linear_backward(ctypes.byref(a), W, pb.linear_scratch_bytes(), None, None)


def test_linear_operands_in_scratch(lib):
    # split products write their partial sums there while the operands are read
    end = W + pb.linear_scratch_bytes()
    for at in (W, W + 4096, end - 16):
        for kw in (dict(x=at), dict(w=at), dict(bias=at), dict(residual=at, ldr=64),
                   dict(pre=at, ldp=64), dict(y=at)):
            assert linear(lib, **kw) == 1, kw
            assert "overlap" in message(lib) and "scratch" in message(lib), kw
        for kw in (dict(dy=at), dict(x=at), dict(w=at), dict(activation=1, pre=at, ldp=128),
                   dict(dx=at), dict(dw=at), dict(db=at)):
            assert linear_back(lib, **kw) == 1, kw
            assert "overlap" in message(lib) and "scratch" in message(lib), kw
    # what a call does not read may be anywhere: x without dw, w without dx, no tokens
    assert linear_back(lib, x=W, dw=None) != 1
    assert linear_back(lib, w=W, dx=None) != 1
    assert linear(lib, m=0, x=W) == 0


# --------------------------------------------------------------------------- rotation

def plan(lib, dh=128):
    p = pb.pb_rope()
    assert lib.pb_rope_init(dh, dh, 0, 1, None, 0, 1e4, None, ctypes.byref(p)) == 0
    return p


def heads(ptr=P, n=4, b=8 * 512, s=512, h=128):
    return ctypes.byref(pb.pb_heads(ptr, n, b, s, h))


def rope_back(lib, eps, gamma=P + (4 << 24)):
    return lib.pb_qk_norm_rope_backward(
        ctypes.byref(plan(lib)), 2, 8, heads(P), None, gamma, None, eps, None,
        heads(P + (1 << 24)), None, heads(P + (2 << 24)), None, P + (5 << 24), None, 0, W,
        pb.qk_norm_rope_scratch_bytes(), None)


def test_backward_of_a_norm_with_a_vanishing_eps(lib):
    # The norm's backward takes rstd^3: for a head of zeros eps^(-3/2), which passes fp32's range
    # from eps = 2e-26 down, and infinity times the head's zero sum is NaN.
    for eps in (1e-30, 1e-40, 2.0 ** -81):
        assert rope_back(lib, eps) == 1, eps
        assert "2^-80" in message(lib)
    assert rope_back(lib, 2.0 ** -80) != 1


def test_views_beyond_all_memory(lib):
    # strides are below 2^40 and tokens below 2^31, but their products pass 64 bits, and the checks
    # for overlaps with them
    far, big = P + (1 << 40), 1 << 40
    p = plan(lib)
    for b, s, kw in ((1 << 15, 1 << 15, dict(b=big)), (1, 1 << 30, dict(s=big)),
                     (1, 4, dict(n=(1 << 31) - 1, h=big))):
        for q, o in ((kw, {}), ({}, kw), (kw, kw)):
            got = lib.pb_qk_norm_rope(ctypes.byref(p), b, s, heads(P, **q), None, None, None, 1e-6,
                                      None, heads(far, **({"s": 4096 * 512, "b": 0} | o)), None,
                                      None)
            assert got == 2 and "2^48" in message(lib), (b, s, q, o, message(lib))


def test_no_tokens_read_no_weights(lib):
    # accumulating over no tokens leaves everything as it is, wherever the weights lie
    dw = P + (4 << 24)
    assert linear_back(lib, m=0, accumulate=1, w=dw) == 0
    assert linear_back(lib, m=0, accumulate=1, w=W) == 0
    assert linear_back(lib, m=0, accumulate=1, dw=W) == 1  # a result in scratch
