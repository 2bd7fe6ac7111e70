"""The serving entry points (attention of packed prompts, paged cache, attention over it) refuse bad
arguments on the host, before anything is enqueued (CPU only; the pointers are made up and never
read)."""

import ctypes
import os

import pytest
import torch

from transformer_block_gb300 import build, pb

P = 0x10000000
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pb.lib()


def message(lib):
    return lib.pb_last_error_message().decode()


# --------------------------------------------------------------------------- packed prompts

def heads(at, n, stride=None, dh=128, head=None):
    return pb.pb_heads(at, n, 0, n * dh if stride is None else stride, dh if head is None else head)


def prompt(lib, scratch=P + 64 * MB, nbytes=None, status=None, **kw):
    a = pb.pb_prompt_args(100, 2, 128, 0, 0.0, heads(P, 8), heads(P + MB, 2), heads(P + 2 * MB, 2),
                          heads(P + 3 * MB, 8), P + 4 * MB)
    for k, v in kw.items():
        setattr(a, k, v)
    if nbytes is None:
        nbytes = pb.prompt_attention_scratch_bytes(max(0, a.tokens), max(0, a.sequences))
    return lib.pb_prompt_attention(ctypes.byref(a), scratch, nbytes, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 1), (dict(sequences=-1), 1), (dict(head_dim=96), 2), (dict(head_dim=256), 2),
    (dict(window=-1), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=3e38), 1), (dict(tokens=2 ** 31 - 1000, nbytes=2 ** 60), 2),
    (dict(sequences=2 ** 24 + 1, nbytes=2 ** 60), 2), (dict(starts=None), 1),
    (dict(starts=P + 4 * MB + 2), 1), (dict(q=heads(None, 8)), 1), (dict(k=heads(P + MB + 8, 2)), 1),
    (dict(v=heads(P + 2 * MB, 2, stride=260)), 1), (dict(v=heads(P + 2 * MB, 2, stride=-256)), 1),
    (dict(q=heads(P, 0)), 1), (dict(v=heads(P + 2 * MB, 4)), 1), (dict(out=heads(P + 3 * MB, 4)), 1),
    (dict(q=heads(P, 7), out=heads(P + 3 * MB, 7)), 1),
    (dict(k=heads(P + MB, 2, stride=0)), 2), (dict(q=heads(P, 8, head=0)), 2),
    (dict(k=heads(P + MB, 2, stride=64)), 2), (dict(k=heads(P + MB, 2, stride=2 ** 39)), 2),
    (dict(out=heads(P + 3 * MB, 8, head=64)), 1), (dict(out=heads(P + 3 * MB, 8, stride=512)), 1),
    (dict(out=heads(P, 8)), 1), (dict(out=heads(P + MB, 8)), 1), (dict(out=heads(P + 2 * MB, 8)), 1),
    (dict(out=heads(P + 4 * MB - 4096, 8)), 1), (dict(scratch=None), 1), (dict(scratch=P + 64 * MB + 8), 1),
    (dict(nbytes=100), 3), (dict(scratch=P), 1), (dict(scratch=P + 3 * MB), 1),
    (dict(scratch=P + 4 * MB), 1),
])
def test_prompts_refused(lib, kw, code):
    assert prompt(lib, **kw) == code and message(lib)


def test_prompt_groups_and_nothing(lib):
    wide = dict(q=heads(P, 129), k=heads(P + 8 * MB, 1), v=heads(P + 9 * MB, 1),
                out=heads(P + 10 * MB, 129), starts=P + 20 * MB)
    assert prompt(lib, **wide) == 2 and "128" in message(lib)
    # no tokens or no sequences do nothing, whatever else is given
    assert prompt(lib, tokens=0, starts=None, scratch=None) == 0
    assert prompt(lib, sequences=0, starts=None, scratch=None) == 0
    assert lib.pb_prompt_attention(None, None, 0, None, None) == 1
    n = ctypes.c_size_t()
    assert lib.pb_prompt_attention_scratch_bytes(-1, 1, ctypes.byref(n)) == 1
    assert lib.pb_prompt_attention_scratch_bytes(1, -1, ctypes.byref(n)) == 1
    assert lib.pb_prompt_attention_scratch_bytes(1, 1, None) == 1
    assert lib.pb_prompt_attention_scratch_bytes(0, 0, ctypes.byref(n)) == 0


def test_prompt_columns_of_one_buffer(lib):
    # q, k, v side by side are inputs and may touch; out as other columns of it is apart by its strides
    row = 8 * 128 + 2 * 256 + 8 * 128
    q = pb.pb_heads(P, 8, 0, row, 128)
    k, v = (pb.pb_heads(P + 2 * (1024 + i * 256), 2, 0, row, 128) for i in range(2))
    out = pb.pb_heads(P + 2 * 1536, 8, 0, row, 128)
    assert prompt(lib, q=q, k=k, v=v, out=out) == 4  # past the checks, no driver
    assert prompt(lib, q=q, k=k, v=v, out=pb.pb_heads(P + 2 * 1528, 8, 0, row, 128)) == 1


# --------------------------------------------------------------------------- cache

FAR = P + (1 << 32)


def cache(**kw):
    c = pb.pb_cache(2, 50, 16, 4, 64, 8, 12, P, P + 16 * MB, P + 32 * MB, P + 33 * MB, P + 34 * MB,
                    P + 35 * MB)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def need(lib, c):
    n = ctypes.c_size_t()
    assert lib.pb_cache_scratch_bytes(ctypes.byref(c), ctypes.byref(n)) == 0
    return n.value


def calls(lib, c, n=2, slots=FAR, starts=FAR + MB, path=FAR + 2 * MB, kept=FAR + 3 * MB,
          scratch=FAR + 4 * MB, nbytes=None, tokens=5):
    b = 1 << 40 if nbytes is None else nbytes
    r = ctypes.byref(c)
    return {lib.pb_cache_extend(r, n, slots, starts, scratch, b, None),
            lib.pb_cache_fork(r, n, slots, starts, scratch, b, None),
            lib.pb_cache_truncate(r, n, slots, starts, scratch, b, None),
            keep(lib, c, n, slots, starts, path, kept, scratch, b, tokens)}


def keep(lib, c, n=2, slots=FAR, starts=FAR + MB, path=FAR + 2 * MB, kept=FAR + 3 * MB,
         scratch=FAR + 4 * MB, nbytes=1 << 40, tokens=5):
    return lib.pb_cache_keep(ctypes.byref(c), n, slots, starts, tokens, path, kept, scratch, nbytes,
                             None)


@pytest.mark.parametrize("kw,code", [
    (dict(layers=0), 1), (dict(pages=0), 1), (dict(page_size=0), 1), (dict(kv_heads=0), 1),
    (dict(slots=0), 1), (dict(slot_pages=0), 1), (dict(head_dim=96), 2), (dict(head_dim=256), 2),
    (dict(slots=2 ** 16 + 1), 2), (dict(pages=2 ** 20 + 1), 2), (dict(page_size=2 ** 27), 2),
    (dict(kv_heads=65536), 2), (dict(layers=65536), 2),
    (dict(pages=2 ** 20, page_size=2 ** 14, kv_heads=2 ** 8), 2), (dict(k=None), 1), (dict(v=P + 8), 1),
    (dict(table=None), 1), (dict(lengths=P + 33 * MB + 2), 1), (dict(refs=None), 1),
    (dict(status=None), 1), (dict(v=P + MB // 4), 1), (dict(table=P + 4096), 1),
    (dict(lengths=P + 32 * MB), 1), (dict(status=P + 33 * MB + 28), 1),
])
def test_caches_refused(lib, kw, code):
    c = cache(**kw)
    assert calls(lib, c) == {code} and message(lib)
    k = pb.pb_heads(FAR + 8 * MB, c.kv_heads, 4096, 256, 64)
    assert lib.pb_cache_write(ctypes.byref(c), 0, 1, 1, FAR, FAR + MB, 5, ctypes.byref(k),
                              ctypes.byref(k), None) == code
    a = attention_args()
    assert lib.pb_cache_attention(ctypes.byref(c), ctypes.byref(a), FAR + 64 * MB, 1 << 40,
                                  None) == code
    n = ctypes.c_size_t()
    got = lib.pb_cache_scratch_bytes(ctypes.byref(c), ctypes.byref(n))
    assert got in (0, code)  # buffers are not looked at there
    assert lib.pb_cache_attention_scratch_bytes(ctypes.byref(c), ctypes.byref(n)) == got


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(n=9), 1), (dict(slots=None), 1), (dict(slots=FAR + 2), 1),
    (dict(starts=None), 1), (dict(scratch=None), 1), (dict(scratch=FAR + 4 * MB + 16), 1),
    (dict(nbytes=64), 3), (dict(scratch=P), 1), (dict(scratch=P + 33 * MB), 1), (dict(slots=P), 1),
    (dict(starts=P + 34 * MB), 1), (dict(slots=FAR + 4 * MB), 1), (dict(starts=FAR + 4 * MB + 256), 1),
])
def test_cache_calls_refused(lib, kw, code):
    assert calls(lib, cache(), **kw) == {code} and message(lib)


def test_keep_and_write_refused(lib):
    c = cache()
    r = ctypes.byref(c)
    assert keep(lib, c, tokens=-1) == 1
    for kw in (dict(path=None), dict(kept=None), dict(path=P), dict(kept=FAR + 4 * MB)):
        assert keep(lib, c, **kw) == 1, kw
    row = 4 * 64
    good = pb.pb_heads(FAR + 8 * MB, 4, 5 * row, row, 64)

    def write(layer=0, layers=2, n=1, slots=FAR, starts=FAR + MB, tokens=5, k=good, v=good):
        return lib.pb_cache_write(r, layer, layers, n, slots, starts, tokens,
                                  None if k is None else ctypes.byref(k),
                                  None if v is None else ctypes.byref(v), None)

    for kw in (dict(layer=-1), dict(layers=3), dict(layer=1), dict(layer=2 ** 31 - 1), dict(layers=-1),
               dict(tokens=-1), dict(tokens=2 ** 30 + 1), dict(n=-1), dict(n=9), dict(slots=None),
               dict(starts=None), dict(k=None), dict(v=None), dict(slots=P),
               dict(k=pb.pb_heads(FAR, 3, 5 * row, row, 64)), dict(v=pb.pb_heads(None, 4, 0, row, 64)),
               dict(v=pb.pb_heads(FAR + 8, 4, 0, row, 64)), dict(k=pb.pb_heads(FAR, 4, 0, row + 4, 64)),
               dict(k=pb.pb_heads(P, 4, 5 * row, row, 64)),
               dict(v=pb.pb_heads(P + 34 * MB, 4, 5 * row, row, 64))):
        assert write(**kw) == 1 and message(lib), kw
    for kw in (dict(layers=0), dict(n=0, slots=None, starts=None), dict(tokens=0)):
        assert write(**kw) == 0, kw


def test_no_sequences(lib):
    assert calls(lib, cache(), n=0, slots=None, starts=None, path=None, kept=None,
                 scratch=None) == {0}
    assert lib.pb_cache_scratch_bytes(None, None) == 1
    assert need(lib, cache()) >= 4 * 8 * 12


# --------------------------------------------------------------------------- attention over it

def attention_args(**kw):
    a = pb.pb_cache_attention_args(0, 2, 5, 0, 0.0, heads(FAR, 8, dh=64), heads(FAR + MB, 8, dh=64),
                                   FAR + 2 * MB, FAR + 3 * MB, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(layer=-1), 1), (dict(layer=2), 1), (dict(sequences=-1), 1), (dict(sequences=9), 1),
    (dict(tokens=-1), 1), (dict(tokens=2 ** 30 + 1), 1), (dict(tokens=2 ** 30), 2),
    (dict(window=-1), 1), (dict(scale=-0.5), 1), (dict(scale=float("nan")), 1),
    (dict(q=heads(None, 8, dh=64)), 1), (dict(q=heads(FAR + 8, 8, dh=64)), 1),
    (dict(q=heads(FAR, 6, dh=64), out=heads(FAR + MB, 6, dh=64)), 1),
    (dict(out=heads(FAR + MB, 4, dh=64)), 1), (dict(out=heads(FAR, 8, dh=64)), 1),
    (dict(out=heads(FAR + MB, 8, stride=0, dh=64)), 1), (dict(out=heads(P + MB // 4, 8, dh=64)), 1),
    (dict(out=heads(P + 34 * MB, 8, dh=64)), 1), (dict(slots=None), 1), (dict(starts=None), 1),
    (dict(slots=FAR + 2 * MB + 1), 1), (dict(parents=FAR + 2), 1), (dict(starts=FAR + MB), 1),
    (dict(parents=FAR + MB + 64), 1), (dict(slots=FAR + 64 * MB), 1), (dict(parents=FAR + 65 * MB), 1),
])
def test_attention_refused(lib, kw, code):
    c = cache()
    a = attention_args(**kw)
    if kw.get("tokens") == 2 ** 30:  # views that long must not meet
        a.q, a.out = heads(FAR + (1 << 50), 8, dh=64), heads(FAR + (1 << 52), 8, dh=64)
    assert lib.pb_cache_attention(ctypes.byref(c), ctypes.byref(a), FAR + 64 * MB, 1 << 40,
                                  None) == code and message(lib)


def test_attention_scratch_refused(lib):
    c, a = cache(), attention_args()
    for scratch, nbytes, code in ((None, 1 << 40, 1), (FAR + 64 * MB + 16, 1 << 40, 1),
                                  (FAR + 64 * MB, 1000, 3), (FAR, 1 << 40, 1), (FAR + MB, 1 << 40, 1),
                                  (P, 1 << 40, 1), (P + 33 * MB, 1 << 40, 1)):
        assert lib.pb_cache_attention(ctypes.byref(c), ctypes.byref(a), scratch, nbytes, None) == code
    assert lib.pb_cache_attention(ctypes.byref(c), None, FAR, 1 << 40, None) == 1
    for kw in (dict(sequences=0), dict(tokens=0)):
        b = attention_args(slots=None, starts=None, **kw)
        assert lib.pb_cache_attention(ctypes.byref(c), ctypes.byref(b), None, 0, None) == 0


# --------------------------------------------------------------------------- binding

def test_binding_refuses():
    bf = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pb._token_heads(bf.float(), 4, 2, 64, "q")
    with pytest.raises(ValueError):
        pb._token_heads(bf, 4, 3, 64, "q")
    with pytest.raises(ValueError):
        pb._token_heads(bf.transpose(1, 2), 4, 64, 2, "q")
    for bad in (torch.zeros(3), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(0, dtype=torch.int32),
                torch.zeros(6, dtype=torch.int32)[::2], torch.zeros(3, dtype=torch.int64)):
        with pytest.raises(ValueError):
            pb._sequences(bad)
        with pytest.raises(ValueError):
            pb._ints(bad, 3, "slots")
    for bad in (0, -1):
        with pytest.raises(ValueError):
            pb._window(bad)
        with pytest.raises(ValueError):
            pb._scale(bad)
    for bad in (float("nan"), float("inf"), 2.0 ** -127, 1e-300, 2.0 ** 127.5):
        with pytest.raises(ValueError):
            pb._scale(bad)
    assert pb._scale(None) == 0 and pb._scale(2.0 ** -126) > 0
    assert pb._window(None) == 0 and pb._window(2 ** 40) == 2 ** 31 - 1
    i32 = dict(dtype=torch.int32)
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    ok = (k, k.clone(), torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(4, **i32))
    pb.Cache(*ok)
    for at, bad in ((1, k[:, :3]), (1, k.float()), (2, ok[2].long()), (2, ok[2][0]), (3, ok[2][0]),
                    (4, ok[3]), (0, k.transpose(1, 2))):
        with pytest.raises(ValueError):
            pb.Cache(*[bad if i == at else t for i, t in enumerate(ok)])


@pytest.mark.parametrize("name", ["prompt.cu", "cache.cu", "cache_attention.cu"])
def test_dependent_launches_read_coherently(name):
    # These kernels may begin while the launch before them still writes what they read: no load
    # through the read-only path.
    body = open(os.path.join(os.path.dirname(build.__file__), "csrc", name)).read()
    assert "launch_dependent(" in body
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in body, (name, word)
