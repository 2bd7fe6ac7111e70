"""Reads and writes of the rotation, linear and AdamW calls where element offsets pass 2^32: the data
is random everywhere, so a value from an offset that has lost its upper bits (2^31 or 2^32 elements
before its place) gives another result. And the linear layer's forms from several host threads,
each result against the same call made alone."""

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def test_rotation_reads_its_own_heads():
    s, h, d = 66000, 512, 128  # 4.33e9 values
    g = gen(1)
    x = torch.randn(1, s, h, d, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(1, s, h, d, generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.randint(0, 100000, (1, 1, s), generator=g, device="cuda", dtype=torch.int32)
    gamma = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    rope = pb.Rope(d)
    y, _ = pb.qk_norm_rope(rope, x, None, pos, gamma)
    dx, _, dgamma, _ = pb.qk_norm_rope_backward(rope, x, None, pos, dy, None, gamma)
    # heads are independent: the same bits from a call on a few tokens alone
    for t in (0, 464, 2 ** 31 // (h * d), 2 ** 32 // (h * d) - 1, 2 ** 32 // (h * d), s - 40):
        part = slice(t, t + 40)
        a, b, p = x[:, part].clone(), dy[:, part].clone(), pos[:, :, part].contiguous()
        assert torch.equal(y[:, part], pb.qk_norm_rope(rope, a, None, p, gamma)[0]), t
        assert torch.equal(dx[:, part], pb.qk_norm_rope_backward(rope, a, None, p, b, None,
                                                                 gamma)[0]), t
    # dgamma: the part of the tokens beyond 2^32 is what is missing without them
    del y, dx
    n = 2 ** 32 // (h * d)
    front = pb.qk_norm_rope_backward(rope, x[:, :n], None, pos[:, :, :n].contiguous(), dy[:, :n],
                                     None, gamma)[2].double()
    back = pb.qk_norm_rope_backward(rope, x[:, n:].clone(), None, pos[:, :, n:].contiguous(),
                                    dy[:, n:].clone(), None, gamma)[2].double()
    # partial sums of 34 million values of standard deviation 1: 2^-24 of each partial sum
    # (sqrt(34e6) = 5800 in the mean) a step of chains of some 10,000, in random directions
    room = 5800 * 2.0 ** -24 * 10000 ** 0.5 * 4
    assert float((dgamma.double() - front - back).abs().max()) <= room
    assert float(back.abs().max()) > 100 * room


def test_linear_reads_its_own_rows():
    m, n = 131100, 32776  # 4.297e9 values
    g = gen(2)
    big = torch.randn(m, n, generator=g, device="cuda", dtype=torch.bfloat16)
    edge = 2 ** 31 // n
    rows = torch.tensor([0, 1, 63, edge, edge + 1, 2 ** 32 // n,
                         2 ** 32 // n + 1, m - 1], device="cuda")
    cols = torch.tensor([0, 1, 255, 16384, n - 1], device="cuda")

    def close(got, a, b, k):
        # half a bf16 step, or fp32 sums cut off 2^-22 of their magnitudes for every 16 of k
        s = a.double().abs() @ b.double().abs()
        half = 2.0 ** -8 if got.dtype is torch.bfloat16 else 2.0 ** -24
        ref = a.double() @ b.double()
        assert ((got.double() - ref).abs() <= half * ref.abs() + (k / 16 + 100) * 2.0 ** -22 * s).all()

    # as x, as dy, and as the weights of three tokens
    w = torch.randn(n, 64, generator=g, device="cuda").to(torch.bfloat16)
    close(pb.linear(big, w)[rows], big[rows], w, n)
    x = torch.randn(m, 64, generator=g, device="cuda").to(torch.bfloat16)
    wt = w.t().contiguous()
    dx, dw, db = pb.linear_backward(big, x, wt, bias=True)
    close(dx[rows], big[rows], wt.t(), n)
    close(dw[:, cols], x.t(), big[:, cols], m)
    ref = big[:, cols].double().sum(0)
    room = (m / 512 + 80) * 2.0 ** -24 * big[:, cols].double().abs().sum(0)
    assert ((db[cols].double() - ref).abs() <= room).all()
    few = torch.randn(3, m // 8 * 8, generator=g, device="cuda").to(torch.bfloat16)
    close(pb.linear(few, big[:m // 8 * 8])[:, cols], few, big[:m // 8 * 8, cols], m)
    few = torch.randn(3, n, generator=g, device="cuda").to(torch.bfloat16)
    y = pb.linear(few, big, layout=pb.PB_WEIGHT_OUT_IN)
    close(y[:, rows], few, big[rows].t(), n)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_steps_its_own_values(bits):
    n = 2 ** 32 + 123456
    g = gen(3)
    p = torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16)
    grad = torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16)
    st = pb.adamw_states(p, bits)
    opt = pb.AdamW([dict(param=p, grad=grad, weight_decay=0.1, **st)])
    # whole state blocks; offsets that lose bits from 2^31 or 2^32 on lead to the first ones
    parts = [slice(0, 8192), slice(2 ** 31 - 4096, 2 ** 31 + 4096),
             slice(2 ** 32 - 4096, 2 ** 32 + 4096), slice(n // 256 * 256 - 4096, n)]
    alone = []
    for part in parts:
        q, d = p[part].clone(), grad[part].clone()
        s = pb.adamw_states(q, bits)
        alone.append((q, s, pb.AdamW([dict(param=q, grad=d, weight_decay=0.1, **s)])))
    for step in (1, 2):
        opt.step(lr=0.01, step=step)
        for _, _, o in alone:
            o.step(lr=0.01, step=step)
    for part, (q, s, _) in zip(parts, alone):
        assert torch.equal(p[part], q)
        for k in ("m", "v"):
            assert torch.equal(st[k][part].view(torch.uint8) if bits == 8 else st[k][part],
                               s[k].view(torch.uint8) if bits == 8 else s[k])
            if bits == 8:
                blocks = slice(part.start // 256, -(-part.stop // 256))
                assert torch.equal(st[k + "_scale"][blocks], s[k + "_scale"])
    norm = opt.grad_norm(max_norm=1e9)
    total = sum(float(grad[c:c + 2 ** 28].double().square().sum()) for c in range(0, n, 2 ** 28))
    # squares of bf16 values are exact in fp32; a thread's four sums are chains of some 5,000,
    # rounded 2^-25 of the sum each in random directions, and the root halves it: far below 2^-17
    assert abs(float(norm[0]) - total ** 0.5) <= 2.0 ** -17 * total ** 0.5
    assert abs(total - n) < n * 1e-3


def test_linear_from_several_host_threads():
    g = gen(4)
    x = torch.randn(200, 4096, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(4096, 8192, generator=g, device="cuda").to(torch.bfloat16) * 0.02
    narrow = w[:, :640].contiguous()

    def calls(scratch):
        out = []
        for s in (None, scratch):
            for t in (1, 3, 20, 32):
                out.append(pb.linear(x[:t], w, activation="gelu", scratch=s))
                out.append(pb.linear(x[:t], narrow, out_dtype=torch.float32, scratch=s))
            out.append(pb.linear(x, narrow, scratch=s))
            out += pb.linear_backward(out[-1], x, narrow, bias=True, scratch=s)
        return out

    def new_scratch():
        return torch.empty(pb.linear_scratch_bytes(), dtype=torch.uint8, device="cuda")

    want = calls(new_scratch())
    torch.cuda.synchronize()
    wrong, done = [], []

    def work():
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            scratch = new_scratch()
            for _ in range(20):
                got = calls(scratch)
                torch.cuda.current_stream().synchronize()
                wrong.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))
            done.append(True)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and len(done) == 4
