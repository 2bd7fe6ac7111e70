"""How far a key or a value that is not finite reaches in the serving attentions. A key's scores are
replaced where a token does not see it, so it reaches the tokens that see it and no others. A value
meets weights of zero (0 x NaN is NaN), so it reaches every token whose tile of rows is computed with
its tile of keys: earlier tokens, and with a window later ones. All other results keep their bits."""

import pytest
import torch

from tests import test_gpu_cache_attention as ca
from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("hq,hk,dh,window", [(2, 2, 128, 1), (8, 2, 64, 1), (8, 2, 128, 100),
                                             (6, 2, 64, 129), (3, 3, 64, 300), (4, 1, 128, None)])
def test_prompts(hq, hk, dh, window, bad):
    before, n = 37, 700
    s = ints([0, before, before + n])
    q, k, v = ca.randn(1, before + n, hq, dh), ca.randn(2, before + n, hk, dh), \
        ca.randn(3, before + n, hk, dh)
    want = pb.prompt_attention(q, k, v, s, window=window)
    w, rows = window or n, 128 // (hq // hk)  # tokens of a tile of rows
    i = torch.arange(n)
    first = i // rows * rows
    lo = (first - w + 1).clamp(min=0) // 128
    hi = ((first + rows).clamp(max=n) - 1) // 128
    for j in (0, 1, 63, 127, 128, 255, 256, 400, 699):
        sees = ((j <= i) & (j > i - w)).cuda()
        beside = ((lo <= j // 128) & (j // 128 <= hi)).cuda()
        for what in "kv":
            x = dict(k=k, v=v)
            x[what] = x[what].clone()
            x[what][before + j] = bad
            got = pb.prompt_attention(q, x["k"], x["v"], s, window=window)
            assert torch.equal(got[:before], want[:before])
            got = got[before:]
            kept = ~(beside if what == "v" else sees)
            assert torch.equal(got[kept], want[before:][kept]), (j, what)
            if what == "v":  # a weight is above zero for what is seen
                assert not bool(torch.isfinite(got[sees]).any()), j


def test_first_value_behind_a_window_of_one():
    # 128 tokens that see themselves only share a tile: the first one's value reaches the others
    q, k, v = (ca.randn(i, 300, 1, 64) for i in range(3))
    want = pb.prompt_attention(q, k, v, window=1)
    v[0] = float("nan")
    got = pb.prompt_attention(q, k, v, window=1)
    assert bool(torch.isnan(got[0]).all())
    assert torch.equal(got[128:], want[128:])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("counts,tree,window", [((1, 1), False, 200), ((1, 1), False, None),
                                                ((70, 20), False, 33), ((16, 60), True, 5),
                                                ((64, 3), True, None)])
def test_over_a_cache(counts, tree, window, bad):
    lengths = [700, 333]
    c, data = ca.fill(lengths, 2, 64, 24)
    t = sum(counts)
    q = ca.randn(9, t, 8, 64)
    starts = [0, counts[0], t]
    parents = [j // 2 - 1 if j else -1 for n in counts for j in range(n)] if tree else None
    up = None if parents is None else ints(parents)

    def run():
        out = c.attention(q, ints([0, 1]), ints(starts), parents=up, window=window)
        assert c.fault() == 0
        return out

    want = run()
    n, count = lengths[0], counts[0]
    seen = ca.visible(n, count, None if parents is None else parents[:count], window)
    w = window or n
    for j in (0, 63, 64, 400, 630, 640, 699):
        page, row = int(c.table[0, j // 24]), j % 24
        for pool, what in ((c.k, "k"), (c.v, "v")):
            old = pool[0, page, :, row].clone()
            pool[0, page, :, row] = bad
            got = run()
            pool[0, page, :, row] = old
            assert torch.equal(got[count:], want[count:])
            if what == "k":
                kept = ~seen[:, j]
            else:  # a block reads no tile behind the window of its first token at most
                kept = torch.full((count,), j // 64 < max(0, n - count - w + 1) // 64, device="cuda")
                assert not bool(torch.isfinite(got[:count][seen[:, j]]).any())
            assert torch.equal(got[:count][kept], want[:count][kept]), (j, what)
