"""Long sequences through the serving attentions, where the bars of single values no longer show a
piece that is left out: results shrink with the root of the number of keys, the bars do not.

Planted values. With k = 0 every weight is 2^0 = 1, exactly, also in bf16; v is 1 in one column of a
key and 0 elsewhere, so a result is (keys seen that have the column) / (keys seen), both counted
exactly in fp32. What is left: the quotient and the product (2^-24 each) and the result's rounding,
2^-8 of it. At most 40 keys share a column (the others come in further runs), so one key left out or
counted twice moves a value by 1/40 = 2.5 % of itself.

Random values. A row's error is that of its weights' roundings (2^-8 of each at most) and of its own
(2^-8). The roundings do not know v, whose values are independent, so the errors of the keys add up as
the keys' values themselves do: their norm stays below 2^-8 of the row's norm, with the row's own
rounding 2^-7; errors of scores in fp32 (below 2^-10 of a weight, as in the operators' tests) add
2^-10. A tile of 64 keys left out of n moves the row by the root of 64 / n of its norm: 2.2 % at 131072
keys, three times the bar."""

import random

import pytest
import torch

from tests import test_gpu_cache_attention as ca
from tests import test_gpu_prompt_attention as pa
from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu
NORM = 2.0 ** -7 + 2.0 ** -10


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def planted(n, heads, dh, run, runs):
    """[n, heads, dh]: key j has column j (one further in each head) in run (j / dh) mod runs."""
    j = torch.arange(n, device="cuda")
    v = torch.zeros(n, heads, dh, dtype=torch.bfloat16, device="cuda")
    for h in range(heads):
        v[j, h, (j + h) % dh] = ((j // dh + h) % runs == run).to(torch.bfloat16)
    return v


def runs_for(n, dh):
    return -(-n // (40 * dh))


def put(c, pool, slot, x):
    """The tokens x [n, heads, dh] of a slot, in the cache's last layer."""
    page = c.k.shape[3]
    used = -(-len(x) // page)
    pad = torch.full((used * page, *x.shape[1:]), float("nan"), dtype=torch.bfloat16, device="cuda")
    pad[:len(x)] = x
    pool[-1, c.table[slot, :used].long()] = pad.view(used, page, *x.shape[1:]).transpose(1, 2)


def name(case):
    return f"{len(case[0])}x{case[0][0]}-" + "-".join(
        f"{len(x)}x{x[0]}" if isinstance(x, list) else str(x) for x in case[1:])


# lengths, new tokens, heads of q, of k, dh, page, tree, window
CACHES = [
    ([40000], [1], 4, 1, 128, 64, False, None),
    ([131072], [1], 4, 1, 128, 64, False, None),
    ([131072], [1], 8, 2, 64, 16, False, None),
    ([50000], [16], 4, 2, 64, 128, True, None),
    ([50000], [64], 2, 1, 128, 24, True, None),
    ([30011, 5, 20000], [3, 3, 3], 16, 4, 128, 48, False, None),
    ([30011, 20000], [300, 1], 8, 2, 64, 64, False, 15000),
    ([9000 - 251 * i for i in range(33)], [1] * 33, 8, 2, 128, 64, False, None),
    ([9000 - 251 * i for i in range(33)], [1 + i % 7 for i in range(33)], 6, 2, 64, 100, True, 4000),
]


def cache_case(lengths, counts, tree, hk, dh, page):
    c, data = ca.fill(lengths, hk, dh, page)
    slots = list(range(len(lengths)))
    rng = random.Random(len(lengths))
    rng.shuffle(slots)
    counts = [counts[s] for s in slots]
    starts = pa.starts_of(counts)
    parents = [rng.randint(-1, j - 1) if j else -1 for n in counts for j in range(n)] if tree else None
    return c, data, slots, starts, parents


@pytest.mark.parametrize("case", CACHES, ids=name)
def test_every_key_of_a_cache_counts_once(case):
    lengths, counts, hq, hk, dh, page, tree, window = case
    c, data, slots, starts, parents = cache_case(lengths, counts, tree, hk, dh, page)
    for s, n in enumerate(lengths):
        put(c, c.k, s, torch.zeros(n, hk, dh, dtype=torch.bfloat16, device="cuda"))
    q = ca.randn(5, starts[-1], hq, dh)
    runs = runs_for(max(lengths), dh)
    for run in range(runs):
        values = [planted(n, hk, dh, run, runs) for n in lengths]
        for s, v in enumerate(values):
            put(c, c.v, s, v)
        out = c.attention(q, ints(slots), ints(starts), window=window,
                          parents=None if parents is None else ints(parents))
        assert c.fault() == 0
        for s, a, z in zip(slots, starts, starts[1:]):
            seen = ca.visible(lengths[s], z - a, None if parents is None else parents[a:z],
                              window).double()
            want = torch.einsum("tn,nhd->thd", seen, values[s].double())
            want = (want / seen.sum(1).view(-1, 1, 1)).repeat_interleave(hq // hk, 1)
            err = (out[a:z].double() - want).abs()
            assert bool((err <= want * (2.0 ** -8 + 2.0 ** -22)).all()), (s, run, float(err.max()))


@pytest.mark.parametrize("case", CACHES, ids=name)
def test_rows_over_a_long_cache(case):
    lengths, counts, hq, hk, dh, page, tree, window = case
    c, data, slots, starts, parents = cache_case(lengths, counts, tree, hk, dh, page)
    q = ca.randn(5, starts[-1], hq, dh)
    out = c.attention(q, ints(slots), ints(starts), window=window,
                      parents=None if parents is None else ints(parents))
    assert c.fault() == 0
    for s, a, z in zip(slots, starts, starts[1:]):
        seen = ca.visible(lengths[s], z - a, None if parents is None else parents[a:z], window)
        want, _ = ca.reference(q[a:z], *data[s], seen, dh ** -0.5)
        err = (out[a:z].double() - want).norm(dim=-1)
        assert bool((err <= NORM * want.norm(dim=-1)).all()), (s, float((err / want.norm(dim=-1)).max()))


# lengths, heads of q, of k, dh, window
PROMPTS = [
    ([16384], 4, 1, 128, None),
    ([16384], 3, 1, 64, None),
    ([9000, 1, 5000, 0, 2049], 2, 2, 128, 1000),
    ([9000, 1, 5000, 0, 2049], 8, 1, 64, 5000),
    ([100 + 13 * i for i in range(140)], 4, 2, 64, None),
]


@pytest.mark.parametrize("case", PROMPTS, ids=name)
def test_every_key_of_prompts_counts_once(case):
    lengths, hq, hk, dh, window = case
    s = pa.starts_of(lengths)
    q, k = pa.randn(1, s[-1], hq, dh), torch.zeros(s[-1], hk, dh, dtype=torch.bfloat16, device="cuda")
    runs = runs_for(min(max(lengths), window or max(lengths)), dh)
    for run in range(runs):
        v = torch.cat([planted(n, hk, dh, run, runs) for n in lengths])
        out = pb.prompt_attention(q, k, v, ints(s), window=window)
        for a, z in zip(s, s[1:]):
            if z == a:
                continue
            n = z - a
            w = min(window or n, n)
            total = v[a:z].double().cumsum(0)
            seen = total.clone()
            seen[w:] -= total[:n - w]
            number = torch.arange(1, n + 1, device="cuda").clamp(max=w).view(-1, 1, 1)
            want = (seen / number).repeat_interleave(hq // hk, 1)
            err = (out[a:z].double() - want).abs()
            assert bool((err <= want * (2.0 ** -8 + 2.0 ** -22)).all()), (a, z, run, float(err.max()))


@pytest.mark.parametrize("case", [([8192], 4, 1, 128, None), ([8192], 3, 1, 64, None),
                                  ([5000, 300, 8000], 2, 2, 128, 1000)] + PROMPTS[-1:],
                         ids=name)
def test_rows_of_long_prompts(case):
    lengths, hq, hk, dh, window = case
    s = pa.starts_of(lengths)
    q, k, v = pa.randn(1, s[-1], hq, dh), pa.randn(2, s[-1], hk, dh), pa.randn(3, s[-1], hk, dh)
    out = pb.prompt_attention(q, k, v, ints(s), window=window)
    for a, z in zip(s, s[1:]):
        want, _ = pa.reference(q, k, v, a, z - a, window, dh ** -0.5)
        err = (out[a:z].double() - want).norm(dim=-1)
        assert bool((err <= NORM * want.norm(dim=-1)).all()), (a, float((err / want.norm(dim=-1)).max()))
