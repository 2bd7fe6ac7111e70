"""Host threads that change one cache at the same time, on one stream: copies of shared pages and
moved rows are each call's own."""

import threading

import pytest
import torch

from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_threads_change_one_cache_on_one_stream():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    page, layers, heads, dh, own, threads = 16, 2, 3, 64, 4, 3
    c = pb.Cache.empty(layers, 60, page, heads, dh, 1 + threads * own, 4)
    c.k.zero_()
    c.v.zero_()

    def rows(seed, n):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        return [torch.randn(layers, n, heads, dh, generator=g, device="cuda").to(torch.bfloat16)
                for _ in range(2)]

    # slot 0: 20 tokens, so the samples of it share a partly filled page
    base = rows(1, 20)
    c.extend(ints([0]), ints([0, 20]))
    c.write(*base, ints([0]), ints([0, 20]))
    torch.cuda.synchronize()
    errors, flags = [], []

    def work(i):
        try:
            torch.cuda.set_device(0)
            mine = list(range(1 + i * own, 1 + (i + 1) * own))
            sl, zeros, src = ints(mine), ints([0] * own), ints([0] * own)
            at = torch.tensor(mine, device="cuda")
            # the threads' calls have lists of different lengths: 3, 4 or 5 drafts each
            drafts = 3 + i
            starts = ints([drafts * j for j in range(own + 1)])
            paths = [[0, 2], [1], [], list(range(drafts))]
            path = ints(sum([p + [0] * (drafts - len(p)) for p in paths], []))
            kept = ints([len(p) for p in paths])
            for step in range(60):
                new = rows(100 * i + step + 2, drafts * own)
                c.truncate(sl, zeros)
                c.fork(src, sl)
                c.extend(sl, starts)
                c.write(*new, sl, starts)
                c.keep(sl, starts, path, kept)
                pages = c.table[at, :2].long()
                for pool, old, x in zip((c.k, c.v), base, new):
                    got = pool[:, pages].transpose(3, 4).reshape(layers, own, 2 * page, heads, dh)
                    for j, p in enumerate(paths):
                        want = torch.cat([old, x[:, [drafts * j + u for u in p]]], 1)
                        flags.append((got[:, j, :want.shape[1]] == want).all())
        except BaseException as e:  # reported by the test
            errors.append(e)

    them = [threading.Thread(target=work, args=(i,)) for i in range(threads)]
    for t in them:
        t.start()
    for t in them:
        t.join()
    assert not errors, errors
    assert c.fault() == 0
    assert len(flags) == threads * 60 * 2 * own and bool(torch.stack(flags).all())
    assert c.lengths.tolist() == [20] + [22, 21, 20, 23] + [22, 21, 20, 24] + [22, 21, 20, 25]
