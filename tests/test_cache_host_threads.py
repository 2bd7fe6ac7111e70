"""The binding keeps calls that change one cache apart: extend, keep and fork are several launches that
hand one another a list in the cache's scratch, so the launches of one call must not come between
those of another, whatever stream they are on (CPU only; the library's calls are counted, not made)."""

import threading
import time

import pytest
import torch

from transformer_block_gb300 import build, pb

CHANGES = ("pb_cache_extend", "pb_cache_write", "pb_cache_keep", "pb_cache_fork", "pb_cache_truncate")


class Counting:
    """The library, but for the calls that change a cache: how many of them run at once."""

    def __init__(self, real):
        self.real, self.guard = real, threading.Lock()
        self.busy, self.most, self.calls, self.fail = {}, {}, [], False

    def __getattr__(self, name):
        if name not in CHANGES:
            return getattr(self.real, name)

        def call(plan, *args):
            key = plan
            with self.guard:
                self.calls.append(name)
                self.busy[key] = self.busy.get(key, 0) + 1
                self.most[key] = max(self.most.get(key, 0), self.busy[key])
            time.sleep(0.002)
            with self.guard:
                self.busy[key] -= 1
            return 1 if self.fail else 0

        return call


@pytest.fixture
def counting(monkeypatch):
    build.build()
    counted = Counting(pb.lib())
    monkeypatch.setattr(pb, "lib", lambda: counted)
    monkeypatch.setattr(pb, "_here", lambda *tensors: None)
    monkeypatch.setattr(pb, "_stream", lambda stream: None)
    return counted


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def small():
    i32 = dict(dtype=torch.int32)
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    return pb.Cache(k, k.clone(), torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(4, **i32))


def change(c):
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    c.extend(ints(0), ints(0, 1))
    c.write(x, x, ints(0), ints(0, 1))
    c.keep(ints(0), ints(0, 1), ints(0), ints(1))
    c.fork(ints(0), ints(1))
    c.truncate(ints(1), ints(0))


def in_threads(n, work):
    errors = []

    def run(i):
        try:
            work(i)
        except BaseException as e:  # reported by the test
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_calls_on_one_cache_follow_one_another(counting):
    c = small()
    in_threads(4, lambda i: [change(c) for _ in range(3)])
    assert counting.most == {c._plan: 1}
    assert sorted(counting.calls) == sorted(4 * 3 * CHANGES)


def test_a_refused_call_leaves_the_cache_free(counting):
    c = small()
    counting.fail = True
    with pytest.raises(pb.PbError):
        c.extend(ints(0), ints(0, 1))
    counting.fail = False
    done = threading.Thread(target=change, args=(c,), daemon=True)
    done.start()
    done.join(20)
    assert not done.is_alive()


def test_caches_are_independent(counting):
    # a call on one cache does not wait for a call on another
    one, other = small(), small()
    with one._changing:
        free = threading.Thread(target=change, args=(other,), daemon=True)
        free.start()
        free.join(20)
        assert not free.is_alive()


def test_what_runs_inside_a_call_may_change_the_cache(counting, monkeypatch):
    # a finalizer or a signal's handler runs on the thread that is in a call, and frees a slot
    c = small()

    def freeing(stream):
        monkeypatch.setattr(pb, "_stream", lambda stream: None)
        c.truncate(ints(1), ints(0))

    monkeypatch.setattr(pb, "_stream", freeing)
    done = threading.Thread(target=c.extend, args=(ints(0), ints(0, 1)), daemon=True)
    done.start()
    done.join(20)
    assert not done.is_alive()
    assert counting.calls == ["pb_cache_truncate", "pb_cache_extend"]
