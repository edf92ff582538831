"""fork, free and compact with more requests than one block works: what a block of the cluster finds
reaches the others, and the tables equal the list model's."""
import numpy as np
import pytest
import torch

from test_gpu_cache import BOUNDS, OK, i32, make, rows_of

pytestmark = pytest.mark.gpu
N, PS = 2500, 16                                        # requests 0 .. 1023 are block 0's, and so on


def tables(c, m):
    assert c.lens.tolist() == m.lens and c.ref.tolist() == m.ref
    assert c.page_table.tolist() == [p + [-1] * (m.maxp - len(p)) for p in m.pages]


def filled(seed=0):
    """A cache of 2N slots, the first N of which hold 0 to 2 pages."""
    rng = np.random.default_rng(seed)
    c, m = make(3 * N, PS, 2 * N, 3, 8, torch.bfloat16)
    cnt = rng.integers(0, 2 * PS + 1, N)
    cnt[[0, 5, 2000]] = 20, 3, 17
    off = [0] + np.cumsum(cnt).tolist()
    src = rows_of(rng, off[-1], 8, torch.bfloat16)
    c.append(i32(range(N)), i32(off), *(t.cuda() for t in src))
    assert c.check_device_error() == OK
    at = 0
    for s in range(N):                                  # the model's append, without its rows
        m.lens[s], n = int(cnt[s]), -(-int(cnt[s]) // PS)
        m.pages[s] = list(range(at, at + n))
        at += n
    m.ref = [1] * at + [0] * (3 * N - at)
    tables(c, m)
    return rng, c, m


def test_fork_and_free_of_many_slots():
    rng, c, m = filled()
    src = rng.integers(0, N, N).tolist()                # sources repeat, across blocks too
    dst = (N + rng.permutation(N)).tolist()
    c.fork(i32(src), i32(dst))
    m.fork(src, dst)
    assert c.check_device_error() == OK
    tables(c, m)
    gone = rng.permutation(2 * N)[:N].tolist()
    c.free(i32(gone))
    m.free(gone)
    assert c.check_device_error() == OK
    tables(c, m)


@pytest.mark.parametrize("at", [0, 1023, 1024, 2000, N - 1])
def test_one_bad_request_refuses_all(at):
    """Wherever the bad request is, every block refuses, and the call after is as if it had not been."""
    _, c, m = filled()
    src, dst = list(range(N)), list(range(N, 2 * N))
    other = (at + 1300) % N                             # a request of another block

    def swap(x, v):
        return x[:at] + [v] + x[at + 1:]

    calls = [
        lambda: c.free(i32(swap(src, 2 * N))), lambda: c.free(i32(swap(src, -1))),
        lambda: c.free(i32(swap(src, src[other]))),                         # a slot named twice
        lambda: c.fork(i32(swap(src, 2 * N)), i32(dst)), lambda: c.fork(i32(src), i32(swap(dst, -5))),
        lambda: c.fork(i32(src), i32(swap(dst, dst[other]))),               # a destination named twice
        lambda: c.fork(i32(swap(src, dst[other])), i32(dst)),               # a source that is a destination
        lambda: c.fork(i32(src), i32(swap(dst, 5))),                        # a destination that is not empty
        lambda: c.compact(i32(swap(src, src[other])), i32([0] * (N + 1)), i32([])),
        lambda: c.compact(i32(swap(src, 2 * N)), i32([0] * (N + 1)), i32([])),
    ]
    for k, call in enumerate(calls):
        call()
        assert c.check_device_error() == BOUNDS, k
        tables(c, m)
    c.fork(i32(src), i32(dst))
    m.fork(src, dst)
    assert c.check_device_error() == OK
    tables(c, m)


def test_compact_of_many_slots():
    rng, c, m = filled(1)
    rows = [torch.cat([c.k[p] for p in m.pages[s]]).cpu()[:m.lens[s]] if m.lens[s] else torch.zeros(0, 8, dtype=torch.bfloat16)
            for s in range(N)]
    slots = rng.permutation(N).tolist()
    keep, off = [], [0]
    for s in slots:
        keep += np.sort(rng.permutation(m.lens[s])[:rng.integers(0, min(m.lens[s], PS) + 1)]).tolist()
        off.append(len(keep))
    m.compact(slots, off, keep)
    c.compact(i32(slots), i32(off), i32(keep))
    assert c.check_device_error() == OK
    tables(c, m)
    for i, s in enumerate(slots):
        if off[i] < off[i + 1]:
            assert torch.equal(c.k[m.pages[s][0]].cpu()[:m.lens[s]], rows[s][keep[off[i]:off[i + 1]]])
