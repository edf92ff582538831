"""Page operators of the history cache against a plain model that keeps every history as a list:
tables, counts and rows are equal, whatever the order of calls."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
OK, BOUNDS, FULL = 0, -5, -7


class Model:
    """The cache's rules in lists: lowest free page first, a shared page copied before it is written."""

    def __init__(self, n_pages, ps, n_slots, max_pages, D, dtype):
        self.ps, self.maxp = ps, max_pages
        self.k = torch.zeros(n_pages, ps, D, dtype=dtype)
        self.v, self.ts = self.k.clone(), torch.zeros(n_pages, ps, dtype=torch.int64)
        self.pages, self.lens, self.ref = [[] for _ in range(n_slots)], [0] * n_slots, [0] * n_pages

    def take(self):
        p = self.ref.index(0)
        self.ref[p] = 1
        return p

    def row(self, s, r):
        return self.pages[s][r // self.ps], r % self.ps

    def append(self, slots, off, k, v, ts, rows=None):
        held = list(self.ref)                           # sharing is judged before the call
        old = []
        freed = []
        for i, s in enumerate(slots):
            cnt, n = off[i + 1] - off[i], self.lens[s]
            old.append(n)
            if cnt and n % self.ps and held[self.pages[s][-1]] > 1:
                freed.append((s, self.pages[s][-1], n))
                self.pages[s][-1] = self.take()
            while len(self.pages[s]) * self.ps < n + cnt:
                self.pages[s].append(self.take())
            self.lens[s] = n + cnt
        for s, p, n in freed:
            q = self.pages[s][n // self.ps]
            for t in (self.k, self.v, self.ts):
                t[q] = t[p]
            self.ref[p] -= 1
        for i, s in enumerate(slots):
            for r in range(off[i], off[i + 1]):
                f = r if rows is None else rows[r]
                p, o = self.row(s, old[i] + r - off[i])
                if 0 <= f < len(k):
                    self.k[p, o], self.v[p, o], self.ts[p, o] = k[f], v[f], ts[f]
                else:
                    self.k[p, o], self.v[p, o], self.ts[p, o] = 0, 0, 0

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.pages[b], self.lens[b] = list(self.pages[a]), self.lens[a]
            for p in self.pages[b]:
                self.ref[p] += 1

    def compact(self, slots, off, keep):
        fresh, gone = [], []
        for i, s in enumerate(slots):
            fresh.append([self.take() for _ in range(-(-(off[i + 1] - off[i]) // self.ps))])
        for i, s in enumerate(slots):
            for e, r in enumerate(keep[off[i]:off[i + 1]]):
                p, o = fresh[i][e // self.ps], e % self.ps
                if 0 <= r < self.lens[s]:
                    a, b = self.row(s, r)
                    for t in (self.k, self.v, self.ts):
                        t[p, o] = t[a, b]
                else:
                    for t in (self.k, self.v, self.ts):
                        t[p, o] = 0
            gone += self.pages[s]
        for p in gone:
            self.ref[p] -= 1
        for i, s in enumerate(slots):
            self.pages[s], self.lens[s] = fresh[i], off[i + 1] - off[i]

    def free(self, slots):
        for s in slots:
            for p in self.pages[s]:
                self.ref[p] -= 1
            self.pages[s], self.lens[s] = [], 0


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def same(c, m):
    assert c.lens.tolist() == m.lens
    assert c.ref.tolist() == m.ref
    want = [p + [-1] * (m.maxp - len(p)) for p in m.pages]
    assert c.page_table.tolist() == want
    k, v, ts = c.k.cpu(), c.v.cpu(), c.ts.cpu()
    assert torch.equal(k, m.k) and torch.equal(v, m.v) and torch.equal(ts, m.ts)


def make(n_pages, ps, n_slots, max_pages, D, dtype):
    from hstu_jagged_pointwise_b200 import ops
    return ops.PagedCache(n_pages, ps, n_slots, max_pages, D, dtype), Model(n_pages, ps, n_slots, max_pages, D, dtype)


def rows_of(rng, n, D, dtype):
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    return (torch.randn(n, D, generator=g).to(dtype), torch.randn(n, D, generator=g).to(dtype),
            torch.randint(0, 2**62, (n,), generator=g))


@pytest.mark.parametrize("ps,D,dtype", [(16, 8, torch.bfloat16), (32, 520, torch.bfloat16), (64, 1032, torch.float32), (128, 64, torch.bfloat16)])
def test_random_calls_equal_the_model(ps, D, dtype):
    """Forty calls of random kinds, sizes and slots; forks of forks, appends to shared pages, cuts of
    shared histories; the whole pool is compared after each."""
    rng = np.random.default_rng(ps)
    n_slots, max_pages = 9, 5
    c, m = make(60, ps, n_slots, max_pages, D, dtype)
    for step in range(40):
        kind = rng.choice(["append", "append", "append", "fork", "compact", "free"])
        slots = rng.permutation(n_slots)[:rng.integers(1, n_slots + 1)].tolist()
        if kind == "append":
            cnt = [int(min(rng.choice([0, 1, ps - 1, ps, ps + 1, 2 * ps + 3]), max_pages * ps - m.lens[s])) for s in slots]
            off = [0] + np.cumsum(cnt).tolist()
            gather = rng.random() < 0.5
            src = rows_of(rng, off[-1] + (5 if gather else 0), D, dtype)
            rows = rng.integers(0, off[-1] + 5, off[-1]).tolist() if gather else None
            m.append(slots, off, *src, rows)
            c.append(i32(slots), i32(off), *(t.cuda() for t in src), rows=None if rows is None else i32(rows))
        elif kind == "fork":
            empty = [s for s in range(n_slots) if m.lens[s] == 0]
            full = [s for s in range(n_slots) if m.lens[s] > 0]
            if not empty or not full:
                continue
            src = rng.choice(full, len(empty)).tolist()
            m.fork(src, empty)
            c.fork(i32(src), i32(empty))
        elif kind == "compact":
            keep, off = [], [0]
            for s in slots:
                n = m.lens[s]
                j = int(rng.integers(0, n + 1))
                keep += (np.sort(rng.permutation(n)[:j]) if rng.random() < 0.7 else rng.integers(0, max(n, 1), j)).tolist()
                off.append(len(keep))
            m.compact(slots, off, keep)
            c.compact(i32(slots), i32(off), i32(keep))
        else:
            m.free(slots)
            c.free(i32(slots))
        assert c.check_device_error() == OK, (step, kind)
        same(c, m)


def filled(n_pages=12, ps=16, n_slots=5, max_pages=4, D=64):
    c, m = make(n_pages, ps, n_slots, max_pages, D, torch.bfloat16)
    src = rows_of(np.random.default_rng(0), 50, D, torch.bfloat16)
    m.append([0, 1], [0, 30, 50], *src)
    c.append(i32([0, 1]), i32([0, 30, 50]), *(t.cuda() for t in src))
    same(c, m)
    return c, m, [t.cuda() for t in src]


def test_refused_requests_change_nothing():
    c, m, (k, v, ts) = filled()
    n = lambda *x: i32(x)
    cases = [
        (lambda: c.free(n(0, 0)), BOUNDS), (lambda: c.free(n(5)), BOUNDS), (lambda: c.free(n(-1)), BOUNDS),
        (lambda: c.fork(n(0), n(1)), BOUNDS),                       # the destination is not empty
        (lambda: c.fork(n(0, 0), n(2, 2)), BOUNDS), (lambda: c.fork(n(2), n(2)), BOUNDS), (lambda: c.fork(n(9), n(2)), BOUNDS),
        (lambda: c.fork(n(0, 2), n(2, 3)), BOUNDS),                 # a destination is a source
        (lambda: c.append(n(2, 2), n(0, 25, 50), k, v, ts), BOUNDS), (lambda: c.append(n(2, 3), n(0, 30, 20), k, v, ts), BOUNDS),
        (lambda: c.append(n(2, 3), n(1, 25, 50), k, v, ts), BOUNDS), (lambda: c.append(n(2, 3), n(0, 25, 49), k, v, ts), BOUNDS),
        (lambda: c.append(n(0), n(0, 50), k, v, ts), BOUNDS),       # 80 rows in a slot of 64
        (lambda: c.append(n(2, 3), n(0, 2**31 - 1, 50), k, v, ts), BOUNDS),
        (lambda: c.compact(n(0, 0), n(0, 1, 2), n(0, 1)), BOUNDS), (lambda: c.compact(n(0), n(0, 3), n(0, 1)), BOUNDS),
    ]
    for call, want in cases:
        call()
        assert c.check_device_error() == want
        same(c, m)
        assert c.check_device_error() == OK
    # a pool that runs out: 4 of 11 pages are held
    c, m, (k, v, ts) = filled(n_pages=11)
    c.append(n(2, 3, 4), n(0, 17, 33, 50), k, v, ts)                # 2 + 1 + 2 pages
    m.append([2, 3, 4], [0, 17, 33, 50], k.cpu(), v.cpu(), ts.cpu())
    same(c, m)
    c.compact(n(0, 1), n(0, 30, 50), n(*range(30), *range(20)))     # four fresh pages, two are free
    assert c.check_device_error() == FULL
    same(c, m)
    c.append(n(2), n(0, 40), k[:40], v[:40], ts[:40])
    m.append([2], [0, 40], k[:40].cpu(), v[:40].cpu(), ts[:40].cpu())
    assert c.check_device_error() == OK
    same(c, m)
    c.append(n(3), n(0, 40), k[:40], v[:40], ts[:40])
    assert c.check_device_error() == FULL
    same(c, m)


def test_source_rows_out_of_range_are_zero_and_flagged():
    c, m, (k, v, ts) = filled()
    rows = [3, -1, 49, 50, 2**31 - 1]
    c.append(i32([2]), i32([0, 5]), k, v, ts, rows=i32(rows))
    m.append([2], [0, 5], k.cpu(), v.cpu(), ts.cpu(), rows)
    assert c.check_device_error() == BOUNDS
    same(c, m)
    c.compact(i32([0]), i32([0, 4]), i32([29, 30, -5, 0]))
    m.compact([0], [0, 4], [29, 30, -5, 0])
    assert c.check_device_error() == BOUNDS
    same(c, m)


def test_empty_requests():
    c, m, (k, v, ts) = filled()
    e = i32([])
    c.free(e), c.fork(e, e), c.append(e, i32([0]), k[:0], v[:0], ts[:0]), c.compact(e, i32([0]), e)
    c.append(i32([3, 0]), i32([0, 0, 0]), k[:0], v[:0], ts[:0])
    c.compact(i32([3]), i32([0, 0]), e)
    c.fork(i32([3]), i32([4]))
    assert c.check_device_error() == OK
    same(c, m)


def test_beam_step_shares_and_splits_pages():
    """Four beams of one history append different events: the shared last page splits into four, the
    source keeps its own, and the full pages stay shared."""
    c, m, (k, v, ts) = filled(n_pages=20, n_slots=8)
    c.fork(i32([0] * 4), i32([2, 3, 4, 5]))
    m.fork([0] * 4, [2, 3, 4, 5])
    off = [0, 1, 2, 3, 4]
    c.append(i32([2, 3, 4, 5]), i32(off), k[:4], v[:4], ts[:4])
    m.append([2, 3, 4, 5], off, k[:4].cpu(), v[:4].cpu(), ts[:4].cpu())
    same(c, m)
    assert m.ref[m.pages[0][0]] == 5 and m.ref[m.pages[0][1]] == 1
    c.free(i32([0]))
    m.free([0])
    same(c, m)


def test_captured_replayed_and_on_another_stream():
    """A captured fork, append and free replays on what the tables hold then."""
    c, m, (k, v, ts) = filled(n_pages=20)
    src, dst, off = i32([0, 1]), i32([2, 3]), i32([0, 3, 6])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.fork(src, dst)
        c.free(dst)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    kk, vv, tt = k[:6].clone(), v[:6].clone(), ts[:6].clone()
    with torch.cuda.graph(g):
        c.fork(src, dst)
        c.append(dst, off, kk, vv, tt)
    g.replay()
    m.fork([0, 1], [2, 3])
    m.append([2, 3], [0, 3, 6], kk.cpu(), vv.cpu(), tt.cpu())
    assert c.check_device_error() == OK
    same(c, m)
    c.free(dst)
    m.free([2, 3])
    kk.copy_(k[10:16])
    g.replay()
    m.fork([0, 1], [2, 3])
    m.append([2, 3], [0, 3, 6], kk.cpu(), vv.cpu(), tt.cpu())
    same(c, m)
    g.replay()                                          # the destinations are not empty now: refused, then appended again
    assert c.check_device_error() == BOUNDS
    m.append([2, 3], [0, 3, 6], kk.cpu(), vv.cpu(), tt.cpu())
    same(c, m)
    del g


def test_many_slots_and_pages():
    """More requests than a CTA has threads, and free pages far into the pool."""
    n, ps = 2500, 16
    c, m = make(6000, ps, 2 * n, 3, 8, torch.bfloat16)
    rng = np.random.default_rng(3)
    cnt = rng.integers(0, 2 * ps + 1, n)
    off = [0] + np.cumsum(cnt).tolist()
    src = rows_of(rng, off[-1], 8, torch.bfloat16)
    slots = rng.permutation(2 * n)[:n].tolist()
    c.append(i32(slots), i32(off), *(t.cuda() for t in src))
    assert c.check_device_error() == OK
    pages = [-(-int(x) // ps) for x in cnt]
    first = [0] + np.cumsum(pages).tolist()
    table = c.page_table.cpu().numpy()
    for i, s in enumerate(slots):
        assert table[s, :pages[i]].tolist() == list(range(first[i], first[i + 1])) and (table[s, pages[i]:] == -1).all()
    assert c.ref.cpu().tolist() == [1] * first[-1] + [0] * (6000 - first[-1])
    got = torch.cat([c.k[first[i]:first[i + 1]].reshape(-1, 8)[:int(cnt[i])] for i in range(n)]).cpu()
    assert torch.equal(got, src[0])
    odd = slots[1::2]
    c.free(i32(odd))
    assert c.check_device_error() == OK
    assert int(c.ref.sum()) == sum(pages[0::2]) and int(c.lens.sum()) == int(sum(cnt[0::2]))


def test_python_checks():
    c, m, (k, v, ts) = filled()
    s, off = i32([2]), i32([0, 4])
    with pytest.raises(ValueError):
        c.append(s.cpu(), off, k[:4], v[:4], ts[:4])
    with pytest.raises(ValueError):
        c.append(s, off, k[:4].float(), v[:4], ts[:4])
    with pytest.raises(ValueError):
        c.append(s, off, k[:4], v[:3], ts[:4])
    with pytest.raises(ValueError):
        c.append(s, off, k[:8:2], v[:4], ts[:4])
    with pytest.raises(ValueError):
        c.append(s, i32([0]), k[:4], v[:4], ts[:4])
    with pytest.raises(ValueError):
        c.append(s, off, k[:4, :32].contiguous(), v[:4], ts[:4])
    with pytest.raises(ValueError):
        c.fork(s, i32([3, 4]))
    with pytest.raises(ValueError):
        c.compact(s, i32([0]), i32([0]))
    with pytest.raises(ValueError):
        c.free(s.long())
    same(c, m)
