"""One workspace for several caches and for both the page operators and the scorer, in stream order:
no call depends on what another has left there."""
import numpy as np
import pytest
import torch

from test_gpu_cache import OK, i32, make, rows_of, same
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


def share(*objects):
    """All of them work in one buffer, the size of the largest one's workspace."""
    ws = torch.zeros(max(o.ws.numel() for o in objects), dtype=torch.uint8, device="cuda")
    for o in objects:
        o.ws, o._ws = ws, (ws.data_ptr(), ws.numel())
    return ws


def grown(case):
    """The case's cache after an append of 3 rows to slot 0 and a fork, and the scores over it."""
    g = torch.Generator().manual_seed(3)
    c, s = case.cache, case.scorer()
    kv = [torch.randn(3, case.D, generator=g).bfloat16().cuda() for _ in range(2)]
    ts = torch.tensor([5, 6, 7], dtype=torch.int64, device="cuda") + int(case.hts[0][-1])
    return c, s, kv, ts


def test_page_operators_and_scorer_share_a_workspace():
    def steps(shared):
        case = Case([40, 129, 300], [5, 70, 20], 2, 64, 16, seed=9)
        c, s, kv, ts = grown(case)
        if shared:
            share(c, s)
        out = []
        x = case.tensors()

        def score():
            out.append(s.score(*x, out=dict(y=torch.full_like(x[0], 7), o_pre=torch.full_like(x[0], 7))))
            assert s.check_device_error() == OK

        for _ in range(2):                              # after a page operator, and after the scorer itself
            c.append(i32([0]), i32([0, 1]), kv[0][:1], kv[1][:1], ts[:1])
            assert c.check_device_error() == OK
            score()
            score()
        c.fork(i32([0]), i32([3]))
        assert c.check_device_error() == OK
        score()
        c.free(i32([3]))
        assert c.check_device_error() == OK
        score()
        c.compact(i32([2, 1]), i32([0, 2, 4]), i32([5, 290, 0, 128]))
        assert c.check_device_error() == OK
        score()
        return out, c

    a, ca = steps(False)
    b, cb = steps(True)
    for x, y in zip(a, b):
        assert torch.equal(x["y"], y["y"]) and torch.equal(x["o_pre"], y["o_pre"])
    assert torch.equal(ca.lens, cb.lens) and torch.equal(ca.ref, cb.ref) and torch.equal(ca.page_table, cb.page_table)


def test_two_caches_share_a_workspace():
    """Caches of few and of many slots and pages, each call after one of the other."""
    rng = np.random.default_rng(2)
    pairs = [make(40, 16, 6, 4, 8, torch.bfloat16), make(400, 32, 130, 3, 16, torch.float32), make(70, 64, 40, 2, 8, torch.bfloat16)]
    share(*(c for c, _ in pairs))
    for step in range(4):
        for c, m in pairs:
            n = len(m.lens) // 2
            slots = list(range(n))
            off = [0] + np.cumsum(rng.integers(0, 9, n)).tolist()
            src = rows_of(rng, off[-1], c.row_elems, c.dtype)
            m.append(slots, off, *src)
            c.append(i32(slots), i32(off), *(t.cuda() for t in src))
            assert c.check_device_error() == OK
        for c, m in pairs:
            dst = list(range(len(m.lens) // 2, 2 * (len(m.lens) // 2)))
            src = rng.integers(0, len(m.lens) // 2, len(dst)).tolist()
            m.fork(src, dst)
            c.fork(i32(src), i32(dst))
            assert c.check_device_error() == OK
        for c, m in pairs:
            dst = list(range(len(m.lens) // 2, 2 * (len(m.lens) // 2)))
            keep = [r for s in dst for r in range(m.lens[s] // 2)]
            off = [0] + np.cumsum([m.lens[s] // 2 for s in dst]).tolist()
            m.compact(dst, off, keep)
            c.compact(i32(dst), i32(off), i32(keep))
            assert c.check_device_error() == OK
            same(c, m)
        for c, m in pairs:
            dst = list(range(len(m.lens) // 2, 2 * (len(m.lens) // 2)))
            m.free(dst)
            c.free(i32(dst))
            assert c.check_device_error() == OK
            same(c, m)


def test_workspace_need_not_be_clear():
    """Only the 256 bytes of the control block have to start at zero."""
    c, m = make(20, 16, 5, 4, 8, torch.bfloat16)
    case = Case([40, 129], [5, 70], 1, 128, 32, seed=11)
    want = case.run()
    s = case.scorer()
    for o in (c, s):
        o.ws[256:] = 0xff
    src = rows_of(np.random.default_rng(0), 50, 8, torch.bfloat16)
    m.append([0, 1], [0, 30, 50], *src)
    c.append(i32([0, 1]), i32([0, 30, 50]), *(t.cuda() for t in src))
    assert c.check_device_error() == OK
    c.ws[256:] = 0xff
    m.fork([0, 0], [2, 3])
    c.fork(i32([0, 0]), i32([2, 3]))
    assert c.check_device_error() == OK
    c.ws[256:] = 0xff
    m.compact([3, 0], [0, 2, 3], [0, 29, 5])
    c.compact(i32([3, 0]), i32([0, 2, 3]), i32([0, 29, 5]))
    assert c.check_device_error() == OK
    c.ws[256:] = 0xff
    m.free([2])
    c.free(i32([2]))
    assert c.check_device_error() == OK
    same(c, m)
    got = s.score(*case.tensors())
    assert s.check_device_error() == OK
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["o_pre"], want["o_pre"])


def test_trees_changed_in_place():
    """A scorer whose tensors get other trees, slots and rules, called and replayed, equals a new one."""
    rule = ([0, 4, 2], [30, 100, 5])
    case = Case([40, 129, 300], [6, 70, 20], 2, 64, 16, rule=rule, seed=9)
    s = case.scorer()
    x = case.tensors()
    first = s.score(*x)
    g, out = torch.cuda.CUDAGraph(), {n: torch.empty_like(t) for n, t in first.items()}
    with torch.cuda.graph(g):
        s.score(*x, out=out)
    other = Case([40, 129, 300], [25, 1, 70], 2, 64, 16, shape="chain", rule=([1, 0, 3], [400, 7, 64]), slots=[2, 0, 1], seed=9)
    for name, new in (("slots", other.slots), ("node_offsets", other.off), ("parent", other.parent), ("node_ts", other.node_ts),
                      ("n_sink", other.S), ("window", other.Wn)):
        getattr(s, name).copy_(torch.as_tensor(new))
    new = other.scorer()
    want = new.score(*x)
    g.replay()
    again = s.score(*x)
    assert s.check_device_error() == OK and new.check_device_error() == OK
    for n, t in want.items():
        assert torch.equal(again[n], t) and torch.equal(out[n], t), n
    assert not torch.equal(first["y"], want["y"])
    del g
