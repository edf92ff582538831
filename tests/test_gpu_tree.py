"""Tree scorer over the paged cache against the fp64 oracle: each node is the last row of a causal
(or window) layer over its history and its path.  The pool holds NaN wherever no row lives."""
import numpy as np
import pytest
import torch

import oracle
from hstu_jagged_pointwise_b200 import workloads as W
from parity import assert_bf16, bf16

pytestmark = pytest.mark.gpu
BIG = 2**31 - 1


def parents(rng, m, shape):
    if shape == "forest":
        return np.full(m, -1, np.int32)
    if shape == "chain":
        return np.arange(-1, m - 1, dtype=np.int32)
    return np.array([rng.integers(-1, i) if i else -1 for i in range(m)], np.int32)      # any earlier node, or none


class Case:
    """A cache of histories `lens` in pages of random places, trees of `nodes` nodes on them."""

    def __init__(self, lens, nodes, H, d, ps, shape="random", rule=None, seed=0, spare_slots=1, slots=None):
        from hstu_jagged_pointwise_b200 import ops
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        D, B = H * d, len(nodes)
        self.H, self.d, self.D, self.ps, self.lens, self.nodes = H, d, D, ps, lens, nodes
        self.alpha = float(max(lens) + 3)
        self.slots = np.asarray(range(B) if slots is None else slots, np.int32)
        self.S, self.Wn = (None, None) if rule is None else (np.asarray(rule[0], np.int32), np.asarray(rule[1], np.int32))
        need = [-(-n // ps) for n in lens]
        n_pages, max_pages = sum(need) + 2, max(max(need), 1) + 1
        c = self.cache = ops.PagedCache(n_pages, ps, len(lens) + spare_slots, max_pages, D)
        order = rng.permutation(n_pages)
        table = np.full((len(lens) + spare_slots, max_pages), -1, np.int32)
        k, v = torch.full((n_pages, ps, D), float("nan"), dtype=torch.bfloat16), torch.full((n_pages, ps, D), float("nan"), dtype=torch.bfloat16)
        ts = torch.full((n_pages, ps), -2**63, dtype=torch.int64)
        ref = torch.zeros(n_pages, dtype=torch.int32)
        self.hk, self.hv, self.hts, at = [], [], [], 0
        for s, n in enumerate(lens):
            pg = order[at:at + need[s]]
            at += need[s]
            table[s, :need[s]] = pg
            ref[pg] = 1
            self.hk.append(W.randn(gen, (n, D), torch.bfloat16))
            self.hv.append(W.randn(gen, (n, D), torch.bfloat16))
            self.hts.append(W.increasing_ts(rng, n))
            for r in range(n):
                k[pg[r // ps], r % ps], v[pg[r // ps], r % ps] = self.hk[s][r], self.hv[s][r]
                ts[pg[r // ps], r % ps] = int(self.hts[s][r])
        c.k.copy_(k), c.v.copy_(v), c.ts.copy_(ts), c.ref.copy_(ref)
        c.page_table.copy_(torch.as_tensor(table))
        c.lens[:len(lens)] = torch.as_tensor(np.asarray(lens, np.int32)).cuda()
        self.off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.T = int(self.off[-1])
        self.parent = np.concatenate([parents(rng, m, shape) for m in nodes] + [np.zeros(0, np.int32)]).astype(np.int32)
        last = [self.hts[s][-1] if lens[s] else W.T0 for s in self.slots]
        self.node_ts = np.concatenate([last[b] + rng.integers(1, 3601, m) for b, m in enumerate(nodes)] + [np.zeros(0, np.int64)]).astype(np.int64)
        self.q, self.k, self.v, self.u = (W.randn(gen, (self.T, D), torch.bfloat16) for _ in range(4))
        self.rab_pos, self.rab_time = W.rab_tables(gen)
        self.rab_pos, self.rab_time = self.rab_pos * 20, self.rab_time * 20       # biases that matter
        self.gamma, self.beta = W.ln_affine(gen, D, True)

    def scorer(self, **kw):
        from hstu_jagged_pointwise_b200 import ops
        t = lambda a: None if a is None else torch.as_tensor(a).cuda()
        args = dict(n_sink=t(self.S), window=t(self.Wn))
        args.update(kw)
        return ops.TreeScorer(self.cache, t(self.slots), t(self.off), t(self.parent), t(self.node_ts), self.H, self.d, self.alpha,
                              max(max(self.nodes), 1), **args)

    def tensors(self):
        return [x.cuda() for x in (self.q, self.k, self.v, self.u, self.rab_pos, self.rab_time, self.gamma, self.beta)]

    def run(self, **kw):
        s = self.scorer(**kw)
        out = s.score(*self.tensors())
        assert s.check_device_error() == 0
        return out

    def path(self, t, b):
        p, a = [], t - int(self.off[b])
        while a >= 0:
            p.append(int(self.off[b]) + a)
            a = int(self.parent[int(self.off[b]) + a])
        return p[::-1]

    def reference(self, rows):
        """Y of the listed nodes in fp64, and with bf16 tensor-core operands."""
        ys, ms = [], []
        for t in rows:
            b = int(np.searchsorted(self.off, t, side="right") - 1)
            s, path = int(self.slots[b]), self.path(t, b)
            k, v = torch.cat([self.hk[s], self.k[path]]), torch.cat([self.hv[s], self.v[path]])
            n = len(k)
            q = torch.zeros(n, self.D)
            q[-1] = self.q[t].float()
            ts = np.concatenate([self.hts[s], self.node_ts[path]])
            kind, ns, nr = oracle.MASK_CAUSAL, None, None
            if self.Wn is not None:
                kind, ns, nr = oracle.MASK_WINDOW, [self.S[b]], [self.Wn[b]]
            args = ([0, n], self.H, self.d, self.d, q, k.float(), v.float(), ts, self.rab_pos, self.rab_time, kind, ns, nr, self.alpha, [n - 1])
            ys.append(oracle.attn_fwd_raw(*args)[0])
            with oracle.bf16_operands():
                ms.append(oracle.attn_fwd_raw(*args)[0])
        return np.array(ys).reshape(-1, self.D), np.array(ms).reshape(-1, self.D)

    def check(self, out, rows=None):
        rows = list(range(self.T)) if rows is None else list(rows)
        y, m = self.reference(rows)
        u = oracle.f32(self.u)[rows]
        o = oracle.ln_mul_fwd(y, u, self.gamma, self.beta)[0]
        om = oracle.ln_mul_fwd(m, u, self.gamma, self.beta)[0]
        idx = torch.as_tensor(rows, dtype=torch.int64).cuda()
        assert_bf16(out["y"][idx], y, "y", bf16(m))
        assert_bf16(out["o_pre"][idx], o, "o_pre", bf16(om))


LENS = [0, 1, 15, 127, 128, 129, 300, 700]
NODES = [5, 1, 16, 17, 0, 33, 65, 3]


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_odd_histories_and_trees(ps, d):
    """Histories that end inside a page and a tile, none at all; trees of none to more than a group."""
    c = Case(LENS, NODES, 2, d, ps, seed=ps + d)
    c.check(c.run())


@pytest.mark.parametrize("shape", ["forest", "chain", "random"])
def test_tree_shapes(shape):
    c = Case([260, 40], [70, 130], 1, 128, 32, shape=shape, seed=5)
    out = c.run()
    c.check(out)


# sinks and windows: nothing visible, only sinks, only itself, a window that ends inside a tile, sinks
# that reach the window, both past the history, a gap of several tiles, a window shorter than the path
RULES = ([0, 4, 0, 3, 130, BIG, 20, 1], [0, 0, 1, 100, 60, 0, 64, 3])


@pytest.mark.parametrize("ps,d", [(16, 128), (64, 64), (128, 128)])
def test_window_with_sinks(ps, d):
    c = Case([300, 200, 257, 600, 300, 90, 900, 500], [9, 8, 7, 20, 30, 6, 40, 12], 2, d, ps, shape="random", rule=RULES, seed=ps)
    out = c.run()
    c.check(out)
    nothing = slice(int(c.off[0]), int(c.off[1]))
    assert torch.count_nonzero(out["y"][nothing]) == 0
    want = (c.beta * c.u[nothing].float()).to(torch.bfloat16)
    assert torch.equal(out["o_pre"][nothing].cpu(), want)


def test_rows_outside_the_window_are_never_used():
    """Evicted pages (-1 in the table) and NaN in every row that no node may see."""
    lens, S, Wn = [1000, 700], [5, 40], [150, 200]
    c = Case(lens, [20, 9], 1, 128, 16, shape="forest", rule=(S, Wn), seed=3)
    table = c.cache.page_table.cpu().numpy()
    k, v, ts = c.cache.k.cpu(), c.cache.v.cpu(), c.cache.ts.cpu()
    for s, n in enumerate(lens):
        for r in range(S[s], n - Wn[s] + 1):
            k[table[s, r // 16], r % 16] = float("nan")
            v[table[s, r // 16], r % 16] = float("inf")
            ts[table[s, r // 16], r % 16] = 2**63 - 1
        for e in range(-(-S[s] // 16), (n - Wn[s] + 1) // 16):
            table[s, e] = -1
    c.cache.k.copy_(k), c.cache.v.copy_(v), c.cache.ts.copy_(ts), c.cache.page_table.copy_(torch.as_tensor(table))
    c.check(c.run())


def test_no_rule_equals_a_window_past_everything_bit_for_bit():
    c = Case([300, 65], [30, 4], 2, 128, 64, seed=8)
    a = c.run()
    t = lambda x: torch.full((2,), x, dtype=torch.int32, device="cuda")
    b = c.run(n_sink=t(0), window=t(BIG))
    e = c.run(n_sink=t(BIG), window=t(0))
    for n in ("y", "o_pre"):
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], e[n])


def test_long_history_split_over_the_gpu():
    """One node over 40,000 rows: the history is cut into parts that add up; twice the same bits."""
    c = Case([40000], [1], 2, 128, 128, seed=2)
    s = c.scorer()
    a = s.score(*c.tensors())
    b = s.score(*c.tensors())
    assert s.check_device_error() == 0
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["o_pre"], b["o_pre"])
    c.check(a)


def test_extreme_times():
    c = Case([200, 130], [40, 20], 1, 64, 32, seed=4)
    c.hts[0] = np.sort(np.random.default_rng(0).integers(-2**62, 2**62, 200))
    ts, table = c.cache.ts.cpu(), c.cache.page_table.cpu().numpy()
    for r in range(200):
        ts[table[0, r // 32], r % 32] = int(c.hts[0][r])
    c.cache.ts.copy_(ts)
    c.node_ts[:20] = 2**63 - 1 - np.arange(20)
    c.node_ts[20:40] = -2**63 + np.arange(20)
    c.check(c.run())


def test_one_node_trees_are_the_mfalcon_scorer():
    """The same users through ops.MFalcon: equal up to the order of the sums and one rounding of Y."""
    from hstu_jagged_pointwise_b200 import ops
    c = Case([300, 1, 0, 150], [40, 3, 7, 130], 2, 128, 64, shape="forest", seed=6)
    out = c.run()
    cu = lambda x, dt: torch.as_tensor(np.asarray(x, dt)).cuda()
    ho = np.concatenate([[0], np.cumsum(c.lens)])
    m = ops.MFalcon(cu(ho, np.int32), cu(np.concatenate(c.hts), np.int64), cu(c.off, np.int32), cu(c.node_ts, np.int64), 2, 128, c.alpha, 256,
                    300, 130)
    q, k, v, u, rp, rt, g, b = c.tensors()
    ref = m.score(torch.cat(c.hk).cuda(), torch.cat(c.hv).cuda(), q, k, v, u, rp, rt, g, b)
    # both hold bf16 P (2^-9 a term, at random) and round Y once (2^-9): within 5e-3 of one another
    for n in ("y", "o_pre"):
        e = (out[n].float() - ref[n].float()).norm() / ref[n].float().norm()
        assert float(e) <= 5e-3, (n, float(e))
    c.check(out)


def test_shared_slots_and_wide_rows():
    """Three trees on one history; 64 heads of 128."""
    c = Case([200, 90], [3, 20, 1, 2], 2, 64, 32, seed=9, slots=[0, 1, 0, 0])
    c.check(c.run())
    w = Case([150], [3], 64, 128, 64, seed=9)
    w.check(w.run())


def test_cache_then_scorer_run_as_one():
    """Serving a step: a history is appended, forked into beams, each beam grows by a node of the last
    tree, and the next node is scored.  It equals scoring the path as one tree."""
    from hstu_jagged_pointwise_b200 import ops
    c = Case([150], [4], 2, 128, 16, shape="chain", seed=10)
    whole = c.run()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache = ops.PagedCache(40, 16, 4, 12, c.D)
    hts = torch.as_tensor(c.hts[0]).cuda()
    cache.append(i32(0), i32(0, 100), c.hk[0][:100].cuda(), c.hv[0][:100].cuda(), hts[:100])
    cache.append(i32(0), i32(0, 50), c.hk[0][100:].cuda(), c.hv[0][100:].cuda(), hts[100:])
    cache.fork(i32(0, 0), i32(1, 2))
    k, v, nts = c.k.cuda(), c.v.cuda(), torch.as_tensor(c.node_ts).cuda()
    cache.append(i32(1, 2), i32(0, 2, 5), k, v, nts, rows=i32(0, 1, 0, 1, 2))
    q, _, _, u, rp, rt, g, b = c.tensors()
    for slot, node in ((1, 2), (2, 3)):
        t = ops.TreeScorer(cache, i32(slot), i32(0, 1), i32(-1), nts[node:node + 1].clone(), 2, 128, c.alpha, 1)
        one = lambda x: x[node:node + 1].clone()
        out = t.score(one(q), one(k), one(v), one(u), rp, rt, g, b)
        assert t.check_device_error() == 0
        # the path's terms move from fp32 into the bf16 product: 2^-9 of a few of 150 terms, and two roundings
        for n in ("y", "o_pre"):
            e = (out[n].float() - whole[n][node:node + 1].float()).norm() / whole[n][node:node + 1].float().norm()
            assert float(e) <= 5e-3, (n, float(e))
    # the history itself is unchanged, and cutting it to its sinks and window changes nothing the window sees
    assert cache.lens.tolist() == [150, 152, 153, 0]
    keep = list(range(4)) + list(range(50, 150))
    cache.fork(i32(0), i32(3))
    cache.compact(i32(3), i32(0, len(keep)), i32(*keep))
    assert cache.check_device_error() == 0 and cache.lens.tolist() == [150, 152, 153, 104]


def test_flagged_calls_write_nothing_and_the_next_is_clean():
    c = Case([300, 200], [20, 9], 1, 64, 64, rule=([4, 2], [100, 50]), seed=1)
    good = c.run()
    s = c.scorer()
    args = c.tensors()

    def refused(tensor, at, value):
        keep = tensor[at].clone()
        tensor[at] = value
        out = dict(y=torch.full_like(good["y"], 7.0), o_pre=torch.full_like(good["y"], 7.0))
        s.score(*args, out=out)
        assert s.check_device_error() == -5, (at, value)
        assert bool((out["y"] == 7.0).all()) and bool((out["o_pre"] == 7.0).all())
        tensor[at] = keep

    for value in (-1, 3, BIG):
        refused(s.slots, 1, value)
    for value in (-2, 5, BIG):
        refused(s.parent, 5, value)
    refused(s.node_offsets, 0, 1)
    refused(s.node_offsets, 1, -1)
    refused(s.node_offsets, 1, 25)                    # a tree past max_nodes
    refused(s.node_offsets, 2, 28)
    refused(s.window, 0, -1)
    refused(s.n_sink, 1, -3)
    refused(c.cache.lens, 0, -1)
    refused(c.cache.lens, 0, 10**6)
    refused(c.cache.page_table, (0, 4), -1)           # the window's last page
    refused(c.cache.page_table, (0, 0), 10**6)        # the sinks' page
    again = s.score(*args)
    assert s.check_device_error() == 0
    assert torch.equal(again["y"], good["y"]) and torch.equal(again["o_pre"], good["o_pre"])


def test_captured_replayed_streams_and_growth():
    """One captured call replayed while the history grows; two scorers at once on two streams."""
    c = Case([100, 40], [6, 6], 2, 128, 32, seed=12)
    s = c.scorer()
    args = c.tensors()
    first = s.score(*args)
    out = {n: torch.zeros_like(first[n]) for n in first}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.score(*args, out=out)
    g.replay()
    assert torch.equal(out["y"], first["y"])
    extra = 7
    gen = torch.Generator().manual_seed(1)
    k, v = W.randn(gen, (extra, c.D), torch.bfloat16), W.randn(gen, (extra, c.D), torch.bfloat16)
    ts = c.hts[1][-1] + 1 + np.arange(extra)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    c.cache.append(i32(1), i32(0, extra), k.cuda(), v.cuda(), torch.as_tensor(ts).cuda())
    g.replay()
    assert s.check_device_error() == 0 and c.cache.check_device_error() == 0
    c.hk[1], c.hv[1], c.hts[1] = torch.cat([c.hk[1], k]), torch.cat([c.hv[1], v]), np.concatenate([c.hts[1], ts])
    c.check(out)
    other = c.scorer()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for st, sc in zip(streams, (s, other)):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(5):
                r = sc.score(*args)
            outs.append(r)
    torch.cuda.synchronize()
    assert torch.equal(outs[0]["y"], out["y"]) and torch.equal(outs[1]["o_pre"], out["o_pre"])
    del g


def test_timeout_is_reported_and_the_context_stays_usable():
    from hstu_jagged_pointwise_b200 import capi
    c = Case([300, 200], [20, 9], 1, 128, 64, seed=1)
    s = c.scorer()
    args = c.tensors()
    good = s.score(*args)
    out = dict(y=torch.full_like(good["y"], 7.0), o_pre=torch.full_like(good["y"], 7.0))
    with capi.wait_fault(2_000_000):
        s.score(*args, out=out)
        torch.cuda.synchronize()
    assert s.check_device_error() == -4
    assert bool((out["o_pre"] == 7.0).all())
    again = s.score(*args)
    assert s.check_device_error() == 0 and torch.equal(again["y"], good["y"])


def test_no_trees_no_nodes():
    from hstu_jagged_pointwise_b200 import ops
    c = Case([50], [3], 1, 64, 16, seed=1)
    e32, e64 = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    tables = c.tensors()[4:]
    for slots, off in ((e32, torch.zeros(1, dtype=torch.int32, device="cuda")), (torch.zeros(2, dtype=torch.int32, device="cuda"),
                                                                                 torch.zeros(3, dtype=torch.int32, device="cuda"))):
        s = ops.TreeScorer(c.cache, slots, off, e32, e64, 1, 64, 1.0, 0)
        out = s.score(x, x, x, x, *tables)
        assert out["y"].shape == (0, 64) and s.check_device_error() == 0


def test_python_checks():
    from hstu_jagged_pointwise_b200 import ops
    c = Case([50, 20], [3, 2], 1, 64, 16, rule=([0, 0], [5, 5]), seed=1)
    s = c.scorer()
    q, k, v, u, rp, rt, g, b = c.tensors()
    for bad in ((q.float(), k, v, u, rp, rt, g, b), (q[:4], k, v, u, rp, rt, g, b), (q, k, v, u, rp[:5], rt, g, b), (q, k, v, u, rp, rt, g.double(), b),
                (q.cpu(), k, v, u, rp, rt, g, b), (q, k.t().contiguous().t(), v, u, rp, rt, g, b)):
        with pytest.raises(ValueError):
            s.score(*bad)
    with pytest.raises(ValueError):
        c.scorer(window=None)
    with pytest.raises(ValueError):
        c.scorer(n_sink=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        s.score(q, k, v, u, rp, rt, g, b, out=dict(y=q.float(), o_pre=q))
    with pytest.raises(Exception):
        ops.TreeScorer(c.cache, s.slots, s.node_offsets, s.parent, s.node_ts, 2, 64, 1.0, 3)      # H*d is not the cache's


def test_pool_past_32_bit_offsets():
    """A pool of 5 GB for keys and as much for values, whose low pages are taken: pages at its end are
    filled, forked, cut and scored."""
    from hstu_jagged_pointwise_b200 import ops
    n_pages, ps, H, d = 20500, 128, 8, 128
    D = H * d
    cache = ops.PagedCache(n_pages, ps, 3, 8, D)
    assert cache.k.numel() * 2 > 2**32
    cache.ref[:20480] = 1
    c = Case([300], [3], H, d, 64, seed=21)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    hk, hv, ts = c.hk[0].cuda(), c.hv[0].cuda(), torch.as_tensor(c.hts[0]).cuda()
    cache.append(i32(0), i32(0, 300), hk, hv, ts)
    cache.fork(i32(0), i32(1))
    cache.compact(i32(1), i32(0, 300), torch.arange(300, dtype=torch.int32, device="cuda"))
    assert cache.check_device_error() == 0
    assert cache.page_table[0, :3].tolist() == [20480, 20481, 20482] and cache.page_table[1, :3].tolist() == [20483, 20484, 20485]
    assert torch.equal(cache.k[20483:20486].reshape(-1, D)[:300], hk) and torch.equal(cache.v[20480:20483].reshape(-1, D)[:300], hv)
    for slot in (0, 1):
        s = ops.TreeScorer(cache, i32(slot), torch.as_tensor(c.off).cuda(), torch.as_tensor(c.parent).cuda(), torch.as_tensor(c.node_ts).cuda(),
                           H, d, c.alpha, 3)
        out = s.score(*c.tensors())
        assert s.check_device_error() == 0
        c.check(out)


def test_rows_and_tables_of_other_callers_are_left_alone():
    """Slots that a call does not name, pages of others and rows behind the last keep their bits."""
    c = Case([70, 33, 100], [4, 2, 3], 1, 64, 32, seed=14)
    before = [t.clone() for t in (c.cache.k, c.cache.v, c.cache.ts, c.cache.page_table, c.cache.lens, c.cache.ref)]
    out = dict(y=torch.full((c.T + 5, c.D), 9.0, dtype=torch.bfloat16, device="cuda"), o_pre=torch.full((c.T + 5, c.D), 9.0, dtype=torch.bfloat16, device="cuda"))
    s = c.scorer()
    s.score(*c.tensors(), out={n: t[:c.T] for n, t in out.items()})
    assert s.check_device_error() == 0
    for t in out.values():
        assert bool((t[c.T:] == 9.0).all())
    after = (c.cache.k, c.cache.v, c.cache.ts, c.cache.page_table, c.cache.lens, c.cache.ref)
    for a, b in zip(before, after):
        assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a, b.view(torch.int16) if b.dtype == torch.bfloat16 else b)


@pytest.mark.parametrize("B,m,lo,hi,d,ps", [(64, 1, 4096, 8192, 128, 128), (48, 1, 4000, 8000, 64, 64), (40, 33, 2000, 4096, 128, 32),
                                            (40, 130, 1000, 3000, 128, 128), (40, 200, 1000, 3000, 64, 16)])
def test_many_items_an_sm(B, m, lo, hi, d, ps):
    """Forests over histories that end inside a tile, with NaN behind their last rows, so many that each
    SM works through a dozen items with HBM busy: the same bits each time, and every head of every node
    near the sum in 64 bits.  The rounding of P and of Y to bf16 are up to 2^-8 of a term or entry each,
    tanh's error 2^-11: independent, they are under 2^-7 of a head's norm together, and twice that is
    allowed; 32 keys of 8192 left out are 2^-4 of it."""
    from hstu_jagged_pointwise_b200 import ops
    rng, g, H = np.random.default_rng(B + m), torch.Generator(device="cuda").manual_seed(m), 4
    lens = rng.integers(lo, hi + 1, B)
    lens[:3] = [lo, hi, hi // 128 * 128]
    D, per = H * d, -(-hi // ps)
    order = torch.as_tensor(rng.permutation(B * per)).cuda()
    c = ops.PagedCache(B * per, ps, B, per, D)
    c.k.copy_(torch.randn(B * per, ps, D, generator=g, device="cuda"))
    c.v.copy_(torch.randn(B * per, ps, D, generator=g, device="cuda"))
    hts = W.T0 + torch.cumsum(torch.randint(1, 7200, (B, per * ps), generator=g, device="cuda"), 1)
    table = order.view(B, per)
    c.ts[table] = hts.view(B, per, ps)
    for b, n in enumerate(lens):
        last = table[b, n // ps:]
        if len(last):
            c.k[last[0], n % ps:], c.v[last[0], n % ps:] = float("nan"), float("nan")
    c.page_table.copy_(table)
    c.lens.copy_(torch.as_tensor(lens))
    T = B * m
    q, k, v, u = (torch.randn(T, D, generator=g, device="cuda").bfloat16() for _ in range(4))
    rp, rt = torch.randn(511, generator=g, device="cuda"), torch.randn(64, generator=g, device="cuda")
    ga, be = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")
    node_ts = (hts[torch.arange(B), torch.as_tensor(lens).long() - 1] + 1).repeat_interleave(m)
    s = ops.TreeScorer(c, i32(np.arange(B)), i32(np.arange(B + 1) * m), i32(np.full(T, -1)), node_ts, H, d, float(hi), m)
    outs = [s.score(q, k, v, u, rp, rt, ga, be) for _ in range(8)]
    assert s.check_device_error() == 0
    for o in outs[1:]:
        assert torch.equal(o["y"], outs[0]["y"]) and torch.equal(o["o_pre"], outs[0]["o_pre"])
    for b in range(B):
        n, at = int(lens[b]), slice(b * m, (b + 1) * m)
        K, V = (x[table[b]].view(-1, H, d)[:n].double() for x in (c.k, c.v))
        qb, kb, vb = (x[at].view(m, H, d).double() for x in (q, k, v))
        pidx = torch.clamp(torch.arange(n, device="cuda") - n, min=-255) + 255
        bucket = torch.as_tensor([int(x).bit_length() for x in (node_ts[b * m] - hts[b, :n]).tolist()], device="cuda")
        z = torch.einsum("mhd,jhd->mhj", qb, K) + (rp[pidx].double() + rt[bucket].double())
        zs = (qb * kb).sum(-1) + rp[255].double() + rt[0].double()
        y = (torch.einsum("mhj,jhd->mhd", z * torch.sigmoid(z), V) + (zs * torch.sigmoid(zs))[..., None] * vb) / float(hi)
        e = (outs[0]["y"][at].view(m, H, d).double() - y).norm(dim=-1) / y.norm(dim=-1)
        assert e.max().item() <= 2**-6, (b, n, e.max().item())
