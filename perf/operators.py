"""What is measured of the windowed attention, the paged history cache and the tree scorer.

Three groups of operators of jagged HSTU pointwise attention (no softmax: Y = sum mask * SiLU(z) v / alpha):
  window_fwd, window_bwd   the attention layer whose rows see the last W tokens and the first S ("sinks"), and its gradient
  refill, beams, compact   the page operators of a user-history cache: free + append, fork + append + free, fork + compact + free
  tree                     a tree of candidate tokens (each sees the cached history, its ancestors and itself) scored over the pages

Where `own` is false `run` computes them with elementary torch operations on padded tensors, in 32 bits
(64 for the bias gradients' long sums), rounded once at the end."""
import random
from types import SimpleNamespace

import numpy as np
import torch

own = False

P, NB, EPS = 256, 64, 1e-5            # rab_pos has 2P-1 entries, rab_time NB
T0, GAP = 1_700_000_000, 3600.0       # first event, mean gap in seconds
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest training batch of this repository's tests, in fp32: latency of a few short rows
        dict(name="window_fwd tiny f32", op="window_fwd", n=4, lo=17, hi=255, mix=1, H=2, d=32, dtype="f32", sinks=4, window=32),
        # a training batch after Stochastic Length (rows of at most 776 events)
        dict(name="window_fwd sl-batch", op="window_fwd", n=64, lo=16, hi=776, mix=2, H=4, d=128, dtype="bf16", sinks=4, window=256),
        # long histories: most key tiles lie outside the window
        dict(name="window_fwd long", op="window_fwd", n=8, lo=1024, hi=4096, mix=3, H=8, d=128, dtype="bf16", sinks=8, window=512),
        # a small odd batch of narrow heads, rows of one token among them
        dict(name="window_bwd odd d64", op="window_bwd", n=12, lo=1, hi=301, mix=4, H=3, d=64, dtype="bf16", sinks=3, window=50),
        # the gradient of long histories
        dict(name="window_bwd long", op="window_bwd", n=8, lo=1024, hi=4096, mix=5, H=4, d=128, dtype="bf16", sinks=4, window=512),
        # histories of a batch of users written into freshly released pages
        dict(name="refill 64x2048", op="refill", n=64, lo=1024, hi=2048, mix=6, H=4, d=128, dtype="bf16", page=64),
        # a step of a beam search: four beams a user, three new events each, the shared last page copied first
        dict(name="beams 64x4", op="beams", n=64, lo=200, hi=2048, mix=7, H=4, d=128, dtype="bf16", page=32, beams=4, add=3),
        # a cached history cut down to 776 of its events
        dict(name="compact 64 to 776", op="compact", n=64, lo=1024, hi=2048, mix=8, H=4, d=128, dtype="bf16", page=64, keep=776),
        # one user, one new event: latency
        dict(name="tree one token", op="tree", n=1, lo=2048, hi=2048, mix=9, H=4, d=128, page=64, nlo=1, nhi=1, depth=1, sinks=0, window=0),
        # a batch of single events over long histories: the cache is read once
        dict(name="tree 64 tokens", op="tree", n=64, lo=4096, hi=8192, mix=10, H=4, d=128, page=128, nlo=1, nhi=1, depth=1, sinks=0, window=0),
        # trees of some dozens of candidates, four levels deep, under a window with sinks, small pages, narrow heads
        dict(name="tree window d64", op="tree", n=48, lo=0, hi=2048, mix=11, H=6, d=64, page=16, nlo=5, nhi=61, depth=4, sinks=4, window=700),
        # ranking: a thousand candidates a user
        dict(name="tree ranking", op="tree", n=32, lo=1500, hi=2048, mix=12, H=4, d=128, page=128, nlo=900, nhi=1024, depth=2, sinks=0, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["window_fwd", "window_fwd", "window_bwd", "refill", "beams", "compact", "tree", "tree", "tree"])
    mix = rng.randrange(1 << 20)
    if op in ("window_fwd", "window_bwd"):
        f32 = op == "window_fwd" and rng.random() < 0.25
        hi = _log(rng, 16, 300 if f32 else 4096)
        n = max(1, min(_log(rng, 1, 64), 18_000 // hi))
        d = rng.choice([32, 64, 128]) if f32 else rng.choice([64, 128])
        return dict(op=op, n=n, lo=rng.randint(0, hi), hi=hi, mix=mix, H=rng.randint(1, 4), d=d, dtype="f32" if f32 else "bf16",
                    sinks=rng.choice([0, 1, 4, 17, 130]), window=_log(rng, 1, 1024))
    H, d = rng.randint(1, 4), rng.choice([64, 128])
    if op in ("refill", "beams", "compact"):
        hi = _log(rng, 30, 2048)
        c = dict(op=op, n=_log(rng, 1, 64), lo=rng.randint(0, hi), hi=hi, mix=mix, H=H, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]),
                 page=rng.choice([16, 32, 64, 128]))
        if c["dtype"] == "f32":
            c["H"] = min(H, 2)
        if op == "beams":
            c.update(beams=rng.randint(1, 4), add=rng.randint(1, 9))
        if op == "compact":
            c.update(keep=rng.randint(1, 776))
        return c
    hi = _log(rng, 16, 8192)
    nhi = _log(rng, 1, 900)
    n = max(1, min(_log(rng, 1, 64), 300_000 // hi, 30_000_000 // (hi * nhi), 24_000 // nhi))
    return dict(op="tree", n=n, lo=rng.randint(0, hi), hi=hi, mix=mix, H=H, d=d, page=rng.choice([16, 32, 64, 128]), nlo=rng.randint(0, nhi),
                nhi=nhi, depth=min(nhi, rng.randint(1, 8)), sinks=rng.choice([0, 0, 1, 4, 130]), window=rng.choice([0, 0, _log(rng, 1, 4096)]))


# Sizes follow from the case alone.

def _lens(c, lo="lo", hi="hi", salt=0):
    r = random.Random(c["mix"] * 7 + salt)
    v = [r.randint(c[lo], c[hi]) for _ in range(c["n"])]
    v[r.randrange(c["n"])] = c[hi]
    return v


def _rules(c):
    """Sinks and window of each row: around the case's."""
    r = random.Random(c["mix"] * 7 + 1)
    return ([max(0, c["sinks"] - r.randrange(3)) for _ in range(c["n"])],
            [max(1, c["window"] - r.randrange(1 + c["window"] // 8)) for _ in range(c["n"])])


def _offsets(lens):
    return [0] + np.cumsum(lens).tolist()


def _levels(c, m):
    """Depth of each of m nodes: as many on each level as on any other."""
    return np.arange(m) * min(c["depth"], m) // max(m, 1)


def _parents(c, nodes, rng):
    """Tree of each user: level by level, each node under a random node of the level above, -1 at the first level."""
    out = []
    for m in nodes:
        lev = _levels(c, m)
        first = np.searchsorted(lev, lev)                 # first node of the own level
        prev = np.searchsorted(lev, lev - 1)              # and of the level above
        pick = prev + np.floor(rng.random_sample(m) * np.maximum(first - prev, 1)).astype(np.int64)
        out.append(np.where(lev > 0, pick, -1))
    return np.concatenate(out).astype(np.int32) if out else np.zeros(0, np.int32)


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _times(g, shape):
    """Increasing event times along the last axis."""
    gaps = 1 + torch.empty(shape, device="cuda").exponential_(1.0 / GAP, generator=g).floor().to(torch.int64)
    return T0 + torch.cumsum(gaps, -1)


def _tables(g, D):
    return dict(rab_pos=_randn(g, 2 * P - 1, scale=0.02), rab_time=_randn(g, NB, scale=0.02), gamma=1 + _randn(g, D, scale=0.1),
                beta=_randn(g, D, scale=0.1))


def _pages_of(lens, page):
    return [-(-n // page) for n in lens]


def _pool(c, g, dtype, n_slots, lens, spare, seed):
    """A cache whose first slots hold `lens` rows in pages of random order, `spare` pages free."""
    page, D = c["page"], c["H"] * c["d"]
    held = _pages_of(lens, page)
    n_pages, max_pages = max(sum(held) + spare, 1), max(-(-(c["hi"] + c.get("add", 0)) // page), 1)
    if own:
        from hstu_jagged_pointwise_b200 import ops
        m = ops.PagedCache(n_pages, page, n_slots, max_pages, D, dtype)
    else:
        m = SimpleNamespace(k=torch.zeros(n_pages, page, D, dtype=dtype, device="cuda"), v=torch.zeros(n_pages, page, D, dtype=dtype, device="cuda"),
                            ts=torch.zeros(n_pages, page, dtype=torch.int64, device="cuda"), lens=_i32([0] * n_slots), ref=_i32([0] * n_pages),
                            page_table=torch.full((n_slots, max_pages), -1, dtype=torch.int32, device="cuda"))
    order = np.random.RandomState(seed).permutation(n_pages)
    table, ref, at = np.full((n_slots, max_pages), -1, np.int32), np.zeros(n_pages, np.int32), 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        ref[order[at:at + h]] = 1
        at += h
    m.k.copy_(torch.randn(n_pages, page, D, generator=g, device="cuda"))
    m.v.copy_(torch.randn(n_pages, page, D, generator=g, device="cuda"))
    m.page_table.copy_(torch.from_numpy(table))
    m.ref.copy_(torch.from_numpy(ref))
    m.lens.copy_(_i32(list(lens) + [0] * (n_slots - len(lens))))
    t = _times(g, (n_slots, max_pages * page))           # row r of slot b gets time t[b, r]
    for b, h in enumerate(held):
        if h:
            m.ts[m.page_table[b, :h].long()] = t[b, :h * page].view(h, page)
    return m, t


def prepare(case, seed):
    c, g = case, _gen(seed)
    D, n = c["H"] * c["d"], c["n"]
    dtype = DTYPES[c.get("dtype", "bf16")]
    lens = _lens(c)
    s = SimpleNamespace(case=c, op=c["op"], H=c["H"], d=c["d"], n=n, lens=lens)
    if s.op in ("window_fwd", "window_bwd"):
        T = sum(lens)
        s.T, s.longest, s.alpha, s.dtype = T, max(max(lens), 1), float(max(max(lens), 1)), dtype
        s.off = _i32(_offsets(lens))
        s.ts = torch.cat([_times(g, (m,)) for m in lens])
        s.q, s.k, s.v, s.u = (_randn(g, T, D, dtype=dtype) for _ in range(4))
        s.sinks, s.window = map(_i32, _rules(c))
        vars(s).update(_tables(g, D))
        if s.op == "window_bwd":
            s.dy = _randn(g, T, D, dtype=dtype)
        if own:
            from hstu_jagged_pointwise_b200 import ops
            s.layer = ops.Layer(s.off, s.ts, s.H, s.d, dtype, s.alpha, s.longest, mask_kind="window", n_static=s.sinks, n_realtime=s.window)
        return s
    if s.op == "tree":
        nodes = _lens(c, "nlo", "nhi", 2)
        s.m, t = _pool(c, g, dtype, n, lens, 3, seed)
        T = sum(nodes)
        s.T, s.nodes, s.alpha = T, max(max(nodes), 1), float(c["hi"] + c["depth"])
        s.slots, s.off = torch.arange(n, dtype=torch.int32, device="cuda"), _i32(_offsets(nodes))
        s.parent = torch.from_numpy(_parents(c, nodes, np.random.RandomState(seed))).cuda()
        user = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(nodes, device="cuda"), output_size=T)
        last = t[torch.arange(n, device="cuda"), torch.clamp(s.m.lens[:n].long() - 1, min=0)]
        s.node_ts = last[user] + 1 + (torch.rand(T, generator=g, device="cuda") * GAP).to(torch.int64)
        s.q, s.k, s.v, s.u = (_randn(g, T, D, dtype=dtype) for _ in range(4))
        s.sinks = s.window = None
        if c["window"]:
            s.sinks, s.window = map(_i32, _rules(c))
        vars(s).update(_tables(g, D))
        if own:
            from hstu_jagged_pointwise_b200 import ops
            s.scorer = ops.TreeScorer(s.m, s.slots, s.off, s.parent, s.node_ts, s.H, s.d, s.alpha, s.nodes, n_sink=s.sinks, window=s.window)
        return s
    if s.op == "refill":
        s.m, _ = _pool(c, g, dtype, n, lens, 5, seed)
        s.slots, s.off, s.T = torch.arange(n, dtype=torch.int32, device="cuda"), _i32(_offsets(lens)), sum(lens)
    elif s.op == "beams":
        K = c["beams"]
        fresh = -(-c["add"] // c["page"]) + 1             # pages a beam can need: its new rows' and the copy of the shared one
        s.m, _ = _pool(c, g, dtype, n * (1 + K), lens, n * K * fresh, seed)
        s.src = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(K)
        s.slots = torch.arange(n, n * (1 + K), dtype=torch.int32, device="cuda")
        s.off, s.T = _i32(_offsets([c["add"]] * (n * K))), n * K * c["add"]
    else:
        kept = [min(c["keep"], m) for m in lens]
        s.m, _ = _pool(c, g, dtype, 2 * n, lens, sum(_pages_of(kept, c["page"])), seed)
        s.src, s.slots = torch.arange(n, dtype=torch.int32, device="cuda"), torch.arange(n, 2 * n, dtype=torch.int32, device="cuda")
        r = np.random.RandomState(seed)
        idx = [np.sort(r.permutation(m)[:j]) for m, j in zip(lens, kept)]
        s.keep_off, s.keep, s.T = _i32(_offsets(kept)), torch.from_numpy(np.concatenate(idx).astype(np.int32)).cuda(), sum(kept)
        return s
    s.k, s.v, s.ts = _randn(g, s.T, D, dtype=dtype), _randn(g, s.T, D, dtype=dtype), _times(g, (s.T,))
    return s


# ----------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if s.op == "window_fwd":
        if own:
            f = s.layer.forward(s.q, s.k, s.v, s.u, s.rab_pos, s.rab_time, s.gamma, s.beta)
            return dict(y=f["y"], o_pre=f["o_pre"])
        return plain_window_fwd(s)
    if s.op == "window_bwd":
        if own:
            return s.layer.backward_from_dy(s.q, s.k, s.v, s.rab_pos, s.rab_time, s.dy)
        return plain_window_bwd(s)
    if s.op == "tree":
        if own:
            return s.scorer.score(s.q, s.k, s.v, s.u, s.rab_pos, s.rab_time, s.gamma, s.beta)
        return plain_tree(s)
    m = s.m
    if s.op == "refill":
        if own:
            m.free(s.slots)
            m.append(s.slots, s.off, s.k, s.v, s.ts)
        else:
            plain_free(m, s.slots)
            plain_append(m, s.slots, s.off, s.T, s.k, s.v, s.ts)
        return _cache_out(m)
    if s.op == "beams":
        if own:
            m.fork(s.src, s.slots)
            m.append(s.slots, s.off, s.k, s.v, s.ts)
            out = _tables_out(m)
            m.free(s.slots)
        else:
            plain_fork(m, s.src, s.slots)
            plain_append(m, s.slots, s.off, s.T, s.k, s.v, s.ts)
            out = _tables_out(m)
            plain_free(m, s.slots)
        return {**_cache_out(m), "grown": out}
    if own:
        m.fork(s.src, s.slots)
        m.compact(s.slots, s.keep_off, s.keep)
        out = _tables_out(m)
        m.free(s.slots)
    else:
        plain_fork(m, s.src, s.slots)
        plain_compact(m, s.slots, s.keep_off, s.keep)
        out = _tables_out(m)
        plain_free(m, s.slots)
    return {**_cache_out(m), "grown": out}


def _cache_out(m):
    return dict(k=m.k, v=m.v, ts=m.ts, page_table=m.page_table, lens=m.lens, ref=m.ref)


def _tables_out(m):
    """The tables between the calls of one pass (the later calls change them in place)."""
    return dict(page_table=m.page_table.clone(), lens=m.lens.clone(), ref=m.ref.clone())


# ----------------------------------------------------------------------------- plain forms: attention

def _padded(off, n, longest):
    """Row index [n, longest] of each padded position, and which are real."""
    at = torch.arange(longest, device="cuda")
    ok = at[None] < (off[1:] - off[:-1])[:, None]
    return torch.where(ok, off[:-1, None].long() + at[None], 0), ok


def _heads(x, idx, H, d):
    """[n, H, longest, d] in 32 bits from rows x[idx]."""
    return x[idx].float().view(*idx.shape, H, d).transpose(1, 2)


def _bucket(ti, tj):
    """min(NB-1, bit length of |ti - tj|), by comparison with the powers of two."""
    powers = torch.tensor([1 << e for e in range(63)], dtype=torch.int64, device="cuda")
    return torch.clamp(torch.bucketize((ti - tj).abs(), powers, right=True), max=NB - 1)


def _norm_mul(s, y, u):
    mu = y.mean(-1, keepdim=True)
    var = ((y - mu) ** 2).mean(-1, keepdim=True)
    return ((y - mu) * torch.rsqrt(var + EPS) * s.gamma + s.beta) * u


def _window_scores(s):
    idx, ok = _padded(s.off, s.n, s.longest)
    q, k, v = (_heads(x, idx, s.H, s.d) for x in (s.q, s.k, s.v))
    i = torch.arange(s.longest, device="cuda")
    back = i[:, None] - i[None]                                                        # i - j
    seen = (i[None] < s.sinks[:, None])[:, None, :] | (back[None] < s.window[:, None, None])
    seen = seen & (back >= 0)[None] & ok[:, None, :] & ok[:, :, None]
    pidx = torch.clamp(-back, -(P - 1), P - 1) + P - 1
    ts = s.ts[idx] if s.T else idx
    tb = _bucket(ts[:, :, None], ts[:, None, :])
    z = q @ k.transpose(-1, -2)
    z += s.rab_pos[pidx]
    z += s.rab_time[tb][:, None]
    return idx, ok, q, k, v, seen[:, None], pidx, tb, z


def _rows(x, ok, T):
    """[T, H*d] from [n, H, longest, d]."""
    return x.transpose(1, 2).reshape(*ok.shape, -1)[ok]


def plain_window_fwd(s):
    idx, ok, q, k, v, seen, _, _, z = _window_scores(s)
    a = torch.where(seen, z * torch.sigmoid(z), 0.0)
    y = _rows(a @ v, ok, s.T) / s.alpha
    return dict(y=y.to(s.dtype), o_pre=_norm_mul(s, y, s.u.float()).to(s.dtype))


def plain_window_bwd(s):
    idx, ok, q, k, v, seen, pidx, tb, z = _window_scores(s)
    dy = _heads(s.dy, idx, s.H, s.d) / s.alpha
    sg = torch.sigmoid(z)
    a = torch.where(seen, z * sg, 0.0)
    dv = a.transpose(-1, -2) @ dy
    dz = torch.where(seen, (dy @ v.transpose(-1, -2)) * (sg * (1 + z * (1 - sg))), 0.0)
    dq, dk = dz @ k, dz.transpose(-1, -2) @ q
    by_pair = dz.sum(1, dtype=torch.float64)
    d_pos = torch.bincount(pidx.flatten(), by_pair.sum(0).flatten(), minlength=2 * P - 1)
    d_time = torch.bincount(tb.flatten(), by_pair.flatten(), minlength=NB)
    return dict(dq=_rows(dq, ok, s.T).to(s.dtype), dk=_rows(dk, ok, s.T).to(s.dtype), dv=_rows(dv, ok, s.T).to(s.dtype),
                d_rab_pos=d_pos.float(), d_rab_time=d_time.float())


def plain_tree(s):
    m, page = s.m, s.m.k.shape[1]
    idx, ok = _padded(s.off, s.n, s.nodes)
    q, k, v = (_heads(x, idx, s.H, s.d) for x in (s.q, s.k, s.v))
    # ancestors of each node, itself among them: paths of parent steps
    up = torch.where(ok, s.parent[idx], -1)
    steps = torch.eye(s.nodes, device="cuda") + (up[:, :, None] == torch.arange(s.nodes, device="cuda")).float()
    anc = (torch.linalg.matrix_power(steps, max(s.case["depth"] - 1, 1)) > 0) & ok[:, :, None]
    depth = anc.sum(-1) - 1
    # the history's rows, gathered from the pages
    n = m.lens[s.slots.long()].long()
    table = m.page_table[s.slots.long()].long()
    pg = torch.clamp(table, min=0)
    hk = m.k[pg].float().view(s.n, -1, s.H, s.d).transpose(1, 2)
    hv = m.v[pg].float().view(s.n, -1, s.H, s.d).transpose(1, 2)
    ht = m.ts[pg].view(s.n, -1)
    j = torch.arange(hk.shape[2], device="cuda")
    pos = n[:, None] + depth                                                           # [n, nodes]
    ts = s.node_ts[idx]
    seen_h = (j[None] < n[:, None])[:, None, :].expand(-1, s.nodes, -1)
    seen_t = anc
    if s.window is not None:
        seen_h = seen_h & ((j[None] < s.sinks[:, None])[:, None, :] | (pos[:, :, None] - j < s.window[:, None, None]))
        seen_t = seen_t & ((pos < s.sinks[:, None])[:, None, :] | (pos[:, :, None] - pos[:, None, :] < s.window[:, None, None]))
    hv = torch.where((j[None] < n[:, None])[:, None, :, None], hv, 0.0)                # what lies past the history is no one's
    zh = q @ hk.transpose(-1, -2)
    zh += (s.rab_pos[torch.clamp(j - pos[:, :, None], -(P - 1), P - 1) + P - 1] + s.rab_time[_bucket(ts[:, :, None], ht[:, None, :])])[:, None]
    y = torch.where(seen_h[:, None], zh * torch.sigmoid(zh), 0.0) @ hv
    zt = q @ k.transpose(-1, -2)
    zt += (s.rab_pos[torch.clamp(pos[:, None, :] - pos[:, :, None], -(P - 1), P - 1) + P - 1] + s.rab_time[_bucket(ts[:, :, None], ts[:, None, :])])[:, None]
    y += torch.where(seen_t[:, None], zt * torch.sigmoid(zt), 0.0) @ v
    y = _rows(y, ok, s.T) / s.alpha
    return dict(y=y.to(torch.bfloat16), o_pre=_norm_mul(s, y, s.u.float()).to(torch.bfloat16))


# ----------------------------------------------------------------------------- plain forms: pages

def _held(m, slots):
    """Which entries of these slots' page-table rows hold pages."""
    page = m.k.shape[1]
    n = (m.lens[slots.long()] + page - 1) // page
    return torch.arange(m.page_table.shape[1], device="cuda")[None] < n[:, None]


def plain_free(m, slots):
    s = slots.long()
    pages = m.page_table[s][_held(m, slots)].long()
    m.ref.index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    m.page_table[s] = -1
    m.lens[s] = 0


def plain_fork(m, src, dst):
    pages = m.page_table[src.long()][_held(m, src)].long()
    m.ref.index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    m.page_table[dst.long()] = m.page_table[src.long()]
    m.lens[dst.long()] = m.lens[src.long()]


def _take(m, need):
    """For each request its place in the list of free pages, lowest page first, and that list."""
    free = torch.argsort(m.ref != 0, stable=True)
    return torch.cumsum(need, 0) - need, free


def _targets(m, slots, off, T, old):
    """Pool row of each of T new rows: row r of request q goes to position old[q] + r of its slot."""
    page = m.k.shape[1]
    cnt = (off[1:] - off[:-1]).long()
    q = torch.repeat_interleave(torch.arange(cnt.numel(), device="cuda"), cnt, output_size=T)
    at = old.long()[q] + torch.arange(T, device="cuda") - off[q].long()
    return q, m.page_table[slots.long()[q], at // page].long() * page + at % page


def plain_append(m, slots, off, T, k, v, ts):
    page, D, s = m.k.shape[1], m.k.shape[2], slots.long()
    old, cnt = m.lens[s].long(), (off[1:] - off[:-1]).long()
    p_old, p_new = (old + page - 1) // page, (old + cnt + page - 1) // page
    last = m.page_table[s, torch.clamp(p_old - 1, min=0)].long()
    split = (old % page != 0) & (cnt > 0) & (m.ref[torch.clamp(last, min=0)] > 1)     # a shared page that would be written: copied first
    base, free = _take(m, p_new - p_old + split)
    col = torch.arange(m.page_table.shape[1], device="cuda")[None]
    first = (p_old - split.long())[:, None]
    fresh = (col >= first) & (col < p_new[:, None])
    pages = free[torch.where(fresh, base[:, None] + col - first, 0)]
    m.page_table[s] = torch.where(fresh, pages.int(), m.page_table[s])
    src, dst = last[split], free[base[split]]
    m.k[dst], m.v[dst], m.ts[dst] = m.k[src], m.v[src], m.ts[src]
    m.ref.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    m.ref[pages[fresh]] = 1
    m.lens[s] = (old + cnt).int()
    _, to = _targets(m, slots, off, T, old)
    m.k.view(-1, D)[to], m.v.view(-1, D)[to], m.ts.view(-1)[to] = k, v, ts


def plain_compact(m, slots, keep_off, keep):
    page, D, s = m.k.shape[1], m.k.shape[2], slots.long()
    cnt, T = (keep_off[1:] - keep_off[:-1]).long(), keep.numel()
    q = torch.repeat_interleave(torch.arange(cnt.numel(), device="cuda"), cnt, output_size=T)
    frm = m.page_table[s[q], keep.long() // page].long() * page + keep.long() % page
    gone = m.page_table[s][_held(m, slots)].long()
    need = (cnt + page - 1) // page
    base, free = _take(m, need)
    col = torch.arange(m.page_table.shape[1], device="cuda")[None]
    fresh = col < need[:, None]
    pages = free[torch.where(fresh, base[:, None] + col, 0)]
    m.ref.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    m.ref[pages[fresh]] = 1
    m.page_table[s] = torch.where(fresh, pages.int(), -1)
    m.lens[s] = cnt.int()
    _, to = _targets(m, slots, keep_off, T, torch.zeros_like(cnt))
    m.k.view(-1, D)[to], m.v.view(-1, D)[to], m.ts.view(-1)[to] = m.k.view(-1, D)[frm], m.v.view(-1, D)[frm], m.ts.view(-1)[frm]


# ----------------------------------------------------------------------------- what cannot be done without

def _pairs(n, S, W):
    """Visible pairs of a row of n tokens: token i sees min(i + 1, W) of the window and the sinks before it."""
    i = np.arange(n)
    return int((np.minimum(i + 1, W) + np.minimum(S, np.maximum(i + 1 - W, 0))).sum())


def work(case):
    c = case
    D, lens = c["H"] * c["d"], _lens(case)
    eb = 4 if c.get("dtype") == "f32" else 2
    if c["op"] in ("window_fwd", "window_bwd"):
        T = sum(lens)
        pairs = sum(_pairs(n, S, W) for n, S, W in zip(lens, *_rules(c)))
        tables = 4 * (2 * P - 1 + NB)
        if c["op"] == "window_fwd":                       # q, k, v, u in; y, o_pre out
            return dict(bytes=6 * T * D * eb + 8 * T + tables + 8 * D, flops=4 * c["d"] * c["H"] * pairs)
        return dict(bytes=7 * T * D * eb + 8 * T + 2 * tables, flops=10 * c["d"] * c["H"] * pairs)
    row = 2 * D * eb + 8
    if c["op"] == "refill":
        return dict(bytes=2 * row * sum(lens), flops=0)
    if c["op"] == "beams":
        split = sum(c["beams"] * (n % c["page"]) for n in lens)     # rows of the shared pages that are written on
        return dict(bytes=2 * row * (split + c["n"] * c["beams"] * c["add"]), flops=0)
    if c["op"] == "compact":
        return dict(bytes=2 * row * sum(min(c["keep"], n) for n in lens), flops=0)
    nodes = _lens(c, "nlo", "nhi", 2)
    seen = rows = 0
    for n, m, S, W in zip(lens, nodes, *(_rules(c) if c["window"] else ([0] * c["n"], [1 << 30] * c["n"]))):
        lev = _levels(c, m)
        w = np.clip(W - 1 - lev, 0, n)                     # of the history, the window's part
        seen += int((w + np.minimum(S, n - w)).sum()) + int((np.minimum(lev + 1, W)).sum())
        rows += (min(n, min(n, W - 1) + S) if m else 0)
    T = sum(nodes)
    return dict(bytes=row * rows + 6 * T * D * 2 + 12 * T, flops=4 * c["d"] * c["H"] * seen)


# ----------------------------------------------------------------------------- the definition in 64 bits

def _bits(x):
    """Bit length of whole numbers below 2^52, from the exponent."""
    return torch.clamp(torch.frexp(x.double())[1], max=NB - 1).long()


def _silu64(z):
    return z / (1 + torch.exp(-z))


def _ln64(s, y, u):
    y = y - y.mean(1, keepdim=True)
    return (y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * s.gamma.double() + s.beta.double()) * u.double()


def _exact_window(s):
    T, H, d = s.T, s.H, s.d
    off, S, W = s.off.tolist(), s.sinks.tolist(), s.window.tolist()
    rp, rt = s.rab_pos.double(), s.rab_time.double()
    y = torch.zeros(T, H * d, dtype=torch.float64, device="cuda")
    if s.op == "window_bwd":
        dq, dk, dv = (torch.zeros_like(y) for _ in range(3))
        dp, dt = torch.zeros_like(rp), torch.zeros_like(rt)
    for b in range(s.n):
        a0, a1 = off[b], off[b + 1]
        if a0 == a1:
            continue
        i = torch.arange(a1 - a0, device="cuda")
        delta = i[None, :] - i[:, None]                    # j - i
        mask = (delta <= 0) & ((delta > -W[b]) | (i[None, :] < S[b]))
        pi = delta.clamp(1 - P, P - 1) + (P - 1)
        t = s.ts[a0:a1]
        tb = _bits((t[None, :] - t[:, None]).abs())
        bias = rp[pi] + rt[tb]
        for h in range(H):
            c = slice(h * d, (h + 1) * d)
            q, k, v = s.q[a0:a1, c].double(), s.k[a0:a1, c].double(), s.v[a0:a1, c].double()
            z = q @ k.T + bias
            if s.op == "window_fwd":
                y[a0:a1, c] = (_silu64(z) * mask) @ v / s.alpha
                continue
            g = s.dy[a0:a1, c].double()
            dv[a0:a1, c] = (_silu64(z) * mask).T @ g / s.alpha
            e = torch.exp(-z)
            dz = mask * (g @ v.T) / s.alpha * ((1 + e + z * e) / (1 + e) ** 2)
            dq[a0:a1, c], dk[a0:a1, c] = dz @ k, dz.T @ q
            dp += torch.bincount(pi.flatten(), dz.flatten(), minlength=2 * P - 1)
            dt += torch.bincount(tb.flatten(), dz.flatten(), minlength=NB)
    if s.op == "window_bwd":
        return dict(dq=dq, dk=dk, dv=dv, d_rab_pos=dp, d_rab_time=dt)
    return dict(y=y, o_pre=_ln64(s, y, s.u))


def _exact_tree(s):
    m, page = s.m, s.m.k.shape[1]
    off, par, H, d = s.off.tolist(), s.parent.tolist(), s.H, s.d
    S = s.sinks.tolist() if s.window is not None else [0] * s.n
    W = s.window.tolist() if s.window is not None else [1 << 40] * s.n
    lens = m.lens.tolist()
    rp, rt = s.rab_pos.double(), s.rab_time.double()
    y = torch.zeros(s.T, H * d, dtype=torch.float64, device="cuda")
    for b, slot in enumerate(s.slots.tolist()):
        a0, a1 = off[b], off[b + 1]
        if a0 == a1:
            continue
        n, cnt = lens[slot], a1 - a0
        seen = np.zeros((cnt, cnt), bool)
        depth = np.zeros(cnt, np.int64)
        for i in range(cnt):
            p = par[a0 + i]
            if p >= 0:
                seen[i] = seen[p]
                depth[i] = depth[p] + 1
            seen[i, i] = True
        pages = m.page_table[slot, :-(-n // page)].long()
        hk, hv, ht = m.k[pages].view(-1, H * d)[:n], m.v[pages].view(-1, H * d)[:n], m.ts[pages].view(-1)[:n]
        K, V, t = torch.cat([hk, s.k[a0:a1]]), torch.cat([hv, s.v[a0:a1]]), torch.cat([ht, s.node_ts[a0:a1]])
        at = n + torch.from_numpy(depth).cuda()
        pos = torch.cat([torch.arange(n, device="cuda"), at])
        mask = torch.cat([torch.ones(cnt, n, dtype=torch.bool, device="cuda"), torch.from_numpy(seen).cuda()], 1)
        mask &= (pos[None] < S[b]) | (at[:, None] - pos[None] < W[b])
        bias = rp[(pos[None] - at[:, None]).clamp(1 - P, P - 1) + P - 1] + rt[_bits((t[None] - s.node_ts[a0:a1, None]).abs())]
        for h in range(H):
            c = slice(h * d, (h + 1) * d)
            z = s.q[a0:a1, c].double() @ K[:, c].double().T + bias
            y[a0:a1, c] = (_silu64(z) * mask) @ V[:, c].double() / s.alpha
    return dict(y=y, o_pre=_ln64(s, y, s.u))


def exact(case, seed):
    if case["op"] in ("refill", "beams", "compact"):       # copies and whole numbers: nothing is computed
        return None
    s = prepare(case, seed)
    return _exact_tree(s) if s.op == "tree" else _exact_window(s)
