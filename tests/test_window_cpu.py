"""Window mask with sinks, without a GPU: the oracle's rule and gradient pinned to hand-worked
tables, to the causal mask and to finite differences, and the library's refusals."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
from hstu_jagged_pointwise_b200 import workloads as W

capi = pytest.importorskip("hstu_jagged_pointwise_b200.capi")


def _mask(L, S, R):
    m, pi, _, _ = oracle.indices([0, L], np.arange(L), oracle.MASK_WINDOW, [S], [R])
    return m.reshape(L, L), pi.reshape(L, L)


def test_window_mask_hand_table():
    """Six tokens, one sink, a window of two, worked by hand."""
    want = ["100000", "110000", "111000", "101100", "100110", "100011"]
    m, pi = _mask(6, 1, 2)
    np.testing.assert_array_equal(m, [[int(c) for c in r] for r in want])
    i, j = np.mgrid[:6, :6]
    np.testing.assert_array_equal(pi, j - i + 255)          # positions are indices


@pytest.mark.parametrize("L,S,R", [(7, 0, 0), (7, 0, 1), (7, 3, 0), (7, 9, 0), (7, 0, 7), (7, 0, 2**31 - 1), (1, 0, 0), (1, 1, 0)])
def test_window_mask_limits(L, S, R):
    """No window and no sinks see nothing; a window of one sees itself; all sinks, or a window
    as long as the row, is the causal mask."""
    m, _ = _mask(L, S, R)
    tri = np.tril(np.ones((L, L), np.uint8))
    if S >= L or R >= L:
        want = tri
    else:
        want = tri * ((np.arange(L)[None] < S) | (np.subtract.outer(np.arange(L), np.arange(L)) < R))
    np.testing.assert_array_equal(m, want)


def test_window_forward_equals_rows_of_the_causal_oracle():
    """A token under the window equals the last token of a causal row made of what it sees, where
    the position bias is constant (sinks move closer when the gap is cut out)."""
    w = W.make_window([23], [2], [5], H=1, d=8, dtype=torch.float32, seed=4, alpha=3.0)
    w.rab_pos = torch.full_like(w.rab_pos, 0.3)
    y = oracle.attn_fwd(w)
    for i in (0, 4, 6, 11, 22):
        seen = [j for j in range(i + 1) if j < 2 or i - j < 5]
        c = W.make_causal([len(seen)], H=1, d=8, dtype=torch.float32, seed=0, alpha=3.0, ts_list=[w.ts[seen]])
        c.q, c.k, c.v, c.rab_pos, c.rab_time = w.q[seen], w.k[seen], w.v[seen], w.rab_pos, w.rab_time
        np.testing.assert_allclose(y[i], oracle.attn_fwd(c)[-1], rtol=1e-12, atol=1e-13)


def test_window_gradient_finite_differences():
    """Every gradient of L = sum(Y * g) by central differences (Y is smooth; step 1e-4 on values of
    order one leaves an error of order 1e-8)."""
    w = W.make_window([1, 9, 6], [0, 2, 1], [1, 3, 0], H=2, d=4, dtype=torch.float32, seed=5, alpha=2.0)
    g = np.random.default_rng(0).standard_normal((w.T, w.D))
    dq, dk, dv, drp, drt = oracle.attn_bwd(w, g)
    rng = np.random.default_rng(1)
    for name, grad in (("q", dq), ("k", dk), ("v", dv), ("rab_pos", drp), ("rab_time", drt)):
        base = getattr(w, name).double().numpy().copy()
        flat = np.argsort(-np.abs(grad).ravel())[:8] if name.startswith("rab") else rng.integers(0, grad.size, 10)
        for e in flat:
            at = np.unravel_index(e, base.shape)
            v = []
            for step in (1e-3, -1e-3):
                x = base.copy()
                x[at] += step
                setattr(w, name, torch.as_tensor(x, dtype=torch.float32))
                x32 = getattr(w, name).double().numpy()[at]
                v.append((float((oracle.attn_fwd(w) * g).sum()), x32))
            setattr(w, name, torch.as_tensor(base, dtype=torch.float32))
            num = (v[0][0] - v[1][0]) / (v[0][1] - v[1][1])
            assert abs(num - grad[at]) <= 1e-5 * max(1.0, np.abs(grad).max()), (name, at, num, grad[at])
    assert np.all(dk[0:0] == 0)
    m, _, _, po = oracle.indices(w.offsets, w.ts, oracle.MASK_WINDOW, w.n_static, w.n_realtime)
    assert m.sum() > 0


def test_window_library_refusals():
    """The kind needs both arrays; sizes and workspaces are checked as for the other kinds."""
    d = capi.HstuDims(B=1, T=4, H=1, d_qk=64, d_v=64, dtype=capi.HSTU_BF16, n_pos=256, n_tbuckets=64, max_seq_len=4,
                      alpha=1.0, ln_eps=1e-5)
    assert capi.LIB.hstu_attn_workspace_bytes(C.byref(d), capi.HSTU_MASK_WINDOW, 0) > 0
    assert capi.LIB.hstu_attn_workspace_bytes(C.byref(d), capi.HSTU_MASK_WINDOW, 1) > 0
    buf = (C.c_int32 * 4)()
    a = C.addressof(buf)
    for ns, nr in ((None, a), (a, None), (None, None)):
        m = capi.HstuMaskSpec(kind=capi.HSTU_MASK_WINDOW, n_static=ns, n_realtime=nr)
        assert capi.LIB.hstu_attn_fwd(C.byref(d), C.byref(m), *[None] * 15, 0, None) == capi.HSTU_ERR_INVALID_ARG
        assert capi.LIB.hstu_attn_bwd_dy(C.byref(d), C.byref(m), *[None] * 14, 0, None) in (
            capi.HSTU_ERR_INVALID_ARG, capi.HSTU_ERR_WORKSPACE)
    m = capi.HstuMaskSpec(kind=capi.HSTU_MASK_WINDOW, n_static=a, n_realtime=a)
    assert capi.LIB.hstu_attn_fwd(C.byref(d), C.byref(m), *[None] * 15, 0, None) == capi.HSTU_ERR_WORKSPACE
    assert capi.LIB.hstu_debug_indices(1, capi.HSTU_MASK_WINDOW, a, a, None, a, 256, 64, a, a, a, a, None) == \
        capi.HSTU_ERR_INVALID_ARG


def test_window_python_refusals():
    ops = pytest.importorskip("hstu_jagged_pointwise_b200.ops")
    with pytest.raises((ValueError, AttributeError)):
        ops.make_mask("window")
    with pytest.raises(ValueError):
        ops.make_mask("window", torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
