"""Window mask with sinks on the GPU against the fp64 oracle: forward, backward, fp32 and bf16,
odd lengths, empty windows, sinks that end inside a tile, captured and side-stream calls."""
import numpy as np
import pytest
import torch

import oracle
from hstu_jagged_pointwise_b200 import workloads as W
from parity import assert_bf16, assert_f32, bf16, dev, errors, run_layer, storage_bwd, storage_fwd

pytestmark = pytest.mark.gpu

# lengths, sinks, windows: rows of 0 and 1 tokens, tile edges, W = S = 0, W or S past the row,
# sinks that end inside a 32-, 64- and 128-key block
BATCHES = {
    "edges": ([0, 1, 127, 128, 129, 0], [0, 0, 3, 0, 1, 2], [0, 1, 5, 128, 64, 7]),
    "nothing": ([5, 200, 130], [0, 0, 0], [0, 0, 0]),
    "sinks_only": ([300, 140, 40], [4, 130, 50], [0, 0, 0]),
    "window_only": ([700, 33], [0, 0], [100, 1]),
    "mixed": ([517, 390, 257, 1000], [4, 33, 200, 95], [96, 1, 129, 64]),
    "wide": ([300, 260], [0, 2**31 - 1], [2**31 - 1, 0]),
}


def _batch(name, **kw):
    lens, s, w = BATCHES[name]
    return W.make_window(lens, s, w, random_affine=True, with_grad=True, **kw)


def test_debug_indices_bit_exact():
    from hstu_jagged_pointwise_b200 import ops
    w = W.make_window([61, 1, 190], [4, 0, 33], [9, 1, 70], H=1, d=64, seed=3)
    d = dev(w)
    got = ops.debug_indices(d["offsets"], d["ts"], "window", d["n_static"], d["n_realtime"])
    want = oracle.indices(w.offsets, w.ts, oracle.MASK_WINDOW, w.n_static, w.n_realtime)
    for g, x in zip(got[:3], want[:3]):
        np.testing.assert_array_equal(g.cpu().numpy(), x)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", sorted(BATCHES))
def test_bf16_forward_backward(name, d):
    w = _batch(name, H=2, d=d, seed=len(name))
    out, _, _ = run_layer(w, backward=True)
    ref = oracle.layer_bwd(w)
    _, o, _, _ = oracle.layer_fwd(w)
    sf, sb = storage_fwd(w), storage_bwd(w)
    assert_bf16(out["y"], ref["y"], "y", sf["y"])
    assert_bf16(out["o_pre"], o, "o_pre", sf["o_pre"])
    for n in ("dq", "dk", "dv", "du"):
        assert_bf16(out[n], ref[n], n, sb[n])
    # sums of dz = dY.V SiLU' over pairs of both signs, with Y and dY stored in bf16 (2^-9 each): where the
    # sum cancels, those two roundings alone exceed 5e-3 of it (the model: 5.24e-3 for window_only, d = 64,
    # seed 11), so the composed-layer bound applies; from a given dY see test_bias_gradients_keep_fp32
    for n in ("d_rab_pos", "d_rab_time"):
        assert_bf16(out[n], ref[n], n, sb[n], chain=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", ["edges", "sinks_only", "mixed"])
def test_bias_gradients_keep_fp32(name, d):
    """From a bf16 dY the bias gradients are fp32 sums of fp32 terms: S and dP are 128-term fp32 sums of
    exact products (2^-24 * sqrt(128) relative to their terms, which reach ~8 x the result), exp and the
    reciprocal add a few 2^-22, the sums another 2^-24 a term: some 2^-19 = 2e-6 a term at random, bounded
    here by 2e-5 of the gradient's norm."""
    w = _batch(name, H=2, d=d, seed=7)
    _, layer, t = run_layer(w)
    got = layer.backward_from_dy(t["q"], t["k"], t["v"], t["rab_pos"], t["rab_time"], t["grad"])
    assert layer.check_device_error() == 0
    dq, dk, dv, drp, drt = oracle.attn_bwd(w, oracle.f32(w.grad))
    assert errors(got["d_rab_pos"], drp)[0] <= 2e-5
    assert errors(got["d_rab_time"], drt)[0] <= 2e-5
    with oracle.bf16_operands():
        m = oracle.attn_bwd(w, oracle.f32(w.grad))
    for n, ref, model in zip(("dq", "dk", "dv"), (dq, dk, dv), m):
        assert_bf16(got[n], ref, n, bf16(model))


@pytest.mark.parametrize("d", [32, 64, 128])
def test_fp32_forward_backward(d):
    w = _batch("mixed", H=1, d=d, dtype=torch.float32, seed=9)
    out, _, _ = run_layer(w, backward=True)
    ref = oracle.layer_bwd(w)
    y, o, mu, rs = oracle.layer_fwd(w)
    assert_f32(out["y"], y, "y")
    assert_f32(out["o_pre"], o, "o_pre")
    for n in ("dq", "dk", "dv", "du", "d_rab_pos", "d_rab_time"):
        assert_f32(out[n], ref[n], n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_window_as_long_as_the_row_is_the_causal_kind(dtype):
    """The same arithmetic in the same order: bit for bit in the forward."""
    lens = [300, 129, 64, 1]
    w = W.make_window(lens, [0, 500, 0, 1], [300, 0, 1 << 20, 0], H=2, d=64, dtype=dtype, seed=2)
    c = W.make_causal(lens, H=2, d=64, dtype=dtype, seed=2)
    a, b = run_layer(w)[0], run_layer(c)[0]
    for n in ("y", "o_pre", "mean", "rstd"):
        assert torch.equal(a[n], b[n]), n


def test_row_that_sees_nothing_is_zero():
    w = W.make_window([70, 200], [0, 0], [0, 0], H=2, d=128, seed=1, random_affine=True, with_grad=True)
    out, _, _ = run_layer(w, backward=True)
    assert torch.count_nonzero(out["y"]) == 0
    for n in ("dq", "dk", "dv", "d_rab_pos", "d_rab_time"):
        assert torch.count_nonzero(out[n]) == 0, n
    want = (w.beta * w.u.float()).to(torch.bfloat16)
    assert torch.equal(out["o_pre"].cpu(), want)


def test_long_row_short_window_sampled():
    """20,000 tokens under a window of 100 with 5 sinks: tiles far apart, positions past the clamp."""
    w = W.make_window([20000, 37], [5, 0], [100, 10], H=2, d=128, seed=6)
    out, _, _ = run_layer(w)
    rows = np.unique(np.concatenate([np.arange(0, 20037, 331), [0, 1, 99, 100, 104, 105, 127, 128, 19999, 20000, 20036]]))
    with oracle.bf16_operands():
        model = bf16(oracle.attn_fwd(w, rows))
    assert_bf16(out["y"][torch.as_tensor(rows).cuda()], oracle.attn_fwd(w, rows), "y", model)


def test_extreme_timestamps():
    ts = [np.array([0, 1, 2**31 - 1, 2**31, 2**40, 2**62, 2**63 - 1] + list(range(2**63 - 400, 2**63 - 1)), np.int64),
          np.sort(np.random.default_rng(0).integers(-2**62, 2**62, 300))]
    w = W.make_window([len(t) for t in ts], [3, 40], [90, 100], H=1, d=64, seed=8, ts_list=ts, with_grad=True)
    out, _, _ = run_layer(w, backward=True)
    ref, sb = oracle.layer_bwd(w), storage_bwd(w)
    for n in ("y", "dq", "dk", "dv"):
        assert_bf16(out[n], ref[n], n, sb[n])


def test_negative_sizes_are_flagged_and_the_next_call_is_clean():
    w = W.make_window([40, 50], [2, 2], [8, 8], H=1, d=64, seed=1)
    good, layer, d = run_layer(w)
    for name in ("n_static", "n_realtime"):
        keep = d[name].clone()
        d[name][1] = -1
        y = torch.full_like(good["y"], 7.0)
        layer.forward(d["q"], d["k"], d["v"], d["u"], d["rab_pos"], d["rab_time"], d["gamma"], d["beta"],
                      out=dict(good, y=y, o_pre=torch.empty_like(y)))
        assert layer.check_device_error() == -5
        assert bool((y == 7.0).all())
        d[name].copy_(keep)
    again = layer.forward(d["q"], d["k"], d["v"], d["u"], d["rab_pos"], d["rab_time"], d["gamma"], d["beta"])
    assert layer.check_device_error() == 0
    assert torch.equal(again["y"], good["y"])


def test_group_norm():
    w = W.with_group_norm(W.make_window([200, 90], [4, 0], [64, 20], H=2, d=64, seed=5, with_grad=True), seed=5, groups=3)
    out, _, _ = run_layer(w, backward=True)
    ref, sf, sb = oracle.layer_bwd(w), storage_fwd(w), storage_bwd(w)
    assert_bf16(out["o_pre"], oracle.layer_fwd(w)[1], "o_pre", sf["o_pre"])
    for n in ("dq", "dk", "dv", "du"):
        assert_bf16(out[n], ref[n], n, sb[n])


def test_noalloc_entry_point():
    import ctypes as C

    from hstu_jagged_pointwise_b200 import capi
    w = W.make_window([200, 90], [4, 0], [64, 20], H=2, d=64, seed=5)
    out, layer, d = run_layer(w)
    y, o = torch.empty_like(out["y"]), torch.empty_like(out["o_pre"])
    mean, rstd = torch.empty_like(out["mean"]), torch.empty_like(out["rstd"])
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    P = lambda t: C.c_void_p(t.data_ptr())
    rc = capi.LIB.hstu_attn_fwd_noalloc(C.byref(layer.dims), C.byref(layer.mask), P(d["q"]), P(d["k"]), P(d["v"]), P(d["u"]),
                                        P(d["offsets"]), P(d["ts"]), P(d["rab_pos"]), P(d["rab_time"]), P(d["gamma"]),
                                        P(d["beta"]), P(y), P(o), P(mean), P(rstd), P(st),
                                        C.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0 and int(st.item()) == 0
    assert torch.equal(y, out["y"]) and torch.equal(o, out["o_pre"])


def test_captured_replayed_and_on_another_stream():
    w = _batch("mixed", H=2, d=128, seed=3)
    ref, layer, d = run_layer(w)
    args = (d["q"], d["k"], d["v"], d["u"], d["rab_pos"], d["rab_time"], d["gamma"], d["beta"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = layer.forward(*args)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a["y"], ref["y"])
    out = {n: torch.zeros_like(ref[n]) for n in ("y", "o_pre", "mean", "rstd")}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(*args, out=out)
        grads = layer.backward(*args, out, d["grad"])
    d["q"].mul_(0.5)
    g.replay()
    g.replay()
    want = layer.forward(*args)
    wg = layer.backward(*args, want, d["grad"])
    assert layer.check_device_error() == 0
    assert torch.equal(out["o_pre"], want["o_pre"]) and torch.equal(grads["dk"], wg["dk"])
    del g


def test_whole_layer_with_window():
    """ops.HSTULayer runs with the window kind and equals its parts."""
    from hstu_jagged_pointwise_b200 import ops
    w = W.make_window([200, 77], [4, 0], [50, 20], H=2, d=64, seed=4, with_grad=True)
    lw = W.make_layer(w, 128, seed=4)
    d = dev(w)
    layer = ops.HSTULayer(d["offsets"], d["ts"], 128, w.H, w.d, w.alpha, w.max_len, mask_kind="window",
                          n_static=d["n_static"], n_realtime=d["n_realtime"])
    params = dict(w1=lw.w1.cuda(), b1=lw.b1.cuda(), w2=lw.w2.cuda(), b2=lw.b2.cuda(), rab_pos=d["rab_pos"],
                  rab_time=d["rab_time"], ln_gamma=d["gamma"], ln_beta=d["beta"])
    s = layer.forward(lw.x.cuda(), params)
    g = layer.backward(s, torch.ones_like(s["out"]), params)
    assert layer.check_device_error() == 0
    sub = W.make_window([200, 77], [4, 0], [50, 20], H=2, d=64, seed=4)
    for n in ("q", "k", "v", "u"):
        setattr(sub, n, s["f1"][n].cpu())
    assert_bf16(s["attn"]["y"], oracle.attn_fwd(sub), "y", storage_fwd(sub)["y"])
    assert all(torch.isfinite(t.float()).all() for t in g.values())


@pytest.mark.parametrize("d", [64, 128])
def test_long_rows_with_sinks_backward(d):
    """Rows long enough that the queries of the sinks' key tile are worked in chunks (more than 512
    tokens, 1 to 128 sinks), beside rows where they are not: one of exactly 512, one with 129 sinks,
    one with none; dK and dV are the same bits twice."""
    w = W.make_window([2500, 512, 513, 1100, 1300, 40, 700], [4, 3, 128, 129, 0, 5, 1], [100, 50, 64, 30, 200, 7, 0], H=2, d=d, seed=11,
                      random_affine=True, with_grad=True)
    _, layer, t = run_layer(w)
    runs = [layer.backward_from_dy(t["q"], t["k"], t["v"], t["rab_pos"], t["rab_time"], t["grad"]) for _ in range(2)]
    assert layer.check_device_error() == 0
    ref = oracle.attn_bwd(w, oracle.f32(w.grad))
    with oracle.bf16_operands():
        model = oracle.attn_bwd(w, oracle.f32(w.grad))
    for n, r, m in zip(("dq", "dk", "dv"), ref, model):
        assert_bf16(runs[0][n], r, n, bf16(m))
    for n, r in zip(("d_rab_pos", "d_rab_time"), ref[3:]):
        assert errors(runs[0][n], r)[0] <= 2e-5, n
    for n in ("dk", "dv"):
        assert torch.equal(runs[0][n], runs[1][n])


def test_two_layers_on_two_streams_and_replayed():
    """Two layers' forward and backward called in turn on two streams, and as two graphs replayed side by
    side, many times with nothing waited for between: each has what it has alone (dQ and the bias
    gradients up to the order of their sums), and the next call in a stream sees the one before done."""
    from hstu_jagged_pointwise_b200 import ops
    cases = [W.make_window([1500, 700, 33, 1], [4, 0, 2, 1], [100, 64, 50, 3], H=2, d=128, seed=5, random_affine=True, with_grad=True),
             W.make_window([900, 5, 513], [1, 3, 130], [40, 2, 300], H=3, d=64, seed=6, random_affine=True, with_grad=True)]
    work, want = [], []
    for w in cases:
        fwd, layer, t = run_layer(w)
        args = [t[n] for n in ("q", "k", "v", "u", "rab_pos", "rab_time", "gamma", "beta")]

        def call(layer=layer, t=t, args=args):
            o = dict(layer.forward(*args))
            o.update(layer.backward(*args, o, t["grad"]))
            return o
        work.append(call)
        want.append({k: v.clone() for k, v in call().items()})
    torch.cuda.synchronize()
    exact = ("y", "o_pre", "dk", "dv", "du")

    def check(got):
        for o, ref in zip(got, want):
            for n, x in ref.items():
                if n in exact:
                    assert torch.equal(o[n], x), n
                else:
                    assert errors(o[n], x.double().cpu().numpy())[0] <= 1e-2, n
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = work[i]()
    torch.cuda.synchronize()
    check(got)
    graphs, outs = [], []
    for i, s in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(work[i]())
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    check(outs)
