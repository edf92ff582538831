"""Window kind: what does not depend on timing is the same bits however calls overlap, what does stays
within the order of its sums, and the bias gradients hold where times span all of 64 bits."""
import numpy as np
import pytest
import torch

import oracle
from hstu_jagged_pointwise_b200 import workloads as W
from parity import assert_bf16, bf16, errors, run_layer

pytestmark = pytest.mark.gpu

EXACT = ("y", "o_pre", "mean", "rstd", "dk", "dv", "du", "d_gamma", "d_beta")


def equal_up_to_order(got, want, n):
    """dQ is a sum of at most five key tiles' shares (window of up to 300 and the sinks'), added in any
    order in fp32: two orders differ by at most 2 * 4 * 2^-24 times the shares' absolute sum, which is
    bounded by five times the largest share; shares up to 12 times the largest sum give 2^-15 of it.  The
    rounding to bf16 then adds at most one whole step, 2^-7 of the value.
    A bias gradient sums some 10^3 reductions of both signs: sqrt(1e3) * 2^-24 = 2e-6 of its norm."""
    a, b = got.double(), want.double()
    if n == "dq":
        assert bool(((a - b).abs() <= 2.0**-7 * b.abs() + 2.0**-15 * b.abs().max()).all()), n
    else:
        assert errors(got, b.cpu().numpy())[0] <= 1e-5, n


def check(got, want):
    for n, x in want.items():
        if n in EXACT:
            assert torch.equal(got[n], x), n
        else:
            equal_up_to_order(got[n], x, n)


def test_overlapping_calls_give_what_each_gives_alone():
    """Two layers' forward and backward in turn on two streams, called and replayed side by side with
    nothing waited for between; the outputs of every call are kept and compared."""
    cases = [W.make_window([1500, 700, 33, 1], [4, 0, 2, 1], [100, 64, 50, 3], H=2, d=128, seed=5, random_affine=True, with_grad=True),
             W.make_window([900, 5, 513], [1, 3, 130], [40, 2, 300], H=3, d=64, seed=6, random_affine=True, with_grad=True)]
    work, want = [], []
    for w in cases:
        _, layer, t = run_layer(w)
        args = [t[n] for n in ("q", "k", "v", "u", "rab_pos", "rab_time", "gamma", "beta")]

        def call(layer=layer, t=t, args=args):
            o = dict(layer.forward(*args))
            o.update(layer.backward(*args, o, t["grad"]))
            return o
        work.append(call)
        want.append({k: v.clone() for k, v in call().items()})
        assert layer.check_device_error() == 0
    assert set(EXACT) | {"dq", "d_rab_pos", "d_rab_time"} == set(want[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    kept = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                kept[i].append(work[i]())
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i, s in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(work[i]())
        graphs.append(g)
    for _ in range(10):
        for i, (g, s) in enumerate(zip(graphs, streams)):
            with torch.cuda.stream(s):
                g.replay()
                kept[i].append({k: v.clone() for k, v in outs[i].items()})
    torch.cuda.synchronize()
    for i in range(2):
        assert len(kept[i]) == 20
        for got in kept[i]:
            check(got, want[i])
    del graphs


@pytest.mark.parametrize("d", [64, 128])
def test_bias_gradients_of_extreme_times(d):
    """Times from -2^62 to 2^63 - 1, whose differences pass 32 bits, so that pairs are worked one by one:
    the bias gradients are fp32 sums of fp32 terms as elsewhere (some 2^-19 a term at random, bounded by
    2e-5 of the norm)."""
    ts = [np.array([0, 1, 2**31 - 1, 2**31, 2**40, 2**62, 2**63 - 1] + list(range(2**63 - 400, 2**63 - 1)), np.int64),
          np.sort(np.random.default_rng(0).integers(-2**62, 2**62, 300)),
          np.sort(np.random.default_rng(1).integers(0, 2**34, 700))]
    w = W.make_window([len(t) for t in ts], [3, 40, 2], [90, 100, 130], H=2, d=d, seed=8, ts_list=ts, with_grad=True)
    _, layer, t = run_layer(w)
    got = layer.backward_from_dy(t["q"], t["k"], t["v"], t["rab_pos"], t["rab_time"], t["grad"])
    assert layer.check_device_error() == 0
    ref = oracle.attn_bwd(w, oracle.f32(w.grad))
    with oracle.bf16_operands():
        model = oracle.attn_bwd(w, oracle.f32(w.grad))
    for n, r, m in zip(("dq", "dk", "dv"), ref, model):
        assert_bf16(got[n], r, n, bf16(m))
    for n, r in zip(("d_rab_pos", "d_rab_time"), ref[3:]):
        assert errors(got[n], r)[0] <= 2e-5, n


def test_rules_of_other_batches_are_refused():
    """Sinks and windows for fewer or more rows than the batch has: the device would read past them."""
    from hstu_jagged_pointwise_b200 import ops
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    ts = torch.arange(9, dtype=torch.int64, device="cuda")
    rule = lambda n: torch.ones(n, dtype=torch.int32, device="cuda")
    for s, w in ((1, 2), (2, 1), (3, 2), (2, 3), (0, 2)):
        with pytest.raises(ValueError):
            ops.Layer(off, ts, 1, 64, torch.bfloat16, 5.0, 5, mask_kind="window", n_static=rule(s), n_realtime=rule(w))
        with pytest.raises(ValueError):
            ops.HSTULayer(off, ts, 64, 1, 64, 5.0, 5, mask_kind="window", n_static=rule(s), n_realtime=rule(w))
    ops.Layer(off, ts, 1, 64, torch.bfloat16, 5.0, 5, mask_kind="window", n_static=rule(2), n_realtime=rule(2))
