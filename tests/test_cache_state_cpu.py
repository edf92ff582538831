"""What the page operators and the tree scorer rely on between their blocks and between calls, as far
as it shows without a GPU."""
import ctypes as C
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "hstu_jagged_pointwise_b200", "csrc", "cache")


def bodies(src, marker):
    """Bodies of the functions whose declaration holds `marker`, by name."""
    out = {}
    for m in re.finditer(marker + r"[^;{]*?\b(\w+)\s*\([^)]*\)\s*\{", src):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[at], 0)
            at += 1
        out[m.group(1)] = src[m.end():at]
    return out


def test_no_remote_store_before_every_block_of_the_cluster_has_started():
    """A block's shared memory may be written by another block of its cluster after that one has started
    and before it has left: a barrier of the cluster comes before the first such store, and one after
    each.  Two calls in a row keep their flags apart."""
    src = open(os.path.join(CSRC, "pages.cu")).read()
    kernels = bodies(src, r"__cluster_dims__")
    assert set(kernels) == {"fork_kernel", "free_kernel"}
    for name, body in kernels.items():
        assert "map_shared_rank" not in body                        # the helper alone stores remotely
        assert 0 <= body.find("this_cluster().sync()") < body.find("cluster_any("), name
        rounds = re.findall(r"cluster_any\(\w+, (\d)\)", body)
        assert rounds == [str(i) for i in range(body.count("cluster_any("))] and len(rounds) <= 2, name
    helper = bodies(src, r"__device__ bool")["cluster_any"]
    assert helper.count("map_shared_rank") == 1 and helper.find("map_shared_rank") < helper.find("cl.sync()")


def test_items_of_overlapping_trees_are_counted_in_64_bits():
    """Bad offsets are found tree by tree, while others claim work items.  Offsets 0, T, 0, T, ... make
    every second tree valid by itself; a call that the host accepts then claims more than 2^31 items."""
    capi = pytest.importorskip("hstu_jagged_pointwise_b200.capi")
    mem = (C.c_uint8 * 4096)()
    base = (C.addressof(mem) + 255) // 256 * 256
    cache = capi.HstuPageCache(n_pages=8, page_size=16, n_slots=4, max_pages=4, row_elems=8192, dtype=capi.HSTU_BF16, k=base, v=base,
                               ts=base, page_table=base, lens=base, ref=base)
    d = capi.HstuTreeDims(B=(1 << 20) + 1, T=8192, H=64, d=128, n_pos=256, n_tbuckets=64, max_nodes=8192, alpha=5.0, ln_eps=1e-5)
    assert capi.CACHE.hstu_tree_workspace_bytes(C.byref(d), C.byref(cache)) > 0
    groups = -(-d.max_nodes // 128)
    assert (d.B + 1) // 2 * d.H * groups > 2**31
    prep = bodies(open(os.path.join(CSRC, "tree.cu")).read(), r"__global__ void __launch_bounds__\(kPrepThreads\)")["tree_prep_kernel"]
    assert re.search(r"long long base = .*\(long long\)atomicAdd\(items_claimed\(p\.ctrl\), \(unsigned long long\)cnt\)", prep)
    assert prep.find("base + cnt > p.max_items") < prep.find("s_base = (int)base")
