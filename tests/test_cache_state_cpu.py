"""What the page operators and the tree scorer rely on between their blocks and between calls, as far
as it shows without a GPU."""
import os
import re

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
