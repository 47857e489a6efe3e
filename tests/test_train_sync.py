"""How the two CTAs of a pair order their memory, read off the kernel's source (CPU): an order that is missing shows in
results rarely or never, so no run can be relied on to fail for it."""
import os
import re

import grouped_gemm_swiglu_b200 as moe

SRC = os.path.join(os.path.dirname(moe.__file__), "csrc", "ffn.cu")


def test_zeroed_rows_reach_the_other_cta_at_cluster_scope():
    """Rank 1 zeroes rows of its operands with ordinary shared-memory stores, and rank 0 issues the MMAs that read them:
    what carries the order, the barrier `fix`, is arrived on with a release and waited for with an acquire at cluster scope."""
    with open(SRC) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    uses = [m for m in re.findall(r"(\w+)\((?:lead\()?&fix\[\w+\]", code) if m != "mbar_init"]
    assert sorted(uses) == ["mbar_arrive_cluster", "warp_wait_cl"]
    wait = re.search(r"bool warp_wait_cl\(.*?\n}", code, re.S).group(0)
    assert "mbar_wait_cl(" in wait and "__syncwarp()" in wait
    # and the stores are handed to the asynchronous proxy before the arrival
    zero = re.search(r"void zero_k_rows\(.*?\n}", code, re.S).group(0)
    assert zero.index("make_uint4(0, 0, 0, 0)") < zero.index("fence_proxy_async_smem()") < zero.index("__syncwarp()")
