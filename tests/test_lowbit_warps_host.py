"""Instructions of the low-bit tensor-core kernel that a whole warp must execute together
follow a __syncwarp() where its lanes may have left a wait each for itself. Read
from the source: no run can show that the compiler will go on reuniting them."""

import os
import re

import pytest

pytestmark = pytest.mark.cpu
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "register_tiled_matrix_gb300", "csrc", "lowbit_tc.cu")


def kernel():
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    return text[text.index("lowbit_tc_kernel("):text.index("CUresult (*EncodeTiledFn)")]


def test_tensor_memory_loads():
    text = kernel()
    load = text.index("tmem_ld_32x32b_x32(")
    wait = text.rindex("wait_on(", 0, load)
    assert "__syncwarp();" in text[wait:load]


def test_barriers_after_the_roles():
    text = kernel()
    roles = text.index("if (wg == 0)")
    between = text[text.rindex("cp_async_wait<0>();"):text.index("cluster_sync();", roles)]
    assert "__syncwarp();" in between


def test_copies_do_not_outlive_their_block():
    """After a timeout a CTA stays, once all its roles are through, for as long as a wait may
    take (a copy that is late cannot be made to order)."""
    text = kernel()
    end = text[text.rindex("__syncthreads();"):]
    stay = re.search(r"if \(threadIdx.x == 0 && \*abort\) \{[^}]*< p\.limit_ns\)", end)
    assert stay and stay.start() < end.index("cluster_sync();")


def test_arrivals_across_a_pair():
    """Each arrival at the leading CTA says what its helper's contract covers."""
    whole = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    assert whole.count("mbar_arrive_cluster_tmem_free(") == 1
    assert whole.count("mbar_arrive_cluster_stage_written(") == 1
    text = kernel()
    assert len(re.findall(r"arrive_set<PAIR>\(tempty_at", text)) == 1
    publish = text[text.index("auto publish"):text.index("arrive_stage<PAIR>(written)")]
    assert publish.index("fence_proxy_async_shared();") < publish.index("__syncwarp();")
    assert text.count("arrive_stage<PAIR>(") == 1
