"""Rules that the kernels' sources keep and that no run shows reliably (no GPU needed)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_weight_dequant_gb300", "csrc")


def source(name):
    """A file of the kernels without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_warps_of_the_projection_agree_after_every_wait():
    """elect.sync, tcgen05.ld and the cluster's barriers take whole warps, and a lane gives up by its own clock."""
    text = source("qgemm_scaled.cuh")
    assert "mbar_wait_bounded(" not in text and "mbar_try_wait" not in text
    assert text.count("mbar_wait_warp(") > 10
    assert text.count("mbar_test(") == text.count("__all_sync(0xffffffffu, mbar_test(")
    assert re.search(r"mbar_wait_warp\([^{]*\{\s*return __all_sync\(", source("qgemv_ptx.cuh"))
