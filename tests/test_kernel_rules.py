"""Rules that the kernels' sources keep and that no run shows reliably (no GPU needed)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_weight_dequant_gb300", "csrc")


def source(name):
    """A file of the kernels without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_every_lane_comes_to_elect_in_the_projection():
    """elect.sync takes whole warps, and a lane gives up a wait by its own clock: what it saw is asked for after the election."""
    text = source("qgemm_scaled.cuh")
    assert text.count("elect_one()") > 10
    assert not re.search(r"&&[^;{}]*elect_one\(\)", text), "an election that some lanes skip"
