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


def test_dependent_launches_read_nothing_through_the_non_coherent_path():
    """Such a kernel is there while the one before it still writes what it will read; the non-coherent path (ld.global.nc, which the
    compiler also takes for const __restrict__ pointers) is for memory that does not change during a kernel's life."""
    names = [n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")) and "pdl_wait" in source(n)]
    assert {"qgemm_scaled.cuh", "qgemv_sample.cuh", "qgemv_rows.cuh", "qgemv_attn.cuh", "qgemv_pages.cuh", "qgemv_lora.cuh"} <= set(names)
    for name in names + ["qgemv_elems.cuh", "qgemv_serve.cuh"]:
        for word in ("__ldg", "ld.global.nc", "__restrict__"):
            assert word not in source(name), (name, word)


def test_aligned_cluster_barriers_of_divergent_code_follow_a_warp_barrier():
    """barrier.cluster.*.aligned takes whole warps; these kernels come to theirs from code whose lanes go different ways."""
    names = [n for n in os.listdir(CSRC) if "barrier.cluster" in source(n)]
    assert {"qgemm_scaled.cuh", "qgemv_sample.cuh", "qgemv_lora.cuh", "qgemm_tc.cuh"} <= set(names)
    for name in names:
        text = source(name)
        functions = re.findall(r"\{\s*(?:__syncwarp\(\);\s*)?asm volatile\(\"barrier\.cluster", text)
        assert functions and all("__syncwarp" in f for f in functions), name
        assert text.count('asm volatile("barrier.cluster') == len(functions), name
