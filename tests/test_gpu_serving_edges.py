"""Edges of the serving operators: first copies of every ring stage, weights far below the largest, inner
sums far apart, codes at ties, sizes that are refused.  References in 64 bits; the tolerances' terms are those
of test_gpu_serving.py (u half an ulp of the output's type, steps(n) for an fp32 sum of n terms)."""
import math

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv
from test_gpu_serving import attend_case, check_attend, h  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ attention: barriers
@pytest.mark.parametrize("typ,dim", [("bf16", 128), ("f16", 256), ("e4m3", 64)])
def test_the_first_copies_of_every_stage_are_waited_for(h, typ, dim):  # noqa: F811
    """Shares of one to a few tiles per warp, so that what is copied first is most of what there is: right, and
    the same bits in every one of many launches."""
    qt = "f16" if typ == "e4m3" else typ
    for lens in ([1] * 40, [16, 33, 47, 64, 129, 200] * 20, [700] * 30):
        got, lse, q, ref, scale, d = attend_case(h, lens, 8, 2, dim, typ, qt, 16, seed=len(lens))
        check_attend(got, lse, q, ref, scale, rows=range(0, len(lens), 7))
        out, first = d.keep[2], got.clone()
        for _ in range(40):
            out.fill_(math.nan)
            qgemv.attn_decode(h, d)
            assert torch.equal(got, first)
    assert qgemv.check_error(h) == qgemv.OK
