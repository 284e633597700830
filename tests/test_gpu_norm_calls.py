"""Calls of the norm that its description allows beside the usual ones: a sum without a residual, outputs over inputs in every
combination, an eps of 0, one row with strides of its own."""
import os
import sys

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_scaled as scaled  # noqa: E402

pytestmark = pytest.mark.gpu
h = scaled.h
WIDTHS = [(3, 64), (5, 512), (2, 528), (700, 1040), (3, 20480)]


def plain(x, res, w, eps, offset=0.0):
    s = x.double() + (0 if res is None else res.double())
    return s, s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps) * (1 if w is None else offset + w.double())


@pytest.mark.parametrize("rows,N", WIDTHS)
@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_outputs_over_inputs(h, rows, N, typ):
    dtype = scaled.TYPES[typ]
    g = scaled.gen(rows + N)
    x, res, w = scaled.randn(g, rows, N).to(dtype), scaled.randn(g, rows, N).to(dtype), scaled.randn(g, N)
    s, t = plain(x, res, w, 1e-6, 0.5)
    half = scaled.HALF_ULP[dtype] * 1.01 + 2.0 ** -24
    for sum_over, y_over in (("res", "x"), ("x", "res"), (None, "x"), (None, "res"), ("x", None), ("res", None)):
        at = {"x": x.clone(), "res": res.clone()}
        total = at[sum_over] if sum_over else torch.empty_like(x)
        y = at[y_over] if y_over else torch.empty_like(x)
        qgemv.run_norm(h, qgemv.norm_desc(at["x"], w, 1e-6, y=y, res=at["res"], res_out=total, offset=0.5))
        torch.cuda.synchronize()
        scaled.within(total, s, s.abs() * half + scaled.TINY[dtype], "sum")
        scaled.within(y, t, t.abs() * (half + 2.0 ** -18) + scaled.TINY[dtype], "norm")


@pytest.mark.parametrize("rows,N", WIDTHS)
def test_a_sum_without_a_residual(h, rows, N):
    g = scaled.gen(N)
    x = scaled.randn(g, rows, N).half()
    total, y = torch.empty(rows, N, device="cuda"), torch.empty_like(x)
    qgemv.run_norm(h, qgemv.norm_desc(x, None, 0.0, y=y, res_out=total))
    torch.cuda.synchronize()
    _, t = plain(x, None, None, 0.0)
    assert torch.equal(total, x.float())
    scaled.within(y, t, t.abs() * (scaled.HALF_ULP[torch.float16] * 1.01 + 2.0 ** -18) + scaled.TINY[torch.float16], "norm")


def test_refused_calls(h):
    x = torch.zeros(4, 64, device="cuda")
    other = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(qgemv.QgemvError):
        qgemv.run_norm(h, qgemv.norm_desc(x, None, 1e-5))  # nothing to write
    with pytest.raises(TypeError):
        qgemv.norm_desc(x, None, 1e-5, y=x, res=x, res_out=other)
    with pytest.raises(ValueError):
        qgemv.norm_desc(x, None, 1e-5, y=x[:, :32])
    with pytest.raises(ValueError):
        qgemv.norm_desc(x, None, 1e-5, codes=torch.zeros(4, 64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qgemv.QgemvError):
        qgemv.run_norm(h, qgemv.norm_desc(x[:1].expand(4, 64), None, 1e-5, y=x))  # rows at a stride of 0
