"""Host-side checks of the entry points of projections in 8 bits and of sampling (no GPU needed): layouts, and
every refusal.  A refused call reads nothing but the description and a few numbers of the handle, so a block of
zeros stands in for the handle."""
import ctypes

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv
from quantized_weight_dequant_gb300.build import build_library

PTR = 1 << 20  # an aligned address that no refused call follows


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_library()


@pytest.fixture(scope="module")
def handle():
    return ctypes.create_string_buffer(1 << 16)


def call(name, handle, desc):
    return getattr(qgemv.lib(), "qgemv_" + name)(ctypes.addressof(handle), desc, None)


def norm(**kw):
    d = dict(x=PTR, res=PTR, res_out=PTR, weight=PTR, y=PTR, codes=PTR, scale=PTR, x_stride=256, res_stride=256, res_out_stride=256,
             y_stride=256, codes_stride=256, scale_stride=2, rows=3, N=256, eps=1e-5, offset=0.0, in_type=2, res_type=2, weight_type=2, out=2)
    d.update(kw)
    return qgemv.Norm(**d)


def quant(**kw):
    d = dict(x=PTR, up=PTR, codes=PTR, scale=PTR, x_stride=256, up_stride=256, codes_stride=256, scale_stride=2, rows=3, N=256, in_type=2)
    d.update(kw)
    return qgemv.Quant(**d)


def scaled(**kw):
    d = dict(x=PTR, x_scale=PTR, W=PTR, w_scale=PTR, y=PTR, x_stride=256, x_scale_stride=2, y_stride=100, M=3, N=100, K=256, out=0)
    d.update(kw)
    return qgemv.Scaled(**d)


def sample(**kw):
    d = dict(logits=PTR, stride=101, u=PTR, temperature=PTR, top_k=PTR, top_p=PTR, min_p=PTR, tokens=PTR, logprobs=PTR, rows=3, V=101, type=0)
    d.update(kw)
    return qgemv.Sample(**d)


MAKE = {"run_norm": norm, "quant_rows": quant, "run_scaled": scaled, "sample": sample}


@pytest.mark.parametrize("name", list(MAKE))
def test_null_handles_and_descriptions_are_refused(name, handle):
    fn = getattr(qgemv.lib(), "qgemv_" + name)
    assert fn(None, MAKE[name](), None) == qgemv.ERR_INVALID_ARG
    assert fn(ctypes.addressof(handle), None, None) == qgemv.ERR_INVALID_ARG


def test_structures_have_the_c_layout():
    """Sizes on an LP64 machine: the fields in their order with natural alignment."""
    assert ctypes.sizeof(qgemv.Norm) == 7 * 8 + 7 * 8 + 7 * 4 + 4
    assert ctypes.sizeof(qgemv.Quant) == 4 * 8 + 6 * 8 + 8
    assert ctypes.sizeof(qgemv.Scaled) == 5 * 8 + 6 * 8 + 8
    assert ctypes.sizeof(qgemv.Sample) == 9 * 8 + 8 + 2 * 4


INVALID, SHAPE, ALIGN = qgemv.ERR_INVALID_ARG, qgemv.ERR_BAD_SHAPE, qgemv.ERR_MISALIGNED


@pytest.mark.parametrize("change,status", [
    (dict(x=0), INVALID), (dict(y=0, codes=0), INVALID), (dict(scale=0), INVALID), (dict(in_type=3), INVALID), (dict(res_type=-1), INVALID),
    (dict(weight_type=7), INVALID), (dict(out=3), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(offset=float("nan")), INVALID), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(N=0), SHAPE), (dict(N=65544), SHAPE),
    (dict(N=248), SHAPE), (dict(N=255, codes=0), SHAPE), (dict(x_stride=248), SHAPE), (dict(res_stride=0), SHAPE), (dict(res_out_stride=255), SHAPE),
    (dict(y_stride=-256), SHAPE), (dict(codes_stride=240), SHAPE), (dict(scale_stride=1), SHAPE), (dict(x_stride=1 << 41), SHAPE),
    (dict(x=PTR + 8), ALIGN), (dict(x_stride=260), ALIGN), (dict(res=PTR + 2), ALIGN), (dict(res_out_stride=257), ALIGN),
    (dict(y=PTR + 4), ALIGN), (dict(codes=PTR + 8), ALIGN), (dict(codes_stride=264), ALIGN), (dict(weight=PTR + 4), ALIGN), (dict(scale=PTR + 2), ALIGN)])
def test_norm_refusals(handle, change, status):
    assert call("run_norm", handle, norm(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=0), INVALID), (dict(codes=0), INVALID), (dict(scale=0), INVALID), (dict(in_type=3), INVALID), (dict(rows=-1), SHAPE),
    (dict(N=8), SHAPE), (dict(N=0), SHAPE), (dict(N=264), SHAPE), (dict(x_stride=255), SHAPE), (dict(up_stride=0), SHAPE), (dict(codes_stride=255), SHAPE),
    (dict(scale_stride=1), SHAPE), (dict(rows=(1 << 31) - 1, N=8192, x_stride=8192, up_stride=8192, codes_stride=8192, scale_stride=64), SHAPE),
    (dict(x=PTR + 8), ALIGN), (dict(up=PTR + 8), ALIGN), (dict(codes=PTR + 8), ALIGN), (dict(x_stride=260), ALIGN), (dict(up_stride=257), ALIGN),
    (dict(codes_stride=264), ALIGN), (dict(scale=PTR + 1), ALIGN)])
def test_quant_refusals(handle, change, status):
    assert call("quant_rows", handle, quant(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=0), INVALID), (dict(x_scale=0), INVALID), (dict(W=0), INVALID), (dict(w_scale=0), INVALID), (dict(y=0), INVALID), (dict(out=3), INVALID),
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=0), SHAPE), (dict(N=1 << 31), SHAPE), (dict(K=0), SHAPE), (dict(K=8), SHAPE), (dict(K=255), SHAPE),
    (dict(x_stride=240), SHAPE), (dict(x_scale_stride=1), SHAPE), (dict(y_stride=99), SHAPE), (dict(x=PTR + 8), ALIGN), (dict(W=PTR + 8), ALIGN),
    (dict(y=PTR + 4), ALIGN), (dict(x_stride=264), ALIGN), (dict(x_scale=PTR + 2), ALIGN), (dict(w_scale=PTR + 2), ALIGN)])
def test_projection_refusals(handle, change, status):
    assert call("run_scaled", handle, scaled(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(logits=0), INVALID), (dict(u=0), INVALID), (dict(tokens=0), INVALID), (dict(type=3), INVALID), (dict(rows=-1), SHAPE), (dict(V=0), SHAPE),
    (dict(V=(1 << 20) + 1, stride=1 << 21), SHAPE), (dict(stride=100), SHAPE), (dict(rows=1 << 30), SHAPE), (dict(logits=PTR + 4), ALIGN),
    (dict(u=PTR + 2), ALIGN), (dict(temperature=PTR + 1), ALIGN), (dict(top_k=PTR + 2), ALIGN), (dict(top_p=PTR + 2), ALIGN),
    (dict(min_p=PTR + 2), ALIGN), (dict(tokens=PTR + 2), ALIGN), (dict(logprobs=PTR + 2), ALIGN)])
def test_sample_refusals(handle, change, status):
    assert call("sample", handle, sample(**change)) == status


@pytest.mark.parametrize("name,rows", [("run_norm", "rows"), ("quant_rows", "rows"), ("run_scaled", "M"), ("sample", "rows")])
def test_no_rows_are_no_work(name, rows, handle):
    assert call(name, handle, MAKE[name](**{rows: 0})) == qgemv.OK


def test_descriptions_refuse_tensors_of_the_host():
    x = torch.zeros(2, 64, dtype=torch.float16)
    codes, scale = torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(2, 1)
    with pytest.raises(TypeError):
        qgemv.norm_desc(x, x[0], 1e-5, y=x)
    with pytest.raises(TypeError):
        qgemv.quant_desc(x, codes, scale)
    with pytest.raises(TypeError):
        qgemv.scaled_desc(codes, scale, codes, scale, x)
    with pytest.raises(TypeError):
        qgemv.sample_desc(x, scale[:, 0], torch.zeros(2, dtype=torch.int32))
