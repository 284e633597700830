"""Host-side checks of the serving entry points (no GPU needed): null arguments are refused before
anything is launched, and the Python descriptions refuse tensors that are not on the device."""
import ctypes

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv
from quantized_weight_dequant_gb300.build import build_library


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_library()


@pytest.mark.parametrize("name,struct", [("page_plan", qgemv.PagePlan), ("kv_store", qgemv.KvStore),
                                         ("attn_decode", qgemv.AttnDecode), ("run_lora", qgemv.Lora)])
def test_null_handles_and_descriptions_are_refused(name, struct):
    fn = getattr(qgemv.lib(), "qgemv_" + name)
    assert fn(None, struct(), None) == qgemv.ERR_INVALID_ARG
    assert fn(None, None, None) == qgemv.ERR_INVALID_ARG


def test_the_new_status_has_a_text():
    assert qgemv.status_string(qgemv.ERR_BAD_INDEX) == "a kernel met an index out of range"


def test_structures_have_the_c_layout():
    """Sizes on an LP64 machine: the fields in their order with natural alignment."""
    assert ctypes.sizeof(qgemv.KvCache) == 4 * 8 + 2 * 8 + 5 * 4 + 4
    assert ctypes.sizeof(qgemv.PagePlan) == 13 * 8 + 3 * 4 + 4
    assert ctypes.sizeof(qgemv.KvStore) == ctypes.sizeof(qgemv.KvCache) + 12 * 8 + 6 * 4
    assert ctypes.sizeof(qgemv.AttnDecode) == ctypes.sizeof(qgemv.KvCache) + 8 * 8 + 6 * 4
    assert ctypes.sizeof(qgemv.Lora) == 13 * 8 + 4 * 4


def test_descriptions_refuse_tensors_of_the_host():
    i32 = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 64, dtype=torch.float16)
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        qgemv.kv_cache(cache, cache)
    with pytest.raises(TypeError):
        qgemv.page_plan_desc(i32, i32, i32[:, None], i32, i32[:1], 16, i32, i32.long(), i32)
    with pytest.raises(TypeError):
        qgemv.lora_desc(x, x[None, :1].expand(1, 8, 64).contiguous(), torch.zeros(1, 5, 8).half(), i32, torch.zeros(2, 5))
