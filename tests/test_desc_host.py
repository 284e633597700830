"""Descriptions of the serving operators and of the layer in 8 bits: sizes past 32 bits are refused where their field has no more."""
import ctypes

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv


class Rows:
    """What a description asks of a device tensor, for sizes that no test allocates."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float16):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


F32, I32 = torch.float32, torch.int32


def norm(N):
    return qgemv.norm_desc(Rows(1, N), None, 1e-5, y=Rows(1, N))


def sample(V):
    return qgemv.sample_desc(Rows(1, V), Rows(1, dtype=F32), Rows(1, dtype=I32))


def cache(pages):
    k = Rows(pages, 1, 16, 64)
    return qgemv.kv_cache(k, k)


def lora(adapters):
    return qgemv.lora_desc(Rows(1, 64), Rows(adapters, 8, 64), Rows(adapters, 32, 8), Rows(1, dtype=I32), Rows(1, 32))


@pytest.mark.parametrize("make,field", [(norm, "N"), (sample, "V"), (cache, "pages"), (lora, "adapters")])
def test_sizes_past_32_bits_are_refused(make, field):
    assert getattr(make(4096), field) == 4096
    assert getattr(make((1 << 31) - 1), field) == (1 << 31) - 1  # the library refuses what it cannot do
    for n in (1 << 31, (1 << 32) + 4096, 1 << 40):
        with pytest.raises(ValueError, match="32 bits"):
            make(n)


def test_fields_by_name_are_checked_too():
    assert qgemv.Sample(V=5).V == 5 and qgemv.Norm().N == 0
    with pytest.raises(ValueError):
        qgemv.Sample(V=(1 << 32) + 5)
    assert issubclass(qgemv.Scaled, ctypes.Structure) and qgemv.Scaled(N=1 << 32).N == 1 << 32  # 64 bits there
