"""Log probabilities of tokens that are nearly certain, relative to themselves: log(p) close to 0 is what the other tokens have.

Tolerance: the share in fp32 half an ulp, the logarithm two ulps, below 2^-22 of the value; the other tokens' weights to 2^-32 of
themselves and rounded down to 2^-43 of the largest, V 2^-43 in all."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_sample as plain  # noqa: E402

pytestmark = pytest.mark.gpu
h = plain.h


@pytest.mark.parametrize("V", [2, 50, 5000, 60000])
@pytest.mark.parametrize("far", [0.1, 1.0, 4.0, 9.0, 16.0, 20.0])
def test_nearly_certain_tokens(h, V, far):
    g = torch.Generator().manual_seed(V)
    rows = 6
    x = torch.rand(rows, V, generator=g) * 2 - far - math.log(V)
    x[:, V // 2] = 2.0
    u = [0.5] * rows
    k = [0, V, min(V, 2), 0, min(V, 200), min(V, 3000)]
    p = [1.0, 1.0, 1.0, 1.0 - 2.0 ** -24, 1.0, 0.99999988]
    tokens, lp = plain.draw(h, x.cuda(), u, k=k, p=p)
    for r in range(rows):
        want, want_lp = plain.reference(x[r], 0.5, 1.0, k[r], plain.f32(p)[r])
        by = torch.sort(x[r].double(), descending=True).values[:k[r] or V]
        w = torch.exp(by - by[0])
        if p[r] < 1:
            w = w[:max(1, int((torch.cumsum(w, 0) - w < plain.f32(p)[r] * w.sum()).sum()))]
        if want == V // 2:  # (the reference's quotient loses what is missing from 1, too)
            want_lp = math.log1p(-float(w[1:].sum() / w.sum())) if len(w) > 1 else 0.0
        assert tokens[r] == want
        assert abs(lp[r] - want_lp) <= abs(want_lp) * 2.0 ** -22 + V * 2.0 ** -43, (r, lp[r], want_lp)
