"""Draws whose candidates do not fit where they are looked for first: lists that overflow, candidates in one part of the row alone, cuts
that ask for more tokens than a mask has left.  Against the plain sampler in 64 bits, with its tolerances."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_sample as plain  # noqa: E402

pytestmark = pytest.mark.gpu
h = plain.h
INF = float("inf")
ROWS = [1, 40, 310]  # rows of eight CTAs, of four and of one


def check_first(h, x, u, n=8, **kw):
    """The first n rows against the plain sampler, all rows drawn."""
    rows = x.shape[0]
    full = {a: [v[i % len(v)] for i in range(rows)] for a, v in kw.items()}
    got = plain.draw(h, x, u, **full)
    n = min(n, rows)
    plain.check(h, x[:n], u[:n], **{a: v[:n] for a, v in full.items()})
    again = plain.draw(h, x[:n], u[:n], **{a: v[:n] for a, v in full.items()})
    assert got[0][:n] == again[0] and got[1][:n] == again[1]


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", ROWS)
def test_first_lists_that_overflow(h, typ, rows):
    """Hardly any spread: thousands of tokens share the bucket of the k-th, and the exact cut's list comes after one that was too long."""
    V = 60000 if rows < 300 else 20000
    x, g = plain.rows_of(rows, rows, V, typ, spread=1e-3)
    x[:, ::500] += 0.03125
    u = torch.rand(rows, generator=g).tolist()
    check_first(h, x, u, k=[50, 3, 400, 1], T=[1.0, 30.0, 5.0, 0.7])
    check_first(h, x, u, k=[50, 300, 256], p=[0.9, 0.4, 0.99, 1.0])
    check_first(h, x, u, k=[60, 7], p=[0.5, 0.97, 0.8], low=[0.99, 0.0], T=[2.0, 40.0, 0.05])


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("part", [0, 3, 7])
def test_what_a_mask_leaves_is_one_range(h, typ, rows, part):
    """One CTA of the cluster has all candidates, more than its list holds and fewer than all lists together."""
    V = 120000 if rows < 300 else 24000
    x, g = plain.rows_of(rows + part, rows, V, typ, spread=1.0)
    x[:, :part * V // 8] = -INF
    x[:, (part + 1) * V // 8:] = -INF
    u = torch.rand(rows, generator=g).tolist()
    check_first(h, x, u, p=[0.9, 0.5, 0.99, 0.7])
    check_first(h, x, u, p=[0.9, 0.6], T=[2.0, 8.0, 0.8], low=[0.0, 0.01, 0.2])
    check_first(h, x, u, k=[10000, 4500, 2000], p=[0.95, 0.8])
    check_first(h, x, u, k=[4097, 9000])
    check_first(h, x, u, k=[255, 1000, 60], p=[0.9, 1.0, 0.5])  # most threads have no token, the others all of them


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("left", [1, 9, 300, 5000])
def test_more_asked_for_than_a_mask_has_left(h, typ, rows, left):
    V = 50000 if rows < 300 else 9000
    x, g = plain.rows_of(rows + left, rows, V, typ)
    far = torch.rand(rows, V, generator=g).cuda()
    x.masked_fill_(far > far.kthvalue(min(left, V - 1), dim=1, keepdim=True).values, -INF)
    u = torch.rand(rows, generator=g).tolist()
    for k in ([left + 1, 2 * left + 7, V - 1], [max(1, left - 1), left, left + 1]):
        check_first(h, x, u, k=k)
        check_first(h, x, u, k=k, p=[0.9, 1.0, 0.3, 0.999], low=[0.0, 0.05])
    x[:, 77] = INF  # one infinite logit: all others weigh nothing
    check_first(h, x, u, k=[left + 1, 2], p=[0.9, 1.0])
