"""The values of the example's attention block (examples/decode_step.py), each stage against 64 bits on what the stage
before it gave: projections with adapters, rotated and stored rows, attention over what the cache holds, and the
output projection.  Activations of a size that leaves scores of a few units, so that an output is an average of
many tokens and its tolerance is small beside it."""
import os
import sys

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv
from test_gpu_decode_step import turn
from test_gpu_serving import F8, HALF_ULP, TINY, attend_reference, steps, within

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def with_adapters(h, b, x, w, n, k, A, B, ids):
    """A projection and its rows' adapters, and what both kinds of terms add up to."""
    plain = torch.empty(x.shape[0], n, device="cuda")
    qgemv.run_gemm(h, b.fmt, x, x.shape[0], w, n, k, plain)
    y, size = plain.double(), plain.double().abs()
    for t, a in enumerate(ids.tolist()):
        if a >= 0:
            low = A[a].double() @ x[t].double()
            y[t] += B[a].double() @ low
            near = steps(k) * (A[a].double().abs() @ x[t].double().abs()) + (2.0 ** -21 + steps(A.shape[1])) * low.abs()
            size[t] += 2.0 ** 22 * (B[a].double().abs() @ near)
    return y, 2.0 ** -22 * (size + y.abs())


@pytest.mark.parametrize("cache", [torch.float16, torch.uint8])
def test_every_stage_of_a_few_steps(cache):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from decode_step import AttentionBlock
    h = qgemv.create(0)
    R, dim, hq, hk, page = 5, 64, 8, 2, 16
    b = AttentionBlock(h, R, hidden=512, q_heads=hq, kv_heads=hk, dim=dim, adapters=3, rank=8, pages=60, page=page, max_len=256, cache=cache)
    g = torch.Generator(device="cuda").manual_seed(2)
    f8 = cache == torch.uint8

    def stored(where):
        """k and v in 64 bits of the cache's tokens (pages, places)."""
        at = (where[0], slice(None), where[1])
        if f8:
            return [c[at].view(F8).double() * s[at].double()[..., None] for c, s in ((b.k, b.cache.keep[2]), (b.v, b.cache.keep[3]))]
        return [c[at].double() for c in (b.k, b.v)]

    history = [[torch.empty(0, hk, dim, device="cuda", dtype=torch.float64)] * 2 for _ in range(R)]
    unit = None
    for fresh in ([20, 0, 33, 1, 64], [1] * R, [1] * R, [0, 40, 0, 16, 1], [1] * R):
        s = b.plan(torch.tensor(fresh, dtype=torch.int32, device="cuda"), sum(fresh))
        s.x.copy_(torch.randn(s.x.shape, generator=g, device="cuda"))
        s.ids.copy_(torch.randint(-1, 3, s.ids.shape, generator=g, device="cuda"))
        if unit is None:  # the size of x that gives queries and keys of about one
            probe = torch.empty_like(s.qkv)
            qgemv.run_gemm(h, b.fmt, s.x, s.capacity, b.w_qkv, b.n_qkv, b.hidden, probe)
            unit = 1 / float(probe.std())
        s.x.mul_(unit)
        before = b.lens.tolist()
        b.run(s)
        assert qgemv.check_error(h) == qgemv.OK
        y, tol = with_adapters(h, b, s.x, b.w_qkv, b.n_qkv, b.hidden, b.a_qkv, b.b_qkv, s.ids)
        within(s.qkv, y, tol, "qkv")
        # rotated and stored rows, against the projection's own
        rows = s.qkv.double().view(-1, hq + 2 * hk, dim)
        pos = torch.cat([torch.arange(n, n + f, device="cuda") for n, f in zip(before, fresh)])
        q, k, v = turn(rows[:, :hq], pos, dim), turn(rows[:, hq:hq + hk], pos, dim), rows[:, hq + hk:]
        # the angles' cosines and sines are rounded to fp32 and the pairs summed there: 2^-22 of both of a pair
        pair = lambda x: 2.0 ** -22 * (x.abs() + x.abs().roll(dim // 2, -1))  # noqa: E731
        within(s.q, q, 2.0 ** -11 * q.abs() + pair(rows[:, :hq]) + 2.0 ** -25, "q")
        for got, want, slack in zip(stored((s.slots // page, s.slots % page)), (k, v), (pair(rows[:, hq:hq + hk]), 0.0)):
            if f8:  # 3 stored bits, subnormals in steps of 2^-9 of the scale
                within(got, want, (2.0 ** -4 * want.abs() + want.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10) * 1.001 + slack, "stored")
            else:
                within(got, want, 2.0 ** -11 * want.abs() + slack + 2.0 ** -25, "stored")
        at = 0
        for r, f in enumerate(fresh):
            n = before[r] + f
            t = torch.arange(n, device="cuda")
            now = stored((b.table[r].long()[t // page], t % page))
            new = stored((s.slots[at:at + f] // page, s.slots[at:at + f] % page))
            # what was there is there still, and the new tokens follow it
            history[r] = [torch.cat([o, x]) for o, x in zip(history[r], new)]
            assert torch.equal(now[0], history[r][0]) and torch.equal(now[1], history[r][1])
            at += f
            if fresh != [1] * R:
                continue
            for kv in range(hk):
                mine = slice(kv * (hq // hk), (kv + 1) * (hq // hk))
                o, _, pv, qk = attend_reference(s.q[r, mine].double(), now[0][:, kv], now[1][:, kv], b.scale)
                tokens, score = steps(n) + 2.0 ** -20, steps(dim) * qk + 2.0 ** -21 * qk
                tol = HALF_ULP[s.out.dtype] * o.abs() + TINY[s.out.dtype] + (2 * score[:, None] + 2 * tokens + 2.0 ** -16) * pv
                assert (tol <= 2.0 ** -8 * pv).all()  # far below what is averaged
                within(s.out[r, mine], o, tol, f"out of {r}")
        if fresh == [1] * R:
            y, tol = with_adapters(h, b, s.out.view(R, -1), b.w_out, b.hidden, b.n_q, b.a_out, b.b_out, s.ids)
            within(s.y, y, tol, "y")
    h.close()
