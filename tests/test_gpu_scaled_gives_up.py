"""Projections in 8 bits whose waits run out: wherever that happens, the call ends, reports it, and what runs next finds nothing of it.
With a limit of 0 a wait gives up unless it is over at once; with some thousand nanoseconds it does so in the middle of a call."""
import os
import sys

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_scaled as scaled  # noqa: E402

pytestmark = pytest.mark.gpu
h = scaled.h
FEW = [(3, 300, 1024), (3, 40000, 1024), (20, 4096, 4096), (64, 256, 4096), (64, 28672, 640), (1, 4096, 4096)]
MANY = [(65, 300, 1024), (128, 4096, 14336), (300, 4096, 14336), (512, 4096, 4096), (1500, 20000, 640), (4096, 5000, 1040)]
LIMITS = [0, 500, 2_000, 6_000, 20_000, 60_000]


@pytest.mark.parametrize("M,N,K", FEW + MANY)
@pytest.mark.parametrize("stall", [0, 1])
def test_waits_of_any_length_end(h, M, N, K, stall):
    x, xs, W, ws = scaled.operands(scaled.gen(M + N + K), M, N, K)
    want, y = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    good, tried = qgemv.scaled_desc(x, xs, W, ws, want), qgemv.scaled_desc(x, xs, W, ws, y)
    qgemv.run_scaled(h, good)
    torch.cuda.synchronize()
    assert qgemv.check_error(h) == qgemv.OK
    again = torch.empty_like(want)
    for limit in LIMITS:
        qgemv.set_option(h, qgemv.OPT_SPIN_LIMIT_NS, limit)
        qgemv.set_option(h, qgemv.OPT_TEST_STALL, stall)
        try:
            y.fill_(7)
            qgemv.run_scaled(h, tried)
            status = qgemv.check_error(h)
        finally:
            qgemv.set_option(h, qgemv.OPT_TEST_STALL, 0)
            qgemv.set_option(h, qgemv.OPT_SPIN_LIMIT_NS, 1_000_000_000)
        if stall:
            assert status == qgemv.ERR_TIMEOUT
        else:  # either it was in time or it says that it was not
            assert status == qgemv.ERR_TIMEOUT or (status == qgemv.OK and torch.equal(y, want))
        again.fill_(7)
        qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, again))
        assert qgemv.check_error(h) == qgemv.OK and torch.equal(again, want)


@pytest.mark.parametrize("M", [1, 30, 64])
@pytest.mark.parametrize("pdl", [0, 1])
def test_the_kernel_before_does_not_count_as_waiting(h, M, pdl):
    """A projection that is there early, beside a long draw that leaves it room, waits for that one's end without a limit."""
    N, K = 512, 512
    x, xs, W, ws = scaled.operands(scaled.gen(M), M, N, K)
    want, y = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, want))
    logits = torch.randn(2, 1 << 20, device="cuda")  # two clusters, some 100 us
    u, tokens = torch.rand(2, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    draw = qgemv.sample_desc(logits, u, tokens, top_p=torch.full((2,), 0.9, device="cuda"))
    desc = qgemv.scaled_desc(x, xs, W, ws, y)
    qgemv.sample(h, draw)
    assert qgemv.check_error(h) == qgemv.OK
    qgemv.set_option(h, qgemv.OPT_PDL, pdl)
    qgemv.set_option(h, qgemv.OPT_SPIN_LIMIT_NS, 25_000)  # the projection's own waits are below 10 us
    try:
        for _ in range(3):
            qgemv.sample(h, draw)
            qgemv.run_scaled(h, desc)
            assert qgemv.check_error(h) == qgemv.OK
            assert torch.equal(y, want)
    finally:
        qgemv.set_option(h, qgemv.OPT_PDL, 0)
        qgemv.set_option(h, qgemv.OPT_SPIN_LIMIT_NS, 1_000_000_000)
