"""The operators of the MLP in 8 bits and of the next token in a row, as a decode step runs them: each stage against the plain
implementation of what it was given, and the run captured in a graph, with dependent launches, on another stream and beside a
second handle against the same run alone, bit for bit."""
import os
import sys

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import test_gpu_sample as tokens  # noqa: E402
import test_gpu_scaled as scaled  # noqa: E402

pytestmark = pytest.mark.gpu
h = scaled.h
BF16 = torch.bfloat16


def block(h, rows, hidden=512, inner=640, vocab=1000, residual=BF16, seed=0):
    from decode_step import TokenBlock
    g = scaled.gen(seed + rows)
    attended = scaled.randn(g, rows, hidden)
    b = TokenBlock(h, attended, inner, vocab, residual, seed)
    b.attended, b.before = attended, (scaled.randn(g, rows, hidden) * 2).to(residual)
    b.u.copy_(torch.rand(rows, generator=g, device="cuda"))
    b.temperature.copy_(0.5 + torch.rand(rows, generator=g, device="cuda"))
    b.top_p.copy_(0.5 + 0.6 * torch.rand(rows, generator=g, device="cuda"))
    b.top_k.copy_(torch.randint(-20, 50, (rows,), generator=g, device="cuda"))
    return b


def results(b):
    return [t.clone() for t in (b.hidden, b.x[0].view(torch.uint8), b.x[1], b.gate_up, b.act[0].view(torch.uint8), b.act[1], b.down, b.last[0].view(torch.uint8),
                                b.last[1], b.logits, b.tokens, b.logprobs)]


def run(b):
    b.hidden.copy_(b.before)
    b.run()
    torch.cuda.synchronize()
    return results(b)


def same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def normed(t, w):
    return t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-5) * w.double()


@pytest.mark.parametrize("rows", [1, 5, 64, 130])
@pytest.mark.parametrize("residual", [BF16, torch.float32])
def test_every_stage(h, rows, residual):
    b = block(h, rows, residual=residual)
    inner = b.act[0].shape[1]
    b.hidden.copy_(b.before)
    stages = []
    for call, desc in b.calls:
        call(h, desc)
        torch.cuda.synchronize()
        stages.append(b.hidden.clone())
    half = scaled.HALF_ULP[residual] * 1.01 + 2.0 ** -24
    first = b.attended.double() + b.before.double()
    scaled.within(stages[0], first, first.abs() * half, "residual")
    scaled.check_codes(b.x[0].view(torch.uint8), b.x[1], normed(first, b.n_mlp), 2.0 ** -18, "norm")
    for x, w, y in ((b.x, b.w_up, b.gate_up), (b.act, b.w_down, b.down), (b.last, b.w_head, b.logits)):
        ref, size = scaled.projection_reference(x[0].view(torch.uint8), x[1], w[0].view(torch.uint8), w[1])
        scaled.within(y, ref, scaled.projection_tolerance(ref, size, x[0].shape[1], BF16), "projection")
    gate, up = b.gate_up.double().split(inner, 1)
    scaled.check_codes(b.act[0].view(torch.uint8), b.act[1], gate / (1 + torch.exp(-gate)) * up, 2.0 ** -20, "gated")
    second = b.down.double() + stages[0].double()
    scaled.within(b.hidden, second, second.abs() * half, "residual")
    scaled.check_codes(b.last[0].view(torch.uint8), b.last[1], normed(second, b.n_last), 2.0 ** -18, "last norm")
    logits = b.logits.cpu()
    for r in range(rows):
        want, lp = tokens.reference(logits[r], *(float(t[r]) for t in (b.u, b.temperature)), int(b.top_k[r]), float(b.top_p[r]))
        assert int(b.tokens[r]) == want and abs(float(b.logprobs[r]) - lp) <= 2.0 ** -22 * (1 + abs(lp))


@pytest.mark.parametrize("rows", [1, 7, 70])
@pytest.mark.parametrize("pdl", [0, 1])
def test_replayed_runs_are_the_eager_ones(h, rows, pdl):
    b = block(h, rows, vocab=9000)
    qgemv.set_option(h, qgemv.OPT_PDL, pdl)
    try:
        run(b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.run()
            b.run()  # the second takes up what the first left
        for seed in range(3):
            g = scaled.gen(100 + seed)
            b.attended.copy_(scaled.randn(g, *b.attended.shape))
            b.u.copy_(torch.rand(rows, generator=g, device="cuda"))
            qgemv.set_option(h, qgemv.OPT_PDL, 0)
            b.hidden.copy_(b.before)
            b.run()
            b.run()
            torch.cuda.synchronize()
            want = results(b)
            b.tokens.fill_(-7)
            b.hidden.copy_(b.before)
            graph.replay()
            torch.cuda.synchronize()
            same(want, results(b))
    finally:
        qgemv.set_option(h, qgemv.OPT_PDL, 0)
    assert qgemv.check_error(h) == qgemv.OK


def test_two_handles_and_two_streams_at_once(h):
    """Nothing is shared between calls: two graphs of one handle and a run of another, all at once, many times."""
    other = qgemv.create(0)
    blocks = [block(h, 40, seed=1), block(h, 90, seed=2), block(other, 3, vocab=40000, seed=3)]
    want = [run(b) for b in blocks]
    graphs = []
    for b in blocks[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.hidden.copy_(b.before)
            b.run()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in blocks]
    for b in blocks:
        b.tokens.fill_(-7)
    torch.cuda.synchronize()
    for _ in range(20):
        for i, b in enumerate(blocks):
            with torch.cuda.stream(streams[i]):
                if i < 2:
                    graphs[i].replay()
                else:
                    b.hidden.copy_(b.before)
                    b.run()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        same(w, results(b))
    assert qgemv.check_error(h) == qgemv.OK and qgemv.check_error(other) == qgemv.OK
    other.close()


def test_calls_on_a_named_stream(h):
    b = block(h, 6)
    want = run(b)
    b.tokens.fill_(-7)
    b.hidden.copy_(b.before)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for call, desc in b.calls:
        call(h, desc, stream=s.cuda_stream)
    s.synchronize()
    same(want, results(b))


@pytest.mark.parametrize("M,N,K", [(3, 300, 1024), (3, 40000, 1024), (64, 256, 4096), (300, 600, 2048), (1000, 4096, 512)])
def test_a_projection_that_gives_up_waiting_reports_it_and_recovers(h, M, N, K):
    want = scaled.run_projection(h, M, N, K)
    x, xs, W, ws = scaled.operands(scaled.gen(M + 3 * N + 7 * K), M, N, K)
    y = torch.empty(M, N, device="cuda")
    qgemv.set_option(h, qgemv.OPT_SPIN_LIMIT_NS, 2_000_000)
    qgemv.set_option(h, qgemv.OPT_TEST_STALL, 1)
    try:
        qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, y))
        torch.cuda.synchronize()
        assert qgemv.check_error(h) == qgemv.ERR_TIMEOUT
    finally:
        qgemv.set_option(h, qgemv.OPT_TEST_STALL, 0)
        qgemv.set_option(h, qgemv.OPT_SPIN_LIMIT_NS, 1_000_000_000)
    got = scaled.run_projection(h, M, N, K)
    assert qgemv.check_error(h) == qgemv.OK
    assert torch.equal(want, got)
