"""Projections in 8 bits by every kernel and launch that the library chooses among: tiles of every size, shared by several CTAs or not,
several to a pair of CTAs, with remainders of rows, columns and blocks, odd strides of y and scales that are not 16-byte aligned.
Against the plain projection in 64 bits, with its tolerances."""
import os
import re
import sys

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_scaled as scaled  # noqa: E402

pytestmark = pytest.mark.gpu
h = scaled.h
F8, INF = scaled.F8, float("inf")

FEW = [(1, 300, 1040), (1, 40000, 640), (30, 1000, 4096), (31, 33000, 400), (64, 500, 2064), (33, 40000, 528)]
MANY = [(4096, 5000, 1040), (1500, 20000, 640), (200, 40000, 256), (257, 19500, 384), (66, 28672, 4096),  # several tiles to a pair
        (300, 4096, 14336), (512, 4096, 14336), (300, 4000, 14000), (129, 4100, 12288),                   # 256 columns, shared
        (128, 4096, 14336), (300, 600, 2048), (300, 2000, 9008), (65, 100, 5008),                         # shared by two to four pairs
        (65, 12000, 512), (700, 5000, 512), (129, 10000, 2048), (2500, 1000, 5008), (513, 4096, 4096), (512, 4096, 4096)]    # one to a pair


def plan(h, M, N, K):
    words = dict(w.split("=") for w in qgemv.describe_scaled(h, M, N, K).split())
    return words.pop("path"), {a: int(b) for a, b in words.items()}


def kind(h, M, N, K):
    path, p = plan(h, M, N, K)
    several = path == "many" and p["share"] == 1 and p["tiles"] > p["ctas"] // 2
    return path, p["rows"] if path == "few" else p["columns"], "shared" if p["share"] > 1 else "several" if several else "single"


def test_the_shapes_reach_every_launch(h):
    want = {("few", rows, s) for rows in (16, 32, 64) for s in ("single", "shared")}
    want |= {("many", columns, s) for columns in (128, 256) for s in ("single", "several", "shared")}
    assert {kind(h, *c) for c in FEW + MANY} == want
    shares = {(kind(h, *c)[1], plan(h, *c)[1]["share"]) for c in MANY}
    assert len([s for s in shares if s[1] > 1]) >= 3


def test_descriptions(h):
    path, p = plan(h, 5, 1000, 4096)
    assert path == "few" and p["rows"] == 16 and p["columns"] == 128 and p["tiles"] == 8 and p["ctas"] == 8 * p["share"]
    path, p = plan(h, 4096, 28672, 4096)
    assert path == "many" and p["tiles"] == 16 * (28672 // p["columns"]) and p["ctas"] % 2 == 0
    assert qgemv.describe_scaled(h, 0, 5, 16) == "path=none"
    for M, N, K in ((-1, 1, 16), (1, 0, 16), (1, 1, 8), (1, 1, 24), (1 << 31, 1, 16), (1, 1 << 31, 16), ((1 << 31) - 1, (1 << 31) - 1, 16)):
        with pytest.raises(qgemv.QgemvError):
            qgemv.describe_scaled(h, M, N, K)
    assert re.match(r"path=\w+ rows=\d+", qgemv.describe_scaled(h, 1 << 20, 1 << 10, 1 << 20))


@pytest.mark.parametrize("M,N,K", FEW + MANY)
@pytest.mark.parametrize("typ,pad,y_pad", [("f32", 0, 0), ("bf16", 16, 3), ("f16", 16, 8)])
def test_every_launch(h, M, N, K, typ, pad, y_pad):
    scaled.run_projection(h, M, N, K, typ, pad=pad, y_pad=y_pad, seed=1)


@pytest.mark.parametrize("M,N,K", FEW + MANY)
def test_repeated_calls_are_equal_and_nan_stays_in_its_rows(h, M, N, K):
    g = scaled.gen(M + N)
    x, xs, W, ws = scaled.operands(g, M, N, K)
    ys = [torch.empty(M, N, device="cuda") for _ in range(3)]
    for y in ys:
        qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, y))
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
    x[M // 2, K - 3] = 0x7f
    W[N - 2, K - 1] = 0xff
    W[N // 3, 0] = 0x7f
    xs[M - 1, xs.shape[1] - 1] = INF
    qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, ys[1]))
    torch.cuda.synchronize()
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[M // 2], bad[:, N - 2], bad[:, N // 3], bad[M - 1] = True, True, True, True
    assert torch.equal(ys[1][~bad], ys[0][~bad]) and not ys[1][bad].isfinite().any()


@pytest.mark.parametrize("M,N,K", [(1, 300, 1040), (33, 40000, 528), (1500, 20000, 640), (300, 4000, 14000), (200, 40000, 256)])
def test_captured_and_replayed(h, M, N, K):
    """Beside eager calls of the same handle on another stream, with and without early weights."""
    g = scaled.gen(K)
    x, xs, W, ws = scaled.operands(g, M, N, K)
    want, y, other = (torch.empty(M, N, device="cuda") for _ in range(3))
    qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, want))
    torch.cuda.synchronize()
    desc, beside = qgemv.scaled_desc(x, xs, W, ws, y), qgemv.scaled_desc(x, xs, W, ws, other)
    stream = torch.cuda.Stream()
    for pdl in (0, 1):
        qgemv.set_option(h, qgemv.OPT_PDL, pdl)
        try:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                qgemv.run_scaled(h, desc)
                qgemv.run_scaled(h, desc)
            y.fill_(7), other.fill_(7)
            torch.cuda.synchronize()
            for _ in range(5):
                graph.replay()
                qgemv.run_scaled(h, beside, stream=stream)
            torch.cuda.synchronize()
        finally:
            qgemv.set_option(h, qgemv.OPT_PDL, 0)
        assert torch.equal(y, want) and torch.equal(other, want) and qgemv.check_error(h) == qgemv.OK
