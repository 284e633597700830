"""GPU parity of the sampler against a plain one in 64 bits: tokens are equal, log probabilities within the
rounding of fp32 (2^-24 of the value and of the ratio under the logarithm, with a margin of four)."""
import math

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from quantized_weight_dequant_gb300.build import build_library
    build_library()
    handle = qgemv.create(0)
    yield handle
    handle.close()


def reference(logits, u, T=1.0, k=0, p=1.0, low=0.0):
    """One row, all in 64 bits: (token, log probability)."""
    x = logits.double()
    x = torch.where(x.isnan(), -INF, x)
    if not (x > -INF).any():
        return -1, -INF
    by, order = torch.sort(x, descending=True, stable=True)
    if not T > 0:
        return int(order[0]), 0.0
    T = max(T, 2.0 ** -64)
    n = int((by > -INF).sum())
    if 0 < k:
        n = min(n, k)
    w = torch.where(by[:n] == by[0], 1.0, torch.exp((by[:n] - by[0]) / T))
    w = torch.where(w < 2.0 ** -43, 0.0, w)  # weights are whole numbers of 2^-43, rounded down
    if p < 1:
        n = max(1, int((torch.cumsum(w, 0) - w < max(p, 0.0) * w.sum()).sum()))
        w = w[:n]
    if low > 0:
        n = int((w >= min(low, 1.0)).sum())
        w = w[:n]
    index, back = torch.sort(order[:n])
    run = torch.cumsum(w[back], 0)
    u = min(max(u, 0.0), 1.0) if u == u else 0.0
    at = int((run <= u * run[-1]).sum())
    if at >= n:  # u = 1: the last token with a weight
        at = int((w[back] > 0).nonzero()[-1])
    return int(index[at]), math.log(float(w[back][at] / run[-1]))


def draw(h, logits, u, T=None, k=None, p=None, low=None, stream=None, logprobs=True):
    f = lambda v, dtype=torch.float32: None if v is None else torch.tensor(v, dtype=dtype, device="cuda")  # noqa: E731
    rows = logits.shape[0]
    tokens = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), 7.0, device="cuda") if logprobs else None
    qgemv.sample(h, qgemv.sample_desc(logits, f(u), tokens, temperature=f(T), top_k=f(k, torch.int32), top_p=f(p), min_p=f(low),
                                      logprobs=lp), stream=stream)
    torch.cuda.synchronize()
    return tokens.tolist(), lp.tolist() if logprobs else None


def f32(v):
    return [float(x) for x in torch.tensor(v, dtype=torch.float32)]


def check(h, logits, u, T=None, k=None, p=None, low=None):
    tokens, lp = draw(h, logits, u, T, k, p, low)
    x = logits.cpu()
    for r in range(x.shape[0]):
        want, want_lp = reference(x[r], f32(u)[r], f32(T)[r] if T else 1.0, k[r] if k else 0, f32(p)[r] if p else 1.0, f32(low)[r] if low else 0.0)
        assert tokens[r] == want, (r, tokens[r], want, u[r], T and T[r], k and k[r], p and p[r], low and low[r])
        if math.isfinite(want_lp):
            assert abs(lp[r] - want_lp) <= 2.0 ** -22 * (1 + abs(want_lp)), (r, lp[r], want_lp)
        else:
            assert lp[r] == want_lp


def rows_of(seed, rows, V, typ, spread=2.2, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, V, generator=g) * spread + torch.where(torch.rand(rows, V, generator=g) < 0.002, 8.0 * torch.rand(rows, V, generator=g), 0.0)
    base = torch.full((rows, V + pad), 99.0)
    base[:, :V] = x
    return base.to(TYPES[typ]).cuda()[:, :V], g


def settings(g, rows, V):
    rand = lambda: torch.rand(rows, generator=g).tolist()  # noqa: E731
    T = [0.0 if a < 0.1 else 0.3 + 1.5 * b for a, b in zip(rand(), rand())]
    k = [0 if a < 0.3 else 1 + int(V ** b) for a, b in zip(rand(), rand())]
    p = [1.0 if a < 0.3 else b for a, b in zip(rand(), rand())]
    low = [0.0 if a < 0.5 else b * b for a, b in zip(rand(), rand())]
    return dict(u=rand(), T=T, k=k, p=p, low=low)


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V", [(1, 1), (7, 2), (40, 31), (40, 32), (40, 33), (64, 500), (9, 513), (33, 4095), (3, 4097), (5, 8193), (2, 32000),
                                    (13, 50001), (200, 2500), (320, 1000)])
def test_mixed_settings(h, typ, rows, V):
    x, g = rows_of(rows + V, rows, V, typ, pad=V % 3)
    check(h, x, **settings(g, rows, V))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["k", "p", "low", "T", "none"])
def test_one_setting_at_a_time(h, typ, what):
    rows, V = 24, 20000
    x, g = rows_of(3, rows, V, typ)
    s = settings(g, rows, V)
    check(h, x, u=s["u"], **({} if what == "none" else {what: s[what]}))


@pytest.mark.parametrize("V", [1, 5, 64, 5000, 70000])
def test_equal_logits(h, V):
    """Equal logits: cuts and draws go by index."""
    n = 16
    x = torch.full((n, V), -3.25, device="cuda")
    u = [(i + 0.5) / n for i in range(n)]
    tokens, lp = draw(h, x, u)
    assert tokens == [int(V * v) for v in u]
    assert all(abs(v + math.log(V)) < 1e-5 for v in lp)
    k = [1 + i * V // n for i in range(n)]
    tokens, _ = draw(h, x, u, k=k)
    assert tokens == [int(min(a, V) * v) for a, v in zip(k, u)]
    p = [(i + 1) / 32 for i in range(n)]  # a part of V tokens, rounded up
    tokens, _ = draw(h, x, u, p=p)
    assert tokens == [int(math.ceil(V * a) * v) for a, v in zip(p, u)]


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
def test_few_values_many_ties(h, typ):
    rows, V = 32, 9000
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-6, 3, (rows, V), generator=g).to(TYPES[typ]).cuda()
    s = settings(g, rows, V)
    s["p"] = [min(v, 0.97) for v in s["p"]]
    check(h, x, **s)


@pytest.mark.parametrize("V", [40, 3000, 30000])
def test_masks_of_every_kind(h, V):
    """-inf, NaN, the lowest value, +inf, rows with a single token or none."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn(12, V, generator=g) * 2
    x[0, 1:] = -INF
    x[1] = -INF
    x[2] = NAN
    x[3, ::2] = NAN
    x[4, 5:] = torch.finfo(torch.float32).min
    x[5, 3] = INF
    x[6, 3], x[6, 30] = INF, INF
    x[7, :V // 2] = -INF
    x[8] = torch.finfo(torch.float32).min
    x[9] = torch.where(torch.rand(V, generator=g) < 0.9, -INF, x[9])
    x[10] *= 1e30
    x[11] = -0.0
    x[11, 1::2] = 0.0
    x = x.cuda()
    u = [(i * 0.37 + 0.11) % 1 for i in range(12)]
    check(h, x, u)
    check(h, x, u, k=[7] * 12)
    check(h, x, u, p=[0.6] * 12)
    check(h, x, u, k=[V - 1] * 12, p=[0.9] * 12, low=[1e-3] * 12)
    check(h, x, u, T=[0.0] * 12)


def test_settings_at_their_ends(h):
    V = 3000
    x, g = rows_of(1, 1, V, "f32")
    x = x.expand(24, V).contiguous()
    x[:, 100] = 9.5
    x[:, 200] = 9.5
    u = [0.3, 0.0, 1 - 2.0 ** -24, 0.7] * 6
    check(h, x, u, T=[0.0, -1.0, NAN, 1e-30, 2.0 ** -64, 2.0 ** -70, INF, 1e30, 1e-3, 50.0, 0.01, 1e4] * 2)
    check(h, x, u, k=[0, -5, 1, 2, 3, V - 1, V, V + 1, 2 ** 31 - 1, -2 ** 31, 10, 4] * 2)
    check(h, x, u, p=[0.0, -1.0, 1e-30, 2.0 ** -30, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, NAN, INF, 0.999, 1e-3] * 2)
    check(h, x, u, low=[0.0, -1.0, NAN, 1.0, 2.0, INF, 1e-30, 0.5, 1e-9, 1e-4, 0.999, 0.1] * 2)
    check(h, x, u, T=[0.05] * 24, k=[1, 50, 1000, 2999] * 6)


def test_random_numbers_out_of_range(h):
    x = torch.zeros(6, 10, device="cuda")
    x[:, 4] = 1.0
    assert draw(h, x, [-1.0, -INF, NAN, 1.0, 2.0, INF])[0] == [0, 0, 0, 9, 9, 9]


def test_every_draw_of_a_small_row(h):
    """u over a fine grid: each token's share of the draws is its probability."""
    n = 4096
    row = torch.tensor([0.5, -1.0, 2.0, -INF, 2.0, 0.25, 1.0])
    x = row.repeat(n, 1).cuda()
    u = [(i + 0.5) / n for i in range(n)]
    tokens, _ = draw(h, x, u, logprobs=False)
    want = torch.cumsum(torch.softmax(row.double(), 0), 0)
    assert tokens == [int((want <= v).sum()) for v in u]


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_the_longest_rows(h, typ):
    V = 1 << 20
    x, g = rows_of(2, 2, V, typ)
    check(h, x, u=[0.3, 0.8])
    check(h, x, u=[0.6, 0.2], k=[1000, 3], p=[0.9, 1.0])
    check(h, x, u=[0.6, 0.2], p=[0.9, 0.99], T=[1.5, 0.7])
    flat = torch.zeros(1, V, device="cuda")
    assert draw(h, flat, [0.999])[0] == [int(0.999 * V)]


def test_logits_far_apart_and_rows_past_the_grid(h):
    far = 1 << 31
    g = torch.Generator().manual_seed(4)
    x = torch.randn(3, 700, generator=g).half().cuda()
    xf = torch.as_strided(torch.zeros(2 * far + 700, dtype=torch.float16, device="cuda"), (3, 700), (far, 1))
    xf.copy_(x)
    assert draw(h, xf, [0.2, 0.5, 0.9], k=[30, 0, 5]) == draw(h, x, [0.2, 0.5, 0.9], k=[30, 0, 5])
    n = 70000
    many = torch.randn(n, 8, generator=g).cuda()
    assert draw(h, many, [0.0] * n, T=[0.0] * n)[0] == many.argmax(1).tolist()


def test_clusters_of_every_size_agree(h):
    """The same rows alone, a few and many at a time: other splits, the same results."""
    V = 40000
    x, g = rows_of(6, 320, V, "f32")
    s = settings(g, 320, V)
    whole = draw(h, x, **s)
    for rows in (1, 10, 40, 100, 160):
        part = draw(h, x[:rows], **{a: b[:rows] for a, b in s.items()})
        assert part[0] == whole[0][:rows] and part[1] == whole[1][:rows]


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V", [(1, 150000), (40, 60000), (310, 9000)])
def test_large_nuclei(h, typ, rows, V):
    """Nearly all of a row stays: more candidates than lists hold."""
    x, g = rows_of(rows, rows, V, typ, spread=1.0, pad=1)
    u = torch.rand(rows, generator=g).tolist()
    n = list(range(rows))
    check(h, x[:24], u[:24], p=[0.9 + 0.1 * (i % 7) / 7 for i in n][:24])
    check(h, x[:24], u[:24], k=[V - 1 - 97 * i for i in n][:24], p=[0.99] * min(rows, 24), low=[1e-3 * (i % 3) for i in n][:24])
    tokens, lp = draw(h, x, u, p=[0.97] * rows)
    again, lp2 = draw(h, x[:24], u[:24], p=[0.97] * min(rows, 24))
    assert tokens[:24] == again and lp[:24] == lp2


@pytest.mark.parametrize("spread", [1e-4, 0.004, 60.0, 300.0])
@pytest.mark.parametrize("rows,V", [(3, 20000), (310, 7000)])
def test_bf16_values_beyond_the_table(h, spread, rows, V):
    """Logits below 2^-8 or above 2^7 in magnitude, all of them or many, some masked."""
    x, g = rows_of(5, rows, V, "bf16", spread=spread)
    x[:, ::3] = -INF
    u = torch.rand(rows, generator=g).tolist()
    check(h, x[:12], u[:12], T=[0.5 + spread] * min(rows, 12), p=[0.5 + 0.04 * i for i in range(min(rows, 12))])
    check(h, x[:12], u[:12], T=[0.5 + spread] * min(rows, 12))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_top_k_beyond_the_lists(h, typ):
    x, g = rows_of(11, 6, 100000, typ)
    u = torch.rand(6, generator=g).tolist()
    check(h, x, u, k=[4095, 4096, 4097, 20000, 40000, 99999])
    check(h, x, u, k=[257, 512, 2049, 5000, 33000, 70000], p=[0.5, 0.9, 0.99, 0.999, 0.8, 0.95])


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V", [(7, 90), (5, 30000), (320, 6000), (2, 120000)])
def test_several_infinite_logits(h, typ, rows, V):
    """Equal and infinite logits are cut by count, mass and index like finite ones."""
    x, g = rows_of(rows, rows, V, typ)
    at = [V // 7 * i for i in range(1, 6)]
    x[:, at] = INF
    u = [(i % 10 + 0.5) / 10 for i in range(rows)]
    n = min(rows, 12)
    for kw in (dict(), dict(k=[1] * n), dict(k=[2, 3, 600] * n), dict(p=[0.0, 0.3, 0.6, 0.99] * n), dict(k=[4, V - 1] * n, p=[0.5, 0.9, 0.2] * n, low=[1.0] * n)):
        check(h, x[:n], u[:n], **{a: v[:n] for a, v in kw.items()})
    tokens, _ = draw(h, x, u, k=[3] * rows)
    assert tokens == [at[int(3 * v)] for v in u]
