"""GPU parity of the row operators (norm with residual, quantisation) and of the 8-bit projection against plain
implementations in 64 bits.  Tolerances are derived from the arithmetic:
  * norm: a sum of N squares is taken in chains of at most 64 and a tree of at most 12 steps: below 80 roundings
    of 2^-24, halved by the root; with the residual's, the root's, the reciprocal's and the products' roundings
    below 2^-18 of a value in all, then half an ulp of the output;
  * codes: half a step of e4m3, 2^-4 of the value or half the smallest step (2^-10 of the scale);
  * projection: products are exact; a matrix instruction sums 32 of them and the accumulator with an error below
    2^-21 of their absolute sum, four to a block: 2^-19, then 2^-24 for each of the block's scalings and sums."""
import math

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float(err[bad].max())} against "
                           f"{float(tol.expand_as(err)[bad].max())} at {bad.nonzero()[0].tolist()}")


def wide(rows, cols, pad, dtype, fill=0):
    """[rows, cols] inside rows of cols + pad elements, and all of it."""
    base = torch.full((rows, cols + pad), fill, dtype=torch.float32, device="cuda").to(dtype)
    return base[:, :cols], base


def blocks(x):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 128)).reshape(x.shape[0], -1, 128)


def check_codes(codes, scale, ref, rel, what):
    """Codes and scales against the values `ref`, of which the kernel's differ by `rel` at most."""
    top = blocks(ref).abs().amax(-1)
    want = torch.where(top > 0, top / 448.0, 1.0).clamp(min=2.0 ** -126)
    within(scale, want, want * (rel + 2.0 ** -23), what + " scale")
    s = scale.double().repeat_interleave(128, 1)[:, :ref.shape[1]]
    within(codes.view(F8).double() * s, ref, ref.abs() * (2.0 ** -4 + 2 * rel + 2.0 ** -22) + s * 2.0 ** -10, what + " codes")


# ------------------------------------------------------------------------------------ norm
def run_norm(h, rows, N, x="bf16", res="bf16", w="bf16", y="bf16", codes=True, pad=0, seed=0, offset=0.0, eps=1e-5, stream=None):
    g = gen(seed + 31 * rows + N)
    xv, _ = wide(rows, N, pad, TYPES[x])
    xv.copy_(randn(g, rows, N) * torch.exp(randn(g, rows, 1)))
    rv = ro = None
    if res:
        rv, _ = wide(rows, N, 2 * pad, TYPES[res])
        rv.copy_(randn(g, rows, N) * 3)
        ro, ro_all = wide(rows, N, pad, TYPES[res], 7)
    wv = (1 + 0.3 * randn(g, N)).to(TYPES[w]) if w else None
    yv = y_all = cv = c_all = sv = s_all = None
    if y:
        yv, y_all = wide(rows, N, pad, TYPES[y], 7)
    if codes:
        cv, c_all = wide(rows, N, 2 * pad, torch.uint8, 7)
        sv, s_all = wide(rows, -(-N // 128), 3 if pad else 0, torch.float32, 7)
    t = xv.double() + (rv.double() if res else 0)
    ref = t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)
    if w:
        ref = ref * (offset + wv.double())
    qgemv.run_norm(h, qgemv.norm_desc(xv, wv, eps, y=yv, codes=cv, scale=sv, res=rv, res_out=ro, offset=offset), stream=stream)
    torch.cuda.synchronize()
    what = f"norm {rows} x {N}"
    if res:
        within(ro, t, t.abs() * (HALF_ULP[TYPES[res]] * 1.01 + 2.0 ** -24) + TINY[TYPES[res]], what + " sum")
        assert (ro_all[:, N:] == 7).all()
    if y:
        within(yv, ref, ref.abs() * (HALF_ULP[TYPES[y]] * 1.01 + 2.0 ** -18) + TINY[TYPES[y]], what)
        assert (y_all[:, N:] == 7).all()
    if codes:
        check_codes(cv, sv, ref, 2.0 ** -18, what)
        assert (c_all[:, N:] == 7).all() and (s_all[:, -(-N // 128):] == 7).all()


@pytest.mark.parametrize("N", [16, 64, 112, 128, 144, 256, 272, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 14336, 16400, 40960, 65536])
@pytest.mark.parametrize("rows", [1, 5])
def test_norm_widths(h, rows, N):
    run_norm(h, rows, N)
    run_norm(h, rows, N, x="f32", res="f32", w="f32", y="f32", pad=16, seed=1)


@pytest.mark.parametrize("N", [8, 24, 136, 2056, 4104, 65528])
def test_norm_without_codes(h, N):
    run_norm(h, 7, N, codes=False)
    run_norm(h, 2, N, codes=False, x="f16", res="", y="f32", pad=8)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("res", ["", "f32", "f16", "bf16"])
@pytest.mark.parametrize("w", ["", "f32", "f16", "bf16"])
@pytest.mark.parametrize("y", ["", "f32", "f16", "bf16"])
def test_norm_types(h, x, res, w, y):
    run_norm(h, 9, 1040, x, res, w, y, pad=16, offset=1.0 if w == "f16" else 0.0)
    run_norm(h, 3, 4112, x, res, w, y)


def test_norm_many_rows(h):
    run_norm(h, 2111, 4096, y="")
    run_norm(h, 70001, 128, codes=False)
    run_norm(h, 1000, 8192, x="f32", res="bf16", y="f16")


def test_norm_in_place(h):
    g = gen(5)
    for N in (256, 4096):
        x, res = randn(g, 6, N).bfloat16(), randn(g, 6, N).bfloat16()
        w = randn(g, N).bfloat16()
        y, total = torch.empty_like(x), torch.empty_like(res)
        qgemv.run_norm(h, qgemv.norm_desc(x, w, 1e-6, y=y, res=res, res_out=total))
        x1, res1 = x.clone(), res.clone()
        qgemv.run_norm(h, qgemv.norm_desc(x1, w, 1e-6, y=x1, res=res1, res_out=res1))
        x2, res2 = x.clone(), res.clone()
        qgemv.run_norm(h, qgemv.norm_desc(x2, w, 1e-6, y=res2, res=res2, res_out=x2))
        torch.cuda.synchronize()
        assert torch.equal(x1, y) and torch.equal(res1, total)
        assert torch.equal(res2, y) and torch.equal(x2, total)


def test_norm_of_zeros_infinities_and_nan(h):
    for N in (256, 4096):
        x = torch.zeros(4, N, dtype=torch.float32, device="cuda")
        x[1, 3], x[2, 5], x[3] = INF, NAN, 1e-30
        y = torch.empty_like(x)
        codes, scale = torch.empty(4, N, dtype=F8, device="cuda"), torch.empty(4, N // 128, device="cuda")
        qgemv.run_norm(h, qgemv.norm_desc(x, None, 1e-6, y=y, codes=codes, scale=scale))
        torch.cuda.synchronize()
        assert (y[0] == 0).all() and (codes[0].float() == 0).all() and (scale[0] == 1).all()
        assert y[1, 3].isnan() and (y[1, 4:] == 0).all() and y[2].isnan().all()
        assert scale[1, 0] == 1 and codes[1, 3].float().isnan() and codes[2].float().isnan().all()
        within(y[3], torch.full((N,), 1e-27, dtype=torch.float64, device="cuda"), torch.tensor(1e-33, device="cuda"), "small rows")


# ------------------------------------------------------------------------------------ quantisation
def quantise(h, x, up=None, pad=0):
    rows, N = x.shape
    codes, c_all = wide(rows, N, pad, torch.uint8, 7)
    scale, s_all = wide(rows, -(-N // 128), 1 if pad else 0, torch.float32, 7)
    qgemv.quant_rows(h, qgemv.quant_desc(x, codes, scale, up=up))
    torch.cuda.synchronize()
    assert (c_all[:, N:] == 7).all() and (s_all[:, scale.shape[1]:] == 7).all()
    return codes, scale


@pytest.mark.parametrize("rows,N", [(1, 16), (3, 64), (2, 128), (5, 144), (7, 1040), (64, 14336), (1, 4096), (333, 2064), (40000, 48), (2, 200000)])
@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
def test_quantised_rows_are_the_rounded_quotients(h, rows, N, typ):
    g = gen(rows + N)
    x, _ = wide(rows, N, 32, TYPES[typ])
    x.copy_(randn(g, rows, N) * torch.exp(2 * randn(g, rows, 1)))
    if rows > 1:
        x[1, :min(128, N)] = 0
    codes, scale = quantise(h, x, pad=16)
    top = blocks(x.float()).abs().amax(-1)
    # rounded once (a division of fp32 by a number is a product with its reciprocal on the GPU): 53 bits are more than
    # twice 24 and two, so that the second rounding of the quotient changes nothing
    want = torch.where(top > 0, (top.double() / 448.0).float(), 1.0)
    assert torch.equal(scale, want)
    q = x.float() / want.repeat_interleave(128, 1)[:, :N]
    assert torch.equal(codes.view(F8).float(), q.to(F8).float())


@pytest.mark.parametrize("rows,N", [(1, 16), (5, 144), (64, 14336), (9, 2064), (1300, 6144)])
@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
def test_gated_rows(h, rows, N, typ):
    """silu(g) u: the exponential within 2 ulp, a sum, a quotient and a product: below 2^-20 of it."""
    g = gen(3 * rows + N)
    both = (randn(g, rows, 2 * N) * 4).to(TYPES[typ])
    both[0, 0], both[0, 1] = -80.0, 60.0
    codes, scale = quantise(h, both[:, :N], both[:, N:], pad=32)
    gate, up = both[:, :N].double(), both[:, N:].double()
    check_codes(codes, scale, gate / (1 + torch.exp(-gate)) * up, 2.0 ** -20, f"gated {rows} x {N}")


def test_quantised_infinities_nan_and_small_rows(h):
    x = torch.ones(4, 384, device="cuda")
    x[0, 5], x[1, 130], x[2, 260], x[3] = INF, -INF, NAN, 1e-41
    codes, scale = quantise(h, x)
    c = codes.view(F8).float()
    assert torch.equal(scale[0], torch.tensor([1, 1 / 448, 1 / 448], device="cuda"))
    assert c[0, 5] == 448 and c[0, 6] == 1 and c[1, 130] == -448 and scale[1, 1] == 1
    assert c[2, 260].isnan() and c[2, 261] == 1 and scale[2, 2] == 1 and (c[2, :256] == 448).all()
    assert (scale[3] == 2.0 ** -126).all() and (c[3] == 0).all()
    big = torch.full((1, 128), -200.0, device="cuda")  # e^200 is infinite: -0
    codes, scale = quantise(h, big, big)
    assert (codes.view(F8).float() == 0).all() and (scale == 1).all()


# ------------------------------------------------------------------------------------ projection
def operands(g, M, N, K, pad=0):
    x, _ = wide(M, K, pad, torch.uint8)
    x.copy_((randn(g, M, K) * 60).clamp(-448, 448).to(F8).view(torch.uint8))
    W = (randn(g, N, K) * 60).clamp(-448, 448).to(F8).view(torch.uint8)
    xs, _ = wide(M, -(-K // 128), 3 if pad else 0, torch.float32)
    xs.copy_(torch.exp(randn(g, M, -(-K // 128))) * 1e-2)
    ws = torch.exp(randn(g, -(-N // 128), -(-K // 128))) * 1e-3
    return x, xs, W, ws


def projection_reference(x, xs, W, ws):
    a = x.view(F8).double() * xs.double().repeat_interleave(128, 1)[:, :x.shape[1]]
    b = W.view(F8).double() * ws.double().repeat_interleave(128, 0)[:W.shape[0]].repeat_interleave(128, 1)[:, :W.shape[1]]
    return a @ b.t(), a.abs() @ b.abs().t()


def projection_tolerance(ref, size, K, typ):
    return size * (2.0 ** -19 + (-(-K // 128) + 4) * 2.0 ** -24) + ref.abs() * HALF_ULP[typ] * 1.01 + TINY[typ]


def run_projection(h, M, N, K, typ="f32", pad=0, y_pad=0, seed=0, stream=None):
    g = gen(seed + M + 3 * N + 7 * K)
    x, xs, W, ws = operands(g, M, N, K, pad)
    y, y_all = wide(M, N, y_pad, TYPES[typ], 7)
    qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, y), stream=stream)
    torch.cuda.synchronize()
    ref, size = projection_reference(x, xs, W, ws)
    within(y, ref, projection_tolerance(ref, size, K, TYPES[typ]), f"projection {M} x {N} x {K}")
    assert (y_all[:, N:] == 7).all()
    return y


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 257, 300])
@pytest.mark.parametrize("N,K", [(256, 512), (200, 400)])
def test_projection_rows(h, M, N, K):
    run_projection(h, M, N, K)


@pytest.mark.parametrize("N,K", [(1, 16), (1, 4096), (3, 112), (127, 128), (128, 144), (129, 256), (77, 2064), (1000, 1040), (4096, 128), (130, 16384),
                                 (513, 5000 // 16 * 16), (6144, 1024)])
@pytest.mark.parametrize("M", [1, 5, 37, 150])
@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
def test_projection_shapes(h, M, N, K, typ):
    run_projection(h, M, N, K, typ, pad=16, y_pad=3)


@pytest.mark.parametrize("M,N,K,typ", [(64, 28672, 4096, "bf16"), (37, 4096, 14336, "f32"), (1, 4096, 4096, "f32"), (1000, 4096, 1024, "bf16"),
                                       (513, 6144, 4096, "f16"), (2048, 1000, 1040, "f32"), (4100, 512, 256, "bf16"), (1, 28672, 4096, "f16")])
def test_projection_sizes(h, M, N, K, typ):
    run_projection(h, M, N, K, typ)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_projection_scales_of_very_different_size(h, M):
    """Blocks 2^100 apart, and scales of zero: what a small block adds is not lost for its own rows."""
    N, K = 300, 640
    g = gen(M)
    x, xs, W, ws = operands(g, M, N, K)
    xs[:, 1] *= 2.0 ** -60
    ws[0] *= 2.0 ** -40
    xs[:, 2] = 0
    xs[0] *= 2.0 ** 50
    y = torch.empty(M, N, device="cuda")
    qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, y))
    torch.cuda.synchronize()
    ref, size = projection_reference(x, xs, W, ws)
    within(y, ref, projection_tolerance(ref, size, K, torch.float32), "projection")


@pytest.mark.parametrize("M", [1, 3, 40, 300])
@pytest.mark.parametrize("N,K", [(300, 640), (512, 4096)])
def test_projection_keeps_nan_and_infinities_to_their_rows(h, M, N, K):
    g = gen(M)
    x, xs, W, ws = operands(g, M, N, K)
    y, y2 = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, y))
    x2, W2, ws2, xs2 = x.clone(), W.clone(), ws.clone(), xs.clone()
    x2[M // 2, 5] = 0x7f
    W2[17, 300] = 0xff
    xs2[M - 1, 3] = INF
    qgemv.run_scaled(h, qgemv.scaled_desc(x2, xs2, W2, ws2, y2))
    torch.cuda.synchronize()
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[M // 2], bad[:, 17], bad[M - 1] = True, True, True
    assert torch.equal(y2[~bad], y[~bad])
    assert y2[M // 2].isnan().all() and y2[:, 17].isnan().all() and (~y2[M - 1].isfinite()).all()


def test_projection_is_deterministic(h):
    for M, N, K in ((1, 4096, 4096), (33, 2000, 8192), (130, 1000, 2048), (600, 3000 // 16 * 16, 1024)):
        g = gen(M)
        x, xs, W, ws = operands(g, M, N, K)
        ys = [torch.empty(M, N, device="cuda") for _ in range(4)]
        for y in ys:
            qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, y))
        torch.cuda.synchronize()
        assert all(torch.equal(y, ys[0]) for y in ys[1:])


def test_projection_of_rows_far_apart(h):
    """Rows of x, its scales and y whose offsets pass 2^32 elements."""
    M, N, K, far = 3, 96, 256, 1 << 31
    g = gen(1)
    x, xs, W, ws = operands(g, M, N, K)
    big = torch.zeros(2 * far + K, dtype=torch.uint8, device="cuda")
    xf = torch.as_strided(big, (M, K), (far, 1))
    xf.copy_(x)
    ybig = torch.zeros(2 * far + N, dtype=torch.bfloat16, device="cuda")
    yf = torch.as_strided(ybig, (M, N), (far, 1))
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qgemv.run_scaled(h, qgemv.scaled_desc(x, xs, W, ws, y))
    qgemv.run_scaled(h, qgemv.scaled_desc(xf, xs, W, ws, yf))
    torch.cuda.synchronize()
    assert torch.equal(y, yf)


@pytest.mark.parametrize("op", ["norm", "quant"])
def test_rows_far_apart(h, op):
    far, N = 1 << 31, 512
    g = gen(2)
    x = randn(g, 3, N).half()
    xf = torch.as_strided(torch.zeros(2 * far + N, dtype=torch.float16, device="cuda"), (3, N), (far, 1))
    xf.copy_(x)
    got = []
    for v in (x, xf):
        codes, scale = torch.empty(3, N, dtype=F8, device="cuda"), torch.empty(3, N // 128, device="cuda")
        if op == "norm":
            qgemv.run_norm(h, qgemv.norm_desc(v, None, 1e-5, codes=codes, scale=scale))
        else:
            qgemv.quant_rows(h, qgemv.quant_desc(v, codes, scale))
        torch.cuda.synchronize()
        got.append((codes.view(torch.uint8), scale))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("rows,N", [(3000, 4096), (1301, 2048), (25000, 256), (1300, 20480)])
def test_norm_of_many_rows_in_place(h, rows, N):
    """CTAs that go on to further rows read those before they have written the first."""
    g = gen(rows)
    x, res, w = randn(g, rows, N).bfloat16(), randn(g, rows, N).bfloat16(), randn(g, N)
    out = [torch.empty_like(x), torch.empty_like(res), torch.empty(rows, N, dtype=F8, device="cuda"), torch.empty(rows, N // 128, device="cuda")]
    qgemv.run_norm(h, qgemv.norm_desc(x, w, 1e-6, y=out[0], codes=out[2], scale=out[3], res=res, res_out=out[1]))
    codes, scale = torch.empty_like(out[2]), torch.empty_like(out[3])
    qgemv.run_norm(h, qgemv.norm_desc(x, w, 1e-6, y=x, codes=codes, scale=scale, res=res, res_out=res))
    torch.cuda.synchronize()
    assert torch.equal(x, out[0]) and torch.equal(res, out[1]) and torch.equal(scale, out[3])
    assert torch.equal(codes.view(torch.uint8), out[2].view(torch.uint8))


def test_gated_ends(h):
    """Gates from where the exponential ends to the infinities; NaN, infinite and large partners."""
    gate = torch.tensor([-87.0, -86.5, -80.0, -30.0, -1e-30, 0.0, 1e-30, 30.0, 88.0, 89.0, 200.0, 1e30, -50.0, -60.0, -70.0, -75.0], device="cuda")
    up = torch.tensor([1e30, 1e33, -1e30, 1e9, 1e30, 5.0, 1e30, -1.0, 1.0, 1.0, -1.0, 1.0, 1e20, 1e22, 1e25, -1e28], device="cuda")
    rows = torch.zeros(16, 128, device="cuda")  # a value to a row, and its scale with it
    rows[:, 0] = gate
    ups = torch.zeros(16, 128, device="cuda")
    ups[:, 0] = up
    codes, scale = quantise(h, rows, ups)
    ref = torch.zeros(16, 128, dtype=torch.float64, device="cuda")
    ref[:, 0] = gate.double() / (1 + torch.exp(-gate.double())) * up.double()
    check_codes(codes, scale, ref, 2.0 ** -20, "gated ends")
    rows[:, 0] = torch.tensor([INF, -INF, NAN, -88.0, -100.0, -3e38, INF, 1.0, 1.0] + [0.0] * 7, device="cuda")
    ups[:, 0] = torch.tensor([2.0, 1.0, 1.0, 1.0, 1.0, 1.0, 0.0, INF, NAN] + [0.0] * 7, device="cuda")
    codes, _ = quantise(h, rows, ups)
    c = codes.view(F8).float()[:, 0]
    assert c[0] == 448 and c[7] == 448 and c[[1, 2, 6, 8]].isnan().all() and (c[3:6] == 0).all()
    # every gate from where the exponential passes the largest number: 0 times a finite partner
    far = -torch.linspace(88, 1000, 128 * 512, device="cuda").reshape(512, 128)
    codes, scale = quantise(h, far, torch.ones_like(far))
    assert (codes.view(F8).float() == 0).all() and (scale == 1).all()
