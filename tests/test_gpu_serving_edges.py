"""Edges of the serving operators: first copies of every ring stage, weights far below the largest, inner
sums far apart, codes at ties, sizes that are refused.  References in 64 bits; the tolerances' terms are those
of test_gpu_serving.py (u half an ulp of the output's type, steps(n) for an fp32 sum of n terms)."""
import math

import pytest
import torch

import test_gpu_serving
from quantized_weight_dequant_gb300 import qgemv
from test_gpu_serving import (F8, HALF_ULP, TINY, TYPES, attend_case, attend_reference, check_attend, gen, h, ints,  # noqa: F401
                              lora_case, make_cache, plan_on_gpu, randn, steps, within)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ attention: barriers
@pytest.mark.parametrize("typ,dim", [("bf16", 128), ("f16", 256), ("e4m3", 64)])
def test_the_first_copies_of_every_stage_are_waited_for(h, typ, dim):  # noqa: F811
    """Shares of one to a few tiles per warp, so that what is copied first is most of what there is: right, and
    the same bits in every one of many launches."""
    qt = "f16" if typ == "e4m3" else typ
    for lens in ([1] * 40, [16, 33, 47, 64, 129, 200] * 20, [700] * 30):
        got, lse, q, ref, scale, d = attend_case(h, lens, 8, 2, dim, typ, qt, 16, seed=len(lens))
        check_attend(got, lse, q, ref, scale, rows=range(0, len(lens), 7))
        out, first = d.keep[2], got.clone()
        for _ in range(40):
            out.fill_(math.nan)
            qgemv.attn_decode(h, d)
            assert torch.equal(got, first)
    assert qgemv.check_error(h) == qgemv.OK


# ------------------------------------------------------------------------------ attention: weights far below the largest
def sink_case(g, typ, gaps, page, dim, pages):
    """A cache of `pages` pages, whose token 0 scores gaps[i] above all others against query i and has the value 0."""
    kc, vc, ks, vs = make_cache(g, typ, pages, 1, page, dim)
    v = 1 + 0.25 * randn(g, pages, 1, page, dim)
    k = torch.zeros_like(v)
    v[0, 0, 0], k[0, 0, 0, 0] = 0, 1
    if typ == "e4m3":
        for c, x in ((kc, k), (vc, v)):
            c.copy_(x.to(F8).view(torch.uint8))
        ks.fill_(1)
        vs.fill_(1)
        k, v = k.to(F8).double(), v.to(F8).double()
    else:
        kc.copy_(k)
        vc.copy_(v)
        k, v = kc.double(), vc.double()
    q = torch.zeros(1, len(gaps), dim, device="cuda", dtype=torch.bfloat16 if typ == "bf16" else torch.float16)
    q[0, :, 0] = torch.tensor(gaps, device="cuda").to(q.dtype)
    return kc, vc, ks, vs, k[:, 0], v[:, 0], q


@pytest.mark.parametrize("typ", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("heads", [8, 12])
def test_many_small_weights_beside_one_large_add_up(h, typ, heads):  # noqa: F811
    """One token of value 0 outweighs each of thousands of others by 10 to 22 nats: what is left of the output is
    theirs alone, each with a weight down to 2^-32 of the largest, which fp16 parts round to 2^-39 of it.  So many
    requests that most (request, head)s are one warp's, in which the large one comes first."""""
    page, dim, n, requests = 64, 64, 4003, 1500
    gaps = [10 + 12 * i / (heads - 1) for i in range(heads)]
    kc, vc, ks, vs, k, v, q = sink_case(gen(41), typ, gaps, page, dim, 9)
    row = torch.cat([torch.zeros(1, device="cuda"), 1 + torch.arange(-(-n // page) - 1, device="cuda") % 8]).int()
    table = row[None].repeat(requests, 1)
    out, lse = torch.empty(requests, heads, dim, device="cuda", dtype=q.dtype), torch.empty(requests, heads, device="cuda")
    qgemv.attn_decode(h, qgemv.attn_decode_desc(qgemv.kv_cache(kc, vc, ks, vs), q.repeat(requests, 1, 1), table, ints([n] * requests),
                                                out, 1.0, lse=lse))
    assert qgemv.check_error(h) == qgemv.OK
    kk, vv = (x[row.long()].reshape(-1, dim)[:n] for x in (k, v))
    o, want, pv, qk = attend_reference(q[0].double(), kk, vv, 1.0)
    score = steps(dim) * qk + 2.0 ** -21 * qk
    tokens = steps(n) + 2.0 ** -20
    within(lse, want, score + tokens + 2.0 ** -22 * want.abs(), "lse")
    lost = n * 2.0 ** -39 * vv.abs().amax()
    within(out, o, HALF_ULP[out.dtype] * o.abs() + TINY[out.dtype] + (2 * score[:, None] + 2 * tokens + 2.0 ** -16) * pv + lost, "out")


@pytest.mark.parametrize("order", [1, -1])
def test_small_value_scales_beside_large_ones_keep_their_part(h, order):  # noqa: F811
    """Value scales 2^60 apart, where the tokens of the largest have zeros: a weight times its scale is rounded to
    2^-25 beside a largest of 2^14, by each of the n tokens and for the largest code."""
    g = gen(22)
    n, page, dim = 200, 16, 64
    kc, vc, ks, vs = make_cache(g, "e4m3", 13, 1, page, dim)
    k, v = ((randn(g, n, dim) * 100).clamp(-440, 440).to(F8) for _ in range(2))
    size = torch.linspace(-50, 10, n, device="cuda") * order
    sk, sv = torch.full((n,), 0.01, device="cuda"), torch.exp2(size)
    v = torch.where((size > -9)[:, None] & (torch.arange(dim, device="cuda") % 2 == 1), torch.zeros((), device="cuda"), v.float()).to(F8)
    t = torch.arange(n, device="cuda")
    kc[t // page, 0, t % page], vc[t // page, 0, t % page] = k.view(torch.uint8), v.view(torch.uint8)
    ks[t // page, 0, t % page], vs[t // page, 0, t % page] = sk, sv
    q = (randn(g, 1, 4, dim) * 0.5).half()
    out = torch.empty_like(q)
    table = torch.arange(13, dtype=torch.int32, device="cuda")[None].contiguous()
    # so many requests of it that most heads are one warp's
    many, outs = q.repeat(1500, 1, 1), out.repeat(1500, 1, 1)
    qgemv.attn_decode(h, qgemv.attn_decode_desc(qgemv.kv_cache(kc, vc, ks, vs), many, table.repeat(1500, 1), ints([n] * 1500), outs, 0.5))
    kk, vv = k.double() * sk.double()[:, None], v.double() * sv.double()[:, None]
    o, _, pv, qk = attend_reference(q[0].double(), kk, vv, 0.5)
    score = steps(dim) * qk + 2.0 ** -21 * qk
    p = torch.softmax(q[0].double() @ kk.t() * 0.5, -1)
    lost = n * 2.0 ** -39 * 448 * (p * sv.double()).amax(-1)
    tol = HALF_ULP[out.dtype] * o.abs() + TINY[out.dtype] + (2 * score[:, None] + 2 * steps(n) + 2.0 ** -16) * pv + lost[:, None]
    # outputs past fp16's range are infinities
    far, inside = o.abs() - tol >= 65520, o.abs() + tol < 65504
    assert torch.equal(outs[:, far].double(), (torch.sign(o[far]) * math.inf).expand(1500, -1))
    within(outs[:, inside], o[inside], tol[inside], "out")


# ------------------------------------------------------------------------------ adapters: inner sums far apart
def spread_case(g, rows, typ, rank, K=64, N=90):
    """Rows of x with one element each, so that an inner sum is one exact product.  Columns of A from K / 2 on make
    sums over 2^38 apart, with the inverse in B as far as it goes; every third output has the small ones only."""
    dt = TYPES[typ]
    size = torch.exp2(torch.linspace(14, -24, rank, device="cuda"))
    A = randn(g, 2, rank, K)
    A[:, :, K // 2:] *= size[:, None]
    B = randn(g, 2, N, rank) * 0.4 * (1 / size).clamp(2.0 ** -14, 2.0 ** 15)
    B[:, ::3] *= size < 2.0 ** -10
    x = torch.zeros(rows, K, device="cuda")
    x[torch.arange(rows), torch.randint(0, K, (rows,), generator=g, device="cuda")] = randn(g, rows) + 3
    return x.to(dt), A.to(dt), B.to(dt)


def spread_reference(x, A, B, ids):
    """The outputs in 64 bits and their tolerance: 21 bits of every inner sum, an fp32 sum over them."""
    low = torch.einsum("mk,mjk->mj", x.double(), A.double()[ids.long()])
    Bm = B.double()[ids.long()]
    ref = torch.einsum("mj,mnj->mn", low, Bm)
    return ref, (2.0 ** -21 + steps(A.shape[1])) * torch.einsum("mj,mnj->mn", low.abs(), Bm.abs()) + 2.0 ** -22 * ref.abs()


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("rows,rank", [(20, 16), (200, 72), (300, 16), (300, 64), (500, 72), (300, 128)])
def test_inner_sums_far_below_the_rows_largest_keep_their_bits(h, rows, rank, typ):  # noqa: F811
    g = gen(rows + rank)
    x, A, B = spread_case(g, rows, typ, rank)
    ids = (torch.arange(rows, device="cuda") // 3 % 2).int()
    y = torch.empty(rows, 90, device="cuda")
    qgemv.run_lora(h, qgemv.lora_desc(x, A, B, ids, y))
    assert qgemv.check_error(h) == qgemv.OK
    ref, tol = spread_reference(x, A, B, ids)
    within(y, ref, tol, "y")


@pytest.mark.parametrize("rows", [40, 400])
def test_inner_sums_far_apart_of_ragged_ranks_ignore_what_lies_past_them(h, rows):  # noqa: F811
    x, A, B = spread_case(gen(rows), rows, "f16", 72)
    ids, ranks = (torch.arange(rows, device="cuda") % 3 - 1).int(), ints([37, 67])
    for a, r in enumerate(ranks.tolist()):
        A[a, r:], B[a, :, r:] = 0, 0
    ref, tol = spread_reference(x, A, B, ids.clamp(min=0))
    for a, r in enumerate(ranks.tolist()):
        A[a, r:], B[a, :, r:] = math.nan, math.nan
    y = torch.empty(rows, 90, device="cuda")
    qgemv.run_lora(h, qgemv.lora_desc(x, A, B, ids, y, ranks=ranks))
    assert qgemv.check_error(h) == qgemv.OK
    there = (ids >= 0)[:, None]
    within(y, ref * there, tol * there, "y")


@pytest.mark.parametrize("rows", [24, 320])
def test_a_row_of_far_apart_sums_leaves_its_neighbours_as_they_are(h, rows):  # noqa: F811
    """The rows of one adapter whose sums are near one another come out bit for bit as without the others."""
    g = gen(5)
    x, A, B = spread_case(g, rows, "f16", 32)
    ids, base = torch.zeros(rows, dtype=torch.int32, device="cuda"), randn(g, rows, 90)
    near = (x[:, :32] != 0).any(1)
    alone, together = torch.empty(rows, 90, device="cuda"), torch.empty(rows, 90, device="cuda")
    qgemv.run_lora(h, qgemv.lora_desc(x, A, B, ids, together, base=base))
    qgemv.run_lora(h, qgemv.lora_desc(torch.where(near[:, None], x, torch.zeros_like(x)), A, B, ids, alone, base=base))
    assert torch.equal(alone[near], together[near]) and qgemv.check_error(h) == qgemv.OK
    assert torch.equal(alone[~near], base[~near])
    ref, tol = spread_reference(x, A, B, ids)
    within(together, ref + base.double(), tol + 2.0 ** -22 * base.double().abs(), "y")


@pytest.mark.parametrize("rows", [5, 300])
@pytest.mark.parametrize("sign", [1, -1])
def test_bf16_inner_sums_up_to_the_end_of_fp32_stay_finite(h, rows, sign):  # noqa: F811
    """Sums of (2 - 2^-9) 2^127, which fp32 holds and bf16 rounds to infinity, brought back by the adapter's scale;
    beside them, infinite ones stay with their rows."""
    x, A = torch.zeros(rows, 16, device="cuda"), torch.zeros(1, 8, 16, device="cuda")
    x[:, 0], x[:, 9] = sign * (2 - 2.0 ** -7) * 2.0 ** 63, sign * 1.5 * 2.0 ** 63
    A[:, :, 0], A[:, :, 9] = 2.0 ** 64, 2.0 ** 56
    x[3] *= 4
    B = torch.zeros(1, 40, 8, device="cuda")
    B[0, torch.arange(40), torch.arange(40) % 8] = torch.exp2(-torch.arange(40, device="cuda") / 8.0)
    x, A, B = x.bfloat16(), A.bfloat16(), B.bfloat16()
    y = torch.empty(rows, 40, device="cuda")
    scale = torch.full((1,), 2.0 ** -100, device="cuda")
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    qgemv.run_lora(h, qgemv.lora_desc(x, A, B, ids, y, scales=scale))
    ref = (2.0 ** -100 * sign * (2 - 2.0 ** -9) * 2.0 ** 127 * B[0].double().sum(-1)).expand(rows - 1, -1)
    within(torch.cat([y[:3], y[4:]]), ref, (2.0 ** -21 + steps(8)) * ref.abs(), "y")  # one product each
    assert not y[3].isfinite().any() and qgemv.check_error(h) == qgemv.OK


# ------------------------------------------------------------------------------ sizes
@pytest.mark.parametrize("requests", [2 ** 30 + 1, 2 ** 31 - 128, 2 ** 31 - 1])
def test_more_requests_than_the_kernels_can_number_are_refused(h, requests):  # noqa: F811
    def none(*n):
        return torch.zeros(n, dtype=torch.int32, device="cuda")

    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    plan = qgemv.page_plan_desc(none(2), none(2), none(2, 3), none(5), none(1), 16, none(2), slots, none(4))
    plan.requests = requests
    assert qgemv.page_plan(h, plan, check=False) == qgemv.ERR_BAD_SHAPE
    k, q = torch.zeros(3, 2, 16, 64, dtype=torch.float16, device="cuda"), torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    attend = qgemv.attn_decode_desc(qgemv.kv_cache(k, k.clone()), q, none(2, 3), none(2), torch.empty_like(q), 0.1)
    attend.requests = requests
    assert qgemv.attn_decode(h, attend, check=False) == qgemv.ERR_BAD_SHAPE
    assert qgemv.check_error(h) == qgemv.OK


# ------------------------------------------------------------------------------ store: codes
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_e4m3_codes_are_the_rounded_quotients_by_the_scale(h, src, dim):  # noqa: F811
    """Scale and codes of unrotated heads bit for bit: max|x| / 448 and x / scale, each rounded to fp32 once, and
    the quotient to e4m3.  Small whole numbers, so that many quotients are near the middle of two codes."""
    g = gen(dim)
    t, hk, page = 3000, 4, 16
    kc, vc, ks, vs = make_cache(g, "e4m3", t // page + 3, hk, page, dim)
    k = torch.randint(-300, 301, (t, hk, dim), generator=g, device="cuda").to(TYPES[src])
    v = (randn(g, t, hk, dim) * torch.exp2(torch.randint(-20, 10, (t, hk, 1), generator=g, device="cuda"))).to(TYPES[src])
    if src == "f32":  # scales down to the least, and values that are not normal
        v[:40] *= torch.exp2(torch.arange(40, device="cuda") * -3.0)[:, None, None]
    slots = torch.randperm(kc.shape[0] * page, generator=g, device="cuda")[:t].contiguous()
    qgemv.kv_store(h, qgemv.kv_store_desc(qgemv.kv_cache(kc, vc, ks, vs), k.flatten(1), v.flatten(1), slots, ints([0] * t)))
    assert qgemv.check_error(h) == qgemv.OK
    for x, codes, scales in ((k, kc, ks), (v, vc, vs)):
        top = x.float().abs().amax(-1)
        # in 64 bits first: torch divides by a plain number as by its reciprocal
        scale = torch.where(top > 0, (top.double() / 448).float(), 1.0).clamp(min=2.0 ** -126)
        at = (slots // page, slice(None), slots % page)
        assert torch.equal(scales[at], scale)
        assert torch.equal(codes[at].view(F8).float(), (x.double() / scale[..., None].double()).float().to(F8).float())


# ------------------------------------------------------------------------------ page plan: broken tables
def test_page_plan_counts_tokens_whose_page_is_negative(h):  # noqa: F811
    """Positions go on past a page that the caller's table or stack has wrong: its tokens are not stored, those of
    the next page are."""
    got = plan_on_gpu(h, [20, 3], [14, 20], [[7, -1, -1], [5, -1, -1]], [9, -6, 2], 16, 34)
    assert qgemv.check_error(h) == qgemv.ERR_BAD_INDEX
    # request 0: tokens 20 .. 31 in page -1, 32 and 33 in page 2; request 1: 3 .. 15 in page 5, 16 .. 22 in page -6
    assert got["slots"] == [-1] * 12 + [32, 33] + [80 + i for i in range(3, 16)] + [-1] * 7
    assert got["positions"] == list(range(20, 34)) + list(range(3, 23))
    assert got["lens"] == [34, 23] and got["counts"] == [34, 34, 2, 0]
    assert got["table"] == [[7, -1, 2], [5, -6, -1]]


# ------------------------------------------------------------------------------ forms beside the usual ones
@pytest.mark.parametrize("rows,used,rank,typ,out,form", [
    (300, 5, 16, "f16", "f32", "inplace"), (300, 290, 16, "bf16", "f32", "inplace"), (700, 3, 64, "bf16", "bf16", "inplace"),
    (450, 4, 128, "f16", "f16", "inplace"), (300, 5, 16, "f16", "f32", "none"), (600, 40, 40, "bf16", "bf16", "none"),
    (513, 6, 32, "f16", "f16", "base"), (400, 2, 72, "bf16", "f16", "base")])
def test_adapters_of_many_rows_in_place_without_a_base_and_in_16_bits(h, rows, used, rank, typ, out, form):  # noqa: F811
    lora_case(h, rows, used, used + 1, rank, 264, 190, typ, out, inplace=form == "inplace", base=form != "none", pad=2)
    assert qgemv.check_error(h) == qgemv.OK


def test_many_rows_without_an_adapter_keep_the_base_in_place(h):  # noqa: F811
    y, ids, base, _ = lora_case(h, 400, 0, 3, 16, 128, 100, "f16", "f32", ids=[-1] * 150 + [2, -1, 0] * 20 + [-1] * 190, inplace=True)
    assert torch.equal(y[ids < 0].double(), base[ids < 0]) and qgemv.check_error(h) == qgemv.OK


@pytest.mark.parametrize("gap", [4, 60])
def test_an_e4m3_cache_whose_scales_have_gaps_between_pages(h, gap):  # noqa: F811
    """Stored and attended to; the gaps hold NaN and stay as they are."""
    g = gen(gap)
    page, hk, dim, n = 16, 2, 64, 83
    kc, vc, _, _ = make_cache(g, "e4m3", 9, hk, page, dim, 32)
    wide = [torch.full((9, hk * page + gap), math.nan, device="cuda") for _ in range(2)]
    ks, vs = (x[:, :hk * page].unflatten(1, (hk, page)) for x in wide)
    cache = qgemv.kv_cache(kc, vc, ks, vs)
    mine = torch.randperm(9, generator=g, device="cuda")[:6]
    t = torch.arange(n, device="cuda")
    k, v = randn(g, n, hk * dim).bfloat16(), randn(g, n, hk * dim).bfloat16()
    qgemv.kv_store(h, qgemv.kv_store_desc(cache, k, v, mine[t // page] * page + t % page, t.int()))
    q = (randn(g, 1, 4, dim) * 2).bfloat16()
    out, lse = torch.empty_like(q), torch.empty(1, 4, device="cuda")
    qgemv.attn_decode(h, qgemv.attn_decode_desc(cache, q, mine.int()[None].contiguous(), ints([n]), out, 0.125, lse=lse))
    assert qgemv.check_error(h) == qgemv.OK
    at = (mine[t // page], slice(None), t % page)
    stored = [c[at].view(F8).double() * s[at].double()[..., None] for c, s in ((kc, ks), (vc, vs))]
    for got, x in zip(stored, (k, v)):
        x = x.double().unflatten(1, (hk, dim))
        within(got, x, (2.0 ** -4 * x.abs() + x.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10) * 1.001, "stored")
    check_attend(out, lse, q, [stored], 0.125)
    assert all(x[:, hk * page:].isnan().all() for x in wide)


@pytest.mark.parametrize("src,typ,qt", [("bf16", "bf16", "bf16"), ("f32", "e4m3", "f16"), ("f16", "f16", "f16")])
def test_store_of_many_tokens_of_heads_of_256(h, src, typ, qt):  # noqa: F811
    check = test_gpu_serving.test_store_rotates_rounds_once_and_writes_only_its_slots
    check(h, 1201, 3, 2, 256, 256, True, src, typ, qt, 32, 0)
    check(h, 1201, 3, 2, 256, 192, False, src, typ, qt, 32, 32)


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [4, 12])
def test_an_infinite_value_that_is_seen_stays_with_its_element(h, typ, heads):  # noqa: F811
    """It gives an infinity or NaN there (inf times the low part of a weight, which may be 0 or negative), and leaves the
    head's other elements, and requests that do not see it, as they are."""
    def edit(table, lens, q, kc, vc):
        vc[table[0, 1].item(), 0, 3, 5] = math.inf

    sound, *_ = attend_case(h, [60, 45], heads, 1, 64, typ, typ, 16, seed=8)
    got, lse, q, ref, scale, _ = attend_case(h, [60, 45], heads, 1, 64, typ, typ, 16, seed=8, edit=edit)
    assert not got[0, :, 5].isfinite().any()
    rest = torch.arange(64, device="cuda") != 5
    assert torch.equal(got[0][:, rest], sound[0][:, rest]) and torch.equal(got[1], sound[1])
