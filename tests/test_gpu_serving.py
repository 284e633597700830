"""GPU parity of the serving operators (page plan, cache store, paged attention, adapters)
against plain implementations in 64 bits, at the sizes, strides and masks where they can go
wrong, and their refusals.  Tolerances are derived from the arithmetic: u is half an ulp of the
output's type, products of 16-bit values are exact in fp32, and a sum of n terms that is taken
in steps of 16 has at most n / 16 + 32 roundings of at most 2^-22 of its absolute terms."""
import math

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
NAN = float("nan")


def steps(n):
    return (n / 16 + 32) * 2.0 ** -22


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


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float(err[bad].max())} against "
                           f"{float(tol.expand_as(err)[bad].max())} at {bad.nonzero()[0].tolist()}")


# ------------------------------------------------------------------------------ page plan
def plan_reference(cached, fresh, table, stack, page, cap):
    table, stack = [list(r) for r in table], list(stack)
    slots, positions, owners, lens, offsets = [], [], [], [], [0]
    taken = missing = 0
    for r, (c, f) in enumerate(zip(cached, fresh)):
        c, f, kept, stuck = max(c, 0), max(f, 0), 0, False
        for i in range(min(f, max(0, cap - offsets[-1]))):
            pos = c + i
            fits = pos // page < len(table[r])
            if fits and pos % page == 0:
                if stack:
                    table[r][pos // page] = stack.pop()
                    taken += 1
                else:
                    stuck, missing = True, missing + 1
            ok = fits and not stuck
            kept += ok
            slots.append(table[r][pos // page] * page + pos % page if ok else -1)
            positions.append(pos if ok else -1)
            owners.append(r)
        lens.append(c + kept)
        offsets.append(offsets[-1] + f)
    rest = cap - len(slots)
    planned = sum(v >= 0 for v in slots)
    return dict(table=table, lens=lens, offsets=offsets, slots=slots + [-1] * rest, positions=positions + [-1] * rest,
                owners=owners + [-1] * rest, counts=[offsets[-1], planned, taken, missing])


def plan_on_gpu(h, cached, fresh, table, stack, page, cap, stream=None):
    n = len(cached)
    width = len(table[0]) if n else 1
    wide = torch.full((max(n, 1), width + 5), -7, dtype=torch.int32, device="cuda")  # rows further apart than wide
    tab = wide[:n, :width]
    if n:
        tab.copy_(ints(table))
    free = ints(list(stack) + [-99] * 3)
    out = {k: torch.full((s,), -5, dtype=torch.int64 if k == "slots" else torch.int32, device="cuda")
           for k, s in (("lens", n), ("offsets", n + 1), ("slots", cap), ("positions", cap), ("owners", cap), ("counts", 4))}
    d = qgemv.page_plan_desc(ints(cached), ints(fresh), tab, free, ints([len(stack)]), page, **out)
    qgemv.page_plan(h, d, stream=stream)
    torch.cuda.synchronize()
    assert (wide[:, width:] == -7).all()
    return {"table": tab.tolist(), **{k: v.tolist() for k, v in out.items()}}


def plan_inputs(n, cached_hi, fresh_hi, page, seed, spare=0, width=None, pages=None):
    r = torch.Generator().manual_seed(seed)
    draw = lambda hi: torch.randint(0, hi + 1, (n,), generator=r).tolist()  # noqa: E731
    cached, fresh = draw(cached_hi), draw(fresh_hi)
    have = [-(-c // page) for c in cached]
    need = sum(-(-(c + f) // page) - b for c, f, b in zip(cached, fresh, have))
    ids = torch.randperm(sum(have) + max(0, need + spare) + 3, generator=r).tolist()
    width = width or max([-(-(c + f) // page) for c, f in zip(cached, fresh)] + [1]) + 2
    table = [[ids.pop() if j < b else -1 for j in range(width)] for b in have]
    return cached, fresh, table, ids[:max(0, need + spare)]


@pytest.mark.parametrize("n,cached_hi,fresh_hi,page,pad,spare", [
    (1, 0, 1, 16, 0, 0), (1, 500, 700, 16, 3, 2), (3, 40, 0, 8, 5, 1), (64, 900, 1, 16, 0, 4), (511, 60, 3, 16, 1, 0),
    (513, 70, 9, 1, 0, 0), (700, 100, 40, 48, 77, -9), (40, 300, 2000, 64, 0, -200), (2, 0, 5000, 7, 0, 0),
    (1030, 33, 1, 32, 4, -1030), (5, 10, 100000, 128, 2, 0)])
def test_page_plan_matches_a_host_allocator(h, n, cached_hi, fresh_hi, page, pad, spare):
    cached, fresh, table, stack = plan_inputs(n, cached_hi, fresh_hi, page, 17 * n + page, spare)
    cap = sum(fresh) + pad
    want = plan_reference(cached, fresh, table, stack, page, cap)
    got = plan_on_gpu(h, cached, fresh, table, stack, page, cap)
    for k in want:
        assert got[k] == want[k], k
    assert qgemv.check_error(h) == qgemv.OK


def test_page_plan_cuts_at_the_capacity_and_at_the_end_of_a_row(h):
    cached, fresh, table, stack = plan_inputs(30, 50, 60, 16, 3)
    for cap in (0, 1, 17, sum(fresh[:7]), sum(fresh) - 1):
        want = plan_reference(cached, fresh, table, stack, 16, cap)
        got = plan_on_gpu(h, cached, fresh, table, stack, 16, cap)
        assert got == want, cap
    short = [row[:4] for row in table]  # rows of 64 positions
    assert plan_on_gpu(h, cached, fresh, short, stack, 16, sum(fresh)) == plan_reference(cached, fresh, short, stack, 16, sum(fresh))


def test_page_plan_counts_negative_lengths_as_none_and_takes_no_requests(h):
    cached, fresh, table, stack = [-3, 5, 0, 20], [2, -1, 0, 13], [[-1, -1, -1]] * 4, [4, 9, 2, 7, 11]
    table = [[-1, -1, -1], [30, -1, -1], [-1, -1, -1], [31, 32, -1]]
    assert plan_on_gpu(h, cached, fresh, table, stack, 16, 20) == plan_reference(cached, fresh, table, stack, 16, 20)
    got = plan_on_gpu(h, [], [], [], [1], 16, 6)
    assert got["slots"] == [-1] * 6 and got["offsets"] == [0] and got["counts"] == [0, 0, 0, 0]


def test_page_plan_reports_a_negative_page(h):
    got = plan_on_gpu(h, [5], [2], [[-1, -1]], [3], 16, 2)
    assert got["slots"] == [-1, -1] and qgemv.check_error(h) == qgemv.ERR_BAD_INDEX
    assert qgemv.check_error(h) == qgemv.OK


# ------------------------------------------------------------------------------ cache store
def make_cache(g, typ, pages, heads, page, dim, gap=0):
    """k, v, k_scale, v_scale with `gap` elements between pages, all poisoned."""
    if typ == "e4m3":
        k, v = (torch.full((pages, heads * page * dim + gap), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.full((pages, heads, page), NAN, device="cuda") for _ in range(2))
    else:
        k, v = (torch.full((pages, heads * page * dim + gap), NAN, dtype=TYPES[typ], device="cuda") for _ in range(2))
        ks = vs = None
    view = lambda t: t[:, :heads * page * dim].unflatten(1, (heads, page, dim))  # noqa: E731
    return view(k), view(v), ks, vs


def rope_table(n, rot):
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def turn(x, table, pos, rot, interleaved):
    """The rotation in 64 bits and the absolute terms behind each element."""
    half = rot // 2
    c, s = table.double()[pos.long()][:, None, :half], table.double()[pos.long()][:, None, half:]
    ia = torch.arange(half, device="cuda") * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else half)
    y, z = x.clone(), x.abs()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    z[..., ia], z[..., ib] = a.abs() + b.abs(), a.abs() + b.abs()
    return y, z


STORES = [  # tokens, hq, hk, dim, rot, interleaved, source, cache, q type, page, gap
    (1, 1, 1, 64, 64, False, "f32", "f16", "f16", 16, 0), (5, 4, 2, 128, 128, True, "f16", "f16", "f16", 8, 64),
    (67, 7, 1, 256, 128, False, "bf16", "bf16", "bf16", 48, 0), (300, 8, 8, 64, 32, True, "f32", "bf16", "bf16", 32, 8),
    (1, 4, 4, 128, 64, False, "bf16", "e4m3", "bf16", 16, 16), (129, 3, 3, 64, 64, True, "f16", "e4m3", "f16", 128, 0),
    (33, 2, 1, 256, 256, False, "f32", "e4m3", "bf16", 16, 0), (40, 0, 2, 128, 0, False, "f32", "f16", None, 16, 0),
    (31, 5, 2, 128, 0, False, "bf16", "e4m3", "f16", 64, 0), (9, 6, 2, 128, 16, False, "f16", "f16", "bf16", 16, 0)]


@pytest.mark.parametrize("t,hq,hk,dim,rot,inter,src,typ,qt,page,gap", STORES)
def test_store_rotates_rounds_once_and_writes_only_its_slots(h, t, hq, hk, dim, rot, inter, src, typ, qt, page, gap):
    g = gen(t + dim)
    pages = t // page + 3
    kc, vc, ks, vs = make_cache(g, typ, pages, hk, page, dim, gap)
    rows = (randn(g, t, (hq + 2 * hk) * dim + 16) * 3).to(TYPES[src])
    if t > 2:
        rows[2] = 0  # a head of zeros (scale 1)
    q, k, v = rows[:, :hq * dim], rows[:, hq * dim:(hq + hk) * dim], rows[:, (hq + hk) * dim:(hq + 2 * hk) * dim]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:t].contiguous()
    pos = torch.randperm(4096, generator=g, device="cuda")[:t].int()
    if t > 4:
        slots[3], pos[4], slots[4] = -1, -1, -1
    table = rope_table(4096, rot) if rot else None
    qo = torch.full((t, hq, dim + 8), NAN, dtype=TYPES[qt], device="cuda")[..., :dim].contiguous() if hq else None
    d = qgemv.kv_store_desc(qgemv.kv_cache(kc, vc, ks, vs), k, v, slots, pos, table, inter, q if hq else None, qo)
    qgemv.kv_store(h, d)
    assert qgemv.check_error(h) == qgemv.OK
    for name, x, heads in (("q", q, hq), ("k", k, hk), ("v", v, hk)):
        if not heads:
            continue
        x = x.double().reshape(t, heads, dim)
        ref, terms = turn(x, table, pos.clamp(min=0), rot, inter) if rot and name != "v" else (x, x.abs())
        near = 2.0 ** -22 * terms
        if name == "q":
            ref = ref * (pos >= 0)[:, None, None]
            within(qo, ref, HALF_ULP[qo.dtype] * ref.abs() + near + TINY[qo.dtype], "q")
            continue
        cache, scale = (kc, ks) if name == "k" else (vc, vs)
        ok = slots >= 0
        page_of, at = slots[ok] // page, slots[ok] % page
        got, ref, near = cache[page_of, :, at], ref[ok], near[ok]
        untouched = torch.ones(pages, page, dtype=torch.bool, device="cuda")
        untouched[page_of, at] = False
        rest = cache.transpose(1, 2)[untouched]
        if typ == "e4m3":
            top = ref.abs().amax(-1, keepdim=True)
            sc = scale[page_of, :, at][..., None]
            want = torch.where(top > 0, top / 448, 1.0)
            within(sc, want, 2.0 ** -21 * want, name + " scale")
            # 3 stored bits, subnormals in steps of 2^-9
            within(got.view(F8).double() * sc, ref, (2.0 ** -4 * ref.abs()).clamp(min=1e-30) * 1.001 + sc * 2.0 ** -10 + near, name)
            assert (rest == 0x7F).all() and scale.transpose(1, 2)[untouched].isnan().all()
        else:
            within(got, ref, HALF_ULP[got.dtype] * ref.abs() + near + TINY[got.dtype], name)
            assert rest.isnan().all()


def test_store_reports_slots_and_positions_out_of_range_and_stores_nothing_there(h):
    g = gen(5)
    kc, vc, _, _ = make_cache(g, "f16", 4, 2, 16, 64)
    rows = randn(g, 6, 256)
    q, k, v = rows[:, :128], rows[:, 128:], rows[:, 128:]
    qo = torch.full((6, 2, 64), NAN, dtype=torch.float16, device="cuda")
    table = rope_table(50, 64)

    def once(slots, pos):
        kc.fill_(NAN)
        d = qgemv.kv_store_desc(qgemv.kv_cache(kc, vc), k, v, ints(slots, torch.int64), ints(pos), table, False, q, qo)
        qgemv.kv_store(h, d)
        return qgemv.check_error(h), int((~kc.isnan()).any(-1).any(1).sum())

    assert once([0, 1, 2, 3, 4, 63], [0, 1, 2, 3, 4, 49]) == (qgemv.OK, 6)
    assert once([0, 64, 2, -5, 4, 2 ** 40], [0] * 6) == (qgemv.ERR_BAD_INDEX, 3)
    assert once([0, 1, 2, 3, 4, 5], [0, 50, 2, 3, -2, 5]) == (qgemv.ERR_BAD_INDEX, 6)
    assert (qo[1] == 0).all() and (qo[4] == 0).all()
    assert once([-1] * 6, [-1] * 6) == (qgemv.OK, 0)
    assert (qo == 0).all()


def test_store_scale_of_heads_that_are_not_finite_or_too_small(h):
    kc, vc, ks, vs = make_cache(None, "e4m3", 1, 1, 16, 64)
    rows = torch.zeros(4, 64, device="cuda")
    rows[0, 3], rows[1, 5], rows[2, 7], rows[3, 9] = math.inf, NAN, 1e-45, 448.0 * 3
    d = qgemv.kv_store_desc(qgemv.kv_cache(kc, vc, ks, vs), rows, rows, ints([0, 1, 2, 3], torch.int64), ints([0] * 4))
    qgemv.kv_store(h, d)
    assert ks[0, 0, :4].tolist() == [1.0, 1.0, 1.0, 3.0]
    got = kc[0, 0, :4].view(F8).float()
    assert got[0, 3] == 448 and got[1, 5].isnan() and got[2].abs().max() == 0 and got[3, 9] == 448
    assert got[3].count_nonzero() == 1


# ------------------------------------------------------------------------------ attention
def attend_reference(q, k, v, scale):
    """q [heads, dim], k and v [tokens, dim] in 64 bits -> out, lse, sum of p |v|, sum |q k| of the largest score."""
    w = q @ k.t() * scale
    lse = torch.logsumexp(w, -1)
    p = torch.softmax(w, -1)
    return p @ v, lse, p @ v.abs(), (q.abs() @ k.abs().t()).amax(-1) * abs(scale)


def attend_case(h, lens, hq, hk, dim, typ, qt, page, window=0, scale=None, seed=1, stride=0, gap=0, stream=None, spike=0.0,
                edit=None, width=None):
    g = gen(seed)
    n = len(lens)
    have = [-(-v // page) for v in lens]
    pages = sum(have) + 4
    kc, vc, ks, vs = make_cache(g, typ, pages, hk, page, dim, gap)
    ids = torch.randperm(pages, generator=g, device="cuda").int().tolist()
    width = width or max(have + [1]) + 1
    table = torch.full((n, width + 3), -1, dtype=torch.int32, device="cuda")
    scale = dim ** -0.5 if scale is None else scale
    ref = []
    q = (randn(g, n, hq * dim + stride) * 2).to(TYPES[qt])[:, :hq * dim].unflatten(1, (hq, dim))
    for r, length in enumerate(lens):
        mine = [ids.pop() for _ in range(have[r])]
        table[r, :have[r]] = ints(mine)
        t = torch.arange(length, device="cuda")
        pg, at = ints(mine, torch.int64)[t // page] if length else t, t % page
        k, v = randn(g, length, hk, dim), randn(g, length, hk, dim)
        if spike and length:
            k[length // 2] *= spike
        if typ == "e4m3":
            sk, sv = (randn(g, length, hk).abs() * 0.01 + 0.002 for _ in range(2))
            k, v = ((x * 100).clamp(-440, 440).to(F8) for x in (k, v))
            kc[pg, :, at], vc[pg, :, at], ks[pg, :, at], vs[pg, :, at] = k.view(torch.uint8), v.view(torch.uint8), sk, sv
            k, v = k.double() * sk.double()[..., None], v.double() * sv.double()[..., None]
        else:
            k, v = k.to(TYPES[typ]), v.to(TYPES[typ])
            kc[pg, :, at], vc[pg, :, at] = k, v
            k, v = k.double(), v.double()
        lo = max(0, length - window) if window else 0
        ref.append((k[lo:], v[lo:]))  # outside of these tokens the cache holds NaN, or tokens before the window
        if window and lo:
            cut = t[:lo]
            if typ == "e4m3":
                kc[pg[cut], :, at[cut]], ks[pg[cut], :, at[cut]], vs[pg[cut], :, at[cut]] = 0x7F, NAN, NAN
                vc[pg[cut], :, at[cut]] = 0x7F
            else:
                kc[pg[cut], :, at[cut]], vc[pg[cut], :, at[cut]] = NAN, NAN
    out = torch.full((n, hq * dim + stride), NAN, dtype=TYPES[qt], device="cuda")
    lse = torch.full((n, hq), NAN, device="cuda")
    lens_d = ints(lens)
    if edit:
        edit(table, lens_d, q, kc, vc)
    d = qgemv.attn_decode_desc(qgemv.kv_cache(kc, vc, ks, vs), q, table[:, :width], lens_d,
                               out[:, :hq * dim].unflatten(1, (hq, dim)), scale, window, lse)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    qgemv.attn_decode(h, d, stream=stream)
    torch.cuda.synchronize()
    got = out[:, :hq * dim].unflatten(1, (hq, dim))
    assert not stride or out[:, hq * dim:].isnan().all()
    return got, lse, q, ref, scale, d


def check_attend(got, lse, q, ref, scale, rows=None):
    n, hq, dim = got.shape
    for r in range(n) if rows is None else rows:
        k, v = ref[r]
        hk = k.shape[1]
        if k.shape[0] == 0:
            assert (got[r] == 0).all() and (lse[r] == -math.inf).all(), r
            continue
        for g in range(hk):
            mine = slice(g * (hq // hk), (g + 1) * (hq // hk))
            o, l, pv, qk = attend_reference(q[r, mine].double(), k[:, g], v[:, g], scale)
            score = steps(dim) * qk + 2.0 ** -21 * qk  # error of a score
            tokens = steps(k.shape[0]) + 2.0 ** -20
            within(lse[r, mine], l, score + tokens + 2.0 ** -22 * l.abs(), f"lse of {r}")
            # weights: two 16-bit parts (2^-17), their scores twice (numerator and sum)
            tol = HALF_ULP[got.dtype] * o.abs() + TINY[got.dtype] + (2 * score[:, None] + 2 * tokens + 2.0 ** -16) * pv
            within(got[r, mine], o, tol, f"out of {r}")


ATTENDS = [  # lens, hq, hk, dim, cache, q, page, window
    ([1], 1, 1, 64, "f16", "f16", 16, 0), ([0], 4, 2, 128, "bf16", "bf16", 16, 0), ([7, 0, 16, 17], 8, 2, 128, "f16", "f16", 8, 0),
    ([15, 16, 17, 31, 33, 64, 100], 32, 8, 128, "bf16", "bf16", 16, 0), ([1000], 32, 8, 128, "f16", "f16", 16, 0),
    ([5000, 3, 0, 777], 8, 1, 128, "bf16", "bf16", 48, 0), ([130, 9], 16, 1, 256, "f16", "f16", 16, 0),
    ([90, 200], 5, 1, 64, "bf16", "bf16", 32, 0), ([60, 300, 1], 24, 2, 64, "f16", "f16", 64, 0),
    ([513, 40], 40, 1, 64, "bf16", "bf16", 16, 0), ([33, 1000], 16, 16, 64, "f16", "f16", 32, 0),
    ([1, 2, 500, 64], 8, 2, 128, "e4m3", "bf16", 16, 0), ([700, 31], 16, 1, 128, "e4m3", "f16", 64, 0),
    ([257, 0, 8], 4, 4, 64, "e4m3", "f16", 8, 0), ([100, 4], 12, 2, 256, "e4m3", "bf16", 16, 0),
    ([900, 10, 129, 128, 127], 8, 2, 128, "f16", "f16", 16, 128), ([300, 5000], 4, 1, 64, "e4m3", "bf16", 128, 100),
    ([40, 41, 42], 8, 8, 256, "bf16", "bf16", 8, 1), ([3000], 2, 2, 128, "bf16", "bf16", 1024, 2999)]


@pytest.mark.parametrize("lens,hq,hk,dim,typ,qt,page,window", ATTENDS)
def test_attention_matches_64_bits_and_sees_nothing_outside(h, lens, hq, hk, dim, typ, qt, page, window):
    got, lse, q, ref, scale, _ = attend_case(h, lens, hq, hk, dim, typ, qt, page, window, stride=8, gap=16 if dim == 128 else 0)
    assert qgemv.check_error(h) == qgemv.OK
    check_attend(got, lse, q, ref, scale)


@pytest.mark.parametrize("n,hi,hq,hk,dim,typ,page", [(200, 90, 8, 2, 128, "f16", 16), (300, 700, 4, 2, 64, "bf16", 32),
                                                     (7, 20000, 16, 4, 128, "e4m3", 16), (33, 2500, 32, 8, 128, "bf16", 64),
                                                     (600, 40, 2, 1, 256, "f16", 16), (2100, 30, 1, 1, 64, "bf16", 8)])
def test_attention_of_many_ragged_requests(h, n, hi, hq, hk, dim, typ, page):
    r = torch.Generator().manual_seed(n)
    lens = torch.randint(0, hi + 1, (n,), generator=r).tolist()
    got, lse, q, ref, scale, _ = attend_case(h, lens, hq, hk, dim, typ, "bf16" if typ == "bf16" else "f16", page, seed=n)
    assert qgemv.check_error(h) == qgemv.OK
    check_attend(got, lse, q, ref, scale)


@pytest.mark.parametrize("n,length,hq,hk,dim,typ", [
    (64, 480, 32, 8, 128, "bf16"), (64, 481, 16, 8, 128, "f16"), (40, 1500, 16, 8, 256, "e4m3"), (20, 450, 8, 2, 128, "e4m3")])
def test_attention_of_requests_of_one_length(h, n, length, hq, hk, dim, typ):
    """Heads as long as the longest that stay whole, one token longer, and where some of the GPU is idle."""
    got, lse, q, ref, scale, _ = attend_case(h, [length] * n, hq, hk, dim, typ, "f16" if typ == "e4m3" else typ, 16, seed=length)
    check_attend(got, lse, q, ref, scale)
    assert qgemv.check_error(h) == qgemv.OK


def test_attention_of_one_long_request_split_over_the_gpu(h):
    got, lse, q, ref, scale, _ = attend_case(h, [100003], 8, 1, 128, "f16", "f16", 16)
    check_attend(got, lse, q, ref, scale)


@pytest.mark.parametrize("lens,hq,hk,dim,typ", [([60000], 1, 1, 64, "f16"), ([90001], 8, 1, 128, "e4m3"), ([70000], 16, 1, 256, "bf16"),
                                                ([30, 50001, 2, 40000], 4, 1, 128, "bf16"), ([9000, 9000, 9000], 16, 1, 64, "e4m3")])
def test_attention_pieces_of_many_ctas_join_in_groups(h, lens, hq, hk, dim, typ):
    qt = "f16" if typ == "e4m3" else typ
    got, lse, q, ref, scale, d = attend_case(h, lens, hq, hk, dim, typ, qt, 16, seed=11)
    check_attend(got, lse, q, ref, scale)
    first = got.clone()
    for _ in range(3):
        qgemv.attn_decode(h, d)
    torch.cuda.synchronize()
    assert torch.equal(first, got) and qgemv.check_error(h) == qgemv.OK


@pytest.mark.parametrize("typ,qt", [("f16", "f16"), ("bf16", "bf16"), ("e4m3", "bf16")])
def test_attention_with_one_key_that_outweighs_the_rest(h, typ, qt):
    got, lse, q, ref, scale, _ = attend_case(h, [2000, 50], 8, 2, 128, typ, qt, 16, spike=4.0, scale=0.5)
    check_attend(got, lse, q, ref, scale)


def test_attention_with_large_bf16_queries_over_an_8_bit_cache(h):
    def grow(table, lens, q, kc, vc):
        q.mul_(2.0 ** 20)  # past fp16's range
    got, lse, q, ref, scale, _ = attend_case(h, [300], 8, 2, 128, "e4m3", "bf16", 16, scale=2.0 ** -24, edit=grow)
    check_attend(got, lse, q, ref, scale)


@pytest.mark.parametrize("order", [1, -1])
def test_attention_over_value_scales_of_very_different_size(h, order):
    """Tokens whose values are 2^60 apart, the small ones with the larger scores or the other way round: the
    weights keep their precision against the largest contribution."""
    g = gen(21)
    n, page, dim = 200, 16, 64
    kc, vc, ks, vs = make_cache(g, "e4m3", 13, 1, page, dim)
    k, v = ((randn(g, n, dim) * 100).clamp(-440, 440).to(F8) for _ in range(2))
    sk = torch.full((n,), 0.01, device="cuda")
    size = torch.linspace(-50, 10, n, device="cuda")
    sv = torch.exp2(size * order if order > 0 else size.flip(0)).contiguous()
    t = torch.arange(n, device="cuda")
    kc[t // page, 0, t % page], vc[t // page, 0, t % page] = k.view(torch.uint8), v.view(torch.uint8)
    ks[t // page, 0, t % page], vs[t // page, 0, t % page] = sk, sv
    q = (randn(g, 1, 4, dim) * 3).half()
    out, lse = torch.empty_like(q), torch.empty(1, 4, device="cuda")
    table = torch.arange(13, dtype=torch.int32, device="cuda")[None].contiguous()
    qgemv.attn_decode(h, qgemv.attn_decode_desc(qgemv.kv_cache(kc, vc, ks, vs), q, table, ints([n]), out, 0.5, lse=lse))
    kk, vv = k.double() * sk.double()[:, None], v.double() * sv.double()[:, None]
    o, want, pv, qk = attend_reference(q[0].double(), kk, vv, 0.5)
    score = steps(dim) * qk + 2.0 ** -21 * qk
    within(lse[0], want, score + steps(n) + 2.0 ** -20 + 2.0 ** -22 * want.abs(), "lse")
    # a weight below 2^-14 of the largest is rounded to 2^-25 of it, by each of the n tokens and for the largest code
    p = torch.softmax(q[0].double() @ kk.t() * 0.5, -1)
    lost = n * 2.0 ** -25 * 448 * (p * sv.double()).amax(-1)
    tol = HALF_ULP[out.dtype] * o.abs() + TINY[out.dtype] + (2 * score[:, None] + 2 * steps(n) + 2.0 ** -16) * pv + lost[:, None]
    # outputs past fp16's range are infinities
    far, inside = o.abs() - tol >= 65520, o.abs() + tol < 65504
    assert torch.equal(out[0][far].double(), torch.sign(o[far]) * math.inf)
    within(out[0][inside], o[inside], tol[inside], "out")


def test_attention_rows_with_infinite_scores(h):
    def edit(table, lens, q, kc, vc):
        kc[table[0, 0].item(), :, :2] = -math.inf  # tokens 0 and 1 of request 0: every score -inf
        q[0].abs_()
    got, lse, q, ref, scale, _ = attend_case(h, [2, 30], 4, 1, 64, "f16", "f16", 16, edit=edit)
    assert (got[0] == 0).all() and (lse[0] == -math.inf).all()
    check_attend(got, lse, q, ref, scale, rows=[1])


def test_attention_skips_pages_outside_the_cache_and_reports_them(h):
    def edit(table, lens, q, kc, vc):
        table[0, 1] = kc.shape[0]
        table[1, 0] = -4
    got, lse, q, ref, scale, _ = attend_case(h, [40, 20, 33], 8, 2, 128, "bf16", "bf16", 16, edit=edit)
    assert qgemv.check_error(h) == qgemv.ERR_BAD_INDEX
    keep = [torch.cat([x[:16], x[32:]]) for x in ref[0]], [x[16:] for x in ref[1]]
    check_attend(got, lse, q, [*keep, ref[2]], scale)


def test_attention_clamps_lengths_out_of_range_and_reports_them(h):
    def edit(table, lens, q, kc, vc):
        lens[0], lens[1] = 1000, -5
    got, lse, q, ref, scale, _ = attend_case(h, [48, 20], 8, 2, 128, "f16", "f16", 16, edit=edit, width=3)
    assert qgemv.check_error(h) == qgemv.ERR_BAD_INDEX
    check_attend(got, lse, q, [ref[0], (ref[1][0][:0], ref[1][1][:0])], scale)


@pytest.mark.parametrize("typ", ["bf16", "e4m3"])
def test_store_and_attention_past_32_bits_of_cache(h, typ):
    """Pages more than 2^32 elements into the cache."""
    page, hk, dim = 64, 8, 128
    pages = 2 ** 32 // (page * hk * dim) + 40
    dt = torch.uint8 if typ == "e4m3" else torch.bfloat16
    kc, vc = (torch.empty(pages, hk, page, dim, dtype=dt, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(pages, hk, page, device="cuda") for _ in range(2)) if typ == "e4m3" else (None, None)
    cache = qgemv.kv_cache(kc, vc, ks, vs)
    g = gen(31)
    n = 150
    mine = torch.tensor([pages - 1, 3, pages - 20], device="cuda")
    t = torch.arange(n, device="cuda")
    slots = mine[t // page] * page + t % page
    k, v = (randn(g, n, hk * dim).bfloat16() for _ in range(2))
    qgemv.kv_store(h, qgemv.kv_store_desc(cache, k, v, slots, t.int()))
    q = (randn(g, 1, hk * 2, dim) * 2).bfloat16()
    out, lse = torch.empty_like(q), torch.empty(1, hk * 2, device="cuda")
    table = mine.int()[None].contiguous()
    qgemv.attn_decode(h, qgemv.attn_decode_desc(cache, q, table, ints([n]), out, dim ** -0.5, lse=lse))
    assert qgemv.check_error(h) == qgemv.OK
    at = (mine[t // page], slice(None), t % page)
    if typ == "e4m3":
        stored = [c[at].view(F8).double() * s[at].double()[..., None] for c, s in ((kc, ks), (vc, vs))]
    else:
        stored = [c[at].double() for c in (kc, vc)]
        assert torch.equal(kc[at].reshape(n, -1), k) and torch.equal(vc[at].reshape(n, -1), v)
    check_attend(out, lse, q, [stored], dim ** -0.5)


def test_attention_repeats_bit_for_bit_on_another_stream_and_in_a_graph(h):
    side = torch.cuda.Stream()
    lens = [4000, 17, 900, 0, 2500, 1]
    a, la, q, ref, scale, d = attend_case(h, lens, 32, 8, 128, "bf16", "bf16", 16, seed=4)
    b, lb, *_ = attend_case(h, lens, 32, 8, 128, "bf16", "bf16", 16, seed=4, stream=side)
    assert torch.equal(a, b) and torch.equal(la, lb)
    out = d.keep[2]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qgemv.attn_decode(h, d)
    out.fill_(NAN)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, b)


# ------------------------------------------------------------------------------ adapters
def lora_case(h, rows, used, loaded, rank, K, N, typ, out, seed=1, ids=None, ranks=None, base=True, inplace=False, pad=0, scales=True):
    g = gen(seed)
    dt, ot = TYPES[typ], TYPES[out]
    x = randn(g, rows, K + 8).to(dt)[:, :K]
    ranks = ints(ranks) if ranks is not None else None
    r_of = ranks.clamp(0, rank).tolist() if ranks is not None else [rank] * loaded
    A, B = (randn(g, loaded, rank, K) * K ** -0.5).to(dt), (randn(g, loaded, N, rank) * 0.3).to(dt)
    for a, r in enumerate(r_of):  # past an adapter's rank
        A[a, r:], B[a, :, r:] = NAN, NAN
    if ids is None:
        pool = torch.randperm(loaded, generator=g, device="cuda")[:used]
        ids = torch.cat([pool, pool[torch.randint(0, used, (rows,), generator=g, device="cuda")]])[:rows].int()
        ids = ids[torch.randperm(rows, generator=g, device="cuda")].contiguous()
    else:
        ids = ints(ids)
    sc = torch.rand(loaded, generator=g, device="cuda") + 0.5 if scales else None
    wide = torch.full((rows, N + pad), NAN, device="cuda").to(ot)
    y = wide[:, :N]
    b = None
    if base:
        b = torch.empty_like(wide)[:, :N]
        b.copy_(randn(g, rows, N).to(ot))
    b64 = b.double() if base else torch.zeros(rows, N, device="cuda", dtype=torch.float64)
    if inplace:
        y.copy_(b)
        b = y
    d = qgemv.lora_desc(x, A, B, ids, y, base=b, ranks=ranks, scales=sc)
    qgemv.run_lora(h, d)
    torch.cuda.synchronize()
    assert not pad or wide[:, N:].isnan().all()
    ref, tol = b64.clone(), torch.zeros_like(b64)
    for a in set(ids.tolist()):
        if not 0 <= a < loaded:
            continue
        m, r = (ids == a).nonzero()[:, 0], r_of[a]
        s = float(sc[a]) if scales else 1.0
        low = x[m].double() @ A[a, :r].double().t()
        near = steps(K) * (x[m].double().abs() @ A[a, :r].double().abs().t())
        if r:
            # the inner sums keep fp32's relative precision against the row's largest of them
            near = near + 2.0 ** -21 * low.abs().amax(-1, keepdim=True)
        Bd = B[a, :, :r].double()
        ref[m] += s * (low @ Bd.t())
        tol[m] += s * (near @ Bd.abs().t() + steps(r) * (low.abs() @ Bd.abs().t()))
    within(y, ref, tol + HALF_ULP[ot] * ref.abs() + 2.0 ** -22 * (b64.abs() + ref.abs()) + TINY[ot], "y")
    return y, ids, b64, d


LORAS = [  # rows, used, loaded, rank, K, N, type, out
    (1, 1, 1, 8, 8, 1, "f16", "f32"), (1, 1, 3, 16, 4096, 6144, "f16", "f32"), (2, 1, 2, 16, 1024, 77, "bf16", "f32"),
    (7, 3, 4, 24, 264, 130, "f16", "f16"), (9, 9, 9, 64, 2056, 999, "bf16", "bf16"), (33, 2, 2, 8, 512, 64, "bf16", "f32"),
    (64, 40, 41, 32, 1024, 520, "f16", "f32"), (65, 3, 5, 128, 640, 300, "bf16", "f32"), (130, 130, 130, 16, 256, 96, "f16", "f32"),
    (200, 1, 1, 40, 776, 1001, "f16", "f32"), (513, 7, 9, 64, 512, 200, "bf16", "f32"), (1000, 4, 4, 32, 136, 65, "f16", "bf16")]


@pytest.mark.parametrize("rows,used,loaded,rank,K,N,typ,out", LORAS)
def test_adapters_match_64_bits(h, rows, used, loaded, rank, K, N, typ, out):
    lora_case(h, rows, used, loaded, rank, K, N, typ, out, pad=8 if N % 2 else 0)
    assert qgemv.check_error(h) == qgemv.OK


def test_adapters_of_more_rows_than_the_workspace_holds_at_once(h):
    lora_case(h, 130001, 3, 3, 8, 16, 9, "f16", "f32")
    lora_case(h, 30011, 2, 2, 128, 24, 40, "bf16", "bf16", pad=8)


@pytest.mark.parametrize("rank,typ", [(8, "f16"), (64, "bf16"), (128, "f16")])
def test_adapters_of_ragged_ranks_ignore_what_lies_past_them(h, rank, typ):
    ranks = [0, 1, rank, rank // 2 + 1, rank - 1, 2 * rank, -3]
    y, ids, base, _ = lora_case(h, 60, 7, 7, rank, 328, 210, typ, "f32", ranks=ranks, scales=False)
    for a in (0, 6):
        assert torch.equal(y[ids == a].double(), base[ids == a])


def test_adapters_in_place_without_a_base_and_without_scales(h):
    lora_case(h, 40, 5, 6, 16, 512, 333, "f16", "f32", inplace=True)
    lora_case(h, 40, 5, 6, 16, 512, 333, "bf16", "bf16", inplace=True)
    lora_case(h, 40, 5, 6, 16, 512, 333, "f16", "f32", base=False, scales=False)


def test_adapter_rows_without_an_adapter_keep_the_base(h):
    ids = [-1, 2, -1, -1, 0, 2] + [-1] * 70
    y, ids, base, _ = lora_case(h, 76, 0, 3, 16, 128, 100, "f16", "f32", ids=ids)
    assert torch.equal(y[ids < 0].double(), base[ids < 0])
    y, ids, base, _ = lora_case(h, 5, 0, 3, 16, 128, 100, "f16", "f32", ids=[-1] * 5)
    assert torch.equal(y.double(), base) and qgemv.check_error(h) == qgemv.OK
    y, ids, base, _ = lora_case(h, 5, 0, 3, 16, 128, 100, "f16", "f32", ids=[0, 3, -2, 2, 1 << 30])
    assert torch.equal(y[1:3].double(), base[1:3]) and qgemv.check_error(h) == qgemv.ERR_BAD_INDEX


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** 10])
def test_adapters_keep_small_and_large_inner_sums(h, size):
    """Inner sums near fp16's ends: the second product takes them in full precision all the same."""
    g = gen(8)
    x, A = randn(g, 20, 512).half(), (randn(g, 2, 16, 512) * size).half()
    B = (randn(g, 2, 90, 16) / size).half()
    y, ids = torch.empty(20, 90, device="cuda"), ints([0, 1] * 10)
    qgemv.run_lora(h, qgemv.lora_desc(x, A, B, ids, y))
    for m in range(20):
        a = m % 2
        low = A[a].double() @ x[m].double()
        near = steps(512) * (A[a].double().abs() @ x[m].double().abs()) + 2.0 ** -21 * low.abs().max()
        ref = B[a].double() @ low
        within(y[m], ref, B[a].double().abs() @ (near + steps(16) * low.abs()) + 2.0 ** -22 * ref.abs(), f"row {m}")


@pytest.mark.parametrize("rows", [20, 300])
@pytest.mark.parametrize("typ", ["f16", "bf16"])
def test_infinities_and_nan_stay_with_their_adapter_and_row(h, rows, typ):
    """Neighbouring rows of other adapters, and of none, come out bit for bit as beside sound ones."""
    g = gen(12)
    x, A, B = randn(g, rows, 256).to(TYPES[typ]), randn(g, 5, 32, 256).to(TYPES[typ]), randn(g, 5, 70, 32).to(TYPES[typ])
    base, ids = randn(g, rows, 70), ints([(m * 7 + m // 6) % 6 - 1 for m in range(rows)])

    def run():
        y = torch.empty(rows, 70, device="cuda")
        qgemv.run_lora(h, qgemv.lora_desc(x, A, B, ids, y, base=base))
        torch.cuda.synchronize()
        return y

    sound = run()
    assert sound.isfinite().all()
    B[1, 3, :] = float("inf")
    B[2] = NAN
    A[3, 5, 9] = float("inf")
    x[9] = NAN
    sick = (ids >= 1) & (ids <= 3)
    sick[9] = True
    y = run()
    assert torch.equal(y[~sick], sound[~sick])
    others = y[ids == 1][:, [n for n in range(70) if n != 3]]
    assert others.isfinite().all() and not y[ids == 1][:, 3].isfinite().any()
    assert not y[(ids == 2) | (ids == 3)].isfinite().any()


def test_adapters_repeat_bit_for_bit_in_a_graph(h):
    y, _, _, d = lora_case(h, 70, 20, 20, 32, 1024, 700, "bf16", "f32", seed=3)
    first = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qgemv.run_lora(h, d)
    y.fill_(NAN)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, y)


# ------------------------------------------------------------------------------ refusals
def test_refusals_launch_nothing(h):
    L = qgemv.lib()
    BAD, ARG, ALIGN = qgemv.ERR_BAD_SHAPE, qgemv.ERR_INVALID_ARG, qgemv.ERR_MISALIGNED

    def tries(fn, make, edits):
        for want, edit in edits:
            d = make()
            for name, value in edit.items():
                part = d
                *path, last = name.split(".")
                for p in path:
                    part = getattr(part, p)
                setattr(part, last, value)
            assert fn(h.ptr, d, None) == want, edit
        assert fn(None, make(), None) == ARG and fn(h.ptr, None, None) == ARG

    i32 = lambda *n: torch.full(n, 0, dtype=torch.int32, device="cuda")  # noqa: E731
    half = lambda *n: torch.zeros(*n, dtype=torch.float16, device="cuda")  # noqa: E731
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    tries(L.qgemv_page_plan, lambda: qgemv.page_plan_desc(i32(2), i32(2), i32(2, 3), i32(5), i32(1), 16, i32(2), slots, i32(4)),
          [(BAD, {"requests": -1}), (BAD, {"page_size": 0}), (BAD, {"table_width": 0}), (BAD, {"table_stride": 2}),
           (BAD, {"capacity": -1}), (BAD, {"capacity": 1 << 31}), (ARG, {"cached": None}), (ARG, {"counts": None}),
           (ARG, {"slots": None}), (ARG, {"free_count": None}), (ALIGN, {"slots": slots.data_ptr() + 8})])
    k, v = half(3, 2, 16, 64), half(3, 2, 16, 64)
    rows, qo = half(4, 256), half(4, 2, 64)
    rope = torch.zeros(10, 64, device="cuda")
    caches = [(ARG, {"cache.k": None}), (ARG, {"cache.type": 0}), (ARG, {"cache.type": 4}), (ARG, {"cache.type": 3}),
              (BAD, {"cache.pages": 0}), (BAD, {"cache.page_size": 12}), (BAD, {"cache.page_size": 24}), (BAD, {"cache.head_dim": 96}),
              (BAD, {"cache.kv_heads": 0}), (BAD, {"cache.page_stride": 100}), (ALIGN, {"cache.page_stride": 2 * 16 * 64 + 4}),
              (ALIGN, {"cache.v": v.data_ptr() + 2})]
    tries(L.qgemv_kv_store, lambda: qgemv.kv_store_desc(qgemv.kv_cache(k, v), rows[:, :128], rows[:, 128:], slots, i32(4), rope,
                                                        q=rows[:, :128], q_out=qo),
          caches + [(BAD, {"tokens": -1}), (ARG, {"k": None}), (ARG, {"q": None}), (ARG, {"slots": None}), (ARG, {"in_type": 3}),
                    (ARG, {"q_type": 0}), (ARG, {"interleaved": 2}), (BAD, {"rot_dim": 8}), (BAD, {"rot_dim": 80}), (BAD, {"q_heads": 0}),
                    (BAD, {"k_stride": 64}), (BAD, {"rope_positions": 0}), (ALIGN, {"k_stride": 250}), (ALIGN, {"q": rows.data_ptr() + 4})])
    q, out = half(2, 4, 64), half(2, 4, 64)
    tries(L.qgemv_attn_decode, lambda: qgemv.attn_decode_desc(qgemv.kv_cache(k, v), q, i32(2, 3), i32(2), out, 0.1),
          caches + [(BAD, {"requests": -1}), (BAD, {"q_heads": 3}), (BAD, {"q_heads": 0}), (BAD, {"table_width": 0}), (BAD, {"q_stride": 64}),
                    (ARG, {"type": 0}), (ARG, {"type": 2}), (ARG, {"window": -1}), (ARG, {"scale": NAN}), (ARG, {"q": None}),
                    (ARG, {"lens": None}), (ALIGN, {"out_stride": 260}), (ALIGN, {"out": out.data_ptr() + 8})])
    x, A, B, y = half(3, 64), half(2, 16, 64), half(2, 24, 16), torch.zeros(3, 24, device="cuda")
    tries(L.qgemv_run_lora, lambda: qgemv.lora_desc(x, A, B, i32(3), y),
          [(BAD, {"rows": -1}), (BAD, {"N": 0}), (BAD, {"K": 60}), (BAD, {"K": 0}), (BAD, {"rank": 12}), (BAD, {"rank": 136}), (BAD, {"rank": 0}),
           (BAD, {"adapters": 0}), (BAD, {"x_stride": 32}), (BAD, {"y_stride": 8}), (ARG, {"type": 0}), (ARG, {"out": 3}), (ARG, {"A": None}),
           (ARG, {"x": None}), (ARG, {"ids": None}), (ALIGN, {"x": x.data_ptr() + 8}), (ALIGN, {"x_stride": 68}), (ALIGN, {"B": B.data_ptr() + 2})])
    assert qgemv.check_error(h) == qgemv.OK


def test_empty_calls_do_nothing(h):
    k, v = (torch.zeros(3, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    rows = torch.empty(0, 128, device="cuda")
    qgemv.kv_store(h, qgemv.kv_store_desc(qgemv.kv_cache(k, v), rows, rows, none.long(), none))
    q = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    qgemv.attn_decode(h, qgemv.attn_decode_desc(qgemv.kv_cache(k, v), q, torch.empty(0, 3, dtype=torch.int32, device="cuda"), none, q, 1.0))
    A, B = (torch.zeros(1, 8, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    qgemv.run_lora(h, qgemv.lora_desc(q[:, 0], A, B.transpose(1, 2).contiguous(), none, torch.empty(0, 64, device="cuda")))
    assert qgemv.check_error(h) == qgemv.OK


def test_descriptions_refuse_wrong_tensors():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        qgemv.kv_cache(k, k.bfloat16())
    with pytest.raises(TypeError):
        qgemv.kv_cache(k.to(torch.uint8), k.to(torch.uint8))
    with pytest.raises(TypeError):
        qgemv.kv_cache(k.transpose(1, 2), k.transpose(1, 2))
    c, q = qgemv.kv_cache(k, k), torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    lens, table = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        qgemv.attn_decode_desc(c, q, table, lens.long(), q, 1.0)
    with pytest.raises(ValueError):
        qgemv.attn_decode_desc(c, q, table[:1], lens, q, 1.0)
    with pytest.raises(ValueError):
        qgemv.lora_desc(k[0, 0], k[0], k[0], lens, k[0, 0])


def test_attention_that_gives_up_waiting_reports_it_and_recovers(h):
    lens = [700, 30]
    want, lse, *_ = attend_case(h, lens, 8, 2, 128, "f16", "f16", 16, seed=9)
    qgemv.set_option(h, qgemv.OPT_SPIN_LIMIT_NS, 2_000_000)
    qgemv.set_option(h, qgemv.OPT_TEST_STALL, 1)
    try:
        attend_case(h, lens, 8, 2, 128, "f16", "f16", 16, seed=9)
        assert qgemv.check_error(h) == qgemv.ERR_TIMEOUT
    finally:
        qgemv.set_option(h, qgemv.OPT_TEST_STALL, 0)
        qgemv.set_option(h, qgemv.OPT_SPIN_LIMIT_NS, 1_000_000_000)
    got, lse2, *_ = attend_case(h, lens, 8, 2, 128, "f16", "f16", 16, seed=9)
    assert qgemv.check_error(h) == qgemv.OK
    assert torch.equal(want, got) and torch.equal(lse, lse2)
