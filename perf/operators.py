"""The operators around the quantised projections of one decode step, as measured cases.

Four operators of a serving step, each in its plain form (elementary torch operations in 32 bits)
and as a call of the library:

  plan    block tables and slot maps from request lengths, pages taken from a free list
  store   q and k rotated, k and v written into the paged key-value cache through the slot map
  attend  attention of one new token per request over the paged cache
  lora    low-rank adapters of many requests added to a shared projection's output

Head layouts and widths are those of the projections that the library is benchmarked on
(hidden 4096: 32 query and 8 key-value heads of 128, QKV 6144 wide; MLP 12288 and 14336 wide)
and common variations of them.
"""
import math
import random

import torch

own = False

F32, F16, BF16, E4M3 = "f32", "f16", "bf16", "e4m3"
_TORCH = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
_BYTES = {F32: 4, F16: 2, BF16: 2, E4M3: 1}
_handles = {}


def _handle():
    """The library handle that a program keeps for its device."""
    from quantized_weight_dequant_gb300 import qgemv
    d = torch.cuda.current_device()
    if d not in _handles:
        _handles[d] = qgemv.create(d)
    return _handles[d]


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 requests: the smallest planning call, all latency
        dict(name="plan decode 64", op="plan", requests=64, cached_hi=8000, fresh_hi=1, long_share=0.0, page=16, pad=0,
             short=0),
        # decode requests mixed with prompt chunks, the token arrays padded for a captured step
        dict(name="plan mixed 1024", op="plan", requests=1024, cached_hi=16000, fresh_hi=4096, long_share=0.25, page=32,
             pad=1111, short=37),
        # what follows the QKV projection of 64 decode requests: fp32 rows of 6144 into an fp16 cache
        dict(name="store decode 64 f16", op="store", tokens=64, q_heads=32, kv_heads=8, dim=128, rot=128, pairs="halves",
             src=F32, kv=F16, q=F16, page=16, pad=3),
        # a prompt of 8191 tokens into an 8-bit cache, pairs side by side
        dict(name="store prompt 8191 e4m3", op="store", tokens=8191, q_heads=32, kv_heads=8, dim=128, rot=128,
             pairs="neighbours", src=BF16, kv=E4M3, q=BF16, page=64, pad=0),
        # a single user's chat at a thousand tokens: latency
        dict(name="attend 1 x 1000 f16", op="attend", requests=1, len_lo=1000, len_hi=1000, empty=0, q_heads=32, kv_heads=8,
             dim=128, kv=F16, q=F16, page=16, window=0),
        # continuous batching: 64 requests of very different lengths, two slots idle
        dict(name="attend 64 ragged bf16", op="attend", requests=64, len_lo=1, len_hi=6000, empty=2, q_heads=32, kv_heads=8,
             dim=128, kv=BF16, q=BF16, page=16, window=0),
        # many short requests of a model with one key-value head per query head and a sliding window
        dict(name="attend 256 window f16", op="attend", requests=256, len_lo=9, len_hi=900, empty=0, q_heads=16, kv_heads=16,
             dim=64, kv=F16, q=F16, page=32, window=300),
        # long documents in an 8-bit cache
        dict(name="attend 16 long e4m3", op="attend", requests=16, len_lo=9000, len_hi=70000, empty=0, q_heads=32, kv_heads=8,
             dim=128, kv=E4M3, q=BF16, page=64, window=0),
        # the largest: 32 requests of about 32 thousand tokens, 8 query heads per key-value head
        dict(name="attend 32 x 33k bf16", op="attend", requests=32, len_lo=24000, len_hi=44000, empty=0, q_heads=64,
             kv_heads=8, dim=128, kv=BF16, q=BF16, page=16, window=0),
        # one request with an adapter on its QKV projection: latency
        dict(name="lora 1 row r16", op="lora", rows=1, used=1, loaded=32, rank=16, ragged=False, none=0, K=4096, N=6144,
             typ=F16),
        # a decode batch in which nearly every request brings its own adapter, of ranks up to 64
        dict(name="lora 64 rows of 48 r64", op="lora", rows=64, used=48, loaded=64, rank=64, ragged=True, none=5, K=4096,
             N=12288, typ=BF16),
        # prompt chunks of four requests on the widest projection
        dict(name="lora 2048 rows of 4 r32", op="lora", rows=2048, used=4, loaded=16, rank=32, ragged=False, none=0, K=4096,
             N=14336, typ=F16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "attend", "attend", "lora"])
    if op == "plan":
        c = dict(op=op, requests=_log(rng, 1, 1024), cached_hi=_log(rng, 1, 30000), fresh_hi=_log(rng, 1, 4096),
                 long_share=rng.choice([0.0, 0.25]), page=rng.choice([8, 16, 32, 64, 128]), pad=rng.choice([0, 17, 300]),
                 short=rng.choice([0, 0, 5]))
        return c
    if op == "store":
        kv = rng.choice([F16, BF16, E4M3])
        dim = rng.choice([64, 128, 128, 256])
        hk = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 8191), q_heads=hk * rng.choice([1, 2, 4, 7]), kv_heads=hk, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), pairs=rng.choice(["halves", "neighbours"]),
                    src=rng.choice([F32, F16, BF16]), kv=kv, q=kv if kv != E4M3 else rng.choice([F16, BF16]),
                    page=rng.choice([8, 16, 32, 64, 128]), pad=rng.choice([0, 1, 9]))
    if op == "attend":
        kv = rng.choice([F16, BF16, E4M3])
        hk = rng.choice([1, 2, 4, 8, 8])
        group = rng.choice([1, 2, 4, 5, 8, 16])
        dim = rng.choice([64, 128, 128, 256])
        r = _log(rng, 1, 256)
        hi = _log(rng, 1, max(2, min(100000, 300000000 // (r * hk * dim))))  # tokens x heads x dim stay below the largest listed
        return dict(op=op, requests=r, len_lo=max(1, hi // rng.choice([1, 3, 100])), len_hi=hi, empty=rng.choice([0, 0, 1]) if r > 1 else 0,
                    q_heads=hk * group, kv_heads=hk, dim=dim, kv=kv, q=kv if kv != E4M3 else rng.choice([F16, BF16]),
                    page=rng.choice([8, 16, 32, 64, 128]), window=rng.choice([0, 0, 0, 127, 4096]))
    rows = _log(rng, 1, 2048)
    used = min(rows, _log(rng, 1, 64))
    K, N = rng.choice([(4096, 6144), (4096, 4096), (4096, 12288), (14336, 4096), (1024, 1000), (2056, 77)])
    return dict(op=op, rows=rows, used=used, loaded=used + rng.choice([0, 3]), rank=rng.choice([8, 16, 32, 64]),
                ragged=rng.choice([True, False]), none=rng.choice([0, 1, 3]) if rows > used + 3 else 0, K=K, N=N,
                typ=rng.choice([F16, BF16]))


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly over their logarithm."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _plan_lengths(case):
    """(cached, fresh) of the case, before their order is drawn."""
    n = case["requests"]
    cached = [v - 1 for v in _spread(n, 1, case["cached_hi"] + 1)]
    long = int(n * case["long_share"])
    fresh = _spread(long, 1, case["fresh_hi"]) if long else []
    fresh = fresh + [1 if case["long_share"] else case["fresh_hi"] if n == 1 else 1 + (i * 7919) % case["fresh_hi"]
                     for i in range(n - long)]
    return cached, fresh[:n]


def _cdiv(a, b):
    return -(-a // b)


def _lens(case):
    n = case["requests"] - case["empty"]
    return [0] * case["empty"] + _spread(n, case["len_lo"], case["len_hi"])


def _ranks(case):
    """Rank of the adapters in the order in which they are used."""
    return [max(1, case["rank"] >> (i % 3)) - (1 if i % 4 == 3 and case["rank"] >> (i % 3) > 1 else 0) if case["ragged"] else case["rank"]
            for i in range(case["loaded"])]


def work(case):
    if case["op"] == "plan":
        cached, fresh = _plan_lengths(case)
        tokens, n = sum(fresh), case["requests"]
        pages = tokens // case["page"] + n // 2
        return {"bytes": 8 * n + 8 * n + 4 * n + 16 * (tokens + case["pad"]) + 8 * pages, "flops": 0}
    if case["op"] == "store":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        per = (hq + 2 * hk) * d * _BYTES[case["src"]] + hq * d * 2 + 2 * hk * d * _BYTES[case["kv"]] + 12 + 4 * case["rot"]
        per += 8 * hk if case["kv"] == E4M3 else 0
        return {"bytes": t * per, "flops": 3 * t * (hq + hk) * case["rot"]}
    if case["op"] == "attend":
        seen = sum(min(n, case["window"]) if case["window"] else n for n in _lens(case))
        hk, hq, d = case["kv_heads"], case["q_heads"], case["dim"]
        per = 2 * hk * d * _BYTES[case["kv"]] + (8 * hk if case["kv"] == E4M3 else 0)
        return {"bytes": seen * per + case["requests"] * hq * (4 * d + 4) + 4 * seen // case["page"], "flops": 4 * seen * hq * d}
    m, k, n = case["rows"], case["K"], case["N"]
    rank = sum(_ranks(case)[:case["used"]])
    return {"bytes": rank * (k + n) * 2 + m * k * 2 + m * n * 8 + 4 * m,
            "flops": 2 * (m - case["none"]) * (rank / case["used"]) * (k + n)}


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    order = random.Random(seed)
    s = {"case": dict(case)}
    {"plan": _prepare_plan, "store": _prepare_store, "attend": _prepare_attend, "lora": _prepare_lora}[case["op"]](case, g, order, s)
    return s


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * scale


def _prepare_plan(case, g, order, s):
    cached, fresh = _plan_lengths(case)
    order.shuffle(cached)
    order.shuffle(fresh)
    n, p = case["requests"], case["page"]
    have = [_cdiv(c, p) for c in cached]
    want = sum(_cdiv(c + f, p) - h for c, f, h in zip(cached, fresh, have))
    width = _cdiv(max(cached) + max(fresh), p) + 3
    free = max(1, want + 50 - (case["short"] + 50 if case["short"] else 0))  # `short` pages too few
    ids = torch.randperm(sum(have) + free + 100, generator=g, device="cuda").to(torch.int32)
    s["cached"], s["fresh"], have_d = _ints(cached), _ints(fresh), _ints(have)
    col = torch.arange(width, device="cuda")[None]
    at = (torch.cumsum(have_d, 0) - have_d)[:, None] + col
    s["table"] = torch.where(col < have_d[:, None], ids[at.clamp(max=ids.numel() - 1)], -1).to(torch.int32).contiguous()
    s["free"] = ids[sum(have):sum(have) + free + 100].contiguous()  # a stack with room above its top
    s["free_count"] = _ints([free])
    cap = s["cap"] = sum(fresh) + case["pad"]
    s["out"] = {"lens": torch.empty(n, dtype=torch.int32, device="cuda"),
                "offsets": torch.empty(n + 1, dtype=torch.int32, device="cuda"),
                "slots": torch.empty(cap, dtype=torch.int64, device="cuda"),
                "positions": torch.empty(cap, dtype=torch.int32, device="cuda"),
                "owners": torch.empty(cap, dtype=torch.int32, device="cuda"),
                "counts": torch.empty(4, dtype=torch.int32, device="cuda")}
    if own:
        from quantized_weight_dequant_gb300 import qgemv
        s["desc"] = qgemv.page_plan_desc(s["cached"], s["fresh"], s["table"], s["free"], s["free_count"], p, **s["out"])


def _cache(case, pages, fill):
    """(k, v, k_scale, v_scale): pages of [kv_heads, page, dim]; 8-bit ones as bytes with a scale per token and head."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case["kv"] != E4M3:
        return fill(shape, _TORCH[case["kv"]]), fill(shape, _TORCH[case["kv"]]), None, None
    scale = lambda: fill(shape[:3], torch.float32).abs() * 2e-3 + 5e-3  # noqa: E731
    k, v = ((fill(shape, torch.float16) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    return k, v, scale(), scale()


def _rope(positions, rot):
    """cos and sin of position x frequency: [positions, rot], the cosines first."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _prepare_store(case, g, order, s):
    t, hq, hk, d, p = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    src = _randn(g, t, (hq + 2 * hk) * d, scale=1.5).to(_TORCH[case["src"]])  # one fused projection's rows
    s["q"], s["k"], s["v"] = src[:, :hq * d], src[:, hq * d:(hq + hk) * d], src[:, (hq + hk) * d:]
    pages = _cdiv(t, p) + 5
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(case, pages, lambda shape, dtype: _randn(g, *shape).to(dtype))
    slots = torch.randperm(pages * p, generator=g, device="cuda")[:t]
    if t > 64:  # prompts fill pages in order
        page = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(t, device="cuda") + 3
        slots = page[i // p] * p + i % p
    s["positions"] = (torch.randperm(16384, generator=g, device="cuda")[:t] if t <= 64
                      else torch.arange(t, device="cuda") + 100).to(torch.int32)
    pad = min(case["pad"], t - 1)
    if pad:  # rows of a padded step: no slot, no position
        slots[-pad:] = -1
        s["positions"][-pad:] = -1
    s["slots"] = slots.contiguous()
    s["rope"] = _rope(16384, case["rot"])
    s["q_out"] = torch.empty(t, hq, d, dtype=_TORCH[case["q"]], device="cuda")
    if own:
        from quantized_weight_dequant_gb300 import qgemv
        cache = qgemv.kv_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["desc"] = qgemv.kv_store_desc(cache, s["k"], s["v"], s["slots"], s["positions"], s["rope"],
                                        interleaved=case["pairs"] == "neighbours", q=s["q"], q_out=s["q_out"])


def _prepare_attend(case, g, order, s):
    lens = _lens(case)
    order.shuffle(lens)
    n, p = case["requests"], case["page"]
    have = [_cdiv(v, p) for v in lens]
    pages = sum(have) + 7
    width = max(have + [1]) + 2
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(
        case, pages, lambda shape, dtype: _randn(g, *shape, dtype=dtype))
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    have_d, col = _ints(have), torch.arange(width, device="cuda")[None]
    at = (torch.cumsum(have_d, 0) - have_d)[:, None] + col
    s["table"] = torch.where(col < have_d[:, None], ids[at.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    s["lens"], s["width"] = _ints(lens), max(have + [1])
    s["scale"] = case["dim"] ** -0.5
    s["q"] = _randn(g, n, case["q_heads"], case["dim"], scale=2.0).to(_TORCH[case["q"]])
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(n, case["q_heads"], dtype=torch.float32, device="cuda")
    if own:
        from quantized_weight_dequant_gb300 import qgemv
        cache = qgemv.kv_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["desc"] = qgemv.attn_decode_desc(cache, s["q"], s["table"], s["lens"], s["out"], scale=s["scale"],
                                           window=case["window"], lse=s["lse"])


def _prepare_lora(case, g, order, s):
    m, k, n, r, used, loaded = (case[x] for x in ("rows", "K", "N", "rank", "used", "loaded"))
    typ = _TORCH[case["typ"]]
    s["x"] = _randn(g, m, k).to(typ)
    s["A"] = (_randn(g, loaded, r, k) * k ** -0.5).to(typ)
    s["B"] = (_randn(g, loaded, n, r) * 0.3).to(typ)
    s["base"] = _randn(g, m, n)
    who = list(range(loaded))
    order.shuffle(who)
    ranks = [0] * loaded
    for i, v in enumerate(_ranks(case)):
        ranks[who[i]] = v
    ids = [who[i * used // (m - case["none"])] for i in range(m - case["none"])]  # every used adapter, in runs of rows
    ids += [-1] * case["none"]
    if m <= 256:
        order.shuffle(ids)
    s["ids"], s["ranks"] = _ints(ids), _ints(ranks)
    s["scales"] = torch.rand(loaded, generator=g, device="cuda") * 1.5 + 0.5
    s["y"] = torch.empty(m, n, dtype=torch.float32, device="cuda")
    if own:
        from quantized_weight_dequant_gb300 import qgemv
        s["desc"] = qgemv.lora_desc(s["x"], s["A"], s["B"], s["ids"], s["y"], base=s["base"], ranks=s["ranks"], scales=s["scales"])


# ------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "store": _plain_store, "attend": _plain_attend, "lora": _plain_lora}[op](s)
    from quantized_weight_dequant_gb300 import qgemv
    if op == "plan":
        qgemv.page_plan(_handle(), s["desc"])
        return {"table": s["table"], **s["out"]}
    if op == "store":
        qgemv.kv_store(_handle(), s["desc"])
        return _stored(s, s["q_out"])
    if op == "attend":
        qgemv.attn_decode(_handle(), s["desc"])
        return {"out": s["out"], "lse": s["lse"]}
    qgemv.run_lora(_handle(), s["desc"])
    return {"y": s["y"]}


def _stored(s, q):
    if s["case"]["kv"] != E4M3:
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
    f8 = torch.float8_e4m3fn
    return {"q": q, "k": s["k_cache"].view(f8), "v": s["v_cache"].view(f8), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_plan(s):
    p, cap, free = s["case"]["page"], s["cap"], s["free"]
    table, width = s["table"], s["table"].shape[1]
    c, f = s["cached"].long().clamp(min=0), s["fresh"].long().clamp(min=0)
    end = torch.cumsum(f, 0)
    off = end - f
    f1 = torch.minimum(torch.minimum(f, (cap - off).clamp(min=0)), (width * p - c).clamp(min=0))
    have = (c + p - 1) // p
    need = (c + f1 + p - 1) // p - have
    base = torch.cumsum(need, 0) - need
    got = torch.minimum(need, (s["free_count"].long() - base).clamp(min=0))
    f2 = torch.where(got < need, (have + got) * p - c, f1)
    top = s["free_count"].long() - 1 - base
    col = torch.arange(width, device="cuda")[None]
    j = col - have[:, None]
    fresh_page = free[(top[:, None] - j).clamp(0, free.numel() - 1)]
    new_table = torch.where((j >= 0) & (j < got[:, None]), fresh_page, table)
    t = torch.arange(cap, device="cuda")
    owner = torch.searchsorted(end, t, right=True)
    inside = owner < c.numel()
    own_r = owner.clamp(max=c.numel() - 1)
    i = t - off[own_r]
    pos = c[own_r] + i
    page = new_table[own_r, (pos // p).clamp(max=width - 1)].long()
    ok = inside & (i < f2[own_r])
    return {"table": new_table, "lens": (c + f2).int(), "offsets": torch.cat([off, end[-1:]]).int(),
            "slots": torch.where(ok, page * p + pos % p, -1), "positions": torch.where(ok, pos, -1).int(),
            "owners": torch.where(inside, owner, -1).int(),
            "counts": torch.stack([end[-1], f2.sum(), got.sum(), (need - got).sum()]).int()}


def _rotate(x, cos, sin, rot, pairs):
    """x [tokens, heads, dim] with its first `rot` values turned by the angles of cos, sin [tokens, 1, rot / 2]."""
    if pairs == "halves":
        a, b, rest = x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_store(s):
    case = s["case"]
    t, hq, hk, d, p, rot = (case[x] for x in ("tokens", "q_heads", "kv_heads", "dim", "page", "rot"))
    pos, slots = s["positions"].long(), s["slots"]
    cs = s["rope"][pos.clamp(min=0)][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    q = _rotate(s["q"].float().reshape(t, hq, d), cos, sin, rot, case["pairs"])
    q = torch.where((pos >= 0)[:, None, None], q, 0.0).to(_TORCH[case["q"]])
    k = _rotate(s["k"].float().reshape(t, hk, d), cos, sin, rot, case["pairs"])
    v = s["v"].float().reshape(t, hk, d)
    # rows without a slot write the first row's values to the first row's slot once more
    row = torch.where(slots >= 0, torch.arange(t, device="cuda"), 0)
    page, at = slots[row] // p, slots[row] % p
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        if case["kv"] == E4M3:
            top = x.abs().amax(-1)
            sc = torch.where(top > 0, top / 448.0, 1.0)
            scale[page, :, at] = sc[row]
            cache[page, :, at] = (x / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)[row]
        else:
            cache[page, :, at] = x.to(cache.dtype)[row]
    return _stored(s, q)


def _plain_attend(s):
    case = s["case"]
    n, hq, hk, d, p = (case[x] for x in ("requests", "q_heads", "kv_heads", "dim", "page"))
    tab = s["table"][:, :s["width"]].long().clamp(min=0)
    span = s["width"] * p

    def rows(cache, scale):  # [requests, kv_heads, positions, dim] in 32 bits
        x = cache[tab]
        x = (x.view(torch.float8_e4m3fn).float() * scale[tab][..., None]) if case["kv"] == E4M3 else x.float()
        return x.transpose(1, 2).reshape(n, hk, span, d)

    t = torch.arange(span, device="cuda")[None]
    lens = s["lens"].long()[:, None]
    seen = (t < lens) & (t >= lens - case["window"]) if case["window"] else t < lens
    seen = seen[:, None, None]
    q = s["q"].float().reshape(n, hk, hq // hk, d)
    score = torch.matmul(q, rows(s["k_cache"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, rows(s["v_cache"], s["v_scale"])) / torch.where(total > 0, total, 1.0)
    return {"out": out.reshape(n, hq, d).to(s["q"].dtype), "lse": (top + torch.log(total)).reshape(n, hq)}


def _plain_lora(s):
    case = s["case"]
    m, r, loaded = case["rows"], case["rank"], case["loaded"]
    low = torch.matmul(s["x"].float(), s["A"].float().reshape(loaded * r, -1).t()).reshape(m, loaded, r)
    mine = s["ids"][:, None] == torch.arange(loaded, device="cuda")[None]
    mine = mine[..., None] & (torch.arange(r, device="cuda")[None] < s["ranks"][:, None])[None]
    low = torch.where(mine, low * s["scales"][:, None], 0.0).reshape(m, loaded * r)
    return {"y": s["base"] + torch.matmul(low, s["B"].float().transpose(1, 2).reshape(loaded * r, -1))}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"plan": _exact_plan, "store": _exact_store, "attend": _exact_attend, "lora": _exact_lora}[case["op"]](case, s)


def _exact_plan(case, s):
    """Request by request, as an allocator on the host would."""
    p, cap = case["page"], s["cap"]
    cached, fresh, table = s["cached"].tolist(), s["fresh"].tolist(), s["table"].tolist()
    stack = s["free"].tolist()[:int(s["free_count"][0])]
    slots, positions, owners, lens, offsets = [], [], [], [], [0]
    taken = short = 0
    for r, (c, f) in enumerate(zip(cached, fresh)):
        kept, stuck = 0, False
        for i in range(f):
            pos = c + i
            if len(slots) < cap:
                fits = pos // p < len(table[r])
                if fits and pos % p == 0:
                    if stack:
                        table[r][pos // p] = stack.pop()
                        taken += 1
                    else:
                        stuck, short = True, short + 1
                ok = fits and not stuck
                kept += ok
                slots.append(table[r][pos // p] * p + pos % p if ok else -1)
                positions.append(pos if ok else -1)
                owners.append(r)
        lens.append(c + kept)
        offsets.append(offsets[-1] + f)
    rest = cap - len(slots)
    i32 = torch.int32
    return {"table": _ints(table), "lens": _ints(lens), "offsets": _ints(offsets), "slots": _ints(slots + [-1] * rest, torch.int64),
            "positions": _ints(positions + [-1] * rest), "owners": _ints(owners + [-1] * rest),
            "counts": _ints([offsets[-1], sum(v >= 0 for v in slots), taken, short], i32)}


def _exact_store(case, s):
    t, hq, hk, d, p, rot = (case[x] for x in ("tokens", "q_heads", "kv_heads", "dim", "page", "rot"))
    half = rot // 2
    ok = s["slots"] >= 0
    table = s["rope"].double()[s["positions"].long().clamp(min=0)]
    first = torch.arange(half, device="cuda") * (2 if case["pairs"] == "neighbours" else 1)
    second = first + (1 if case["pairs"] == "neighbours" else half)

    def turn(x):
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(table[:, :half], table[:, half:])[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q = turn(s["q"].double().reshape(t, hq, d)) * (s["positions"] >= 0).double()[:, None, None]
    k, v = turn(s["k"].double().reshape(t, hk, d)), s["v"].double().reshape(t, hk, d)
    page, at = s["slots"][ok] // p, s["slots"][ok] % p
    got = {"q": q}
    for name, x in (("k", k), ("v", v)):
        if case["kv"] == E4M3:
            got[name] = None  # codes: what they stand for depends on the scale's own rounding
            sc = s[name + "_scale"].double()
            top = x.abs().amax(-1)
            sc[page, :, at] = torch.where(top > 0, top / 448.0, torch.ones_like(top))[ok]
            got[name + "_scale"] = sc
        else:
            c = s[name + "_cache"].double()
            c[page, :, at] = x[ok]
            got[name] = c
    return got


def _exact_attend(case, s):
    hq, hk, d, p = (case[x] for x in ("q_heads", "kv_heads", "dim", "page"))
    out = torch.zeros(case["requests"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["requests"], hq), -math.inf, dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n <= lo:
            continue
        t = torch.arange(lo, n, device="cuda")
        page, at = s["table"][r].long()[t // p], t % p
        for h in range(hk):
            k, v = s["k_cache"][page, h, at], s["v_cache"][page, h, at]
            if case["kv"] == E4M3:
                k = k.view(torch.float8_e4m3fn).double() * s["k_scale"].double()[page, h, at][:, None]
                v = v.view(torch.float8_e4m3fn).double() * s["v_scale"].double()[page, h, at][:, None]
            mine = slice(h * (hq // hk), (h + 1) * (hq // hk))
            w = (s["q"][r, mine].double() @ k.double().t()) * s["scale"]
            lse[r, mine] = torch.logsumexp(w, -1)
            out[r, mine] = torch.softmax(w, -1) @ v.double()
    return {"out": out, "lse": lse}


def _exact_lora(case, s):
    y = s["base"].double()
    ids = s["ids"]
    for a in sorted(set(ids.tolist()) - {-1}):
        rows, r = (ids == a).nonzero()[:, 0], int(s["ranks"][a])
        low = s["x"][rows].double() @ s["A"][a, :r].double().t()
        y[rows] += float(s["scales"][a]) * (low @ s["B"][a, :, :r].double().t())
    return {"y": y}
