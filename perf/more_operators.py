"""What a decode step with 8-bit projections adds to the serving operators, as measured cases.

Four operators, each in its plain form (elementary torch operations in 32 bits, sampling in 64) and as a
call of the library:

  norm    root-mean-square norm with the residual's addition, into 16 or 32 bits or into e4m3 with a scale per 128
  quant   rows, or the gated product silu(gate) * up, into e4m3 with a scale per 128
  fp8     a projection of such rows: e4m3 weights with a scale for each block of 128 x 128
  sample  the next token of each request: temperature, top-k, top-p and min-p from one given random number a row

Widths are those of the projections that the library is benchmarked on (hidden 4096, QKV 6144 wide,
MLP 12288 and 14336 wide, gate and up 28672) and generic vocabularies.
"""
import math
import random

import torch

own = False

F32, F16, BF16 = "f32", "f16", "bf16"
_TORCH = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
_BYTES = {F32: 4, F16: 2, BF16: 2}
_F8 = torch.float8_e4m3fn
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
        # one token before its QKV projection in 8 bits: the smallest call, all latency
        dict(name="norm 1 x 4096 to e4m3", op="norm", rows=1, N=4096, x=BF16, res=BF16, w=BF16, y="", codes=True),
        # 64 decode requests: fp32 rows of the output projection into the fp16 rows of the next one
        dict(name="norm 64 x 4096 f32 to f16", op="norm", rows=64, N=4096, x=F32, res=F16, w=F32, y=F16, codes=False),
        # a prompt's tokens, the residual stream kept in bf16, the next projection in 8 bits
        dict(name="norm 8191 x 4096 to e4m3", op="norm", rows=8191, N=4096, x=BF16, res=BF16, w=BF16, y="", codes=True),
        # 64 decode requests between gate and up and the MLP's second projection
        dict(name="quant 64 x 14336 gated", op="quant", rows=64, N=14336, x=BF16, gated=True),
        # a prompt's attention output before the output projection
        dict(name="quant 8191 x 4096", op="quant", rows=8191, N=4096, x=BF16, gated=False),
        # a single request's attention output projection: latency
        dict(name="fp8 1 x 4096 x 4096", op="fp8", M=1, N=4096, K=4096, y=F32),
        # gate and up of 64 decode requests
        dict(name="fp8 64 x 28672 x 4096", op="fp8", M=64, N=28672, K=4096, y=BF16),
        # an odd batch through the MLP's second projection, K long and N short
        dict(name="fp8 37 x 4096 x 14336", op="fp8", M=37, N=4096, K=14336, y=F32),
        # gate and up of a prompt: the largest, all matrix instructions
        dict(name="fp8 4096 x 28672 x 4096", op="fp8", M=4096, N=28672, K=4096, y=BF16),
        # one request's next token: latency
        dict(name="sample 1 x 32000", op="sample", rows=1, V=32000, x=F32, k_hi=50, p_lo=0.8, min_p=0.0, greedy=0.0, masked=0.0),
        # 64 requests with settings of their own, some of them greedy, some without a limit
        dict(name="sample 64 x 128000 mixed", op="sample", rows=64, V=128000, x=F32, k_hi=1000, p_lo=0.7, min_p=0.02, greedy=0.1,
             masked=0.0),
        # a large batch in bf16 (many equal logits) with part of the vocabulary masked, nucleus only
        dict(name="sample 509 x 50001 top-p", op="sample", rows=509, V=50001, x=BF16, k_hi=0, p_lo=0.85, min_p=0.0, greedy=0.0,
             masked=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "fp8", "fp8", "sample", "sample"])
    if op == "norm":
        codes = rng.choice([True, True, False])
        return dict(op=op, rows=_log(rng, 1, 8191), N=rng.choice([64, 1040, 2048, 4096, 4112, 8192, 14336]), x=rng.choice([F32, F16, BF16]),
                    res=rng.choice(["", F32, F16, BF16, BF16]), w=rng.choice([F32, F16, BF16]),
                    y=rng.choice(["", F16, BF16]) if codes else rng.choice([F32, F16, BF16]), codes=codes)
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 8191), N=rng.choice([64, 1040, 4096, 6144, 12288, 14336]), x=rng.choice([F32, F16, BF16]),
                    gated=rng.choice([True, False]))
    if op == "fp8":
        N, K = rng.choice([(6144, 4096), (4096, 4096), (4096, 12288), (4096, 14336), (28672, 4096), (1000, 1040), (77, 2064), (1024, 1024)])
        return dict(op=op, M=_log(rng, 1, 4096), N=N, K=K, y=rng.choice([F32, F16, BF16]))
    rows = _log(rng, 1, 512)
    return dict(op=op, rows=rows, V=_log(rng, 500, min(200000, 26000000 // rows)), x=rng.choice([F32, F16, BF16]), k_hi=rng.choice([0, 0, 64, 5000]),
                p_lo=rng.choice([1.0, 0.5, 0.9]), min_p=rng.choice([0.0, 0.0, 0.05]), greedy=rng.choice([0.0, 0.2]),
                masked=rng.choice([0.0, 0.0, 0.9]))


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "norm":
        m, n = case["rows"], case["N"]
        per = _BYTES[case["x"]] + (2 * _BYTES[case["res"]] if case["res"] else 0) + (_BYTES[case["y"]] if case["y"] else 0)
        per += 1 if case["codes"] else 0
        return {"bytes": m * n * per + n * _BYTES[case["w"]] + (4 * m * _cdiv(n, 128) if case["codes"] else 0), "flops": 5 * m * n}
    if case["op"] == "quant":
        m, n = case["rows"], case["N"]
        return {"bytes": m * n * ((2 if case["gated"] else 1) * _BYTES[case["x"]] + 1) + 4 * m * _cdiv(n, 128), "flops": (5 if case["gated"] else 2) * m * n}
    if case["op"] == "fp8":
        m, n, k = case["M"], case["N"], case["K"]
        blocks = _cdiv(k, 128)
        return {"bytes": n * k + m * k + m * n * _BYTES[case["y"]] + 4 * blocks * (m + _cdiv(n, 128)), "flops": 2 * m * n * k}
    m, v = case["rows"], case["V"]
    return {"bytes": m * v * _BYTES[case["x"]] + 28 * m, "flops": 4 * m * v}


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    {"norm": _prepare_norm, "quant": _prepare_quant, "fp8": _prepare_fp8, "sample": _prepare_sample}[case["op"]](case, g, s)
    return s


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _activations(g, m, n):
    """Rows as a layer gives them: each of its own size, a few columns far larger than the others."""
    size = torch.exp(_randn(g, m, 1) * 0.3)
    far = torch.where(_rand(g, 1, n) < 0.004, 12.0, 1.0)
    return _randn(g, m, n) * size * far


def _prepare_norm(case, g, s):
    m, n = case["rows"], case["N"]
    s["x"] = _activations(g, m, n).to(_TORCH[case["x"]])
    s["res"] = (_activations(g, m, n) * 2.0).to(_TORCH[case["res"]]) if case["res"] else None
    s["w"] = (1.0 + 0.2 * _randn(g, n)).to(_TORCH[case["w"]])
    s["eps"] = 1e-5
    empty = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    s["out"] = {"res": empty((m, n), _TORCH[case["res"]]) if case["res"] else None,
                "y": empty((m, n), _TORCH[case["y"]]) if case["y"] else None,
                "codes": empty((m, n), _F8) if case["codes"] else None,
                "scale": empty((m, _cdiv(n, 128)), torch.float32) if case["codes"] else None}
    if own:
        from quantized_weight_dequant_gb300 import qgemv
        o = s["out"]
        s["desc"] = qgemv.norm_desc(s["x"], s["w"], s["eps"], y=o["y"], codes=o["codes"], scale=o["scale"], res=s["res"], res_out=o["res"])


def _prepare_quant(case, g, s):
    m, n = case["rows"], case["N"]
    s["x"] = _activations(g, m, 2 * n if case["gated"] else n).to(_TORCH[case["x"]])  # gate and up: two halves of one projection's rows
    s["out"] = {"codes": torch.empty((m, n), dtype=_F8, device="cuda"),
                "scale": torch.empty((m, _cdiv(n, 128)), dtype=torch.float32, device="cuda")}
    if own:
        from quantized_weight_dequant_gb300 import qgemv
        x = s["x"]
        s["desc"] = qgemv.quant_desc(x[:, :n], s["out"]["codes"], s["out"]["scale"], up=x[:, n:] if case["gated"] else None)


def _by_128(x):
    """[rows, columns] as [rows, blocks, 128], zeros behind the last column."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 128)).reshape(x.shape[0], -1, 128)


def _to_codes(y):
    """e4m3 codes and a scale for each 128 columns of a row."""
    b = _by_128(y)
    top = b.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, 1.0)
    return (b / scale[..., None]).reshape(y.shape[0], -1)[:, :y.shape[1]].to(_F8).contiguous(), scale


def _prepare_fp8(case, g, s):
    m, n, k = case["M"], case["N"], case["K"]
    s["x"], s["xs"] = _to_codes(_activations(g, m, k))
    # weights in blocks of 128 x 128, each of its own size
    nb, kb = _cdiv(n, 128), _cdiv(k, 128)
    w = _randn(g, n, k)
    s["W"] = (w * (448.0 / 5.5)).clamp(-448, 448).to(_F8)
    s["ws"] = torch.exp(_randn(g, nb, kb) * 0.4) * (k ** -0.5 * 5.5 / 448.0)
    s["y"] = torch.empty(m, n, dtype=_TORCH[case["y"]], device="cuda")
    if own:
        from quantized_weight_dequant_gb300 import qgemv
        s["desc"] = qgemv.scaled_desc(s["x"], s["xs"], s["W"], s["ws"], s["y"])


def _prepare_sample(case, g, s):
    m, v = case["rows"], case["V"]
    # a broad bulk and some tokens that the model thinks likely
    x = _randn(g, m, v) * 2.2 + torch.where(_rand(g, m, v) < 0.0005, 1.0, 0.0) * (4.0 + 5.0 * _rand(g, m, v))
    if case["masked"]:  # tokens that a grammar forbids
        x = torch.where(_rand(g, m, v) < case["masked"], -math.inf, x)
    s["x"] = x.to(_TORCH[case["x"]])
    s["temperature"] = 0.6 + 0.6 * _rand(g, m)
    if case["greedy"]:
        s["temperature"] = torch.where(_rand(g, m) < case["greedy"], 0.0, s["temperature"])
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if case["k_hi"]:  # one row in four has no limit
        k = torch.exp(_rand(g, m) * math.log(case["k_hi"])).round().to(torch.int32)
        s["top_k"] = k if m == 1 else torch.where(_rand(g, m) < 0.25, 0, k)
    if case["p_lo"] < 1:
        s["top_p"] = (case["p_lo"] + (1.2 - case["p_lo"]) * _rand(g, m)).clamp(max=1.0)
    if case["min_p"]:
        s["min_p"] = torch.where(_rand(g, m) < 0.5, case["min_p"], 0.0)
    s["u"] = _rand(g, m)
    s["out"] = {"tokens": torch.empty(m, dtype=torch.int32, device="cuda"), "logprobs": torch.empty(m, dtype=torch.float32, device="cuda")}
    if own:
        from quantized_weight_dequant_gb300 import qgemv
        s["desc"] = qgemv.sample_desc(s["x"], s["u"], s["out"]["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                                      top_p=s["top_p"], min_p=s["min_p"], logprobs=s["out"]["logprobs"])


# ------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "quant": _plain_quant, "fp8": _plain_fp8, "sample": _plain_sample}[op](s)
    from quantized_weight_dequant_gb300 import qgemv
    if op == "norm":
        qgemv.run_norm(_handle(), s["desc"])
        return s["out"]
    if op == "quant":
        qgemv.quant_rows(_handle(), s["desc"])
        return s["out"]
    if op == "fp8":
        qgemv.run_scaled(_handle(), s["desc"])
        return {"y": s["y"]}
    qgemv.sample(_handle(), s["desc"])
    return s["out"]


def _plain_norm(s):
    case = s["case"]
    t = s["x"].float()
    got = {"res": None, "y": None, "codes": None, "scale": None}
    if case["res"]:
        t = t + s["res"].float()
        got["res"] = t.to(s["res"].dtype)
    y = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + s["eps"]) * s["w"].float()
    if case["y"]:
        got["y"] = y.to(_TORCH[case["y"]])
    if case["codes"]:
        got["codes"], got["scale"] = _to_codes(y)
    return got


def _plain_quant(s):
    n, x = s["case"]["N"], s["x"].float()
    if s["case"]["gated"]:
        x = x[:, :n] / (1.0 + torch.exp(-x[:, :n])) * x[:, n:]
    codes, scale = _to_codes(x)
    return {"codes": codes, "scale": scale}


def _plain_fp8(s):
    m, n, k = (s["case"][x] for x in ("M", "N", "K"))
    x = (_by_128(s["x"].float()) * s["xs"][..., None]).reshape(m, -1)[:, :k]
    w = (_by_128(s["W"].float()) * s["ws"].repeat_interleave(128, 0)[:n, :, None]).reshape(n, -1)[:, :k]
    return {"y": torch.matmul(x, w.t()).to(s["y"].dtype)}


def _plain_sample(s):
    """In 64 bits: a draw is decided by whether a running sum lies on this or that side of a border."""
    x = s["x"].double()
    top = x.amax(-1, keepdim=True)
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    w = torch.exp((x - top) / torch.where(greedy, 1.0, t))
    by, order = torch.sort(w, dim=-1, descending=True, stable=True)
    # the order is the logits': equal logits have equal weights, lower indexes first
    rank = torch.arange(x.shape[1], device="cuda")[None]
    keep = torch.ones_like(by, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = (rank < k) | (k <= 0)
    mass = torch.where(keep, by, 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cumsum(mass, -1) - mass
        keep = keep & ((before < p * mass.sum(-1, keepdim=True)) | (p >= 1) | (rank == 0))
    if s["min_p"] is not None:
        keep = keep & (by >= s["min_p"].double()[:, None])
    keep = keep & torch.where(greedy, rank == 0, True)
    kept = torch.zeros_like(w).scatter(1, order, torch.where(keep, by, 0.0))
    run = torch.cumsum(kept, -1)
    total = run[:, -1:]
    token = (run <= s["u"].double()[:, None] * total).sum(-1)
    return {"tokens": token.int(), "logprobs": torch.log(kept.gather(1, token[:, None]) / total)[:, 0].float()}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "quant": _exact_quant, "fp8": _exact_fp8, "sample": _exact_sample}[case["op"]](case, s)


def _exact_scales(y):
    """The largest of each 128 columns over 448; the codes follow from its rounding and have no value of their own."""
    return torch.stack([c.abs().amax(-1) / 448.0 for c in y.split(128, dim=1)], 1)


def _exact_norm(case, s):
    t = s["x"].double()
    if case["res"]:
        t = t + s["res"].double()
    n = t.shape[1]
    y = t / torch.sqrt((t * t).sum(-1, keepdim=True) / n + s["eps"]) * s["w"].double()
    return {"res": t if case["res"] else None, "y": y if case["y"] else None, "codes": None, "scale": _exact_scales(y) if case["codes"] else None}


def _exact_quant(case, s):
    x = s["x"].double()
    if case["gated"]:
        gate, up = x.chunk(2, dim=1)
        x = gate * torch.sigmoid(gate) * up
    return {"codes": None, "scale": _exact_scales(x)}


def _exact_fp8(case, s):
    m, n, k = case["M"], case["N"], case["K"]
    col = torch.arange(k, device="cuda") // 128
    x = s["x"].double() * s["xs"].double()[:, col]
    w = s["W"].double()
    for r in range(0, n, 128):
        w[r:r + 128] *= s["ws"].double()[r // 128, col]
    return {"y": x @ w.t()}


def _exact_sample(case, s):
    """Row by row, candidate by candidate."""
    tokens, logprobs = [], []
    for r in range(case["rows"]):
        x = s["x"][r].double()
        t = float(s["temperature"][r])
        k = int(s["top_k"][r]) if s["top_k"] is not None else 0
        p = float(s["top_p"][r]) if s["top_p"] is not None else 1.0
        low = float(s["min_p"][r]) if s["min_p"] is not None else 0.0
        by, order = torch.sort(x, descending=True, stable=True)
        if t <= 0:
            tokens.append(int(order[0]))
            logprobs.append(0.0)
            continue
        n = min(k, x.numel()) if k > 0 else x.numel()
        n = max(1, min(n, int((by > -math.inf).sum())))
        w = torch.exp((by[:n] - by[0]) / t)
        if p < 1:
            n = max(1, int((torch.cumsum(w, 0) - w < p * w.sum()).sum()))
            w = w[:n]
        if low > 0:
            n = max(1, int((w >= low).sum()))
            w = w[:n]
        index, back = torch.sort(order[:n])
        run = torch.cumsum(w[back], 0)
        at = min(n - 1, int(torch.searchsorted(run, float(s["u"][r]) * run[-1:], right=True)))
        tokens.append(int(index[at]))
        logprobs.append(math.log(float(w[back][at] / run[-1])))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32, device="cuda"),
            "logprobs": torch.tensor(logprobs, dtype=torch.float64, device="cuda")}
