"""The serving operators as they are used together (examples/decode_step.py): prompts and single
tokens of a few requests through page plan, quantised projection, adapters, cache store and
paged attention, against a history kept request by request in 64 bits."""
import os
import sys

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def turn(x, pos, dim):
    f = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    a = pos.double()[:, None] * f
    z = torch.complex(x[..., :dim // 2], x[..., dim // 2:]) * torch.polar(torch.ones_like(a), a)[:, None]
    return torch.cat([z.real, z.imag], -1)


@pytest.mark.parametrize("cache", [torch.float16, torch.uint8])
def test_a_few_steps_of_an_attention_block(cache):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from decode_step import AttentionBlock
    h = qgemv.create(0)
    R, dim, hq, hk = 5, 64, 8, 2
    b = AttentionBlock(h, R, hidden=512, q_heads=hq, kv_heads=hk, dim=dim, adapters=3, rank=8, pages=60, page=16, max_len=256, cache=cache)
    g = torch.Generator(device="cuda").manual_seed(1)
    history = [(torch.empty(0, hk, dim, device="cuda", dtype=torch.float64),) * 2 for _ in range(R)]
    for it, fresh in enumerate(([20, 0, 33, 1, 64], [1] * R, [1] * R, [0, 40, 0, 16, 1], [1] * R)):
        s = b.plan(torch.tensor(fresh, dtype=torch.int32, device="cuda"), sum(fresh))
        s.x.copy_(torch.randn(s.x.shape, generator=g, device="cuda").half())
        s.ids.copy_(torch.randint(-1, 3, s.ids.shape, generator=g, device="cuda"))
        before = b.lens.tolist()
        b.run(s)
        assert qgemv.check_error(h) == qgemv.OK
        assert b.lens.tolist() == [x + f for x, f in zip(before, fresh)]
        used = [p for row, n in zip(b.table.tolist(), b.lens.tolist()) for p in row[:-(-n // 16)]]
        assert len(set(used)) == len(used) and int(b.free_count) == 60 - len(used)
        # the projection with its adapters, from the same call without them
        plain = torch.empty_like(s.qkv)
        qgemv.run_gemm(h, b.fmt, s.x, s.capacity, b.w_qkv, b.n_qkv, b.hidden, plain)
        want = plain.double()
        for t, a in enumerate(s.ids.tolist()):
            if a >= 0:
                want[t] += b.b_qkv[a].double() @ (b.a_qkv[a].double() @ s.x[t].double())
        # inner sums of 512 exact products in fp32, then 8 of them: far below 1e-5 of the largest output
        assert (s.qkv.double() - want).abs().max() <= 1e-5 * want.abs().max()
        rows = s.qkv.double().view(-1, hq + 2 * hk, dim)
        at = 0
        for r, f in enumerate(fresh):
            pos = torch.arange(before[r], before[r] + f, device="cuda")
            new = rows[at:at + f]
            k, v = turn(new[:, hq:hq + hk], pos, dim), new[:, hq + hk:]
            history[r] = tuple(torch.cat([o, n]) for o, n in zip(history[r], (k, v)))
            if fresh == [1] * R:
                q = turn(new[:, :hq], pos, dim)[0].view(hk, hq // hk, dim)
                kk, vv = history[r]
                p = torch.softmax(torch.einsum("hgd,thd->hgt", q, kk) * b.scale, -1)
                ref = torch.einsum("hgt,thd->hgd", p, vv).reshape(hq, dim)
                # keys and values are rounded once (fp16 2^-11, e4m3 2^-4 of a value or less), queries to fp16: a score is
                # off by at most that of sum |q k|, a weight by twice as much, the output by that of sum p |v|
                u = 2.0 ** -11 if cache == torch.float16 else 2.0 ** -4
                score = (u + 2.0 ** -11) * (torch.einsum("hgd,thd->hgt", q.abs(), kk.abs()) * b.scale).amax(-1).reshape(hq, 1)
                pv = torch.einsum("hgt,thd->hgd", p, vv.abs()).reshape(hq, dim)
                tol = (torch.expm1(2 * score) + u) * (pv + vv.abs().amax()) + 2.0 ** -10 * ref.abs()
                assert ((s.out[r].double() - ref).abs() <= tol).all(), (it, r)
            at += f
    h.close()


def test_the_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, os.path.join(root, "examples", "decode_step.py"), "--requests", "7", "--steps", "3"],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "us per step" in out.stdout, out.stdout + out.stderr
