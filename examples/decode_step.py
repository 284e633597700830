"""Decode step of one layer for many requests, with quantised projections.

One layer's attention as a serving loop runs it: pages of the key-value cache are planned on
the GPU, the QKV projection (quantised weights) is joined by each request's low-rank adapter,
its rows are rotated and stored in the cache, every new token attends to its request's pages,
and the output projection closes the block.  The MLP follows with projections in 8 bits: the norm
takes up the residual and hands over codes, the gated product is quantised as it is formed; and from
the normed last hidden state come the logits, of which each request's next token is drawn by its own
temperature, top-k and top-p.  Prompts and single tokens go through the same calls of the attention;
a step of single tokens is captured in a CUDA graph and replayed.

    python examples/decode_step.py [--requests 64] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_weight_dequant_gb300 import qgemv, synth  # noqa: E402


class AttentionBlock:
    """Quantised QKV and output projections, their adapters, and a paged cache for `requests` requests."""

    def __init__(self, handle, requests, hidden=4096, q_heads=32, kv_heads=8, dim=128, fmt=synth.Q4_K, adapters=8,
                 rank=16, pages=4096, page=16, max_len=4096, cache=torch.float16, seed=0):
        self.h, self.fmt, self.hidden, self.page, self.requests = handle, fmt, hidden, page, requests
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n_qkv, self.n_q = (q_heads + 2 * kv_heads) * dim, q_heads * dim
        self.w_qkv = torch.from_numpy(synth.make_weights(fmt, self.n_qkv, hidden, seed=seed + 1)).cuda()
        self.w_out = torch.from_numpy(synth.make_weights(fmt, hidden, self.n_q, seed=seed + 2)).cuda()

        def pair(n, k):
            a = torch.randn(adapters, rank, k, generator=g, device="cuda") * k ** -0.5
            return a.half(), (torch.randn(adapters, n, rank, generator=g, device="cuda") * 0.05).half()

        self.a_qkv, self.b_qkv = pair(self.n_qkv, hidden)
        self.a_out, self.b_out = pair(hidden, self.n_q)
        shape = (pages, kv_heads, page, dim)
        scales = (None, None)
        if cache == torch.uint8:  # e4m3 codes with a scale per token and head
            scales = tuple(torch.zeros(shape[:3], device="cuda") for _ in range(2))
        self.k, self.v = (torch.zeros(shape, dtype=cache, device="cuda") for _ in range(2))
        self.cache = qgemv.kv_cache(self.k, self.v, *scales)
        angle = torch.arange(max_len, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        # the allocator's state: lengths and tables of the requests, a stack of free pages
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.table = torch.full((requests, -(-max_len // page)), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=g, device="cuda").int()
        self.free_count = torch.full((1,), pages, dtype=torch.int32, device="cuda")
        self.scale = dim ** -0.5

    def plan(self, fresh, capacity):
        """Buffers and descriptions of a step that brings fresh[r] new tokens to request r, `capacity` in all."""
        s = Step()
        i32 = dict(dtype=torch.int32, device="cuda")
        s.capacity, s.fresh = capacity, fresh
        s.new_lens, s.counts = torch.empty(self.requests, **i32), torch.empty(4, **i32)
        s.slots = torch.empty(capacity, dtype=torch.int64, device="cuda")
        s.positions, s.owners, s.offsets = torch.empty(capacity, **i32), torch.empty(capacity, **i32), torch.empty(self.requests + 1, **i32)
        s.x = torch.zeros(capacity, self.hidden, dtype=torch.float16, device="cuda")
        s.ids = torch.full((capacity,), -1, **i32)  # adapter of each token
        s.qkv = torch.empty(capacity, self.n_qkv, device="cuda")
        s.q = torch.empty(capacity, self.q_heads, self.dim, dtype=torch.float16, device="cuda")
        s.pages = qgemv.page_plan_desc(self.lens, fresh, self.table, self.free, self.free_count, self.page, s.new_lens, s.slots,
                                       s.counts, s.offsets, s.positions, s.owners)
        s.add_qkv = qgemv.lora_desc(s.x, self.a_qkv, self.b_qkv, s.ids, s.qkv, base=s.qkv)
        n_kv = self.kv_heads * self.dim
        s.store = qgemv.kv_store_desc(self.cache, s.qkv[:, self.n_q:self.n_q + n_kv], s.qkv[:, self.n_q + n_kv:], s.slots,
                                      s.positions, self.rope, q=s.qkv[:, :self.n_q], q_out=s.q)
        if capacity == self.requests:  # one token each: row r is request r
            s.out = torch.empty_like(s.q)
            s.y = torch.empty(capacity, self.hidden, device="cuda")
            s.attend = qgemv.attn_decode_desc(self.cache, s.q, self.table, s.new_lens, s.out, self.scale)
            s.add_out = qgemv.lora_desc(s.out.view(capacity, -1), self.a_out, self.b_out, s.ids, s.y, base=s.y)
        return s

    def run(self, s):
        """The step's kernels, all on the current stream; nothing is allocated and nothing waits."""
        h = self.h
        qgemv.page_plan(h, s.pages)
        qgemv.run_gemm(h, self.fmt, s.x, s.capacity, self.w_qkv, self.n_qkv, self.hidden, s.qkv)
        qgemv.run_lora(h, s.add_qkv)
        qgemv.kv_store(h, s.store)
        if s.capacity == self.requests:
            qgemv.attn_decode(h, s.attend)
            qgemv.run_gemm(h, self.fmt, s.out, s.capacity, self.w_out, self.hidden, self.n_q, s.y)
            qgemv.run_lora(h, s.add_out)
        # the requests' new state
        self.lens.copy_(s.new_lens)
        self.free_count.sub_(s.counts[2:3])


class Step:
    pass


def e4m3_blocks(w):
    """Codes of a weight matrix and its scales, one for 128 x 128."""
    n, k = w.shape
    padded = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128)).view(-(-n // 128), 128, -(-k // 128), 128)
    scale = (padded.abs().amax((1, 3)) / 448).clamp(min=2.0 ** -126)
    codes = (padded / scale[:, None, :, None]).view(-(-n // 128) * 128, -1)[:n, :k].contiguous()
    return codes.to(torch.float8_e4m3fn), scale.contiguous()


class TokenBlock:
    """Residual, norm and gated MLP with projections in 8 bits, then the last norm, the logits and the next tokens.  `attended`
    [rows][hidden] is what the attention adds to the residual `hidden`, which ends as the layer's output."""

    def __init__(self, handle, attended, inner=14336, vocab=32000, residual=torch.bfloat16, seed=0):
        self.h, (rows, hidden) = handle, attended.shape
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(n, k):
            return e4m3_blocks(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)

        def norm_weight():
            return (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).bfloat16()

        def codes_of(n):
            return torch.empty(rows, n, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, -(-n // 128), device="cuda")

        self.w_up, self.w_down, self.w_head = weights(2 * inner, hidden), weights(hidden, inner), weights(vocab, hidden)
        self.n_mlp, self.n_last = norm_weight(), norm_weight()
        self.hidden = torch.zeros(rows, hidden, dtype=residual, device="cuda")
        self.x, self.act, self.last = codes_of(hidden), codes_of(inner), codes_of(hidden)
        self.gate_up = torch.empty(rows, 2 * inner, dtype=torch.bfloat16, device="cuda")
        self.down = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
        self.u, self.temperature, self.top_p = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"), torch.ones(rows, device="cuda")
        self.top_k = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.tokens, self.logprobs = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
        self.calls = [
            (qgemv.run_norm, qgemv.norm_desc(attended, self.n_mlp, 1e-5, codes=self.x[0], scale=self.x[1], res=self.hidden, res_out=self.hidden)),
            (qgemv.run_scaled, qgemv.scaled_desc(*self.x, *self.w_up, self.gate_up)),
            (qgemv.quant_rows, qgemv.quant_desc(self.gate_up[:, :inner], *self.act, up=self.gate_up[:, inner:])),
            (qgemv.run_scaled, qgemv.scaled_desc(*self.act, *self.w_down, self.down)),
            (qgemv.run_norm, qgemv.norm_desc(self.down, self.n_last, 1e-5, codes=self.last[0], scale=self.last[1], res=self.hidden, res_out=self.hidden)),
            (qgemv.run_scaled, qgemv.scaled_desc(*self.last, *self.w_head, self.logits)),
            (qgemv.sample, qgemv.sample_desc(self.logits, self.u, self.tokens, temperature=self.temperature, top_k=self.top_k, top_p=self.top_p,
                                             logprobs=self.logprobs))]

    def run(self):
        for call, desc in self.calls:
            call(self.h, desc)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--prompt", type=int, default=200)
    args = ap.parse_args()
    handle = qgemv.create(torch.cuda.current_device())
    block = AttentionBlock(handle, args.requests, pages=args.requests * 40)
    g = torch.Generator(device="cuda").manual_seed(7)
    prompts = torch.randint(1, args.prompt + 1, (args.requests,), generator=g, device="cuda").int()
    first = block.plan(prompts, int(prompts.sum()))
    first.x.copy_(torch.randn(first.x.shape, generator=g, device="cuda").half())
    block.run(first)  # the prompts' keys and values (their attention belongs to the prompt's own kernel)
    step = block.plan(torch.ones(args.requests, dtype=torch.int32, device="cuda"), args.requests)
    step.ids.copy_(torch.randint(-1, 8, (args.requests,), generator=g, device="cuda"))
    step.x.copy_(torch.randn(step.x.shape, generator=g, device="cuda").half())
    token = TokenBlock(handle, step.y)
    token.u.copy_(torch.rand(args.requests, generator=g, device="cuda"))
    token.top_p.fill_(0.9)
    block.run(step)
    token.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.run(step)
        token.run()
    begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
    torch.cuda.synchronize()
    begin.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert qgemv.check_error(handle) == qgemv.OK
    print(f"{args.requests} requests, lengths {int(block.lens.min())} to {int(block.lens.max())}, "
          f"{int(block.free_count)} pages free: {begin.elapsed_time(end) * 1e3 / args.steps:.1f} us per step of one layer and the next tokens")
    handle.close()


if __name__ == "__main__":
    main()
