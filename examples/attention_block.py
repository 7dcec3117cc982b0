"""The attention block of a decoder layer, served from a paged MXFP4 key/value cache.

Everything a layer does around its attention, on one stream and with no allocation after set-up:

    x -> act_quant -> QKV GEMM (MXFP4 weights) -> norm + rotation of queries and keys
      -> append to the cache -> attention over the cache -> act_quant -> output GEMM + residual

A prompt goes through in one call, then one token of every sequence at a time; the weights are
random.  Run from the repository's root on a GPU:

    python examples/attention_block.py
"""
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_act_amd as mx  # noqa: E402


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


def _bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda")


class AttentionBlock:
    def __init__(self, hidden=2048, q_heads=16, kv_heads=4, head_dim=128, pages=256, page_size=64,
                 max_positions=8192, max_tokens=4096, batch=2, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.hq, self.hk, self.D, self.hidden = q_heads, kv_heads, head_dim, hidden
        self.page_size, self.batch = page_size, batch

        def weight(n, k):                                   # bf16 -> MXFP4 [n, k / 2] + E8M0 [n, k / 32]
            w = torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k)
            q, s = _u8(n, k // 2), _u8(n, k // 32)
            mx.mx_act_quant_fp4(w.to(torch.bfloat16), q, s)
            return q, s

        self.wqkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.wo = weight(hidden, q_heads * head_dim)
        self.q_norm = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        self.k_norm = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        angle = torch.arange(max_positions, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        shape = (pages, kv_heads, page_size)
        self.cache = mx.MxKvCacheFp4(*(_u8(*shape, head_dim // n) for n in (2, 32, 2, 32)))
        # buffers for up to max_tokens tokens a call
        width = (q_heads + 2 * kv_heads) * head_dim
        self.xq, self.xs = _u8(max_tokens, hidden), _u8(max_tokens, hidden // 32)
        self.qkv, self.out = _bf16(max_tokens, width), _bf16(max_tokens, q_heads, head_dim)
        self.oq = _u8(max_tokens, q_heads * head_dim)
        self.os = _u8(max_tokens, q_heads * head_dim // 32)
        need = mx.mx_attn_fp4_workspace_size(batch, max_tokens, q_heads, kv_heads, head_dim)
        self.workspace = _u8(need)                          # zero before its first use

    def forward(self, x, y, positions, slots, table, lens, q_starts=None, max_q=None):
        """x, y: bf16 [tokens, hidden] (the block's input and output); positions int32 [tokens]; slots
        int64 [tokens] (where each token's key and value go); table int32 [batch, width] and lens int32
        [batch] (after this call's tokens); q_starts int32 [batch + 1] with max_q, or None for max_q
        tokens of each sequence."""
        T, hq, hk, D = x.shape[0], self.hq, self.hk, self.D
        qkv = self.qkv[:T]
        mx.mx_act_quant(x, self.xq[:T], self.xs[:T])
        mx.mx_gemm_fp8_fp4(self.xq[:T], self.xs[:T], *self.wqkv, qkv)
        heads = qkv.view(T, hq + 2 * hk, D)
        q, k, v = heads[:, :hq], heads[:, hq:hq + hk], heads[:, hq + hk:]
        mx.mx_qk_norm_rope(q, k, positions, self.cos, self.sin, q, k, self.q_norm, self.k_norm)
        mx.mx_kv_append_fp4(self.cache, k, v, slots)
        out = self.out[:T]
        mx.mx_attn_fp4(self.cache, q, table, lens, out, self.workspace, q_starts=q_starts, max_q=max_q)
        mx.mx_act_quant(out.view(T, hq * D), self.oq[:T], self.os[:T])
        mx.mx_gemm_fp8_fp4_bias_residual(self.oq[:T], self.os[:T], *self.wo, x, y)


class Sequences:
    """Page tables of a batch of sequences, pages handed out in turn."""

    def __init__(self, block, max_len):
        self.page_size, self.width = block.page_size, -(-max_len // block.page_size)
        order = torch.randperm(block.batch * self.width).view(block.batch, self.width)
        self.table = order.to(torch.int32).cuda()

    def slots(self, seq, positions):
        """Cache slots of tokens of sequences `seq` at `positions` (both int64, on the GPU)."""
        return self.table[seq, positions // self.page_size].long() * self.page_size + \
            positions % self.page_size


def run(lens=(300, 211), steps=8, seed=0, **config):
    """A prompt of each sequence in one call, then `steps` tokens of every sequence, one a call; and the
    same tokens all as one prompt.  Returns the two [tokens, hidden] results of the steps' tokens."""
    block = AttentionBlock(batch=len(lens), seed=seed, **config)
    B, total = len(lens), [n + steps for n in lens]
    seqs = Sequences(block, max(total))
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = [torch.randn((n, block.hidden), generator=g, device="cuda").to(torch.bfloat16) for n in total]

    def prompt(news):
        seq = torch.cat([torch.full((n,), b, device="cuda") for b, n in enumerate(news)])
        pos = torch.cat([torch.arange(n, device="cuda") for n in news])
        starts = torch.tensor([0, *torch.tensor(news).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        xs = torch.cat([t[:n] for t, n in zip(x, news)])
        y = torch.empty_like(xs)
        block.forward(xs, y, pos.to(torch.int32), seqs.slots(seq, pos), seqs.table,
                      torch.tensor(news, dtype=torch.int32, device="cuda"), starts, max(news))
        return y, starts

    prompt(list(lens))
    seq = torch.arange(B, device="cuda")
    stepped = []
    for i in range(steps):
        pos = torch.tensor([n + i for n in lens], device="cuda")
        xs = torch.stack([t[n + i] for t, n in zip(x, lens)])
        y = torch.empty_like(xs)
        block.forward(xs, y, pos.to(torch.int32), seqs.slots(seq, pos), seqs.table,
                      (pos + 1).to(torch.int32))
        stepped.append(y)
    whole, starts = prompt(total)
    rows = [int(starts[b + 1]) - steps + i for i in range(steps) for b in range(B)]
    return torch.cat(stepped), whole[rows]


def main():
    stepped, whole = run()
    off = (stepped.float() - whole.float()).norm() / whole.float().norm()
    print(f"{len(stepped)} tokens, step by step against one prompt: relative difference {off:.2e}")
    block = AttentionBlock(batch=16, pages=16 * 64)
    seqs = Sequences(block, 4096)
    pos = torch.full((16,), 4000, device="cuda")
    x = torch.randn((16, block.hidden), device="cuda").to(torch.bfloat16)
    y, slots = torch.empty_like(x), seqs.slots(torch.arange(16, device="cuda"), pos)
    args = (x, y, pos.to(torch.int32), slots, seqs.table, (pos + 1).to(torch.int32))
    block.forward(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(*args)
    graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(100):
        graph.replay()
    torch.cuda.synchronize()
    print(f"16 sequences of 4001 tokens, one token each: {(time.perf_counter() - t) * 1e4:.1f} us a step (graph)")


if __name__ == "__main__":
    main()
