"""The attention operators together with the library's quantizers and GEMMs, as
examples/attention_block.py runs them."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_util import note
from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(mx):
    spec = importlib.util.spec_from_file_location("attention_block",
                                                  os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("config", [dict(hidden=512, q_heads=6, kv_heads=2, head_dim=64, pages=40, page_size=16,
                                         max_positions=512, max_tokens=512),
                                    dict(hidden=1024, q_heads=8, kv_heads=1, head_dim=128, pages=24, page_size=48,
                                         max_positions=512, max_tokens=600)])
def test_steps_give_what_one_prompt_gives(example, config):
    # The same tokens through the cache one by one and at once.  GEMMs of other row counts may round
    # a bf16 value the other way (2^-8 of it); what a stored code amplifies of that, 2^-2 of a key or
    # value in a few places, averages out over the keys: 2^-6 of the result's norm is far above both.
    note(f"attention block {config}")
    stepped, whole = example.run(lens=(70, 33), steps=5, **config)
    torch.cuda.synchronize()
    assert torch.isfinite(whole).all()
    off = (stepped.float() - whole.float()).norm() / whole.float().norm()
    assert float(off) < 2.0 ** -6


def test_block_against_the_float64_chain(mx, example):
    # From the QKV projection's bf16 output on: norm, rotation, cache and attention in float64, with
    # the cache as stored.
    block = example.AttentionBlock(hidden=256, q_heads=4, kv_heads=2, head_dim=64, pages=8, page_size=16,
                                   max_positions=64, max_tokens=64, batch=1)
    seqs = example.Sequences(block, 50)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((50, 256), generator=g, device="cuda").to(torch.bfloat16)
    y, pos = torch.empty_like(x), torch.arange(50, device="cuda")
    note("attention block against float64")
    qkv = torch.empty((50, 8 * 64), dtype=torch.bfloat16, device="cuda")
    xq, xs = (torch.empty((50, n), dtype=torch.uint8, device="cuda") for n in (256, 8))
    mx.mx_act_quant(x, xq, xs)
    mx.mx_gemm_fp8_fp4(xq, xs, *block.wqkv, qkv)
    block.forward(x, y, pos.to(torch.int32), seqs.slots(torch.zeros_like(pos), pos), seqs.table,
                  torch.tensor([50], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    h = qkv.view(50, 8, 64).cpu().double().numpy()
    cos, sin, p = block.cos.cpu().numpy(), block.sin.cpu().numpy(), pos.cpu().numpy()
    one = np.ones(64)
    q, _ = A.norm_rope(h[:, :4], one, p, cos, sin)
    k, _ = A.norm_rope(h[:, 4:6], one, p, cos, sin)
    c = [t.cpu().numpy() for t in (block.cache.k, block.cache.k_scale, block.cache.v, block.cache.v_scale)]
    table = seqs.table.cpu().numpy()
    # what is stored: keys within one E2M1 rounding (2^-2 of the value plus a quarter step, the step at
    # most 2^-1 of the block's largest / 3) of the exact ones, values as the quantizer gives them
    kc, vc = A.cache_rows(c[0], c[1], table[0], 50), A.cache_rows(c[2], c[3], table[0], 50)
    top = np.abs(k).reshape(50, 2, 2, 32).max(-1).repeat(32, -1).transpose(1, 0, 2)
    kt = k.transpose(1, 0, 2)
    assert (np.abs(kc - kt) <= 0.25 * np.abs(kt) + top / 6 + 2.0 ** -6).all()
    _, _, want_v = A.quantize_fp4(h[:, 6:].astype(np.float32))
    assert np.array_equal(vc, want_v.transpose(1, 0, 2))
    out, _, mag, size = A.attention(q, *c, table, [50], [0, 50], 64 ** -0.5)
    got = block.out[:50].cpu().double().numpy()
    # queries were rounded to bf16 once: a score moves by at most 2^-8 of its terms' magnitudes, and
    # the weights by e^(2 d) of that
    d = (2.0 ** -8 * size)[..., None]
    assert (np.abs(got - out) <= 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + np.expm1(2 * d)) * mag * 2 + 2.0 ** -20).all()
