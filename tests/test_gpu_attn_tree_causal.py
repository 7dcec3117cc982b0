"""mx_attn_tree_fp4 of chains beside mx_attn_fp4's causal mask: the same attention, but not always the same order of
sums (trees are cut into other runs, and two wavefronts may share a block's rows), so not the same bits in general."""
import numpy as np
import pytest
import torch

from attention_util import Paged, attention_close, bf16, f64, oracle
from draft_util import forest, ints
from gpu_util import note
from oracle import draft_oracle as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,group,dim,window", [(5, 4, 128, 0), (40, 4, 128, 0), (33, 4, 64, 0), (3, 5, 256, 0), (9, 3, 256, 0),
                                                (16, 4, 128, 0), (130, 1, 64, 0), (1, 8, 128, 70), (1, 70, 128, 70)])
def test_chains_and_causal_masks_lie_as_close_as_their_bounds_say(mx, n, group, dim, window):
    # either is within attention_close's bound of the exact value, so they are within twice that of each other; a
    # window is the same where it takes nothing of the tree: one node's
    rng = np.random.default_rng(n + dim)
    lens = [n, 100 + n, 1200]
    parents, starts = forest(rng, [n] * 3, "chain")
    mask, pos = D.tree_mask(parents, starts, -(-n // 32), lens)
    paged = Paged(rng, lens, 2, dim, 16)
    cache, table, seq = mx.MxKvCacheFp4(*paged.tensors()), ints(paged.table), ints(lens)
    q = bf16(rng.standard_normal((3 * n, 2 * group, dim))).cuda()
    ws = torch.zeros(mx.mx_attn_fp4_workspace_size(3, n, 2 * group, 2, dim), dtype=torch.uint8, device="cuda")
    tree, causal = torch.full_like(q, float("nan")), torch.full_like(q, float("nan"))
    sums = [torch.full(q.shape[:2], float("nan"), device="cuda") for _ in range(2)]
    note(f"attn tree beside causal n={n} group={group} D={dim}")
    mx.mx_attn_tree_fp4(cache, q, ints(mask), table, seq, tree, ws, window=window, positions=ints(pos), lse=sums[0])
    mx.mx_attn_fp4(cache, q, table, seq, causal, ws, window=window, lse=sums[1])
    torch.cuda.synchronize()
    ref = oracle(paged, q, starts, dim ** -0.5, window=window)
    attention_close(tree, sums[0], ref, "tree")
    attention_close(causal, sums[1], ref, "causal")
    o, _, mag, top = ref
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 4 * 2.0 ** -20 * top[..., None]) * mag + 2.0 ** -126 * (1 + 1e4 * 192)
    assert (np.abs(f64(tree) - f64(causal)) <= 2 * tol).all()
