"""mx_attn_tree_fp4 against the float64 oracle, within the bounds that attention_close derives: trees of
every size around the mask's words and the tiles, few and many rows, all head sizes, windows, masks that
leave rows empty or are no trees, sequences shorter than their trees, ragged batches, strides, junk beyond
the lengths, streams, graphs, refusals."""
import numpy as np
import pytest
import torch

from attention_util import Paged, attention_close, bf16, f64
from draft_util import forest, ints
from gpu_util import note
from oracle import draft_oracle as D

pytestmark = pytest.mark.gpu


def run(mx, paged, q, mask, starts, max_q, ws=None, positions=None, out=None, ragged=True, **how):
    cache = mx.MxKvCacheFp4(*paged.tensors())
    B, (N, H) = len(paged.lens), q.shape[:2]
    if ws is None:
        n = mx.mx_attn_fp4_workspace_size(B, max_q, H, paged.heads, paged.D)
        ws = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((N, H), float("nan"), device="cuda")
    mask = mask if isinstance(mask, torch.Tensor) else ints(mask)
    mx.mx_attn_tree_fp4(cache, q, mask, ints(paged.table), ints(paged.lens), out, ws,
                        q_starts=ints(starts) if ragged else None, max_q=max_q,
                        positions=None if positions is None else ints(positions), lse=lse, **how)
    torch.cuda.synchronize()
    return out, lse


def compare(mx, rng, lens, sizes, hk, group, dim, page, kind="tree", window=0, mask=None, positions=None,
            max_q=None, what="", **how):
    parents, starts = forest(rng, sizes, kind)
    max_q = max_q or max(sizes)
    words = -(-max_q // 32)
    made, pos = D.tree_mask(parents, starts, words, lens)
    mask = made if mask is None else mask
    positions = pos if positions is None else positions
    paged = Paged(rng, lens, hk, dim, page)
    q = bf16(rng.standard_normal((starts[-1], hk * group, dim))).cuda()
    note(f"attn tree D={dim} sizes={sizes[:6]} group={group} hk={hk} page={page} window={window} {what}")
    out, lse = run(mx, paged, q, mask, starts, max_q, window=window,
                   positions=positions if window else None, **how)
    ref = D.attention(f64(q), paged.k, paged.ks, paged.v, paged.vs, paged.table, lens, starts, dim ** -0.5,
                      mask, window, positions)
    attention_close(out, lse, ref, what)
    return out, lse, ref


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,group", [(1, 1), (2, 8), (7, 2), (16, 1), (16, 4), (31, 1), (32, 2), (33, 1)])
def test_few_rows(mx, dim, n, group):
    rng = np.random.default_rng(100 * n + dim + group)
    lens = [n, n + 1, n + 31, n + 32, n + 90, 128 + n // 2, 300]
    compare(mx, rng, lens, [n] * len(lens), 2, group, dim, 16, ragged=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,group", [(26, 4), (33, 8), (64, 2), (65, 3), (129, 1), (40, 16)])
def test_many_rows(mx, dim, n, group):
    rng = np.random.default_rng(100 * n + dim + group)
    lens = [n, n + 40, n + 64, 260 + n]
    compare(mx, rng, lens, [n] * len(lens), 1, group, dim, 32, ragged=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_hundreds_of_nodes(mx, dim):
    rng = np.random.default_rng(dim + 7)
    compare(mx, rng, [650, 620, 700], [610, 20, 333], 1, 1, dim, 16)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", ["chain", "star"])
def test_other_shapes_of_trees(mx, dim, kind):
    rng = np.random.default_rng(dim)
    compare(mx, rng, [200, 70, 64], [12, 1, 20], 2, 2, dim, 48, kind)
    compare(mx, rng, [200, 90, 64], [70, 1, 50], 1, 3, dim, 16, kind)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 20, 64, 150, 1000, 2 ** 31 - 1])
def test_windows(mx, dim, window):
    rng = np.random.default_rng(dim + window % 1000)
    compare(mx, rng, [5, 40, 129, 300, 260], [5, 9, 3, 8, 0], 2, 3, dim, 16, window=window)
    compare(mx, rng, [70, 71, 390], [70, 33, 70], 2, 2, dim, 16, window=window)


@pytest.mark.parametrize("sizes,group", [([6, 3], 4), ([50, 70], 3)])
def test_positions_outside_the_tree_are_clamped(mx, sizes, group):
    rng = np.random.default_rng(4)
    N = sum(sizes)
    wild = rng.integers(-2 ** 31, 2 ** 31, N).astype(np.int32)
    wild[:3] = [2 ** 31 - 1, -2 ** 31, 0]
    compare(mx, rng, [300, 170], sizes, 2, group, 128, 16, window=40, positions=wild)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,group", [(9, 2), (70, 3)])
def test_any_mask_and_rows_that_see_nothing(mx, dim, n, group):
    # views that no tree has, bits past the nodes set, no text before: some rows see no key at all
    rng = np.random.default_rng(dim + n)
    words = -(-n // 32) + 1
    mask = rng.integers(-2 ** 31, 2 ** 31, (3 * n, words)).astype(np.int32)
    mask[::4] = 0
    _, lse, ref = compare(mx, rng, [n, n + 3, n + 100], [n] * 3, 2, group, dim, 16, mask=mask)
    assert np.isneginf(f64(lse)[0]).all() and not np.isneginf(f64(lse)[-1]).any()


@pytest.mark.parametrize("n,group", [(9, 2), (70, 3)])
def test_sequences_shorter_than_their_trees(mx, n, group):
    # the first nodes are no cached tokens: nobody sees them
    rng = np.random.default_rng(n)
    compare(mx, rng, [0, 1, n - 1, n, 3], [n] * 5, 2, group, 128, 16)
    compare(mx, rng, [0, 1, n - 1, n, 3], [n] * 5, 2, group, 128, 16, window=5)


def test_ragged_batches_of_many_lengths(mx):
    rng = np.random.default_rng(5)
    sizes = [12, 0, 3, 9, 1, 12, 5, 0]
    compare(mx, rng, [3000, 0, 3, 130, 1100, 17, 5, 640], sizes, 2, 7, 128, 16)
    compare(mx, rng, [2000, 0, 3, 130, 1100, 17, 5, 640], sizes, 2, 2, 64, 64, max_q=40)


@pytest.mark.parametrize("dim,n,hk,group", [(64, 40, 33, 2), (128, 40, 33, 2), (256, 33, 33, 1)])
@pytest.mark.parametrize("window", [0, 900])
def test_batches_that_are_dealt_and_joined(mx, dim, n, hk, group, window):
    # nearly all keys are one sequence's: runs of its tiles go to all workgroups, and are joined
    rng = np.random.default_rng(dim + hk + window)
    lens, sizes = [2200, 700, 0, 130], [n, 3, 0, n // 2]
    out, lse, _ = compare(mx, rng, lens, sizes, hk, group, dim, 32, window=window)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,group", [(60, 2), (105, 2), (50, 6)])
def test_few_rows_beside_many(mx, dim, n, group):
    # blocks with all, half, one more than half, few and none of their rows, of short texts and of long ones that
    # are dealt to all workgroups: 120 rows are a block of 128, 210 one of 256, 300 one and a part of the next
    rng = np.random.default_rng(dim + n)
    half = (64 if n * group <= 128 else 128) // group
    sizes = [n, 1, 0, half, half + 1, 5, n, 3]
    lens = [2300, 2200, 30, 1500, 700, 64, 129, 40]
    compare(mx, rng, lens, sizes, 37, group, dim, 32, what="dealt")
    compare(mx, rng, [130, 1, 7, 200, 90, 64, 300, 40], sizes, 3, group, dim, 16, what="not dealt")
    compare(mx, rng, [3100, 900], [half, n], 1, group, dim, 64, what="split", window=800 if n == 60 else 0)


def test_one_long_sequence_is_split(mx):
    rng = np.random.default_rng(8)
    compare(mx, rng, [4001], [26], 1, 8, 128, 64)
    compare(mx, rng, [4001], [9], 1, 4, 128, 64)
    compare(mx, rng, [3001], [40], 1, 4, 256, 64)


def test_a_chain_gives_what_the_causal_mask_gives(mx):
    # the same kernels take the same tokens in the same order: the same bits
    rng = np.random.default_rng(9)
    for n, group, dim in ((5, 4, 128), (40, 4, 128), (33, 4, 64), (3, 5, 256)):
        lens = [n, 100, 257]
        parents, starts = forest(rng, [n] * 3, "chain")
        mask, _ = D.tree_mask(parents, starts, 2, lens)
        paged = Paged(rng, lens, 2, dim, 16)
        q = bf16(rng.standard_normal((3 * n, 2 * group, dim))).cuda()
        note(f"attn tree against causal n={n}")
        out, lse = run(mx, paged, q, mask, starts, n, ragged=False)
        ref = D.attention(f64(q), paged.k, paged.ks, paged.v, paged.vs, paged.table, lens, starts, dim ** -0.5, mask)
        attention_close(out, lse, ref)
        ws = torch.zeros(mx.mx_attn_fp4_workspace_size(3, n, 2 * group, 2, dim), dtype=torch.uint8, device="cuda")
        causal = torch.empty_like(out)
        mx.mx_attn_fp4(mx.MxKvCacheFp4(*paged.tensors()), q, ints(paged.table), ints(lens), causal, ws)
        attention_close(causal, None, ref)


@pytest.mark.parametrize("n,group", [(6, 4), (50, 4)])
def test_strides_and_one_mask_for_all(mx, n, group):
    rng = np.random.default_rng(n)
    lens, starts = [n + 60, n + 9], [0, n, 2 * n]
    paged = Paged(rng, lens, 2, 128, 16, gap=32 * 16)
    wide = bf16(rng.standard_normal((2 * n, 2 * group + 3, 128))).cuda()
    q = wide[:, 1:1 + 2 * group]
    words = -(-n // 32)
    rows = rng.integers(-2 ** 31, 2 ** 31, (2 * n, words)).astype(np.int32)
    buf = torch.full((2 * n, 2 * group + 1, 136), 42.0, dtype=torch.bfloat16, device="cuda")
    masks = ints(np.pad(rows, ((0, 0), (3, 2))))[:, 3:3 + words]
    for mask, dense in ((masks, rows), (ints(rows[:1]).expand(2 * n, words), np.repeat(rows[:1], 2 * n, 0))):
        note(f"attn tree strides n={n}")
        out, lse = run(mx, paged, q, mask, starts, n, out=buf[:, :2 * group, :128])
        ref = D.attention(f64(q), paged.k, paged.ks, paged.v, paged.vs, paged.table, lens, starts, 128 ** -0.5, dense)
        attention_close(out, lse, ref)
        rest = buf.clone()
        rest[:, :2 * group, :128] = 42.0
        assert (rest == 42.0).all()


@pytest.mark.parametrize("group", [1, 20])
def test_masks_beyond_32_bits(mx, group):
    # a mask whose last rows lie past 2^32 bytes
    rng = np.random.default_rng(14)
    n, lens = 4, [90]
    paged = Paged(rng, lens, 1, 128, 16)
    parents, starts = forest(rng, [n])
    rows, pos = D.tree_mask(parents, starts, 1, lens)
    big = torch.zeros((n - 1) * (1 << 29) + 1, dtype=torch.int32, device="cuda")
    mask = torch.as_strided(big, (n, 1), (1 << 29, 1))
    mx.mx_tree_mask(ints(parents), mask, max_q=n)
    torch.cuda.synchronize()
    assert np.array_equal(mask.cpu().numpy(), rows)
    q = bf16(rng.standard_normal((n, group, 128))).cuda()
    note(f"attn tree mask 6 GiB group={group}")
    out, lse = run(mx, paged, q, mask, starts, n)
    ref = D.attention(f64(q), paged.k, paged.ks, paged.v, paged.vs, paged.table, lens, starts, 128 ** -0.5, rows)
    attention_close(out, lse, ref)


def test_rows_behind_the_last_sequence_are_left_alone(mx):
    rng = np.random.default_rng(10)
    for n, group in ((5, 4), (40, 4)):
        paged = Paged(rng, [100, 60], 1, 128, 16)
        starts = [0, n, 2 * n - 2]
        q = bf16(rng.standard_normal((2 * n + 3, group, 128))).cuda()
        parents, _ = forest(rng, [n, n - 2])
        mask, _ = D.tree_mask(parents, starts, 2)
        padded = np.concatenate([mask, np.full((5, 2), -1, np.int32)])
        note(f"attn tree rows behind n={n}")
        out, lse = run(mx, paged, q, padded, starts, n)
        used = slice(0, starts[-1])
        ref = D.attention(f64(q)[used], paged.k, paged.ks, paged.v, paged.vs, paged.table, [100, 60], starts,
                          128 ** -0.5, mask)
        attention_close(out[used], lse[used], ref)
        assert torch.isnan(out[starts[-1]:].float()).all() and torch.isnan(lse[starts[-1]:]).all()


@pytest.mark.parametrize("n,group", [(6, 4), (50, 4)])
def test_a_nan_node_reaches_only_its_descendants(mx, n, group):
    rng = np.random.default_rng(n + 1)
    paged = Paged(rng, [100 + n], 1, 128, 16)
    parents, starts = forest(rng, [n])
    mask, _ = D.tree_mask(parents, starts, 2)
    t = 100 + 2                                            # node 2
    paged.ks[paged.table[0, t // 16], :, t % 16] = 255
    paged.k[paged.table[0, t // 16], :, t % 16] = 0
    q = bf16(rng.standard_normal((n, group, 128))).cuda()
    note(f"attn tree NaN node n={n}")
    out, lse = run(mx, paged, q, mask, starts, n)
    ref = D.attention(f64(q), paged.k, paged.ks, paged.v, paged.vs, paged.table, [100 + n], starts, 128 ** -0.5, mask)
    assert np.isnan(ref[0]).any() and not np.isnan(ref[0]).all()
    attention_close(out, lse, ref)


@pytest.mark.parametrize("n,lens", [(8, [3000, 9]), (60, [2500, 64])])
def test_streams_graphs_and_repeated_bits(mx, n, lens):
    rng = np.random.default_rng(12)
    paged = Paged(rng, lens, 2, 128, 16)
    cache, table, seq = mx.MxKvCacheFp4(*paged.tensors()), ints(paged.table), ints(lens)
    q = bf16(rng.standard_normal((2 * n, 8, 128))).cuda()
    parents, starts = forest(rng, [n, n])
    mask = ints(D.tree_mask(parents, starts, 2)[0])
    size = mx.mx_attn_fp4_workspace_size(2, n, 8, 2, 128)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out, side, graph = torch.empty_like(q), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    note(f"attn tree captured n={n}")
    with torch.cuda.graph(graph, stream=side):
        mx.mx_attn_tree_fp4(cache, q, mask, table, seq, out, ws)
    for step in range(4):
        seq.copy_(torch.tensor([lens[0] - 300 * step, lens[1] - step], dtype=torch.int32))
        parents, _ = forest(rng, [n, n])
        mask.copy_(torch.from_numpy(D.tree_mask(parents, starts, 2)[0]))
        q.copy_(bf16(rng.standard_normal((2 * n, 8, 128))))
        eager = torch.empty_like(q)
        mx.mx_attn_tree_fp4(cache, q, mask, table, seq, eager, torch.zeros_like(ws))
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), step
    with torch.cuda.stream(side):
        mx.mx_attn_tree_fp4(cache, q, mask, table, seq, out, ws)
    side.synchronize()
    assert torch.equal(out, eager)


def test_refusals(mx):
    rng = np.random.default_rng(13)
    paged = Paged(rng, [40], 2, 128, 16)
    q = bf16(rng.standard_normal((3, 4, 128))).cuda()
    ws = torch.zeros(mx.mx_attn_fp4_workspace_size(1, 3, 4, 2, 128), dtype=torch.uint8, device="cuda")
    mask, pos = ints(np.ones((3, 1))), ints([37, 38, 38])
    good = dict(cache=mx.MxKvCacheFp4(*paged.tensors()), q=q, mask=mask, page_table=ints(paged.table),
                seq_lens=ints([40]), out=torch.empty_like(q), workspace=ws)

    def refused(status=None, **change):
        with pytest.raises((mx.MxError, TypeError)) as e:
            mx.mx_attn_tree_fp4(**{**good, **change})
        assert status is None and e.type is TypeError or e.value.status == status

    refused(mx.MX_ERR_DEVICE, q=q.cpu())
    refused(mx.MX_ERR_DEVICE, mask=mask.cpu())
    refused(None, mask=mask.long())
    refused(None, mask=None)
    refused(mx.MX_ERR_SHAPE, mask=mask[:2])
    refused(mx.MX_ERR_SHAPE, mask=mask[:, :0])
    refused(mx.MX_ERR_STRIDE, mask=ints(np.ones((3, 4)))[:, ::2])
    refused(mx.MX_ERR_NULL, window=4)                                # without positions
    refused(mx.MX_ERR_SHAPE, window=4, positions=pos[:2])
    refused(None, window=4, positions=pos.long())
    refused(mx.MX_ERR_SHAPE, window=-1, positions=pos)
    refused(mx.MX_ERR_SHAPE, max_q=2)
    refused(mx.MX_ERR_SHAPE, max_q=40, q_starts=ints([0, 3]))         # a word too few
    refused(mx.MX_ERR_SHAPE, max_q=65537, q_starts=ints([0, 3]), mask=ints(np.ones((3, 2049))))
    refused(mx.MX_ERR_WORKSPACE, workspace=None)
    refused(mx.MX_ERR_SHAPE, scale=float("nan"))
    refused(None, seq_lens=ints([40]).long())
