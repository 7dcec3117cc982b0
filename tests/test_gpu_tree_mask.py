"""mx_tree_mask against the oracle (exact): sizes around the words' edges, ragged sequences, strides,
nodes whose parent is none, rows behind the last sequence, graphs, refusals."""
import numpy as np
import pytest
import torch

from draft_util import forest, ints
from gpu_util import note
from oracle import draft_oracle as D

pytestmark = pytest.mark.gpu


def check(mx, parents, starts, lens, words, max_q, spare=0, gap=0, with_starts=True, **how):
    N = len(parents)
    buf = torch.full((N + spare, words + gap), -77, dtype=torch.int32, device="cuda")
    pos = torch.full((N + spare,), -77, dtype=torch.int32, device="cuda")
    padded = np.concatenate([parents, np.zeros(spare, np.int32)])
    mx.mx_tree_mask(ints(padded), buf[:, :words], seq_lens=ints(lens), positions=pos,
                    q_starts=ints(starts) if with_starts else None, max_q=max_q, **how)
    torch.cuda.synchronize()
    mask, want = D.tree_mask(parents, starts, words, lens)
    assert np.array_equal(buf[:N, :words].cpu().numpy(), mask)
    assert np.array_equal(pos[:N].cpu().numpy(), want)
    rest = buf.clone()
    rest[:N, :words] = -77
    assert (rest == -77).all() and (pos[N:] == -77).all()


@pytest.mark.parametrize("kind", ["tree", "chain", "star"])
@pytest.mark.parametrize("n,words", [(1, 1), (2, 3), (31, 1), (32, 1), (33, 2), (64, 2), (65, 3), (200, 7),
                                     (1000, 32), (1024, 33)])
def test_sizes(mx, kind, n, words):
    rng = np.random.default_rng(n)
    parents, starts = forest(rng, [n], kind)
    note(f"tree mask {kind} n={n}")
    check(mx, parents, starts, [n + 5], words, n, with_starts=False)


def test_ragged_batches_and_what_lies_behind_them(mx):
    rng = np.random.default_rng(1)
    sizes = [0, 1, 40, 7, 0, 96, 33, 0]
    parents, starts = forest(rng, sizes)
    note("tree mask ragged")
    check(mx, parents, starts, [9, 0, 40, 1000, 3, 2 ** 31 - 1, 33, 5], 3, 96, spare=5, gap=2)


def test_many_sequences(mx):
    rng = np.random.default_rng(2)
    sizes = rng.integers(0, 6, 3000).tolist()
    parents, starts = forest(rng, sizes)
    note("tree mask 3000 sequences")
    check(mx, parents, starts, rng.integers(0, 10 ** 6, 3000).tolist(), 1, 5)


def test_parents_that_are_none(mx):
    parents = np.array([5, -1, 2, 3, 1, 2 ** 31 - 1, -2 ** 31, 4, 7, 9], np.int32)
    note("tree mask bad parents")
    check(mx, parents, [0, 10], [10], 1, 10)


def test_sequences_longer_than_max_q_are_cut(mx):
    rng = np.random.default_rng(4)
    parents, _ = forest(rng, [20, 8], "chain")
    mask = torch.full((28, 1), -77, dtype=torch.int32, device="cuda")
    note("tree mask cut")
    mx.mx_tree_mask(ints(parents), mask, q_starts=ints([0, 20, 28]), max_q=8)
    got = mask.cpu().numpy()[:, 0]
    want = [(1 << (i + 1)) - 1 for i in range(8)]
    assert got[:8].tolist() == want and got[20:].tolist() == want and (got[8:20] == -77).all()


def test_stream_and_graph(mx):
    rng = np.random.default_rng(5)
    sizes = [26] * 4
    parents, starts = forest(rng, sizes)
    p, mask, pos, lens = ints(parents), ints(np.zeros((104, 1))), ints(np.zeros(104)), ints([30, 40, 50, 60])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    note("tree mask captured")
    with torch.cuda.graph(graph, stream=side):
        mx.mx_tree_mask(p, mask, seq_lens=lens, positions=pos, max_q=26)
    for _ in range(3):
        parents, starts = forest(rng, sizes)
        p.copy_(torch.from_numpy(parents))
        lens.add_(3)
        graph.replay()
        torch.cuda.synchronize()
        want = D.tree_mask(parents, starts, 1, lens.tolist())
        assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[1])


def test_refusals(mx):
    p, mask, lens, pos = ints([-1, 0, 0]), ints(np.zeros((3, 2))), ints([9]), ints([0] * 3)
    good = dict(parents=p, mask=mask, seq_lens=lens, positions=pos, max_q=3)

    def refused(status=None, **change):
        with pytest.raises((mx.MxError, TypeError)) as e:
            mx.mx_tree_mask(**{**good, **change})
        assert status is None and e.type is TypeError or e.value.status == status

    refused(mx.MX_ERR_DEVICE, parents=p.cpu())
    refused(None, parents=p.long())
    refused(None, mask=mask.float())
    refused(mx.MX_ERR_SHAPE, mask=ints(np.zeros((2, 2))))
    refused(mx.MX_ERR_SHAPE, mask=ints(np.zeros((3, 0))))
    refused(mx.MX_ERR_STRIDE, mask=ints(np.zeros((3, 4)))[:, ::2])
    refused(mx.MX_ERR_STRIDE, mask=ints(np.zeros((1, 2))).expand(3, 2))
    refused(mx.MX_ERR_NULL, seq_lens=None)
    refused(mx.MX_ERR_NULL, positions=None)
    refused(mx.MX_ERR_SHAPE, positions=pos[:2])
    refused(mx.MX_ERR_SHAPE, max_q=2)
    refused(mx.MX_ERR_SHAPE, max_q=1025, q_starts=ints([0, 3]), mask=ints(np.zeros((3, 40))))
    refused(None, max_q=None, q_starts=ints([0, 3]))
    refused(None, max_q=None, seq_lens=None, positions=None)
