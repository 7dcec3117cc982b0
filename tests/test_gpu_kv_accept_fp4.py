"""mx_kv_accept_fp4 against the oracle, byte for byte and with every other byte untouched: paths of every
kind, moves across pages, layers in one launch and several, strides, offsets, wild tables, graphs."""
import numpy as np
import pytest
import torch

from draft_util import ints
from gpu_util import note
from oracle import draft_oracle as D

pytestmark = pytest.mark.gpu


def paths(rng, sizes, width, how="any"):
    """Paths as verification writes them, and their counts."""
    path, count = np.full((len(sizes), width), -1, np.int32), np.zeros(len(sizes), np.int32)
    for b, n in enumerate(sizes):
        if n == 0:
            continue
        k = {"any": int(rng.integers(1, min(n, width) + 1)), "all": min(n, width), "root": 1}[how]
        path[b, :k] = [0] + sorted(rng.choice(np.arange(1, n), k - 1, replace=False).tolist())
        count[b] = k
    return path, count


def caches(rng, layers, pages, heads, page, dim):
    return [[rng.integers(0, 256, (pages, heads, page, w), dtype=np.uint8) for w in (dim // 2, dim // 32) * 2]
            for _ in range(layers)]


def check(mx, cs, table, lens, sizes, path, count, max_q, tensors=None, ragged=True, lens_out=True):
    starts = [0, *np.cumsum(sizes).tolist()]
    ts = tensors or [[torch.from_numpy(a).cuda() for a in c] for c in cs]
    new = torch.full((len(lens),), -77, dtype=torch.int32, device="cuda") if lens_out else None
    mx.mx_kv_accept_fp4([mx.MxKvCacheFp4(*t) for t in ts], ints(table), ints(lens), ints(path), ints(count),
                        lens_out=new, q_starts=ints(starts) if ragged else None, max_q=max_q)
    torch.cuda.synchronize()
    for layer, (c, t) in enumerate(zip(cs, ts)):
        want, lengths = D.accept(c, table, lens, starts, path, count)
        for i, (a, b) in enumerate(zip(t, want)):
            got = a.cpu().numpy()
            assert np.array_equal(got, b), (layer, i, np.argwhere(got != b)[:3])
    if lens_out:
        assert np.array_equal(new.cpu().numpy(), lengths)


def setup(rng, lens, page, spare=1):
    counts = [-(-n // page) for n in lens]
    order = rng.permutation(sum(counts) + spare)
    table = np.full((len(lens), max(counts) + 1), -9, np.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, len(order)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 48])
@pytest.mark.parametrize("how", ["any", "all", "root"])
def test_paths(mx, dim, page, how):
    rng = np.random.default_rng(dim + page)
    sizes = [1, 2, 9, 26, 0, 64, 40, 17, 100]
    lens = [s + int(rng.integers(0, 70)) for s in sizes]
    table, pages = setup(rng, lens, page)
    path, count = paths(rng, sizes, 100, how)
    note(f"accept D={dim} page={page} {how}")
    check(mx, caches(rng, 1, pages, 3, page, dim), table, lens, sizes, path, count, 100)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_neighbouring_moves_that_lie_on_each_other(mx, dim):
    # every row but the first moves by one or a few places, over many chunks of a wavefront's
    rng = np.random.default_rng(dim)
    for skip in (1, 2, 5):
        n = 1024
        path = np.full((1, n), -1, np.int32)
        k = n - skip
        path[0, :k] = [0, *range(1 + skip, n)]
        table, pages = setup(rng, [n + 10], 16)
        note(f"accept shifted D={dim} by {skip}")
        check(mx, caches(rng, 1, pages, 2, 16, dim), table, [n + 10], [n], path, np.array([k], np.int32), n, ragged=False)


@pytest.mark.parametrize("layers", [2, 5, 64, 65, 130])
def test_layers(mx, layers):
    rng = np.random.default_rng(layers)
    sizes, lens = [8, 30], [20, 45]
    table, pages = setup(rng, lens, 16)
    path, count = paths(rng, sizes, 12)
    note(f"accept {layers} layers")
    check(mx, caches(rng, layers, pages, 2, 16, 64), table, lens, sizes, path, count, 30)


def test_layers_side_by_side_in_one_tensor(mx):
    # [pages, layers, heads, page, bytes]: a layer's pages lie far apart, other layers' between them
    rng = np.random.default_rng(7)
    sizes, lens = [8, 30], [20, 45]
    table, pages = setup(rng, lens, 16)
    path, count = paths(rng, sizes, 30)
    cs = caches(rng, 3, pages, 2, 16, 128)
    whole = [torch.stack([torch.from_numpy(c[i]) for c in cs], 1).cuda() for i in range(4)]
    note("accept layers in one tensor")
    check(mx, cs, table, lens, sizes, path, count, 30, tensors=[[w[:, i] for w in whole] for i in range(3)])


def test_wild_arguments_stay_inside(mx):
    # entries that are no page, lengths beyond the table, below the nodes and negative, nodes that are none,
    # counts beyond the path: skipped, nothing else is touched
    rng = np.random.default_rng(8)
    sizes = [10] * 7
    lens = [30, 10 ** 9, 4, -5, 31, 32, 33]
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 7], [-1, 8], [9, 10 ** 8], [10, 11]], np.int32)
    path, count = paths(rng, sizes, 10)
    path[6, 1:4] = [3, 2 ** 31 - 1, 6]
    path[5, 1:3] = [-7, 5]
    count[:] = [10 ** 9, 5, 5, 5, 5, 5, 5]
    path[0] = [0, 2, 3, 5, 6, 7, 9, -1, -1, -1]
    note("accept wild")
    check(mx, caches(rng, 2, 12, 2, 16, 128), table, lens, sizes, path, count, 10)
    check(mx, caches(rng, 2, 12, 2, 16, 128), table, lens, sizes, path, -count, 10, lens_out=False)


def test_offsets_beyond_32_bits(mx):
    rng = np.random.default_rng(10)
    sizes, lens = [20], [60]
    table = np.array([[3, 1, 0, 2]], np.int32)
    path, count = paths(rng, sizes, 20, "any")
    path[0, :4], count[0] = [0, 5, 9, 18], 4
    cs = caches(rng, 1, 4, 2, 16, 128)
    stride = 1 << 31
    big = torch.zeros(4 * stride, dtype=torch.uint8, device="cuda")
    ts = []
    for i, a in enumerate(cs[0]):
        p, h, s, w = a.shape
        t = torch.as_strided(big, (p, h, s, w), (stride, s * w, w, 1), storage_offset=(1 << 20) * i)
        t.copy_(torch.from_numpy(a))
        ts.append(t)
    note("accept 4 GiB offsets")
    check(mx, cs, table, lens, sizes, path, count, 20, tensors=[ts])


def test_more_wavefronts_than_a_grid_has(mx):
    # 64 layers x 65535 sequences: the grid's wavefronts take several each
    rng = np.random.default_rng(13)
    B, n = 65535, 4
    cs = caches(rng, 64, 4, 1, 16, 64)
    lens, table = np.zeros(B, np.int32), np.full((B, 1), -1, np.int32)
    path, count = np.full((B, n), -1, np.int32), np.zeros(B, np.int32)
    for b, page in ((0, 0), (40000, 2), (B - 1, 3)):
        lens[b], table[b, 0], path[b, :2], count[b] = 16, page, [0, 3], 2
    note("accept 64 layers x 65535 sequences")
    check(mx, cs, table, lens, [n] * B, path, count, n, ragged=False)


def test_graph_and_stream(mx):
    rng = np.random.default_rng(11)
    sizes, lens = [12, 30], [40, 45]
    starts = [0, 12, 42]
    table, pages = setup(rng, lens, 16)
    cs = caches(rng, 2, pages, 2, 16, 128)
    ts = [[torch.from_numpy(a).cuda() for a in c] for c in cs]
    handles = [mx.MxKvCacheFp4(*t) for t in ts]
    path, count = paths(rng, sizes, 30)
    dev = [ints(path), ints(count)]
    tb, ln, st, new = ints(table), ints(lens), ints(starts), ints([0, 0])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    note("accept captured")
    with torch.cuda.graph(graph, stream=side):
        mx.mx_kv_accept_fp4(handles, tb, ln, *dev, lens_out=new, q_starts=st, max_q=30)
    for _ in range(4):
        path, count = paths(rng, sizes, 30)
        dev[0].copy_(torch.from_numpy(path))
        dev[1].copy_(torch.from_numpy(count))
        graph.replay()
        torch.cuda.synchronize()
        for i, t in enumerate(ts):
            cs[i], lengths = D.accept(cs[i], table, lens, starts, path, count)
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(t, cs[i]))
        assert np.array_equal(new.cpu().numpy(), lengths)


def test_refusals(mx):
    rng = np.random.default_rng(12)
    c = [mx.MxKvCacheFp4(*(torch.from_numpy(a).cuda() for a in x)) for x in caches(rng, 2, 4, 2, 16, 128)]
    other = mx.MxKvCacheFp4(*(torch.from_numpy(a).cuda() for a in caches(rng, 1, 4, 1, 16, 128)[0]))
    good = dict(caches=c, page_table=ints([[0, 1]]), seq_lens=ints([20]), path=ints([[0, 2]]), count=ints([2]), max_q=4)

    def refused(status=None, **change):
        with pytest.raises((mx.MxError, TypeError)) as e:
            mx.mx_kv_accept_fp4(**{**good, **change})
        assert status is None and e.type is TypeError or e.value.status == status

    mx.mx_kv_accept_fp4(**good)
    mx.mx_kv_accept_fp4(**{**good, "caches": []})
    refused(None, caches=[c[0], None])
    refused(mx.MX_ERR_SHAPE, caches=[c[0], other])
    refused(mx.MX_ERR_STRIDE, caches=[c[0], c[1], c[0]])             # one cache twice
    refused(None, page_table=ints([[0, 1]]).long())
    refused(mx.MX_ERR_SHAPE, page_table=ints([0, 1]))
    refused(mx.MX_ERR_SHAPE, seq_lens=ints([20, 20]))
    refused(mx.MX_ERR_DEVICE, seq_lens=ints([20]).cpu())
    refused(mx.MX_ERR_SHAPE, path=ints([0, 2]))
    refused(mx.MX_ERR_SHAPE, count=ints([2, 2]))
    refused(mx.MX_ERR_STRIDE, path=ints([[0, 2, 3, 3]])[:, ::2])
    refused(mx.MX_ERR_STRIDE, lens_out=good["seq_lens"])
    refused(mx.MX_ERR_SHAPE, max_q=1025)
    refused(None, max_q=None)
