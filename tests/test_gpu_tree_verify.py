"""mx_tree_verify against the oracle, token for token.  Inputs are random, so no random number lies within
the rounding of 64-bit sums (2^-40 of a row's probability at these sizes) of where a decision turns but for
those placed there on purpose, in numbers that every sum holds exactly."""
import numpy as np
import pytest
import torch

from draft_util import forest, ints, softmax
from gpu_util import note
from oracle import draft_oracle as D

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def workspace(mx, B):
    return torch.zeros(mx.mx_tree_verify_workspace_size(B), dtype=torch.uint8, device="cuda")


def run(mx, target, draft, tokens, parents, u, s, starts, width, max_q, ws=None, ragged=True, **how):
    B = len(starts) - 1
    path, out = (torch.full((B, width), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    count = torch.full((B,), -77, dtype=torch.int32, device="cuda")
    mx.mx_tree_verify(target, draft, ints(tokens), ints(parents), torch.from_numpy(u).cuda(),
                      torch.from_numpy(s).cuda(), path, out, count, workspace(mx, B) if ws is None else ws,
                      q_starts=ints(starts) if ragged else None, max_q=max_q, **how)
    torch.cuda.synchronize()
    return path.cpu().numpy(), out.cpu().numpy(), count.cpu().numpy()


def case(rng, sizes, V, dtype, mode, kind="tree", sharp=3.0, apart=1.0):
    parents, starts = forest(rng, sizes, kind)
    N = len(parents)
    z = sharp * rng.standard_normal((N, V))
    target = torch.from_numpy(softmax(z)).to(TYPES[dtype])
    draft = torch.from_numpy(softmax(z + apart * rng.standard_normal((N, V)))).to(TYPES[dtype])
    tokens = np.zeros(N, np.int32)
    d64 = draft.double().numpy()
    for b in range(len(sizes)):
        kids = {}
        for i in range(starts[b] + 1, starts[b + 1]):
            kids.setdefault(starts[b] + parents[i], []).append(i)
        for up, its in kids.items():
            w = d64[up] / d64[up].sum()
            if mode == "chosen":
                order = np.argsort(-d64[up], kind="stable")
                tokens[its] = [order[k % V] for k in range(len(its))]
            else:
                left = int((w > 0).sum())
                for k, i in enumerate(its):
                    if mode == "distinct" and k < left:
                        x = rng.choice(V, p=w / w.sum())
                        w = w.copy()
                        w[x] = 0
                    else:
                        x = rng.choice(V, p=d64[up] / d64[up].sum())
                    tokens[i] = x
    return (target, None if mode == "chosen" else draft, tokens, parents, rng.random(N).astype(np.float32),
            rng.random(len(sizes)).astype(np.float32), starts)


def compare(mx, c, width, max_q, mode, what="", on_gpu=None, **how):
    target, draft, tokens, parents, u, s, starts = c
    f8 = lambda t: None if t is None else t.double().numpy()
    want = D.verify(f8(target), f8(draft), tokens, parents, u, s, starts, width, mode != "distinct")
    t, d = on_gpu or (target.cuda(), None if draft is None else draft.cuda())
    got = run(mx, t, d, tokens, parents, u, s, starts, width, max_q, replacement=mode != "distinct", **how)
    for name, a, b in zip(("path", "tokens", "count"), got, want):
        assert np.array_equal(a, b), f"{what} {name}: {np.argwhere(a != b)[:4]}"
    return want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", ["drawn", "distinct", "chosen"])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 1000, 4097, 8193])
def test_trees_over_vocabularies(mx, dtype, mode, V):
    rng = np.random.default_rng(V + len(mode))
    sizes = [1, 2, 5, 12, 26, 0, 33, 40, 3, 9, 17, 64, 20, 20, 20, 20]
    if V >= 4097:
        sizes = [1, 26, 0, 12, 33, 9]
    c = case(rng, sizes, V, dtype, mode, sharp=1.5)
    note(f"verify {mode} {dtype} V={V}")
    want = compare(mx, c, max(sizes), max(sizes), mode)
    if V > 2 and mode != "chosen":             # flat rows: a chosen draft is rarely what the target draws
        assert 1 < want[2].max()


@pytest.mark.parametrize("mode", ["drawn", "distinct", "chosen"])
def test_many_small_walks(mx, mode):
    # several rejections in a row, descents after them, leaves, places that end
    rng = np.random.default_rng(17)
    sizes = rng.integers(0, 30, 600).tolist()
    c = case(rng, sizes, 40, "fp32", mode, sharp=1.0, apart=1.5)
    for width in (30, 3, 1):
        note(f"verify {mode} 600 sequences, width {width}")
        want = compare(mx, c, width, 30, mode)
        assert width == 1 or want[2].max() == (3 if width == 3 else want[2].max()) > 2


@pytest.mark.parametrize("kind,sizes", [("chain", [5] * 9), ("star", [30] * 9), ("chain", [200, 1]),
                                        ("star", [1024]), ("chain", [1024])])
@pytest.mark.parametrize("mode", ["drawn", "distinct", "chosen"])
def test_chains_and_stars(mx, kind, sizes, mode):
    rng = np.random.default_rng(sizes[0])
    c = case(rng, sizes, 1100 if sizes[0] < 500 else 1500, "fp32", mode, kind, apart=0.3 if kind == "chain" else 3.0)
    note(f"verify {kind} {sizes} {mode}")
    compare(mx, c, sizes[0], sizes[0], mode)


@pytest.mark.parametrize("dtype,V,mode", [("fp32", 100003, "distinct"), ("fp32", 131072, "drawn"),
                                          ("bf16", 151937, "chosen"), ("fp16", 65537, "drawn"),
                                          ("bf16", 262143, "distinct")])
def test_large_vocabularies_in_slices(mx, dtype, V, mode):
    rng = np.random.default_rng(V)
    c = case(rng, [6, 1, 11], V, dtype, mode, apart=1.5)
    note(f"verify {mode} {dtype} V={V}")
    compare(mx, c, 11, 11, mode)
    ws = workspace(mx, 3)
    compare(mx, c, 11, 11, mode, ws=ws)
    for _ in range(3):                                     # the workspace is left as it has to be
        compare(mx, c, 11, 11, mode, ws=ws)


@pytest.mark.parametrize("mode", ["drawn", "distinct", "chosen"])
def test_batches_whose_rows_are_not_cut(mx, mode):
    rng = np.random.default_rng(31)
    sizes = rng.integers(1, 6, 140).tolist()
    c = case(rng, sizes, 20011, "bf16", mode, apart=2.0)
    note(f"verify {mode} 140 sequences, whole rows")
    compare(mx, c, 5, 5, mode)


@pytest.mark.parametrize("dtype,least", [("fp32", 2.0 ** -149), ("bf16", 2.0 ** -133), ("fp16", 2.0 ** -24)])
def test_the_smallest_probabilities(mx, dtype, least):
    # rows of subnormal numbers alone: their sums are exact, and multiples of the smallest one
    rng = np.random.default_rng(32)
    V, n = 5003, 64
    k = rng.integers(0, 8, (n, V))
    t = torch.from_numpy(k * least).to(TYPES[dtype])
    assert (t.double() == torch.from_numpy(k * least)).all()
    s = (rng.integers(0, 1 << 10, n) / 1024).astype(np.float32)
    upto = k.cumsum(-1)
    want = [int(np.nonzero(upto[i] > float(s[i]) * upto[i, -1])[0][0]) for i in range(n)]
    note(f"verify subnormal {dtype}")
    got = run(mx, t.cuda(), None, np.zeros(n), -np.ones(n), np.zeros(n, np.float32), s, list(range(n + 1)), 1, 1)
    assert got[1][:, 0].tolist() == want


def test_where_the_next_token_falls(mx):
    # 2^12 equal probabilities: every sum is exact, the number 2^-12 k falls on a border
    V = 4096
    target = torch.full((1, V), 1 / V)
    for V0 in (4096, 4095, 3333):
        t = target[:, :V0].contiguous()
        for s, want in ((0.0, 0), (0.99999994, V0 - 1), (1.0, V0 - 1), (float("nan"), V0 - 1), (-1.0, 0)):
            got = run(mx, t.cuda(), None, [0], [-1], np.zeros(1, np.float32), np.array([s], np.float32), [0, 1], 1, 1)
            assert got[1][0, 0] == want, (V0, s)
    note("verify borders")
    k = np.arange(4096, dtype=np.float32) / 4096
    n = len(k)
    got = run(mx, target.expand(n, V).cuda().contiguous(), None, np.zeros(n), -np.ones(n), np.zeros(n, np.float32), k,
              list(range(n + 1)), 1, 1)
    assert np.array_equal(got[1][:, 0], np.arange(n))      # sums up to v have to exceed k: the k-th


def test_every_place_of_a_row(mx):
    # all of the probability on one token, at every place around the chunks' edges
    V, places = 20011, [0, 1, 3, 4, 255, 256, 4095, 4096, 4097, 8191, 8192, 12287, 12288, 20007, 20008, 20010]
    for dtype in TYPES.values():
        t = torch.zeros((len(places), V), dtype=dtype)
        t[torch.arange(len(places)), torch.tensor(places)] = 1
        n = len(places)
        note(f"verify places {dtype}")
        for s in (0.0, 0.5, 0.99):
            got = run(mx, t.cuda(), None, np.zeros(n), -np.ones(n), np.zeros(n, np.float32), np.full(n, s, np.float32),
                      list(range(n + 1)), 2, 1)
            assert got[1][:, 0].tolist() == places and (got[1][:, 1] == -1).all() and got[2].tolist() == [1] * n


def test_edges_by_hand(mx):
    one = torch.tensor([[0.25, 0.5, 0.25, 0.0]] * 3)
    u, s = np.array([0, .9, .9], np.float32), np.zeros(1, np.float32)

    def go(target=one, draft=one, tokens=(0, 1, 2), parents=(-1, 0, 1), u=u, s=0.0, width=3):
        p, t, c = run(mx, target.cuda(), None if draft is None else draft.cuda(), tokens, parents,
                      np.asarray(u, np.float32), np.array([s], np.float32), [0, 3], width, 3)
        k = c[0]
        assert (p[0, k:] == -1).all() and (t[0, k:] == -1).all()
        return p[0, :k].tolist(), t[0, :k].tolist()

    note("verify by hand")
    assert go() == ([0, 1, 2], [1, 2, 0])
    assert go(width=2) == ([0, 1], [1, 0])
    assert go(tokens=(0, 9, 2)) == ([0], [0])                       # no such token; p - q leaves nothing
    assert go(tokens=(0, -1, 2)) == ([0], [0])
    assert go(tokens=(0, 3, 2), draft=None) == ([0], [0])
    assert go(s=0.25) == ([0, 1, 2], [1, 2, 1])
    assert go(target=0 * one) == ([0], [-1])
    assert go(draft=0 * one) == ([0, 1, 2], [1, 2, 0])              # what the draft calls impossible
    assert go(draft=None, tokens=(0, 1, 1), parents=(-1, 0, 0), u=(0, .6, 0), s=.5) == ([0], [2])   # twice
    assert go(parents=(-1, 0, 2)) == ([0, 1], [1, 0])               # a node that is its own parent
    assert go(parents=(-1, 7, -3)) == ([0], [0])
    assert go(u=(0, float("nan"), .9)) == ([0], [0])                # no number: rejected
    bad = torch.tensor([[float("nan"), 0.5, float("inf"), -1.0]] * 3)
    assert go(target=bad, u=(0, .9, 0)) == ([0, 1], [1, 1])
    assert go(target=bad, draft=bad, u=(0, .9, 0), s=.5) == ([0, 1], [1, 1])
    # the chosen draft has all but what its type loses: nothing is left without it
    assert go(target=torch.tensor([[0.9, 0, 0, 0]] * 3), draft=None, tokens=(0, 0, 1), parents=(-1, 0, 0),
              u=(0, .95, .5), s=.3) == ([0], [0])


def test_strides_and_alignment(mx):
    rng = np.random.default_rng(21)
    for dtype in TYPES:
        for V, off in ((1000, 1), (4099, 3), (9001, 5)):
            c = case(rng, [9, 4, 12], V, dtype, "drawn")
            N = len(c[3])
            wide = torch.full((2, N, V + 7), float("inf"), dtype=TYPES[dtype], device="cuda")
            t, d = wide[0, :, off:off + V], wide[1, :, off:off + V]
            t.copy_(c[0])
            d.copy_(c[1])
            note(f"verify strides {dtype} V={V}")
            compare(mx, c, 12, 12, "drawn", on_gpu=(t, d))
    c = case(rng, [9, 9], 500, "fp32", "drawn")
    row = c[1][:1]
    note("verify one draft row for all")
    compare(mx, (c[0], row.expand(18, 500), *c[2:]), 9, 9, "drawn",
            on_gpu=(c[0].cuda(), row.cuda().expand(18, 500)), ragged=False)


def test_offsets_beyond_32_bits(mx):
    # the last rows lie past 2^32 bytes of their matrix
    rng = np.random.default_rng(22)
    V, N = 300, 6
    c = case(rng, [3, 3], V, "bf16", "drawn")
    big = torch.zeros((N - 1) * (1 << 29) + V, dtype=torch.bfloat16, device="cuda")
    t = torch.as_strided(big, (N, V), (1 << 29, 1))
    t.copy_(c[0])
    note("verify 4 GiB offsets")
    compare(mx, c, 3, 3, "drawn", on_gpu=(t, c[1].cuda()))


def test_rows_behind_the_last_sequence_and_batches_without_nodes(mx):
    rng = np.random.default_rng(23)
    c = case(rng, [5, 0, 7], 300, "fp32", "drawn")
    target, draft, tokens, parents, u, s, starts = c
    pad = lambda a: np.concatenate([a, np.full(4, 1, a.dtype)])
    nan = torch.full((4, 300), float("nan"))
    note("verify rows behind")
    want = D.verify(target.double().numpy(), draft.double().numpy(), tokens, parents, u, s, starts, 7)
    got = run(mx, torch.cat([target, nan]).cuda(), torch.cat([draft, nan]).cuda(), pad(tokens), pad(parents), pad(u), s,
              starts, 7, 7)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    e = np.zeros(0, np.float32)
    path, out, count = run(mx, torch.zeros((0, 9), device="cuda"), None, e, e, e, s, [0, 0, 0, 0], 4, 0)
    assert (path == -1).all() and (out == -1).all() and (count == 0).all()


def test_streams_graphs_and_an_attention_workspace(mx):
    rng = np.random.default_rng(24)
    V, sizes = 50001, [9, 12, 5]
    ws = torch.zeros(mx.mx_attn_fp4_workspace_size(3, 12, 32, 8, 128), dtype=torch.uint8, device="cuda")
    assert ws.numel() >= mx.mx_tree_verify_workspace_size(3)
    c = case(rng, sizes, V, "fp32", "distinct")
    dev = [c[0].cuda(), c[1].cuda(), ints(c[2]), ints(c[3]), torch.from_numpy(c[4]).cuda(), torch.from_numpy(c[5]).cuda()]
    outs = [ints(np.zeros((3, 12))), ints(np.zeros((3, 12))), ints(np.zeros(3))]
    starts = ints(c[6])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    note("verify captured")
    with torch.cuda.graph(graph, stream=side):
        mx.mx_tree_verify(*dev, *outs, ws, q_starts=starts, max_q=12, replacement=False)
    for step in range(4):
        c = case(rng, sizes, V, "fp32", "distinct")
        for t, a in zip(dev, c):
            t.copy_(a if isinstance(a, torch.Tensor) else torch.from_numpy(a))
        for t in outs:
            t.fill_(-77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = D.verify(c[0].double().numpy(), c[1].double().numpy(), *c[2:6], c[6], 12, False)
        assert all(np.array_equal(t.cpu().numpy(), w) for t, w in zip(outs, want)), step
        with torch.cuda.stream(side):
            mx.mx_tree_verify(*dev, *outs, ws, q_starts=starts, max_q=12, replacement=False)
        side.synchronize()
        assert all(np.array_equal(t.cpu().numpy(), w) for t, w in zip(outs, want)), step
    assert not ws[:1 << 23].any()                          # the counters are zero again


def test_calls_at_once_on_several_streams(mx):
    # each with a workspace of its own; their workgroups share the chip, and some have to wait for others
    rng = np.random.default_rng(25)
    streams, calls = [torch.cuda.Stream() for _ in range(4)], []
    for i, (sizes, V) in enumerate((([9] * 16, 30011), ([12] * 5, 60000), ([30] * 2, 100003), ([26] * 60, 5000))):
        c = case(rng, sizes, V, "fp32", "distinct", apart=2.0)
        dev = [c[0].cuda(), c[1].cuda(), ints(c[2]), ints(c[3]), torch.from_numpy(c[4]).cuda(),
               torch.from_numpy(c[5]).cuda()]
        outs = [ints(np.zeros((len(sizes), max(sizes)))) for _ in range(2)] + [ints(np.zeros(len(sizes)))]
        want = D.verify(c[0].double().numpy(), c[1].double().numpy(), *c[2:6], c[6], max(sizes), False)
        calls.append((dev, outs, workspace(mx, len(sizes)), want))
    torch.cuda.synchronize()
    note("verify on four streams")
    for _ in range(20):
        for (dev, outs, ws, _), st in zip(calls, streams):
            with torch.cuda.stream(st):
                mx.mx_tree_verify(*dev, *outs, ws, replacement=False)
    torch.cuda.synchronize()
    for dev, outs, ws, want in calls:
        assert all(np.array_equal(t.cpu().numpy(), w) for t, w in zip(outs, want))
        assert not ws[:1 << 23].any()


def test_refusals(mx):
    t = torch.full((3, 8), 0.125, device="cuda")
    f = torch.zeros(3, device="cuda")
    good = dict(target=t, draft=t, tokens=ints([0] * 3), parents=ints([-1, 0, 1]), accept_u=f, sample_u=f[:1],
                path=ints(np.zeros((1, 3))), tokens_out=ints(np.zeros((1, 3))), count=ints([0]),
                workspace=workspace(mx, 1))

    def refused(status=None, **change):
        with pytest.raises((mx.MxError, TypeError)) as e:
            mx.mx_tree_verify(**{**good, **change})
        assert status is None and e.type is TypeError or e.value.status == status

    refused(mx.MX_ERR_DEVICE, target=t.cpu())
    refused(None, target=t.double(), draft=None)
    refused(None, draft=t.bfloat16())
    refused(mx.MX_ERR_SHAPE, draft=t[:2])
    refused(mx.MX_ERR_SHAPE, target=t[0], draft=None)
    refused(mx.MX_ERR_STRIDE, target=torch.zeros(3, 16, device="cuda")[:, ::2])
    refused(mx.MX_ERR_STRIDE, target=t[:1].expand(3, 8))
    refused(None, tokens=ints([0] * 3).long())
    refused(mx.MX_ERR_SHAPE, parents=ints([0] * 4))
    refused(None, accept_u=f.double())
    refused(mx.MX_ERR_SHAPE, sample_u=f[:1].view(1, 1))
    refused(mx.MX_ERR_SHAPE, sample_u=f[:2], path=ints(np.zeros((2, 3))), tokens_out=ints(np.zeros((2, 3))),
            count=ints([0, 0]))
    refused(mx.MX_ERR_SHAPE, path=ints(np.zeros((2, 3))))
    refused(mx.MX_ERR_SHAPE, path=ints(np.zeros((1, 0))), tokens_out=ints(np.zeros((1, 0))))
    refused(mx.MX_ERR_SHAPE, tokens_out=ints(np.zeros((1, 2))))
    refused(mx.MX_ERR_STRIDE, path=ints(np.zeros((1, 6)))[:, ::2])
    refused(mx.MX_ERR_SHAPE, count=ints([0, 0]))
    refused(mx.MX_ERR_WORKSPACE, workspace=None)
    refused(mx.MX_ERR_WORKSPACE, workspace=good["workspace"][:-8])
    refused(mx.MX_ERR_SHAPE, max_q=1025, q_starts=ints([0, 3]))
    refused(None, q_starts=ints([0, 3]))
    refused(mx.MX_ERR_SHAPE, target=t[:, :0], draft=None)
