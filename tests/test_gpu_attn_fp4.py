"""Attention over the paged MXFP4 cache (mx_attn_fp4) against the float64 oracle: lengths around
every tile edge, groups and head sizes, masks that leave rows empty, windows, ragged queries, pages
that end inside a tile, strides, junk beyond the lengths, NaN tokens, streams and graphs."""
import numpy as np
import pytest
import torch

from attention_util import Paged, attention_close, bf16, f64, oracle
from gpu_util import note

pytestmark = pytest.mark.gpu

LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 700]


def run(mx, paged, q, starts=None, max_q=None, ws=None, lse=True, out=None, **how):
    cache = mx.MxKvCacheFp4(*paged.tensors())
    B, N, H = len(paged.lens), q.shape[0], q.shape[1]
    mq = max_q if max_q is not None else N // B
    if ws is None:
        n = mx.mx_attn_fp4_workspace_size(B, mq, H, paged.heads, paged.D)
        ws = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    l = torch.full((N, H), float("nan"), device="cuda") if lse else None
    table = torch.from_numpy(paged.table).cuda()
    lens = torch.tensor(paged.lens, dtype=torch.int32, device="cuda")
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    mx.mx_attn_fp4(cache, q, table, lens, out, ws, q_starts=st, max_q=max_q, lse=l, **how)
    torch.cuda.synchronize()
    return out, l


def queries(rng, n, heads, D, scale=1.0):
    return bf16(scale * rng.standard_normal((n, heads, D))).cuda()


def uniform(n, B):
    return [n * i for i in range(B + 1)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 7, 16])
def test_single_tokens_at_every_length(mx, D, group):
    rng = np.random.default_rng(100 + D + group)
    paged = Paged(rng, LENS, 2, D, 16)
    q = queries(rng, len(LENS), 2 * group, D)
    note(f"attn tokens D={D} group={group}")
    out, lse = run(mx, paged, q)
    ref = oracle(paged, q, uniform(1, len(LENS)), D ** -0.5)
    attention_close(out, lse, ref)
    assert not f64(out)[0].any() and np.isneginf(f64(lse)[0]).all()     # a sequence without keys


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,group,page", [(2, 8, 48), (3, 5, 16), (4, 12, 32), (5, 13, 64), (9, 16, 16)])
def test_a_few_queries(mx, D, nq, group, page):
    # sequences shorter than their queries: the first rows' positions are negative, they see nothing
    rng = np.random.default_rng(7 * D + nq)
    lens = [0, 1, 3, 4, 31, 33, 66, 130, 290]
    paged = Paged(rng, lens, 1, D, page)
    q = queries(rng, nq * len(lens), group, D)
    note(f"attn few D={D} nq={nq} group={group} page={page}")
    out, lse = run(mx, paged, q)
    attention_close(out, lse, oracle(paged, q, uniform(nq, len(lens)), D ** -0.5))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 37), (True, 64), (True, 200)])
def test_masks(mx, D, causal, window):
    rng = np.random.default_rng(D + window)
    for nq, lens, group in ((3, [1, 40, 129, 300], 4), (70, [70, 71, 165, 390], 2)):
        paged = Paged(rng, lens, 2, D, 16)
        q = queries(rng, nq * len(lens), 2 * group, D)
        note(f"attn masks D={D} nq={nq} causal={causal} window={window}")
        out, lse = run(mx, paged, q, causal=causal, window=window)
        attention_close(out, lse, oracle(paged, q, uniform(nq, len(lens)), D ** -0.5, causal=causal,
                                         window=window), f"nq {nq}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_prompts(mx, D, group):
    rng = np.random.default_rng(3 * D + group)
    news = [1, 63, 64, 65, 130, 0, 257]
    lens = [1, 63, 80, 65, 131, 40, 257]
    starts = [0, *np.cumsum(news).tolist()]
    paged = Paged(rng, lens, 1, D, 32)
    q = queries(rng, starts[-1], group, D)
    note(f"attn prompts D={D} group={group}")
    out, lse = run(mx, paged, q, starts=starts, max_q=257)
    attention_close(out, lse, oracle(paged, q, starts, D ** -0.5))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_chunk_against_a_long_past_is_split(mx, D):
    # one block of rows for each head: the keys are dealt to many workgroups and joined
    rng = np.random.default_rng(D)
    paged = Paged(rng, [3001, 1700], 1, D, 64)
    q = queries(rng, 2 * 96, 1, D)
    note(f"attn chunk D={D}")
    out, lse = run(mx, paged, q)
    attention_close(out, lse, oracle(paged, q, uniform(96, 2), D ** -0.5))


@pytest.mark.parametrize("D,nq,hk,group,page", [(64, 70, 33, 2, 32), (128, 70, 33, 2, 64), (128, 35, 65, 2, 16),
                                                (256, 40, 33, 1, 48)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1500)])
def test_chunks_of_very_different_lengths_are_dealt(mx, D, nq, hk, group, page, causal, window):
    # nearly all keys are one sequence's: its blocks' tiles are dealt to all workgroups, runs begin and
    # end inside of them, and the rows of most heads are joined from several parts
    rng = np.random.default_rng(11 * D + hk + window)
    lens, news = [2200, 900, 0, 130], [nq, 3, 0, nq // 2]
    starts = [0, *np.cumsum(news).tolist()]
    paged = Paged(rng, lens, hk, D, page)
    q = queries(rng, starts[-1], hk * group, D)
    ws = torch.zeros(mx.mx_attn_fp4_workspace_size(4, nq, hk * group, hk, D), dtype=torch.uint8, device="cuda")
    note(f"attn dealt D={D} nq={nq} hk={hk} group={group} causal={causal} window={window}")
    how = dict(starts=starts, max_q=nq, ws=ws, causal=causal, window=window)
    out, lse = run(mx, paged, q, **how)
    attention_close(out, lse, oracle(paged, q, starts, D ** -0.5, causal=causal, window=window))
    again, lse2 = run(mx, paged, q, **how)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_ragged_tokens_split_over_many_workgroups(mx):
    rng = np.random.default_rng(5)
    lens = [9000, 0, 1, 130, 4097, 17, 2, 640]
    paged = Paged(rng, lens, 2, 128, 16)
    q = queries(rng, len(lens), 8, 128)
    note("attn ragged")
    out, lse = run(mx, paged, q)
    attention_close(out, lse, oracle(paged, q, uniform(1, len(lens)), 128 ** -0.5))


def test_more_sequences_than_threads(mx):
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 40, 700).tolist()
    news = [int(x) for x in rng.integers(0, 2, 700)]
    starts = [0, *np.cumsum(news).tolist()]
    paged = Paged(rng, lens, 1, 64, 16)
    q = queries(rng, starts[-1], 2, 64)
    note("attn 700 sequences, about half without queries")
    out, lse = run(mx, paged, q, starts=starts, max_q=1)
    attention_close(out, lse, oracle(paged, q, starts, 64 ** -0.5))


def test_scores_of_every_size(mx):
    # large scores: the running maximum moves; equal ones; a scale of zero and a negative one
    rng = np.random.default_rng(8)
    paged = Paged(rng, [600, 129], 1, 128, 16, lo=118, hi=130)
    for scale, size in ((1.0, 3.0), (0.0, 1.0), (-0.05, 1.0), (0.3, 0.0)):
        for nq in (1, 40):
            q = queries(rng, 2 * nq, 4, 128, size)
            note(f"attn scale={scale} size={size} nq={nq}")
            out, lse = run(mx, paged, q, scale=scale)
            attention_close(out, lse, oracle(paged, q, uniform(nq, 2), scale), f"{scale} {size} {nq}")


@pytest.mark.parametrize("nq", [1, 2, 50])
def test_strides(mx, nq):
    # queries inside a packed projection, outputs with gaps that stay untouched, pages with gaps, a
    # page table that is a slice of a wider one
    rng = np.random.default_rng(nq)
    lens = [100, 77]
    paged = Paged(rng, lens, 2, 128, 16, gap=48 * 16)
    wide = queries(rng, 2 * nq, 6 + 4, 128)
    q = wide[:, :6]
    buf = torch.full((2 * nq, 7, 136), 42.0, dtype=torch.bfloat16, device="cuda")
    paged.table = np.ascontiguousarray(np.pad(paged.table, ((0, 0), (0, 3)), constant_values=-1))
    note(f"attn strides nq={nq}")
    out, lse = run(mx, paged, q, out=buf[:, :6, :128])
    attention_close(out, lse, oracle(paged, q, uniform(nq, 2), 128 ** -0.5))
    rest = buf.clone()
    rest[:, :6, :128] = 42.0
    assert (rest == 42.0).all()


@pytest.mark.parametrize("nq", [1, 3, 40])
def test_a_nan_token_reaches_only_queries_that_see_it(mx, nq):
    rng = np.random.default_rng(nq + 50)
    lens = [200, 200]
    paged = Paged(rng, lens, 1, 128, 16)
    t = 200 - max(1, nq // 2)                        # of the second sequence; early queries miss it
    paged.ks[paged.table[1, t // 16], :, t % 16] = 255
    paged.k[paged.table[1, t // 16], :, t % 16] = 0
    q = queries(rng, 2 * nq, 2, 128)
    note(f"attn NaN token nq={nq}")
    out, lse = run(mx, paged, q)
    ref = oracle(paged, q, uniform(nq, 2), 128 ** -0.5)
    assert np.isnan(ref[0]).any()
    attention_close(out, lse, ref)


def test_bad_tables_and_lengths_stay_inside_the_cache(mx):
    # lengths beyond the table are cut to it, negative ones are none, entries that are no page read
    # page 0: results are defined only in so far as nothing else is touched
    rng = np.random.default_rng(9)
    paged = Paged(rng, [64, 64, 64], 1, 64, 16, width_extra=0)
    q = queries(rng, 3, 2, 64)
    want = oracle(paged, q, uniform(1, 3), 0.125)
    paged.lens = [64, 10 ** 6, -5]
    note("attn lengths out of range")
    out, lse = run(mx, paged, q)
    for i in (0, 1):
        attention_close(out[i:i + 1], lse[i:i + 1], tuple(a[i:i + 1] for a in want))
    assert not f64(out)[2].any()
    note("attn page out of range")
    got = []
    for entry in (10 ** 7, -1, 0):
        paged.table[0, 1] = entry
        got.append(run(mx, paged, q)[0])
    for o in got[:2]:
        assert torch.equal(o.view(torch.int16), got[2].view(torch.int16)) and torch.equal(o[1], out[1])


def test_offsets_beyond_32_bits(mx):
    # a cache of more than 2^32 bytes, the sequence's pages at its far end
    rng = np.random.default_rng(10)
    paged = Paged(rng, [150], 1, 128, 64, spare=0, width_extra=0)
    stride = 1 << 31                                   # bytes from page to page
    pages = len(paged.k)
    big = [torch.zeros(stride * pages, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ts = []
    for i, a in enumerate((paged.k, paged.ks, paged.v, paged.vs)):
        p, h, s, w = a.shape
        t = torch.as_strided(big[i // 2], (p, h, s, w), (stride, s * w, w, 1),
                             storage_offset=(1 << 20) * (i % 2))
        t.copy_(torch.from_numpy(a))
        ts.append(t)
    q = queries(rng, 1, 4, 128)
    paged.tensors = lambda: ts
    note("attn 4 GiB offsets")
    out, lse = run(mx, paged, q)
    attention_close(out, lse, oracle(paged, q, [0, 1], 128 ** -0.5))
    q = queries(rng, 150, 1, 128)
    out, lse = run(mx, paged, q)
    attention_close(out, lse, oracle(paged, q, [0, 150], 128 ** -0.5))


@pytest.mark.parametrize("nq,lens", [(1, [5000, 3]), (64, [4000, 64])])
def test_workspace_is_left_reusable_and_bits_repeat(mx, nq, lens):
    rng = np.random.default_rng(11)
    paged = Paged(rng, lens, 2, 128, 16)
    q = queries(rng, 2 * nq, 4, 128)
    n = mx.mx_attn_fp4_workspace_size(2, nq, 4, 2, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    note(f"attn repeat nq={nq}")
    first, lse = run(mx, paged, q, ws=ws)
    for _ in range(3):
        again, lse2 = run(mx, paged, q, ws=ws)
        assert torch.equal(first, again) and torch.equal(lse, lse2)
    # another problem through the same workspace
    other = Paged(rng, [2500, 2600], 2, 128, 16)
    q2 = queries(rng, 2 * nq, 4, 128)
    out, l = run(mx, other, q2, ws=ws)
    attention_close(out, l, oracle(other, q2, uniform(nq, 2), 128 ** -0.5))


def test_one_workspace_for_calls_of_all_sizes(mx):
    # few rows, many rows in parts, other batches and head sizes in turn
    rng = np.random.default_rng(14)
    ws = torch.zeros(max(mx.mx_attn_fp4_workspace_size(8, 200, 8, 2, d) for d in (64, 128, 256)),
                     dtype=torch.uint8, device="cuda")
    for D, lens, nq in ((128, [900, 2000], 100), (128, [1500] * 8, 1), (256, [1100], 40), (64, [2600, 5, 700], 3),
                        (256, [3000, 1], 2), (128, [2500], 1), (64, [900], 200), (128, [1500, 800] * 4, 2)):
        paged = Paged(rng, lens, 2, D, 16)
        q = queries(rng, nq * len(lens), 8, D)
        note(f"attn shared workspace D={D} nq={nq} batch={len(lens)}")
        out, lse = run(mx, paged, q, ws=ws)
        attention_close(out, lse, oracle(paged, q, uniform(nq, len(lens)), D ** -0.5), f"{D} {nq}")


def test_streams_and_graph_replay(mx):
    rng = np.random.default_rng(12)
    paged = Paged(rng, [1000, 700], 2, 128, 16)
    cache = mx.MxKvCacheFp4(*paged.tensors())
    q = queries(rng, 2, 8, 128)
    want, _ = run(mx, paged, q, lse=False)
    table = torch.from_numpy(paged.table).cuda()
    lens = torch.tensor(paged.lens, dtype=torch.int32, device="cuda")
    ws = torch.zeros(mx.mx_attn_fp4_workspace_size(2, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    note("attn on a side stream")
    with torch.cuda.stream(side):
        mx.mx_attn_fp4(cache, q, table, lens, out, ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    note("attn captured")
    with torch.cuda.graph(graph, stream=side):
        mx.mx_attn_fp4(cache, q, table, lens, out, ws)
    for step in range(4):
        # lengths change between replays: the deal is made on the device
        lens.copy_(torch.tensor([1000 - 100 * step, 700 - 13 * step], dtype=torch.int32))
        q.copy_(queries(rng, 2, 8, 128))
        eager = torch.empty_like(q)
        mx.mx_attn_fp4(cache, q, table, lens, eager, torch.zeros_like(ws))
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), step


def test_binding_refusals(mx):
    rng = np.random.default_rng(13)
    paged = Paged(rng, [40], 2, 128, 16)
    k, ks, v, vs = paged.tensors()
    cache = mx.MxKvCacheFp4(k, ks, v, vs)
    q = queries(rng, 1, 4, 128)
    table = torch.from_numpy(paged.table).cuda()
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    ws = torch.zeros(mx.mx_attn_fp4_workspace_size(1, 1, 4, 2, 128), dtype=torch.uint8, device="cuda")
    good = dict(cache=cache, q=q, page_table=table, seq_lens=lens, out=torch.empty_like(q), workspace=ws)

    def refused(status=None, **change):
        with pytest.raises((mx.MxError, TypeError)) as e:
            mx.mx_attn_fp4(**{**good, **change})
        assert status is None and e.type is TypeError or e.value.status == status

    refused(mx.MX_ERR_DEVICE, q=q.cpu())
    refused(None, q=q.float())
    refused(mx.MX_ERR_SHAPE, q=queries(rng, 1, 3, 128), out=torch.empty(1, 3, 128, dtype=torch.bfloat16, device="cuda"))
    refused(mx.MX_ERR_SHAPE, out=torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda"))
    refused(mx.MX_ERR_SHAPE, q=q[..., :64], out=torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda"))
    refused(None, seq_lens=lens.long())
    refused(mx.MX_ERR_SHAPE, seq_lens=lens.repeat(2))
    refused(mx.MX_ERR_STRIDE, page_table=table.t().contiguous().t() if table.shape[1] > 1 and table.shape[0] > 1
            else torch.zeros(1, 8, dtype=torch.int32, device="cuda")[:, ::2])
    refused(mx.MX_ERR_WORKSPACE, workspace=None)
    refused(mx.MX_ERR_WORKSPACE, workspace=ws[:1 << 23])
    refused(mx.MX_ERR_SHAPE, window=5, causal=False)
    refused(mx.MX_ERR_SHAPE, window=-1)
    refused(mx.MX_ERR_SHAPE, max_q=2)                               # 2 rows in q expected
    refused(None, q_starts=torch.zeros(2, dtype=torch.int32, device="cuda"))     # without max_q
    refused(mx.MX_ERR_ALIGN, q=torch.empty(4 * 128 + 8, dtype=torch.bfloat16, device="cuda")[4:-4].view(1, 4, 128))
    refused(mx.MX_ERR_SHAPE, scale=float("inf"))
    for bad in (dict(k=k[:, :, :, :48]), dict(ks=ks[:, :1]), dict(v=v[:, :, :8]), dict(vs=vs.float())):
        with pytest.raises((mx.MxError, TypeError)):
            mx.MxKvCacheFp4(**{**dict(k=k, k_scale=ks, v=v, v_scale=vs), **{
                {"ks": "k_scale", "vs": "v_scale"}.get(n, n): t for n, t in bad.items()}})
    with pytest.raises(mx.MxError) as e:                            # tokens of a page apart
        mx.MxKvCacheFp4(*(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, ks, v, vs)))
    assert e.value.status == mx.MX_ERR_STRIDE
