"""Attention over the paged MXFP4 cache (mx_attn_fp4) at the edges of what it accepts, against the
float64 oracle with the bounds of attention_util.attention_close."""
import numpy as np
import pytest
import torch

from attention_util import Paged, attention_close, f64, oracle
from gpu_util import note
from oracle.attention_oracle import cache_rows
from test_gpu_attn_fp4 import queries, run, uniform

pytestmark = pytest.mark.gpu


def evict(paged, news, window):
    """Drops what lies before each sequence's oldest window: bytes 0xFF (every scale NaN), pages that
    hold nothing else -1 in the table, and page 0, which is read in their place, 0xFF throughout."""
    arrays = (paged.k, paged.ks, paged.v, paged.vs)
    page = paged.page_size
    free = next(i for i in range(len(paged.k)) if i not in paged.table)
    for a in arrays:
        a[free] = a[0]
        a[0] = 0xFF
    paged.table[paged.table == 0] = free
    for b, (length, n) in enumerate(zip(paged.lens, news)):
        low = max(length - n + 1 - window, 0)
        for t in range(min(low, length)):
            for a in arrays:
                a[paged.table[b, t // page], :, t % page] = 0xFF
        paged.table[b, :low // page] = -1


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,group,window", [(1, 4, 1), (1, 8, 50), (1, 16, 501), (4, 8, 50), (5, 6, 200),
                                             (70, 2, 50), (70, 4, 333), (300, 1, 37)])
def test_what_lies_before_the_window_is_never_used(mx, D, nq, group, window):
    # windows that begin inside a page, inside a step and inside a tile, and whole pages before them
    rng = np.random.default_rng(D + nq + window)
    lens = [nq + n for n in (0, 1, 17, 100, 395, 600, 1177)]
    paged = Paged(rng, lens, 2, D, 16)
    evict(paged, [nq] * len(lens), window)
    q = queries(rng, nq * len(lens), 2 * group, D)
    note(f"attn evicted D={D} nq={nq} group={group} window={window}")
    out, lse = run(mx, paged, q, window=window)
    ref = oracle(paged, q, uniform(nq, len(lens)), D ** -0.5, window=window)
    assert not np.isnan(ref[0]).any()
    attention_close(out, lse, ref)


@pytest.mark.parametrize("D,nq,hk,page", [(128, 70, 33, 16), (256, 40, 33, 16)])
def test_what_lies_before_the_window_is_never_used_in_a_deal(mx, D, nq, hk, page):
    rng = np.random.default_rng(D + nq)
    lens, news = [2600, 900, 0, 130], [nq, 3, 0, nq // 2]
    starts = [0, *np.cumsum(news).tolist()]
    paged = Paged(rng, lens, hk, D, page)
    evict(paged, news, 2205)
    q = queries(rng, starts[-1], 2 * hk, D)
    note(f"attn evicted, dealt D={D} nq={nq}")
    out, lse = run(mx, paged, q, starts=starts, max_q=nq, window=2205)
    attention_close(out, lse, oracle(paged, q, starts, D ** -0.5, window=2205))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,group", [(4, 4), (9, 6), (70, 2), (300, 1)])
def test_the_widest_windows_hide_nothing(mx, D, nq, group):
    # sequences shorter than their queries: the first positions are negative
    rng = np.random.default_rng(D + nq)
    lens = [0, 1, nq // 3, nq - 1, nq, nq + 200]
    paged = Paged(rng, lens, 2, D, 16)
    q = queries(rng, nq * len(lens), 2 * group, D)
    note(f"attn widest windows D={D} nq={nq} group={group}")
    want, want_lse = run(mx, paged, q)
    attention_close(want, want_lse, oracle(paged, q, uniform(nq, len(lens)), D ** -0.5))
    for window in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - nq):
        out, lse = run(mx, paged, q, window=window)
        assert torch.equal(out, want) and torch.equal(lse, want_lse), window


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("sign", ["both", "negative"])
def test_the_largest_score_wins_however_large(mx, D, nq, sign):
    """Scores so large, and so far apart, that a row's output is the value of its largest score alone.

    A score's fp32 sum and its product with the scale are off by at most d = 2^-20 scale sum |q k| each
    (the rounded product by 2^-24 of it): a row whose largest score is more than 4 d + 200 above the
    next has one weight, all others being below 2^-200 of it (0 in fp32).  Its output is that value:
    the same bits from maxima of 2^28 (in base 2) on, where the weight is 1; below, the weight is 2 to
    the power of the maximum's rounding error and rounded to bf16 once, and attention_close's bound
    holds: 2^-8 for that and 2^-8 for the result's rounding.  Its log-sum-exp is the score."""
    rng = np.random.default_rng(D + nq)
    lens = [600, 1500, 129]
    paged = Paged(rng, lens, 1, D, 16, lo=124, hi=130, junk=0x7F)
    if sign == "negative":
        paged.k &= 0x77                                       # keys above 0, queries below
    q = queries(rng, nq * len(lens), 4, D)
    if sign == "negative":
        q = -q.abs()
    for e in (20, 27, 28, 29, 31, 33, 60, 95):
        scale = 2.0 ** e / D
        note(f"attn scores of 2^{e} D={D} nq={nq} sign={sign}")
        out, lse = run(mx, paged, q, scale=scale)
        got, got_lse, rows = f64(out), f64(lse), 0
        for b, n in enumerate(lens):
            k = cache_rows(paged.k, paged.ks, paged.table[b], n)[0]
            v = cache_rows(paged.v, paged.vs, paged.table[b], n)[0]
            for i in range(nq):
                seen = n - nq + i + 1
                for h in range(4):
                    x = f64(q[b * nq + i, h])
                    s = scale * (k[:seen] @ x)
                    d = 2.0 ** -20 * scale * (np.abs(k[:seen]) @ np.abs(x)).max()
                    first, second = np.sort(s)[::-1][:2]
                    if first - second <= 4 * d + 200:
                        continue
                    rows += 1
                    where = (e, b, i, h)
                    value = v[s.argmax()]
                    tol = 0 if abs(first) * np.log2(np.e) >= 2.0 ** 28 * (1 + 2.0 ** -18) else 2.0 ** -7 * np.abs(value)
                    assert (np.abs(got[b * nq + i, h] - value) <= tol).all(), where
                    assert abs(got_lse[b * nq + i, h] - first) <= 2 * d, where
        assert rows > nq * len(lens) * 2                      # of 4 heads


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,nq,group", [(65, 1, 4), (130, 2, 5), (300, 1, 16)])
def test_more_than_64_sequences_cut_between_workgroups(mx, D, B, nq, group):
    # the deal of more than 64 sequences, with units of up to 40 tiles where a run is a few
    rng = np.random.default_rng(D + B)
    lens = rng.integers(0, 1500, B).tolist()
    lens[3], lens[B // 2], lens[B - 1] = 5000, 3333, 4001
    news = [int(n) for n in rng.integers(0, nq + 1, B)]
    news[3] = news[B - 1] = nq
    starts = [0, *np.cumsum(news).tolist()]
    paged = Paged(rng, lens, 1, D, 32)
    q = queries(rng, starts[-1], group, D)
    tiles = [(n // 128 + 2) for n, m in zip(lens, news) if m]
    assert max(tiles) > 4 * (sum(tiles) // 256 + 1)                # one is cut whatever the number of workgroups
    ws = torch.zeros(mx.mx_attn_fp4_workspace_size(B, nq, group, 1, D), dtype=torch.uint8, device="cuda")
    note(f"attn {B} sequences cut D={D} nq={nq} group={group}")
    how = dict(starts=starts, max_q=nq, ws=ws)
    out, lse = run(mx, paged, q, **how)
    attention_close(out, lse, oracle(paged, q, starts, D ** -0.5))
    again, lse2 = run(mx, paged, q, **how)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,nq,hk,lens", [(1, 150, 2, [2500]), (4, 70, 33, [2600, 900, 0, 130])])
def test_many_rows_on_other_streams_and_in_graphs(mx, D, B, nq, hk, lens):
    # keys in parts, joined by a second launch: split, and dealt by lengths that change between replays
    rng = np.random.default_rng(D + B)
    news = [nq, 3, 0, nq // 2][:B]
    starts = [0, *np.cumsum(news).tolist()]
    paged = Paged(rng, lens, hk, D, 32)
    cache = mx.MxKvCacheFp4(*paged.tensors())
    q = queries(rng, starts[-1], 2 * hk, D)
    want, _ = run(mx, paged, q, starts=starts, max_q=nq, lse=False)
    table = torch.from_numpy(paged.table).cuda()
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ds = torch.tensor(starts, dtype=torch.int32, device="cuda")
    ws = torch.zeros(mx.mx_attn_fp4_workspace_size(B, nq, 2 * hk, hk, D), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    note(f"attn many rows on a side stream D={D} B={B}")
    with torch.cuda.stream(side):
        mx.mx_attn_fp4(cache, q, table, dl, out, ws, q_starts=ds, max_q=nq)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    note("attn many rows captured")
    with torch.cuda.graph(graph, stream=side):
        mx.mx_attn_fp4(cache, q, table, dl, out, ws, q_starts=ds, max_q=nq)
    for step, share in enumerate((1.0, 0.5, 0.9, 0.05, 1.0)):
        dl.copy_(torch.tensor([int(n * share) for n in lens], dtype=torch.int32))
        q.copy_(queries(rng, starts[-1], 2 * hk, D))
        eager = torch.empty_like(q)
        mx.mx_attn_fp4(cache, q, table, dl, eager, torch.zeros_like(ws), q_starts=ds, max_q=nq)
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), step
