"""The draft operators together with the append and the attention, as a decoding loop uses them: whole steps
in one captured graph, nothing read back between them, against the same text decoded token by token."""
import numpy as np
import pytest
import torch

from draft_util import ints, random_parents, softmax
from gpu_util import note
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu


class Model:
    """A target and a draft that look at the last token alone, and layers whose keys, values and queries
    are functions of the token: what a cache has to hold for a text is known."""

    def __init__(self, rng, vocab, layers, hk, group, dim, positions):
        self.vocab, self.layers, self.hk, self.group, self.dim = vocab, layers, hk, group, dim
        z = 1.5 * rng.standard_normal((vocab, vocab))
        self.target = torch.from_numpy(softmax(z)).float().cuda()
        self.draft = torch.from_numpy(softmax(z + 0.7 * rng.standard_normal((vocab, vocab)))).float().cuda()
        self.order = self.draft.sort(-1, descending=True).indices.to(torch.int32)
        make = lambda heads: torch.from_numpy(rng.standard_normal((layers, vocab, heads, dim))).to(torch.bfloat16).cuda()
        self.k, self.v, self.q = make(hk), make(hk), make(hk * group)
        f = 10000.0 ** (-np.arange(0, dim, 2) / dim)
        a = np.arange(positions)[:, None] * f
        self.cos, self.sin = (torch.from_numpy(x.astype(np.float32)).cuda() for x in (np.cos(a), np.sin(a)))

    def caches(self, mx, pages, page):
        t = [torch.zeros((self.layers, pages, self.hk, page, w), dtype=torch.uint8, device="cuda")
             for w in (self.dim // 2, self.dim // 32) * 2]
        return t, [mx.MxKvCacheFp4(*(x[i] for x in t)) for i in range(self.layers)]


def slots_of(table, at, page):
    """Slots of tokens `at` [batch, n] (long) of each sequence."""
    return (table.long().gather(1, at // page) * page + at % page).flatten()


@pytest.mark.parametrize("dim,hk,group,n,page", [(128, 2, 4, 12, 16), (64, 2, 3, 40, 48), (256, 1, 2, 20, 32)])
def test_steps_in_one_graph_give_what_single_tokens_give(mx, dim, hk, group, n, page):
    rng = np.random.default_rng(dim + n)
    B, vocab, layers, steps, prompt = 3, 50, 3, 6, [7, 30, 1]
    m = Model(rng, vocab, layers, hk, group, dim, 512)
    width = -(-(max(prompt) + steps * n + n) // page)
    table = ints(rng.permutation(B * width + 1)[:B * width].reshape(B, width))
    t, caches = m.caches(mx, B * width + 1, page)
    text = [rng.integers(0, vocab, p + 1).tolist() for p in prompt]          # the last one is not cached yet
    # the prompts' keys and values
    for layer, cache in enumerate(caches):
        for b, p in enumerate(prompt):
            ids = torch.tensor(text[b][:p], device="cuda")
            mx.mx_kv_append_fp4(cache, m.k[layer, ids], m.v[layer, ids],
                                slots_of(table[b:b + 1], torch.arange(p, device="cuda")[None], page),
                                torch.arange(p, dtype=torch.int32, device="cuda"), m.cos, m.sin)
    # one tree for all steps: its shape in the parents, its tokens from the draft's order
    parents = np.stack([random_parents(rng, n, 5) for _ in range(B)])
    rank = np.zeros((B, n), int)
    for b in range(B):
        for i in range(1, n):
            rank[b, i] = int((parents[b, 1:i] == parents[b, i]).sum())
    par, rk = torch.from_numpy(parents).cuda(), torch.from_numpy(rank).cuda()
    flat, N = ints(parents.reshape(-1)), B * n
    lens, new_lens = ints([p + n for p in prompt]), ints([0] * B)            # with the tree's nodes
    root = ints([x[-1] for x in text])
    words = -(-n // 32)
    mask, pos = ints(np.zeros((N, words))), ints([0] * N)
    q = torch.zeros((layers, N, hk * group, dim), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(max(mx.mx_attn_fp4_workspace_size(B, n, hk * group, hk, dim), mx.mx_tree_verify_workspace_size(B)),
                     dtype=torch.uint8, device="cuda")
    accept_u, sample_u = torch.zeros(N, device="cuda"), torch.zeros(B, device="cuda")
    path, said, count = ints(np.zeros((B, n))), ints(np.zeros((B, n))), ints([0] * B)
    tokens, tree = ints(np.zeros((B, n))), torch.arange(n, device="cuda")

    def step():
        tokens[:, 0] = root
        for i in range(1, n):
            tokens[:, i] = m.order[tokens.gather(1, par[:, i:i + 1].long())[:, 0].long(), rk[:, i]]
        mx.mx_tree_mask(flat, mask, seq_lens=lens, positions=pos, max_q=n)
        ids = tokens.flatten().long()
        slots = slots_of(table, (lens - n).long()[:, None] + tree, page)
        for layer, cache in enumerate(caches):
            mx.mx_kv_append_fp4(cache, m.k[layer, ids], m.v[layer, ids], slots, pos, m.cos, m.sin)
            mx.mx_qk_norm_rope(m.q[layer, ids], None, pos, m.cos, m.sin, q[layer], None)
            mx.mx_attn_tree_fp4(cache, q[layer], mask, table, lens, out[layer], ws, max_q=n)
        mx.mx_tree_verify(m.target[ids], None, tokens.flatten(), flat, accept_u, sample_u, path, said, count, ws, max_q=n)
        mx.mx_kv_accept_fp4(caches, table, lens, path, count, lens_out=new_lens, max_q=n)

    keep = [x.clone() for x in t]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                        # torch's own first calls, outside the capture
        step()
    side.synchronize()
    for x, y in zip(t, keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    note(f"draft steps captured D={dim} n={n}")
    with torch.cuda.graph(graph, stream=side):
        step()
    went = 0
    for s in range(steps):
        u, v = rng.random(N).astype(np.float32), rng.random(B).astype(np.float32)
        accept_u.copy_(torch.from_numpy(u))
        sample_u.copy_(torch.from_numpy(v))
        base = (lens - n).tolist()
        graph.replay()
        torch.cuda.synchronize()
        ids = tokens.cpu().numpy().reshape(-1)
        target = m.target.double().cpu().numpy()[ids]
        want = O.verify(target, None, ids, parents.reshape(-1), u, v, [n * b for b in range(B + 1)], n)
        for a, b in zip((path, said, count), want):
            assert np.array_equal(a.cpu().numpy(), b), s
        assert new_lens.tolist() == [x + int(c) for x, c in zip(base, want[2])]
        # the attention of the accepted nodes is that of their text, token by token
        fresh, singles = m.caches(mx, B * width + 1, page)
        for b in range(B):
            k = int(want[2][b])
            whole = text[b] + want[1][b, :k - 1].tolist()            # up to the last accepted node
            assert len(whole) == base[b] + k
            idx = torch.tensor(whole, device="cuda")
            at = torch.arange(len(whole), device="cuda")
            for layer, single in enumerate(singles):
                mx.mx_kv_append_fp4(single, m.k[layer, idx], m.v[layer, idx], slots_of(table[b:b + 1], at[None], page),
                                    at.to(torch.int32), m.cos, m.sin)
                o = torch.zeros((k, hk * group, dim), dtype=torch.bfloat16, device="cuda")
                nodes = torch.from_numpy(want[0][b, :k]).long().cuda() + n * b
                mx.mx_attn_fp4(single, q[layer, nodes], table[b:b + 1], ints([len(whole)]), o,
                               torch.zeros_like(ws), max_q=k)
                torch.cuda.synchronize()
                # Other tilings: both are off from the exact mean by at most 2^-7 of the mean of |v| (their
                # weights' and own roundings); values are below 4.
                off = (o.float() - out[layer, nodes].float()).abs().max()
                assert float(off) <= 2 * 2.0 ** -7 * 4, (s, b, layer)
            text[b] += want[1][b, :k].tolist()
            went += k - 1
        # and the cache holds the text's bytes
        for x, y in zip(t, fresh):
            for b in range(B):
                tok = torch.arange(len(text[b]) - 1, device="cuda")
                pg, of = table[b].long()[tok // page], tok % page
                assert torch.equal(x[:, pg, :, of], y[:, pg, :, of]), (s, b)
        root.copy_(ints([x[-1] for x in text]))
        lens.copy_(new_lens + n)
    assert went > 3                                      # some drafts stood
