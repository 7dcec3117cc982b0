"""The operators of a decoding step with a tree of drafted tokens, as cases that can be measured.

Four operators around the paged MXFP4 cache: masks and positions of trees given by their nodes'
parents ("mask"), attention of a tree's nodes over the cache ("attn"), verification of the drafted
tokens against the target's probabilities from given random numbers ("verify"), and the move of the
accepted path's keys and values to their places in every layer's cache ("accept").

`own` False runs their plain forms in elementary torch operations; `own` True makes the calls a user
of block_scaled_precision_act_amd makes.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------------- cases

def _mask(name, B, n, ragged):
    return dict(name=name, op="mask", B=B, n=n, ragged=ragged, L=2000, lmin=n)


def _attn(name, B, n, L, lmin, hq, hk, D, page, window=0, ragged=False, lse=False):
    return dict(name=name, op="attn", B=B, n=n, L=L, lmin=lmin, hq=hq, hk=hk, D=D, page=page,
                window=window, ragged=ragged, lse=lse)


def _verify(name, B, n, V, dtype, draft, chain=False, ragged=False):
    return dict(name=name, op="verify", B=B, n=n, V=V, dtype=dtype, draft=draft, chain=chain,
                ragged=ragged)


def _accept(name, layers, B, n, L, lmin, h, D, page, ragged=False):
    return dict(name=name, op="accept", layers=layers, B=B, n=n, L=L, lmin=lmin, h=h, D=D, page=page,
                ragged=ragged)


def listed():
    return [
        # the tree of one reply: all latency
        _mask("mask_tree", 1, 26, False),
        # many requests' trees of up to 129 nodes (five words a mask)
        _mask("mask_batch", 128, 129, True),
        # a small tree behind a short text
        _attn("attn_tree_short", 1, 8, 1000, 1000, 32, 8, 128, 16),
        # trees of up to 12 nodes for 41 sequences of very different lengths, an odd group of heads
        _attn("attn_tree_ragged", 41, 12, 8192, 16, 56, 8, 128, 16, ragged=True),
        # a window of the past, heads of 64, no shared heads
        _attn("attn_tree_window", 32, 26, 6144, 1536, 12, 12, 64, 32, window=4096),
        # heads of 256, an odd number of nodes
        _attn("attn_tree_wide", 2, 33, 32768, 20000, 16, 2, 256, 64, lse=True),
        # long contexts, trees of 64 nodes
        _attn("attn_tree_long", 4, 64, 131073, 120001, 32, 8, 128, 64, lse=True),
        # a chain of four drafted tokens of one reply
        _verify("verify_chain", 1, 5, 32000, "fp32", "drawn", chain=True),
        # trees whose nodes' children are drawn without replacement, an odd vocabulary
        _verify("verify_tree", 16, 26, 100003, "fp32", "distinct"),
        # trees of the draft's most probable tokens: no draft distribution
        _verify("verify_chosen", 41, 64, 131072, "bf16", "chosen", ragged=True),
        # one layer, one sequence
        _accept("accept_layer", 1, 1, 8, 1000, 1000, 8, 128, 16),
        # every layer of a model at once, 41 sequences
        _accept("accept_layers", 32, 41, 64, 512, 300, 8, 128, 64, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    D = rng.choice((64, 128, 128, 256))
    hk = rng.choice((1, 2, 4, 8, 12))
    hq = hk * rng.choice((1, 2, 4, 5, 7, 8, 16))
    page = rng.choice((16, 32, 48, 64, 128))
    op = rng.choice(("mask", "attn", "attn", "attn", "verify", "verify", "verify", "accept"))
    ragged = rng.random() < 0.5
    if op == "mask":
        n = _log(rng, 1, 200)
        c = _mask("", _log(rng, 1, 128 * 129 // n), n, ragged)
    elif op == "attn":
        cache = 4 * 120001 * 8 * 128 // (hk * D)            # cached tokens of the largest case
        pairs = 4 * 64 * 120001 * 32 * 128 // (hq * D)      # (query, token) pairs of the largest case
        n, B = _log(rng, 1, 128), _log(rng, 1, 64)
        if B * n * n > pairs:
            B = 1
        most = max(n, min(131073, cache // B, pairs // (B * n)))
        L = _log(rng, n, most)
        lmin = L if rng.random() < 0.4 else _log(rng, 1, L)
        window = _log(rng, 16, 4096) if rng.random() < 0.25 else 0
        c = _attn("", B, n, L, lmin, hq, hk, D, page, window=window, ragged=ragged and B > 1,
                  lse=rng.random() < 0.3)
    elif op == "verify":
        draft = rng.choice(("drawn", "distinct", "chosen"))
        V, n = _log(rng, 2000, 200000), _log(rng, 1, 64)
        B = _log(rng, 1, max(1, min(64, (1 if draft == "chosen" else 0.15) * 41 * 64 * 131072 // (n * V))))
        c = _verify("", B, n, V, rng.choice(("fp32", "fp32", "bf16", "fp16")), draft,
                    chain=rng.random() < 0.4, ragged=ragged and B > 1)
    else:
        n = _log(rng, 1, 128)
        L = _log(rng, n, 600)
        B = _log(rng, 1, 41)
        layers = _log(rng, 1, max(1, min(70, 32 * 41 * 512 * 8 * 128 // (B * L * hk * D))))
        c = _accept("", layers, B, n, L, _log(rng, n, L), hk, D, page, ragged)
    del c["name"]
    return c


def _lens(c):
    """(cached tokens, nodes among them) of each sequence."""
    lens, news = [], []
    for i in range(c["B"]):
        u, w = (i * 0.6180339887) % 1.0, (i * 0.7548776662) % 1.0
        news.append(1 + int((c["n"] - 1) * w) if c["ragged"] and i else c["n"])
        if "L" in c:
            lens.append(c["L"] if i == 0 else c["lmin"] + int((c["L"] - c["lmin"]) * u))
    return lens, news


# --------------------------------------------------------------------------------------- inputs

def _ints(values):
    return torch.as_tensor(values, dtype=torch.int32, device="cuda")


def _parents(g, B, n, chain=False):
    """Parents [B, n] of trees in order of their levels (a few children a node), on the host."""
    i = torch.arange(n)
    if chain:
        p = (i - 1).expand(B, n)
    else:
        p = ((i - 1) * (0.1 + 0.5 * torch.rand((B, n), generator=g))).long()
    return torch.where(i == 0, torch.full_like(p, -1), p)


def _ancestors(parents):
    """For parents [B, n]: which nodes [B, n, n] are a node's ancestors or itself, on the host."""
    B, n = parents.shape
    seen = torch.zeros((B, n, n), dtype=torch.bool)
    rows = torch.arange(B)
    for i in range(n):
        if i:
            seen[:, i] = seen[rows, parents[:, i]]
        seen[:, i, i] = True
    return seen


def _words(bits):
    """Truth values [..., n] as int32 words [..., ceil(n / 32)], the lowest bit first."""
    n = bits.shape[-1]
    b = torch.nn.functional.pad(bits.long(), (0, -n % 32)).unflatten(-1, (-1, 32))
    w = (b << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _quantise(x):
    """x fp32 [..., D] -> packed E2M1 codes [..., D / 2], low nibble first, and E8M0 [..., D / 32]."""
    b = x.unflatten(-1, (-1, 32))
    bits = b.abs().amax(-1).clamp_min(1e-4).view(torch.int32)
    byte = (bits >> 23) - 2 + ((bits & 0x7FFFFF) > 0x400000)
    y = b * ((254 - byte) << 23).view(torch.float32)[..., None]
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5))
    code = (code + 8 * torch.signbit(y)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], byte.to(torch.uint8)


def _pages(g, lens, page):
    """A page table [B, width] with the pages dealt in any order, and the number of pages."""
    counts = [-(-n // page) for n in lens]
    pages, width = sum(counts) + 2, max(counts)
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    table, at = [], 0
    for n in counts:
        table.append(order[at:at + n] + [0] * (width - n))
        at += n
    return _ints(table), pages


def prepare(case, seed):
    c = case
    host = torch.Generator()
    host.manual_seed(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, news = _lens(c)
    B, n = c["B"], c["n"]
    total = sum(news)
    starts = [0]
    for m in news:
        starts.append(starts[-1] + m)
    s = {"case": c, "starts": _ints(starts)}
    if lens:
        s["lens"] = _ints(lens)
    node = torch.arange(n) < torch.tensor(news)[:, None]              # [B, n]: the sequences' nodes
    if c["op"] != "accept":
        parents = _parents(host, B, n, c.get("chain", False))
        s["parents"] = parents[node].to(torch.int32).cuda()
    if c["op"] == "mask":
        s["mask"] = torch.empty((total, -(-n // 32)), dtype=torch.int32, device="cuda")
        s["pos"] = torch.empty(total, dtype=torch.int32, device="cuda")
    if c["op"] == "attn":
        hk, D, page = c["hk"], c["D"], c["page"]
        seen = _ancestors(parents)
        s["mask"] = _words(seen)[node].cuda()
        depth = seen.sum(-1) - 1
        s["pos"] = (torch.tensor(lens)[:, None] - torch.tensor(news)[:, None] + depth)[node].to(torch.int32).cuda()
        s["table"], pages = _pages(g, lens, page)
        chan = torch.exp(0.5 * torch.randn((hk, 1, D), generator=g, device="cuda"))
        shape = (pages, hk, page, D)
        s["cache"] = [*_quantise(torch.randn(shape, generator=g, device="cuda") * chan),
                      *_quantise(torch.randn(shape, generator=g, device="cuda") + 0.3 * chan)]
        s["q"] = torch.randn((total, c["hq"], D), generator=g, device="cuda").to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((total, c["hq"]), device="cuda") if c["lse"] else None
        if own:
            import block_scaled_precision_act_amd as mx
            m = mx.mx_attn_fp4_workspace_size(B, n, c["hq"], hk, D)
            s["ws"] = torch.zeros(max(m, 256), dtype=torch.uint8, device="cuda")
            s["handle"] = mx.MxKvCacheFp4(*s["cache"])
    if c["op"] == "verify":
        V, dtype = c["V"], TYPES[c["dtype"]]
        z = 4 * torch.randn((total, V), generator=g, device="cuda")
        s["target"] = torch.softmax(z, -1).to(dtype)
        z += 1.2 * torch.randn((total, V), generator=g, device="cuda")   # the draft's opinion
        # the children of a node, in order: which of its drafts a node is
        child = torch.zeros((B, n), dtype=torch.long)
        for i in range(1, n):
            child[:, i] = (parents[:, 1:i] == parents[:, i:i + 1]).sum(-1)
        most = min(V, int(child.max()) + 1)
        if c["draft"] == "chosen":
            s["draft"] = None
            drafts = z.topk(most, -1).indices
        else:
            s["draft"] = torch.softmax(z, -1).to(dtype)
            drafts = torch.multinomial(s["draft"].float(), most, c["draft"] == "drawn", generator=g)
        row = torch.tensor(starts[:-1])[:, None] + parents.clamp_min(0)
        s["tokens"] = drafts[row[node].cuda(), child[node].clamp_max(most - 1).cuda()].to(torch.int32)
        s["accept_u"] = torch.rand(total, generator=g, device="cuda")
        s["sample_u"] = torch.rand(B, generator=g, device="cuda")
        s["path"], s["new"] = (torch.empty((B, n), dtype=torch.int32, device="cuda") for _ in range(2))
        s["count"] = torch.empty(B, dtype=torch.int32, device="cuda")
        if own:
            import block_scaled_precision_act_amd as mx
            s["ws"] = torch.zeros(mx.mx_tree_verify_workspace_size(B), dtype=torch.uint8, device="cuda")
    if c["op"] == "accept":
        layers, h, D, page = c["layers"], c["h"], c["D"], c["page"]
        s["table"], pages = _pages(g, lens, page)
        s["cache"] = [torch.randint(0, 256, (layers, pages, h, page, w), dtype=torch.uint8, generator=g,
                                    device="cuda") for w in (D // 2, D // 32, D // 2, D // 32)]
        # a path of a tree in order of its levels: every node past the root comes from behind the
        # path's own places, so that a second call finds what the first one found
        path, count = [], []
        for m, u in zip(news, torch.rand((B, 9), generator=host).tolist()):
            k = min(1 + int(8 * u[0]), (m + 1) // 2)
            steps = sorted(range(k, m), key=lambda i: (i * (0.5 + u[1])) % 1.0)[:k - 1]
            path.append([0] + sorted(steps) + [-1] * (n - k))
            count.append(k)
        s["path"], s["count"] = _ints(path), _ints(count)
        s["new_lens"] = torch.empty_like(s["lens"])
        if own:
            import block_scaled_precision_act_amd as mx
            s["handles"] = [mx.MxKvCacheFp4(*(t[i] for t in s["cache"])) for i in range(layers)]
    return s


# ---------------------------------------------------------------------------------- plain forms

def _tree_mask(s):
    c, starts, parents = s["case"], s["starts"].long(), s["parents"].long()
    n, total = c["n"], s["parents"].shape[0]
    node = torch.arange(total, device="cuda")
    seq = torch.searchsorted(starts, node, right=True) - 1
    local = node - starts[seq]
    up = torch.where((parents >= 0) & (parents < local), parents, -1)
    seen = torch.zeros((total, n), dtype=torch.bool, device="cuda")
    at = local
    for _ in range(n):                      # all nodes step to their parents together
        seen[node, at.clamp_min(0)] |= at >= 0
        at = torch.where(at >= 0, up[(starts[seq] + at).clamp_min(0)], -1)
    first = s["lens"].long() - (starts[1:] - starts[:-1])
    return _words(seen), (first[seq] + seen.sum(-1) - 1).to(torch.int32)


def _values(codes, scales):
    """What packed codes [..., D / 2] and E8M0 bytes [..., D / 32] stand for, fp32 [..., D]."""
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    v = torch.stack([t[(codes & 15).int()], t[(codes >> 4).int()]], -1).flatten(-2)
    e = (scales.int() << 23).view(torch.float32)
    return (v.unflatten(-1, (-1, 32)) * e[..., None]).flatten(-2)


def _attention(s):
    c, q = s["case"], s["q"].float()
    B, n, hk, D = c["B"], c["n"], c["hk"], c["D"]
    G = c["hq"] // hk
    lens, starts, table = s["lens"].long(), s["starts"].long(), s["table"].long()
    k, ks, v, vs = (t[table].transpose(1, 2).flatten(2, 3) for t in s["cache"])   # [B, hk, L, .]
    k, v = _values(k, ks), _values(v, vs)
    at = (starts[:-1, None] + torch.arange(n, device="cuda")).clamp_max(q.shape[0] - 1)    # [B, n]
    rows = q[at].view(B, n, hk, G, D).permute(0, 2, 3, 1, 4)
    sc = rows.reshape(B, hk, G * n, D) @ k.transpose(-1, -2)
    sc = sc.view(B, hk, G, n, -1) * (1 / math.sqrt(D))
    t = torch.arange(sc.shape[-1], device="cuda")
    first = lens - (starts[1:] - starts[:-1])
    past = (t < first[:, None])[:, None].expand(B, n, -1)
    if c["window"]:
        past = past & (t > s["pos"][at][..., None] - c["window"])
    bits = ((s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).flatten(1)
    inside = t - first[:, None]                                                   # [B, L]
    tree = bits[at].gather(2, inside.clamp(0, bits.shape[1] - 1)[:, None].expand(B, n, -1)) != 0
    seen = past | (tree & ((inside >= 0) & (t < lens[:, None]))[:, None])
    sc = sc.masked_fill(~seen.view(B, 1, 1, n, -1), -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.masked_fill(m == -math.inf, 0))
    total = p.sum(-1, keepdim=True)
    o = (p / total.masked_fill(total == 0, 1)).view(B, hk, G * n, -1) @ v
    o = o.view(B, hk, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, hk * G, D)
    tok = torch.arange(q.shape[0], device="cuda")
    seq = torch.searchsorted(starts, tok, right=True) - 1
    o = o[seq, tok - starts[seq]].to(torch.bfloat16)
    if not c["lse"]:
        return o
    lse = (m + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, n, hk * G)
    return o, lse[seq, tok - starts[seq]]


def _weights(rows):
    """Probabilities in 64 bits; what is none (negative, infinite, not a number) counts as 0."""
    r = rows.double()
    return r.masked_fill(~((r > 0) & (r < math.inf)), 0)


def _verified(s):
    """All sequences at once, node by node: a node is looked at when its parent has been accepted."""
    c, target, draft = s["case"], s["target"], s["draft"]
    B, n, V = c["B"], c["n"], c["V"]
    total = target.shape[0]
    starts, parents, tokens = s["starts"].long(), s["parents"].long(), s["tokens"].long()
    base, size = starts[:-1], starts[1:] - starts[:-1]
    seqs = torch.arange(B, device="cuda")
    f8 = dict(dtype=torch.float64, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    factor, left, mass = torch.zeros(B, **f8), torch.ones(B, **f8), torch.ones(B, **f8)
    gone = torch.zeros((B, V), dtype=torch.bool, device="cuda")          # rejected, of chosen drafts
    path, new = (torch.full((B, n), -1, dtype=torch.long, device="cuda") for _ in range(2))
    path[:, 0] = torch.where(size > 0, 0, -1)
    count = (size > 0).long()
    for i in range(1, n):
        row, at = (base + i).clamp_max(total - 1), (base + cur).clamp_max(total - 1)
        mine = (i < size) & (parents[row] == cur)
        x, u = tokens[row], s["accept_u"][row].double()
        real = (x >= 0) & (x < V)
        x = x.clamp(0, V - 1)
        p = _weights(target[at, x]) * real
        if draft is None:
            w = p.masked_fill(gone[seqs, x], 0)
            ok = mine & (w > 0) & (u * left < w)
            no = mine & ~ok
            left = torch.where(no, (left - w).clamp_min(0), left)
            gone[seqs, x] |= no & real
        else:
            q = _weights(draft[at, x]) * real
            w = (p - factor * q).clamp_min(0)
            ok = mine & (mass > 0) & (w > 0) & (u * q * left < w * mass)
            no = mine & ~ok & (mass > 0)
            factor = torch.where(no, factor + left / mass, factor)
            if c["draft"] == "distinct":
                mass = torch.where(no, mass - q, mass)
            rest = (_weights(target[at]) - factor[:, None] * _weights(draft[at])).clamp_min(0).sum(-1)
            left = torch.where(no, rest, left)
        place = count.clamp_max(n - 1)
        path[seqs, place] = torch.where(ok, i, path[seqs, place])
        place = (count - 1).clamp_min(0)
        new[seqs, place] = torch.where(ok, x, new[seqs, place])
        count = count + ok
        cur = torch.where(ok, i, cur)
        factor = factor.masked_fill(ok, 0)
        left, mass = left.masked_fill(ok, 1), mass.masked_fill(ok, 1)
        gone &= ~ok[:, None]
    at = (base + cur).clamp_max(total - 1)
    p = _weights(target[at])
    rest = p.masked_fill(gone, 0) if draft is None else \
        (p - factor[:, None] * _weights(draft[at])).clamp_min(0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p)
    upto = rest.cumsum(-1)
    t = s["sample_u"].double() * upto[:, -1]
    token = (upto <= t[:, None]).sum(-1)
    last = ((rest > 0) * torch.arange(V, device="cuda")).amax(-1)
    token = torch.where(token < V, token, last)
    token = torch.where(rest.sum(-1) > 0, token, -1)
    place = (count - 1).clamp_min(0)
    new[seqs, place] = torch.where(size > 0, token, new[seqs, place])
    return path.to(torch.int32), new.to(torch.int32), count.to(torch.int32)


def _accepted(s):
    c, page, path = s["case"], s["case"]["page"], s["path"].long()
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(path.shape[1], device="cuda")
    kept = (i < s["count"].long()[:, None]) & (path >= 0)
    src, dst = (first[:, None] + torch.where(kept, x, 0) for x in (path, i))     # else: the root, to itself
    table = s["table"].long()
    at, to = table.gather(1, src // page), table.gather(1, dst // page)
    for t in s["cache"]:
        t[:, to, :, dst % page] = t[:, at, :, src % page]
    s["new_lens"].copy_(first + s["count"])
    return s["cache"], s["new_lens"]


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _run_own(s)
    return {"mask": _tree_mask, "attn": _attention, "verify": _verified, "accept": _accepted}[op](s)


def _run_own(s):
    import block_scaled_precision_act_amd as mx
    c = s["case"]
    if c["op"] == "mask":
        mx.mx_tree_mask(s["parents"], s["mask"], seq_lens=s["lens"], positions=s["pos"],
                        q_starts=s["starts"], max_q=c["n"])
        return s["mask"], s["pos"]
    if c["op"] == "attn":
        mx.mx_attn_tree_fp4(s["handle"], s["q"], s["mask"], s["table"], s["lens"], s["out"], s["ws"],
                            q_starts=s["starts"], max_q=c["n"], window=c["window"],
                            positions=s["pos"] if c["window"] else None, lse=s["lse"])
        return (s["out"], s["lse"]) if c["lse"] else s["out"]
    if c["op"] == "verify":
        mx.mx_tree_verify(s["target"], s["draft"], s["tokens"], s["parents"], s["accept_u"],
                          s["sample_u"], s["path"], s["new"], s["count"], s["ws"],
                          q_starts=s["starts"], max_q=c["n"], replacement=c["draft"] == "drawn")
        return s["path"], s["new"], s["count"]
    mx.mx_kv_accept_fp4(s["handles"], s["table"], s["lens"], s["path"], s["count"],
                        lens_out=s["new_lens"], q_starts=s["starts"], max_q=c["n"])
    return s["cache"], s["new_lens"]


# --------------------------------------------------------------------------------- what it takes

def work(case):
    c = case
    lens, news = _lens(c)
    total = sum(news)
    if c["op"] == "mask":
        return {"bytes": total * (8 + 4 * -(-c["n"] // 32)) + 8 * c["B"], "flops": total}
    if c["op"] == "attn":
        tokens = pairs = 0
        for L, n in zip(lens, news):
            past = max(0, L - n)
            if c["window"]:
                past = min(past, c["window"] - 1)
            tokens += min(L, past + n)
            pairs += n * past + n                    # of the tree a node sees itself at least
        row = 2 * c["hk"] * (c["D"] // 2 + c["D"] // 32)
        return {"bytes": tokens * row + 4 * total * c["hq"] * c["D"], "flops": 4 * pairs * c["hq"] * c["D"]}
    if c["op"] == "verify":
        # one row of each a sequence: what the last token is drawn from
        rows = 1 if c["draft"] == "chosen" else 2
        width = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": c["B"] * c["V"] * width * rows + total * (12 + 2 * width) + c["B"] * (8 + 8 * c["n"]),
                "flops": 4 * c["B"] * c["V"]}
    moved = sum(max(0, min(4, (n + 1) // 2) - 1) for n in news)      # four of a path on the mean
    return {"bytes": 2 * moved * c["layers"] * c["h"] * 2 * (c["D"] // 2 + c["D"] // 32) + 12 * c["B"],
            "flops": 0}


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definitions, sequence by sequence and node by node, in float64."""
    c, s = case, prepare(case, seed)
    lens, news = _lens(c)
    return {"mask": _exact_mask, "attn": _exact_attn, "verify": _exact_verify,
            "accept": _exact_accept}[c["op"]](c, s, lens, news)


def _exact_mask(c, s, lens, news):
    parents, at, masks, places = s["parents"].tolist(), 0, [], []
    width = -(-c["n"] // 32)
    for L, n in zip(lens, news):
        sets = []
        for i, up in enumerate(parents[at:at + n]):
            sets.append({i} | (sets[up] if 0 <= up < i else set()))
            whole = sum(1 << j for j in sets[i])
            masks.append(np.array([(whole >> (32 * w)) & 0xFFFFFFFF for w in range(width)], np.uint32))
            places.append(L - n + len(sets[i]) - 1)
        at += n
    return torch.from_numpy(np.stack(masks).view(np.int32)).cuda(), _ints(places)


def _exact_attn(c, s, lens, news):
    D, hk, page = c["D"], c["hk"], c["page"]
    G, at, outs, sums = c["hq"] // hk, 0, [], []
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device="cuda", dtype=torch.float64) / 2
    words = s["mask"].cpu().numpy().view(np.uint32)
    for b, (L, n) in enumerate(zip(lens, news)):
        mine = s["table"][b, :-(-L // page)].long()
        kv = []
        for codes, bytes_ in ((s["cache"][0], s["cache"][1]), (s["cache"][2], s["cache"][3])):
            raw = codes[mine].movedim(1, 0).reshape(hk, -1, D // 2)[:, :L].long()
            nib = torch.empty((hk, L, D), dtype=torch.int64, device="cuda")
            nib[..., 0::2], nib[..., 1::2] = raw % 16, raw // 16
            e = bytes_[mine].movedim(1, 0).reshape(hk, -1, D // 32)[:, :L].long() - 127
            val = half[nib % 8] * (1 - 2 * (nib // 8))
            kv.append(torch.ldexp(val, e.repeat_interleave(32, -1)))
        hide = np.zeros((n, L), bool)
        place = s["pos"][at:at + n].tolist()
        for i in range(n):
            if c["window"]:
                hide[i, :max(0, min(L - n, place[i] - c["window"] + 1))] = True
            for j in range(max(0, n - L), n):
                hide[i, L - n + j] = not words[at + i, j // 32] >> (j % 32) & 1
        q = s["q"][at:at + n].double().view(n, hk, G, D).permute(1, 2, 0, 3)
        at += n
        z = torch.matmul(q.reshape(hk, G * n, D), kv[0].mT).view(hk, G, n, L) / math.sqrt(D)
        z = z.masked_fill(torch.from_numpy(hide).cuda(), -math.inf)
        lse = torch.logsumexp(z, -1)
        z = torch.exp(z - lse.masked_fill(lse == -math.inf, 0)[..., None])
        o = torch.matmul(z.view(hk, G * n, L), kv[1]).view(hk, G, n, D)
        outs.append(o.permute(2, 0, 1, 3).reshape(n, c["hq"], D))
        sums.append(lse.permute(2, 0, 1).reshape(n, c["hq"]))
    o = torch.cat(outs)
    return (o, torch.cat(sums)) if c["lse"] else o


def _exact_verify(c, s, lens, news):
    """With the distributions themselves: what is left of the target's after a rejection is
    normalised, and so is the draft's after a drawn token has left it."""
    n, V = c["n"], c["V"]
    tokens, parents = s["tokens"].tolist(), s["parents"].tolist()
    u = s["accept_u"].double().tolist()
    path, new, count = np.full((c["B"], n), -1), np.full((c["B"], n), -1), np.zeros(c["B"], int)

    def row(m, i):
        return m[i].double().cpu().numpy()

    base = 0
    for b, size in enumerate(news):
        here, steps, said = 0, [0], []
        while True:
            r, scale = row(s["target"], base + here), None
            q = None if s["draft"] is None else row(s["draft"], base + here)
            step = None
            for i in range(here + 1, size):
                if parents[base + i] != here:
                    continue
                x = tokens[base + i]
                chance = r[x] if scale is None else r[x] / scale
                if r[x] > 0 and u[base + i] * (1.0 if q is None else q[x]) < chance:
                    step = i
                    break
                if q is None:
                    r[x] = 0.0
                    scale = (1.0 if scale is None else scale) - chance * (1.0 if scale is None else scale)
                else:
                    r = np.maximum((r if scale is None else r / scale) - q, 0.0)
                    scale = r.sum()
                    if c["draft"] == "distinct":
                        q = q / (1.0 - q[x])
                        q[x] = 0.0
            if step is None:
                break
            here = step
            steps.append(step)
            said.append(tokens[base + step])
        upto = np.cumsum(r)
        said.append(int(np.searchsorted(upto, s["sample_u"][b].double().item() * upto[-1], side="right")))
        path[b, :len(steps)], new[b, :len(said)], count[b] = steps, said, len(steps)
        base += size
    return _ints(path), _ints(new), _ints(count)


def _exact_accept(c, s, lens, news):
    page, path, count = c["page"], s["path"].tolist(), s["count"].tolist()
    table, after = s["table"].tolist(), [t.clone() for t in s["cache"]]
    for b, (L, n) in enumerate(zip(lens, news)):
        for i in range(count[b]):
            (p0, t0), (p1, t1) = divmod(L - n + path[b][i], page), divmod(L - n + i, page)
            for old, t in zip(s["cache"], after):
                t[:, table[b][p1], :, t1] = old[:, table[b][p0], :, t0]
    return after, _ints([L - n + k for L, n, k in zip(lens, news, count)])
