"""The attention operators around a paged MXFP4 key/value cache, as cases that can be measured.

Four operators: the per-head norm of queries and keys with the position rotation in the same pass
("norm_rope"), its gradients ("norm_rope_back"), appending keys and values to the 4-bit cache with
the rotation applied on the way ("append"), and attention over that cache ("attn").

`own` False runs their plain forms in elementary torch operations (fp32, one rounding at the end);
`own` True makes the calls a user of block_scaled_precision_act_amd makes.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0


# ---------------------------------------------------------------------------------------- cases

def _norm(name, op, T, hq, hk, D, rot, inter, norm):
    return dict(name=name, op=op, T=T, hq=hq, hk=hk, D=D, rot=rot, inter=inter, norm=norm)


def _append(name, T, h, D, rot, inter, page):
    return dict(name=name, op="append", T=T, h=h, D=D, rot=rot, inter=inter, page=page)


def _attn(name, B, nq, L, lmin, hq, hk, D, page, causal=True, window=0, ragged=False, lse=False):
    return dict(name=name, op="attn", B=B, nq=nq, L=L, lmin=lmin, hq=hq, hk=hk, D=D, page=page,
                causal=causal, window=window, ragged=ragged, lse=lse)


def listed():
    return [
        # one new token of one sequence: what a chat reply pays per layer, all latency
        _norm("norm_rope_token", "norm_rope", 1, 32, 8, 128, 128, False, True),
        # a prompt of 16384 tokens, queries and keys of one layer
        _norm("norm_rope_prompt", "norm_rope", 16384, 32, 8, 128, 128, False, True),
        # training on an odd number of tokens, pairs side by side, half of the head rotated
        _norm("norm_rope_back_odd", "norm_rope_back", 4099, 12, 12, 64, 32, True, True),
        # a training step's microbatch
        _norm("norm_rope_back_train", "norm_rope_back", 16384, 32, 8, 128, 128, False, True),
        # one new token for each of 41 sequences (the A4W4 decode shapes' M; 4608 = 3 * 12 * 128)
        _append("append_41_tokens", 41, 12, 128, 128, False, 16),
        # a prompt of 16384 tokens into the cache
        _append("append_prompt", 16384, 8, 128, 128, False, 64),
        # one token of one short sequence: latency
        _attn("attn_token_short", 1, 1, 1000, 1000, 32, 8, 128, 16),
        # one token for each of 41 sequences of very different lengths, an odd group of heads
        _attn("attn_tokens_ragged", 41, 1, 8192, 1, 56, 8, 128, 16),
        # long contexts, one token each: the cache is read once
        _attn("attn_tokens_long", 4, 1, 131073, 120001, 32, 8, 128, 64),
        # a few drafted tokens checked at once, a window of the past, heads of 64, no shared heads
        _attn("attn_draft_window", 32, 4, 6144, 1536, 12, 12, 64, 32, window=4096),
        # a chunk of a long prompt against what is cached already, heads of 256
        _attn("attn_chunk", 2, 512, 32768, 20000, 16, 2, 256, 64, ragged=True, lse=True),
        # a whole prompt
        _attn("attn_prompt", 1, 8192, 8192, 8192, 32, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    D = rng.choice((64, 128, 128, 256))
    rot = rng.choice((D, D, D // 2))
    inter = rng.random() < 0.3
    hk = rng.choice((1, 2, 4, 8, 12))
    hq = hk * rng.choice((1, 2, 4, 5, 7, 8, 16))
    page = rng.choice((16, 32, 48, 64, 128))
    op = rng.choice(("norm_rope", "norm_rope_back", "append", "attn", "attn", "attn"))
    if op.startswith("norm"):
        T = _log(rng, 1, max(1, 16384 * 40 * 128 // ((hq + hk) * D)))
        c = _norm("", op, T, hq, hk, D, rot, inter, rng.random() < 0.8)
    elif op == "append":
        c = _append("", _log(rng, 1, 16384 * 8 * 128 // (hk * D)), hk, D, rot, inter, page)
    else:
        kind = rng.choice(("tokens", "tokens", "chunk", "prompt"))
        cache = 4 * 131073 * 8 * 128 // (hk * D)            # cached tokens of the largest case
        pairs = 8192 * 8192 * 32 * 128 // (hq * D) // 2     # (query, key) pairs of the largest case
        window = _log(rng, 16, 4096) if rng.random() < 0.25 else 0
        if kind == "tokens":
            nq, B = rng.choice((1, 1, 1, 2, 3, 4)), _log(rng, 1, 128)
        elif kind == "chunk":
            nq, B = _log(rng, 5, 1024), _log(rng, 1, 8)
        else:
            nq, B = _log(rng, 16, min(4096, math.isqrt(pairs))), rng.choice((1, 1, 2, 3))
        most = max(nq, min(131073, cache // B, pairs // (B * nq)))
        L = nq if kind == "prompt" else _log(rng, nq, most)
        if B * nq * L > pairs:
            B = 1
        lmin = L if rng.random() < 0.4 else _log(rng, 1, L)
        c = _attn("", B, nq, L, lmin, hq, hk, D, page, causal=window > 0 or rng.random() < 0.85,
                  window=window, ragged=B > 1 and nq > 1 and rng.random() < 0.5,
                  lse=rng.random() < 0.3)
    del c["name"]
    return c


def _lens(c):
    """(cached tokens, new tokens among them) of each sequence of an attention case."""
    lens, news = [], []
    for i in range(c["B"]):
        u, w = (i * 0.6180339887) % 1.0, (i * 0.7548776662) % 1.0
        lens.append(c["L"] if i == 0 else c["lmin"] + int((c["L"] - c["lmin"]) * u))
        news.append(1 + int((c["nq"] - 1) * w) if c["ragged"] and i else c["nq"])
    return lens, news


# --------------------------------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _tables(P, rot):
    f = THETA ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * f
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, D = case, case["D"]
    s = {"case": c}
    if c["op"].startswith("norm"):
        T, hq, hk = c["T"], c["hq"], c["hk"]
        # queries, keys (and values) side by side, as a projection of [T, hidden] leaves them
        qkv = (_randn(g, T, (hq + 2 * hk) * D) * 1.7).to(torch.bfloat16)
        s["q"] = qkv[:, :hq * D].view(T, hq, D)
        s["k"] = qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
        s["cos"], s["sin"] = _tables(max(T, 4096), c["rot"])
        s["pos"] = (torch.arange(T, device="cuda") + (4096 - T if T < 64 else 0)).to(torch.int32)
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"] = (1 + 0.2 * _randn(g, D)).to(torch.bfloat16)
            s["kw"] = (1 + 0.2 * _randn(g, D)).to(torch.bfloat16)
        if c["op"] == "norm_rope":
            s["out"] = [torch.empty((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, hk)]
        else:
            s["dq"] = (0.01 * _randn(g, T, hq, D)).to(torch.bfloat16)
            s["dk"] = (0.01 * _randn(g, T, hk, D)).to(torch.bfloat16)
            s["grad"] = [torch.empty((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, hk)]
            s["dw"] = [torch.empty(D, device="cuda") if c["norm"] else None for _ in "qk"]
            if own:
                import block_scaled_precision_act_amd as mx
                n = mx.mx_qk_norm_rope_backward_workspace_size(T, hq, hk, D)
                s["ws"] = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")
        return s
    h, page = (c["h"], c["page"]) if c["op"] == "append" else (c["hk"], c["page"])
    if c["op"] == "append":
        T = c["T"]
        pages = -(-T // page) + 3
        chan = torch.exp(0.5 * _randn(g, h, D))
        kv = torch.cat([_randn(g, T, h, D) * chan, _randn(g, T, h, D) + 0.3 * chan], 1)
        kv = kv.to(torch.bfloat16)
        s["k"], s["v"] = kv[:, :h], kv[:, h:]
        s["cos"], s["sin"] = _tables(max(T, 4096), c["rot"])
        s["pos"] = (torch.arange(T, device="cuda") + (4096 - T if T < 64 else 0)).to(torch.int32)
        if T < 64:          # a token of each sequence: slots anywhere
            s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
        else:               # a prompt: page after page, the pages in any order
            order = torch.randperm(pages, generator=g, device="cuda")
            t = torch.arange(T, device="cuda")
            s["slots"] = order[t // page] * page + t % page
        s["cache"] = [torch.zeros((pages, h, page, D // n), dtype=torch.uint8, device="cuda")
                      for n in (2, 32, 2, 32)]
        s["out"] = [torch.empty((T, h, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    else:
        lens, news = _lens(c)
        counts = [-(-n // page) for n in lens]
        pages, width = sum(counts) + 2, max(counts)
        order = torch.randperm(pages, generator=g, device="cuda").tolist()
        table, at = [], 0
        for n in counts:
            table.append(order[at:at + n] + [0] * (width - n))
            at += n
        s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = [0]
        for n in news:
            starts.append(starts[-1] + n)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        chan = torch.exp(0.5 * _randn(g, h, 1, D))
        s["cache"] = [*_quantise(_randn(g, pages, h, page, D) * chan),
                      *_quantise(_randn(g, pages, h, page, D) + 0.3 * chan)]
        s["q"] = _randn(g, starts[-1], c["hq"], D).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((starts[-1], c["hq"]), device="cuda") if c["lse"] else None
        if own:
            import block_scaled_precision_act_amd as mx
            n = mx.mx_attn_fp4_workspace_size(c["B"], c["nq"], c["hq"], c["hk"], D)
            s["ws"] = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")
    if own:
        import block_scaled_precision_act_amd as mx
        s["handle"] = mx.MxKvCacheFp4(*s["cache"])
    return s


# ---------------------------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, rot, inter):
    """Rotates the first `rot` of each head of x [T, H, D] by cos, sin [T, rot / 2]."""
    c, s = cos[:, None], sin[:, None]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


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


def _values(codes, scales):
    """What packed codes [..., D / 2] and E8M0 bytes [..., D / 32] stand for, fp32 [..., D]."""
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                     device=codes.device)
    v = torch.stack([t[(codes & 15).int()], t[(codes >> 4).int()]], -1).flatten(-2)
    s = (scales.int() << 23).view(torch.float32)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _norm_rope(x, w, cos, sin, rot, inter):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(x, cos, sin, rot, inter).to(torch.bfloat16)


def _norm_rope_back(dy, x, w, cos, sin, rot, inter):
    dn, x = _rotate(dy.float(), cos, -sin, rot, inter), x.float()
    if w is None:
        return dn.to(torch.bfloat16), None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dw = (dn * x * r).sum((0, 1))
    gr = dn * w.float()
    dx = r * (gr - x * (r * r * (gr * x).mean(-1, keepdim=True)))
    return dx.to(torch.bfloat16), dw


def _attention(s):
    c, q = s["case"], s["q"].float()
    B, nq, hk, D = c["B"], c["nq"], c["hk"], c["D"]
    G = c["hq"] // hk
    lens, starts, table = s["lens"].long(), s["starts"].long(), s["table"].long()
    k, ks, v, vs = (t[table].transpose(1, 2).flatten(2, 3) for t in s["cache"])   # [B, hk, L, .]
    k, v = _values(k, ks), _values(v, vs)
    at = starts[:-1, None] + torch.arange(nq, device="cuda")
    rows = q[at.clamp_max(q.shape[0] - 1)].view(B, nq, hk, G, D).permute(0, 2, 3, 1, 4)
    sc = rows.reshape(B, hk, G * nq, D) @ k.transpose(-1, -2)
    sc = sc.view(B, hk, G, nq, -1) * (1 / math.sqrt(D))
    t = torch.arange(sc.shape[-1], device="cuda")
    place = (lens - (starts[1:] - starts[:-1]))[:, None] + torch.arange(nq, device="cuda")
    seen = (t < lens[:, None]).view(B, 1, -1).expand(B, nq, -1)
    if c["causal"]:
        seen = seen & (t <= place[..., None])
    if c["window"]:
        seen = seen & (t > place[..., None] - c["window"])
    sc = sc.masked_fill(~seen.view(B, 1, 1, nq, -1), -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.masked_fill(m == -math.inf, 0))
    total = p.sum(-1, keepdim=True)
    o = (p / total.masked_fill(total == 0, 1)).view(B, hk, G * nq, -1) @ v
    o = o.view(B, hk, G, nq, D).permute(0, 3, 1, 2, 4).reshape(B, nq, hk * G, D)
    tok = torch.arange(q.shape[0], device="cuda")
    seq = torch.searchsorted(starts, tok, right=True) - 1
    o = o[seq, tok - starts[seq]].to(torch.bfloat16)
    if not c["lse"]:
        return o
    lse = (m + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, nq, hk * G)
    return o, lse[seq, tok - starts[seq]]


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s)
    if c["op"] == "attn":
        return _attention(s)
    cos, sin = s["cos"][s["pos"].long()], s["sin"][s["pos"].long()]
    how = (cos, sin, c["rot"], c["inter"])
    if c["op"] == "norm_rope":
        return [_norm_rope(s["q"], s["qw"], *how), _norm_rope(s["k"], s["kw"], *how)]
    if c["op"] == "norm_rope_back":
        dq, dqw = _norm_rope_back(s["dq"], s["q"], s["qw"], *how)
        dk, dkw = _norm_rope_back(s["dk"], s["k"], s["kw"], *how)
        return [dq, dk] + ([dqw, dkw] if c["norm"] else [])
    kc, ks = _quantise(_rotate(s["k"].float(), *how))
    vc, vs = _quantise(s["v"].float())
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    for cache, new in zip(s["cache"], (kc, ks, vc, vs)):
        cache[page, :, off] = new
    return {"cache": s["cache"], "k": _values(kc, ks).to(torch.bfloat16),
            "v": _values(vc, vs).to(torch.bfloat16)}


def _run_own(s):
    import block_scaled_precision_act_amd as mx
    c = s["case"]
    if c["op"] == "attn":
        mx.mx_attn_fp4(s["handle"], s["q"], s["table"], s["lens"], s["out"], s["ws"],
                       q_starts=s["starts"], max_q=c["nq"], causal=c["causal"],
                       window=c["window"], lse=s["lse"])
        return (s["out"], s["lse"]) if c["lse"] else s["out"]
    if c["op"] == "append":
        mx.mx_kv_append_fp4(s["handle"], s["k"], s["v"], s["slots"], s["pos"], s["cos"], s["sin"],
                            k_out=s["out"][0], v_out=s["out"][1], interleaved=c["inter"])
        return {"cache": s["cache"], "k": s["out"][0], "v": s["out"][1]}
    if c["op"] == "norm_rope":
        mx.mx_qk_norm_rope(s["q"], s["k"], s["pos"], s["cos"], s["sin"], *s["out"], s["qw"], s["kw"],
                           eps=EPS, interleaved=c["inter"])
        return s["out"]
    mx.mx_qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["cos"], s["sin"],
                                *s["grad"], s["qw"], s["kw"], *s["dw"], s["ws"], eps=EPS,
                                interleaved=c["inter"])
    return s["grad"] + (s["dw"] if c["norm"] else [])


# --------------------------------------------------------------------------------- what it takes

def work(case):
    c, D = case, case["D"]
    if c["op"].startswith("norm"):
        n = c["T"] * (c["hq"] + c["hk"]) * D
        table = c["T"] * (c["rot"] * 4 + 4)
        if c["op"] == "norm_rope":
            return {"bytes": 4 * n + table, "flops": 8 * n}
        return {"bytes": 6 * n + table, "flops": 16 * n}
    if c["op"] == "append":
        n = c["T"] * c["h"] * D
        return {"bytes": 4 * n + 2 * n * (1 / 2 + 1 / 32) + 4 * n + c["T"] * (c["rot"] * 4 + 12),
                "flops": 10 * n}
    tokens = pairs = new = 0
    for L, n in zip(*_lens(c)):
        first = L - n                                   # the first new token's place
        lo = max(0, first + 1 - c["window"]) if c["window"] else 0
        tokens += max(0, L - lo)
        new += n
        for i in range(n):
            hi = min(L, first + i + 1) if c["causal"] else L
            pairs += max(0, hi - (max(0, first + i + 1 - c["window"]) if c["window"] else 0))
    return {"bytes": 2 * tokens * c["hk"] * (D // 2 + D // 32) + 4 * new * c["hq"] * D,
            "flops": 4 * pairs * c["hq"] * D}


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definitions in float64, sequence by sequence and rotation by complex numbers."""
    c, s, f8 = case, prepare(case, seed), torch.float64

    def turn(x, sign=1):
        rot, p = c["rot"], s["pos"].long()
        z = torch.complex(s["cos"][p].to(f8), sign * s["sin"][p].to(f8))[:, None]
        head, rest = x[..., :rot], x[..., rot:]
        if c["inter"]:
            y = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * z)
            y = y.flatten(-2)
        else:
            y = torch.complex(*(t.contiguous() for t in head.chunk(2, -1))) * z
            y = torch.cat([y.real, y.imag], -1)
        return torch.cat([y, rest], -1)

    def four_bits(x):
        b = x.unflatten(-1, (-1, 32))
        top = b.abs().amax(-1, keepdim=True).clamp_min(float(torch.tensor(1e-4)))
        m, e = torch.frexp(top / 6)                     # top / 6 = m 2^e with m in [1/2, 1)
        e = e - (m == 0.5).to(e.dtype)
        y = torch.ldexp(b, -e)
        step = 0.5 + 0.5 * (y.abs() >= 2) + (y.abs() >= 4)
        return torch.ldexp(torch.round(y / step) * step, e).flatten(-2)

    if c["op"] == "norm_rope":
        res = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.to(f8)
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(f8)
            res.append(turn(x))
        return res
    if c["op"] == "norm_rope_back":
        grads, weights = [], []
        for x, w, dy in ((s["q"], s["qw"], s["dq"]), (s["k"], s["kw"], s["dk"])):
            x, dn = x.to(f8), turn(dy.to(f8), -1)
            if w is None:
                grads.append(dn)
                continue
            size = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
            unit = x / size                             # dx = (g - unit <g, unit> / D) / size
            weights.append((dn * unit).sum(0).sum(0))
            gw = dn * w.to(f8)
            grads.append((gw - unit * (gw * unit).mean(-1, keepdim=True)) / size)
        return grads + weights
    if c["op"] == "append":
        return {"cache": [None] * 4, "k": four_bits(turn(s["k"].to(f8))),
                "v": four_bits(s["v"].to(f8))}
    lens, news = _lens(c)
    D, hk, page = c["D"], c["hk"], c["page"]
    G, at, outs, sums = c["hq"] // hk, 0, [], []
    table = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device="cuda", dtype=f8) / 2
    for b, (L, n) in enumerate(zip(lens, news)):
        own_pages = s["table"][b, :-(-L // page)].long()
        kv = []
        for codes, bytes_ in ((s["cache"][0], s["cache"][1]), (s["cache"][2], s["cache"][3])):
            raw = codes[own_pages].movedim(1, 0).reshape(hk, -1, D // 2)[:, :L].long()
            nib = torch.empty((hk, L, D), dtype=torch.int64, device="cuda")
            nib[..., 0::2], nib[..., 1::2] = raw % 16, raw // 16
            e = bytes_[own_pages].movedim(1, 0).reshape(hk, -1, D // 32)[:, :L].long() - 127
            val = table[nib % 8] * (1 - 2 * (nib // 8))
            kv.append(torch.ldexp(val, e.repeat_interleave(32, -1)))
        q = s["q"][at:at + n].to(f8).view(n, hk, G, D).permute(1, 2, 0, 3)
        at += n
        z = torch.matmul(q.reshape(hk, G * n, D), kv[0].mT).view(hk, G, n, L) / math.sqrt(D)
        key = torch.arange(L, device="cuda")[None]
        p = torch.arange(L - n, L, device="cuda")[:, None]
        hide = torch.zeros((n, L), dtype=torch.bool, device="cuda")
        if c["causal"]:
            hide |= key > p
        if c["window"]:
            hide |= key <= p - c["window"]
        z = z.masked_fill(hide, -math.inf)
        lse = torch.logsumexp(z, -1)
        z = torch.exp(z - lse.masked_fill(lse == -math.inf, 0)[..., None])
        o = torch.matmul(z.view(hk, G * n, L), kv[1]).view(hk, G, n, D)
        outs.append(o.permute(2, 0, 1, 3).reshape(n, c["hq"], D))
        sums.append(lse.permute(2, 0, 1).reshape(n, c["hq"]))
    o = torch.cat(outs)
    return (o, torch.cat(sums)) if c["lse"] else o
