"""Float64 oracle of the draft operators, from their definitions, node by node.  It shares nothing with
the HIP path: verification is written with the normalised distributions themselves, where the kernel
keeps what is left of the target's in one factor."""
import numpy as np

from .attention_oracle import cache_rows


def ancestors(parents):
    """For each node the set of itself and its ancestors."""
    sets = []
    for i, up in enumerate(parents):
        sets.append({i} | (sets[up] if 0 <= up < i else set()))
    return sets


def tree_mask(parents, starts, words, lens=None):
    """int32 mask [nodes, words], int32 positions [nodes] (or None)."""
    N = len(parents)
    mask, pos = np.zeros((N, words), np.uint32), np.zeros(N, np.int32)
    for b in range(len(starts) - 1):
        q0, q1 = starts[b], starts[b + 1]
        for i, s in enumerate(ancestors(parents[q0:q1])):
            for j in s:
                mask[q0 + i, j // 32] |= np.uint32(1 << (j % 32))
            if lens is not None:
                pos[q0 + i] = lens[b] - (q1 - q0) + len(s) - 1
    return mask.view(np.int32), pos if lens is not None else None


def attention(q, k_codes, k_scales, v_codes, v_scales, page_table, seq_lens, starts, scale, mask,
              window=0, positions=None):
    """out, lse, the weighted mean of |v| and the largest scale * sum |q k| of each row, as
    attention_oracle.attention gives them, for queries whose view of each other `mask` says."""
    N, hq, D = q.shape
    q, words = np.asarray(q, np.float64), np.asarray(mask).view(np.uint32)
    hk = k_codes.shape[1]
    out, lse = np.zeros((N, hq, D)), np.full((N, hq), -np.inf)
    mag, top = np.zeros((N, hq, D)), np.zeros((N, hq))
    for b, L in enumerate(seq_lens):
        k = cache_rows(k_codes, k_scales, page_table[b], L)
        v = cache_rows(v_codes, v_scales, page_table[b], L)
        n = starts[b + 1] - starts[b]
        for i in range(n):
            row, seen = starts[b] + i, np.zeros(L, bool)
            for t in range(L):
                j = t - (L - n)
                seen[t] = words[row, j // 32] >> (j % 32) & 1 if j >= 0 else \
                    not window or t > min(max(positions[row], L - n), L - 1) - window
            if not seen.any():
                continue
            for h in range(hq):
                kk, vv = k[h // (hq // hk), seen], v[h // (hq // hk), seen]
                s = scale * (kk @ q[row, h])
                m = s.max()
                p = np.exp(s - m)
                out[row, h] = p @ vv / p.sum()
                mag[row, h] = p @ np.abs(vv) / p.sum()
                lse[row, h] = m + np.log(p.sum())
                top[row, h] = abs(scale) * (np.abs(kk) @ np.abs(q[row, h])).max()
    return out, lse, mag, top


def _clean(row):
    row = np.asarray(row, np.float64)
    return np.where((row > 0) & np.isfinite(row), row, 0.0)


def verify_one(target, draft, tokens, parents, accept_u, sample_u, width, replacement):
    """Path and emitted tokens of one sequence; target and draft fp64 [n, V] (draft None: chosen)."""
    n = len(parents)
    if n == 0:
        return [], []
    V = target.shape[1]
    here, path, said = 0, [0], []
    while True:
        p = _clean(target[here])
        r, whole = p.copy(), True             # what is left, normalised unless whole
        q = None if draft is None else _clean(draft[here])
        alive, left, step, gone = True, 1.0, None, set()
        if len(path) < width:
            for i in range(here + 1, n):
                if parents[i] != here:
                    continue
                x, u = tokens[i], float(accept_u[i])
                inside = 0 <= x < V
                if draft is None:
                    w = r[x] if inside else 0.0
                    if w > 0 and u * left < w:
                        step = i
                        break
                    left = max(left - w, 0.0)
                    if inside:
                        r[x] = 0.0
                    continue
                if not alive:
                    continue
                w, d = (r[x], q[x]) if inside else (0.0, 0.0)
                if w > 0 and u * d < w:
                    step = i
                    break
                r = np.maximum(r - q, 0.0)
                if r.sum() > 0:
                    r = r / r.sum()
                if not replacement and inside:
                    alive = 1.0 - d > 0
                    if alive:
                        q[x] = 0.0
                        q = q / (1.0 - d)
        if step is None:
            break
        here = step
        path.append(step)
        said.append(int(tokens[step]))
    if not r.sum() > 0:
        r = p
    if not r.sum() > 0:
        said.append(-1)
        return path, said
    upto = np.cumsum(r)
    past = np.nonzero(upto > float(sample_u) * upto[-1])[0]
    said.append(int(past[0]) if len(past) else int(np.nonzero(r > 0)[0][-1]))
    return path, said


def verify(target, draft, tokens, parents, accept_u, sample_u, starts, width, replacement=True):
    """path, tokens_out int32 [batch, width], count int32 [batch]."""
    B = len(starts) - 1
    path, out = (np.full((B, width), -1, np.int32) for _ in range(2))
    count = np.zeros(B, np.int32)
    for b in range(B):
        s = slice(starts[b], starts[b + 1])
        steps, said = verify_one(target[s], None if draft is None else draft[s], tokens[s], parents[s],
                                 accept_u[s], sample_u[b], width, replacement)
        path[b, :len(steps)], out[b, :len(said)], count[b] = steps, said, len(steps)
    return path, out, count


def accept(cache, table, lens, starts, path, count):
    """The four arrays [pages, heads, page_size, bytes] of a cache after the move; new lengths."""
    pages, page = cache[0].shape[0], cache[0].shape[2]
    covered = table.shape[1] * page
    after, new = [a.copy() for a in cache], np.zeros(len(lens), np.int32)
    for b, L in enumerate(lens):
        n, L = starts[b + 1] - starts[b], min(max(int(L), 0), covered)
        first, k = L - n, min(max(int(count[b]), 0), n, path.shape[1])
        new[b] = max(first + k, 0)
        for i in range(k):
            j = int(path[b, i])
            if not 0 <= j < n or first + i < 0 or first + j >= covered:
                continue
            p0, p1 = table[b, (first + j) // page], table[b, (first + i) // page]
            if 0 <= p0 < pages and 0 <= p1 < pages:
                for old, a in zip(cache, after):
                    a[p1, :, (first + i) % page] = old[p0, :, (first + j) % page]
    return after, new
