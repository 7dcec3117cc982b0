"""Inputs of the attention operators' GPU tests: paged MXFP4 caches, and checks with their bounds."""
import numpy as np
import torch

from oracle import attention_oracle as A


def bf16(x) -> torch.Tensor:
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def tables(rng, rows: int, rot: int):
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(rows)[:, None] * f + rng.uniform(0, 0.1)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


class Paged:
    """A random paged cache (host arrays and GPU tensors): sequences of the given lengths in pages
    that are dealt at random, every byte that belongs to no sequence set to `junk`."""

    def __init__(self, rng, lens, heads, D, page_size, spare=2, width_extra=1, junk=0xFF,
                 lo=120, hi=132, gap=0):
        self.lens, self.heads, self.D, self.page_size = list(lens), heads, D, page_size
        counts = [-(-n // page_size) for n in lens]
        pages = sum(counts) + spare
        order = rng.permutation(pages)
        width = max(counts, default=0) + width_extra
        self.table = np.full((len(lens), width), -7, np.int32)      # unused entries: not a page
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (pages, heads, page_size)
        self.k, self.ks, self.v, self.vs = (np.full(shape + (w,), junk, np.uint8)
                                            for w in (D // 2, D // 32, D // 2, D // 32))
        for b, n in enumerate(lens):
            for t in range(0, n, page_size):
                page, m = self.table[b, t // page_size], min(page_size, n - t)
                for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
                    codes[page, :, :m] = rng.integers(0, 256, (heads, m, D // 2))
                    scales[page, :, :m] = rng.integers(lo, hi + 1, (heads, m, D // 32))
        self.gap = gap

    def tensors(self):
        """The four GPU tensors; `gap` bytes between pages' blocks (a multiple of 16)."""
        out = []
        for a in (self.k, self.ks, self.v, self.vs):
            p, h, s, w = a.shape
            buf = torch.full((p, h * s * w + self.gap), 0xA5, dtype=torch.uint8, device="cuda")
            t = buf[:, :h * s * w].unflatten(1, (h, s, w))
            t.copy_(torch.from_numpy(a))
            out.append(t)
        return out


def attention_close(out, lse, ref, what="", reach=1e4 * 192):
    """Compares bf16 out and fp32 lse (or None) with attention_oracle.attention's four arrays.

    Bounds: a score's fp32 sum of exact products is off by at most d = 2^-20 scale sum |q k| (the
    bound of the library's GEMMs), which scales each weight by at most e^{2 d}; a weight is rounded
    to bf16 once (2^-9 of it, doubled for the sums' fp32 rounding and exp2), so the mean moves by at
    most (2^-8 + 4 d) sum p |v| / sum p; the result is rounded once (2^-8 of it).  A weight below
    fp32's normal range, 2^-126 of the row's largest, counts as zero: that moves the mean by at most
    2^-126 of the sum of all |v| (`reach`).  The lse moves by at most d and the relative error of
    its sum, 2^-18 at these lengths."""
    o, l, mag, top = ref
    o_got = f64(out)
    d = 2.0 ** -20 * top[..., None]
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 4 * d) * mag + 2.0 ** -126 * (1 + reach)
    nan = np.isnan(o)
    assert np.array_equal(np.isnan(o_got), nan), f"{what}: NaN in other places"
    bad = ~(np.abs(o_got - o) <= tol) & ~nan
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outputs, first {np.argwhere(bad)[0]}"
    if lse is not None:
        got = f64(lse)
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(got), empty), f"{what}: lse -inf in other places"
        fine = ~empty & ~np.isnan(l)
        lt = d[..., 0] + 2.0 ** -18 * np.maximum(1, np.abs(l))
        assert (np.abs(got[fine] - l[fine]) <= lt[fine]).all(), f"{what}: lse"


def oracle(paged, q, starts, scale, **how):
    return A.attention(f64(q), paged.k, paged.ks, paged.v, paged.vs, paged.table, paged.lens,
                       starts, scale, **how)
