"""Trees of drafted tokens for the draft operators' tests."""
import numpy as np
import torch


def random_parents(rng, n, reach=6):
    """A tree of n nodes in order of its levels, at most `reach` nodes past a node's first possible child."""
    p = [-1]
    for i in range(1, n):
        p.append(int(rng.integers(max(p[-1], 0), min(i, max(p[-1], 0) + reach))))
    return np.array(p[:n], np.int32)


def forest(rng, sizes, kind="tree"):
    """Parents of all sequences' nodes [nodes] and starts."""
    make = {"tree": lambda n: random_parents(rng, n), "chain": lambda n: np.arange(-1, n - 1, dtype=np.int32),
            "star": lambda n: np.where(np.arange(n) > 0, 0, -1).astype(np.int32)}[kind]
    starts = [0, *np.cumsum(sizes).tolist()]
    return np.concatenate([make(n)[:n] for n in sizes] or [np.zeros(0)]).astype(np.int32), starts


def ints(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)
