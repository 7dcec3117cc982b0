"""mx_kv_accept_fp4 at the ends of what its arguments may be: pages of more than 4 GiB."""
import numpy as np
import pytest
import torch

from draft_util import ints
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_of_more_than_4_gib(mx, dim):
    # one page of one head, whose codes pass 2^32 bytes; nodes on both sides of that byte, then behind it
    rng = np.random.default_rng(dim)
    at = (1 << 33) // dim                                      # the token whose codes begin at byte 2^32
    cache = [torch.zeros((1, 1, at + 160, w), dtype=torch.uint8, device="cuda") for w in (dim // 2, dim // 32) * 2]
    for first, n, path in ((at - 100, 200, [0, 1, 60, 99, 100, 101, 150, 199]), (at - 3, 90, [0, 4, 5, 6, 80, 89]),
                           (at + 30, 120, [0, 2, 3, 64, 119])):
        nodes = slice(first, first + n)
        before = [torch.from_numpy(rng.integers(1, 256, (n, t.shape[3]), dtype=np.uint8)).cuda() for t in cache]
        for t, b in zip(cache, before):
            t[0, 0, nodes] = b
        new = ints([-77])
        note(f"accept in a page of {at + 160} tokens, D={dim}, nodes from {first}")
        mx.mx_kv_accept_fp4(mx.MxKvCacheFp4(*cache), ints([[0]]), ints([first + n]), ints([path]), ints([len(path)]),
                            lens_out=new, max_q=n)
        torch.cuda.synchronize()
        assert new.item() == first + len(path)
        for t, b in zip(cache, before):
            want = b.clone()
            want[:len(path)] = b[torch.tensor(path, device="cuda")]
            assert torch.equal(t[0, 0, nodes], want)
            t[0, 0, nodes] = 0                                 # nothing else is written
            assert not any(bool(part.any()) for part in t.view(-1).split(1 << 30))
