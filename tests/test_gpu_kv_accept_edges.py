"""mx_kv_accept_fp4 at the ends of what its arguments may be: pages of more than 4 GiB, caches that can
be gone over only once, no caches at all."""
import numpy as np
import pytest
import torch

from draft_util import ints
from gpu_util import note
from oracle import draft_oracle as D

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


@pytest.mark.parametrize("of", [iter, lambda cs: (c for c in cs), lambda cs: map(lambda c: c, cs), tuple,
                                lambda cs: dict(enumerate(cs)).values()])
def test_caches_from_any_iterable(mx, of):
    rng = np.random.default_rng(1)
    table, sizes, lens, path, count = np.array([[2, 0], [1, 3]]), [9, 5], [20, 25], [[0, 3, 8], [0, 2, 4]], [3, 2]
    cs = [[rng.integers(0, 256, (4, 2, 16, w), dtype=np.uint8) for w in (64, 4) * 2] for _ in range(3)]
    ts = [[torch.from_numpy(a).cuda() for a in c] for c in cs]
    new = ints([-77, -77])
    note("accept caches from an iterable")
    mx.mx_kv_accept_fp4(of([mx.MxKvCacheFp4(*t) for t in ts]), ints(table), ints(lens), ints(path), ints(count),
                        lens_out=new, q_starts=ints([0, 9, 14]), max_q=9)
    torch.cuda.synchronize()
    for c, t in zip(cs, ts):
        want, lengths = D.accept(c, table, lens, [0, 9, 14], np.array(path), count)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(t, want))
    assert np.array_equal(new.cpu().numpy(), lengths)


def test_iterables_of_what_is_no_cache_are_refused(mx):
    good = mx.MxKvCacheFp4(*(torch.zeros((4, 2, 16, w), dtype=torch.uint8, device="cuda") for w in (64, 4) * 2))
    for caches in (iter([good, None]), (c for c in (good, "k")), None, 5):
        with pytest.raises(TypeError):
            mx.mx_kv_accept_fp4(caches, ints([[0, 1]]), ints([20]), ints([[0, 2]]), ints([2]), max_q=4)


@pytest.mark.parametrize("caches", [list, tuple, lambda: iter(())])
def test_new_lengths_are_written_without_layers(mx, caches):
    sizes = [9, 0, 5, 30, 7, 4, 12, 3]
    lens, count = [20, 11, 25, 12, -3, 2 ** 31 - 1, 40, 9], [3, 0, 5, 2, 1, 4, 100, -8]
    starts = np.cumsum([0, *sizes])
    path, table = np.tile(np.arange(6), (8, 1)), np.full((8, 1), 2 ** 31 - 1)       # a table of nothing
    # no page size to clamp lengths by; counts as elsewhere
    want = [max(max(L, 0) - n + min(max(k, 0), n, 6), 0) for L, n, k in zip(lens, sizes, count)]
    new = ints([-77] * 9)
    note("accept without layers")
    mx.mx_kv_accept_fp4(caches(), ints(table), ints(lens), ints(path), ints(count), lens_out=new[:8], q_starts=ints(starts),
                        max_q=30)
    torch.cuda.synchronize()
    assert new.tolist() == [*want, -77]


def test_new_lengths_without_layers_of_many_sequences_in_a_graph(mx):
    B, n = 65535, 4
    rng = np.random.default_rng(2)
    path, table = ints(np.tile([0, 1, 3, -1], (B, 1))), ints(np.zeros((B, 1)))
    lens, count, new = ints(rng.integers(n, 1000, B)), ints(rng.integers(0, 4, B)), ints(np.full(B, -77))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    note("accept without layers, captured")
    with torch.cuda.graph(graph, stream=side):
        mx.mx_kv_accept_fp4([], table, lens, path, count, lens_out=new, max_q=n)
    for _ in range(3):
        lens.add_(5)
        count.copy_(ints(rng.integers(0, 4, B)))
        new.fill_(-77)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(new, lens - n + count)


def test_lengths_of_caches_of_no_pages(mx):
    # nothing moves, whatever path and table say; lengths end where the table does
    cache = mx.MxKvCacheFp4(*(torch.zeros((0, 2, 16, w), dtype=torch.uint8, device="cuda") for w in (64, 4) * 2))
    new = ints([-77, -77])
    note("accept of no pages")
    mx.mx_kv_accept_fp4([cache], ints([[0, 1], [5, -1]]), ints([20, 99]), ints([[0, 2], [0, 3]]), ints([2, 1]), lens_out=new, max_q=4)
    torch.cuda.synchronize()
    assert new.tolist() == [18, 29]
