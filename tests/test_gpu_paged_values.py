"""Values and table entries at the edges of the paged attention: infinities and NaN in V, also where a row
has one key only."""
import pytest
import torch

from paged_common import Batch, cobs

pytestmark = pytest.mark.gpu


def _put(b, r, t, value, columns=slice(None, None, 7)):
    """V of token t of request r holds `value` in some columns of every head."""
    page = b.p.page
    b.V[r][:, t, columns] = value
    b.v_cache[b.table[r, t // page].item(), :, t % page] = b.V[r][:, t].to(b.v_cache.device)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("G,d,page", [(1, 128, 16), (4, 128, 64), (8, 64, 32), (11, 64, 128), (16, 128, 16)])
def test_values_of_single_tokens(dtype, value, G, d, page):
    """A visible infinity reaches the output as what it is (its weight is a positive number), a hidden one
    does not, and the other columns keep their accuracy."""
    C = cobs()
    lens = [(0, 1), (1, 1), (100, 1), (130, 1), (3000, 1)]
    for W, S in ((0, 0), (40, 3)):
        b = Batch(C, lens, 2 * G, 2, d, page, dtype=dtype, window=W, sinks=S, drop_unseen=False, seed=G)
        for r, t in ((0, 0), (1, 1), (2, 60), (2, 99), (3, 2), (4, 5), (4, 2990)):
            _put(b, r, t, value)
        _put(b, 4, 2999, -value, slice(3, None, 14))
        C.device_error(reset=True)
        b.run()
        assert C.device_error() == 0
        b.check((W, S))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("entry", [-1, -2, -2 ** 31, -2 ** 31 + 1, 1 << 20, 2 ** 31 - 1])
@pytest.mark.parametrize("new", [1, 30])
def test_every_entry_outside_the_cache_counts_as_zeros_and_is_recorded(dtype, entry, new):
    C = cobs()
    b = Batch(C, [(3000, new), (90, 1)], 4, 2, 128, 32, dtype=dtype)
    warm = Batch(C, [(3000, new), (90, 1)], 4, 2, 128, 32, dtype=dtype, seed=1)   # shared memory holds other keys
    for j in (1, 40, 93):
        b.table[0, j] = entry
        b.K[0][:, 32 * j:32 * (j + 1)] = 0
        b.V[0][:, 32 * j:32 * (j + 1)] = 0
    C.device_error(reset=True)
    warm.run()
    assert C.device_error() == 0
    b.run()
    assert C.device_error(reset=True) == 1
    b.check(entry)
    # entries of pages that no row sees may be anything
    b = Batch(C, [(3000, new), (90, 1)], 4, 2, 128, 32, dtype=dtype, window=50, sinks=2)
    b.table[b.table < 0] = entry
    b.run()
    assert C.device_error() == 0
    b.check(entry)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[(3000, 20)], [(700, 32), (40, 5)], [(90, 30), (200, 31), (5, 2)]])
def test_chunks_of_one_row_tile_with_infinite_values(lens, d):
    """The key tiles of at most 128 rows go to two groups of threads, whose accumulators are joined; tiles with
    infinities that some rows do not see are multiplied by the threads. Calls agree bit for bit."""
    C = cobs()
    b = Batch(C, lens, 8, 2, d, 32, window=600, sinks=5, drop_unseen=False)
    for r, (c, n) in enumerate(lens):
        for t in (c + n - 1, c + n // 2, max(0, c - 300), 3):
            _put(b, r, t, float("inf"), slice(t % 5, None, 11))
    b.run()
    b.check()
    first = b.O.clone()
    for _ in range(30):
        b.O.fill_(7.0)
        b.run()
        assert torch.equal(b.O.view(torch.int16), first.view(torch.int16))
    assert C.device_error() == 0
