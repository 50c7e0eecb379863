"""Page tables and token places from request lengths (fs_paged_step_tables): whole numbers, equal to an
allocator that goes request by request."""
import numpy as np
import pytest

from oracle import serving
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


def _cu(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _check(ms, lens, new, width, page, free, budget, count=None, table=None, seed=0):
    rng = np.random.default_rng(seed)
    R = len(lens)
    table = rng.integers(0, 10 ** 6, (R, width)).astype(np.int32) if table is None else table
    stack = rng.permutation(2 * free + 5)[:free].astype(np.int32)
    count = free if count is None else count
    want = serving.step_tables(lens, new, table, stack, count, page, budget)
    t, s = _cu(table), _cu(stack)
    got = ms.paged_step_tables(_cu(lens), _cu(new), t, s, _cu([count]), page, budget)
    assert (t.cpu().numpy() == want[0]).all()
    for g, w, n in zip(got, want[1:], (R + 1, budget, budget, R, 1)):
        assert g.shape == (n,) and g.tolist() == (w if isinstance(w, list) else [w])
    assert (s.cpu().numpy() == stack).all()
    return got


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("R", [1, 2, 31, 33, 511, 512, 513, 1500])
def test_mixed_steps(ms, R, page):
    """Requests that decode, chunks, idle ones; as many pages and tokens as are asked for, or fewer."""
    rng = np.random.default_rng(R + page)
    lens = rng.integers(0, 900, R)
    new = np.where(rng.random(R) < 0.7, 1, np.where(rng.random(R) < 0.5, 0, rng.integers(1, 700, R)))
    new[rng.integers(0, R)] = 900
    need = int((-(-(lens + new) // page) - -(-lens // page)).sum())
    total = int(new.sum())
    for free, budget in ((need, total), (need + 7, total + 100), (need * 2 // 3, total), (need, total * 3 // 4), (1, 3), (0, 0)):
        _check(ms, lens, new, 1900 // page + 1, page, free, budget)


def test_windows_of_places(ms):
    """Requests that start and end inside, at and across the borders of a CTA's 2048 places."""
    for new in ([2047, 1, 2048, 1], [2048, 2048], [1] * 4100, [5000], [2046, 5000, 3], [1, 4095, 4096, 4097]):
        n = len(new)
        for page in (1, 2, 3):
            _check(ms, [page - 1] * n, new, 5100, page, sum(new) + n, sum(new) + 11)


def test_lengths_that_ask_for_nothing(ms):
    """Negative lengths, more tokens than the table can name, lengths whose sum passes 32 bits."""
    big = 2 ** 31 - 1
    _check(ms, [3, -1, 5, big, 100, 0, -2 ** 31, 7], [2, 4, -3, big, 61, 160, 1, 0], 10, 16, 50, 400)
    _check(ms, [0, 0, 0], [160, 161, 160], 10, 16, 50, 320)
    _check(ms, [big, 1], [big, big], 4, 16, 5, 10)


def test_stack_counts_are_clamped(ms):
    for count in (-3, 0, 2, 99, 2 ** 31 - 1):
        _check(ms, [0, 16, 5], [17, 1, 1], 4, 16, 6, 30, count=count)


def test_nothing_to_do(ms):
    _check(ms, [], [], 4, 16, 5, 8)
    _check(ms, [3, 4], [1, 1], 0, 16, 5, 8)
    _check(ms, [3, 4], [1, 1], 4, 16, 0, 8)      # no pages needed, none there
    _check(ms, [3, 4], [0, 0], 4, 16, 5, 0)


def test_many_requests_and_large_pages(ms):
    rng = np.random.default_rng(5)
    _check(ms, rng.integers(0, 50, 20000), rng.integers(0, 3, 20000), 4, 16, 9000, 15000)
    _check(ms, [2 ** 30, 5], [10, 2 ** 20], 3, 2 ** 29 - 10000, 4, 2 ** 20 + 10)


def test_captured_step_by_step(ms):
    """A graph that allocates, replayed with the totals and the count it left; then the same on another stream."""
    import torch
    rng = np.random.default_rng(1)
    R, page, width, F = 9, 4, 30, 200
    lens, new, table, count = _cu(rng.integers(0, 20, R)), _cu(rng.integers(0, 5, R)), _cu(np.full((R, width), -1)), _cu([F])
    stack = _cu(rng.permutation(F))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ms.paged_step_tables(lens, new, table.clone(), stack, count, page, 40)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        starts, rows, pos, totals, left = ms.paged_step_tables(lens, new, table, stack, count, page, 40)
        lens.copy_(totals)
        count.copy_(left)
    hl, ht, hc = lens.tolist(), table.cpu().numpy(), F
    for i in range(6):
        new.copy_(_cu(rng.integers(0, 5, R)))
        want = serving.step_tables(hl, new.tolist(), ht, stack.tolist(), hc, page, 40)
        g.replay()
        torch.cuda.synchronize()
        ht, hl, hc = want[0], want[4], want[5]
        assert (table.cpu().numpy() == ht).all() and starts.tolist() == want[1] and rows.tolist() == want[2]
        assert pos.tolist() == want[3] and lens.tolist() == hl and count.tolist() == [hc]
