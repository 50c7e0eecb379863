"""Attention of chunks whose waits run out: a limit on the kernels' waits, so short that CTAs give up in the middle of their
work.  Every launch ends, what was not computed is NaN, and calls behind it are as if it had not been."""
import ctypes

import numpy as np
import pytest

from tests.helpers import ensure_built
from tests.test_gpu_chunk_attention import call, case

pytestmark = pytest.mark.gpu
DEFAULT = 4 * 10 ** 9
LIMITS = [0, 1000, 3000, 10000, 20000, 30000, 50000, 80000]     # clock cycles; a key tile takes 1000 to 3000


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    min_sampling_gb300.lib.fs_paged_chunk_attention_wait_limit.argtypes = [ctypes.c_int64]
    return min_sampling_gb300


@pytest.fixture
def limit(ms):
    def to(cycles):
        assert ms.lib.fs_paged_chunk_attention_wait_limit(cycles) == 0
    yield to
    to(DEFAULT)


# More tiles for a CTA than are described ahead, cut ones and whole ones; of requests with few rows, with many, with both.
CASES = {"few": ([1, 3, 2, 1] * 50, [300, 70, 20, 900] * 50), "many": ([40, 7, 300, 90] * 35, [150, 60, 350, 100] * 35),
         "both": ([1, 40, 3, 90] * 40, [500, 100, 50, 300] * 40)}


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", CASES)
def test_every_launch_ends(ms, limit, D, kind):
    import torch
    c = case(60, "bf16", *CASES[kind], 16, 8, D, 16)
    hint = dict(max_queries=4 if kind == "few" else None)
    want, lse = call(ms, c, **hint)
    torch.cuda.synchronize()
    for cycles in LIMITS:
        limit(cycles)
        call(ms, c, out=torch.empty_like(want), **hint)
        torch.cuda.synchronize()
        limit(DEFAULT)
        out, l = call(ms, c, **hint)
        assert torch.equal(out, want) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", CASES)
def test_every_row_is_right_or_nan(ms, limit, dtype, D, kind):
    """Nothing of what an output or a workspace held before shows: each head of each token is the answer's bits or NaN, its lse
    too, and rows of no request are as they were."""
    import torch
    if D == 256 and kind != "few":
        pytest.skip("many rows of heads of 256 have no waits of this kind")
    c = case(61, dtype, *CASES[kind], 16, 8, D, 16, lead=2, tail=3)
    hint = dict(max_queries=4 if kind == "few" else None)
    want, lse = call(ms, c, out=torch.full_like(c["q"], 7.0), **hint)
    lost = []
    for cycles in LIMITS + [0] * 4:
        torch.full((1 << 26,), 7.0, device="cuda")    # what the allocator hands out next
        limit(cycles)
        out, l = call(ms, c, out=torch.full_like(c["q"], 7.0), **hint)
        torch.cuda.synchronize()
        limit(DEFAULT)
        gone = torch.isnan(out).all(-1)
        lost.append(int(gone.sum()))
        same = (out == want).all(-1) & (l == lse)
        assert bool((same | (gone & torch.isnan(l))).all()), (cycles, lost)
        n = int(c["starts"][-1])
        assert bool((out[:2] == 7).all()) and bool((out[n:] == 7).all())
    assert max(lost) > 0, lost  # (of no cycles: the first wait that is not over when it is looked at)
