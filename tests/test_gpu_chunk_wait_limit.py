"""Attention of chunks whose waits run out: a limit on the kernels' waits for their own copies and products, so short that
some of them give up.  Every launch ends, and calls behind it are as if it had not been."""
import ctypes

import numpy as np
import pytest

from tests.helpers import ensure_built
from tests.test_gpu_chunk_attention import call, case

pytestmark = pytest.mark.gpu
DEFAULT = 4 * 10 ** 9
LIMITS = [0, 300, 1000, 3000, 10000, 30000]     # clock cycles; a key tile takes 1000 to 3000


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


CASES = {"few": ([1, 3, 2] * 9, [5000, 300, 70] * 9), "many": ([300, 40, 700], [4000, 900, 700]), "both": ([1, 300, 2], [9000, 3000, 50])}


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", CASES)
def test_every_launch_ends(ms, limit, D, kind):
    import torch
    c = case(60, "bf16", *CASES[kind], 8, 2, D, 16)
    want, lse = call(ms, c)
    torch.cuda.synchronize()
    for cycles in LIMITS:
        limit(cycles)
        call(ms, c, out=torch.empty_like(want))
        torch.cuda.synchronize()
        limit(DEFAULT)
        out, l = call(ms, c)
        assert torch.equal(out, want) and torch.equal(l, lse)
