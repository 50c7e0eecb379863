"""Attention of chunks: a request's answer does not depend on the requests beside it in the batch."""
import numpy as np
import pytest

from tests.helpers import ensure_built
from tests.test_gpu_chunk_attention import call, case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [5, 33, 70, 97])      # last tiles of 20 to 132 rows: 4, 20 or 24 of a warp's 32 are the request's
def test_the_next_requests_queries(ms, dtype, D, n):
    """Ragged last tiles beside queries of every size, and beside rows of no request.  So many requests that a CTA has a tile's keys
    from first to last: its rows' maxima grow on the way."""
    import torch
    R = 24
    c = case(40, dtype, [n, 40] * R, [1500, 300] * R, 32, 8, D, 16, tail=64)
    own = torch.zeros(c["q"].shape[0], dtype=torch.bool, device="cuda")
    for r in range(0, 2 * R, 2):
        own[int(c["starts"][r]):int(c["starts"][r + 1])] = True
    want, lse = call(ms, c)
    assert not bool(torch.isnan(want).any())
    for factor in (0.0, 4.0, 40.0, float("inf"), float("nan")):
        q = c["q"].clone()
        q[~own] *= factor
        out, l = call(ms, dict(c, q=q))
        assert torch.equal(out[own], want[own]) and torch.equal(l[own], lse[own]), factor


@pytest.mark.parametrize("D", [64, 128])
def test_many_ragged_requests_into_the_query(ms, D):
    """Each tile's rows behind its request are being written over by the next one's: the same bits as into an output apart."""
    import torch
    rng = np.random.default_rng(42)
    new = rng.integers(1, 90, 120)
    c = case(42, "bf16", new, new + rng.integers(0, 900, 120), 8, 2, D, 16)
    c["q"] *= 30
    c["v"] *= 30
    want, lse = call(ms, c)
    for _ in range(10):
        q = c["q"].clone()
        out, l = call(ms, dict(c, q=q), out=q)
        assert torch.equal(out, want) and torch.equal(l, lse)
