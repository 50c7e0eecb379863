"""Attention over infinite and NaN values in a row's last tokens."""
import pytest

from tests.helpers import ensure_built
from tests.test_gpu_prefix_attention import _call, _case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("own", [5, 40, 64, 67, 130, 700])
@pytest.mark.parametrize("prefix", [0, 100, 600])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinite_values_that_a_query_sees(ms, dtype, prefix, own, D):
    """Infinite and NaN values in the last tokens reach the queries that see them as the sum has them, and no other query."""
    import torch
    Q = 5
    for rows in (2, 12):
        c = _case(34 + own, dtype, [rows], rows, Q, 8, 2, D, [prefix], [own] * rows, 16)
        clean, _ = _call(ms, c)
        inf, nan = float("inf"), float("nan")
        marks = [(0, own - 1, 0, inf), (0, own - 2, 1, -inf), (0, own - 3, 2, inf), (0, own - 1, 2, -inf), (0, own - 4, 3, nan),
                 (0, own - 2, D - 1, inf), (1, own - 4, 5, -inf), (1, own - 1, 5, -inf), (1, own - 5, 6, inf)]
        for b, t, d, x in marks:
            c["v"][int(c["stab"][b, t // 16]), t % 16, 1, d] = x
        want = clean.clone()
        for b, t, d, x in marks:
            for j in range(Q):
                if t <= own - Q + j:
                    want[b, j, 4:, d] += x        # the heads that read head 1
        out, _ = _call(ms, c)
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))
