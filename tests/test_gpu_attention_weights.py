"""Attention over scores of any size."""
import numpy as np
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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [3, 20, 80])     # attend_kernel, tiles of 128 queries, of 256
@pytest.mark.parametrize("exponent", [12, 20, 24, 28, 31, 40, 60])
def test_scores_of_any_size(ms, dtype, rows, exponent):
    """Products q k up to 1.5 * 2^exponent, exact (one non-zero component), the largest once per head and at least 2^(exponent - 1)
    ahead: the next weight is exp(-2^(exponent - 1) / 8) = 0 in any float, so the output is that key's value, but for half a
    step each of two roundings: that key's weight w = 2^r, r the rounding of its score against the maximum's, enters the product
    rounded and the sum as it is (round(w) v / w), and the output's own.  lse: the constants log2(e) and ln 2 and two
    products, within 3 * 2^-24 of itself."""
    import torch
    if dtype == "f16" and exponent > 28:
        pytest.skip("beyond the type")
    n, lo = 600, exponent // 2
    c = _case(32, dtype, [rows], rows, 1, 8, 4, 64, [n], [0] * rows, 16)
    c["q"].zero_()
    c["q"][..., 0] = 2.0 ** lo
    c["k"].zero_()
    pages = torch.from_numpy(c["ptab"][0].astype(np.int64)).cuda()
    t = torch.arange(n, device="cuda")
    val = 2.0 ** (exponent - lo - 1) * (1 + (t % 128) / 128)     # 128 values, exact in 8 bits
    for h in range(4):
        val_h = val.clone()
        val_h[(37 * h + 11) % n] = 2.0 ** (exponent - lo) * 1.5
        c["k"][pages[t // 16], t % 16, h, 0] = val_h.to(c["k"].dtype)
    out, lse = _call(ms, c)
    for h in range(8):
        i = (37 * (h // 2) + 11) % n
        v = c["v"][int(c["ptab"][0, i // 16]), i % 16, h // 2]
        eps = torch.finfo(v.dtype).eps
        assert ((out[:, 0, h].double() - v.double()).abs() <= eps * (1 + eps) * v.double().abs()).all(), (h, out[0, 0, h, :4], v[:4])
    s = 1.5 * 2.0 ** exponent / 8
    assert ((lse.double() - s).abs() <= 2.0 ** -22 * s).all()
