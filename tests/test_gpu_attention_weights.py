"""Attention over scores of any size and weights far below the largest."""
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


def _tail(dtype, rows, Q, n, own, nats, seed=33):
    """One key `nats` ahead of n - 1 equal ones whose values are around 1; its own value is 0 (a sink).  The keys are the
    prefix's, or with `own` each row's."""
    import torch
    c = _case(seed, dtype, [rows], rows, Q, 8, 4, 64, [0 if own else n], [n if own else Q] * rows, 64)
    c["q"].zero_()
    c["q"][..., 0] = nats
    c["k"].zero_()
    c["v"].uniform_(0.5, 1.5)
    for tab in (c["stab"] if own else c["ptab"]):
        c["k"][int(tab[0]), 0, :, 0] = 8.0        # times nats / sqrt(64)
        c["v"][int(tab[0]), 0] = 0
    if not own:
        for tab in c["stab"]:                     # the rows' own tokens: weightless
            c["k"][int(tab[0]), :, :, 0] = -512.0
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,Q,n,own", [(3, 1, 65537, False), (20, 1, 65537, False), (80, 1, 20000, False), (2, 2, 30000, True),
                                          (1, 1, 5000, True)])
@pytest.mark.parametrize("nats", [9.0, 11.0, 14.0, 17.0])
def test_a_long_tail_of_small_weights(ms, dtype, rows, Q, n, own, nats):
    """The tail's weights are rounded to half a step of their own size, down to 2^-25 of the largest.  Tolerance, with h half
    a step: h A (weights) + h |o| (output) + 2 e A (float32: the score's error 68 * 2^-24 * nats, and 2^-16); A = o here."""
    import torch
    c = _tail(dtype, rows, Q, n, own, nats)
    out, lse = _call(ms, c)
    half = torch.finfo(c["q"].dtype).eps / 2
    f = lambda t: t.double().cpu().numpy()
    e = nats * 68 * 2.0 ** -24 + 2.0 ** -16
    w = np.exp(-nats)
    v = f(c["v"])
    for b in {0, rows - 1}:
        tab = c["stab"][b] if own else c["ptab"][0]
        for j in range(Q):
            m = n - (Q - 1 - j) if own else n
            t = np.arange(1, m)
            o = w * v[np.asarray(tab)[t // 64], t % 64].sum(0) / (1 + w * (m - 1))      # [heads, dim]
            got = f(out[b, j]).reshape(4, 2, 64)
            assert (np.abs(got - o[:, None]) <= (2 * half + 2 * e) * np.abs(o[:, None])).all(), \
                (nats, np.abs(got / o[:, None] - 1).max())
            assert np.abs(f(lse[b, j]) - nats - np.log1p(w * (m - 1))).max() <= e + 2.0 ** -22 * nats
