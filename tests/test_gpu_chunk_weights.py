"""Attention of chunks over weights far below the largest: how finely each kernel rounds them.

Every 16th key is `nats` ahead of the others, so that each part of a tile, whichever warp or CTA has it, holds weights of 1 and of
w = exp(-nats); the values of the first kind are 0, so that an output is made of the small ones alone:
  o = w S / (a + w b),   a keys ahead, b others, S the sum of the others' values, all positive.
Tolerance, relative, with h half a step of the type: max(h, u / w) + h + 2 e.  Weights are rounded by h of their own size, in f16 by u at least: they
are 2^11 (tensor cores) or 2^15 times larger in the product, where half the smallest step is 2^-25, so u = 2^-36 or 2^-40; in bf16, with
float32's exponents, u = 0.  h: the output.  e = nats (D + 4) 2^-24 + 2^-16: float32, as in the other tests; twice, for the sum."""
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


# query tokens, heads' dimension, caches that the copy engine has a map for, log2 of u
KERNELS = {"few": (2, 64, True, -40), "few 128": (1, 128, True, -40), "few 256": (2, 256, True, -40), "few, no map": (2, 128, False, -40),
           "tensor cores": (90, 64, True, -36), "tensor cores 128": (90, 128, True, -36), "tensor cores, no map": (50, 128, False, -36),
           "rows": (50, 256, True, -40)}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("n", [700, 30000])
@pytest.mark.parametrize("nats", [9.0, 14.0, 17.0, 20.0])
def test_small_weights(ms, dtype, kernel, n, nats):
    import torch
    new, D, mapped, log_u = KERNELS[kernel]
    c = case(70, dtype, [new], [n], 8, 2, D, 16)
    c["q"].zero_()
    c["q"][..., 0] = nats
    page = torch.from_numpy(c["table"][0].astype(np.int64)).cuda()
    t = torch.arange(n, device="cuda")
    ahead = t % 16 == 5
    c["k"].zero_()
    c["k"][page[t[ahead] // 16], t[ahead] % 16, :, 0] = 8.0      # times nats / 8
    c["v"].uniform_(0.5, 1.5).mul_(2.0 ** 14)                    # (outputs stay above f16's smallest normal number)
    c["v"][page[t[ahead] // 16], t[ahead] % 16] = 0
    v = c["v"][page[t // 16], t % 16].double().cumsum(0)         # [n, heads, dim]
    if not mapped:
        pages, size, H, _ = c["k"].shape
        slot = H * (D + 8) + 8
        k, w = (torch.zeros((pages + 1) * (size * slot + 8), dtype=c["k"].dtype, device="cuda").as_strided(
            (pages, size, H, D), (size * slot + 8, slot, D + 8, 1)) for _ in range(2))
        k.copy_(c["k"]), w.copy_(c["v"])
        c = dict(c, k=k, v=w)
    out, lse = call(ms, c, scale=0.125, max_queries=new)
    w = float(np.exp(-nats))
    half = torch.finfo(c["q"].dtype).eps / 2
    e = nats * (D + 4) * 2.0 ** -24 + 2.0 ** -16
    p = torch.arange(n - new, n, device="cuda")
    a = ahead.double().cumsum(0)[p]
    total = a + w * (p + 1 - a)
    want = (w * v[p] / total[:, None, None]).repeat_interleave(4, 1)
    tol = half + max(half, 2.0 ** log_u / w if dtype == "f16" else 0.0) + 2 * e
    rel = (out.double() / want - 1).abs()
    assert bool((rel <= tol).all()), (float(rel.max()), tol)
    sure = nats + torch.log(total)
    assert bool(((lse.double() - sure[:, None]).abs() <= e + 2.0 ** -22 * sure[:, None]).all())
