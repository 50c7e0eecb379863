"""Sampling from given uniforms where top-p's mass ends in a row's tail."""
import numpy as np
import pytest

from tests.helpers import ensure_built
from tests.test_gpu_uniforms import _check as _check_tokens
from tests.test_gpu_uniforms import _logits, _u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


def _peaked(dtype, B, V, sigma, peak, seed):
    z = _logits(B, V, dtype, seed, sigma)
    if peak is not None:
        z[:, V // 3] = peak
    return z


TAILS = [("bf16", 256000, 3.0, None, 0.9), ("bf16", 256000, 4.0, None, 1.0), ("bf16", 151936, 2.0, 18.0, 1.0),
         ("f32", 151936, 2.0, 18.0, 1.0), ("f16", 128256, 1.0, 25.0, 1.0), ("f32", 256000, 5.0, None, 1.2)]


@pytest.mark.parametrize("case", range(len(TAILS)))
@pytest.mark.parametrize("p", [0.995, 0.999, 0.9999, 0.999999])
def test_top_p_that_ends_in_the_tail(ms, case, p):
    """Confident rows and wide ones: the mass that top-p asks for ends among tokens of little weight."""
    dtype, V, sigma, peak, T = TAILS[case]
    z = _peaked(dtype, 3, V, sigma, peak, 41 + case)
    for kw in (dict(), dict(top_k=5000), dict(top_k=5000, order="top_k_first"), dict(min_p=1e-8)):
        _check_tokens(ms, z, _u(3, 5), temperature=T, top_p=p, few_near=False, **kw)
        _check_tokens(ms, z, np.float32([1 - 2.0 ** -24, 0.9999, 0.999]), temperature=T, top_p=p, few_near=False, **kw)


@pytest.mark.parametrize("case", range(len(TAILS)))
def test_top_p_takes_a_few_passes(ms, case):
    """Wherever the mass ends, a row takes a few passes: 20 times what it takes at top-p 0.5 at most.  There it takes two, the
    second over few segments; at worst six, of which the weighing ones are two to four times as long."""
    import torch
    dtype, V, sigma, peak, T = TAILS[case]
    z = _peaked(dtype, 4, V, sigma, peak, 41 + case)
    u = torch.full((4,), 0.5, device="cuda")

    def time(p):
        t, p = torch.full((4,), T, device="cuda"), torch.full((4,), p, device="cuda")
        best = float("inf")
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            ms.top_k_top_p_sampling_from_uniforms(z, u, t, None, p)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    base = time(0.5)
    for p in (0.9, 0.99, 0.995, 0.999, 0.9995, 0.9999, 0.99999, 0.999999):
        assert time(p) <= 20 * base, (p, time(p), base)
