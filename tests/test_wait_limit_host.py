"""The limit on chunk attention's waits, without a GPU: negative ones are refused."""
import ctypes

from tests.helpers import ensure_built


def test_wait_limit_arguments():
    ensure_built()
    import min_sampling_gb300
    f = min_sampling_gb300.lib.fs_paged_chunk_attention_wait_limit
    f.argtypes = [ctypes.c_int64]
    assert f(-1) == 1 and f(-2 ** 63) == 1
    assert f(4 * 10 ** 9) == 0
