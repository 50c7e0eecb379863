"""Attention of chunks through the C ABI with a caller's workspace: any multiple of 16 bytes, of the size asked for,
and nothing written outside of it."""
import ctypes

import numpy as np
import pytest

from tests.helpers import ensure_built
from tests.test_decode_host import KV, _s
from tests.test_gpu_chunk_attention import call, case

pytestmark = pytest.mark.gpu
P, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    lib = min_sampling_gb300.lib
    lib.fs_paged_chunk_attention.argtypes = [P, P, P, i32, i32, P, i32, i32, P, P, i32, i32, i32, f32, i32, P, P, P, P, sz, P]
    lib.fs_paged_chunk_attention_workspace_bytes.argtypes = [P, i32, i32, i32, i32, i32, P]
    return min_sampling_gb300


@pytest.mark.parametrize("D,gs", [(64, 4), (128, 4), (256, 4), (128, 1)])
@pytest.mark.parametrize("at", [0, 16, 32, 48, 112, 240])
def test_any_multiple_of_16_bytes(ms, D, gs, at):
    """Tiles that are cut across CTAs (their parts lie in the workspace) and whole ones, many rows and few."""
    import torch
    c = case(50, "bf16", [300, 1, 40, 2], [3000, 5000, 700, 3], 2 * gs, 2, D, 16)
    want, lse = call(ms, c)
    cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    q, k, v, table, starts, lens = c["q"], c["k"], c["v"], cu(c["table"]), cu(c["starts"]), cu(c["lens"])
    N, Hq = q.shape[:2]
    kv = KV.pack(k.data_ptr(), v.data_ptr(), 1, k.shape[0], 16, 2, D, *k.stride()[:3], *v.stride()[:3])
    n = sz(0)
    assert ms.lib.fs_paged_chunk_attention_workspace_bytes(kv, N, len(lens), Hq, table.shape[1], N, ctypes.byref(n)) == 0
    ws = torch.full((n.value + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0
    out, l = torch.zeros_like(q), torch.zeros(N, Hq, device="cuda")
    args = [kv, q.data_ptr(), _s(*q.stride()[:2]), N, Hq, table.data_ptr(), len(lens), table.shape[1], starts.data_ptr(), lens.data_ptr(),
            N, 0, 0, D ** -0.5, 1, out.data_ptr(), _s(*out.stride()[:2]), l.data_ptr()]
    stream = torch.cuda.current_stream().cuda_stream
    assert ms.lib.fs_paged_chunk_attention(*args, ws.data_ptr() + at, n.value - 1, stream) == 1
    assert ms.lib.fs_paged_chunk_attention(*args, ws.data_ptr() + at, n.value, stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(l, lse)
    assert bool((ws[:at] == 0x5a).all()) and bool((ws[at + n.value:] == 0x5a).all())
