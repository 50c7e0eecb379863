"""Strides of either sign at the C ABI: tensors read and written backwards give what their flipped copies give."""
import ctypes
import struct

import pytest

from tests.helpers import ensure_built
from tests.test_gpu_prefix_attention import _call, _case

pytestmark = pytest.mark.gpu
KV = struct.Struct("@PPiiiii6q")   # fs_paged_kv
FS_BF16 = 1


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


def _backwards(t, n):
    """Address and strides of t read backwards along its first n dimensions: the same elements as t.flip(range(n))."""
    at = t.data_ptr() + t.element_size() * sum((t.shape[i] - 1) * t.stride(i) for i in range(n))
    return at, [-t.stride(i) for i in range(n)]


def _kv(k, v):
    (ka, ks), (va, vs) = _backwards(k, 3), _backwards(v, 3)
    return KV.pack(ka, va, FS_BF16, *k.shape, *ks, *vs)


def _s(v):
    return (ctypes.c_int64 * len(v))(*v)


@pytest.mark.parametrize("rows", [3, 40])     # without and with the tensor-core kernel
def test_attention_over_negative_strides(ms, rows):
    import torch
    P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib = ctypes.CDLL(ms.LIB_PATH)
    f = lib.fs_shared_prefix_attention
    f.argtypes = [P, P, P, i32, i32, i32, P, i32, P, i32, P, P, i32, P, ctypes.c_float, P, P, P, P, sz, P]
    c = _case(31, "bf16", [rows], rows, 1, 8, 4, 64, [600], [20] * rows, 16)
    cu = lambda x: torch.from_numpy(x).cuda()
    ptab, plens, stab, slens = cu(c["ptab"]), cu(c["plens"]), cu(c["stab"]), cu(c["slens"])
    want, lse = _call(ms, dict(c, q=c["q"].flip(0, 1, 2), k=c["k"].flip(0, 1, 2), v=c["v"].flip(0, 1, 2)))
    kv = _kv(c["k"], c["v"])
    need = sz(0)
    assert lib.fs_shared_prefix_attention_workspace_bytes(kv, i32(rows), i32(1), i32(8), i32(1), i32(ptab.shape[1]),
                                                          i32(stab.shape[1]), ctypes.byref(need)) == 0
    ws = torch.empty(max(need.value, 1), dtype=torch.uint8, device="cuda")
    out, got_lse = torch.zeros_like(c["q"]), torch.zeros(rows, 1, 8, device="cuda")
    qa, qs = _backwards(c["q"], 3)
    oa, os_ = _backwards(out, 3)
    torch.cuda.synchronize()
    st = f(kv, qa, _s(qs), rows, 1, 8, None, 1, ptab.data_ptr(), ptab.shape[1], plens.data_ptr(), stab.data_ptr(),
           stab.shape[1], slens.data_ptr(), 64 ** -0.5, oa, _s(os_), got_lse.data_ptr(), ws.data_ptr(), need.value, None)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(out.flip(0, 1, 2), want) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("dim", [64, 36])     # 16-byte words, single elements
def test_appending_over_negative_strides(ms, dim):
    import torch
    P, i32 = ctypes.c_void_p, ctypes.c_int32
    f = ctypes.CDLL(ms.LIB_PATH).fs_append_paged_kv
    f.argtypes = [P, P, P, P, P, i32, P, i32, i32, P, P, P, P, i32, i32, P, P, i32, P, P, P]
    n, H, Hq, page, pages = 9, 2, 4, 4, 6
    mk = lambda *s: torch.randn(s, device="cuda").bfloat16()
    key, value, query, k, v = mk(n, H, dim), mk(n, H, dim), mk(n, Hq, dim), mk(pages, page, H, dim), mk(pages, page, H, dim)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, pos, rows = i([[0, 1, 2], [5, 4, 3]]), i([0, 1, 2, 3, 7, 11, 0, 4, 8]), i([0] * 6 + [1] * 3)
    inv = torch.tensor([1.0, 0.3, 0.1, 0.01, 0.7, 0.2, 0.5, 0.9], device="cuda")
    wk, wv = k.flip(0, 1, 2), v.flip(0, 1, 2)
    want = ms.append_paged_kv(key.flip(0, 1), value.flip(0, 1), wk, wv, table, pos, rows, inv_freq=inv, query=query.flip(0, 1))
    qo = torch.zeros_like(query)
    (ka, ks), (va, vs), (qa, qs), (oa, os_) = [_backwards(t, 2) for t in (key, value, query, qo)]
    torch.cuda.synchronize()
    st = f(_kv(k, v), ka, _s(ks), va, _s(vs), n, table.data_ptr(), 2, 3, rows.data_ptr(), pos.data_ptr(), None,
           inv.data_ptr(), 16, 0, qa, _s(qs), Hq, oa, _s(os_), None)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(k.flip(0, 1, 2), wk) and torch.equal(v.flip(0, 1, 2), wv) and torch.equal(qo.flip(0, 1), want)
