"""Host-side checks of the decode-step entries, without a GPU: the C ABI refuses bad arguments before
touching the device, and the binding refuses tensors the kernels cannot read."""
import ctypes
import struct

import pytest

from tests.helpers import ensure_built

P, FAKE = ctypes.c_void_p, ctypes.c_void_p(0x1000)   # never dereferenced: every call below is rejected on the host


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import min_sampling_gb300
    lib, sz, i32 = min_sampling_gb300.lib, ctypes.c_size_t, ctypes.c_int32
    lib.fs_top_k_top_p_sampling_from_uniforms.argtypes = [P, i32, ctypes.c_int64, i32, i32, P, i32, P, P, P, P, P, i32, P, P,
                                                          P, sz, P]
    lib.fs_append_paged_kv.argtypes = [P, P, P, P, P, i32, P, i32, i32, P, P, P, P, i32, i32, P, P, i32, P, P, P]
    lib.fs_shared_prefix_attention.argtypes = [P, P, P, i32, i32, i32, P, i32, P, i32, P, P, i32, P, ctypes.c_float, P, P, P,
                                               P, sz, P]
    return min_sampling_gb300


KV = struct.Struct("@PPiiiii6q")   # fs_paged_kv


def _kv(ms, k=0x1000, v=0x1000, dtype=1, pages=4, page=16, heads=2, dim=64, ks=(2048, 128, 64), vs=(2048, 128, 64)):
    return KV.pack(k or 0, v or 0, dtype, pages, page, heads, dim, *ks, *vs)


def _s(*v):
    return (ctypes.c_int64 * len(v))(*v) if v else None


def test_uniforms_arguments(ms):
    def call(x=FAKE, dtype=0, stride=16, b_in=4, V=16, idx=None, b_out=4, u=FAKE, order=0, tok=FAKE, valid=FAKE, ws=FAKE,
             n=1 << 20):
        return ms.lib.fs_top_k_top_p_sampling_from_uniforms(x, dtype, stride, b_in, V, idx, b_out, u, None, None, None, None,
                                                            order, tok, valid, ws, n, None)
    assert call(x=None) == 1 and call(u=None) == 1 and call(tok=None) == 1 and call(valid=None) == 1
    assert call(ws=None) == 1 and call(n=0) == 1
    assert call(dtype=3) == 1 and call(dtype=-1) == 1 and call(V=0) == 1 and call(V=2097153, stride=2097153) == 2
    assert call(b_out=5) == 1 and call(b_out=-1) == 1 and call(b_in=-1) == 1 and call(order=2) == 1
    assert call(stride=15) == 1
    assert call(x=P(0x1001)) == 1 and call(x=P(0x1001), dtype=1) == 1 and call(ws=P(0x1002)) == 1
    assert call(b_in=0, b_out=0, x=None, u=None) == 0
    n = ctypes.c_size_t(0)
    assert ms.lib.fs_from_uniforms_workspace_bytes(0, 64, 151936, ctypes.byref(n)) == 0
    assert n.value == 64 * 8 * -(-(151936 + 3) // 128)
    assert ms.lib.fs_from_uniforms_workspace_bytes(1, 2, 1, ctypes.byref(n)) == 0 and n.value == 16


def test_append_arguments(ms):
    def call(kv=None, key=FAKE, value=FAKE, n=3, table=FAKE, R=4, w=2, rows=FAKE, pos=FAKE, inv=FAKE, rotary=64, inter=0,
             q=FAKE, hq=4, qo=FAKE, ks=_s(128, 64), qs=_s(256, 64)):
        kv = _kv(ms) if kv is None else kv
        return ms.lib.fs_append_paged_kv(kv, key, ks, value, _s(128, 64), n, table, R, w, rows, pos, None, inv,
                                         rotary, inter, q, qs, hq, qo, _s(256, 64), None)
    assert call(key=None) == 1 and call(value=None) == 1 and call(pos=None) == 1 and call(inv=None) == 1
    assert call(table=None) == 1 and call(ks=None) == 1 and call(qs=None) == 1 and call(qo=None) == 1 and call(hq=0) == 1
    assert call(n=-1) == 1 and call(R=-1) == 1 and call(w=-1) == 1
    assert call(rotary=63) == 1 and call(rotary=66) == 1 and call(rotary=-2) == 1 and call(inter=2) == 1
    assert call(rows=None, R=2) == 1
    assert call(kv=_kv(ms, page=0)) == 1 and call(kv=_kv(ms, heads=0)) == 1 and call(kv=_kv(ms, dim=0)) == 1
    assert call(kv=_kv(ms, dtype=7)) == 1 and call(kv=_kv(ms, k=None)) == 1 and call(kv=_kv(ms, pages=-1)) == 1
    assert call(kv=_kv(ms, dim=2048)) == 2 and call(kv=_kv(ms, heads=5000)) == 2
    assert call(n=0, key=None, value=None, pos=None) == 0


def test_attention_arguments(ms):
    def call(kv=None, q=FAKE, qs=_s(512, 512, 64), B=4, Q=1, hq=4, starts=FAKE, G=2, ptab=FAKE, pw=4, pl=FAKE, stab=FAKE,
             sw=2, sl=FAKE, out=FAKE, os=_s(512, 512, 64)):
        kv = _kv(ms) if kv is None else kv
        return ms.lib.fs_shared_prefix_attention(kv, q, qs, B, Q, hq, starts, G, ptab, pw, pl, stab, sw, sl,
                                                 1.0, out, os, None, FAKE, 0, None)
    assert call(q=None) == 1 and call(out=None) == 1 and call(qs=None) == 1 and call(os=None) == 1
    assert call(ptab=None) == 1 and call(pl=None) == 1 and call(stab=None) == 1 and call(sl=None) == 1
    assert call(starts=None) == 1 and call(B=-1) == 1 and call(Q=0) == 1 and call(hq=3) == 1 and call(hq=0) == 1
    assert call(G=-1) == 1 and call(pw=-1) == 1 and call(sw=-1) == 1
    assert call(kv=_kv(ms, dtype=0)) == 2 and call(kv=_kv(ms, dim=96)) == 2 and call(kv=_kv(ms, dtype=9)) == 1
    assert b"64, 128 or 256" in ms.lib.fs_last_error_string()
    assert call(kv=_kv(ms, ks=(2048, 128, 4))) == 1 and call(kv=_kv(ms, v=0x1008)) == 1
    assert call(qs=_s(512, 512, 60)) == 1 and call(out=P(0x1004)) == 1
    assert b"16-byte" in ms.lib.fs_last_error_string()
    assert call(pw=2 ** 30) == 2
    assert call(B=0, q=None) == 0


def test_binding_refuses(ms):
    """Tensors of the wrong type, device, shape or layout (CPU tensors are one of them) never reach the library."""
    import torch
    f, i = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.int32)
    kc = f(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ms.top_k_top_p_sampling_from_uniforms(f(2, 8), f(2))
    with pytest.raises(ValueError, match="2-D"):
        ms.top_k_top_p_sampling_from_uniforms(f(8), f(1))
    with pytest.raises(ValueError, match="CUDA"):
        ms.append_paged_kv(f(1, 2, 64), f(1, 2, 64), kc, kc, i(1, 1), i(1))
    with pytest.raises(ValueError, match="4-D"):
        ms.append_paged_kv(f(1, 2, 64), f(1, 2, 64), kc[0], kc[0], i(1, 1), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        ms.shared_prefix_attention(f(1, 4, 64), kc, kc, i(1, 1), i(1), i(1, 1), i(1))
    for bad in (None, 3, "x"):
        with pytest.raises(ValueError):
            ms.top_k_top_p_sampling_from_uniforms(bad, f(1))
        with pytest.raises(ValueError):
            ms.append_paged_kv(f(1, 2, 64), f(1, 2, 64), bad, kc, i(1, 1), i(1))
        with pytest.raises(ValueError):
            ms.shared_prefix_attention(f(1, 4, 64), bad, kc, i(1, 1), i(1), i(1, 1), i(1))
    with pytest.raises(ValueError, match="order"):
        ms.top_k_top_p_sampling_from_uniforms(f(2, 8), f(2), order="sideways")
