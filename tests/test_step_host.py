"""Host-side checks of the serving-step entries, without a GPU: the C ABI refuses bad arguments before
touching the device, and the binding refuses tensors the kernels cannot read."""
import ctypes

import pytest

from tests.helpers import ensure_built
from tests.test_decode_host import _kv, _s

P, FAKE = ctypes.c_void_p, ctypes.c_void_p(0x1000)   # never dereferenced: every call below is rejected on the host
i32, i64, f32, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import min_sampling_gb300
    lib = min_sampling_gb300.lib
    lib.fs_paged_step_tables.argtypes = [P, P, i32, P, i32, P, i32, P, i32, i32, P, P, P, P, P, P]
    lib.fs_append_paged_kv_normed.argtypes = [P, P, P, P, P, i32, P, i32, i32, P, P, P, P, i32, i32, P, P, i32, P, P, P, P, f32, P]
    lib.fs_paged_chunk_attention.argtypes = [P, P, P, i32, i32, P, i32, i32, P, P, i32, i32, i32, f32, i32, P, P, P, P, sz, P]
    lib.fs_paged_chunk_attention_workspace_bytes.argtypes = [P, i32, i32, i32, i32, i32, P]
    lib.fs_adjust_logits.argtypes = [P, i32, i64, i32, i32, P, i64, i32, P, P, P, P, P, P, P, P, i32, P, i32, P, P, i64, P]
    return min_sampling_gb300


def test_table_arguments(ms):
    def call(lens=FAKE, new=FAKE, R=3, table=FAKE, width=4, free=FAKE, F=8, count=FAKE, page=16, budget=10, starts=FAKE, rows=FAKE,
             pos=FAKE, totals=FAKE, left=FAKE):
        return ms.lib.fs_paged_step_tables(lens, new, R, table, width, free, F, count, page, budget, starts, rows, pos, totals, left, None)
    for bad in (dict(lens=None), dict(new=None), dict(table=None), dict(free=None), dict(count=None), dict(starts=None), dict(rows=None),
                dict(pos=None), dict(totals=None), dict(left=None), dict(R=-1), dict(width=-1), dict(F=-1), dict(page=0), dict(budget=-1)):
        assert call(**bad) == 1, bad
    assert call(width=2 ** 30, page=16) == 2 and call(budget=2 ** 31 - 1) == 2


def test_norm_arguments(ms):
    def call(kv=None, q=FAKE, wq=FAKE, wk=FAKE, eps=1e-6, rotary=64, n=3):
        return ms.lib.fs_append_paged_kv_normed(_kv(ms) if kv is None else kv, FAKE, _s(128, 64), FAKE, _s(128, 64), n, FAKE, 4, 2, FAKE, FAKE,
                                                None, FAKE, rotary, 0, q, _s(256, 64), 4, FAKE, _s(256, 64), wq, wk, eps, None)
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(q=None) == 1
    assert call(rotary=63) == 1 and call(n=-1) == 1 and call(kv=_kv(ms, dtype=7)) == 1 and call(kv=_kv(ms, dim=2048)) == 2
    assert call(n=0) == 0


def test_chunk_arguments(ms):
    def call(kv=None, q=FAKE, qs=_s(256, 64), N=5, hq=4, table=FAKE, R=3, width=4, starts=FAKE, lens=FAKE, most=5, window=0, sinks=0, rest=1,
             out=FAKE, os=_s(256, 64), ws=FAKE, n=0):
        return ms.lib.fs_paged_chunk_attention(_kv(ms) if kv is None else kv, q, qs, N, hq, table, R, width, starts, lens, most, window, sinks,
                                               1.0, rest, out, os, None, ws, n, None)
    for bad in (dict(q=None), dict(qs=None), dict(out=None), dict(os=None), dict(table=None), dict(starts=None), dict(lens=None), dict(N=-1),
                dict(hq=3), dict(hq=0), dict(R=-1), dict(width=-1), dict(most=0), dict(window=-1), dict(sinks=-1), dict(rest=2),
                dict(kv=_kv(ms, dtype=9)), dict(kv=_kv(ms, page=0)), dict(kv=_kv(ms, k=None)), dict(kv=_kv(ms, ks=(2048, 128, 4))),
                dict(qs=_s(256, 60)), dict(out=P(0x1008)), dict(ws=P(0x1008))):
        assert call(**bad) == 1, bad
    assert b"16-byte" in ms.lib.fs_last_error_string()
    assert call(kv=_kv(ms, dtype=0)) == 2 and call(kv=_kv(ms, dim=96)) == 2 and call(width=2 ** 30) == 2
    assert call(N=0, q=None) == 0
    n = sz(7)
    assert ms.lib.fs_paged_chunk_attention_workspace_bytes(_kv(ms), 0, 3, 4, 4, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert ms.lib.fs_paged_chunk_attention_workspace_bytes(_kv(ms), 5, 3, 3, 4, 1, ctypes.byref(n)) == 1
    assert ms.lib.fs_paged_chunk_attention_workspace_bytes(_kv(ms), 5, 3, 4, 4, 1, None) == 1


def test_adjust_arguments(ms):
    def call(x=FAKE, dtype=0, xs=16, B=3, V=16, tok=FAKE, ts=8, L=8, lens=FAKE, prompts=FAKE, rep=FAKE, pres=FAKE, freq=FAKE, bs=FAKE,
             bt=FAKE, bv=FAKE, nb=4, allowed=FAKE, masks=2, rows=FAKE, out=FAKE, os=16):
        return ms.lib.fs_adjust_logits(x, dtype, xs, B, V, tok, ts, L, lens, prompts, rep, pres, freq, bs, bt, bv, nb, allowed, masks, rows, out,
                                       os, None)
    for bad in (dict(x=None), dict(out=None), dict(dtype=3), dict(xs=15), dict(os=15), dict(ts=7), dict(B=-1), dict(V=0), dict(L=-1),
                dict(nb=-1), dict(masks=-1), dict(tok=None), dict(tok=None, lens=None, prompts=None, rep=None, pres=None), dict(bt=None),
                dict(bv=None), dict(bs=None), dict(allowed=None), dict(rows=None), dict(x=P(0x1002)), dict(out=P(0x1001), dtype=1)):
        assert call(**bad) == 1, bad
    assert call(V=2097153, xs=2097153, os=2097153) == 2 and call(L=2 ** 30, ts=2 ** 30) == 2
    assert call(B=0, x=None, out=None) == 0


def test_binding_refuses(ms):
    """Tensors of the wrong type, device, shape or layout (CPU tensors are one of them) never reach the library."""
    import torch
    f, i = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.int32)
    kc = f(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ms.paged_step_tables(i(2), i(2), i(2, 3), i(5), i(1), 16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ms.paged_chunk_attention(f(1, 4, 64), kc, kc, i(1, 1), i(2), i(1))
    with pytest.raises(ValueError, match="4-D"):
        ms.paged_chunk_attention(f(1, 4, 64), kc[0], kc[0], i(1, 1), i(2), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        ms.adjust_logits(f(2, 8))
    with pytest.raises(ValueError, match="2-D"):
        ms.adjust_logits(f(8))
    for bad in (None, 3, "x"):
        with pytest.raises(ValueError):
            ms.paged_step_tables(i(2), i(2), bad, i(5), i(1), 16, 8)
        with pytest.raises(ValueError):
            ms.paged_chunk_attention(f(1, 4, 64), bad, kc, i(1, 1), i(2), i(1))
        with pytest.raises(ValueError):
            ms.adjust_logits(bad)
