"""Appending to a paged cache with the rotation (fs_append_paged_kv) against float64.

Tolerance of a rotated element x cos a - y sin a of type t: half a step of the rounding to t,
eps(t) / 2 of the result, and the float32 arithmetic before it: sine and cosine to 2 units (2^-22),
two products and a sum (3 roundings, 2^-24 each), the angle to 2^-33 turns and its float32 form to
2^-24 of itself (pi 2^-24): (|x| + |y|) * 2^-20 covers their sum.  Copies are exact."""
import numpy as np
import pytest

from oracle import decode
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _np(t):
    return t.double().cpu().numpy()


def _inv(half, base=10000.0):
    return (base ** (-np.arange(half) / max(half, 1))).astype(np.float32)


def _case(seed, dtype, n, H, Hq, D, page, pages, width, R):
    import torch
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(s, generator=g).to(_dt(dtype)).cuda()
    rng = np.random.default_rng(seed)
    table = rng.permutation(pages)[: R * width].reshape(R, width).astype(np.int32)
    # distinct places, a few rows' worth, in any order
    slots = rng.permutation(R * width * page)[:n]
    rows, pos = (slots // (width * page)).astype(np.int32), (slots % (width * page)).astype(np.int32)
    return dict(key=mk(n, H, D), value=mk(n, H, D), query=mk(n, Hq, D) if Hq else None, k=mk(pages, page, H, D),
                v=mk(pages, page, H, D), table=table, rows=rows, pos=pos)


def _check(ms, c, inv, interleaved, rpos=None, rows="given", views=None, query_out=None):
    import torch
    cu = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    eps = torch.finfo(c["key"].dtype).eps
    rows_np = c["rows"] if rows == "given" else None
    want = decode.append(_np(c["key"]), _np(c["value"]), _np(c["k"]), _np(c["v"]), c["table"], c["pos"], rows_np, rpos,
                         [] if inv is None else inv, interleaved, None if c["query"] is None else _np(c["query"]))
    mag = lambda x: np.abs(_np(x)).max(-1, keepdims=True) * 2
    q_in = None if c["query"] is None else c["query"].clone()
    before_k, before_v = _np(c["k"]), _np(c["v"])
    k_view, v_view = views or (c["k"], c["v"])
    q = ms.append_paged_kv(c["key"], c["value"], k_view, v_view, cu(c["table"]), cu(c["pos"]), cu(rows_np),
                           rotary_positions=cu(rpos), inv_freq=cu(inv), interleaved=interleaved, query=c["query"],
                           query_out=query_out)
    kc, vc, qw, wrote = want
    gk, gv = _np(c["k"]), _np(c["v"])
    assert (gv == vc).all()
    keep = np.ones(gk.shape[:2], bool)
    for pg, s in wrote:
        keep[pg, s] = False
    assert (gk[keep] == before_k[keep]).all() and (gv[keep] == before_v[keep]).all()
    top = float(mag(c["key"]).max()) if c["key"].numel() else 0.0
    assert (np.abs(gk - kc) <= eps / 2 * np.abs(kc) + top * 2.0 ** -20).all()
    if q is not None:
        assert (np.abs(_np(q) - qw) <= eps / 2 * np.abs(qw) + mag(q_in) * 2.0 ** -20).all()
        skipped = c["pos"] < 0
        assert torch.equal(q[cu(skipped)], q_in[cu(skipped)])
    return q


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (7, 2, 8, 128, 128), (130, 8, 32, 128, 64), (33, 3, 3, 80, 32),
                                   (5, 1, 0, 128, 0), (9, 5, 10, 30, 18), (4, 2, 4, 256, 256), (3, 64, 128, 16, 16),
                                   (2, 1, 1, 1024, 1024), (6, 1, 2, 1, 0)])
def test_shapes(ms, dtype, interleaved, shape):
    n, H, Hq, D, rotary = shape
    for page in (1, 5, 16):
        c = _case(n + page, dtype, n, H, Hq, D, page, 400, 40, 4)
        _check(ms, c, _inv(rotary // 2) if rotary else None, interleaved)


def test_far_positions_and_frequencies(ms):
    """Angles at positions up to 2^31 - 1 and frequencies from 0 to above 1, signs included."""
    n = 12
    rpos = np.int32([0, 1, 127, 4095, 131071, 10 ** 6, 16777217, 2 ** 30 + 1, 2 ** 31 - 1, -1, -5, -2 ** 31])
    for inv in (_inv(32), np.float32(list(_inv(28)) + [0.0, -0.5, 3.0, 100.0]), _inv(32, 5e6)):
        c = _case(3, "f32", n, 2, 3, 64, 16, 64, 8, 4)
        _check(ms, c, inv, False, rpos=rpos)


def test_frequency_that_is_not_finite_shows(ms):
    c = _case(4, "f32", 2, 1, 1, 8, 4, 16, 4, 2)
    import torch
    inv = torch.tensor([1.0, float("inf"), float("nan"), 0.5], device="cuda")
    cu = lambda x: torch.from_numpy(x).cuda()
    q = ms.append_paged_kv(c["key"], c["value"], c["k"], c["v"], cu(c["table"]), cu(c["pos"]), cu(c["rows"]),
                           inv_freq=inv, query=c["query"])
    assert torch.isnan(q[..., [1, 2, 5, 6]]).all() and torch.isfinite(q[..., [0, 3, 4, 7]]).all()


def test_padding_and_places_that_do_not_exist(ms):
    """Negative positions, rows and pages out of range, positions beyond the table: not written."""
    c = _case(5, "bf16", 12, 2, 4, 64, 16, 64, 8, 4)
    c["pos"][[0, 5]] = [-1, -2 ** 31]
    c["pos"][1] = 8 * 16            # beyond the table
    c["pos"][2] = 2 ** 31 - 1
    c["rows"][3], c["rows"][4], c["rows"][6] = -1, 4, 2 ** 31 - 1
    c["table"][c["rows"][7], c["pos"][7] // 16] = 64
    c["table"][c["rows"][8], c["pos"][8] // 16] = -3
    _check(ms, c, _inv(32), False)
    c = _case(6, "bf16", 4, 2, 4, 64, 16, 64, 8, 4)
    c["pos"][:] = -1
    _check(ms, c, _inv(32), True)


def test_strides_layouts_and_in_place(ms):
    import torch
    for dtype in ("bf16", "f32"):
        c = _case(7, dtype, 10, 4, 8, 64, 16, 64, 8, 4)
        # one fused projection [N, (Hq + 2 H) * D]; pages laid out heads first; keys and values in one tensor
        qkv = torch.cat([c["query"].flatten(1), c["key"].flatten(1), c["value"].flatten(1)], 1)
        c["query"], c["key"], c["value"] = [x.view(10, -1, 64) for x in qkv.split([512, 256, 256], 1)]
        both = torch.stack([c["k"], c["v"]], 1).transpose(2, 3).contiguous().transpose(2, 3)
        c["k"], c["v"] = both[:, 0], both[:, 1]
        out = c["query"]  # rotated in place
        q = _check(ms, c, _inv(32), False, query_out=out)
        assert q is out
        # odd strides and addresses: single elements
        c = _case(8, dtype, 10, 4, 8, 64, 16, 64, 8, 4)
        wide = torch.zeros(10, 4, 67, dtype=c["key"].dtype, device="cuda")
        wide[..., 3:] = c["key"]
        c["key"] = wide[..., 3:]
        _check(ms, c, _inv(32), True)


def test_rows_default_to_the_token(ms):
    c = _case(9, "f16", 4, 2, 4, 64, 16, 64, 8, 4)
    _check(ms, c, _inv(16), False, rows=None)
    import torch
    empty = _case(10, "f16", 0, 2, 4, 64, 16, 64, 8, 4)
    assert _check(ms, empty, _inv(16), False).shape == (0, 4, 64)


def test_offsets_past_32_bits(ms):
    """A cache of more than 2^31 elements: pages at its end."""
    import torch
    page, H, D = 64, 8, 128
    pages = 2 ** 31 // (page * H * D) + 9
    k = torch.zeros(pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    key, val = (torch.randn(3, H, D, device="cuda").bfloat16() for _ in range(2))
    table = torch.tensor([[pages - 1, 0], [pages - 8, 1], [2, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([63, 5, 70], dtype=torch.int32, device="cuda")
    ms.append_paged_kv(key, val, k, v, table, pos)
    for t, (pg, s) in enumerate([(pages - 1, 63), (pages - 8, 5), (pages - 2, 6)]):
        assert torch.equal(k[pg, s], key[t]) and torch.equal(v[pg, s], val[t])
    assert int((k != 0).sum()) == int((key != 0).sum()) and int((v != 0).sum()) == int((val != 0).sum())


def test_captured_and_replayed(ms):
    import torch
    c = _case(11, "bf16", 6, 2, 4, 64, 16, 64, 8, 4)
    cu = lambda x: torch.from_numpy(x).cuda()
    table, rows, pos, inv = cu(c["table"]), cu(c["rows"]), cu(c["pos"]), cu(_inv(32))
    ref = [c["k"].clone(), c["v"].clone()]
    call = lambda k, v: ms.append_paged_kv(c["key"], c["value"], k, v, table, pos, rows, inv_freq=inv, query=c["query"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = call(c["k"], c["v"])
    for step in range(3):
        pos.copy_((pos + 17) % 128)
        g.replay()
        want = call(*ref)
        assert torch.equal(q, want) and torch.equal(c["k"], ref[0]) and torch.equal(c["v"], ref[1])


def test_refusals(ms):
    import torch
    c = _case(12, "bf16", 4, 2, 4, 64, 16, 64, 8, 4)
    cu = lambda x: torch.from_numpy(x).cuda()
    good = dict(key=c["key"], value=c["value"], k_cache=c["k"], v_cache=c["v"], page_table=cu(c["table"]),
                positions=cu(c["pos"]), rows=cu(c["rows"]), inv_freq=cu(_inv(32)), query=c["query"])
    before = c["k"].clone(), c["v"].clone()
    f = ms.append_paged_kv
    for bad in (dict(key=c["key"].half()), dict(key=c["key"][:3]), dict(key=c["key"][..., ::2]), dict(value=c["value"][:, :1]),
                dict(v_cache=c["v"][:5]), dict(k_cache=c["k"].cpu()), dict(k_cache=c["k"].double(), v_cache=c["v"].double()),
                dict(k_cache=c["k"].transpose(2, 3), v_cache=c["v"].transpose(2, 3)), dict(page_table=cu(c["table"]).long()),
                dict(page_table=cu(c["table"])[:, ::2]), dict(page_table=torch.from_numpy(c["table"])),
                dict(positions=cu(c["pos"])[:2]), dict(positions=cu(c["pos"]).long()), dict(rows=cu(c["rows"]).cpu()),
                dict(rows=None, page_table=cu(c["table"])[:3]), dict(inv_freq=cu(_inv(33))), dict(inv_freq=cu(_inv(32)).double()),
                dict(inv_freq=cu(_inv(32))[None]), dict(rotary_positions=cu(c["pos"])[:1]), dict(query=c["query"][..., :32]),
                dict(query=c["query"][:, :0]), dict(query_out=c["query"][:2]), dict(query=None, query_out=c["query"])):
        with pytest.raises(ValueError):
            f(**{**good, **bad})
    assert torch.equal(c["k"], before[0]) and torch.equal(c["v"], before[1])


def test_gradients_and_shared_memory_are_refused(ms):
    """No gradient is lost without a word, no cache or output whose elements share memory is written."""
    import torch
    mk = lambda *s: torch.randn(s, device="cuda")
    t = dict(key=mk(3, 2, 64), value=mk(3, 2, 64), k_cache=mk(4, 8, 2, 64), v_cache=mk(4, 8, 2, 64),
             page_table=torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous(),
             positions=torch.tensor([0, 5, 7], dtype=torch.int32, device="cuda"), query=mk(3, 4, 64))
    kept = t["k_cache"].clone(), t["v_cache"].clone()
    for name in ("key", "value", "k_cache", "v_cache", "query"):
        bad = dict(t, **{name: t[name].clone().requires_grad_()})
        with pytest.raises(ValueError, match="no backward"):
            ms.append_paged_kv(**bad)
    for name in ("k_cache", "v_cache"):
        with pytest.raises(ValueError, match="share memory"):
            ms.append_paged_kv(**dict(t, **{name: t[name][:1].expand_as(t[name])}))
    with pytest.raises(ValueError, match="share memory"):
        ms.append_paged_kv(**t, query_out=t["query"][:, :1].expand_as(t["query"]))
    assert torch.equal(t["k_cache"], kept[0]) and torch.equal(t["v_cache"], kept[1])
    with torch.no_grad():
        q = ms.append_paged_kv(**dict(t, key=t["key"].clone().requires_grad_()))
    assert torch.equal(q, t["query"])
    for i, p in enumerate((0, 5, 7)):
        assert torch.equal(t["k_cache"][i, p], t["key"][i]) and torch.equal(t["v_cache"][i, p], t["value"][i])
