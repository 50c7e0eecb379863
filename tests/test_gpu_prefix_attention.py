"""Attention over a shared prefix (fs_shared_prefix_attention) against float64.

Tolerance of an output o = sum p_j v_j / l, A = sum p_j |v_j| / l, h = eps(t) / 2:
  h A       the weights enter the product rounded to the type
  h |o|     the output's own rounding
  2 e A     e the relative error of a weight in float32: its score's absolute error, D products
            and sums of size S = scale * max_j sum |q k_j| (D 2^-24 S), the scaling to base 2 (4 * 2^-24 S) and 2^x (2^-21);
            twice, for the sum of the weights; the joins and the sums add (joins + 64) 2^-24, within
            2^-16
  f16 only: a weight below 2^-14 of the largest is rounded to a multiple of 2^-24: up to 2^-25 for each of n
            keys, against a sum of weights l' relative to the largest: n 2^-25 max |v| / l'.
lse: e, plus 2^-22 max(1, |lse|)."""
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


def _case(seed, dtype, groups, rows, Q, Hq, H, D, plens, slens, page, sigma=1.0, spare=3):
    """`groups`: rows per group; `rows` rows in all (the last ones may belong to none)."""
    import torch
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    plens, slens = np.int32(plens), np.int32(slens)
    pp, sp = -(-plens // page), -(-slens // page)
    pages = int(pp.sum() + sp.sum()) + spare
    order = rng.permutation(pages).astype(np.int32)
    ptab = np.full((len(plens), max(int(pp.max(initial=0)), 1)), -1, np.int32)   # entries past the length are never read
    stab = np.full((rows, max(int(sp.max(initial=0)), 1)), -1, np.int32)
    at = 0
    for tab, cnt in ((ptab, pp), (stab, sp)):
        for i, m in enumerate(cnt):
            tab[i, :m] = order[at:at + m]
            at += int(m)
    mk = lambda *s: (torch.randn(s, generator=g) * sigma).to(dt).cuda()
    starts = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    return dict(q=mk(rows, Q, Hq, D), k=mk(pages, page, H, D), v=mk(pages, page, H, D), ptab=ptab, plens=plens, stab=stab,
                slens=slens, starts=starts)


def _call(ms, c, **kw):
    import torch
    cu = lambda x: None if x is None else torch.from_numpy(x).cuda()
    none = len(c["plens"]) == 0
    return ms.shared_prefix_attention(c["q"], c["k"], c["v"], None if none else cu(c["ptab"]), None if none else cu(c["plens"]),
                                      cu(c["stab"]), cu(c["slens"]), None if none else cu(c["starts"]), return_lse=True, **kw)


def _check(ms, c, scale=None, rows=None, **kw):
    import torch
    out, lse = _call(ms, c, scale=scale, **kw)
    D, Q, gs = c["q"].shape[-1], c["q"].shape[1], c["q"].shape[2] // c["k"].shape[2]
    sc = D ** -0.5 if scale is None else scale
    f = lambda t: t.float().cpu().numpy()
    kn, vn = f(c["k"]), f(c["v"])
    o, l, A, big, rel = decode.attend(f(c["q"]), kn, vn, c["ptab"], c["plens"], c["stab"], c["slens"], c["starts"], sc)
    h = torch.finfo(c["q"].dtype).eps / 2
    e = big * (D + 4) * 2.0 ** -24 + 2.0 ** -16
    tol = h * A + h * np.abs(o) + (2 * e)[..., None] * A
    if c["q"].dtype == torch.float16:
        n = (max(c["plens"], default=0) + c["slens"].max(initial=0))
        tol += (n * 2.0 ** -25 * np.abs(vn).max() / rel)[..., None]
    got, gl = f(out).astype(np.float64), f(lse).astype(np.float64)
    sel = slice(None) if rows is None else rows
    bad = ~(np.abs(got - o) <= tol)
    assert not bad[sel].any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4], tol[bad][:4])
    empty = np.isneginf(l)
    assert (np.isneginf(gl) == empty)[sel].all()
    gl, l = np.where(empty, 0, gl), np.where(empty, 0, l)
    assert (np.abs(gl - l) <= e + 2.0 ** -22 * np.maximum(1, np.abs(l)))[sel].all()
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (8, 8), (8, 2), (10, 2), (7, 1), (32, 2)])
def test_head_layouts(ms, dtype, D, heads):
    Hq, H = heads
    _check(ms, _case(1, dtype, [5], 5, 1, Hq, H, D, [300], [1, 63, 64, 65, 130], 16))


@pytest.mark.parametrize("page", [1, 5, 16, 64, 100])
@pytest.mark.parametrize("plen", [0, 1, 15, 16, 17, 63, 64, 65, 255, 257, 1000])
def test_lengths_and_pages(ms, page, plen):
    _check(ms, _case(plen + page, "bf16", [3], 3, 1, 4, 2, 64, [plen], [0, 1, 70], page))
    _check(ms, _case(plen + page, "f16", [3], 3, 2, 4, 2, 128, [plen], [2, 33, 64], page))


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 8, 9, 16, 17, 33, 70, 130])
def test_batch_sizes(ms, rows):
    """Every tile size, full and ragged."""
    rng = np.random.default_rng(rows)
    for D in (64, 128):
        _check(ms, _case(rows, "bf16", [rows], rows, 1, 8, 2, D, [777], rng.integers(1, 40, rows), 16))


@pytest.mark.parametrize("Q", [1, 2, 5, 8, 33])
def test_several_tokens_a_row(ms, Q):
    """Causal among a row's own tokens; suffixes shorter than Q leave early queries with less."""
    _check(ms, _case(Q, "bf16", [2, 3], 5, Q, 8, 2, 64, [130, 64], [Q, Q + 1, 64 + Q, max(Q - 1, 0), 0], 16))
    _check(ms, _case(Q, "f16", [2], 2, Q, 4, 4, 128, [0], [Q, max(Q - 2, 0)], 5))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("plen", [40, 2100, 9000])
def test_wide_heads(ms, dtype, plen):
    """Heads of 256: tiles of 16, 32 and 64 queries, few key ranges (tiles of 64 keys) and many (of 32)."""
    rng = np.random.default_rng(plen)
    for rows, Q in ((1, 1), (4, 1), (7, 1), (18, 1), (3, 5), (6, 5), (40, 2)):
        _check(ms, _case(plen + rows, dtype, [rows], rows, Q, 16, 4, 256, [plen], rng.integers(0, 300, rows), 16))
    _check(ms, _case(plen, dtype, [2, 5, 0, 30], 40, 1, 8, 2, 256, [plen, 31, 7, 65], rng.integers(0, 70, 40), 5))


@pytest.mark.parametrize("rows", [1, 90])
def test_wide_heads_unseen_values(ms, rows):
    """NaN and infinite values in tokens behind a query's own, at the border of a tile of keys."""
    import torch
    Q = 5
    for length in (32, 34, 64, 66, 97):
        c = _case(length, "bf16", [rows], rows, Q, 8, 2, 256, [100], [length] * rows, 16)
        want = _check(ms, c)[0][:, :Q - 2].clone()
        for b in range(rows):
            for t, x in ((length - 1, float("nan")), (length - 2, float("inf"))):
                c["v"][int(c["stab"][b, t // 16]), t % 16] = x
        assert torch.equal(_call(ms, c)[0][:, :Q - 2], want)


def test_groups_of_every_size(ms):
    """Empty groups, empty prefixes, rows of no group, many groups."""
    _check(ms, _case(1, "bf16", [3, 0, 1, 4], 10, 1, 8, 2, 128, [500, 10, 0, 65], [1, 2, 3, 4, 5, 6, 7, 8, 0, 64], 16))
    n = 70
    _check(ms, _case(2, "bf16", [1] * n, n, 1, 4, 1, 64, [3 * i for i in range(n)], [i % 5 for i in range(n)], 16))
    c = _case(3, "bf16", [2, 2], 6, 1, 4, 1, 64, [100, 50], [3] * 6, 16)
    c["starts"] = np.int32([1, 3, 5])      # rows 0 and 5 have no prefix
    _check(ms, c)
    _check(ms, _case(4, "f16", [], 5, 1, 4, 2, 64, [], [0, 1, 64, 100, 7], 16))
    c = _case(5, "bf16", [4], 4, 1, 4, 2, 64, [200], [0, 0, 0, 0], 16)
    _check(ms, c)


def test_long_prefix_and_scores_of_every_size(ms):
    for sigma, scale in ((1.0, None), (4.0, None), (1.0, 0.0), (1.0, -0.3), (0.05, None)):
        for rows in (3, 40, 150):
            _check(ms, _case(9, "bf16", [rows], rows, 1, 4, 1, 128, [5000], [20] * rows, 16, sigma), scale=scale)


def test_many_rows_of_one_prefix(ms):
    """Tiles of 64 queries and more per key/value head."""
    rng = np.random.default_rng(3)
    for dtype, D, Hq, H in (("bf16", 128, 8, 2), ("f16", 64, 8, 8), ("bf16", 64, 12, 2)):
        _check(ms, _case(6, dtype, [90, 61], 151, 1, Hq, H, D, [1500, 900], rng.integers(0, 90, 151), 16))


def test_views_and_outputs(ms):
    """Pages laid out heads first, keys and values in one tensor, a strided query and a strided output."""
    import torch
    c = _case(7, "bf16", [4], 4, 2, 8, 2, 64, [100], [5, 9, 70, 2], 16)
    both = torch.stack([c["k"], c["v"]], 1).transpose(2, 3).contiguous().transpose(2, 3)
    c["k"], c["v"] = both[:, 0], both[:, 1]
    wide = torch.zeros(4, 2, 8, 192, dtype=torch.bfloat16, device="cuda")
    wide[..., 64:128] = c["q"]
    c["q"] = wide[..., 64:128]
    res = torch.full((4, 2, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, _ = _check(ms, c, out=res[..., 64:])
    assert out.data_ptr() == res[..., 64:].data_ptr() and bool((res[..., :64] == 7).all())
    one = dict(c, q=c["q"][:, 0])
    out1, lse1 = _call(ms, one)
    assert out1.shape == (4, 8, 64) and lse1.shape == (4, 8)


def test_what_a_query_does_not_see_does_not_reach_it(ms):
    """NaN and infinities behind the lengths, in unused pages, and in the tokens that come after a query."""
    for rows in (3, 50):
        c = _case(8, "bf16", [rows], rows, 3, 4, 2, 64, [100], [3 + i % 20 for i in range(rows)], 16, spare=5)
        clean, _ = _check(ms, c)
        used = set()
        for tab, lens in ((c["ptab"], c["plens"]), (c["stab"], c["slens"])):
            for i, n in enumerate(lens):
                used |= {(int(tab[i, t // 16]), t % 16) for t in range(n)}
        free = np.array([[(pg, s) not in used for s in range(16)] for pg in range(c["k"].shape[0])])
        import torch
        mask = torch.from_numpy(free).cuda()
        c["k"][mask], c["v"][mask] = float("nan"), float("inf")
        out, _ = _call(ms, c)
        assert torch.equal(out, clean)
        # the last token of rows 0 and 1: only their last query sees it
        for b in (0, 1):
            t = int(c["slens"][b]) - 1
            pg = int(c["stab"][b, t // 16])
            c["v"][pg, t % 16] = float("inf") if b == 0 else float("nan")
            c["k"][pg, t % 16, 0] = float("nan")
        out, lse = _call(ms, c)
        for b in (0, 1):
            assert torch.equal(out[b, :2], clean[b, :2])
            assert not torch.isfinite(out[b, 2]).any()
        assert torch.equal(out[2:], clean[2:])


def test_pages_that_do_not_exist_show_as_nan(ms):
    import torch
    for rows in (3, 60):
        c = _case(10, "bf16", [rows - 1, 1], rows, 1, 4, 2, 64, [200, 40], [70] * rows, 16)
        clean, _ = _check(ms, c)
        c["stab"][1, 2], c["ptab"][1, 1] = c["k"].shape[0], -7
        out, lse = _call(ms, c)
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
        assert torch.isnan(out[rows - 1]).all()
        keep = [i for i in range(rows - 1) if i != 1]
        assert torch.equal(out[keep], clean[keep])


def test_lengths_beyond_the_tables_are_clamped(ms):
    import torch
    c = _case(11, "bf16", [3], 3, 1, 4, 2, 64, [160], [32, 32, 32], 16)
    clean, _ = _check(ms, c)
    c["plens"], c["slens"] = np.int32([2 ** 31 - 1]), np.int32([2 ** 31 - 1, 33, 32])
    out, _ = _call(ms, c)
    assert torch.equal(out, clean)
    c["plens"], c["slens"] = np.int32([-1]), np.int32([-5, -2 ** 31, 0])
    out, lse = _call(ms, c)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_no_pages_at_all(ms):
    import torch
    k = torch.zeros(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    out, lse = ms.shared_prefix_attention(q, k, k, z(1, 0), z(1), z(2, 0), z(2), return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    out = ms.shared_prefix_attention(q[:0], k, k, None, None, z(0, 0), z(0))
    assert out.shape == (0, 4, 64)


def test_offsets_past_32_bits(ms):
    """A cache of more than 2^31 elements whose used pages lie at its end."""
    import torch
    page, H, D = 64, 8, 128
    pages = 2 ** 31 // (page * H * D) + 20
    c = _case(12, "bf16", [4], 4, 1, 8, 8, 128, [200], [10, 64, 65, 3], page)
    small = c["k"].shape[0]
    k = torch.zeros(pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[pages - small:], v[pages - small:] = c["k"], c["v"]
    want, _ = _check(ms, c)
    far = dict(c, k=k, v=v, ptab=c["ptab"] + (pages - small), stab=np.where(c["stab"] >= 0, c["stab"] + pages - small, -1).astype(np.int32))
    out, _ = _call(ms, far)
    assert torch.equal(out, want)


def test_the_same_bits_every_time_captured_and_on_two_streams(ms):
    import torch
    cs = [_case(20 + i, "bf16", [20], 20, 1, 8, 2, 128, [3000], [50] * 20, 16) for i in range(2)]
    want = [_call(ms, c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(8):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                got[i].append(_call(ms, c))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1]) for g in got[i])
    # two graphs captured on one stream, replayed at the same time on two others, with new lengths
    cu = lambda x: torch.from_numpy(x).cuda()
    dev = [dict(c, **{n: cu(c[n]) for n in ("ptab", "plens", "stab", "slens", "starts")}) for c in cs]
    call = lambda d: ms.shared_prefix_attention(d["q"], d["k"], d["v"], d["ptab"], d["plens"], d["stab"], d["slens"],
                                                d["starts"])
    graphs, outs = [], []
    for d in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(d))
        graphs.append(g)
    for plen in (3000, 1, 0, 1777):
        for d in dev:
            d["plens"].fill_(plen)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for d, o in zip(dev, outs):
            assert torch.equal(o, call(d))


def test_a_prefix_without_pages_shows_as_nan(ms):
    import torch
    k = torch.zeros(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    for rows in (2, 40):
        q = torch.randn(rows, 4, 64, device="cuda").bfloat16()
        out = ms.shared_prefix_attention(q, k, k, z(1, 40), z(1) + 600, z(rows, 1), z(rows))
        assert bool(torch.isnan(out).all())


def test_refusals(ms):
    import torch
    c = _case(13, "bf16", [2, 2], 4, 1, 8, 2, 64, [100, 30], [5, 9, 70, 2], 16)
    cu = lambda x: torch.from_numpy(x).cuda()
    good = dict(query=c["q"], k_cache=c["k"], v_cache=c["v"], prefix_table=cu(c["ptab"]), prefix_lens=cu(c["plens"]),
                suffix_table=cu(c["stab"]), suffix_lens=cu(c["slens"]), group_starts=cu(c["starts"]))
    f = ms.shared_prefix_attention
    for bad in (dict(query=c["q"].half()), dict(query=c["q"][..., :32]), dict(query=c["q"][:, :, :3]), dict(query=c["q"][:, :0]),
                dict(query=c["q"][0, 0]), dict(query=c["q"].cpu()), dict(k_cache=c["k"][..., ::2], v_cache=c["v"][..., ::2]),
                dict(v_cache=c["v"][:3]), dict(prefix_table=cu(c["ptab"]).long()), dict(prefix_table=None),
                dict(prefix_lens=cu(c["plens"])[:1]), dict(prefix_lens=None), dict(suffix_table=cu(c["stab"])[:3]),
                dict(suffix_lens=cu(c["slens"])[:3]), dict(suffix_lens=torch.from_numpy(c["slens"])), dict(suffix_table=None),
                dict(group_starts=cu(c["starts"])[:2]), dict(group_starts=None), dict(out=c["q"][:2]), dict(out=c["q"].half())):
        with pytest.raises(ValueError):
            f(**{**good, **bad})
    wide = torch.zeros(4, 1, 8, 68, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ms.FsError):      # a stride of 136 bytes
        f(**{**good, "query": wide[..., :64]})
    with pytest.raises(ms.FsError):      # float32, and heads of 32
        f(**{**good, "query": c["q"].float(), "k_cache": c["k"].float(), "v_cache": c["v"].float()})
    with pytest.raises(ms.FsError):
        f(**{**good, **{n: good[n][..., :32].contiguous() for n in ("query", "k_cache", "v_cache")}})


def test_gradients_and_shared_memory_are_refused(ms):
    """No gradient is lost without a word, no output whose elements share memory is written."""
    import torch
    c = _case(13, "bf16", [4], 4, 1, 8, 2, 64, [100], [5, 9, 70, 2], 16)
    want, _ = _call(ms, c)
    for name in ("q", "k", "v"):
        bad = dict(c, **{name: c[name].clone().requires_grad_()})
        with pytest.raises(ValueError, match="no backward"):
            _call(ms, bad)
        with torch.no_grad():
            assert torch.equal(_call(ms, bad)[0], want)
        assert torch.equal(_call(ms, dict(c, **{name: bad[name].detach()}))[0], want)
    with pytest.raises(ValueError, match="share memory"):
        _call(ms, c, out=c["q"][:1].clone().expand_as(c["q"]))
    assert torch.equal(_call(ms, dict(c, q=c["q"].clone()), out=torch.empty_like(c["q"]))[0], want)
    shared = dict(c, q=c["q"][:1].expand_as(c["q"]))     # reading a broadcast query is fine
    assert torch.equal(_call(ms, shared)[0], _call(ms, dict(c, q=shared["q"].contiguous()))[0])
