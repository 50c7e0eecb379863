"""Attention of chunks over a paged cache (fs_paged_chunk_attention) against float64.

Tolerance of an output o = sum p_j v_j, A = sum p_j |v_j|, h = eps(t) / 2, as for attention over shared prefixes:
  h A       the weights enter the product rounded to the type
  h |o|     the output's own rounding
  2 e A     e the relative error of a weight in float32: its score's absolute error, (D + 4) 2^-24 of
            S = scale * max_j sum |q k_j|, and 2^x, the joins and the sums within 2^-16; twice, for the sum of the weights
  f16 only: a weight below 2^-14 of the largest is rounded to a multiple of 2^-24: up to 2^-25 for each of n
            keys, against a sum of weights l' relative to the largest: n 2^-25 max |v| / l'.
lse: e, plus 2^-22 max(1, |lse|)."""
import numpy as np
import pytest

from oracle import serving
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


def case(seed, dtype, new, lens, Hq, H, D, page, sigma=1.0, spare=3, lead=0, tail=0):
    """Requests of `lens` tokens, the last `new` of them queries; rows of no request before and behind."""
    import torch
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    new, lens = np.int32(new), np.int32(lens)
    need = -(-lens // page)
    pages = int(need.sum()) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(int(need.max(initial=0)), 1)), -1, np.int32)   # entries past the length are never read
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += int(m)
    mk = lambda *s: (torch.randn(s, generator=g) * sigma).to(dt).cuda()
    starts = (lead + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
    return dict(q=mk(int(starts[-1]) + tail, Hq, D), k=mk(pages, page, H, D), v=mk(pages, page, H, D), table=table, starts=starts,
                lens=lens)


def call(ms, c, **kw):
    import torch
    cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return ms.paged_chunk_attention(c["q"], c["k"], c["v"], cu(c["table"]), cu(c["starts"]), cu(c["lens"]), return_lse=True, **kw)


def check(ms, c, scale=None, window=None, sinks=0, rows=None, **kw):
    import torch
    out, lse = call(ms, c, scale=scale, window=window, sinks=sinks, **kw)
    D = c["q"].shape[-1]
    lens = np.clip(c["lens"], 0, c["table"].shape[1] * c["k"].shape[1])
    o, l, A, big, rel = serving.chunk_attention(c["q"], c["k"], c["v"], c["table"], c["starts"], lens, window, sinks,
                                                D ** -0.5 if scale is None else scale)
    h = torch.finfo(c["q"].dtype).eps / 2
    e = big * (D + 4) * 2.0 ** -24 + 2.0 ** -16
    tol = h * A + h * o.abs() + (2 * e)[..., None] * A
    if c["q"].dtype == torch.float16:
        tol += (int(lens.max(initial=0)) * 2.0 ** -25 * c["v"].double().abs().max() / rel)[..., None]
    got, gl = out.double(), lse.double()
    sel = slice(None) if rows is None else rows
    bad = ~((got - o).abs() <= tol)
    assert not bool(bad[sel].any()), (torch.argwhere(bad)[:4], got[bad][:4], o[bad][:4], tol[bad][:4])
    empty = torch.isneginf(l)
    assert torch.equal(torch.isneginf(gl)[sel], empty[sel])
    ok = torch.where(empty, True, (gl - l).abs() <= e + 2.0 ** -22 * l.abs().clamp(min=1))
    assert bool(ok[sel].all())
    return out, lse


KINDS = {"one token": ([1] * 5, [1, 63, 64, 65, 300]), "few": ([2, 3, 1], [2, 70, 129]), "chunks": ([130, 40, 1, 300], [130, 500, 77, 301])}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (8, 8), (8, 2), (10, 2), (7, 1), (32, 2), (40, 2), (24, 1), (130, 1)])
@pytest.mark.parametrize("kind", KINDS)
def test_head_layouts(ms, dtype, D, heads, kind):
    check(ms, case(1, dtype, *KINDS[kind], *heads, D, 16))


@pytest.mark.parametrize("page", [1, 3, 4, 5, 8, 16, 32, 64, 100, 128, 256])
@pytest.mark.parametrize("n", [1, 4, 33, 150])
def test_lengths_and_pages(ms, page, n):
    """Lengths around the borders of tiles and pages; no context, some, more queries than tokens."""
    lens = [n, n + 1, n + 14, n + 63, n + 64, n + 65, n + 127, n + 128, n + 129, n + 500, max(n - 2, 0), 0]
    check(ms, case(n + page, "bf16", [n] * len(lens), lens, 4, 2, 64, page))
    check(ms, case(n + page, "f16", [n] * 4, lens[4:8], 8, 2, 128, page))


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 128, 500])
@pytest.mark.parametrize("sinks", [0, 1, 4, 64, 130, 2000])
def test_windows_and_sinks(ms, window, sinks):
    for D, H in ((64, 2), (128, 1)):
        check(ms, case(window, "bf16", [1, 1, 3, 70, 300], [900, 40, 333, 800, 300], 4, H, D, 16), window=window, sinks=sinks)
    check(ms, case(window, "f16", [1, 90, 5], [900, 640, 20], 4, 2, 256, 16), window=window, sinks=sinks)


def test_window_borders(ms):
    """Windows that end at, before and behind the borders of tiles, for single tokens and chunks."""
    for n in (1, 140):
        for window in (126, 127, 128, 129, 255, 256, 257):
            check(ms, case(n, "bf16", [n] * 4, [n + 255, n + 256, n + 257, n + 600], 8, 2, 64, 16), window=window, sinks=3)


@pytest.mark.parametrize("gs", [1, 3, 4, 16, 17, 64])
def test_query_tiles(ms, gs):
    """Rows of one tile of 16, just more, whole and ragged tiles of 128 and 256."""
    for n in (1, 2, 16 // gs + 1, 128 // gs + 1, 256 // gs, 256 // gs + 1, 600 // gs + 1):
        if n > 0:
            check(ms, case(gs + n, "bf16", [n, 1], [n + 100, 300], gs, 1, 128, 16))


def test_many_requests(ms):
    rng = np.random.default_rng(3)
    new = np.where(rng.random(700) < 0.1, rng.integers(0, 60, 700), 1)
    check(ms, case(3, "bf16", new, new + rng.integers(0, 200, 700), 4, 2, 64, 16))
    check(ms, case(4, "f16", new[:90], new[:90] + rng.integers(0, 900, 90), 8, 8, 128, 16), max_queries=60)


def test_long_contexts_cut_into_ranges(ms):
    """One tile over many CTAs: a few rows and many, the joins of up to 300 parts."""
    for D in (64, 128, 256):
        check(ms, case(5, "bf16", [1], [40000], 4, 1, D, 16))
        check(ms, case(6, "bf16", [30, 1], [20000, 9000], 4, 1, D, 64))
    check(ms, case(7, "f16", [300], [9001], 8, 4, 128, 16))


@pytest.mark.parametrize("hint", [1, 4, 5, 100, None])
def test_the_hint_does_not_change_what_is_answered(ms, hint):
    c = case(8, "bf16", [1, 90, 4, 2], [50, 90, 300, 2], 8, 2, 128, 16)
    check(ms, c, max_queries=hint)
    check(ms, case(8, "bf16", [1, 20, 4], [50, 90, 300], 8, 2, 256, 16), max_queries=hint)


@pytest.mark.parametrize("kind", ["one token", "chunks"])
def test_scores_of_every_size(ms, kind):
    for sigma, scale in ((4.0, None), (1.0, 0.0), (1.0, -0.3), (0.05, None), (30.0, None)):
        for dtype in ("bf16", "f16"):
            check(ms, case(9, dtype, *KINDS[kind], 4, 2, 128, 16, sigma), scale=scale)


@pytest.mark.parametrize("kind", ["one token", "chunks"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rising_maxima_and_long_tails(ms, kind, dtype):
    """Keys sorted by their scores, so that the maximum grows in every tile, or is the first key's alone."""
    import torch
    for sign in (1, -1):
        c = case(10, dtype, *KINDS[kind], 2, 1, 64, 16)
        for r, n in enumerate(c["lens"]):
            t = np.arange(n)
            pg = c["table"][r, t // 16]
            c["k"][torch.from_numpy(pg.astype(np.int64)).cuda(), torch.from_numpy(t % 16).cuda(), 0, 0] = \
                torch.from_numpy(sign * np.linspace(-30, 30, n)).to(c["k"].dtype).cuda()
        c["q"][..., 0] = 8
        check(ms, c)


def test_huge_scores(ms):
    """Maxima past 2^20 in base 2: equal scores stay equal."""
    import torch
    for kind in ("one token", "chunks"):
        c = case(11, "bf16", *KINDS[kind], 2, 1, 64, 16)
        c["q"][:], c["k"][:] = 0, 0
        c["q"][..., 0], c["k"][..., 0] = 2.0 ** 14, 3 * 2.0 ** 12
        out, lse = call(ms, c)
        o = serving.chunk_attention(c["q"], c["k"], c["v"], c["table"], c["starts"], c["lens"], None, 0, 64 ** -0.5)
        A = o[2]
        assert bool(((out.double() - o[0]).abs() <= 2.0 ** -8 * (A + o[0].abs()) + 2.0 ** -14 * A).all())
        assert bool(((lse.double() - o[1]).abs() <= 2.0 ** -20 * o[1].abs()).all())


def test_views_and_outputs(ms):
    """Pages laid out heads first, keys and values in one tensor, padded heads, a strided query and output."""
    import torch
    for kind in KINDS:
        for D in (64, 128, 256):
            c = case(12, "bf16", *KINDS[kind], 8, 2, D, 16)
            want, _ = check(ms, c)
            both = torch.stack([c["k"], c["v"]], 1).transpose(2, 3).contiguous().transpose(2, 3)
            wide = torch.zeros(*c["k"].shape[:3], D + 8, dtype=torch.bfloat16, device="cuda")
            wide[..., 8:] = c["k"]
            n, Hq = c["q"].shape[:2]
            fused = torch.zeros(n, Hq, 3 * D, dtype=torch.bfloat16, device="cuda")
            fused[..., D:2 * D] = c["q"]
            res = torch.full((n, Hq, 2 * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
            for k, v in ((both[:, 0], both[:, 1]), (wide[..., 8:], c["v"])):
                out, _ = call(ms, dict(c, k=k, v=v, q=fused[..., D:2 * D]), out=res[..., 8:D + 8])
                assert torch.equal(out, want) and out.data_ptr() == res[..., 8:].data_ptr()
                assert bool((res[..., :8] == 7).all()) and bool((res[..., D + 8:] == 7).all())


def test_strides_without_a_common_row(ms):
    """Caches that the copy engine has no map for: strides with no common divisor of a head or more."""
    import torch
    for kind in KINDS:
        for D in (64, 128, 256):
            c = case(13, "bf16", *KINDS[kind], 8, 2, D, 16)
            pages, page, H, _ = c["k"].shape
            # heads D + 8 apart, slots 8 more than their heads take: the greatest common divisor is 8
            slot = H * (D + 8) + 8
            k, v = (torch.zeros((pages + 1) * (page * slot + 8), dtype=torch.bfloat16, device="cuda").as_strided(
                (pages, page, H, D), (page * slot + 8, slot, D + 8, 1)) for _ in range(2))
            k.copy_(c["k"]), v.copy_(c["v"])
            check(ms, dict(c, k=k, v=v))
            check(ms, dict(c, v=v), window=40, sinks=2)


def test_rows_of_no_request(ms):
    """Left as they are in a given output, zeros in a new one; lse -infinity."""
    import torch
    for kind in KINDS:
        for D in (128, 256):
            c = case(14, "bf16", *KINDS[kind], 8, 2, D, 16, lead=3, tail=9)
            n = int(c["starts"][-1])
            for given in (None, torch.full_like(c["q"], 5.0)):
                out, lse = call(ms, c, out=given)
                inner = dict(c, q=c["q"][3:n].contiguous(), starts=c["starts"] - 3)
                want, wl = check(ms, inner)
                assert torch.equal(out[3:n], want) and torch.equal(lse[3:n], wl)
                for edge in (out[:3], out[n:]):
                    assert bool((edge == (0 if given is None else 5)).all())
                assert bool(torch.isneginf(lse[:3]).all()) and bool(torch.isneginf(lse[n:]).all())


def test_what_a_query_does_not_see_does_not_reach_it(ms):
    """NaN and infinities behind the lengths, in unused pages, below the window, and in tokens that come after a query."""
    import torch
    for kind in ("few", "chunks"):
        for D in (64, 128, 256):
            for kw in (dict(), dict(window=20, sinks=2)):
                c = case(15, "bf16", *KINDS[kind], 8, 2, D, 16, spare=5)
                clean, _ = check(ms, c, **kw)
                free = np.ones(c["k"].shape[:2], bool)
                for r, n in enumerate(c["lens"]):
                    t = np.arange(n)
                    lo = n - int(c["starts"][r + 1] - c["starts"][r]) - (kw.get("window", 10 ** 6) - 1)
                    t = t[(t >= lo) | (t < kw.get("sinks", 0))]
                    free[c["table"][r, t // 16], t % 16] = False
                mask = torch.from_numpy(free).cuda()
                c["k"][mask], c["v"][mask] = float("nan"), float("inf")
                out, _ = call(ms, c, **kw)
                assert torch.equal(out, clean)
                # the last token of request 0: only its last query sees it
                t = int(c["lens"][0]) - 1
                pg, last = int(c["table"][0, t // 16]), int(c["starts"][1]) - 1
                c["k"][pg, t % 16], c["v"][pg, t % 16] = float("nan"), float("inf")
                out, lse = call(ms, c, **kw)
                assert torch.isnan(out[last]).all() and torch.isnan(lse[last]).all()
                others = [i for i in range(out.shape[0]) if i != last]
                assert torch.equal(out[others], clean[others])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,length", [(5, 5), (5, 70), (5, 700), (150, 150), (150, 400)])
@pytest.mark.parametrize("kw", [dict(), dict(window=40, sinks=1)])
def test_infinite_values_that_a_query_sees(ms, D, n, length, kw):
    """Infinite and NaN values among the chunk's own tokens reach the queries that see them as the sum has them, and no other."""
    import torch
    inf, nan = float("inf"), float("nan")
    for dtype in ("bf16", "f16"):
        c = case(16, dtype, [n, 1], [length, 50], 8, 2, D, 16)
        clean, _ = call(ms, c, **kw)
        # (at least `first`: every one of them is seen by some of the queries only, and is taken out of its tile)
        first = length - n
        marks = [(length - 1, 0, inf), (length - 2, 1, -inf), (length - 3, 2, inf), (length - 1, 2, -inf), (length - 4, 3, nan),
                 (length - 2, D - 1, inf), (first + 1, 5, -inf), (first + 1, 6, inf)]
        for t, d, x in marks:
            c["v"][int(c["table"][0, t // 16]), t % 16, 1, d] = x
        want = clean.clone()
        for t, d, x in marks:
            for j in range(n):
                p = length - n + j
                if t <= p and (p - t < kw.get("window", 10 ** 9) or t < kw.get("sinks", 0)):
                    want[j, 4:, d] += x
        out, _ = call(ms, c, **kw)
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


def test_pages_that_do_not_exist_show_where_they_are_seen(ms):
    import torch
    for kind in KINDS:
        for D in (64, 128, 256):
            for window in (None, 30):
                c = case(17, "bf16", *KINDS[kind], 8, 2, D, 16)
                clean, _ = check(ms, c, window=window)
                r = len(c["lens"]) - 1
                for bad, at in ((c["k"].shape[0], 2), (-7, 4)):
                    c["table"][r, at] = bad
                out, lse = call(ms, c, window=window)
                n = int(c["starts"][r + 1] - c["starts"][r])
                for i in range(out.shape[0]):
                    p = int(c["lens"][r]) - n + i - int(c["starts"][r])
                    keys = np.arange(max(0, p - (window or 10 ** 9) + 1), p + 1)
                    lost = i >= c["starts"][r] and bool(np.isin(keys // 16, [2, 4]).any())
                    if lost:
                        assert torch.isnan(out[i]).all() and torch.isnan(lse[i]).all()
                    else:
                        assert torch.equal(out[i], clean[i])


def test_lengths_and_starts_out_of_range(ms):
    """Lengths are clamped to what the table can name, starts to the batch."""
    import torch
    for D in (64, 256):
        c = case(18, "bf16", [1, 40, 2], [160, 160, 160], 8, 2, D, 16)
        clean, _ = check(ms, c)
        out, _ = call(ms, dict(c, lens=np.int32([2 ** 31 - 1, 161, 160])))
        assert torch.equal(out, clean)
        out, lse = call(ms, dict(c, lens=np.int32([-1, -2 ** 31, 0])))
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        out, _ = call(ms, dict(c, starts=np.int32([-5, 1, 41, 10 ** 9])))
        assert torch.equal(out, clean)
        out, _ = call(ms, dict(c, starts=np.int32([0, 1, 41, 41])))       # the last request has no queries
        assert torch.equal(out[:41], clean[:41]) and bool((out[41:] == 0).all())


def test_nothing_to_attend(ms):
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    k = torch.zeros(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.randn(40, 4, 64, device="cuda").bfloat16()
    starts = torch.tensor([0, 1, 40], dtype=torch.int32, device="cuda")
    out, lse = ms.paged_chunk_attention(q, k, k, z(2, 0), starts, z(2), return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    out = ms.paged_chunk_attention(q, k, k, z(2, 3), starts, z(2) + 40)      # pages that are not there
    assert torch.isnan(out).all()
    assert ms.paged_chunk_attention(q[:0], k, k, z(0, 0), z(1), z(0)).shape == (0, 4, 64)
    out, lse = ms.paged_chunk_attention(q, k, k, z(0, 0), z(1), z(0), return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_offsets_past_32_bits(ms):
    """A cache of more than 2^31 elements whose used pages lie at its end."""
    import torch
    page, H, D = 64, 8, 128
    pages = 2 ** 31 // (page * H * D) + 20
    c = case(19, "bf16", [1, 70, 3], [200, 300, 65], 8, 8, D, page)
    small = c["k"].shape[0]
    k = torch.zeros(pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[pages - small:], v[pages - small:] = c["k"], c["v"]
    want, _ = check(ms, c)
    out, _ = call(ms, dict(c, k=k, v=v, table=np.where(c["table"] >= 0, c["table"] + pages - small, -1).astype(np.int32)))
    assert torch.equal(out, want)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_into_the_query(ms, D):
    import torch
    for kind in KINDS:
        for extra in (0, 3000):
            new, lens = KINDS[kind]
            c = case(20, "bf16", new, np.int32(lens) + extra, 8, 2, D, 16)
            want, lse = call(ms, c)
            q = c["q"].clone()
            out, lse2 = call(ms, dict(c, q=q), out=q)
            assert out is q and torch.equal(q, want) and torch.equal(lse, lse2)


def test_the_same_bits_every_time_captured_and_on_two_streams(ms):
    import torch
    cs = [case(21 + i, "bf16", [1, 300, 2], [3000, 900, 50], 8, 2, 128, 16) for i in range(2)]
    want = [call(ms, c) for c in cs]
    torch.cuda.synchronize()
    cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    args = [[c["q"], c["k"], c["v"], cu(c["table"]), cu(c["starts"]), cu(c["lens"])] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(6):
        for i, a in enumerate(args):
            with torch.cuda.stream(streams[i]):
                got[i].append(ms.paged_chunk_attention(*a, return_lse=True))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1]) for g in got[i])
    # two graphs captured on one stream, replayed at the same time on two others, with other lengths
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            outs.append(ms.paged_chunk_attention(*a, return_lse=True))
        graphs.append(g)
    short = dict(cs[0], lens=np.int32([500, 301, 2]))
    args[0][5].copy_(cu(short["lens"]))
    torch.cuda.synchronize()
    for _ in range(3):
        for i, g in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                g.replay()
    torch.cuda.synchronize()
    w0 = call(ms, short)
    assert torch.equal(outs[0][0], w0[0]) and torch.equal(outs[1][0], want[1][0]) and torch.equal(outs[1][1], want[1][1])


def test_more_tiles_than_threads(ms):
    """Requests, and tiles of the tensor cores, of which a thread of the search for a CTA's run has several; none at a run's start."""
    new = np.tile([20, 1, 0, 3, 33], 260)
    check(ms, case(30, "bf16", new, new + np.tile([0, 90, 7], 434)[:1300], 2, 2, 64, 16))
    new = np.concatenate([np.ones(600, int), [700], np.ones(600, int), [17, 300]])
    check(ms, case(31, "bf16", new, new + 40, 2, 1, 64, 16))
    check(ms, case(32, "f16", [3000, 2, 1500], [3000, 3000, 1600], 24, 1, 128, 16), window=100, sinks=3)


def test_steps_behind_one_another(ms):
    """Lengths, starts, tables, queries and caches that change between calls which nobody waits for."""
    import torch
    for D, H in ((64, 4), (128, 1)):
        c = case(33, "bf16", [1, 300, 2, 40, 1], [2600, 600, 50, 700, 900], 4, H, D, 16)
        cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()

        def steps(wait):
            q, k, v, table, starts, lens = c["q"].clone(), c["k"].clone(), c["v"].clone(), cu(c["table"]), cu(c["starts"]), cu(c["lens"])
            outs = []
            for i in range(12):
                outs.append(ms.paged_chunk_attention(q, k, v, table, starts, lens, return_lse=True))
                if wait:
                    torch.cuda.synchronize()
                lens.sub_(1)
                starts[1:5].add_(1 if i % 2 else -1)
                table[:, :3].copy_(table[:, :3].roll(1, 1))
                q.mul_(-1)
                k[i].neg_(), v[i].neg_()
                if wait:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            return outs
        for (o, l), (o2, l2) in zip(steps(False), steps(True)):
            assert torch.equal(o, o2) and torch.equal(l, l2)
