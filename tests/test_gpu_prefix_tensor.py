"""The prefix's part on the tensor cores (33 queries a key/value head and a table of 512 keys on) over what it accepts: page
sizes, layouts, pages that do not exist, groups, far offsets, unused slots.  Same tolerances as the other attention tests."""
import numpy as np
import pytest

from tests.helpers import ensure_built
from tests.test_gpu_prefix_attention import _call, _case, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


@pytest.mark.parametrize("page", [1, 5, 16, 64, 100])
@pytest.mark.parametrize("plen", [512, 513, 575, 577, 641, 1290])
def test_lengths_and_pages(ms, page, plen):
    """128 and 256 queries a tile; pages that end inside a tile of keys."""
    rng = np.random.default_rng(plen)
    _check(ms, _case(plen + page, "bf16", [18], 18, 1, 8, 4, 64, [plen], rng.integers(0, 40, 18), page))
    _check(ms, _case(plen + page, "f16", [40], 40, 2, 8, 4, 128, [plen], rng.integers(0, 40, 40), page))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (8, 8), (10, 2), (7, 1), (32, 2)])
def test_head_layouts(ms, dtype, D, heads):
    Hq, H = heads
    for n in (33, 129):
        rows = -(-n * H // Hq)
        _check(ms, _case(1, dtype, [rows], rows, 1, Hq, H, D, [700], [i % 20 for i in range(rows)], 16))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [20, 80])
def test_lengths_short_of_the_table(ms, dtype, rows):
    """Tables wider than the lengths, as a captured graph has them: few tiles of keys, one, none."""
    for plen in (0, 1, 63, 64, 65, 128, 300):
        c = _case(plen + rows, dtype, [rows], rows, 1, 8, 4, 128, [plen], [i % 5 for i in range(rows)], 16)
        c["ptab"] = np.concatenate([c["ptab"], np.full((1, 100), -1, np.int32)], 1)
        _check(ms, c)


@pytest.mark.parametrize("rows", [20, 80])
def test_views_and_outputs(ms, rows):
    """Pages laid out heads first, keys and values in one tensor, a strided query and a strided output."""
    import torch
    for D in (64, 128):
        c = _case(7, "bf16", [rows], rows, 2, 8, 2, D, [700], [2 + i % 30 for i in range(rows)], 16)
        both = torch.stack([c["k"], c["v"]], 1).transpose(2, 3).contiguous().transpose(2, 3)
        c["k"], c["v"] = both[:, 0], both[:, 1]
        wide = torch.zeros(rows, 2, 8, 3 * D, dtype=torch.bfloat16, device="cuda")
        wide[..., D:2 * D] = c["q"]
        c["q"] = wide[..., D:2 * D]
        res = torch.full((rows, 2, 8, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
        out, _ = _check(ms, c, out=res[..., D:])
        assert out.data_ptr() == res[..., D:].data_ptr() and bool((res[..., :D] == 7).all())


def test_pages_that_do_not_exist_show_as_nan(ms):
    """One bad page, first, middle or last, among good ones: its group's rows are NaN, no other row changes."""
    import torch
    for at, bad in ((0, -1), (20, 2 ** 31 - 1), (43, -2 ** 31), (37, None)):
        for rows in (40, 160):
            half = rows // 2
            c = _case(10, "bf16", [half, half], rows, 1, 8, 4, 64, [700, 690], [70] * rows, 16)
            clean, _ = _check(ms, c)
            c["ptab"][1, at] = c["k"].shape[0] if bad is None else bad
            out, lse = _call(ms, c)
            assert torch.isnan(out[half:]).all() and torch.isnan(lse[half:]).all()
            assert torch.equal(out[:half], clean[:half])


def test_groups_of_every_size(ms):
    """Empty groups, short and empty prefixes, rows of no group."""
    _check(ms, _case(1, "bf16", [3, 0, 50, 100], 153, 1, 8, 2, 128, [700, 10, 0, 650], [i % 70 for i in range(153)], 16))
    _check(ms, _case(2, "f16", [1, 129, 3, 0, 60], 200, 1, 8, 2, 64, [513, 640, 1, 64, 65], [i % 3 for i in range(200)], 5))
    c = _case(3, "bf16", [60, 60], 130, 1, 4, 2, 64, [600, 550], [3] * 130, 16)
    c["starts"] = np.int32([4, 64, 120])      # rows 0 to 3 and 120 to 129 have no prefix
    _check(ms, c)


def test_unused_slots_and_later_tokens_do_not_reach_a_query(ms):
    """NaN and infinities behind the lengths, in unused pages, and in the tokens that come after a query."""
    import torch
    for rows, dtype in ((20, "bf16"), (80, "f16")):
        c = _case(8, dtype, [rows], rows, 3, 8, 2, 64, [701], [3 + i % 20 for i in range(rows)], 16, spare=5)
        clean, _ = _check(ms, c)
        used = set()
        for tab, lens in ((c["ptab"], c["plens"]), (c["stab"], c["slens"])):
            for i, n in enumerate(lens):
                used |= {(int(tab[i, t // 16]), t % 16) for t in range(n)}
        free = np.array([[(pg, s) not in used for s in range(16)] for pg in range(c["k"].shape[0])])
        mask = torch.from_numpy(free).cuda()
        c["k"][mask], c["v"][mask] = float("nan"), float("inf")
        assert torch.equal(_call(ms, c)[0], clean)
        t = int(c["slens"][1]) - 1
        c["v"][int(c["stab"][1, t // 16]), t % 16] = float("nan")
        out, _ = _call(ms, c)
        assert torch.equal(out[1, :2], clean[1, :2]) and torch.isnan(out[1, 2]).all()
        keep = [0] + list(range(2, rows))
        assert torch.equal(out[keep], clean[keep])


def test_nan_and_infinite_values_of_the_prefix(ms):
    import torch
    for rows in (20, 80):
        c = _case(9, "bf16", [rows], rows, 1, 8, 4, 64, [700], [4] * rows, 16)
        clean, _ = _call(ms, c)
        for t, d, x in ((3, 1, float("inf")), (650, 2, -float("inf")), (699, 3, float("nan")), (64, 4, float("inf")), (65, 4, -float("inf"))):
            c["v"][int(c["ptab"][0, t // 16]), t % 16, 1, d] = x
        out, _ = _call(ms, c)
        assert bool((out[:, 0, 2:4, 1] == float("inf")).all()) and bool((out[:, 0, 2:4, 2] == -float("inf")).all())
        assert torch.isnan(out[:, 0, 2:4, 3:5]).all()
        out[:, 0, 2:4, 1:5] = clean[:, 0, 2:4, 1:5]
        assert torch.equal(out, clean)
        c["k"][int(c["ptab"][0, 40]), 7, 3, 9] = float("nan")     # a key that every query of head 3 sees
        out, lse = _call(ms, c)
        assert torch.isnan(out[:, 0, 6:]).all() and torch.isnan(lse[:, 0, 6:]).all()
        assert torch.equal(out[:, 0, :2], clean[:, 0, :2])


def test_offsets_past_32_bits(ms):
    """A cache of more than 2^31 elements whose used pages lie at its end."""
    import torch
    page, H, D = 64, 8, 128
    for rows in (40, 140):
        c = _case(12, "bf16", [rows], rows, 1, 8, 8, 128, [700], [i % 9 for i in range(rows)], page)
        small = c["k"].shape[0]
        pages = 2 ** 31 // (page * H * D) + small + 1
        k = torch.zeros(pages, page, H, D, dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        k[pages - small:], v[pages - small:] = c["k"], c["v"]
        want, _ = _check(ms, c)
        far = dict(c, k=k, v=v, ptab=c["ptab"] + (pages - small),
                   stab=np.where(c["stab"] >= 0, c["stab"] + pages - small, -1).astype(np.int32))
        out, _ = _call(ms, far)
        assert torch.equal(out, want)


def test_captured_with_the_widest_tables(ms):
    """A captured call replayed with lengths from nothing to the table's end."""
    import torch
    cu = lambda x: torch.from_numpy(x).cuda()
    c = _case(14, "bf16", [40, 40], 80, 1, 8, 2, 128, [1500, 1400], [200] * 80, 16)
    d = dict(c, **{n: cu(c[n]) for n in ("ptab", "plens", "stab", "slens", "starts")})
    call = lambda: ms.shared_prefix_attention(d["q"], d["k"], d["v"], d["ptab"], d["plens"], d["stab"], d["slens"], d["starts"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for plen, slen in ((1400, 200), (0, 0), (1, 200), (64, 64), (129, 1), (777, 130)):
        d["plens"].fill_(plen)
        d["slens"].fill_(slen)
        g.replay()
        assert torch.equal(out, call())
        _check(ms, dict(c, plens=np.full(2, plen, np.int32), slens=np.full(80, slen, np.int32)))
