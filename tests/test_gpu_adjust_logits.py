"""Penalties, biases and grammar masks (fs_adjust_logits) against float64.

Tolerance of a logit of type t that changes: eps / 2 of the result, and of the float32 steps before (product or
quotient, the product with the count and its difference in one rounding, presence, bias: 4 roundings of 2^-24) of the largest
magnitude on the way.  Every other logit is copied: equal bits.  -infinity where the mask says so, exactly."""
import numpy as np
import pytest

from oracle import serving
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


def _case(seed, dtype, B, V, history=0, bias=0, masks=None, pad=0, hot=None):
    """bias: entries a row at most; masks: rows of masks."""
    import torch
    rng = np.random.default_rng(seed)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    x = torch.from_numpy(rng.standard_normal((B, V + pad)).astype(np.float32) * 4).to(dt).cuda()[:, :V]
    c = dict(x=x, tokens=None, lens=None, prompts=None, pen={}, bias=None, allowed=None, rows=None)
    if history:
        c["tokens"] = rng.integers(-3, hot or V + 3, (B, history)).astype(np.int32)
        c["lens"] = rng.integers(0, history + 1, B).astype(np.int32)
        c["lens"][0] = history
        c["prompts"] = (c["lens"] * rng.random(B)).astype(np.int32)
        c["pen"] = dict(repetition=(1 + rng.random(B)).astype(np.float32), presence=rng.standard_normal(B).astype(np.float32),
                        frequency=(0.3 * rng.standard_normal(B)).astype(np.float32))
    if bias:
        n = rng.integers(0, bias + 1, B)
        n[-1] = bias
        c["bias"] = (np.concatenate([[0], np.cumsum(n)]).astype(np.int32), rng.integers(-2, V + 2, n.sum()).astype(np.int32),
                     rng.standard_normal(n.sum()).astype(np.float32) * 5)
    if masks is not None:
        c["allowed"] = rng.integers(-2 ** 31, 2 ** 31, (masks, -(-V // 32))).astype(np.int32)
        c["rows"] = rng.integers(-2, max(masks, 1), B).astype(np.int32)
    return c


def _args(c):
    import torch
    cu = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    kw = {k: cu(v) for k, v in c["pen"].items()}
    if c["bias"]:
        kw.update(bias_starts=cu(c["bias"][0]), bias_tokens=cu(c["bias"][1]), bias_values=cu(c["bias"][2]))
    if c["allowed"] is not None:
        kw.update(allowed=cu(c["allowed"]), allowed_rows=cu(c["rows"]))
    return [c["x"], cu(c["tokens"]), cu(c["lens"]), cu(c["prompts"])], kw


def _expect(c):
    """float64 logits, magnitudes, and which change."""
    z0 = c["x"].double().cpu().numpy()
    B, V = z0.shape
    z, big, touched = z0.copy(), np.abs(z0), np.zeros((B, V), bool)
    for b in range(B):
        tok = () if c["tokens"] is None else c["tokens"][b, : np.clip(c["lens"][b], 0, c["tokens"].shape[1]) if c["lens"] is not None else None]
        kw = {k: float(v[b]) for k, v in c["pen"].items()}
        bias = []
        if c["bias"]:
            s = np.clip(c["bias"][0], 0, len(c["bias"][1]))
            bias = [(int(t), float(v)) for t, v in zip(c["bias"][1][s[b]:s[b + 1]], c["bias"][2][s[b]:s[b + 1]])]
        ok = None
        if c["allowed"] is not None and c["rows"][b] >= 0:
            ok = np.zeros(V, bool)
            if c["rows"][b] < len(c["allowed"]):
                ok = np.unpackbits(c["allowed"][c["rows"][b]].view(np.uint8), bitorder="little")[:V].astype(bool)
        z[b], big[b] = serving.adjust_row(z0[b], tok, int(c["prompts"][b]) if c["prompts"] is not None else 0, bias=bias, allowed=ok, **kw)
        t = [int(i) for i in tok if 0 <= i < V] + [i for i, _ in bias if 0 <= i < V]
        touched[b, t] = True
    return z, big, touched


def _near(got, c, want):
    import torch
    z, big, touched = want
    g = got.double().cpu().numpy()
    banned = np.isneginf(z) & ~np.isneginf(c["x"].double().cpu().numpy())
    assert np.isneginf(g[banned]).all()
    keep = ~touched & ~banned
    assert (g[keep] == c["x"].double().cpu().numpy()[keep]).all()
    tol = torch.finfo(got.dtype).eps / 2 * np.abs(z) + 4 * 2.0 ** -24 * big
    sel = touched & ~banned
    assert (np.abs(g[sel] - z[sel]) <= tol[sel]).all()


def _check(ms, c):
    """Into a new tensor, in place, and into a strided one: the same."""
    import torch
    want = _expect(c)
    a, kw = _args(c)
    x0 = c["x"].clone()
    got = ms.adjust_logits(*a, **kw)
    assert got.is_contiguous() and torch.equal(c["x"], x0)
    _near(got, c, want)
    B, V = x0.shape
    buf = torch.full((B, V + 3), 9.0, dtype=x0.dtype, device="cuda")
    out = buf[:, 1:V + 1]
    assert ms.adjust_logits(*a, **kw, out=out) is out
    bits = lambda t: t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)
    assert torch.equal(bits(out), bits(got)) and bool((buf[:, 0] == 9).all()) and bool((buf[:, V + 1:] == 9).all())
    full = c["x"]._base if c["x"]._base is not None else c["x"]
    pad = full.clone()
    assert ms.adjust_logits(*a, **kw, out=a[0]) is a[0]
    assert torch.equal(bits(a[0]), bits(got)) and torch.equal(bits(full[:, V:]), bits(pad[:, V:]))
    a[0].copy_(x0)
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 7, 31, 32, 33, 1000, 4095, 4096, 8193, 32000, 50257])
def test_vocabularies(ms, dtype, V):
    for pad in (0, 1, 8):
        _check(ms, _case(V + pad, dtype, 3, V, history=40, bias=9, masks=2, pad=pad))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("history", [1, 4, 513, 2000, 4096, 4097, 9000])
def test_histories(ms, dtype, history):
    """One CTA a row, several, and more tokens than are staged at once; few and many rows."""
    for B in (1, 5, 70):
        _check(ms, _case(history + B, dtype, B, 3000, history=history))


@pytest.mark.parametrize("parts", ["history", "bias", "masks", "history bias", "history masks", "bias masks", ""])
def test_parts(ms, parts):
    for dtype in TYPES:
        _check(ms, _case(3, dtype, 6, 700, history=60 if "history" in parts else 0, bias=30 if "bias" in parts else 0,
                         masks=4 if "masks" in parts else None, pad=5))


def test_one_token_often_and_full_tables(ms):
    """Histories of one token, of few, and biases for every token: more tokens than a table holds, tables that overflow."""
    _check(ms, _case(1, "f32", 2, 1000, history=5000, hot=1))
    _check(ms, _case(2, "bf16", 3, 1000, history=3000, hot=4))
    _check(ms, _case(3, "f32", 3, 9000, history=20, bias=9000))
    _check(ms, _case(4, "bf16", 2, 40000, history=70000))
    # tokens that all fall into one CTA's share
    c = _case(5, "f32", 1, 200000, history=8000)
    h = np.arange(200000, dtype=np.uint64) * 2654435769 % 2 ** 32
    for split in (1, 2, 3, 4, 5):
        mine = np.nonzero(h >> (32 - split) == 0)[0][:8000]
        c["tokens"][0, : len(mine)] = mine
        _check(ms, c)


def test_counts_past_16_bits(ms):
    c = _case(6, "f32", 1, 50, history=70000, hot=1)
    c["tokens"][:] = 7
    c["lens"][:], c["prompts"][:] = 70000, 100
    c["pen"]["frequency"][:] = 1e-3
    _check(ms, c)


def test_duplicate_biases_and_tokens_out_of_range(ms):
    c = _case(7, "f32", 2, 100, history=5)
    c["tokens"][:] = [[-1, 100, 2 ** 31 - 1, -2 ** 31, 3], [99, 99, 0, 0, -5]]
    c["bias"] = (np.int32([0, 5, 9]), np.int32([3, 3, 100, -1, 3, 0, 50, 0, 99]), np.float32([1, 2, 3, 4, 5, 6, 7, 8, 9]))
    got = _check(ms, c)
    assert float(got[1, 50]) == np.float32(float(c["x"][1, 50])) + np.float32(7)


def test_ranges_of_lengths_starts_and_mask_rows(ms):
    c = _case(8, "f32", 4, 100, history=6, bias=3, masks=2)
    c["lens"][:] = [-1, 99, 3, 0]
    c["prompts"][:] = [-4, 99, -2 ** 31, 2]
    c["bias"] = (np.int32([-5, 2, 4, 99, 3]), c["bias"][1][:4] if len(c["bias"][1]) >= 4 else np.int32([1, 2, 3, 4]), np.float32([1, 2, 3, 4]))
    c["rows"][:] = [-1, 2, 0, -2 ** 31]
    got = _check(ms, c)
    assert bool((got[1] == -float("inf")).all())        # a mask that does not exist allows nothing


def test_no_masks_at_all(ms):
    import torch
    x = torch.randn(2, 40, device="cuda")
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    rows = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    got = ms.adjust_logits(x, allowed=none, allowed_rows=rows)
    assert torch.equal(got[0], x[0]) and bool((got[1] == -float("inf")).all())


def test_values_that_are_not_finite(ms):
    """Infinite and NaN logits go through as the arithmetic has them; a mask overrides them."""
    import torch
    inf, nan = float("inf"), float("nan")
    for dt in (torch.float32, torch.bfloat16):
        x = torch.tensor([[inf, -inf, nan, 1.0, inf, nan, -inf, 2.0]], device="cuda").to(dt)
        tok = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device="cuda")
        got = ms.adjust_logits(x, tok, repetition=2.0, presence=1.0, frequency=0.5)
        assert got[0, 0] == inf and got[0, 1] == -inf and torch.isnan(got[0, 2]) and float(got[0, 3]) == 0.5 - 1.5
        assert got[0, 4] == inf and torch.isnan(got[0, 5]) and got[0, 6] == -inf and got[0, 7] == 2
        mask = torch.tensor([[0x80]], dtype=torch.int32, device="cuda")
        got = ms.adjust_logits(x, tok, repetition=2.0, allowed=mask)
        assert bool((got[0, :7] == -inf).all()) and got[0, 7] == 2


def test_scalars_and_defaults(ms):
    import torch
    c = _case(9, "f32", 3, 64, history=7)
    c["pen"] = {k: np.float32([v] * 3) for k, v in dict(repetition=1.3, presence=0.2, frequency=0.1).items()}
    a, kw = _args(c)
    want = ms.adjust_logits(*a, **kw)
    assert torch.equal(ms.adjust_logits(*a, repetition=1.3, presence=0.2, frequency=0.1), want)
    full = ms.adjust_logits(a[0], a[1], frequency=0.25)
    c2 = dict(c, lens=None, prompts=None, pen=dict(frequency=np.float32([0.25] * 3)))
    _near(full, c2, _expect(c2))
    assert torch.equal(ms.adjust_logits(a[0], a[1][:, :0], repetition=2.0), a[0])
    assert torch.equal(ms.adjust_logits(a[0]), a[0]) and ms.adjust_logits(a[0][:0]).shape == (0, 64)


def test_captured_and_on_two_streams(ms):
    import torch
    cs = [_case(20 + i, "bf16", 20, 9000, history=900, bias=20, masks=7) for i in range(2)]
    args = [_args(c) for c in cs]
    want = [ms.adjust_logits(*a, **kw) for a, kw in args]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(6):
        for i, (a, kw) in enumerate(args):
            with torch.cuda.stream(ss[i]):
                got[i].append(ms.adjust_logits(*a, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])
    graphs, outs = [], []
    for i, (a, kw) in enumerate(args):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=ss[0]):
            outs.append(ms.adjust_logits(*a, **kw))
        graphs.append(g)
    args[0][0][2].zero_()           # lens: no history now
    for _ in range(3):
        for i, g in enumerate(graphs):
            with torch.cuda.stream(ss[i]):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], want[1])
    c0 = dict(cs[0], lens=np.zeros(20, np.int32))
    _near(outs[0], c0, _expect(c0))


@pytest.mark.parametrize("history", [902, 901])
def test_steps_behind_one_another(ms, history):
    """Logits, histories and lengths that change between calls which nobody waits for."""
    import torch
    c = _case(30, "f32", 20, 9001, history=history, bias=20, masks=7)

    def steps(wait):
        (x, tokens, lens, prompts), kw = _args(c)
        x, outs = x.clone(), []
        for i in range(12):
            outs.append(ms.adjust_logits(x, tokens, lens, prompts, **kw))
            if wait:
                torch.cuda.synchronize()
            x.neg_()
            tokens.copy_(tokens.roll(1, 0))
            lens.sub_(1).clamp_(min=0)
            kw["allowed_rows"].copy_(kw["allowed_rows"].roll(1))
            kw["bias_values"].neg_()
            kw["frequency"].mul_(1.5)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs
    for a, b in zip(steps(False), steps(True)):
        assert torch.equal(a, b)
