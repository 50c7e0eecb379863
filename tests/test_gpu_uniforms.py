"""Sampling from given uniforms (fs_top_k_top_p_sampling_from_uniforms) against the float64
definition: the same token on every row.  The kernels decide on weights with a relative error of 5e-10
and an absolute one of 2^-43, so a row whose decisive mass lies within MARGIN of a border
proves nothing and is left out; the drawn rows hardly ever do."""
import numpy as np
import pytest

from oracle import decode
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
MARGIN = 1e-9
INF = float("inf")


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


def _dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _col(x, n, default):
    return np.full(n, default) if x is None else np.broadcast_to(np.asarray(x), (n,))


def _check(ms, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, order="joint", indices=None,
           few_near=True):
    import torch
    dev = logits.device
    put = lambda x, dt: x if x is None or np.isscalar(x) else torch.as_tensor(np.ascontiguousarray(x), dtype=dt, device=dev)
    tok, valid = ms.top_k_top_p_sampling_from_uniforms(
        logits, put(np.asarray(u, np.float32), torch.float32), put(temperature, torch.float32), put(top_k, torch.int32),
        put(top_p, torch.float32), put(min_p, torch.float32), order, put(indices, torch.int32))
    tok, valid = tok.cpu().numpy(), valid.cpu().numpy()
    z = logits.float().cpu().numpy()
    n = len(tok)
    T, K = _col(temperature, n, 1.0).astype(np.float32), _col(top_k, n, 0)
    P, Mp = _col(top_p, n, 1.0).astype(np.float32), _col(min_p, n, 0.0).astype(np.float32)
    near = 0
    for b in range(n):
        r = b if indices is None else int(indices[b])
        want, margin = (-1, INF) if not 0 <= r < len(z) else decode.token_from_uniform(
            z[r], float(np.float32(u[b])), float(T[b]), int(K[b]), float(P[b]), float(Mp[b]), order)
        if margin < MARGIN:
            near += 1
            continue
        assert tok[b] == want, (b, tok[b], want, margin)
        assert valid[b] == (want >= 0)
    if few_near:
        assert near <= max(1, n // 20)
    return tok


def _logits(B, V, dtype, seed, sigma=3.0, pad=0, shift=0):
    """Rows inside a larger buffer: `pad` elements between rows, `shift` before the first."""
    import torch
    g = torch.Generator().manual_seed(seed)
    buf = torch.empty(shift + B * (V + pad)).normal_(generator=g) * sigma
    return buf.to(_dtype(dtype)).cuda()[shift:].view(B, V + pad)[:, :V]


def _u(n, seed):
    return np.random.default_rng(seed).random(n).astype(np.float32) * np.float32(1 - 2.0 ** -24)


FILTERS = [dict(), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=50, top_p=0.9),
           dict(top_k=20, top_p=0.8, min_p=0.02), dict(top_k=1), dict(top_p=0.0), dict(min_p=1.0), dict(top_p=1.0, top_k=0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["joint", "top_k_first"])
@pytest.mark.parametrize("f", range(len(FILTERS)))
def test_filters_and_types(ms, dtype, order, f):
    for V, seed in ((32000, 1), (1000, 2)):
        _check(ms, _logits(6, V, dtype, seed), _u(6, seed + f), temperature=0.8, order=order, **FILTERS[f])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 8, 31, 127, 128, 129, 255, 256, 257, 511, 513, 4099, 70001])
def test_odd_sizes_strides_and_alignments(ms, dtype, V):
    for pad, shift in ((0, 0), (1, 0), (3, 1), (8, 5)):
        for kw in (dict(), dict(top_k=3, top_p=0.7), dict(top_p=0.6), dict(top_k=max(1, V // 2), top_p=0.9)):
            _check(ms, _logits(4, V, dtype, V + pad, 2.0, pad, shift), _u(4, V + pad), order="top_k_first", **kw)


@pytest.mark.parametrize("k", [2, 511, 512, 513, 700, 5000, 31999, 32000, 40000])
@pytest.mark.parametrize("order", ["joint", "top_k_first"])
def test_large_top_k(ms, k, order):
    for dtype in ("f32", "bf16"):
        z = _logits(4, 32000, dtype, k)
        _check(ms, z, _u(4, k), top_k=k, order=order)
        _check(ms, z, _u(4, k + 1), top_k=k, top_p=0.97, min_p=0.001, order=order)


def test_full_size_and_per_row_parameters(ms):
    rng = np.random.default_rng(5)
    for dtype, V in (("f32", 151936), ("bf16", 256000)):
        B = 24
        z = _logits(B, V, dtype, 11)
        kw = dict(temperature=rng.uniform(0.3, 2.0, B).astype(np.float32), top_k=rng.integers(-1, 400, B).astype(np.int32),
                  top_p=rng.uniform(0.2, 1.1, B).astype(np.float32), min_p=(rng.random(B) * 0.02).astype(np.float32))
        for order in ("joint", "top_k_first"):
            _check(ms, z, _u(B, 3), order=order, **kw)
            _check(ms, z, _u(B, 4), order=order, temperature=kw["temperature"], top_p=kw["top_p"])


@pytest.mark.parametrize("sigma", [0.0, 1e-3, 0.05])
def test_flat_rows_and_ties(ms, sigma):
    """Near-flat and constant rows: every token's mass is about 1 / V, and 16-bit values tie by thousands."""
    for dtype in ("f32", "bf16", "f16"):
        for kw in (dict(), dict(top_p=0.5), dict(top_k=100), dict(top_k=10000, top_p=0.3), dict(top_k=7, top_p=0.5)):
            for order in ("joint", "top_k_first"):
                z = _logits(3, 40001, dtype, 3, sigma) + 1
                # a constant row: every running mass is a multiple of 1 / V, and a border is one exactly
                _check(ms, z, _u(3, 8), order=order, **kw, few_near=sigma > 0)
        if sigma == 0.0:
            u = np.float32([0.0, 0.5, 0.9999999, 1 - 2.0 ** -24, 0.123456, 2.0 ** -24, 1e-30, 0.75])
            tok = _check(ms, _logits(8, 40001, dtype, 3, 0.0), u, few_near=False)
            assert (tok == np.floor(u.astype(np.float64) * 40001)).all()


def test_parallel_samples_follow_the_kept_law(ms):
    """Evenly spaced uniforms through `indices` meet each token in proportion to its mass."""
    import torch
    z = _logits(2, 1024, "bf16", 9, 2.0)
    n = 1 << 16
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    for r in range(2):
        idx = np.full(n, r, np.int32)
        tok, valid = ms.top_k_top_p_sampling_from_uniforms(z, torch.from_numpy(u).cuda(), 0.9, 40, 0.9,
                                                           indices=torch.from_numpy(idx).cuda())
        tok = tok.cpu().numpy()
        assert valid.all() and (np.diff(tok) >= 0).all()
        zz = z[r].float().cpu().numpy().astype(np.float64)
        w = np.exp((zz - zz.max()) / np.float64(np.float32(0.9)))
        kept = np.unique(tok)
        cnt = np.bincount(tok, minlength=1024)[kept]
        # each border falls between two neighbouring uniforms
        assert np.abs(cnt / n - w[kept] / w[kept].sum()).max() <= 1.0 / n + 2.0 ** -24
    _check(ms, z, _u(64, 1), indices=np.arange(64, dtype=np.int32) % 2, top_p=0.9)


def test_rows_that_cannot_be_sampled(ms):
    z = _logits(12, 3000, "f32", 4)
    z[0, 17] = float("nan")
    z[1, 2999] = INF
    z[2] = -INF
    z[3, 1:] = -INF            # one finite logit
    z[4, ::2] = -INF           # a mask
    z[5] = -3.4e38             # the type's lowest everywhere: a flat row
    z[6, :] = -3.4e38
    z[6, 5] = 3.4e38
    z[7, 0] = -float("nan")
    u = _u(12, 6)
    u[8], u[9], u[10] = 1.0, -0.25, float("nan")
    for kw in (dict(), dict(top_k=50), dict(top_p=0.9), dict(top_k=50, top_p=0.9), dict(min_p=0.5)):
        _check(ms, z, u, **kw, few_near=False)
    zz = _logits(8, 500, "bf16", 5)
    _check(ms, zz, _u(8, 2), temperature=np.float32([0, -1, float("nan"), 1e-40, INF, 1e30, 2e-38, 1.0]), few_near=False)
    _check(ms, zz, _u(8, 2), top_p=np.float32([float("nan"), -1, 0, 1, 2, 0.5, INF, -INF]), few_near=False)
    _check(ms, zz, _u(8, 2), min_p=np.float32([float("nan"), -1, 0, 1, 2, 0.5, INF, -INF]), few_near=False)
    _check(ms, zz, _u(8, 2), indices=np.int32([0, -1, 8, 7, 2 ** 31 - 1, -2 ** 31, 3, 3]), top_k=5)
    _check(ms, zz, np.float32([0, 2.0 ** -149, 1e-30, 1 - 2.0 ** -24, 0.5, 0, 0, 0]), few_near=False)


def test_largest_vocabulary(ms):
    for dtype in ("f32", "bf16"):
        z = _logits(1, 2097152, dtype, 6)
        for kw in (dict(), dict(top_k=50, top_p=0.9), dict(top_p=0.9), dict(top_k=300000)):
            _check(ms, z, _u(1, 7), **kw)


def test_large_temperatures_and_offsets(ms):
    z = _logits(4, 9000, "f32", 8, 3.0) + 1000.0
    for T in (1e-3, 0.05, 30.0, 1e6):
        for kw in (dict(), dict(top_p=0.8), dict(top_k=2000, top_p=0.9)):
            _check(ms, z, _u(4, 9), temperature=T, **kw)


def test_zeros_of_both_signs_tie(ms):
    import torch
    z = torch.tensor([[-0.0, 0.0, -1.0, -0.0]], device="cuda").expand(3, 4).contiguous()
    for dt in ("f32", "bf16", "f16"):
        tok = _check(ms, z.to(_dtype(dt)), [0.1, 0.5, 0.9], top_k=1)
        assert tok.tolist() == [0, 1, 3]


def test_refusals(ms):
    """What the kernels cannot read is refused by name, before anything is launched."""
    import torch
    z, u = torch.zeros(4, 64, device="cuda"), torch.zeros(4, device="cuda")
    f = ms.top_k_top_p_sampling_from_uniforms
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=z.double()), dict(logits=z[0]), dict(logits=z.t()), dict(logits=z[:1].expand(4, 64)),
                dict(logits=z[:, :0]), dict(logits=z.cpu()), dict(uniforms=u.half()), dict(uniforms=u[:3]),
                dict(uniforms=u.cpu()), dict(uniforms=torch.zeros(8, device="cuda")[::2]), dict(uniforms=None),
                dict(temperature=u.double()), dict(top_k=u), dict(top_k=i32(1, 2)), dict(top_p=i32(1, 1, 1, 1)),
                dict(min_p=u[:2]), dict(indices=i32(0, 1).long()), dict(indices=i32(0, 1)), dict(order="up")):
        with pytest.raises(ValueError):
            f(**{"logits": z, "uniforms": u, **bad})
    with pytest.raises(TypeError):
        f(z, u, top_k="many")
    with pytest.raises(ms.FsError):
        f(torch.zeros(1, 2097153, device="cuda"), u[:1])
    tok, valid = f(z[:0], u[:0])
    assert tok.shape == (0,) and valid.shape == (0,)
    tok, valid = f(z[:0], u[:2], indices=i32(0, 3))     # no input row at all: every output row is out of range
    assert tok.tolist() == [-1, -1] and valid.tolist() == [0, 0]


def test_same_answer_alone_in_a_batch_and_replayed(ms):
    """A row's token depends on the row alone; a captured call replays with new inputs, on another stream."""
    import torch
    z = _logits(300, 20000, "bf16", 12)
    u = torch.from_numpy(_u(300, 5)).cuda()
    call = lambda z, u: ms.top_k_top_p_sampling_from_uniforms(z, u, 0.9, 300, 0.95)[0]
    whole = call(z, u)
    for b in (0, 7, 299):
        assert int(call(z[b:b + 1], u[b:b + 1])) == int(whole[b])
    zs, us = z[:5].clone(), u[:5].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(zs, us)
    for lo in (0, 50, 100):
        zs.copy_(z[lo:lo + 5])
        us.copy_(u[lo:lo + 5])
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        assert torch.equal(out, whole[lo:lo + 5])


def test_calls_on_two_streams_at_once(ms):
    import torch
    z = [_logits(64, 50000, "f32", 20 + i) for i in range(2)]
    u = [torch.from_numpy(_u(64, 30 + i)).cuda() for i in range(2)]
    want = [ms.top_k_top_p_sampling_from_uniforms(z[i], u[i], top_p=0.9)[0] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(ms.top_k_top_p_sampling_from_uniforms(z[i], u[i], top_p=0.9)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
