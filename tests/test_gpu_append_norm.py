"""Norms of queries and keys while appending (fs_append_paged_kv_normed) against float64.

Tolerance of an element of type t, before the rotation n = x r w: the sum of D squares in float32 (D + 1 roundings of
2^-24 of a sum of positive terms, half of that in its root), the reciprocal root (2^-22), the products with the
weights, cosines and the scale (4 roundings); then as without norms the rotation, (|n_x| + |n_y|) 2^-20 in
all for its part, and eps / 2 of the result: eps / 2 |y| + (|n_x| + |n_y|) (2^-20 + (D + 16) 2^-24)."""
import numpy as np
import pytest

from oracle import serving
from tests.helpers import ensure_built
from tests.test_gpu_paged_kv import _case, _inv, _np

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def ms():
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300
    return min_sampling_gb300


def _check(ms, c, inv, interleaved, sides="qk", rpos=None, eps=EPS, query_out=None, seed=0):
    import torch
    cu = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    rng = np.random.default_rng(seed)
    D = c["key"].shape[-1]
    weight = lambda: (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
    wq, wk = weight() if "q" in sides else None, weight() if "k" in sides else None
    half = torch.finfo(c["key"].dtype).eps / 2
    q_in, before_k, before_v = c["query"].clone(), _np(c["k"]), _np(c["v"])
    q = ms.append_paged_kv(c["key"], c["value"], c["k"], c["v"], cu(c["table"]), cu(c["pos"]), cu(c["rows"]),
                           rotary_positions=cu(rpos), inv_freq=cu(inv), interleaved=interleaved, query=c["query"], query_out=query_out,
                           query_norm=cu(wq), key_norm=cu(wk), norm_eps=eps)
    gk, gv, gq = _np(c["k"]), _np(c["v"]), _np(q)
    fr = [] if inv is None else inv
    page = gk.shape[1]

    def near(got, x, w, p):
        n = serving.norm_rotate(x, w, eps, 0, [], interleaved)
        want = serving.norm_rotate(x, w, eps, p, fr, interleaved)
        size = 2 * np.abs(n).max(-1, keepdims=True)
        return (np.abs(got - want) <= half * np.abs(want) + size * (2.0 ** -20 + (D + 16) * 2.0 ** -24)).all()

    for t, pos in enumerate(c["pos"]):
        if pos < 0:
            assert torch.equal(q[t], q_in[t])
            continue
        rp = int(pos if rpos is None else rpos[t])
        assert near(gq[t], _np(q_in[t]), wq, rp)
        r, i = int(c["rows"][t]), int(pos) // page
        if not (0 <= r < c["table"].shape[0] and i < c["table"].shape[1] and 0 <= c["table"][r, i] < gk.shape[0]):
            continue
        pg, s = c["table"][r, i], int(pos) % page
        assert near(gk[pg, s], _np(c["key"][t]), wk, rp) and (gv[pg, s] == _np(c["value"][t])).all()
        before_k[pg, s], before_v[pg, s] = gk[pg, s], gv[pg, s]
    assert (gk == before_k).all() and (gv == before_v).all()     # nothing else was written
    return q


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (7, 2, 8, 128, 128), (130, 8, 32, 128, 64), (33, 3, 3, 80, 32), (5, 1, 2, 128, 0),
                                   (9, 5, 10, 30, 18), (4, 2, 4, 256, 256), (3, 40, 70, 16, 16), (2, 1, 1, 1024, 1024), (6, 1, 2, 1, 0),
                                   (3, 33, 1, 8, 8)])
def test_shapes(ms, dtype, interleaved, shape):
    n, H, Hq, D, rotary = shape
    for page in (1, 16):
        _check(ms, _case(n + page, dtype, n, H, Hq, D, page, 400, 40, 4), _inv(rotary // 2) if rotary else None, interleaved, seed=n)


@pytest.mark.parametrize("n", [607, 608, 1216, 2432, 2600])
def test_tokens_of_a_cta(ms, n):
    """One, two and four tokens a CTA, whole and ragged."""
    _check(ms, _case(n, "bf16", n, 1, 3, 64, 16, 400, 100, 4), _inv(32), False)


@pytest.mark.parametrize("sides", ["q", "k", "qk"])
def test_one_side(ms, sides):
    for dtype in ("f32", "bf16"):
        _check(ms, _case(3, dtype, 20, 2, 6, 128, 16, 64, 8, 4), _inv(64), False, sides)
        _check(ms, _case(3, dtype, 20, 2, 6, 30, 16, 64, 8, 4), _inv(6), True, sides)


def test_sizes_of_the_data(ms):
    """Heads of zeros, large and small heads, eps of 0 and large."""
    c = _case(5, "f32", 6, 2, 4, 64, 16, 64, 8, 4)
    c["key"][1], c["query"][2] = 0, 0
    c["key"][2] *= 1e15
    c["query"][3] *= 1e-15
    _check(ms, c, _inv(32), False)
    _check(ms, c, _inv(32), False, eps=100.0)
    c["key"][1], c["query"][2] = 1, -1
    c["query"][3] = 1
    _check(ms, c, _inv(32), False, eps=0.0)


def test_padding_and_places_that_do_not_exist(ms):
    c = _case(5, "bf16", 12, 2, 4, 64, 16, 64, 8, 4)
    c["pos"][[0, 5]] = [-1, -2 ** 31]
    c["pos"][1], c["pos"][2] = 8 * 16, 2 ** 31 - 1
    c["rows"][3], c["rows"][4] = -1, 4
    c["table"][c["rows"][7], c["pos"][7] // 16] = 64
    _check(ms, c, _inv(32), False)
    _check(ms, c, _inv(32), True, rpos=np.arange(12).astype(np.int32) * 10 ** 8)


def test_in_place_strided_and_unaligned(ms):
    """Queries normed in place out of a fused projection; views that only single elements fit."""
    import torch
    for D, shift in ((128, 0), (128, 1), (1024, 0)):
        c = _case(8, "bf16", 9, 2, 4, D, 16, 64, 8, 4)
        buf = torch.zeros(9, 8 * D + 9, dtype=torch.bfloat16, device="cuda")
        fused = buf[:, shift:shift + 8 * D].unflatten(1, (8, D))
        fused[:, :4], fused[:, 4:6], fused[:, 6:] = c["query"], c["key"], c["value"]
        c["query"], c["key"], c["value"] = fused[:, :4], fused[:, 4:6], fused[:, 6:]
        q = c["query"]
        assert _check(ms, c, _inv(D // 2), False, query_out=q) is q


def test_without_norms_the_same_bits_as_before(ms):
    import torch
    for norms in (dict(), dict(query_norm=None, key_norm=None, norm_eps=5.0)):
        c = _case(9, "bf16", 30, 2, 4, 128, 16, 64, 8, 4)
        cu = lambda x: torch.from_numpy(x).cuda()
        args = [c["key"], c["value"], c["k"].clone(), c["v"].clone(), cu(c["table"]), cu(c["pos"]), cu(c["rows"])]
        q = ms.append_paged_kv(*args, inv_freq=cu(_inv(64)), query=c["query"], **norms)
        args2 = args[:2] + [c["k"].clone(), c["v"].clone()] + args[4:]
        q2 = ms.append_paged_kv(*args2, inv_freq=cu(_inv(64)), query=c["query"])
        assert torch.equal(q, q2) and torch.equal(args[2], args2[2])
