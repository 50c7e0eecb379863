"""The binding's check for tensors that share memory, against the sets of addresses (no GPU)."""
import random

import pytest

from tests.helpers import ensure_built


@pytest.fixture(scope="module")
def shares():
    ensure_built()
    import min_sampling_gb300 as ms
    return ms._native().shares_memory


def _addresses(t):
    import itertools
    return [t.data_ptr() + t.element_size() * sum(i * s for i, s in zip(x, t.stride())) for x in itertools.product(*map(range, t.shape))]


def test_random_views(shares):
    import torch
    rng = random.Random(1)
    buf = torch.zeros(6000, dtype=torch.bfloat16)

    def view():
        d = rng.randint(0, 4)
        shape = [rng.choice([1, 1, 2, 3, 4, 5]) for _ in range(d)]
        if rng.random() < 0.4:      # nested in some order, with gaps
            strides, at = [0] * d, 1
            for i in rng.sample(range(d), d):
                strides[i] = at + rng.choice([0, 0, 1, 3])
                at = strides[i] * shape[i]
        else:
            strides = [rng.choice([0, 1, 1, 2, 3, 4, 6, 8, 12, 30]) for _ in range(d)]
        return buf.as_strided(shape, strides, rng.randint(0, 90))

    seen = set()
    for _ in range(4000):
        a, b = view(), view()
        A, B = _addresses(a), _addresses(b)
        assert shares(a, a) == (len(set(A)) < len(A)), (a.shape, a.stride())
        want = bool(set(A) & set(B))
        assert shares(a, b) == want == shares(b, a), (a.shape, a.stride(), b.shape, b.stride())
        seen.add(want)
    assert seen == {True, False}


def test_layouts_in_use(shares):
    import torch
    qkv = torch.zeros(50, 48 * 128)
    q, k, v = qkv[:, :4096].view(50, 32, 128), qkv[:, 4096:5120].view(50, 8, 128), qkv[:, 5120:].view(50, 8, 128)
    assert not (shares(q, k) or shares(q, v) or shares(k, v) or shares(q, q)) and shares(q, qkv) and shares(qkv[3], v)
    both = torch.zeros(40, 2, 16, 8, 64)
    a, b = both[:, 0], both[:, 1]
    heads_first = both.transpose(2, 3)
    assert not (shares(a, b) or shares(a, a) or shares(heads_first[:, 0], b)) and shares(heads_first[:, 1], b)
    wide = torch.zeros(40, 16, 8, 128)
    assert not shares(wide[..., :64], wide[..., 64:]) and shares(wide[..., :65], wide[..., 64:])
    assert not shares(wide[::2], wide[1::2]) and shares(wide[::2], wide[2:])
    assert shares(wide[:1].expand(4, 16, 8, 128), wide[0]) and shares(t := wide[:1].expand(4, 16, 8, 128), t)
    assert not shares(wide[:0], wide) and not shares(wide[:0], wide[:0])
    far = torch.empty(1, dtype=torch.bfloat16).expand(2 ** 20, 16, 8, 128)     # sizes whose products pass 32 bits
    assert shares(far, wide.bfloat16()) is False


def test_strides_that_do_not_nest_end(shares):
    """Strides without any order: an answer comes soon, and is never a wrong no."""
    import torch
    buf = torch.zeros(1 << 16)
    rng = random.Random(2)
    for _ in range(200):
        a, b = (buf.as_strided([rng.randint(2, 9) for _ in range(4)], [rng.randint(1, 997) for _ in range(4)], rng.randint(0, 999))
                for _ in range(2))
        if set(_addresses(a)) & set(_addresses(b)):
            assert shares(a, b)
