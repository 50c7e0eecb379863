"""What the decode step's entries refuse, and what they tell autograd."""
import pytest

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


def _append_args(dtype=None):
    import torch
    mk = lambda *s: torch.randn(s, device="cuda").to(dtype or torch.bfloat16)
    return dict(key=mk(3, 2, 64), value=mk(3, 2, 64), k_cache=mk(4, 8, 2, 64), v_cache=mk(4, 8, 2, 64),
                page_table=torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                positions=torch.tensor([0, 5, 7], dtype=torch.int32, device="cuda"), query=mk(3, 4, 64))


def _attend_args():
    import torch
    mk = lambda *s: torch.randn(s, device="cuda").bfloat16()
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    return dict(query=mk(3, 4, 64), k_cache=mk(8, 16, 2, 64), v_cache=mk(8, 16, 2, 64), prefix_table=i([0, 1]), prefix_lens=i(30),
                suffix_table=i([2], [3], [4]), suffix_lens=i(3, 16, 1))


# ------------------------------------------------------------------ forward-mode tangents

def test_tangents_are_refused(ms):
    """No forward-mode derivative is lost without a word, whether gradients are recorded or not."""
    import torch
    import torch.autograd.forward_ad as fw
    for f, args, names in ((ms.append_paged_kv, _append_args(torch.float32), ("key", "value", "k_cache", "v_cache", "query")),
                           (ms.shared_prefix_attention, _attend_args(), ("query", "k_cache", "v_cache"))):
        for name in names:
            with fw.dual_level():
                dual = fw.make_dual(args[name], torch.ones_like(args[name]))
                with pytest.raises(ValueError, match="tangent"):
                    f(**dict(args, **{name: dual}))
                with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                    f(**dict(args, **{name: dual}))
                f(**dict(args, **{name: fw.unpack_dual(dual).primal}))


# ------------------------------------------------------------------ versions

def test_written_tensors_get_a_new_version(ms):
    import torch
    t = _append_args()
    before = t["k_cache"]._version, t["v_cache"]._version, t["key"]._version, t["query"]._version
    q = ms.append_paged_kv(**t)
    assert t["k_cache"]._version > before[0] and t["v_cache"]._version > before[1]
    assert t["key"]._version == before[2] and t["query"]._version == before[3]
    res = torch.empty_like(t["query"])
    v = res._version
    assert ms.append_paged_kv(**t, query_out=res) is res and res._version > v and torch.equal(res, q)
    t = _attend_args()
    res = torch.empty_like(t["query"])
    v, kv = res._version, t["k_cache"]._version
    ms.shared_prefix_attention(**t, out=res)
    assert res._version > v and t["k_cache"]._version == kv


def test_a_saved_cache_that_changed_fails_the_backward_pass(ms):
    import torch
    t = _append_args(torch.float32)
    w = torch.ones(64, device="cuda", requires_grad=True)
    y = (t["k_cache"] * w).sum()          # saves the cache for w's gradient
    ms.append_paged_kv(**t)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inference_tensors_work(ms):
    import torch
    with torch.inference_mode():
        t, u = _append_args(), _attend_args()
        ms.append_paged_kv(**t, query_out=torch.empty_like(t["query"]))
        ms.shared_prefix_attention(**u, out=torch.empty_like(u["query"]))
    q = ms.append_paged_kv(**t)           # and outside of it
    assert torch.equal(q, t["query"])


def test_a_refused_call_changes_no_version(ms):
    t = _append_args()
    before = t["k_cache"]._version
    with pytest.raises(ValueError):
        ms.append_paged_kv(**dict(t, positions=t["positions"][:2]))
    assert t["k_cache"]._version == before


# ------------------------------------------------------------------ shared memory

def test_appending_refuses_tensors_that_share_memory(ms):
    import torch
    t = _append_args()
    f = ms.append_paged_kv
    kept = {n: t[n].clone() for n in ("k_cache", "v_cache", "key", "query")}
    dense = t["k_cache"]
    flat = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    strided = lambda st: flat.as_strided(dense.shape, st)
    bad = [dict(k_cache=strided((960, 120, 60, 1))),       # heads of 64, 60 apart
           dict(k_cache=strided((960, 64, 64, 1))),        # slots on top of one another's heads
           dict(v_cache=strided((1000, 128, 64, 1))),      # pages of 1024
           dict(v_cache=dense), dict(k_cache=t["v_cache"]), dict(v_cache=dense.view(32, 2, 64).view(4, 8, 2, 64)),
           dict(query_out=t["query"][:, :1].as_strided((3, 4, 64), (256, 32, 1))),
           dict(query_out=t["k_cache"].view(-1)[:768].view(3, 4, 64)),
           dict(key=t["k_cache"][0, :3]), dict(value=t["v_cache"][1, 1:4]), dict(value=t["k_cache"][3, 5:])]
    qkv = torch.randn(3, 8 * 64 + 64, device="cuda").bfloat16()
    q, k, v = qkv[:, :256].view(3, 4, 64), qkv[:, 256:384].view(3, 2, 64), qkv[:, 384:512].view(3, 2, 64)
    late = qkv[:, 64:320].view(3, 4, 64)
    bad += [dict(query=q, query_out=late), dict(query=q, key=k, query_out=late), dict(query=late, value=v, query_out=qkv[:, 192:448].view(3, 4, 64))]
    for b in bad:
        with pytest.raises(ValueError, match="share"):
            f(**{**t, **b})
    assert all(torch.equal(t[n], x) for n, x in kept.items()) and not bool(flat.any())
    # in one buffer, but apart: fused projections rotated in place, keys and values of a page beside one another,
    # heads of keys and values in turn
    assert f(**{**t, **dict(query=q, key=k, value=v, query_out=q)}) is q
    both = torch.zeros(4, 2, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
    f(**{**t, **dict(k_cache=both[:, 0], v_cache=both[:, 1])})
    assert torch.equal(both[0, 0, 0], t["key"][0]) and torch.equal(both[2, 1, 7], t["value"][2])
    turn = torch.zeros(4, 8, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    f(**{**t, **dict(k_cache=turn[:, :, :, 0], v_cache=turn[:, :, :, 1])})
    assert torch.equal(turn[1, 5, :, 0], t["key"][1]) and torch.equal(turn[1, 5, :, 1], t["value"][1])
    whole = torch.zeros(4, 8, 2, 128, dtype=torch.bfloat16, device="cuda")
    f(**{**t, **dict(k_cache=whole[..., :64], v_cache=whole[..., 64:])})
    assert torch.equal(whole[0, 0], torch.cat([t["key"][0], t["value"][0]], -1))


def test_attention_refuses_outputs_that_share_memory(ms):
    import torch
    t = _attend_args()
    f = ms.shared_prefix_attention
    kept = {n: t[n].clone() for n in ("query", "k_cache", "v_cache")}
    want = f(**t)
    wide = torch.zeros(3, 6, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5] = t["query"]
    for b in (dict(out=t["k_cache"].view(-1)[:768].view(3, 4, 64)), dict(out=t["v_cache"].view(-1)[-768:].view(3, 4, 64)),
              dict(out=torch.zeros(2048, dtype=torch.bfloat16, device="cuda").as_strided((3, 4, 64), (128, 64, 1))),
              dict(query=wide[:, 1:5], out=wide[:, 2:]), dict(query=wide[:, 1:5], out=wide[:, :4])):
        with pytest.raises(ValueError, match="share"):
            f(**{**t, **b})
    assert all(torch.equal(t[n], x) for n, x in kept.items())
    # the query's own memory is fine, and so are neighbours in one buffer
    assert torch.equal(f(**t, out=torch.empty_like(want)), want)
    two = torch.zeros(3, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    two[:, 0] = t["query"]
    assert torch.equal(f(**{**t, **dict(query=two[:, 0], out=two[:, 1])}), want)


@pytest.mark.parametrize("rows,Q", [(3, 1), (3, 5), (34, 1), (34, 3)])
@pytest.mark.parametrize("prefix,own", [(40, 16), (40, 600), (800, 16), (800, 600), (800, 1100)])
def test_attention_into_the_query(ms, rows, Q, prefix, own):
    """`out` may be the query: every plan has read it before it writes."""
    import torch
    from tests.test_gpu_prefix_attention import _call, _case
    for D in (64, 128, 256):
        c = _case(51, "bf16", [rows], rows, Q, 8, 2, D, [prefix], [own] * rows, 16)
        want, lse = _call(ms, c)
        q = c["q"].clone()
        out, lse2 = _call(ms, dict(c, q=q), out=q)
        assert out is q and torch.equal(q, want) and torch.equal(lse, lse2)
