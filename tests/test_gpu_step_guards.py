"""What the serving step's entries refuse, and what they tell autograd."""
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


def _i(*v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _chunk(dtype=None):
    import torch
    mk = lambda *s: torch.randn(s, device="cuda").to(dtype or torch.bfloat16)
    return dict(query=mk(5, 4, 64), k_cache=mk(8, 16, 2, 64), v_cache=mk(8, 16, 2, 64), page_table=_i([0, 1], [2, 3]), query_starts=_i(0, 4, 5),
                lens=_i(20, 17))


def _tables():
    return dict(lens=_i(3, 16), new_lens=_i(1, 1), page_table=_i([0, -1], [1, -1]), free_pages=_i(7, 8, 9), free_count=_i(3), page_size=16,
                max_tokens=4)


def _adjust():
    import torch
    return dict(logits=torch.randn(2, 40, device="cuda"), tokens=_i([1, 2, 3], [4, 4, 5]), lens=_i(3, 2), prompt_lens=_i(1, 0),
                repetition=torch.full((2,), 1.5, device="cuda"), bias_starts=_i(0, 1, 1), bias_tokens=_i(3),
                bias_values=torch.ones(1, device="cuda"), allowed=_i([-1, 3], [7, 0]), allowed_rows=_i(0, -1))


def _norm():
    from tests.test_gpu_decode_guards import _append_args
    import torch
    return dict(_append_args(torch.float32), query_norm=torch.ones(64, device="cuda"), key_norm=torch.ones(64, device="cuda"))


def test_shapes_types_and_values(ms):
    import torch
    for f, base, bads in (
            (ms.paged_step_tables, _tables(), [dict(lens=_i(3)), dict(new_lens=_i(1, 1, 1)), dict(page_table=_i(0, 1)), dict(free_pages=_i([7])),
                                               dict(free_count=_i(1, 2)), dict(page_size=0), dict(max_tokens=-1), dict(lens=_i(3, 16).long()),
                                               dict(free_count=torch.tensor([3], dtype=torch.int32))]),
            (ms.paged_chunk_attention, _chunk(), [dict(query_starts=_i(0, 4)), dict(lens=_i(1, 2, 3)), dict(page_table=_i(0, 1)), dict(window=0),
                                                  dict(window=-4), dict(sinks=-1), dict(max_queries=0), dict(lens=_i(20, 17).float()),
                                                  dict(query=_chunk()["query"][:, :3]), dict(query=_chunk()["query"].half()),
                                                  dict(query=_chunk()["query"][..., :32])]),
            (ms.adjust_logits, _adjust(), [dict(tokens=_i([1, 2, 3])), dict(lens=_i(1)), dict(prompt_lens=_i(1).float()), dict(tokens=None),
                                           dict(bias_starts=_i(0, 1)), dict(bias_values=None), dict(bias_tokens=_i(1, 2)), dict(allowed=_i([1], [2])),
                                           dict(allowed=None), dict(allowed_rows=_i(0)), dict(repetition=torch.ones(2, device="cuda").half()),
                                           dict(logits=torch.zeros(2, 40, device="cuda", dtype=torch.float64)),
                                           dict(logits=torch.zeros(40, 2, device="cuda").T), dict(out=torch.zeros(2, 41, device="cuda")),
                                           dict(out=torch.zeros(2, 40, device="cuda").half()), dict(allowed=_i([1, 2]), allowed_rows=None),
                                           dict(logits=torch.zeros(1, 40, device="cuda").expand(2, 40))]),
            (ms.append_paged_kv, _norm(), [dict(query_norm=torch.ones(63, device="cuda")), dict(key_norm=torch.ones(64, device="cuda").half()),
                                           dict(query=None), dict(norm_eps=-1.0), dict(norm_eps=float("nan")),
                                           dict(key_norm=torch.ones(128, device="cuda")[::2])])):
        f(**base)
        for bad in bads:
            with pytest.raises(ValueError):
                f(**{**base, **bad})
    with pytest.raises(ms.FsError):
        c = _chunk()
        ms.paged_chunk_attention(c["query"][..., :48].contiguous(), c["k_cache"][..., :48].contiguous(), c["v_cache"][..., :48].contiguous(),
                                 c["page_table"], c["query_starts"], c["lens"])


def test_gradients_and_tangents_are_refused(ms):
    import torch
    import torch.autograd.forward_ad as fw
    for f, args, names in ((ms.paged_chunk_attention, _chunk(), ("query", "k_cache", "v_cache")),
                           (ms.adjust_logits, _adjust(), ("logits", "repetition", "bias_values")),
                           (ms.append_paged_kv, _norm(), ("query_norm", "key_norm", "key", "query"))):
        for name in names:
            t = args[name].clone().requires_grad_()
            with pytest.raises(ValueError, match="backward"):
                f(**{**args, name: t})
            with torch.no_grad():
                f(**{**args, name: t})
            with fw.dual_level():
                dual = fw.make_dual(args[name], torch.ones_like(args[name]))
                with pytest.raises(ValueError, match="tangent"):
                    f(**{**args, name: dual})


def test_written_tensors_get_a_new_version(ms):
    import torch
    t = _tables()
    v, w = t["page_table"]._version, t["lens"]._version
    ms.paged_step_tables(**t)
    assert t["page_table"]._version > v and t["lens"]._version == w
    c = _chunk()
    res = torch.empty_like(c["query"])
    v = res._version
    assert ms.paged_chunk_attention(**c, out=res) is res and res._version > v
    a = _adjust()
    v = a["logits"]._version
    ms.adjust_logits(**a)
    assert a["logits"]._version == v
    ms.adjust_logits(**a, out=a["logits"])
    assert a["logits"]._version > v
    with torch.inference_mode():
        ms.adjust_logits(**_adjust(), out=torch.empty(2, 40, device="cuda"))
        ms.paged_step_tables(**_tables())
        ms.paged_chunk_attention(**_chunk(), out=torch.empty(5, 4, 64, device="cuda", dtype=torch.bfloat16))


def test_outputs_that_share_memory_are_refused(ms):
    import torch
    c = _chunk()
    kept = {n: c[n].clone() for n in ("query", "k_cache", "v_cache")}
    wide = torch.zeros(5, 6, 64, dtype=torch.bfloat16, device="cuda")
    for b in (dict(out=c["k_cache"].view(-1)[:1280].view(5, 4, 64)), dict(out=c["v_cache"].view(-1)[-1280:].view(5, 4, 64)),
              dict(query=wide[:, 1:5], out=wide[:, 2:]), dict(out=wide.view(-1)[:1024].as_strided((5, 4, 64), (128, 64, 1)))):
        with pytest.raises(ValueError, match="share"):
            ms.paged_chunk_attention(**{**c, **b})
    assert all(torch.equal(c[n], x) for n, x in kept.items())
    a = _adjust()
    buf = torch.zeros(200, device="cuda")
    for b in (dict(logits=buf[:80].view(2, 40), out=buf[4:84].view(2, 40)), dict(out=buf.as_strided((2, 40), (0, 1))),
              dict(out=buf.as_strided((2, 40), (20, 1))), dict(tokens=buf[:6].view(torch.int32).view(2, 3), out=buf[:80].view(2, 40)),
              dict(repetition=buf[3:5], out=buf[:80].view(2, 40)), dict(allowed=buf[:4].view(torch.int32).view(2, 2), out=buf[2:82].view(2, 40))):
        with pytest.raises(ValueError):
            ms.adjust_logits(**{**a, **b})
    t = _tables()
    room = torch.zeros(20, dtype=torch.int32, device="cuda")
    for b in (dict(lens=room[:2], page_table=room[:4].view(2, 2)), dict(free_pages=room[3:9], page_table=room[:4].view(2, 2)),
              dict(free_count=room[3:4], page_table=room[:4].view(2, 2)), dict(new_lens=room[1:3], page_table=room[:4].view(2, 2))):
        with pytest.raises(ValueError, match="share"):
            ms.paged_step_tables(**{**t, **b})
    ms.paged_step_tables(**{**t, **dict(lens=room[4:6], page_table=room[:4].view(2, 2))})


@pytest.mark.parametrize("name", ["page_table", "query_starts", "lens"])
def test_an_output_over_the_places_is_refused(ms, name):
    import torch
    c = _chunk()
    room = torch.zeros(1280, dtype=torch.bfloat16, device="cuda")
    x = c[name]
    over = room.view(torch.int32)[:x.numel()].view(x.shape)
    over.copy_(x)
    with pytest.raises(ValueError, match="share"):
        ms.paged_chunk_attention(**{**c, name: over}, out=room.view(5, 4, 64))
    assert torch.equal(over, x)
