"""The decode-step operators together, as a serving loop uses them: a prompt's keys and values
appended to shared pages, n samples drawn from its last row, then decode steps that append each sample's
token to its own pages, attend over the shared prefix and the sample's suffix, and draw the next tokens;
the same loop in float64 (its keys, values and logits recomputed from the tokens drawn) must draw the same
tokens, and every attention output must agree."""
import numpy as np
import pytest

from oracle import decode
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_parallel_samples_of_one_prompt(dtype):
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300 as ms
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    g = torch.Generator().manual_seed(1)
    V, H, Hq, D, page, n, prompt, steps = 500, 2, 4, 64, 16, 6, 45, 5
    embed = lambda h: torch.randn(V, h, D, generator=g).to(dt).cuda()
    wk, wv, wq = embed(H), embed(H), embed(Hq)
    head = (torch.randn(Hq * D, V, generator=g) * 0.3).to(dt).cuda()
    inv = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).cuda()
    kc = torch.full((24, page, H, D), float("nan"), dtype=dt, device="cuda")   # unwritten slots are never read
    vc = torch.full_like(kc, float("nan"))
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    perm = np.random.default_rng(2).permutation(24)
    ptab, stab = i32(perm[None, :3]), i32(perm[3:9].reshape(n, 1))
    toks = torch.randint(0, V, (prompt,), generator=g)
    q = ms.append_paged_kv(wk[toks], wv[toks], kc, vc, ptab, i32(np.arange(prompt)), i32(np.zeros(prompt)), inv_freq=inv,
                           query=wq[toks])
    # the prompt's last token attends over the prompt: it is a row with no suffix
    plen = i32([prompt])
    out = ms.shared_prefix_attention(q[-1:], kc, vc, ptab, plen, i32(np.zeros((1, 1))), i32([0]))
    logits = out.flatten(1) @ head
    u = torch.rand(steps + 1, n, generator=g).cuda()
    tok, valid = ms.top_k_top_p_sampling_from_uniforms(logits, u[0], 0.9, 50, 0.95, indices=i32(np.zeros(n)))
    assert bool(valid.all())
    f = lambda t: t.double().cpu().numpy()
    fk, fv, fq = f(wk), f(wv), f(wq)
    inv_np = inv.cpu().numpy()
    hist = [[int(t) for t in toks] for _ in range(n)]

    def expect_tokens(lg, uu, got):
        lg = lg.float().cpu().numpy()
        for b in range(n):
            want, margin = decode.token_from_uniform(lg[b if len(lg) > 1 else 0], float(uu[b]), float(np.float32(0.9)), 50,
                                                     float(np.float32(0.95)))
            assert margin < 1e-9 or int(got[b]) == want

    expect_tokens(logits, u[0], tok)
    for s in range(steps):
        for b in range(n):
            hist[b].append(int(tok[b]))
        t = tok.long()
        pos = i32(np.full(n, s))
        q = ms.append_paged_kv(wk[t], wv[t], kc, vc, stab, pos, rotary_positions=i32(np.full(n, prompt + s)), inv_freq=inv,
                               query=wq[t])
        out, lse = ms.shared_prefix_attention(q, kc, vc, ptab, plen, stab, i32(np.full(n, s + 1)), return_lse=True)
        # the whole step from the tokens alone
        half = torch.finfo(dt).eps / 2
        for b in range(n):
            L = len(hist[b])
            k = np.stack([decode.rotate(fk[x], i, inv_np, False) for i, x in enumerate(hist[b])])
            v = np.stack([fv[x] for x in hist[b]])
            qq = decode.rotate(fq[hist[b][-1]], L - 1, inv_np, False)
            for h in range(Hq):
                sc = k[:, h // 2] @ qq[h] / 8.0
                p = np.exp(sc - sc.max())
                p /= p.sum()
                # rotated keys and queries are rounded to the type: each score is off by up to 2 half (1 + half) sum |q k|,
                # a weight by e^(twice that) - 1; then the operator's own tolerance
                e = np.expm1(2 * (2 * half * 1.01 * (np.abs(k[:, h // 2]) @ np.abs(qq[h])).max() / 8.0 + 2.0 ** -14))
                A = p @ np.abs(v[:, h // 2])
                o = p @ v[:, h // 2]
                assert (np.abs(f(out[b, h]) - o) <= (half + e) * A + half * np.abs(o)).all()
        logits = out.flatten(1) @ head
        tok, valid = ms.top_k_top_p_sampling_from_uniforms(logits, u[s + 1], 0.9, 50, 0.95)
        assert bool(valid.all())
        expect_tokens(logits, u[s + 1], tok)
    assert len({tuple(h) for h in hist}) > 1   # the samples went their own ways
