"""The serving step's operators together: requests of different lengths get their prompts in chunks while
others decode, from page tables made on the GPU to sampled tokens; the same loop in float64, recomputed from the tokens
drawn, must draw the same tokens, and every attention output must agree."""
import numpy as np
import pytest

from oracle import decode, serving
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,window,sinks", [("bf16", None, 0), ("f16", None, 0), ("bf16", 24, 2)])
def test_continuous_batch(dtype, window, sinks):
    ensure_built()
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import min_sampling_gb300 as ms
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    g = torch.Generator().manual_seed(1)
    V, H, Hq, D, page, width, pages, chunk, budget = 300, 2, 8, 64, 8, 12, 60, 25, 64
    embed = lambda h: torch.randn(V, h, D, generator=g).to(dt).cuda()
    wk, wv, wq = embed(H), embed(H), embed(Hq)
    head = (torch.randn(Hq * D, V, generator=g) * 0.3).to(dt).cuda()
    inv = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    nq, nk = (torch.from_numpy((1 + 0.2 * np.random.default_rng(i).standard_normal(D)).astype(np.float32)).cuda() for i in (2, 3))
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    f = lambda t: t.double().cpu().numpy()
    fk, fv, fq, fnq, fnk = f(wk), f(wv), f(wq), f(nq), f(nk)
    prompts = [torch.randint(0, V, (n,), generator=g).tolist() for n in (70, 3, 26, 41)]
    R = len(prompts)
    hist, done = [list(p) for p in prompts], [0] * R           # tokens of each request; how many the cache holds
    kc = torch.full((pages, page, H, D), float("nan"), dtype=dt, device="cuda")   # unwritten slots are never read
    vc = torch.full_like(kc, float("nan"))
    table, stack = i32(np.full((R, width), -1)), i32(np.random.default_rng(4).permutation(pages))
    lens, count = i32(np.zeros(R)), i32([pages])
    inv_t = torch.from_numpy(inv).cuda()
    half = torch.finfo(dt).eps / 2
    drawn = [0] * R
    for step in range(9):
        new = [min(chunk, len(h) - d) for h, d in zip(hist, done)]
        starts, rows, pos, lens, count = ms.paged_step_tables(lens, i32(new), table, stack, count, page, budget)
        st = starts.tolist()
        new = [st[r + 1] - st[r] for r in range(R)]     # all that was asked for, or nothing where the budget ended
        ids = [h[d:d + n] for h, d, n in zip(hist, done, new)]
        toks = torch.tensor(sum(ids, []) + [0] * (budget - st[-1]))
        q = ms.append_paged_kv(wk[toks], wv[toks], kc, vc, table, pos, rows, inv_freq=inv_t, query=wq[toks], query_norm=nq, key_norm=nk)
        out, lse = ms.paged_chunk_attention(q, kc, vc, table, starts, lens, window=window, sinks=sinks, return_lse=True)
        assert bool((out[st[-1]:] == 0).all())
        done = [d + n for d, n in zip(done, new)]
        for r in range(R):
            n = done[r]
            if not new[r]:
                continue
            k = np.stack([serving.norm_rotate(fk[x], fnk, 1e-6, i, inv, False) for i, x in enumerate(hist[r][:n])])
            v = np.stack([fv[x] for x in hist[r][:n]])
            for j in {0, new[r] // 2, new[r] - 1}:
                p = n - new[r] + j
                qq = serving.norm_rotate(fq[hist[r][p]], fnq, 1e-6, p, inv, False)
                t = np.arange(p + 1)
                t = t[(t > p - (window or 10 ** 9)) | (t < sinks)]
                for h in range(Hq):
                    sc = k[t, h // 4] @ qq[h] / 8.0
                    w = np.exp(sc - sc.max())
                    w /= w.sum()
                    # keys and queries are rounded to the type: each score is off by up to 2 half (1 + half) sum |q k|, a weight
                    # by e^(twice that) - 1; then the operator's own tolerance
                    e = np.expm1(2 * (2 * half * 1.01 * (np.abs(k[t, h // 4]) @ np.abs(qq[h])).max() / 8.0 + 2.0 ** -14))
                    A, o = w @ np.abs(v[t, h // 4]), w @ v[t, h // 4]
                    assert (np.abs(f(out[st[r] + j, h]) - o) <= (half + e) * A + half * np.abs(o)).all()
        # requests whose whole text is in the cache draw a token from their last row
        ready = [r for r in range(R) if new[r] and done[r] == len(hist[r])]
        if not ready:
            continue
        logits = out[i32([st[r + 1] - 1 for r in ready]).long()].flatten(1) @ head
        L = max(len(h) for h in hist)
        tokens = i32([hist[r] + [0] * (L - len(hist[r])) for r in ready])
        banned = np.zeros((1, 32 * (-(-V // 32))), np.uint8)
        banned[0, :V] = np.arange(V) % 5 != 0
        mask = i32(np.packbits(banned, axis=1, bitorder="little").view(np.int32))
        adj = ms.adjust_logits(logits, tokens, i32([len(hist[r]) for r in ready]), i32([len(prompts[r]) for r in ready]), repetition=1.3,
                               presence=0.4, frequency=0.2, allowed=mask, allowed_rows=i32([0 if r % 2 else -1 for r in ready]))
        u = torch.rand(len(ready), generator=g)
        tok, valid = ms.top_k_top_p_sampling_from_uniforms(adj, u.cuda(), 0.9, 50, 0.95)
        assert bool(valid.all())
        for i, r in enumerate(ready):
            z, big = serving.adjust_row(f(logits[i]), hist[r], len(prompts[r]), np.float32(1.3), np.float32(0.4), np.float32(0.2),
                                        allowed=None if r % 2 == 0 else banned[0, :V])
            a = f(adj[i])
            assert (np.isneginf(a) == np.isneginf(z)).all()
            fin = np.isfinite(z)
            assert (np.abs(a[fin] - z[fin]) <= half * np.abs(z[fin]) + 2.0 ** -22 * big[fin]).all()
            want, margin = decode.token_from_uniform(adj[i].float().cpu().numpy(), float(u[i]), float(np.float32(0.9)), 50,
                                                     float(np.float32(0.95)))
            assert margin < 1e-9 or int(tok[i]) == want
            if r % 2:
                assert int(tok[i]) % 5 != 0
            hist[r].append(int(tok[i]))
            drawn[r] += 1
    assert min(drawn) >= 4 and int(count[0]) == pages - sum(-(-d // page) for d in done)
