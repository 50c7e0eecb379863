"""The measured cases of the serving-step operators: page tables and token places from request
lengths, norms of queries and keys with the rotation while appending, attention of chunks of new
tokens over a paged cache (with a sliding window and first tokens that stay visible), and
penalties, biases and grammar masks on logits.

Each case is a dict of plain values.  ``run`` makes one pass through the operator: in its
plain form (elementary torch operations) while ``own`` is false, through the package's
public entry points while it is true.  ``exact`` computes the same outputs in 64 bits, apart
from the plain form.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decode step of 64 requests: a token each, a page for those that fill theirs.  Latency.
        dict(name="tables_decode", op="tables", decode=64, chunks=0, chunk=0, context=32768, page=16, budget=64, short=False),
        # A step of a large server: 1500 requests decode, 12 prompts get a chunk, padded to 16384 tokens.
        dict(name="tables_mixed", op="tables", decode=1500, chunks=12, chunk=1201, context=8190, page=16, budget=16384,
             short=False),
        # One decode step of 64 samples: norms, rotation and appending of a token each.
        dict(name="append_norm_decode", op="append", seqs=64, tokens=64, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, dtype="bf16", page=16, context=32768),
        # A prefill of ragged prompts, 8190 tokens together.
        dict(name="append_norm_prefill", op="append", seqs=5, tokens=8190, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, dtype="bf16", page=16, context=2048),
        # One request's row with a history of a thousand tokens: latency.
        dict(name="adjust_one_row", op="adjust", rows=1, vocab=32000, pad=0, dtype="bf16", history=1000, bias=20, masks=0),
        # The benchmark's own batch (64 rows of 151936 logits) with all penalties, long histories and biases.
        dict(name="adjust_penalties", op="adjust", rows=64, vocab=151936, pad=0, dtype="f32", history=4096, bias=300, masks=0),
        # A large batch, half of its rows held to a grammar, rows of an odd vocabulary in a padded buffer.
        dict(name="adjust_grammar", op="adjust", rows=256, vocab=151665, pad=271, dtype="bf16", history=700, bias=0, masks=128),
        # A short prompt's last piece: latency.
        dict(name="chunk_short", op="chunk", decode=0, context=0, chunks=1, chunk=37, past=1000, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", page=16, window=0, sinks=0),
        # A decode step of 64 requests of all lengths up to 8192: the caches' bytes bound it.
        dict(name="chunk_decode", op="chunk", decode=64, context=8192, chunks=0, chunk=0, past=0, q_heads=32, kv_heads=8,
             dim=128, dtype="bf16", page=16, window=0, sinks=0),
        # A whole prompt at once: matrix products bound it.
        dict(name="chunk_prefill", op="chunk", decode=0, context=0, chunks=1, chunk=8190, past=0, q_heads=32, kv_heads=8,
             dim=128, dtype="bf16", page=16, window=0, sinks=0),
        # Chunks of two long prompts beside 47 requests that decode.
        dict(name="chunk_mixed", op="chunk", decode=47, context=6000, chunks=2, chunk=1021, past=16384, q_heads=32, kv_heads=8,
             dim=128, dtype="bf16", page=16, window=0, sinks=0),
        # A sliding window of 1024 with four first tokens, long chunks behind long contexts.
        dict(name="chunk_window", op="chunk", decode=13, context=9000, chunks=4, chunk=2050, past=12000, q_heads=16, kv_heads=8,
             dim=64, dtype="f16", page=64, window=1024, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "adjust", "adjust", "chunk", "chunk", "chunk"])
    if op == "tables":
        chunks = rng.choice([0, 0, rng.randint(1, 12)])
        decode, chunk = _log_int(rng, 1, 1500), _log_int(rng, 2, 1200) if chunks else 0
        total = decode + chunks * chunk
        return dict(op=op, decode=decode, chunks=chunks, chunk=chunk, context=_log_int(rng, 1, 8000),
                    page=rng.choice([1, 5, 16, 64]), budget=max(1, int(total * rng.choice([0.7, 1.0, 1.1]))),
                    short=rng.random() < 0.3)
    dt = rng.choice(["bf16", "f16"])
    if op == "append":
        dim = rng.choice([64, 128, 256])
        kvh = rng.randint(1, 8)
        seqs = rng.randint(1, 64)
        return dict(op=op, seqs=seqs, tokens=max(seqs, _log_int(rng, 1, 4000)), q_heads=kvh * rng.randint(1, 4),
                    kv_heads=kvh, dim=dim, rotary=rng.choice([dim, dim // 2]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f16", "f32"]), page=rng.choice([1, 5, 16, 64]), context=_log_int(rng, 1, 4000))
    if op == "adjust":
        vocab = _log_int(rng, 1000, 256000)
        rows = min(_log_int(rng, 1, 256), max(1, 256 * 151665 // vocab // 2))
        return dict(op=op, rows=rows, vocab=vocab, pad=rng.choice([0, 0, 1, 8, 77]), dtype=rng.choice(["f32", "bf16", "f16"]),
                    history=rng.choice([0, _log_int(rng, 1, 4000), _log_int(rng, 1, 4000)]),
                    bias=rng.choice([0, min(vocab // 2, _log_int(rng, 1, 300))]),
                    masks=rng.choice([0, rng.randint(1, rows)]))
    kvh = rng.randint(1, 8)
    chunks = rng.randint(0, 5)
    return dict(op=op, decode=rng.choice([0, _log_int(rng, 1, 48)]) if chunks else _log_int(rng, 1, 48),
                context=_log_int(rng, 1, 6000), chunks=chunks, chunk=_log_int(rng, 2, 1500) if chunks else 0,
                past=rng.choice([0, _log_int(rng, 1, 6000)]) if chunks else 0, q_heads=kvh * rng.choice([1, 2, 4, 5, 8]),
                kv_heads=kvh, dim=rng.choice([64, 128]), dtype=dt, page=rng.choice([1, 5, 16, 64]),
                **rng.choice([dict(window=0, sinks=0), dict(window=0, sinks=0),
                              dict(window=_log_int(rng, 1, 3000), sinks=rng.choice([0, 1, 4, 130]))]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).cuda()


def _requests(c):
    """Tokens in the cache and new tokens of each request, before the seed's order: requests that decode one token
    with contexts spread up to the case's, then chunks of decreasing length."""
    n, past = [], []
    for i in range(c["decode"]):
        past.append((c["context"] - 1) * (i + 1) // c["decode"])
        n.append(1)
    for i in range(c["chunks"]):
        n.append(max(1, c["chunk"] - (i * c["chunk"]) // (4 * c["chunks"])))
        p = c["past"] if "past" in c else c["context"]
        past.append(p - (i * p) // (3 * c["chunks"]))
    return np.array(past, np.int64), np.array(n, np.int64)


def _tables_inputs(c, seed):
    g = _gen(seed)
    past, n = _requests(c)
    order = torch.randperm(len(n), generator=g, device="cuda").cpu().numpy()
    past, n = past[order], n[order]
    page = c["page"]
    have, want = -(-past // page), -(-(past + n) // page)
    need = int((want - have).sum())
    # The stack of free pages; too few of them for the last requests in some cases.
    free = max(1, need // 2) if c["short"] else need + 1000
    total = int(have.sum()) + free
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = int(want.max()) + 3
    table = np.full((len(n), width), -1, np.int32)
    host, at = ids.cpu().numpy(), 0
    for r, m in enumerate(have):
        table[r, :m] = host[at:at + m]
        at += int(m)
    # The stack's buffer has room for every page.
    stack = torch.cat((ids[at:], ids.new_full((at,), -1)))
    return dict(case=c, lens=_i32(past), new_lens=_i32(n), page_table=torch.from_numpy(table).cuda(), free_pages=stack,
                free_count=_i32([free]))


def _append_inputs(c, seed):
    g = _gen(seed)
    dt = DTYPES[c["dtype"]]
    N, R, page = c["tokens"], c["seqs"], c["page"]
    # Tokens dealt to the sequences in runs, each run behind a context of its own length.
    per = np.full(R, N // R, np.int64)
    per[: N - int(per.sum())] += 1
    start = torch.randint(0, c["context"] + 1, (R,), generator=g, device="cuda").cpu().numpy()
    rows = np.repeat(np.arange(R), per)
    pos = np.concatenate([start[r] + np.arange(per[r]) for r in range(R)])
    pages_of = (start + per + page - 1) // page
    # Only the pages that this call writes are backed by memory of their own; a sequence's earlier
    # pages all name the last page of the pool.
    first = start // page
    owned = (pages_of - first).astype(np.int64)
    total = int(((per + 2 * page - 2) // page).sum()) + 1  # as many as any start within a page can take
    order = torch.randperm(total - 1, generator=g, device="cuda").cpu().numpy()
    table = np.full((R, int(pages_of.max())), total - 1, np.int32)
    at = 0
    for r in range(R):
        table[r, first[r]:pages_of[r]] = order[at:at + owned[r]]
        at += owned[r]
    half = c["rotary"] // 2
    inv = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    H, D = c["kv_heads"], c["dim"]
    weight = lambda: 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
    return dict(case=c, key=_normal(g, (N, H, D), dt) * 3, value=_normal(g, (N, H, D), dt),
                query=_normal(g, (N, c["q_heads"], D), dt) * 2, k_cache=_normal(g, (total, page, H, D), dt),
                v_cache=_normal(g, (total, page, H, D), dt), page_table=torch.from_numpy(table).cuda(), rows=_i32(rows),
                positions=_i32(pos), inv_freq=inv, query_norm=weight(), key_norm=weight())


def _adjust_inputs(c, seed):
    g = _gen(seed)
    B, V, L, M = c["rows"], c["vocab"], c["history"], c["masks"]
    buf = torch.empty((B, V + c["pad"]), dtype=DTYPES[c["dtype"]], device="cuda")
    for i in range(0, B, 64):  # in slices, to keep the fp32 temporaries small
        n = min(64, B - i)
        buf[i:i + n] = (torch.randn((n, V + c["pad"]), generator=g, device="cuda") * 3.0).to(buf.dtype)
    s = dict(case=c, logits=buf[:, :V], tokens=None, lens=None, prompt_lens=None, repetition=None, presence=None, frequency=None,
             bias_starts=None, bias_tokens=None, bias_values=None, allowed=None, allowed_rows=None)
    spread = torch.rand(B, generator=g, device="cuda")
    if L:
        # Histories repeat some tokens often: the square of a uniform number, over the vocabulary.
        u = torch.rand((B, L), generator=g, device="cuda", dtype=torch.float64)
        s["tokens"] = torch.clamp((u * u * V).int(), max=V - 1)
        lens = L - (np.arange(B, dtype=np.int64) * L) // (2 * B)
        s["lens"] = _i32(lens)[torch.randperm(B, generator=g, device="cuda")].contiguous()
        s["prompt_lens"] = (s["lens"] * spread).int()
        s["repetition"] = 1.0 + 0.3 * spread
        s["presence"] = 0.8 * torch.rand(B, generator=g, device="cuda")
        s["frequency"] = 0.3 * torch.rand(B, generator=g, device="cuda")
    if c["bias"]:
        # Distinct tokens of each row, up to the case's count.
        n = np.array([max(1, c["bias"] - (i * c["bias"]) // (2 * B)) for i in range(B)])
        step = V // c["bias"]
        ids = (torch.arange(c["bias"], device="cuda") * step
               + torch.randint(0, step, (B, c["bias"]), generator=g, device="cuda")).int()
        s["bias_starts"] = _i32(np.concatenate([[0], np.cumsum(n)]))
        s["bias_tokens"] = torch.cat([ids[i, :n[i]] for i in range(B)])
        s["bias_values"] = 4.0 * torch.randn(s["bias_tokens"].numel(), generator=g, device="cuda")
    if M:
        s["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (M, (V + 31) // 32), generator=g, device="cuda").int()
        rows = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        rows[torch.randperm(B, generator=g, device="cuda")[:M]] = torch.arange(M, dtype=torch.int32, device="cuda")
        s["allowed_rows"] = rows
    return s


def _chunk_inputs(c, seed):
    g = _gen(seed)
    dt = DTYPES[c["dtype"]]
    past, n = _requests(c)
    order = torch.randperm(len(n), generator=g, device="cuda").cpu().numpy()
    past, n = past[order], n[order]
    lens, page = past + n, c["page"]
    H, D = c["kv_heads"], c["dim"]
    pages_of = -(-lens // page)
    total = int(pages_of.sum())
    ids = torch.randperm(total, generator=g, device="cuda").cpu().numpy().astype(np.int32)
    table = np.zeros((len(n), int(pages_of.max())), np.int32)
    at = 0
    for r, m in enumerate(pages_of):
        table[r, :m] = ids[at:at + m]
        at += int(m)
    starts = np.concatenate([[0], np.cumsum(n)])
    return dict(case=c, query=_normal(g, (int(starts[-1]), c["q_heads"], D), dt), k_cache=_normal(g, (total, page, H, D), dt),
                v_cache=_normal(g, (total, page, H, D), dt), page_table=torch.from_numpy(table).cuda(),
                query_starts=_i32(starts), lens=_i32(lens), host=(starts.tolist(), lens.tolist()), longest=int(n.max()))


_INPUTS = {"tables": _tables_inputs, "append": _append_inputs, "adjust": _adjust_inputs, "chunk": _chunk_inputs}


def prepare(case, seed):
    return _INPUTS[case["op"]](case, seed)


# ------------------------------------------------------------------ one pass

def _tables_own(s):
    import min_sampling_gb300 as ms
    c = s["case"]
    out = ms.paged_step_tables(s["lens"], s["new_lens"], s["page_table"], s["free_pages"], s["free_count"], c["page"],
                               c["budget"])
    return (s["page_table"],) + tuple(out)


def _tables_plain(s):
    c, table = s["case"], s["page_table"]
    page, budget, width = c["page"], c["budget"], table.shape[1]
    lens, new = s["lens"].long(), s["new_lens"].long()
    free = s["free_count"].long().clamp(0, s["free_pages"].numel())
    ok = (new > 0) & (lens >= 0) & (lens + new <= width * page)
    have, want = (lens + page - 1) // page, (lens + new + page - 1) // page
    need, tok = torch.where(ok, want - have, 0), torch.where(ok, new, 0)
    pages = need.cumsum(0)
    ok = ok & ((need == 0) | (pages <= free)) & (tok.cumsum(0) <= budget)
    need, tok = torch.where(ok, need, 0), torch.where(ok, tok, 0)
    first = need.cumsum(0) - need
    j = torch.arange(width, device="cuda")
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    at = (free - 1 - first[:, None] - (j - have[:, None])).clamp(0, s["free_pages"].numel() - 1)
    table.copy_(torch.where(fresh, s["free_pages"][at], table))
    ends = tok.cumsum(0)
    starts = torch.cat((ends.new_zeros(1), ends))
    t = torch.arange(budget, device="cuda")
    row = torch.searchsorted(ends, t, right=True)
    real = row < len(lens)
    row = row.clamp(max=len(lens) - 1)
    pos = torch.where(real, lens[row] + t - starts[row], -1)
    return (table, starts.int(), torch.where(real, row, -1).int(), pos.int(), torch.where(ok, lens + new, lens.clamp(min=0)).int(),
            (free - need.sum()).int())


def _append_own(s):
    import min_sampling_gb300 as ms
    q = ms.append_paged_kv(s["key"], s["value"], s["k_cache"], s["v_cache"], s["page_table"], s["positions"],
                           s["rows"], inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"], query=s["query"],
                           query_norm=s["query_norm"], key_norm=s["key_norm"], norm_eps=EPS)
    return s["k_cache"], s["v_cache"], q


def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rotate(x, cos, sin, rotary, interleaved):
    r, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        out = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = r.chunk(2, dim=-1)
        out = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((out, rest), dim=-1)


def _append_plain(s):
    c = s["case"]
    # The angle of a far position needs more than 32 bits; its cosine and sine do not.
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    k = _rotate(_norm(s["key"], s["key_norm"]), cos, sin, c["rotary"], c["interleaved"])
    q = _rotate(_norm(s["query"], s["query_norm"]), cos, sin, c["rotary"], c["interleaved"])
    pos = s["positions"].long()
    page = s["page_table"][s["rows"].long(), pos // c["page"]].long()
    s["k_cache"][page, pos % c["page"]] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, pos % c["page"]] = s["value"]
    return s["k_cache"], s["v_cache"], q.to(s["query"].dtype)


def _adjust_own(s):
    import min_sampling_gb300 as ms
    return ms.adjust_logits(s["logits"], s["tokens"], s["lens"], s["prompt_lens"], repetition=s["repetition"],
                            presence=s["presence"], frequency=s["frequency"], bias_starts=s["bias_starts"],
                            bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], allowed=s["allowed"],
                            allowed_rows=s["allowed_rows"])


def _adjust_plain(s):
    z = s["logits"].float()
    B, V = z.shape
    if s["tokens"] is not None:
        at = torch.arange(s["tokens"].shape[1], device="cuda")
        there = at < s["lens"][:, None]
        made = there & (at >= s["prompt_lens"][:, None])
        tok = s["tokens"].long()
        seen = torch.zeros_like(z).scatter_add_(1, tok, there.float()) > 0
        count = torch.zeros_like(z).scatter_add_(1, tok, made.float())
        rep = s["repetition"][:, None]
        z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
        z = z - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias_starts"] is not None:
        n = s["bias_tokens"].numel()
        row = torch.searchsorted(s["bias_starts"][1:], torch.arange(n, device="cuda", dtype=torch.int32), right=True)
        b = torch.zeros_like(z)
        b[row, s["bias_tokens"].long()] = s["bias_values"]
        z = z + b
    if s["allowed"] is not None:
        r = s["allowed_rows"].long()
        bits = (s["allowed"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        bits = bits.flatten(1)[:, :V].bool()
        z = torch.where(bits[r.clamp(min=0)] | (r < 0)[:, None], z, float("-inf"))
    return z.to(s["logits"].dtype)


def _chunk_own(s):
    import min_sampling_gb300 as ms
    c = s["case"]
    return ms.paged_chunk_attention(s["query"], s["k_cache"], s["v_cache"], s["page_table"], s["query_starts"], s["lens"],
                                    window=c["window"] or None, sinks=c["sinks"], max_queries=s["longest"], return_lse=True)


def _chunk_plain(s):
    c = s["case"]
    page, H, D = c["page"], c["kv_heads"], c["dim"]
    gs = c["q_heads"] // H
    starts, lens = s["host"]
    out = torch.empty_like(s["query"])
    lse = torch.empty(s["query"].shape[:2], device="cuda")
    for r, n in enumerate(lens):
        pg = s["page_table"][r, : -(-n // page)].long()
        k = s["k_cache"][pg].reshape(-1, H, D)[:n].float().permute(1, 2, 0)
        v = s["v_cache"][pg].reshape(-1, H, D)[:n].float().permute(1, 0, 2)
        for a in range(starts[r], starts[r + 1], 1024):  # in slices, to keep the scores' memory small
            b = min(a + 1024, starts[r + 1])
            q = s["query"][a:b].float().reshape(b - a, H, gs, D).permute(1, 2, 0, 3).reshape(H, -1, D) / math.sqrt(D)
            sc = (q @ k).reshape(H, gs, b - a, n)
            pos = (n - starts[r + 1] + torch.arange(a, b, device="cuda"))[:, None]
            t = torch.arange(n, device="cuda")
            seen = t <= pos
            if c["window"]:
                seen &= (t > pos - c["window"]) | (t < c["sinks"])
            sc = sc.masked_fill(~seen, float("-inf"))
            m = sc.amax(-1, keepdim=True)
            e = torch.exp(sc - m)
            l = e.sum(-1, keepdim=True)
            o = (e.reshape(H, -1, n) @ v).reshape(H, gs, b - a, D) / l
            out[a:b] = o.permute(2, 0, 1, 3).reshape(b - a, -1, D).to(out.dtype)
            lse[a:b] = (m + torch.log(l)).squeeze(-1).permute(2, 0, 1).reshape(b - a, -1)
    return out, lse


_RUN = {("tables", False): _tables_plain, ("tables", True): _tables_own, ("append", False): _append_plain,
        ("append", True): _append_own, ("adjust", False): _adjust_plain, ("adjust", True): _adjust_own,
        ("chunk", False): _chunk_plain, ("chunk", True): _chunk_own}


def run(state):
    return _RUN[state["case"]["op"], bool(own)](state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "tables":
        past, n = _requests(c)
        new_pages = int((-(-(past + n) // c["page"]) - -(-past // c["page"])).sum())
        # Lengths in, totals and starts out; the new pages read and written; a row and a position for each token.
        return {"bytes": 16 * len(n) + 8 * new_pages + 8 * c["budget"], "flops": 8 * (len(n) + c["budget"])}
    e = SIZE[c["dtype"]]
    if c["op"] == "append":
        el = c["tokens"] * c["dim"] * (2 * c["kv_heads"] + c["q_heads"])
        rot = c["tokens"] * (c["kv_heads"] + c["q_heads"])
        return {"bytes": 2 * el * e + 12 * c["tokens"], "flops": rot * (4 * c["dim"] + 3 * c["rotary"])}
    if c["op"] == "adjust":
        B, V = c["rows"], c["vocab"]
        # Every logit read and written; histories, biases and masks read.
        hist = sum(c["history"] - (i * c["history"]) // (2 * B) for i in range(B))
        bias = sum(max(1, c["bias"] - (i * c["bias"]) // (2 * B)) for i in range(B)) if c["bias"] else 0
        return {"bytes": 2 * B * V * e + 4 * hist + 8 * bias + c["masks"] * V // 8, "flops": 2 * B * V + 4 * hist + bias}
    past, n = _requests(c)
    pairs = keys = 0
    for p, m in zip(past.tolist(), n.tolist()):
        pos = np.arange(p, p + m)
        if c["window"]:
            first = np.maximum(pos - c["window"] + 1, 0)
            pairs += int((pos + 1 - first + np.minimum(first, c["sinks"])).sum())
            lo = max(p - c["window"] + 1, 0)
            keys += p + m - lo + min(lo, c["sinks"])
        else:
            pairs += int((pos + 1).sum())
            keys += p + m
    return {"bytes": keys * c["kv_heads"] * c["dim"] * 2 * e + int(n.sum()) * c["q_heads"] * (2 * c["dim"] * e + 4),
            "flops": 4 * pairs * c["q_heads"] * c["dim"]}


# ------------------------------------------------------------------ exact values

def _tables_exact(c, seed):
    s = _tables_inputs(c, seed)
    table, stack = s["page_table"].cpu().numpy(), s["free_pages"].cpu().numpy()
    lens, new, left = s["lens"].tolist(), s["new_lens"].tolist(), int(s["free_count"])
    page, budget = c["page"], c["budget"]
    asked_pages = asked_tokens = 0
    top = left
    starts, rows, pos, after = [0], [], [], []
    for r, (p, n) in enumerate(zip(lens, new)):  # request by request, as an allocator on the host would
        slots = [t for t in range(p, p + n) if t % page == 0]
        asked_pages += len(slots)
        asked_tokens += n
        if asked_tokens <= budget and (not slots or asked_pages <= left):
            for t in slots:
                top -= 1
                table[r, t // page] = stack[top]
            rows += [r] * n
            pos += range(p, p + n)
            after.append(p + n)
        else:
            after.append(p)
        starts.append(len(rows))
    pad = [-1] * (budget - len(rows))
    return torch.from_numpy(table).cuda(), _i32(starts), _i32(rows + pad), _i32(pos + pad), _i32(after), _i32([top])


def _append_exact(c, seed):
    s = _append_inputs(c, seed)
    half = c["rotary"] // 2
    ang = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(ang), ang)

    def rot(x, w):
        x = x.double()
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["dim"] + EPS) * w.double()
        if c["interleaved"]:
            i, j = torch.arange(half, device="cuda") * 2, torch.arange(half, device="cuda") * 2 + 1
        else:
            i = torch.arange(half, device="cuda")
            j = i + half
        y = torch.complex(x[..., i], x[..., j]) * turn
        x[..., i], x[..., j] = y.real, y.imag
        return x

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    H, D, pos = c["kv_heads"], c["dim"], s["positions"].long()
    slot = s["page_table"][s["rows"].long(), pos // c["page"]].long() * c["page"] + pos % c["page"]
    kc.view(-1, H, D).index_copy_(0, slot, rot(s["key"], s["key_norm"]))
    vc.view(-1, H, D).index_copy_(0, slot, s["value"].double())
    return kc, vc, rot(s["query"], s["query_norm"])


def _adjust_exact(c, seed):
    s = _adjust_inputs(c, seed)
    B, V = c["rows"], c["vocab"]
    host = {k: v.cpu().numpy() for k, v in s.items() if isinstance(v, torch.Tensor) and k != "logits"}
    z = s["logits"].double()
    for b in range(B):  # row by row, token by token of its history
        x = z[b].cpu().numpy()
        if c["history"]:
            h = host["tokens"][b, : host["lens"][b]]
            ids, n = np.unique(h[host["prompt_lens"][b]:], return_counts=True)
            u = np.unique(h)
            r = float(host["repetition"][b])
            x[u] = np.where(x[u] > 0, x[u] / r, x[u] * r)
            x[ids] -= float(host["presence"][b]) + float(host["frequency"][b]) * n
        if c["bias"]:
            i, j = host["bias_starts"][b:b + 2]
            x[host["bias_tokens"][i:j]] += host["bias_values"][i:j].astype(np.float64)
        if c["masks"] and host["allowed_rows"][b] >= 0:
            bits = np.unpackbits(host["allowed"][host["allowed_rows"][b]].view(np.uint8), bitorder="little")[:V]
            x[bits == 0] = -np.inf
        z[b] = torch.from_numpy(x).cuda()
    return z


def _chunk_exact(c, seed):
    s = _chunk_inputs(c, seed)
    page, H, D = c["page"], c["kv_heads"], c["dim"]
    gs = c["q_heads"] // H
    starts, lens = s["host"]
    N = starts[-1]
    out = torch.empty((N, c["q_heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((N, c["q_heads"]), dtype=torch.float64, device="cuda")
    kf, vf = s["k_cache"].view(-1, H, D), s["v_cache"].view(-1, H, D)
    for r, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        slot = s["page_table"][r, t // page].long() * page + t % page
        m = starts[r + 1] - starts[r]
        # which keys each of the request's tokens sees, as distances between positions
        back = (n - m + torch.arange(m, device="cuda"))[:, None] - t[None, :]
        hidden = back < 0
        if c["window"]:
            hidden |= (back >= c["window"]) & (t >= c["sinks"])
        k, v = kf[slot].double(), vf[slot].double()
        for h in range(c["q_heads"]):
            sc = s["query"][starts[r]:starts[r + 1], h].double() @ k[:, h // gs].T * D ** -0.5
            sc[hidden] = -math.inf
            out[starts[r]:starts[r + 1], h] = torch.softmax(sc, -1) @ v[:, h // gs]
            lse[starts[r]:starts[r + 1], h] = torch.logsumexp(sc, -1)
    return out, lse


def exact(case, seed):
    return {"tables": _tables_exact, "append": _append_exact, "adjust": _adjust_exact, "chunk": _chunk_exact}[case["op"]](
        case, seed)
