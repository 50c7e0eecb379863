"""The measured cases of the decode-loop operators: sampling from given random numbers,
appending to a paged key/value cache with the rotation applied, and attention for batches
that share a long prefix.

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


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One request of a 32000-token vocabulary: the latency of a single decode step.
        dict(name="sample_one_row", op="sample", rows=1, outs=1, vocab=32000, pad=0, dtype="bf16",
             order="top_k_first", k=50, p=0.9, min_p=0.0, temperature=0.8, sigma=3.0),
        # The benchmark's own batch (64 rows of 151936 logits, top-k 50 then top-p 0.9).
        dict(name="sample_top_k_first", op="sample", rows=64, outs=64, vocab=151936, pad=0, dtype="f32",
             order="top_k_first", k=50, p=0.9, min_p=0.0, temperature=1.0, sigma=3.0),
        # Nucleus sampling alone: every weight of the row counts.  Rows of an odd vocabulary in a padded buffer.
        dict(name="sample_top_p", op="sample", rows=64, outs=64, vocab=151665, pad=271, dtype="bf16",
             order="joint", k=0, p=0.95, min_p=0.0, temperature=0.9, sigma=3.0),
        # Four samples of each prompt's last row, min-p, the 128256-token vocabulary.
        dict(name="sample_min_p_parallel", op="sample", rows=128, outs=512, vocab=128256, pad=0, dtype="f16",
             order="joint", k=0, p=0.0, min_p=0.05, temperature=1.2, sigma=2.5),
        # A large batch with all three filters in the joint order.
        dict(name="sample_joint", op="sample", rows=256, outs=256, vocab=256000, pad=0, dtype="bf16",
             order="joint", k=200, p=0.97, min_p=0.002, temperature=1.0, sigma=3.0),
        # One decode step of 64 samples: 64 tokens appended, their queries rotated.
        dict(name="append_decode", op="append", seqs=64, tokens=64, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, dtype="bf16", page=16, context=32768),
        # A prefill of ragged prompts, 8190 tokens together.
        dict(name="append_prefill", op="append", seqs=5, tokens=8190, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, dtype="bf16", page=16, context=2048),
        # Half of each head rotated, neighbouring pairs, one head of keys to each of queries, odd counts.
        dict(name="append_partial_pairs", op="append", seqs=3, tokens=2049, q_heads=12, kv_heads=12, dim=64,
             rotary=32, interleaved=True, dtype="f16", page=5, context=1000),
        # Four samples of a short prompt: latency.
        dict(name="attend_four_samples", op="attend", groups=1, rows=4, queries=1, q_heads=32, kv_heads=8, dim=128,
             prefix=1000, suffix=37, dtype="bf16", page=16),
        # Sixteen samples of one long prompt: the prefix's bytes bound it.
        dict(name="attend_long_prefix", op="attend", groups=1, rows=16, queries=1, q_heads=32, kv_heads=8, dim=128,
             prefix=65537, suffix=300, dtype="bf16", page=16),
        # Three prompts with samples of their own, five positions a row as chain verification asks (four drafts).
        dict(name="attend_verify_groups", op="attend", groups=3, rows=48, queries=5, q_heads=16, kv_heads=8, dim=64,
             prefix=8190, suffix=700, dtype="f16", page=64),
        # A large batch over one prompt: matrix products bound it.
        dict(name="attend_large_batch", op="attend", groups=1, rows=256, queries=1, q_heads=32, kv_heads=8, dim=128,
             prefix=16384, suffix=512, dtype="bf16", page=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "append", "attend", "attend"])
    dt = rng.choice(["bf16", "f16"])
    if op == "sample":
        vocab = _log_int(rng, 1000, 256000)
        rows = min(_log_int(rng, 1, 256), max(1, 256 * 256000 // vocab // 4))
        return dict(op=op, rows=rows, outs=rows * rng.choice([1, 1, 2]), vocab=vocab, pad=rng.choice([0, 0, 1, 8, 77]),
                    dtype=rng.choice(["f32", "bf16", "f16"]), order=rng.choice(["joint", "top_k_first"]),
                    k=rng.choice([0, 1, _log_int(rng, 2, 500), _log_int(rng, 500, 100000)]),
                    p=rng.choice([0.0, round(rng.uniform(0.3, 0.999), 3)]),
                    min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)]),
                    temperature=round(rng.uniform(0.3, 2.0), 2), sigma=round(rng.uniform(0.5, 4.0), 2))
    if op == "append":
        dim = rng.choice([64, 128])
        kvh = rng.randint(1, 8)
        seqs = rng.randint(1, 64)
        return dict(op=op, seqs=seqs, tokens=max(seqs, _log_int(rng, 1, 8000)), q_heads=kvh * rng.randint(1, 4),
                    kv_heads=kvh, dim=dim, rotary=rng.choice([dim, dim // 2]), interleaved=rng.random() < 0.5,
                    dtype=dt, page=rng.choice([1, 5, 16, 64]), context=_log_int(rng, 1, 4000))
    kvh = rng.randint(1, 8)
    return dict(op=op, groups=rng.randint(1, 4), rows=_log_int(rng, 4, 128), queries=rng.choice([1, 1, 1, 3, 5]),
                q_heads=kvh * rng.choice([1, 2, 4, 5, 8]), kv_heads=kvh, dim=rng.choice([64, 128]),
                prefix=_log_int(rng, 1, 6000), suffix=_log_int(rng, 5, 900), dtype=dt,
                page=rng.choice([1, 5, 16, 64]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _sample_inputs(c, seed):
    g = _gen(seed)
    B, V = c["rows"], c["vocab"]
    buf = torch.empty((B, V + c["pad"]), dtype=DTYPES[c["dtype"]], device="cuda")
    for i in range(0, B, 64):  # in slices, to keep the fp32 temporaries small
        n = min(64, B - i)
        buf[i:i + n] = (torch.randn((n, V + c["pad"]), generator=g, device="cuda") * c["sigma"]).to(buf.dtype)
    n = c["outs"]
    s = dict(case=c, logits=buf[:, :V], uniforms=torch.rand(n, generator=g, device="cuda"))
    spread = torch.rand(n, generator=g, device="cuda")
    # Per-row parameters around the case's, as requests of one batch have them.
    s["temperature"] = (c["temperature"] * (0.9 + 0.2 * spread)).float()
    s["top_k"] = (torch.clamp((c["k"] * (0.5 + spread)).int(), min=1) if c["k"] else None)
    s["top_p"] = (c["p"] * (1.0 - 0.05 * spread)).float() if c["p"] else None
    s["min_p"] = (c["min_p"] * (0.5 + spread)).float() if c["min_p"] else None
    s["indices"] = None if n == B else torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(n // B)
    return s


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
    width = int(pages_of.max())
    # Only the pages that this call writes are backed by memory of their own; a sequence's earlier
    # pages all name the last page of the pool.
    first = start // page
    owned = (pages_of - first).astype(np.int64)
    total = int(((per + 2 * page - 2) // page).sum()) + 1  # as many as any start within a page can take
    order = torch.randperm(total - 1, generator=g, device="cuda").cpu().numpy()
    table = np.full((R, width), total - 1, np.int32)
    at = 0
    for r in range(R):
        table[r, first[r]:pages_of[r]] = order[at:at + owned[r]]
        at += owned[r]
    half = c["rotary"] // 2
    inv = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    H, D = c["kv_heads"], c["dim"]
    return dict(case=c, key=_normal(g, (N, H, D), dt), value=_normal(g, (N, H, D), dt),
                query=_normal(g, (N, c["q_heads"], D), dt),
                k_cache=_normal(g, (total, page, H, D), dt), v_cache=_normal(g, (total, page, H, D), dt),
                page_table=torch.from_numpy(table).cuda(), rows=torch.from_numpy(rows.astype(np.int32)).cuda(),
                positions=torch.from_numpy(pos.astype(np.int32)).cuda(), inv_freq=inv)


def _attend_inputs(c, seed):
    g = _gen(seed)
    dt = DTYPES[c["dtype"]]
    G, B, Q, page = c["groups"], c["rows"], c["queries"], c["page"]
    H, D = c["kv_heads"], c["dim"]
    # Groups of unequal sizes; prefixes up to the case's length; suffixes from Q tokens on.
    cuts = torch.randperm(B - 1, generator=g, device="cuda")[: G - 1].sort().values.cpu().numpy() + 1
    starts = np.concatenate([[0], cuts, [B]]).astype(np.int32)
    plens = np.array([c["prefix"] - (i * c["prefix"]) // (4 * G) for i in range(G)], np.int32)
    lo = min(Q, c["suffix"])
    slens = torch.randint(lo, c["suffix"] + 1, (B,), generator=g, device="cuda").cpu().numpy().astype(np.int32)
    slens[0] = c["suffix"]
    ppages, spages = -(-plens // page), -(-slens // page)
    total = int(ppages.sum() + spages.sum())
    order = torch.randperm(total, generator=g, device="cuda").cpu().numpy().astype(np.int32)
    ptab = np.zeros((G, int(ppages.max())), np.int32)
    stab = np.zeros((B, int(spages.max())), np.int32)
    at = 0
    for t, n in ((ptab, ppages), (stab, spages)):
        for i, m in enumerate(n):
            t[i, :m] = order[at:at + m]
            at += int(m)
    return dict(case=c, query=_normal(g, (B, Q, c["q_heads"], D), dt), k_cache=_normal(g, (total, page, H, D), dt),
                v_cache=_normal(g, (total, page, H, D), dt), prefix_table=torch.from_numpy(ptab).cuda(),
                prefix_lens=torch.from_numpy(plens).cuda(), suffix_table=torch.from_numpy(stab).cuda(),
                suffix_lens=torch.from_numpy(slens).cuda(), group_starts=torch.from_numpy(starts).cuda(),
                host=(starts.tolist(), plens.tolist()))


_INPUTS = {"sample": _sample_inputs, "append": _append_inputs, "attend": _attend_inputs}


def prepare(case, seed):
    return _INPUTS[case["op"]](case, seed)


# ------------------------------------------------------------------ one pass

def _sample_own(s):
    import min_sampling_gb300 as ms
    return ms.top_k_top_p_sampling_from_uniforms(s["logits"], s["uniforms"], s["temperature"], s["top_k"], s["top_p"],
                                                 s["min_p"], s["case"]["order"], s["indices"])


def _sample_plain(s):
    z = s["logits"].double()
    if s["indices"] is not None:
        z = z[s["indices"].long()]
    V = z.shape[1]
    # 64 bits: one rounding of a long sum in 32 moves the border between two tokens of a flat row.
    w = torch.exp((z - z.amax(1, keepdim=True)) / s["temperature"].double()[:, None])
    zs, at = torch.sort(z, dim=1, descending=True)
    keep = torch.ones_like(z, dtype=torch.bool)
    ws = w.gather(1, at)
    if s["top_k"] is not None:
        k = torch.clamp(s["top_k"].long(), max=V)
        tk = zs.gather(1, (k - 1)[:, None])
        keep &= z >= tk
        if s["case"]["order"] == "top_k_first":
            ws = ws * (zs >= tk)
    if s["top_p"] is not None:
        cum = ws.cumsum(1)
        need = s["top_p"].double()[:, None] * cum[:, -1:]
        r = torch.clamp((cum < need).sum(1, keepdim=True), max=V - 1)
        keep &= z >= zs.gather(1, r)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    cum = (w * keep).cumsum(1)
    hit = cum > s["uniforms"].double()[:, None] * cum[:, -1:]
    valid = hit.any(1)
    tok = torch.where(valid, hit.int().argmax(1), torch.full_like(valid, -1, dtype=torch.int64))
    return tok.int(), valid.to(torch.uint8)


def _append_own(s):
    import min_sampling_gb300 as ms
    q = ms.append_paged_kv(s["key"], s["value"], s["k_cache"], s["v_cache"], s["page_table"], s["positions"],
                           s["rows"], inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"], query=s["query"])
    return s["k_cache"], s["v_cache"], q


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
    k = _rotate(s["key"].float(), cos, sin, c["rotary"], c["interleaved"])
    q = _rotate(s["query"].float(), cos, sin, c["rotary"], c["interleaved"])
    pos = s["positions"].long()
    page = s["page_table"][s["rows"].long(), pos // c["page"]].long()
    s["k_cache"][page, pos % c["page"]] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, pos % c["page"]] = s["value"]
    return s["k_cache"], s["v_cache"], q.to(s["query"].dtype)


def _attend_own(s):
    import min_sampling_gb300 as ms
    return ms.shared_prefix_attention(s["query"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_lens"],
                                      s["suffix_table"], s["suffix_lens"], s["group_starts"], return_lse=True)


def _attend_plain(s):
    c = s["case"]
    G, B, Q, page, H, D = c["groups"], c["rows"], c["queries"], c["page"], c["kv_heads"], c["dim"]
    gs = c["q_heads"] // H
    q = s["query"].float().reshape(B, Q, H, gs, D) / math.sqrt(D)
    starts, plens = s["host"]
    m1, l1, o1 = [], [], []
    for g in range(G):  # the prefix once for each group's rows
        pg = s["prefix_table"][g, : -(-plens[g] // page)].long()
        k = s["k_cache"][pg].reshape(-1, H, D)[: plens[g]].float()
        v = s["v_cache"][pg].reshape(-1, H, D)[: plens[g]].float()
        qq = q[starts[g]:starts[g + 1]].permute(2, 0, 1, 3, 4).reshape(H, -1, D)
        sc = qq @ k.permute(1, 2, 0)
        m = sc.amax(-1, keepdim=True)
        e = torch.exp(sc - m)
        n = starts[g + 1] - starts[g]
        back = lambda x: x.reshape(H, n, Q, gs, -1).permute(1, 2, 0, 3, 4)
        m1.append(back(m)), l1.append(back(e.sum(-1, keepdim=True))), o1.append(back(e @ v.permute(1, 0, 2)))
    m1, l1, o1 = torch.cat(m1), torch.cat(l1), torch.cat(o1)
    st = s["suffix_table"].long()
    S = st.shape[1] * page
    k = s["k_cache"][st].reshape(B, S, H, D).float().permute(0, 2, 3, 1)
    v = s["v_cache"][st].reshape(B, S, H, D).float().permute(0, 2, 1, 3)
    qq = q.permute(0, 2, 1, 3, 4).reshape(B, H, Q * gs, D)
    seen = s["suffix_lens"].long()[:, None] - (Q - 1 - torch.arange(Q, device="cuda"))
    mask = torch.arange(S, device="cuda") < seen[..., None]
    mask = mask[:, None, :, None, :].expand(B, H, Q, gs, S).reshape(B, H, Q * gs, S)
    sc = (qq @ k).masked_fill(~mask, float("-inf"))
    back = lambda x: x.reshape(B, H, Q, gs, -1).permute(0, 2, 1, 3, 4)
    m2 = back(sc.amax(-1, keepdim=True))
    mx = torch.maximum(m1, m2)
    e = torch.exp(sc - mx.permute(0, 2, 1, 3, 4).reshape(B, H, Q * gs, 1))
    f = torch.exp(m1 - mx)
    l = l1 * f + back(e.sum(-1, keepdim=True))
    o = (o1 * f + back(e @ v)) / l
    lse = (mx + torch.log(l)).reshape(B, Q, c["q_heads"])
    return o.reshape(B, Q, c["q_heads"], D).to(s["query"].dtype), lse


_RUN = {("sample", False): _sample_plain, ("sample", True): _sample_own, ("append", False): _append_plain,
        ("append", True): _append_own, ("attend", False): _attend_plain, ("attend", True): _attend_own}


def run(state):
    return _RUN[state["case"]["op"], bool(own)](state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "sample":
        # Every logit once; a few operations each (compare, weight, sum).
        return {"bytes": c["rows"] * c["vocab"] * SIZE[c["dtype"]] + c["outs"] * 25, "flops": 4 * c["rows"] * c["vocab"]}
    e = SIZE[c["dtype"]]
    if c["op"] == "append":
        el = c["tokens"] * c["dim"] * (2 * c["kv_heads"] + c["q_heads"])
        return {"bytes": 2 * el * e + 12 * c["tokens"], "flops": 3 * c["tokens"] * c["rotary"] * (c["kv_heads"] + c["q_heads"])}
    # The inputs' lengths: group i's prefix is shorter by i/(4 groups); suffixes are spread evenly up to the longest.
    G, B, Q = c["groups"], c["rows"], c["queries"]
    plens = [c["prefix"] - (i * c["prefix"]) // (4 * G) for i in range(G)]
    slen = (min(Q, c["suffix"]) + c["suffix"]) / 2
    kv = (sum(plens) + B * slen) * c["kv_heads"] * c["dim"] * 2 * e
    qo = B * Q * c["q_heads"] * (2 * c["dim"] * e + 4)
    pairs = B * Q * (sum(plens) / G + slen)
    return {"bytes": int(kv + qo), "flops": int(4 * pairs * c["q_heads"] * c["dim"])}


# ------------------------------------------------------------------ exact values

def _sample_exact(c, seed):
    s = _sample_inputs(c, seed)
    lg = s["logits"].float().cpu().numpy()
    idx = np.arange(c["outs"]) if s["indices"] is None else s["indices"].cpu().numpy()
    par = {k: None if s[k] is None else s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "uniforms")}
    tok = np.full(c["outs"], -1, np.int32)
    ok = np.zeros(c["outs"], np.uint8)
    srt = {}
    for b in range(c["outs"]):
        r = int(idx[b])
        if r not in srt:  # distinct values, descending, with how often each occurs
            v, n = np.unique(lg[r], return_counts=True)
            srt = {r: (v[::-1].astype(np.float64), n[::-1])}
        v, n = srt[r]
        T = float(par["temperature"][b])
        wv = np.exp((v - v[0]) / T)
        cut = -np.inf
        mass = wv * n
        if par["top_k"] is not None:
            j = int(np.searchsorted(np.cumsum(n), min(int(par["top_k"][b]), c["vocab"])))
            cut = max(cut, v[j])
            if c["order"] == "top_k_first":
                mass = mass[: j + 1]
        if par["top_p"] is not None:
            cm = np.cumsum(mass)
            j = min(int(np.searchsorted(cm, float(par["top_p"][b]) * cm[-1])), len(cm) - 1)
            cut = max(cut, v[j])
        if par["min_p"] is not None:
            cut = max(cut, v[np.nonzero(wv >= float(par["min_p"][b]))[0][-1]])
        z = lg[r].astype(np.float64)
        at = np.nonzero(z >= cut)[0]
        cm = np.cumsum(np.exp((z[at] - v[0]) / T))
        j = int(np.searchsorted(cm, float(par["uniforms"][b]) * cm[-1], side="right"))
        tok[b], ok[b] = at[min(j, len(at) - 1)], 1
    return torch.from_numpy(tok).cuda(), torch.from_numpy(ok).cuda()


def _append_exact(c, seed):
    s = _append_inputs(c, seed)
    half = c["rotary"] // 2
    ang = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(ang), ang)

    def rot(x):
        x = x.double().clone()
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
    kc.view(-1, H, D).index_copy_(0, slot, rot(s["key"]))
    vc.view(-1, H, D).index_copy_(0, slot, s["value"].double())
    return kc, vc, rot(s["query"])


def _attend_exact(c, seed):
    s = _attend_inputs(c, seed)
    B, Q, page, H, D = c["rows"], c["queries"], c["page"], c["kv_heads"], c["dim"]
    gs = c["q_heads"] // H
    starts, plens = s["host"]
    out = torch.empty((B, Q, c["q_heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, Q, c["q_heads"]), dtype=torch.float64, device="cuda")
    kf, vf = s["k_cache"].view(-1, H, D), s["v_cache"].view(-1, H, D)

    def slots(table, n):
        t = torch.arange(n, device="cuda")
        return table[t // page].long() * page + t % page

    slens = s["suffix_lens"].tolist()
    for g, n in enumerate(plens):
        sp = slots(s["prefix_table"][g], n)
        kp, vp = kf[sp].double(), vf[sp].double()
        for b in range(starts[g], starts[g + 1]):  # row by row, prefix and suffix as one list of keys
            ss = slots(s["suffix_table"][b], slens[b])
            k, v = torch.cat((kp, kf[ss].double())), torch.cat((vp, vf[ss].double()))
            for i in range(Q):
                m = n + slens[b] - (Q - 1 - i)
                qi = s["query"][b, i].double().view(H, gs, D)
                sc = torch.einsum("hgd,khd->hgk", qi, k[:m]) * D ** -0.5
                p = torch.softmax(sc, -1)
                out[b, i] = torch.einsum("hgk,khd->hgd", p, v[:m]).reshape(-1, D)
                lse[b, i] = torch.logsumexp(sc, -1).reshape(-1)
    return out, lse


def exact(case, seed):
    return {"sample": _sample_exact, "append": _append_exact, "attend": _attend_exact}[case["op"]](case, seed)
