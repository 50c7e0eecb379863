"""One step of a batch of requests of any kind, in float64: page tables from lengths, norms with the
rotation, attention of chunks over a paged cache, penalties, biases and masks on logits.

TEST INFRASTRUCTURE ONLY.  Plain definitions, request by request; attention in torch, so that long cases can run where
their tensors are.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.decode import rotate


def step_tables(lens, new_lens, page_table, free_pages, free_count, page_size, budget):
    """(table, starts, rows, positions, totals, free_left), lists and a copy of the table."""
    table = np.array(page_table)
    width, left = table.shape[1], min(max(int(free_count), 0), len(free_pages))
    top = left
    pages = tokens = 0
    starts, rows, pos, totals = [0], [], [], []
    for r, (p, n) in enumerate(zip(lens, new_lens)):
        p, n = int(p), int(n)
        asks = n > 0 and p >= 0 and p + n <= width * page_size
        need = -(-(p + n) // page_size) - -(-p // page_size) if asks else 0
        if asks:
            pages += need
            tokens += n
        if asks and (need == 0 or pages <= left) and tokens <= budget:
            for j in range(need):
                top -= 1
                table[r, -(-p // page_size) + j] = free_pages[top]
            rows += [r] * n
            pos += range(p, p + n)
            totals.append(p + n)
        else:
            totals.append(max(p, 0))
        starts.append(len(rows))
    pad = [-1] * (budget - len(rows))
    return table, starts, rows + pad, pos + pad, totals, top


def norm_rotate(x, weight, eps, pos, inv_freq, interleaved):
    """x / sqrt(mean(x^2) + eps) * weight over the last axis (None: no norm), rotated by pos * inv_freq."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return rotate(x, pos, inv_freq, interleaved)


def chunk_attention(query, k_cache, v_cache, page_table, query_starts, lens, window, sinks, scale):
    """float64 (out, lse, A, S, rel) of torch tensors: A = sum p |v|, S the largest score sum scale * sum |q k|
    and rel = sum_j exp(s_j - max) of each query.  A query that sees no key: zeros, lse -inf."""
    import torch
    N, Hq, D = query.shape
    H, page = k_cache.shape[2], k_cache.shape[1]
    gs = Hq // H
    new = lambda *s: torch.zeros(s, dtype=torch.float64, device=query.device)
    out, av, lse, big, rel = new(N, Hq, D), new(N, Hq, D), new(N, Hq) - math.inf, new(N, Hq), new(N, Hq) + 1
    for r in range(len(lens)):
        a, b, n = int(query_starts[r]), int(query_starts[r + 1]), int(lens[r])
        if b <= a or n <= 0:
            continue
        t = torch.arange(n, device=query.device)
        pg = torch.as_tensor(page_table[r][: -(-n // page)].astype(np.int64), device=query.device)[t // page]
        k, v = k_cache[pg, t % page].double(), v_cache[pg, t % page].double()
        pos = (n - (b - a) + torch.arange(b - a, device=query.device))[:, None]
        seen = t <= pos
        if window:
            seen &= (t > pos - window) | (t < sinks)
        some = seen.any(1)
        for h in range(Hq):
            q = query[a:b, h].double()
            s = (scale * (q @ k[:, h // gs].T)).masked_fill(~seen, -math.inf)
            m = s.amax(1, keepdim=True)
            m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
            e = torch.exp(s - m)
            l = e.sum(1, keepdim=True)
            d = torch.where(some[:, None], l, torch.ones_like(l))
            out[a:b, h] = e @ v[:, h // gs] / d
            av[a:b, h] = e @ v[:, h // gs].abs() / d
            lse[a:b, h] = torch.where(some, (m + torch.log(d)).squeeze(1), torch.full_like(m.squeeze(1), -math.inf))
            big[a:b, h] = (abs(scale) * (q.abs() @ k[:, h // gs].abs().T)).masked_fill(~seen, 0).amax(1)
            rel[a:b, h] = d.squeeze(1)
    return out, lse, av, big, rel


def adjust_row(z, tokens=(), prompt=0, repetition=1.0, presence=0.0, frequency=0.0, bias=(), allowed=None):
    """One row: (logits, and of each the largest magnitude on the way).  bias: (token, value) pairs in order; allowed: truth
    values, or None."""
    z = np.array(z, np.float64)
    V = z.size
    big = np.abs(z)
    tokens = [int(t) for t in tokens]
    seen = {t for t in tokens if 0 <= t < V}
    count = {}
    for t in tokens[max(prompt, 0):]:
        count[t] = count.get(t, 0) + 1
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        for t in seen:
            z[t] = z[t] / repetition if z[t] > 0 else z[t] * repetition
            big[t] = max(big[t], abs(z[t]))
            c = count.get(t, 0)
            if c:
                z[t] = z[t] - frequency * c - presence
                big[t] = max(big[t], abs(frequency * c), abs(presence), abs(z[t]))
        for t, v in dict(bias).items():
            if 0 <= t < V:
                z[t] += v
                big[t] = max(big[t], abs(v), abs(z[t]))
    if allowed is not None:
        z[~np.asarray(allowed, bool)] = -np.inf
    return z, big
