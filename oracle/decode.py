"""The decode step in float64: sampling from given uniforms, appending to a paged cache
with the rotation, attention over a shared prefix and a row's own suffix.

TEST INFRASTRUCTURE ONLY.  Plain definitions, row by row.
"""
from __future__ import annotations

import math

import numpy as np


def token_from_uniform(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, order="joint"):
    """One row: (token, margin), token -1 for an invalid row.  `margin` is the smallest distance, relative
    to the mass it is measured against, of a decisive running mass from its border."""
    z = np.asarray(z, np.float64)
    bad = np.isnan(z).any() or (z == np.inf).any() or not (z > -np.inf).any()
    bad |= not (0.0 <= u < 1.0) or not (temperature >= 2.0 ** -126) or math.isnan(top_p) or not (min_p <= 1.0)
    if bad:
        return -1, math.inf
    m = z.max()
    with np.errstate(over="ignore", under="ignore"):
        w = np.where(z == -np.inf, 0.0, np.exp(np.where(z == -np.inf, 0.0, (z - m)) / np.float64(temperature)))
    V = z.size
    margin = math.inf
    keep = np.ones(V, bool)
    base = np.ones(V, bool)
    if 0 < top_k < V:
        t = np.partition(z, V - top_k)[V - top_k]
        keep &= z >= t
        if order == "top_k_first":
            base = z >= t
    if top_p < 1.0:
        # mass at or above each distinct value, largest first
        vals, inv = np.unique(z[base], return_inverse=True)
        mass = np.bincount(inv, weights=w[base])[::-1].cumsum()
        need = max(top_p, 0.0) * mass[-1]
        j = min(int(np.searchsorted(mass, need)), mass.size - 1)
        margin = min(margin, float(np.abs(mass - need).min() / mass[-1])) if top_p > 0 else margin
        keep &= z >= vals[::-1][j]
    if min_p > 0.0:
        margin = min(margin, float(np.abs(w - min_p)[z < m].min())) if (z < m).any() else margin
        keep &= w >= min_p
    cum = np.cumsum(np.where(keep, w, 0.0))
    need = u * cum[-1]
    hit = np.nonzero(cum > need)[0]
    if cum[-1] <= 0 or hit.size == 0:
        return -1, margin
    if u > 0:
        margin = min(margin, float(np.abs(cum - need).min() / cum[-1]))
    return int(hit[0]), margin


def rotate(x, pos, inv_freq, interleaved):
    """Rotate the first 2 len(inv_freq) elements of the last axis of x by pos * inv_freq."""
    x = np.array(x, np.float64)
    half = len(inv_freq)
    # the angle in turns: exact products, reduced before they lose digits
    ang = np.array([math.fmod(int(pos) * float(f), 2.0 * math.pi) if abs(int(pos) * float(f)) < 2 ** 20
                    else _angle(int(pos), float(f)) for f in inv_freq])
    c, s = np.cos(ang), np.sin(ang)
    i = np.arange(half) * 2 if interleaved else np.arange(half)
    j = i + 1 if interleaved else i + half
    a, b = x[..., i].copy(), x[..., j].copy()
    x[..., i], x[..., j] = a * c - b * s, b * c + a * s
    return x


def _angle(pos: int, f: float) -> float:
    """pos * f modulo 2 pi with rational arithmetic (pi to 60 digits)."""
    from fractions import Fraction
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    a = Fraction(f) * pos
    return float(a - two_pi * (a // two_pi))


def append(key, value, k_cache, v_cache, page_table, positions, rows, rotary_positions, inv_freq, interleaved, query):
    """float64 copies of the caches after the call, the rotated queries, and the slots written."""
    kc, vc = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    q = None if query is None else np.array(query, np.float64)
    wrote = set()
    pages, page = kc.shape[:2]
    for t, pos in enumerate(positions):
        if pos < 0:
            continue
        rp = int(pos if rotary_positions is None else rotary_positions[t])
        if q is not None:
            q[t] = rotate(q[t], rp, inv_freq, interleaved)
        r, i = int(rows[t]) if rows is not None else t, int(pos) // page
        if not (0 <= r < page_table.shape[0] and i < page_table.shape[1]):
            continue
        pg = int(page_table[r, i])
        if not 0 <= pg < pages:
            continue
        kc[pg, pos % page] = rotate(key[t], rp, inv_freq, interleaved)
        vc[pg, pos % page] = value[t]
        wrote.add((pg, int(pos % page)))
    return kc, vc, q, wrote


def attend(query, k_cache, v_cache, prefix_table, prefix_lens, suffix_table, suffix_lens, group_starts, scale):
    """out, lse and, for tolerances, per element sum_j p_j |v_j|, and per query the largest score sum
    scale * sum |q k| and sum_j exp(s_j - max)."""
    query = np.asarray(query, np.float64)
    B, Q, Hq, D = query.shape
    page, H = k_cache.shape[1], k_cache.shape[2]
    gs = Hq // H
    out, av = np.zeros((B, Q, Hq, D)), np.zeros((B, Q, Hq, D))
    lse, big, rel = np.full((B, Q, Hq), -np.inf), np.zeros((B, Q, Hq)), np.ones((B, Q, Hq))

    def gather(table, n):
        t = np.arange(n)
        pg = np.asarray(table)[t // page]
        return k_cache[pg, t % page].astype(np.float64), v_cache[pg, t % page].astype(np.float64)

    for b in range(B):
        ks, vs = gather(suffix_table[b], int(suffix_lens[b]))
        kp, vp = ks[:0], vs[:0]
        for g in range(len(prefix_lens)):
            if group_starts is None or group_starts[g] <= b < group_starts[g + 1]:
                kp, vp = gather(prefix_table[g], int(prefix_lens[g]))
        for j in range(Q):
            n = max(0, int(suffix_lens[b]) - (Q - 1 - j))
            k, v = np.concatenate([kp, ks[:n]]), np.concatenate([vp, vs[:n]])
            if not len(k):
                continue
            for h in range(Hq):
                s = scale * (k[:, h // gs] @ query[b, j, h])
                m = s.max()
                e = np.exp(s - m)
                out[b, j, h] = (e @ v[:, h // gs]) / e.sum()
                av[b, j, h] = (e @ np.abs(v[:, h // gs])) / e.sum()
                lse[b, j, h] = m + math.log(e.sum())
                big[b, j, h] = abs(scale) * (np.abs(k[:, h // gs]) @ np.abs(query[b, j, h])).max()
                rel[b, j, h] = e.sum()
    return out, lse, av, big, rel
