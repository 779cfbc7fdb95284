"""fp64 numpy forms of the cache operators, written from their definitions one sequence and one
head at a time. Arrays are fp64 (values of 16-bit tensors) or int64; caches are
[num_pages, heads_kv, page_size, head_dim], tables [batch, max_pages].
"""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rotary_dim, theta=10000.0):
    return [theta ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]


def rotate(x, positions, inv_freq, axis_of_pair, pairing, inverse=False):
    """x [b, h, t, d], positions [axes, b, t]: pair i turns by positions[axis of i] * inv_freq[i]."""
    y = np.array(x, dtype=np.float64)
    pairs = len(inv_freq)
    for i, f in enumerate(inv_freq):
        angle = np.asarray(positions[axis_of_pair[i]], dtype=np.float64) * f
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        if inverse:
            s = -s
        a, b = (i, i + pairs) if pairing == "halves" else (2 * i, 2 * i + 1)
        p, q = np.array(x[..., a], dtype=np.float64), np.array(x[..., b], dtype=np.float64)
        y[..., a], y[..., b] = p * c - q * s, q * c + p * s
    return y


def entry(table, b, e, page_size):
    return int(table[b, e // page_size]), e % page_size


def entries(table, b, n, page_size, num_pages):
    """(e, page, place) of the entries 0 .. n-1 that lie on a page of the cache."""
    out = []
    for e in range(n):
        pg, off = entry(table, b, e, page_size)
        if 0 <= pg < num_pages:
            out.append((e, pg, off))
    return out


def decode(q, k, v, table, lens, scale):
    """q [b, hq, d]. Returns out [b, hq, d], lse [b, hq], share [pages, hkv, ps] (the softmax weights
    added per entry and KV head) and the largest scale * sum |q_i k_i| of every row."""
    b, hq, d = q.shape
    pages, hkv, ps, _ = k.shape
    g = hq // hkv
    cap = table.shape[1] * ps
    out, lse = np.zeros((b, hq, d)), np.full((b, hq), -math.inf)
    share, reach = np.zeros((pages, hkv, ps)), np.zeros((b, hq))
    for i in range(b):
        n = min(max(int(lens[i]), 0), cap)
        at = entries(table, i, n, ps, pages)
        if not at:
            continue
        pg, off = np.array([a[1] for a in at]), np.array([a[2] for a in at])
        for h in range(hkv):
            kk, vv, qq = k[pg, h, off], v[pg, h, off], q[i, h * g:(h + 1) * g]
            x = scale * (qq @ kk.T)
            reach[i, h * g:(h + 1) * g] = (scale * (np.abs(qq) @ np.abs(kk).T)).max(axis=1)
            top = x.max(axis=1, keepdims=True)
            p = np.exp(x - top)
            total = p.sum(axis=1, keepdims=True)
            lse[i, h * g:(h + 1) * g] = (top + np.log(total))[:, 0]
            p /= total
            out[i, h * g:(h + 1) * g] = p @ vv
            np.add.at(share, (pg, h, off), p.sum(axis=0))
    return out, lse, share, reach


def evict(arrays, weight, order, table, lens, seen, budget, sinks, recent):
    """arrays: caches [pages, hkv, ps, ...] compacted like weight and order, all in place. Returns the
    new lengths."""
    pages, hkv, ps = weight.shape
    cap = table.shape[1] * ps
    new = np.array(lens)
    used = {}
    for b in range(len(lens)):
        n = min(max(int(lens[b]), 0), cap)
        for s in range(-(-n // ps)):
            used.setdefault(int(table[b, s]), []).append(b)
    refused = set()
    for pg, who in used.items():
        if not 0 <= pg < pages or len(who) > 1:
            refused.update(who)
    for b in range(len(lens)):
        n = min(max(int(lens[b]), 0), cap)
        if n <= budget or b in refused:
            continue
        at = [entry(table, b, e, ps) for e in range(n)]
        for h in range(hkv):
            rank = []
            for e, (pg, off) in enumerate(at):
                o, w = int(order[pg, h, off]), float(weight[pg, h, off])
                safe = o < sinks or o >= int(seen[b]) - recent
                rank.append((0 if safe else 1, 0.0 if safe else -(w if w > 0 else 0.0), e))
            kept = {e for _, _, e in sorted(rank)[:budget]}
            holes = [e for e in range(budget) if e not in kept]
            movers = sorted(e for e in kept if e >= budget)
            assert len(holes) == len(movers)
            for to, frm in zip(holes, movers):
                for x in (*arrays, weight, order):
                    x[at[to][0], h, at[to][1]] = x[at[frm][0], h, at[frm][1]]
        new[b] = budget
    return new
