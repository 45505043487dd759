"""Plain 64-bit forms of the operators between a decode step's weight products.

Written from their definitions (include/q4k.h), row by row and head by head, in numpy;
they share no code with the library.  Arrays are host arrays; a cache is given as its
values: keys and values [n_pages][heads][page_size][D] and the page table.
"""
from __future__ import annotations

import math

import numpy as np


def slot_rows(pool, table_row, n, head):
    """Rows of slots 0 .. n - 1 of one head, [n][D] in 64 bits."""
    size = pool.shape[2]
    j = np.arange(n)
    return pool[table_row[j // size], head, j % size].astype(np.float64)


def attn_decode(k, v, table, lens, q, n_q, scale, softcap=0.0, window=0, k_scale=1.0, v_scale=1.0, weights=None,
                decay=1.0):
    """q [batch][n_q][n_heads][D].  Returns o (like q), the updated weights, and for every output element
    sum_j p_j |v_j| and max_j scale * sum_d |q_d k_jd| (what its rounding errors are measured by)."""
    B, _, H, D = q.shape
    G = H // k.shape[1]
    o, mag, big = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
    w = None if weights is None else weights.astype(np.float64).copy()
    for b in range(B):
        n = max(0, int(lens[b]))
        if w is not None:
            w[b, :, :n] *= decay
        for h in range(H):
            kk, vv = slot_rows(k, table[b], n, h // G) * k_scale, slot_rows(v, table[b], n, h // G) * v_scale
            for i in range(n_q):
                end = n - n_q + 1 + i
                begin = max(0, end - window) if window > 0 else 0
                if end <= begin:
                    continue
                x = q[b, i, h].astype(np.float64)
                s = kk[begin:end] @ x * scale
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                p = np.exp(s - s.max())
                p /= p.sum()
                o[b, i, h] = p @ vv[begin:end]
                mag[b, i, h] = p @ np.abs(vv[begin:end])
                big[b, i, h] = (np.abs(kk[begin:end]) @ np.abs(x)).max() * scale
                if w is not None:
                    w[b, h // G, begin:end] += p
    return o, w, mag, big


def rope(x, table, rope_dim, pairs):
    """x [T][heads][D] fp32 rotated by rows [T][rope_dim] of cosines and sines, every operation rounded to fp32."""
    half = rope_dim // 2
    if half == 0:
        return x.copy()
    y = x.copy()
    c, s = table[:, None, :half], table[:, None, half:]
    ia = np.arange(half) * 2 if pairs else np.arange(half)
    ib = ia + 1 if pairs else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def kv_evict(lens, weights, positions, budget, sinks, recent):
    """Returns new lengths, and for every sequence and head the slots taken over: take[b][h][i] is the old slot whose
    entry lies in slot i afterwards."""
    B, H, _ = weights.shape
    take = [[None] * H for _ in range(B)]
    new = np.minimum(np.maximum(lens, 0), budget)
    for b in range(B):
        n = max(0, int(lens[b]))
        for h in range(H):
            order = []
            newest = max([int(p) for p in positions[b, h, :n]], default=0)
            for j in range(n):
                p, w = int(positions[b, h, j]), float(weights[b, h, j])
                held = p < sinks or p > newest - recent
                order.append((held, math.isnan(w), 0.0 if math.isnan(w) else w, j))
            gone = {t[3] for t in sorted(order)[:n - int(new[b])]}
            m = int(new[b])
            fill = iter([j for j in range(m, n) if j not in gone])
            take[b][h] = [next(fill) if j in gone else j for j in range(m)]
    return new, take


def _norm(x, kind, w, b, eps):
    if kind == 0:
        return x
    if kind == 2:
        x = x - x.mean(1, keepdims=True)
    x = x / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    if w is not None:
        x = x * w
    return x if b is None else x + b


def norm_residual(y, post, post_w, post_b, post_eps, gate, scale, r, pre, pre_w, pre_b, pre_eps):
    """Returns h and pre(h)."""
    d = lambda a: None if a is None else np.asarray(a, np.float64)  # noqa: E731
    h = d(r)
    if y is not None:
        t = _norm(d(y), post, d(post_w), d(post_b), post_eps)
        h = h + scale * (t if gate is None else t * d(gate))
    return h, _norm(h, pre, d(pre_w), d(pre_b), pre_eps)


def sample_weight(d):
    """The whole-number weights of distances d (np.float32), every operation rounded to fp32."""
    f = np.float32
    d = np.asarray(d, f)
    near = d < f(41)
    x = np.where(near, d, f(0))
    n = np.floor(x)
    x = x - n - f(0.5)
    coef = [f(2 ** -0.5 * (-math.log(2)) ** i / math.factorial(i)) for i in range(8)]
    p = np.full_like(x, coef[7])
    for i in range(6, -1, -1):
        p = p * x + coef[i]
    w = ((p.astype(np.float64) * 2 ** 24).astype(np.int64) << 16) >> n.astype(np.int64)
    return np.where(near, w, 0)


def sample(logits, temperature, top_k, top_p, min_p, u):
    """One row; returns (token, prob)."""
    f = np.float32
    zf = np.where(np.isnan(logits), f(-math.inf), np.asarray(logits, f))
    z = zf.tolist()
    top = max(z)
    if top == -math.inf:
        return -1, 0.0
    greedy = not temperature > 0
    with np.errstate(all="ignore"):
        c = f(f(f(1) / f(1 if greedy else temperature)) * f(1.4426950408889634))
        w = sample_weight(np.where(zf == f(top), f(0), (f(top) - zf) * c)).tolist()
    rank = sorted(range(len(z)), key=lambda i: (-z[i], i))
    if greedy:
        top_k, top_p, min_p = 1, 1.0, 0.0
    if top_k > 0:
        rank = rank[:top_k]
    share = lambda x: math.floor(min(max(float(x), 0.0), 1.0) * 2 ** 24)  # noqa: E731
    p_share = 2 ** 24 if math.isnan(top_p) else share(top_p)
    m_share = 0 if math.isnan(min_p) else share(min_p)
    u_share = 0 if math.isnan(u) else min(share(u), 2 ** 24 - 1)
    if p_share < 2 ** 24:
        goal, run, keep = sum(w[i] for i in rank) * p_share >> 24, 0, []
        for i in rank:
            if keep and run >= goal:
                break
            keep.append(i)
            run += w[i]
        rank = keep
    least = w[rank[0]] * m_share >> 24
    kept = sorted(i for i in rank if w[i] >= least)
    total = sum(w[i] for i in kept)
    goal, run = total * u_share >> 24, 0
    for i in kept:
        run += w[i]
        if run > goal:
            return i, w[i] / total
    raise AssertionError("the target lies below the sum")
