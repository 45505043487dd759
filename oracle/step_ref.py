"""Plain forms of the operators of a step that mixes prompts and decode tokens (include/q4k.h), in numpy: whole numbers for
the plan, 64 bits for the rest, a request, adapter or row at a time.  They share no code with the library."""
from __future__ import annotations

import numpy as np

from oracle import decode_ref


def batch_plan(table, max_pages, page_size, n_pages, seq_lens, n_new, first_pos, held, free_pages, count, T):
    """Returns a dict of the outputs: table, held, free_pages, count, after, starts, seq, slot, pos (the last three as long as
    there are tokens)."""
    table, free = np.array(table), np.array(free_pages)
    B, capacity = len(seq_lens), max_pages * page_size
    lens = [min(max(int(n), 0), capacity) for n in seq_lens]
    held = [min(max(int(n), 0), max_pages) for n in held]
    stack = [int(p) for p in free[:min(max(int(count), 0), n_pages)]]
    asked, tokens, want = 0, [], []
    for b in range(B):
        n = max(int(n_new[b]), 0)
        if lens[b] + n > capacity:
            n = 0
        asked += n
        tokens.append(n if asked <= T else 0)
        want.append(0 if n_new[b] < 0 else -(-(lens[b] + tokens[b]) // page_size))
    for b in range(B):
        for j in range(want[b], held[b]):
            if len(stack) < n_pages:
                free[len(stack)] = table[b, j]
                stack.append(int(table[b, j]))
    have, lacking = len(stack), 0
    for b in range(B):
        if want[b] <= held[b]:
            continue
        lacking += want[b] - held[b]
        if lacking > have:
            tokens[b], want[b] = 0, held[b]
        for j in range(held[b], want[b]):
            table[b, j] = stack.pop()
    starts = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int64)
    seq = np.repeat(np.arange(B), tokens)
    i = np.arange(len(seq)) - starts[seq]
    slot = np.array(lens)[seq] + i
    pos = slot if first_pos is None else np.array(first_pos)[seq] + i
    after = [0 if n_new[b] < 0 else lens[b] + tokens[b] for b in range(B)]
    return dict(table=table, held=want, free_pages=free, count=len(stack), after=after, starts=starts, seq=seq, slot=slot, pos=pos)


def in_eight(v):
    """(q, s) of fp32 values [M][D], every operation rounded to fp32."""
    x = np.asarray(v, np.float32).reshape(v.shape[0], -1, 32)
    a = np.abs(x).max(2)
    s = (a / np.float32(127)).astype(np.float32)
    with np.errstate(all="ignore"):
        q = np.minimum(np.rint(np.abs(x) / s[..., None]), 127)
    q = np.where(np.isinf(x), 127, q)
    q = np.where(s[..., None] > 0, np.copysign(q, x), 0)
    return q.reshape(v.shape).astype(np.int8), s


def lora_add(a, b, ranks, scales, ids, x, y):
    """Returns y with the adapters' parts added, and for each element the sum of its products' magnitudes."""
    out, mag = y.astype(np.float64).copy(), np.abs(y).astype(np.float64)
    for t, i in enumerate(ids):
        if not 0 <= i < len(a):
            continue
        r = min(max(int(ranks[i]), 0), a.shape[1])
        inner = a[i, :r].astype(np.float64) @ x[t].astype(np.float64)
        big = np.abs(a[i, :r]).astype(np.float64) @ np.abs(x[t]).astype(np.float64)
        out[t] += float(scales[i]) * (b[i, :, :r].astype(np.float64) @ inner)
        mag[t] += abs(float(scales[i])) * (np.abs(b[i, :, :r]).astype(np.float64) @ big)
    return out, mag


def attn_chunk(k, v, table, starts, lens, q, scale, softcap=0.0, window=0, k_scale=1.0, v_scale=1.0):
    """q [T][heads][D].  Returns o (0 where no sequence has the row), and the two magnitudes of decode_ref.attn_decode."""
    o, mag, big = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    for b in range(len(lens)):
        lo, hi = int(starts[b]), int(starts[b + 1])
        if hi > lo:
            r = decode_ref.attn_decode(k, v, table[b:b + 1], [int(lens[b])], q[None, lo:hi], hi - lo, scale, softcap, window,
                                       k_scale, v_scale)
            o[lo:hi], mag[lo:hi], big[lo:hi] = r[0][0], r[2][0], r[3][0]
    return o, mag, big
