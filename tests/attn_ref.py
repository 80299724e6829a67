"""Plain 64-bit forms of the attention operators (numpy, loops), for the tests. They share
no code with the library; each follows the definition in the public header."""
from __future__ import annotations

import math

import numpy as np


def pages_of(tokens, page):
    return -(-tokens // page)


def kv_plan(kv_len, new_len, table, free, used, page, max_tokens):
    """(table, seq_len, q_start, positions, slots, summary) as integer arrays."""
    S, max_pages = table.shape
    table = table.copy()
    used = min(max(int(used), 0), len(free))
    q_start, seq_len = [0], []
    positions, slots = np.zeros(max_tokens, np.int64), np.full(max_tokens, -1, np.int64)
    given = wanted = asked = 0
    for s in range(S):
        kv, new = max(int(kv_len[s]), 0), max(int(new_len[s]), 0)
        asked += new
        new = min(new, max_tokens - q_start[-1])
        seq_len.append(kv + new)
        for i in range(pages_of(kv, page), pages_of(kv + new, page)):
            wanted += 1
            if i >= max_pages:
                continue
            ok = used + given < len(free)
            table[s, i] = free[used + given] if ok else -1
            given += ok
        for t in range(new):
            pos = kv + t
            positions[q_start[-1] + t] = pos
            if pos // page < max_pages and table[s, pos // page] >= 0:
                slot = int(table[s, pos // page]) * page + pos % page
                if slot < 2 ** 31:
                    slots[q_start[-1] + t] = slot
        q_start.append(q_start[-1] + new)
    summary = [min(x, 2 ** 31 - 1)
               for x in (q_start[-1], used + given, asked - q_start[-1], wanted - given)]
    return table, np.array(seq_len), np.array(q_start), positions, slots, np.array(summary)


def rotate(x, pos, inv_freq, magnitude, interleaved):
    """x [H, D] at one position; also the size |x0| + |x1| behind each element."""
    y, size = x.astype(np.float64).copy(), np.abs(x).astype(np.float64)
    half = len(inv_freq)
    for i in range(half):
        a = float(pos) * float(inv_freq[i])
        c, s = magnitude * math.cos(a), magnitude * math.sin(a)
        d0, d1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[:, d0] = x[:, d0] * c - x[:, d1] * s
        y[:, d1] = x[:, d1] * c + x[:, d0] * s
        size[:, d0] = size[:, d1] = magnitude * (np.abs(x[:, d0]) + np.abs(x[:, d1]))
    return y, size


def attention(q, keys, values, rows, scale, window):
    """One sequence. q [n, Hq, D]; keys and values [len, Hkv, D] with NaN-free places where
    they count; `rows`: bool [len], False where the key's page is missing. Returns out, lse,
    and the sums sum_j w_j |v_j| and max_j |scale| sum_d |q_d k_d| that bound the error."""
    n, Hq, D = q.shape
    length, Hkv = keys.shape[:2]
    G = Hq // Hkv
    out, size = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, reach = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        pos = length - n + i
        first = max(0, pos - window + 1) if window else 0
        seen = [j for j in range(first, pos + 1) if rows[j]]
        if not seen:
            continue
        for h in range(Hq):
            k, v = keys[seen, h // G], values[seen, h // G]
            z = scale * (k @ q[i, h])
            top = z.max()
            if top == -np.inf:
                continue
            w = np.exp(z - top)
            lse[i, h] = top + math.log(w.sum())
            w /= w.sum()
            out[i, h], size[i, h] = w @ v, w @ np.abs(v)
            reach[i, h] = abs(scale) * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, lse, size, reach
