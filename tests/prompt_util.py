"""Oracles in 64 bits (and whole numbers) of page planning, rotary positions and prompt
attention, written from their definitions."""
from __future__ import annotations

import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative to the value


def plan(free, count, table, held, keep, new, page, n_out):
    """One call on copies, request after request: what the call returns, and free, count,
    table and held after it."""
    free, table, held = list(free[:count]), table.copy(), held.copy()
    B, W = table.shape
    bad, need = np.zeros(B, dtype=bool), held.copy()
    cu = [0]
    for b in range(B):
        k, n, h = int(keep[b]), int(new[b]), int(held[b])
        cu.append(cu[-1] + max(0, n))
        bad[b] = k < 0 or n < 0 or h < 0 or h > W or k + n > W * page or k > h * page or cu[-1] > n_out
        if not bad[b]:
            need[b] = -(-(k + n) // page)
            for i in range(need[b], h):
                free.append(int(table[b, i]))
                table[b, i] = -1
    status, wanted, last = np.where(bad, 2, 0), 0, 0
    for b in range(B):
        if need[b] > held[b]:
            wanted += int(need[b] - held[b])
            if wanted > len(free):
                status[b] = 7
            else:
                last = wanted
    got = free[len(free) - last:]
    free = free[:len(free) - last]
    for b in range(B):
        if status[b] == 0:
            for i in range(held[b], need[b]):
                table[b, i] = got.pop(0)
            held[b] = need[b]
    slot, position = np.full(n_out, -1, np.int64), np.full(n_out, -1, np.int32)
    for b in range(B):
        for i in range(max(0, int(new[b]))):
            if cu[b] + i < n_out:
                at = int(keep[b]) + i
                position[cu[b] + i] = at
                if status[b] == 0:
                    slot[cu[b] + i] = int(table[b, at // page]) * page + at % page
    seq_len = np.where(status == 0, keep + new, keep)
    return dict(cu_new=np.minimum(cu, 2 ** 31 - 1), seq_len=seq_len, slot=slot, position=position, status=status,
                free=np.array(free, dtype=np.int64), table=table, held=held)


def rotary(x, position, freq, axis, adjacent, scale):
    """x [T, H, D] rotated, and what each element may be off by (before its last rounding).

    The angle: 2^-24 half turns when its 32-bit phase becomes a float, 2^-31 for the phase's
    lowest bits, 2^-33 turns for the frequency's at the farthest position; sine and cosine
    one unit in the last place, 2^-23: below (pi + 1 + 2) 2^-24 < 7 u in all.  Times the
    scale, two products and a sum: 3 u of (|x| + |y|) more."""
    P = len(freq)
    # angles in numpy's longest type: 11 bits more than float64 and often 60
    turns = position.astype(np.longdouble)[axis].T * (freq.astype(np.longdouble) / (2 * PI))
    turns = ((turns - np.rint(turns)) * 2 * PI).astype(np.float64)[:, None, :]
    c, s = scale * np.cos(turns), scale * np.sin(turns)
    i, j = (2 * np.arange(P), 2 * np.arange(P) + 1) if adjacent else (np.arange(P), np.arange(P) + P)
    out, tol = x.copy(), np.zeros(x.shape)
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    tol[..., i] = tol[..., j] = 10 * U32 * abs(scale) * (np.abs(a) + np.abs(b))
    return out, tol


PI = np.longdouble("3.14159265358979323846264338327950288419716939937510")


def attention(q, k, v, cu_q, cu_k, scale, window=0, sinks=0, bf16=False):
    """out, lse and what they may be off by.

    With u = 2^-24: a score is D products summed in fp32 in some order (truncated at worst,
    which counts twice) and scaled by up to three roundings, |dx| <= 2 (D + 8) u max_j
    sum_d |q k_j| scale; that much relative error in each weight and in their sum; the
    exponential and the sums of n tokens add (n + 32) u.  bf16 only: each weight is rounded
    to 8 bits before it meets its value (U16 of itself) and the result is (U16 of |out|);
    fp32: 4 u |out| for the division."""
    T, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    tol, tol_lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(cu_q) - 1):
        n, m = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        for t in range(n):
            P = m - n + t
            j = np.arange(max(0, P + 1))
            if window:
                j = j[(j > P - window) | (j < sinks)]
            if j.size == 0:
                continue
            row = int(cu_q[b]) + t
            for h in range(H):
                r = slice(h * G, (h + 1) * G)
                K, V, Q = k[cu_k[b] + j, h], v[cu_k[b] + j, h], q[row, r]
                x = Q @ K.T * scale
                top = x.max(1, keepdims=True)
                w = np.exp(x - top)
                l = w.sum(1, keepdims=True)
                o = w @ V / l
                out[row, r], lse[row, r] = o, (top + np.log(l))[:, 0]
                dx = 2 * (D + 8) * U32 * (np.abs(Q) @ np.abs(K).T * scale).max(1, keepdims=True)
                rel = 2 * dx + (j.size + 32) * U32 + (U16 if bf16 else 0.0)
                tol[row, r] = (w @ np.abs(V) / l) * rel + (U16 if bf16 else 4 * U32) * np.abs(o)
                tol_lse[row, r] = (dx + (j.size + 32) * U32 + 4 * U32 * np.abs(top + np.log(l)))[:, 0]
    return out, lse, tol, tol_lse
