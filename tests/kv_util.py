"""Oracle of the 8-bit paged cache in 64-bit numpy, and seeded inputs for its tests."""
from __future__ import annotations

import math

import numpy as np
import torch

EXP_MIN, EXP_MAX = -100, 119
TILE = 128  # tokens whose probabilities share one reference in the tensor-core kernel


def code_table() -> np.ndarray:
    """What the 256 e4m3 codes stand for, from the format's definition."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = -x if c >> 7 else x
    return out


VALUE = code_table()
_FINITE = np.sort(VALUE[:127])  # the non-negative values 0 .. 448, by code


def encode(x: np.ndarray) -> np.ndarray:
    """e4m3 codes of x: the nearest value, the even code on ties, saturating; NaN and
    infinities give the NaN code 0x7F."""
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    hi = np.clip(np.searchsorted(_FINITE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _FINITE[lo], _FINITE[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(x), c | 128, c)
    return np.where(np.isfinite(x), c, 127).astype(np.uint8)


def wanted_scale(amax: float) -> float:
    if amax == 0:
        return 2.0 ** EXP_MIN
    e = EXP_MIN
    while e < EXP_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(codes, scale, x, table, cached, cu):
    """The cache after the append, as copies: codes [P, H, bs, D] uint8, scale [P, H]."""
    codes, scale = codes.copy(), scale.astype(np.float64).copy()
    bs = codes.shape[2]
    for b in range(len(cached)):
        new = x[cu[b]:cu[b + 1]]
        for i in range(cached[b] // bs, -(-(cached[b] + len(new)) // bs) if len(new) else 0):
            page, keep = int(table[b, i]), max(0, int(cached[b]) - i * bs)
            a = i * bs + keep - cached[b]
            part = new[a:a + bs - keep]  # [m, H, D]
            for h in range(codes.shape[1]):
                v = part[:, h]
                s = wanted_scale(np.abs(v[np.isfinite(v)]).max(initial=0.0))
                if keep:
                    s = max(s, scale[page, h])
                    if s > scale[page, h]:
                        codes[page, h, :keep] = encode(VALUE[codes[page, h, :keep]] * (scale[page, h] / s))
                codes[page, h, keep:keep + len(part)] = encode(v / s)
                scale[page, h] = s
    return codes, scale


def read(codes, scale, table_row, positions):
    """[len(positions), H, D] values."""
    bs = codes.shape[2]
    page = table_row[positions // bs]
    return VALUE[codes[page, :, positions % bs]] * scale[page][:, :, None].astype(np.float64)


def attention(q, kc, vc, ks, vs, table, seq_len, cu, scale, window=0, sinks=0, bf16=False):
    """out, lse and the error bound of out (per element) and lse, in 64 bits.

    Bound, with u = 2^-24 and everything relative to sum_j p_j |v_j| = A unless said:
     - a score is D products summed in fp32 in some order (truncated at worst), then
       scaled by at most three roundings: |dx| <= 2 (D + 8) u max_j sum |q k| scale;
       p's error is twice that (its own and the sum's), exp2 and the sums of n tokens
       in fp32 add (n + 32) u;
     - bf16 only.  The queries are split into two e4m3 terms below their row's largest
       magnitude Q: what is left is under 2^-16 Q an element, which changes a score by
       2^-16 Q sum_d |k_jd| scale at most.  The probabilities are split likewise: 2^-8
       of each, or 2^-17 of the tile's largest probability times the tile's largest
       value scale where that is more.  The result is rounded to 8 bits: 2^-9 |out|;
     - fp32: the result's own roundings, 4 u |out|."""
    u = 2.0 ** -24
    H, bs, D = kc.shape[1], kc.shape[2], kc.shape[3]
    T, Hq, _ = q.shape
    G = Hq // H
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    tol, tol_lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(seq_len)):
        n = int(cu[b + 1] - cu[b])
        for t in range(n):
            P = int(seq_len[b]) - n + t
            j = np.arange(max(P + 1, 0))
            if window:
                j = j[(j > P - window) | (j < sinks)]
            if j.size == 0:
                continue
            K, V = read(kc, ks, table[b], j), read(vc, vs, table[b], j)
            vsc = vs[table[b][j // bs]].astype(np.float64)
            for h in range(H):
                r = slice(h * G, (h + 1) * G)
                Q = q[cu[b] + t, r]
                x = Q @ K[:, h].T * scale
                m = np.max(np.where(np.isnan(x), -np.inf, x), axis=1, keepdims=True)
                p = np.exp(x - m)
                l = p.sum(1, keepdims=True)
                o = p @ V[:, h] / l
                row = cu[b] + t
                out[row, r], lse[row, r] = o, (m + np.log(l))[:, 0]
                A = p @ np.abs(V[:, h]) / l
                dx = 2 * (D + 8) * u * (np.abs(Q) @ np.abs(K[:, h]).T * scale).max(1, keepdims=True)
                rel = 2 * dx + (j.size + 32) * u
                tl = dx + (j.size + 32) * u + 4 * u * np.abs(m + np.log(l))
                if bf16:
                    dq = 2.0 ** -16 * np.abs(Q).max(1, keepdims=True) * np.abs(K[:, h]).sum(1).max() * scale
                    rel = rel + 2 * dq + 2.0 ** -8
                    tl = tl + dq
                    floor = np.zeros_like(o)
                    for tile in np.unique(j // TILE):
                        w = j // TILE == tile
                        floor += (p[:, w].max(1, keepdims=True) * vsc[w, h].max() * 2.0 ** -17 / l *
                                  (np.abs(V[w, h]) / vsc[w, h, None]).sum(0))
                    tol[row, r] = A * rel + floor + 2.0 ** -9 * np.abs(o)
                else:
                    tol[row, r] = A * rel + 4 * u * np.abs(o)
                tol_lse[row, r] = tl[:, 0]
    return out, lse, tol, tol_lse


# ------------------------------------------------------------------ inputs
class Inputs:
    """A filled cache and its requests, on the GPU and as numpy arrays."""

    def __init__(self, seed, lens, new, Hq, Hkv, D, page, dtype, extra_pages=3, token_major=False, fused=False,
                 dev="cuda"):
        g = np.random.default_rng(seed)
        self.lens, self.new = np.asarray(lens), np.asarray(new)
        B = len(self.lens)
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        pages = -(-self.lens // page)
        P = int(pages.sum()) + extra_pages
        width = max(1, int(pages.max(initial=0)))
        order = g.permutation(P).astype(np.int32)
        self.table = np.full((B, width), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        self.free = order[at:]
        # codes of normal values in a spread of scales, the keys with a few large channels
        self.kc = encode(g.normal(0, 60, (P, Hkv, page, D)) * np.exp(0.6 * g.normal(size=(1, Hkv, 1, D))))
        self.vc = encode(g.normal(0, 90, (P, Hkv, page, D)))
        self.ks = 2.0 ** g.integers(-8, -5, (P, Hkv)).astype(np.float64)
        self.vs = 2.0 ** g.integers(-9, -4, (P, Hkv)).astype(np.float64)
        T = int(self.cu[-1])
        wide = g.normal(0, 1, (T, Hq + 2 * Hkv, D)) * np.exp(0.5 * g.normal(size=(T, Hq + 2 * Hkv, 1)))
        self.wide = torch.from_numpy(wide).to(dtype).to(dev)
        q = self.wide[:, :Hq]
        self.q = q if fused else q.contiguous()
        self.k_new, self.v_new = self.wide[:, Hq:Hq + Hkv], self.wide[:, Hq + Hkv:]
        self.page, self.token_major, self.dev, self.dtype = page, token_major, dev, dtype

    def cache(self):
        import speculative_decoding_verification_15_gb300 as pkg

        def codes(c):
            t = torch.from_numpy(c).to(self.dev)
            if self.token_major:
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            return t.view(torch.float8_e4m3fn)

        return pkg.KVCache(codes(self.kc), codes(self.vc), self.tensor(self.ks.astype(np.float32)),
                           self.tensor(self.vs.astype(np.float32)))

    def tensor(self, a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(self.dev)

    def q64(self):
        return self.q.double().cpu().numpy()

    def i32(self, a):
        return self.tensor(np.asarray(a, dtype=np.int32))


def codes_of(t) -> np.ndarray:
    return t.contiguous().view(torch.uint8).cpu().numpy()
