"""The 8-bit paged cache in double precision: quantised writes, reads and
attention, straight from their definitions (numpy, no code shared with the
library or with the rest of the oracle).

Pools: codes [NB, P, Hkv, D] and scale bytes [NB, Hkv, P], both uint8; a row is
2^(byte - 127) * e4m3(codes).  Packed row r of sequence b (cu[b] <= r < cu[b+1])
is position seqlens[b] - (cu[b+1] - r)."""
from __future__ import annotations

import numpy as np


def _table() -> np.ndarray:
    """The values of the 256 e4m3 codes: 4 exponent bits (bias 7), 3 mantissa
    bits, no infinity, 0x7F and 0xFF NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if (c & 0x7F) == 0x7F else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if c & 0x80 else x
    return v


E4M3 = _table()


def bf16(bits) -> np.ndarray:
    """bf16 bit patterns (uint16) as float64."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def scales(b) -> np.ndarray:
    """e8m0 bytes as float64."""
    b = np.asarray(b, np.uint8).astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def quantise(bits):
    """Rows of bf16 bits [..., D] -> (codes [..., D], scale bytes [...])."""
    x = bf16(bits)
    fin = np.isfinite(x)
    top = np.where(fin, np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -117, np.int64)
    for t in range(-117, 119):                       # the smallest e with top <= 448 * 2^e
        e = np.where(top > 448 * 2.0 ** t, t + 1, e)
    y = np.where(fin, np.abs(x), 0.0) / np.ldexp(1.0, e)[..., None]
    grid = E4M3[:127]
    mid = (grid[1:] + grid[:-1]) / 2                 # exact in double
    lo = np.searchsorted(mid, y, side="left")        # ties stay below
    tie = (lo < 126) & (y == mid[np.minimum(lo, 125)])
    codes = lo + (tie & (lo % 2 == 1))               # ties go to the even code
    codes = np.where(fin, codes | np.where(np.signbit(x), 0x80, 0), 0x7F)
    return codes.astype(np.uint8), (e + 127).astype(np.uint8)


def places(seqlens, cu, T, table, NB, P):
    """(page, position in page) of every packed row; page -1: dropped, page -2:
    the row belongs to no sequence."""
    B, MP = table.shape
    out = np.full((T, 2), -2, np.int64)
    for b in range(B):
        n = min(max(int(seqlens[b]), 0), MP * P)
        for r in range(max(int(cu[b]), 0), min(int(cu[b + 1]), T)):
            pos = n - (int(cu[b + 1]) - r)
            page = int(table[b, pos // P]) if pos >= 0 else -1
            out[r] = (page, pos % P) if 0 <= page < NB else (-1, 0)
    return out


def append(k, v, table, seqlens, cu, kp, vp, ks, vs):
    """Writes in place: k, v bf16 bits [T, Hkv, D]."""
    at = places(seqlens, cu, k.shape[0], table, kp.shape[0], kp.shape[1])
    for x, codes, sc in ((k, kp, ks), (v, vp, vs)):
        c, s = quantise(x)
        for r, (page, pos) in enumerate(at):
            if page >= 0:
                codes[page, pos] = c[r]
                sc[page, :, pos] = s[r]


def read(kp, vp, ks, vs, table, seqlens, cu, T):
    """float64 k, v [T, Hkv, D]; rows of no sequence are NaN."""
    at = places(seqlens, cu, T, table, kp.shape[0], kp.shape[1])
    outs = []
    for codes, sc in ((kp, ks), (vp, vs)):
        out = np.full((T,) + codes.shape[2:], np.nan)
        for r, (page, pos) in enumerate(at):
            if page >= 0:
                out[r] = E4M3[codes[page, pos]] * scales(sc[page, :, pos])[:, None]
            elif page == -1:
                out[r] = 0.0
        outs.append(out)
    return outs


def _attend(q, k, v, sink, scale):
    """One query [D] over keys [n, D]: (o, lse, sum p|v| / den, largest |q||k| scale)."""
    if k.shape[0] == 0:
        return np.zeros(v.shape[1]), float(sink), np.zeros(v.shape[1]), 0.0
    s = scale * (k @ q)
    m = max(s.max(), sink)
    m = m if np.isfinite(m) else 0.0
    p = np.exp(s - m)
    den = p.sum() + np.exp(sink - m)
    return p @ v / den, m + np.log(den), p @ np.abs(v) / den, float(scale * (np.abs(k) @ np.abs(q)).max())


def decode(q, kp, vp, ks, vs, table, seqlens, sinks, window, scale):
    """q bf16 bits [B, Hq, D].  Returns (out, sum p|v| / den, largest score
    magnitude [B, Hq]), float64; the last two bound a rounded evaluation's error."""
    q = bf16(q)
    B, Hq, D = q.shape
    NB, P, Hkv, _ = kp.shape
    MP = table.shape[1]
    out, mag, top = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Hq))
    for b in range(B):
        n = min(max(int(seqlens[b]), 0), MP * P)
        if n == 0:
            continue
        for hk in range(Hkv):
            k, v = [], []
            for t in range(max(0, n - window), n):
                page = int(table[b, t // P])
                if 0 <= page < NB:
                    k.append(E4M3[kp[page, t % P, hk]] * scales(ks[page, hk, t % P]))
                    v.append(E4M3[vp[page, t % P, hk]] * scales(vs[page, hk, t % P]))
                else:
                    k.append(np.zeros(D))
                    v.append(np.zeros(D))
            k, v = np.array(k), np.array(v)
            for h in range(hk * (Hq // Hkv), (hk + 1) * (Hq // Hkv)):
                out[b, h], _, mag[b, h], top[b, h] = _attend(q[b, h], k, v, float(sinks[h]), scale)
    return out, mag, top


def extend(q, k, v, cu_q, cu_k, sinks, window, scale):
    """Packed chunks with earlier keys: query i of sequence b sits at position
    p = Lk - Lq + i and sees keys max(0, p - window + 1) .. p.  q, k, v bf16 bits.
    Returns (out [T, Hq, D], lse [Hq, T], sum p|v| / den, largest score)."""
    q, k, v = bf16(q), bf16(k), bf16(v)
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, top = np.full((Hq, T), np.nan), np.zeros((T, Hq))
    for b in range(len(cu_q) - 1):
        lq, lk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        for i in range(lq):
            p = lk - lq + i
            rows = slice(int(cu_k[b]) + max(0, p - window + 1), int(cu_k[b]) + max(p + 1, 0))
            r = int(cu_q[b]) + i
            for h in range(Hq):
                out[r, h], lse[h, r], mag[r, h], top[r, h] = _attend(
                    q[r, h], k[rows, h // G], v[rows, h // G], float(sinks[h]), scale)
    return out, lse, mag, top
