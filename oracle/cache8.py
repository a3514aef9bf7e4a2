"""fp64 definitions of the rotated append and of the 8-bit cache (numpy, CPU).

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinity, NaN at
0x7f / 0xff, largest value 448.  A code of a block stands for code * scale; a
block is 16 tokens of one KV head of one page.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _e4m3_table() -> np.ndarray:
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = -v if c & 128 else v
    t[0x7F] = t[0xFF] = np.nan
    return t


E4M3 = _e4m3_table()


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even one; past the largest value it saturates; not finite: NaN."""
    x = np.asarray(x, np.float64)
    mags = E4M3[:0x7F]                      # ascending
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0.0), 448.0)
    hi = np.searchsorted(mags, a)           # first magnitude >= a
    lo = np.maximum(hi - 1, 0)
    up, down = mags[hi] - a, a - mags[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.isfinite(x), code, 0x7F)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def rotate(x, pos, inv_freq, interleaved=False, scale=1.0):
    """x [T][heads][D] turned by pos [T] * inv_freq [dim / 2]."""
    half = len(inv_freq)
    y = np.array(x, np.float64)
    if not half:
        return y
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    first = 2 * np.arange(half) if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    u, w = y[..., first].copy(), y[..., second].copy()
    y[..., first] = scale * (u * c - w * s)
    y[..., second] = scale * (w * c + u * s)
    return y


def block_scale(amax: np.ndarray) -> np.ndarray:
    """The least power of two s in [2^-120, 2^120] with amax / s <= 448."""
    amax = np.asarray(amax, np.float64)
    s = np.full(amax.shape, 2.0 ** -120)
    for e in range(-120, 120):
        s = np.where(amax > 448 * 2.0 ** e, 2.0 ** (e + 1), s)
    return s


def places(table, b, lo, hi, page_size):
    """Pool token rows of positions [lo, hi) of row b."""
    p = np.arange(lo, hi)
    return table[b, p // page_size].astype(np.int64) * page_size + p % page_size


def append_values(x, pages, table, lens, counts, page_size):
    """x [T][Hkv][D] written as is; returns pages as float64 [rows][Hkv][D]."""
    out = np.array(pages, np.float64).reshape(-1, *x.shape[1:])
    t = 0
    for b, n in enumerate(counts):
        out[places(table, b, lens[b], lens[b] + n, page_size)] = x[t:t + n]
        t += n
    return out


def append_q8(x, codes, scales, table, lens, counts, page_size):
    """x fp64 [T][Hkv][D] into codes uint8 [pages][page_size][Hkv][D] and scales [pages][.][Hkv].
    Returns (codes, scales, values before rounding [rows][Hkv][D] in units of the new scale, with NaN where
    the pool was not written)."""
    H, D = x.shape[1:]
    c = codes.reshape(-1, H, D).copy()
    s = scales.reshape(-1, H).astype(np.float64)
    want = np.full(c.shape, np.nan)
    t = 0
    for b, n in enumerate(counts):
        end = lens[b] + n
        for lo in range(lens[b] - lens[b] % BLOCK, end, BLOCK) if n else ():
            a, z = max(lo, lens[b]), min(lo + BLOCK, end)
            new = x[t + a - lens[b]:t + z - lens[b]]
            rows = places(table, b, a, z, page_size)
            blk = rows[0] // BLOCK
            amax = np.where(np.isfinite(new), np.abs(new), 0).max((0, 2))
            size = block_scale(amax)
            if a > lo:   # tokens of the row are there already
                size = np.maximum(size, s[blk])
                held = np.arange(blk * BLOCK, blk * BLOCK + a - lo)
                want[held] = E4M3[c[held]] * (s[blk] / size)[:, None]
                moved = (size != s[blk])[None, :, None]
                c[held] = np.where(moved, e4m3_encode(want[held]), c[held])
            s[blk] = size
            want[rows] = new / size[:, None]
            c[rows] = e4m3_encode(want[rows])
        t += n
    return c.reshape(codes.shape), s.reshape(scales.shape), want


def decode_q8(q, k_codes, v_codes, k_scales, v_scales, table, lens):
    """q fp64 [B][Hq][D]: (out [B][Hq][D], lse [B][Hq])."""
    B, Hq, D = q.shape
    pages, ps, H = k_codes.shape[:3]
    G = Hq // H
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    kf, vf = k_codes.reshape(-1, H, D), v_codes.reshape(-1, H, D)
    ks, vs = k_scales.reshape(-1, H).astype(np.float64), v_scales.reshape(-1, H).astype(np.float64)
    for b in range(B):
        if lens[b] == 0:
            continue
        rows = places(table, b, 0, lens[b], ps)
        for h in range(H):
            k = E4M3[kf[rows, h]] * ks[rows // BLOCK, h][:, None]
            v = E4M3[vf[rows, h]] * vs[rows // BLOCK, h][:, None]
            s = q[b, h * G:(h + 1) * G] @ k.T / np.sqrt(D)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            lse[b, h * G:(h + 1) * G] = m[:, 0] + np.log(p.sum(1))
            out[b, h * G:(h + 1) * G] = p @ v / p.sum(1, keepdims=True)
    return out, lse
