"""Microscaled KV cache in fp64 NumPy: the format, its tiles and attention.

Written from the definitions in ``include/loopvq.h``; shares no code with the
library.
"""
import numpy as np

BLOCK, TILE = 32, 32
FORMATS = {"e4m3": (448.0, -6, 3), "e2m1": (6.0, 0, 1)}   # largest value, least exponent, fraction bits


def mx_table(fmt):
    """Value of every code (NaN for e4m3's two NaN codes)."""
    _, lowest, digits = FORMATS[fmt]
    ebits = 4 if fmt == "e4m3" else 2
    n = 1 << (ebits + digits)
    half = np.empty(n)
    for c in range(n):
        e, f = c >> digits, c & ((1 << digits) - 1)
        half[c] = f * 2.0 ** (lowest - digits) if e == 0 else (1 + f / 2 ** digits) * 2.0 ** (e - 1 + lowest)
    if fmt == "e4m3":
        half[-1] = np.nan
    return np.concatenate([half, -half])


def mx_quantise(x, fmt):
    """x [..., D] -> (codes uint8 [..., D], scale bytes uint8 [..., D/32])."""
    top = FORMATS[fmt][0]
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    ok = np.isfinite(b).all(-1)
    b = np.where(ok[..., None], b, 0.0)
    peak = np.abs(b).max(-1)
    e = np.full(peak.shape, -64)
    for cand in range(-64, 56):          # one more while the block does not fit
        e = np.where(peak > top * 2.0 ** cand, cand + 1, e)
    y = np.clip(b / 2.0 ** e[..., None].astype(np.float64), -top, top)
    tab = mx_table(fmt)
    half = len(tab) // 2
    vals = tab[:half - 1] if fmt == "e4m3" else tab[:half]
    a = np.abs(y)
    hi = np.clip(np.searchsorted(vals, a), 1, len(vals) - 1)
    lo = hi - 1
    up = a - vals[lo] > vals[hi] - a
    tie = a - vals[lo] == vals[hi] - a
    code = np.where(up | (tie & (hi % 2 == 0)), hi, lo)
    code = code + np.where(np.signbit(y), half, 0)
    code = np.where(ok[..., None], code, 0).astype(np.uint8)
    return code.reshape(x.shape), np.where(ok, e + 127, 255).astype(np.uint8)


def mx_values(code, scale, fmt):
    """Codes and scale bytes -> fp64 values."""
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    v = mx_table(fmt)[code].reshape(*scale.shape, BLOCK)
    return (v * s[..., None]).reshape(code.shape)


def mx_tile_bytes(D, fmt):
    return TILE * D * (8 if fmt == "e4m3" else 4) // 8 + TILE * D // BLOCK


def mx_place(n, d, kind, D, fmt):
    """(byte, nibble or None) of the code of token n (0..31), channel d in a tile."""
    sub, b, n16, d32 = n // 16, d // 32, n % 16, d % 32
    if kind == "k":
        ab = n16 % 4 // 2
        g, c = 2 * (n16 // 4) + n16 % 2, d32 // 8
        i = ab * 8 + d32 % 8
    else:
        g, c = d32 // 4, n16 // 4
        i = (d32 % 4) * 4 + n16 % 4
    lane = 4 * g + c
    if fmt == "e4m3":
        return sub * (D // 32) * 512 + (b * 32 + lane) * 16 + i, None
    return sub * (D // 32) * 256 + ((b // 2) * 32 + lane) * 16 + (b % 2) * 8 + i // 2, i % 2


def mx_scale_place(n, b, D, fmt):
    codes = TILE * D * (8 if fmt == "e4m3" else 4) // 8
    return codes + ((n // 4) * (D // 32) + b) * 4 + n % 4


def mx_store(pool, t, h, pos, code, scale, kind, fmt):
    """Writes one token's codes [D] and scales [D/32] at pool position pos of a
    pool [T][H][tiles][tile bytes]."""
    D = code.shape[0]
    tile = pool[t, h, pos // TILE]
    for d in range(D):
        at, nib = mx_place(pos % TILE, d, kind, D, fmt)
        if nib is None:
            tile[at] = code[d]
        else:
            tile[at] = (tile[at] & (0x0F if nib else 0xF0)) | (int(code[d]) << (4 * nib))
    for b in range(D // BLOCK):
        tile[mx_scale_place(pos % TILE, b, D, fmt)] = scale[b]


def mx_attention(q, k, v, sees, pos_q, pos_k, scale, softcap=0.0, slope=None):
    """One query head: q [R][D], k and v [N][D], sees bool [R][N] -> o [R][D], lse [R],
    the weighted magnitudes sum p |v| [R][D], and the largest p |v| of each block
    of channels [R][D]."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        s = scale * (q @ k.T)
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
        if slope is not None:
            s = s - slope * (pos_q[:, None] - pos_k[None, :])
        s = np.where(sees, s, -np.inf)
        top = s.max(-1, keepdims=True) if s.shape[1] else np.full((len(q), 1), -np.inf)
        p = np.where(sees, np.exp(s - np.where(np.isinf(top), 0.0, top)), 0.0)
        l = p.sum(-1)
        R, D = q.shape
        o, a, top_v = np.zeros((R, D)), np.zeros((R, D)), np.zeros((R, D))
        peak = np.repeat(np.abs(v).reshape(len(v), -1, BLOCK).max(-1), BLOCK, axis=1)
        for i in range(R):
            w = p[i, sees[i]] / l[i] if sees[i].any() else p[i, sees[i]]
            o[i] = w @ v[sees[i]]
            a[i] = w @ np.abs(v[sees[i]])
            top_v[i] = (w[:, None] * peak[sees[i]]).max(0, initial=0.0)
        lse = np.where(sees.any(-1), top[:, 0] + np.log(l), -np.inf)
    return o, lse, a, top_v
