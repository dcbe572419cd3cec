"""Oracle of the rotary positions, the 8-bit key-value cache and the attention
over it.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain NumPy in float64:
one token, one pair or one request and head at a time.
"""

import numpy as np

from .attn_oracle import attend, paged_rows


def rope(x, positions, freqs, interleaved, gain):
    """x [T, heads, D] with the first 2 * len(freqs) dimensions turned."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(freqs)
    for t, p in enumerate(positions):
        for i, f in enumerate(freqs):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = np.cos(float(p) * float(f)), np.sin(float(p) * float(f))
            y[t, :, a] = gain * (x[t, :, a] * c - x[t, :, b] * s)
            y[t, :, b] = gain * (x[t, :, a] * s + x[t, :, b] * c)
    return y


def quantize_rows(x):
    """(codes, scales) of rows x [..., D]: s = amax / 127 as float32 (the next
    one below where 127 s would not be a float32), codes the nearest whole
    number to the exact x / s, ties to even; scale NaN, codes 0 for rows that
    are not finite."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x).all(axis=-1)
    x = np.where(finite[..., None], x, 0.0)
    scale = (np.abs(x).max(axis=-1) / 127.0).astype(np.float32)
    most = float(np.finfo(np.float32).max)
    scale = np.where(scale.astype(np.float64) * 127.0 > most, np.nextafter(scale, np.float32(0)), scale)
    step = np.where(scale > 0, scale, np.float32(1)).astype(np.float64)[..., None]
    codes = np.clip(np.rint(x / step), -127, 127)
    codes = np.where(scale[..., None] > 0, codes, 0.0)
    return codes.astype(np.int8), np.where(finite, scale, np.float32(np.nan)).astype(np.float32)


def attention_i8(q, k_codes, v_codes, k_scale, v_scale, block_table, lens, starts, max_len, max_new, scale):
    """q [T, Hq, D] over codes [blocks, Hkv, page, D] and scales [blocks, Hkv,
    page] -> float64 [T, Hq, D]; rows that no request computes are NaN."""
    k = k_codes.astype(np.float64) * k_scale.astype(np.float64)[..., None]
    v = v_codes.astype(np.float64) * v_scale.astype(np.float64)[..., None]
    group = q.shape[1] // k.shape[1]
    out = np.full(q.shape, np.nan)
    for b, t, n in visible(q.shape[0], lens, starts, max_len, max_new):
        kk, vv = (paged_rows(c, block_table[b], n, c.shape[2]) for c in (k, v))
        for h in range(q.shape[1]):
            out[t, h] = attend(q[t, h], kk[:, h // group], vv[:, h // group], scale)
    return out


def visible(tokens, lens, starts, max_len, max_new):
    """(request, row of q, positions it sees) of every row that is computed."""
    rows = []
    for b in range(len(lens)):
        first, end = (b, b + 1) if starts is None else (min(max(int(s), 0), tokens) for s in starts[b:b + 2])
        for i in range(min(max(end - first, 0), max_new)):
            sees = int(lens[b]) - (end - first) + i + 1
            rows.append((b, first + i, max(0, min(sees, max_len))))
    return rows
