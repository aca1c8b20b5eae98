"""fp64 CPU definitions of the serving operators: norm and rotation of queries
and keys, attention with a window and sinks, the 4-bit cache (values and
bytes), pages and slots.  Plain loops and tables; test infrastructure only.
"""

from __future__ import annotations

import numpy as np

from .rbs_oracle import as_f64, rope_rotate

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 non-negative e4m3 values by bit pattern: exponent bias 7, subnormals below 2^-6
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


# ---- norm and rotation


def qk_norm_rope(x, weight, pos, theta: float, eps: float, style: int = 0):
    """x [B, L, H, 128], pos [B, L] -> (rotated rows, size of the pair behind every value) in fp64."""
    x = as_f64(x)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * as_f64(weight)
    out = np.stack([rope_rotate(y[b:b + 1], np.asarray(pos[b]), theta, style)[0] for b in range(x.shape[0])])
    if style == 0:
        pair = np.abs(y[..., :64]) + np.abs(y[..., 64:])
        size = np.concatenate([pair, pair], -1)
    else:
        size = np.repeat(np.abs(y[..., 0::2]) + np.abs(y[..., 1::2]), 2, axis=-1)
    return out, size


# ---- attention over the keys a query may see


def visible(qpos, kpos, window: int, sinks: int):
    q, k = np.asarray(qpos)[:, None], np.asarray(kpos)[None, :]
    see = k <= q
    if window > 0:
        see &= (k > q - window) | (k < sinks)
    return see


def attend(q, k, v, see, scale: float):
    """q [n, 128], k and v [m, 128], see [n, m] -> outputs, ln sum exp, and the error scales
    a = sum_s softmax_s |v_s| per value and z = largest scale * sum |q k| per row."""
    s = scale * (q @ k.T)
    z = scale * (np.abs(q) @ np.abs(k).T)
    out = np.zeros((q.shape[0], v.shape[1]))
    a = np.zeros_like(out)
    lse = np.full(q.shape[0], -np.inf)
    zmax = np.zeros(q.shape[0])
    for i in range(q.shape[0]):
        idx = np.flatnonzero(see[i])
        if idx.size == 0:
            continue
        m = s[i, idx].max()
        p = np.exp(s[i, idx] - m)
        out[i] = p @ v[idx] / p.sum()
        a[i] = p @ np.abs(v[idx]) / p.sum()
        lse[i] = m + np.log(p.sum())
        zmax[i] = z[i, idx].max()
    return out, lse, a, zmax


def window_attention(Q, K, V, window: int, sinks: int, q_offset: int = 0, scale: float | None = None, rows=None):
    """Q [B, Lq, Hq, 128], K, V [B, Lk, Hkv, 128]; rows: the query tokens to compute (all)."""
    Q, K, V = as_f64(Q), as_f64(K), as_f64(V)
    B, Lq, Hq, D = Q.shape
    Hkv = K.shape[2]
    scale = D ** -0.5 if scale is None else scale
    rows = np.arange(Lq) if rows is None else np.asarray(rows)
    out = np.zeros((B, rows.size, Hq, D))
    a = np.zeros_like(out)
    lse = np.zeros((B, Hq, rows.size))
    z = np.zeros((B, Hq, rows.size))
    see = visible(rows + q_offset, np.arange(K.shape[1]), window, sinks)
    cols = np.flatnonzero(see.any(0))
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            o, e, aa, zz = attend(Q[b, rows, h], K[b, cols, g], V[b, cols, g], see[:, cols], scale)
            out[b, :, h], lse[b, h], a[b, :, h], z[b, h] = o, e, aa, zz
    return out, lse, a, z


# ---- the 4-bit format


def _nearest(x, grid):
    """Index of the grid value nearest to x >= 0, the even index of two equally near."""
    up = np.clip(np.searchsorted(grid, x), 1, grid.size - 1)
    d0, d1 = x - grid[up - 1], grid[up] - x
    return np.where((d0 < d1) | ((d0 == d1) & (up % 2 == 1)), up - 1, up)


def quantise(x, g: float = 1.0):
    """x [..., 128] -> codes [..., 128] and scale bits [..., 8] (uint8)."""
    x = as_f64(x)
    r = (x / g).reshape(*x.shape[:-1], 8, 16)
    fine = np.isfinite(r).all(-1)
    r = np.where(fine[..., None], r, 0.0)
    bits = _nearest(np.abs(r).max(-1) / 6.0, E4M3)
    s = E4M3[bits]
    ratio = np.abs(r) / np.where(s > 0, s, 1.0)[..., None]
    code = np.where((s > 0)[..., None], _nearest(ratio, LEVELS), 0)
    code = code + np.where((s > 0)[..., None] & np.signbit(r), 8, 0)
    return code.reshape(x.shape).astype(np.uint8), np.where(fine, bits, 0x7F).astype(np.uint8)


def values(code, bits, g: float = 1.0):
    level = np.concatenate([LEVELS, -LEVELS])[code].reshape(*code.shape[:-1], 8, 16)
    s = np.where(bits == 0x7F, np.nan, E4M3[np.minimum(bits, 126)])
    return (level * s[..., None] * g).reshape(code.shape)


def round_trip(x, g: float = 1.0):
    return values(*quantise(x, g), g)


def write_token(data, slot: int, page: int, head: int, kc, ks, vc, vs) -> None:
    """One token's codes [128] and scales [8] of keys and values into data [num_pages, Hkv, page bytes], byte by byte."""
    off = slot % page
    sub = data[slot // page, head].reshape(-1, 2304)[off // 16]
    t = off % 16
    h, r, j, i = t // 8, t % 8, (t % 8) // 2, t % 2
    for s in range(8):
        for jj in range(4):
            for e in range(2):
                d = 16 * s + 8 * e + 2 * jj
                sub[512 * h + 64 * r + 16 * jj + 2 * s + e] = kc[d] | (kc[d + 1] << 4)
        for rr in range(8):
            d = 16 * s + rr
            sub[1024 + 512 * h + 64 * rr + 16 * j + 8 * i + s] = vc[d] | (vc[d + 8] << 4)
        sub[2048 + 8 * t + s] = ks[s]
        sub[2176 + 16 * (t // 2) + 2 * s + i] = vs[s]


# ---- pages and slots


def extend(table, old, new, free, head: int, max_new: int, page: int):
    """Table after the call, slots, positions, pages taken.  Lengths and pages must be in range."""
    table = table.copy()
    slots = np.full((len(old), max_new), -1, dtype=np.int64)
    pos = np.full((len(old), max_new), -1, dtype=np.int64)
    for b, (o, n) in enumerate(zip(old, new)):
        for e in range(-(-o // page), -(-n // page)):
            table[b, e] = free[head]
            head += 1
        for i in range(min(n - o, max_new)):
            pos[b, i] = o + i
            slots[b, i] = table[b, (o + i) // page] * page + (o + i) % page
    return table, slots, pos, head
