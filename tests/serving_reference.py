"""Plain 64-bit implementations (numpy, one session and row after another) of the serving
operators: logit controls, the 4-bit cache and attention over it.  Written from the definitions in
include/sdcp.h; they share no code with the library."""
import numpy as np

GROUP = 32


def bf16(x):
    """float array -> the nearest bfloat16 (ties to even), as float32; NaN stays."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r).astype(np.float32)


# ---- logit controls -------------------------------------------------------------------

def adjust_row(l, prompt, outputs, drafts, ctl, biases, mask):
    """One row: (adjusted float64 row, the largest magnitude any step of an entry went through,
    whether anything applied)."""
    V = l.shape[0]
    c = np.zeros(V)
    for t in list(outputs) + list(drafts):
        if 0 <= t < V:
            c[t] += 1
    seen = c > 0
    for t in prompt:
        if 0 <= t < V:
            seen[t] = True
    rep, freq, pres = (np.float64(np.float32(x)) for x in ctl)
    with np.errstate(invalid="ignore", over="ignore"):
        z = l.astype(np.float64)
        z = np.where(seen, np.where(z > 0, z / rep, z * rep), z)
        most = np.maximum(np.abs(l), np.abs(z)) + np.abs(freq) * c + np.abs(pres) * (c > 0)
        z = np.where(c > 0, z - freq * c - pres, z)
    applied = seen.copy()
    for t, v in biases:
        z[t] += np.float64(v)
        most[t] += abs(np.float64(v))
        applied[t] = True
    if mask is not None:
        for t in range(V):
            if not (int(mask[t // 32]) >> (t % 32)) & 1:
                z[t], applied[t] = -np.inf, True
    return z, most, applied


# ---- the cache ------------------------------------------------------------------------

def scale_of(byte):
    return (1 + (byte % 8) / 8.0) * 2.0 ** (byte // 8 - 15)


def channel_place(slot, d, P, D):
    """(byte of the code, its shift, byte of the scale) of channel d of a token slot in a block."""
    g, r = divmod(d, GROUP)
    w, e = divmod(r, 8)
    bit = 4 * (e // 2 + 4 * (e % 2))
    return (g * P + slot) * 16 + w * 4 + bit // 8, bit % 8, P * D // 2 + slot * (D // GROUP) + g


def token_values(block, slot, P, D):
    """float64 [D] of a token slot."""
    out = np.zeros(D)
    for d in range(D):
        at, shift, sb = channel_place(slot, d, P, D)
        out[d] = (((int(block[at]) >> shift) & 15) - 8) * scale_of(int(block[sb]))
    return out


def block_values(blocks, P, D):
    """float64 [..., P, D] of whole blocks [..., bytes]."""
    at = np.zeros((P, D), dtype=np.int64)
    sh = np.zeros((P, D), dtype=np.int64)
    sb = np.zeros((P, D), dtype=np.int64)
    for p in range(P):
        for d in range(D):
            at[p, d], sh[p, d], sb[p, d] = channel_place(p, d, P, D)
    n = (blocks[..., at].astype(np.int64) >> sh) & 15
    b = blocks[..., sb].astype(np.int64)
    return (n - 8) * (1 + (b % 8) / 8.0) * 2.0 ** (b // 8 - 15)


def quantise_row(x):
    """float32 [D] -> (codes n [D], scale bytes [D/32]); x / s and the largest / 7 in float32."""
    n = np.zeros(x.shape[0], dtype=np.int64)
    sbs = []
    for g in range(x.shape[0] // GROUP):
        y = x[g * GROUP:(g + 1) * GROUP].astype(np.float32)
        mags = np.abs(y)[~np.isnan(y)]
        most = np.float32(mags.max()) if mags.size else np.float32(0)
        t = np.float32(most / np.float32(7))
        sb = 8
        while sb < 167 and scale_of(sb) < float(t):
            sb += 1
        sbs.append(sb)
        with np.errstate(invalid="ignore"):
            q = np.clip(np.rint(y / np.float32(scale_of(sb))), -7, 7)
        n[g * GROUP:(g + 1) * GROUP] = np.where(np.isnan(y), 0, np.nan_to_num(q)).astype(np.int64)
    return n, np.array(sbs)


def write_token(block, slot, P, D, n, sbs):
    for d in range(D):
        at, shift, sb = channel_place(slot, d, P, D)
        block[at] = (int(block[at]) & ~(15 << shift)) | ((int(n[d]) + 8) << shift)
        block[sb] = sbs[d // GROUP]


def rotate_row(x, row, layout, dtype):
    """x [D] turned by a table row (cosines, then sines) in `dtype` arithmetic, one rounding a step."""
    x = x.astype(dtype)
    out = x.copy()
    if row is None:
        return out
    half = row.shape[0] // 2
    with np.errstate(invalid="ignore"):
        for j in range(half):
            a, b = (j, j + half) if layout == 0 else (2 * j, 2 * j + 1)
            c, s = dtype(row[j]), dtype(row[half + j])
            out[a] = dtype(x[a] * c) - dtype(x[b] * s)
            out[b] = dtype(x[b] * c) + dtype(x[a] * s)
    return out


# ---- attention ------------------------------------------------------------------------

def attend_row(q, keys, values, scale, first, last):
    """q [D] over keys / values [tokens, D] at positions first..last: (out, sum p |v|, the largest
    sum of magnitudes a score is made of)."""
    k, v = keys[first:last + 1], values[first:last + 1]
    s = (k @ q) * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v), (np.abs(k) @ np.abs(q)).max() * abs(scale)
