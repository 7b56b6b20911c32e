"""Plain 64-bit implementations of the operators over the 4-bit pool and of
shared pages, by their definitions (include/pagedkv.h), in numpy."""
import numpy as np

CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def e4m3(byte):
    """Value of e4m3 bytes (0x7f is not a number)."""
    byte = np.asarray(byte).astype(np.int64)
    e, m = byte >> 3 & 15, byte & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((byte & 127) == 127, np.nan, v)
    return np.where(byte & 128, -v, v)


SCALES = e4m3(np.arange(127))  # 0 .. 448


def nearest(x, grid):
    """Index of the nearest grid value, ties to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise(x, by=1.0):
    """x [..][d] -> codes 0 .. 15 [..][d], scale bytes [..][d / 16]."""
    y = np.asarray(x, dtype=np.float64) / by
    g = y.reshape(*y.shape[:-1], -1, 16)
    top = np.abs(g).max(-1) / 6
    nan = np.isnan(top)
    byte = np.clip(nearest(np.minimum(np.where(nan, 1.0, top), 448.0), SCALES), 1, 126)
    with np.errstate(invalid="ignore"):
        q = g / SCALES[byte][..., None]
    code = np.where(np.isnan(q), 0, nearest(np.minimum(np.abs(np.nan_to_num(q, nan=0.0, posinf=9.0, neginf=-9.0)), 6.0), CODES))
    code = code + 8 * (g < 0)  # -0 is written as 0
    return code.reshape(y.shape), np.where(nan, 127, byte)


def offsets(d):
    """Byte and shift of the code of (k|v, token, column), byte of the scale of (k|v, token, group)."""
    tok, col, grp = np.arange(16)[:, None], np.arange(d)[None], np.arange(d // 16)[None]
    half, c, e = tok // 8, tok % 8 // 2, tok % 2
    eighth, within = col // (d // 8), col % (d // 8)
    code = np.stack([tok * (d // 2) + col // 2 + 0 * tok,
                     8 * d + (((half * 8 + eighth) * 4 + c) * 2 + e) * (d // 16) + within // 2])
    q = d // 64
    scale = np.stack([16 * d + (((tok % 8) * 4 + grp // q) * 2 + half) * q + grp % q,
                      17 * d + ((grp * 4 + c) * 2 + half) * 2 + e])
    return code, (col % 2) * 4, scale


def unpack(pool):
    """pool uint8 [nb][hkv][18 d] -> values [nb][2][hkv][16][d]."""
    pool = np.asarray(pool)
    d = pool.shape[-1] // 18
    code, shift, scale = offsets(d)
    out = np.empty((pool.shape[0], 2, pool.shape[1], 16, d))
    for kv in range(2):
        c = pool[..., code[kv]] >> shift & 15
        s = e4m3(pool[..., scale[kv]])
        v = CODES[c & 7] * np.repeat(s, 16, -1)
        out[:, kv] = np.where(c & 8, -v, v)
    return out


def pack_token(pool, slot, k, v, k_by=1.0, v_by=1.0):
    """Writes one token's k, v [hkv][d] into pool, in place."""
    d = k.shape[-1]
    code, _, scale = offsets(d)
    blk, row = slot // 16, slot % 16
    for kv, (x, by) in enumerate(((k, k_by), (v, v_by))):
        c, s = quantise(x, by)
        pool[blk][:, code[kv][row, ::2]] = c[:, ::2] | c[:, 1::2] << 4
        pool[blk][:, scale[kv][row]] = s


def attend(q, values, table, lens, qsl, scale, k_by=1.0, v_by=1.0):
    """Returns (out, bound) [T][hq][d]: 64-bit attention, and what an
    implementation with 32-bit scores and sums, probabilities in fp16 and a bf16
    output may be off by. Rows of no request are NaN, with bound NaN."""
    q = np.asarray(q, dtype=np.float64)
    t, hq, d = q.shape
    hkv = values.shape[2]
    out, tol = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for r, n in enumerate(lens):
        a, b = qsl[r], qsl[r + 1]
        if a == b:
            continue
        blocks = values[np.asarray(table[r][:-(-n // 16)])]
        for h in range(hkv):
            k = blocks[:, 0, h].reshape(-1, d)[:n] * k_by
            v = blocks[:, 1, h].reshape(-1, d)[:n] * v_by
            g = hq // hkv
            for i in range(a, b):
                p = n - (b - a) + (i - a)
                qq = q[i, h * g:(h + 1) * g]
                z = qq @ k[:p + 1].T * scale
                w = np.exp(z - z.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o, mag = w @ v[:p + 1], w @ np.abs(v[:p + 1])
                # scores: 2^-20 of the sum of magnitudes (128 products in 32 bits, q in fp16 against its
                # row's largest), and 2^-22 of the exponent for its own rounding and exp2's
                top = np.abs(qq).max(-1, keepdims=True)
                ds = 2.0 ** -20 * scale * ((np.abs(qq) + 2.0 ** -4 * top) @ np.abs(k[:p + 1]).T).max(-1, keepdims=True)
                ds = ds + 2.0 ** -22 * (z.max(-1, keepdims=True) - z.min(-1, keepdims=True))
                out[i, h * g:(h + 1) * g] = o
                # fp16's half step 2^-11 for p, sums 2^-14, bf16's half step 2^-8 for the output. Below 2^-14
                # fp16's half step stays 2^-25: p is taken against a reference that the largest score is not
                # below, so the row's sum is at least 1 and the output off by at most 2^-25 of the sum of |v|.
                tol[i, h * g:(h + 1) * g] = (2.0 ** -8 * 1.01 * np.abs(o) + mag * (2.0 ** -11 + 2.0 ** -14 + 2.5 * ds)
                                             + 2.0 ** -25 * np.abs(v[:p + 1]).sum(0) + 1e-37)
    return out, tol


def fork(parents, table, lens, shares, free, cursor, width):
    """Returns (table, lens, shares, free, cursor, src, dst)."""
    shares, free = list(shares), list(free)
    children = [[r for r, p in enumerate(parents) if p == q] for q in range(len(lens))]
    for q, n in enumerate(lens):
        c = len(children[q])
        for b in table[q][:n // 16]:
            shares[b] += c - 1
        if n % 16 and c == 0:
            shares[table[q][n // 16]] -= 1
    gone = []
    for q, n in enumerate(lens):
        if children[q]:
            continue
        for b in table[q][:-(-n // 16)]:
            if shares[b] == -1:
                shares[b] = 0
                gone.append(b)
    cursor -= len(gone)
    free[cursor:cursor + len(gone)] = gone
    out, out_lens, src, dst = [], [], [], []
    for r, p in enumerate(parents):
        n = lens[p] if p >= 0 else 0
        line = list(table[p][:-(-n // 16)]) if p >= 0 else []
        s = d = -1
        if n % 16 and children[p][0] != r:
            s, d = line[-1], free[cursor]
            line[-1] = d
            cursor += 1
        out.append(line + [-1] * (width - len(line)))
        out_lens.append(n)
        src.append(s)
        dst.append(d)
    return out, out_lens, shares, free, cursor, src, dst
