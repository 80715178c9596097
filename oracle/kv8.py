"""The 8-bit K/V cache operators in numpy, from their definitions (include/llm_ops.h): quantisation and
requantisation in fp32 exactly as defined there, everything else in 64 bits.

A cache is a dict: fmt ("int8" or "e4m3"), codes k and v as uint8 [pages][Hkv][16][d], scales ks and vs
as float32 [pages][Hkv].
"""
import numpy as np

PAGE = 16
CODE_MAX = {"int8": np.float32(127), "e4m3": np.float32(448)}


def _e4m3_values():
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(b & 0x7F) == 0x7F] = np.nan
    return np.where(b & 0x80, -v, v).astype(np.float32)


E4M3 = _e4m3_values()


def decode(codes, fmt):
    return codes.view(np.int8).astype(np.float32) if fmt == "int8" else E4M3[codes]


def encode(x, fmt):
    """fp32 values to codes: half to even, saturating; NaN becomes 0."""
    x = np.nan_to_num(np.asarray(x, np.float32), nan=0.0, posinf=np.inf, neginf=-np.inf)
    x = np.clip(x, -CODE_MAX[fmt], CODE_MAX[fmt])
    if fmt == "int8":
        return np.rint(x).astype(np.int8).view(np.uint8)
    a = np.abs(x).astype(np.float64)
    # steps of 2^(e - 3) in [2^e, 2^(e + 1)), 2^-9 below 2^-6
    e = np.maximum(np.frexp(a)[1] - 1, -6)
    q = np.rint(a * 2.0 ** (3.0 - e)) * 2.0 ** (e - 3.0)
    code = np.searchsorted(E4M3[:0x7F].astype(np.float64), q).astype(np.uint8)
    return code | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)


def sequences(row_start, kv_len):
    """(sequence, first row, rows, kv) of each sequence."""
    return [(b, int(row_start[b]), int(row_start[b + 1] - row_start[b]), int(kv_len[b])) for b in range(len(kv_len))]


def _touched(n, kv):
    """(logical page, first slot, slots, first row of the sequence's) of every page that its last n tokens lie in."""
    out, first = [], kv - n
    for page in range(first // PAGE, (kv - 1) // PAGE + 1) if n else []:
        s0, s1 = max(first - page * PAGE, 0), min(kv - page * PAGE, PAGE)
        out.append((page, s0, s1 - s0, page * PAGE + s0 - first))
    return out


def append(cache, table, row_start, kv_len, k, v):
    """k, v: float32 [rows][Hkv][d] (16-bit rows converted).  Changes the cache."""
    fmt = cache["fmt"]
    for b, row0, n, kv in sequences(row_start, kv_len):
        for page, s0, cnt, r in _touched(n, kv):
            p = table[b, page]
            for x, codes, scale in ((k, cache["k"], cache["ks"]), (v, cache["v"], cache["vs"])):
                new = x[row0 + r:row0 + r + cnt].astype(np.float32)
                for h in range(new.shape[1]):
                    top = np.abs(new[:, h]).max()
                    fresh = np.float32(top) / CODE_MAX[fmt] if np.isfinite(top) else np.float32(np.nan)
                    old, s = scale[p, h], fresh
                    if s0 > 0:
                        grown = np.isnan(fresh) or fresh > old
                        if grown:
                            with np.errstate(all="ignore"):
                                again = decode(codes[p, h, :s0], fmt) * (old / fresh)
                            codes[p, h, :s0] = encode(again, fmt) if fresh > 0 else 0
                        else:
                            s = old
                    scale[p, h] = s
                    with np.errstate(all="ignore"):
                        codes[p, h, s0:s0 + cnt] = encode(new[:, h] / s, fmt) if s > 0 else 0


def read(cache, table, row_start, kv_len, rows):
    """-> k, v as float32 [rows][Hkv][d] (code * scale rounded to fp32)."""
    out = []
    for codes, scale in ((cache["k"], cache["ks"]), (cache["v"], cache["vs"])):
        x = np.zeros((rows,) + (codes.shape[1], codes.shape[3]), np.float32)
        for b, row0, n, kv in sequences(row_start, kv_len):
            for page, s0, cnt, r in _touched(n, kv):
                p = table[b, page]
                val = decode(codes[p, :, s0:s0 + cnt], cache["fmt"]) * scale[p][:, None, None]
                x[row0 + r:row0 + r + cnt] = val.transpose(1, 0, 2)
        out.append(x)
    return out


def attention(cache, table, row_start, kv_len, q):
    """q: [rows][Hq][d] -> out, lse, and per (row, head) the sums that bounds on the error are made of: the
    weighted sum of |V| and the plain sum of |V| (same shape as out), and the largest sum of |q_i k_i| / sqrt(d)
    over the keys."""
    rows, Hq, d = q.shape
    Hkv = cache["k"].shape[1]
    out, absv, sumv = (np.zeros((rows, Hq, d)) for _ in range(3))
    lse, absqk = np.full((rows, Hq), -np.inf), np.zeros((rows, Hq))
    for b, row0, n, kv in sequences(row_start, kv_len):
        pages = table[b, :-(-kv // PAGE)]
        for g in range(Hkv):
            K = (decode(cache["k"][pages, g], cache["fmt"]).astype(np.float64) * cache["ks"][pages, g].astype(np.float64)[:, None, None])
            V = (decode(cache["v"][pages, g], cache["fmt"]).astype(np.float64) * cache["vs"][pages, g].astype(np.float64)[:, None, None])
            K, V = K.reshape(-1, d), V.reshape(-1, d)
            for i in range(n):
                seen = kv - n + i + 1
                if seen <= 0:
                    continue
                for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                    x = q[row0 + i, h].astype(np.float64)
                    s = K[:seen] @ x / np.sqrt(d)
                    top = s.max()
                    w = np.exp(s - top)
                    lse[row0 + i, h] = top + np.log(w.sum())
                    w /= w.sum()
                    out[row0 + i, h] = w @ V[:seen]
                    absv[row0 + i, h] = w @ np.abs(V[:seen])
                    sumv[row0 + i, h] = np.abs(V[:seen]).sum(0)
                    absqk[row0 + i, h] = (np.abs(K[:seen]) @ np.abs(x)).max() / np.sqrt(d)
    return out, lse, absv, sumv, absqk


def norm_rope(x, gain, eps, base, pos):
    """x [rows][H][d] -> float64."""
    x = x.astype(np.float64)
    d = x.shape[-1]
    if gain is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * gain.astype(np.float64)
    ang = pos.astype(np.float64)[:, None] * base ** (-2.0 * np.arange(d // 2) / d)
    co, si = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([a * co - b * si, b * co + a * si], -1)
