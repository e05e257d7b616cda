"""Plain 64-bit reference of the 4-bit cache: record layout, quantisation, reading, attention.

numpy only, written from the definitions in include/pa.h; nothing here is shared with the CUDA path.  bf16
values travel as float64 (exact).
"""

from __future__ import annotations

import math

import numpy as np

D, B, RECORD = 128, 16, 2208
V_CODES, K_SCALES, V_SCALES = 1024, 2048, 2176
SCALES = sorted({m * 2.0 ** (e - 3) for e in range(-40, 40) for m in range(8, 16)} | {2.0 ** 40})
NIBBLE = [0, 4, 1, 5, 2, 6, 3, 7]       # of dim d of eight


def away(x: float) -> float:
    """Nearest integer, ties away from zero."""
    return math.copysign(math.floor(abs(x) + 0.5), x)


def quantise(x):
    """One set of bf16 values: (codes, s, z); s NaN where one of them is."""
    x = np.asarray(x, np.float64)
    fin = x[np.isfinite(x)]
    lo, hi = min(0.0, *fin, 0.0), max(0.0, *fin, 0.0)
    with np.errstate(over="ignore"):
        span = float(np.float32(hi) - np.float32(lo))
    s = next((t for t in SCALES if 15 * t >= span), SCALES[-1])
    z = int(min(15.0, math.floor(-lo / s + 0.5)))
    codes = [0 if math.isnan(v) else int(min(15.0, max(0.0, away(max(min(v / s, 1e9), -1e9)) + z))) for v in x]
    return np.array(codes), (math.nan if np.isnan(x).any() else s), z


def scale_word(s: float, z: int) -> int:
    if math.isnan(s):
        return 0x7FC0
    m, e = math.frexp(s)                 # m in [0.5, 1): 16 m = 8 .. 15
    return (e - 1 + 127) << 7 | (int(m * 16) - 8) << 4 | z


def k_word(t, ch):
    """Byte offset of the word of dims 8 ch .. 8 ch + 7 of K of token t."""
    return 64 * t + 16 * (ch % 4) + 4 * (ch // 4)


def v_word(t, ch):
    return V_CODES + 64 * t + 16 * ((ch // 4) ^ (t // 2 % 4)) + 4 * (ch % 4)


def put_row(rec, t, k, v):
    """Rows k, v [128] into slot t of a record (uint8 [RECORD], in place)."""
    for x, groups, word, scales in ((k, 4, k_word, K_SCALES + 8 * t), (v, 1, v_word, V_SCALES + 2 * t)):
        for g in range(groups):
            n = D // groups
            codes, s, z = quantise(x[g * n:(g + 1) * n])
            rec[scales + 2 * g:scales + 2 * g + 2] = np.frombuffer(np.uint16(scale_word(s, z)).tobytes(), np.uint8)
            for i in range(0, n, 8):
                w = sum(int(codes[i + d]) << 4 * NIBBLE[d] for d in range(8))
                at = word(t, (g * n + i) // 8)
                rec[at:at + 4] = np.frombuffer(np.uint32(w).tobytes(), np.uint8)


def unpack(rec):
    """Elements K, V [..., 16, 128] in 64 bits of records [..., RECORD]."""
    words = np.ascontiguousarray(rec).view(np.uint32)
    halves = np.ascontiguousarray(rec).view(np.uint16).astype(np.uint32)
    t, d = np.arange(B)[:, None], np.arange(D)[None, :]
    out = []
    for word, scale in ((k_word(t, d // 8), K_SCALES // 2 + 4 * t + d // 32), (v_word(t, d // 8), V_SCALES // 2 + t + 0 * d)):
        code = words[..., word // 4] >> (4 * np.array(NIBBLE)[d % 8]).astype(np.uint32) & 15
        h = halves[..., scale]
        s = ((h & 0xFFF0) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
        out.append(s * (code.astype(np.float64) - (h & 15)))
    return out


def random_records(rng, shape, spread=0.0, exponent=-3):
    """Records of random codes, zero points and scales (of many magnitudes where spread is not 0)."""
    rec = rng.integers(0, 256, shape + (RECORD,), dtype=np.uint8)
    n = (RECORD - K_SCALES) // 2
    e = np.round(spread * rng.standard_normal(shape + (n,))).astype(int) + exponent + 127
    word = e << 7 | rng.integers(0, 8, shape + (n,)) << 4 | rng.integers(3, 13, shape + (n,))
    rec[..., K_SCALES:] = np.ascontiguousarray(word.astype(np.uint16)).view(np.uint8)
    return rec


def attention(q, cache, block_tables, n, scale, first=None):
    """One sequence: q [R, Hq, 128] rows at positions first .. first + R - 1 (None: one row that sees all n tokens).
    Returns (out, A, C): out [R, Hq, 128]; A the softmax-weighted mean of |V|, which times the relative error of a
    weight bounds what rounding the weights does to out; C what a relative error 1 of every sum over codes or zero
    points would do to it (the decode sums c and z apart), in the place of A where that is what rounds."""
    R, Hq, _ = q.shape
    Hkv = cache.shape[1]
    G = Hq // Hkv
    ids = block_tables[: (n + B - 1) // B]
    out, mag, sums = (np.zeros((R, Hq, D)) for _ in range(3))
    if n == 0:
        return out, mag, sums
    for g in range(Hkv):
        K, V = (x.reshape(-1, D)[:n] for x in unpack(cache[ids, g]))
        sv = np.repeat(cache[ids, g][:, V_SCALES:].view(np.uint16).reshape(-1, 1), 1, axis=1)[:n, 0].astype(np.uint32)
        sv = ((sv & 0xFFF0) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
        x = np.einsum("rhd,td->rht", q[:, g * G:(g + 1) * G].astype(np.float64), K) * scale
        if first is not None:
            x = np.where(np.arange(n)[None, None, :] <= first + np.arange(R)[:, None, None], x, -np.inf)
        p = np.exp(x - x.max(axis=-1, keepdims=True))
        p /= p.sum(axis=-1, keepdims=True)
        h = slice(g * G, (g + 1) * G)
        out[:, h], mag[:, h] = p @ V, p @ np.abs(V)
        sums[:, h] = 15 * (p @ sv)[..., None]
    return out, mag, sums
