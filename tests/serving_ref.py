"""Plain 64-bit references of the step plan, the RoPE forms and the block-scaled E4M3 caches.

numpy only, written from the definitions in include/pa.h; nothing here is shared with the CUDA
path.  bf16 values travel as float64 (exact) or as bit patterns where bits are compared.
"""

from __future__ import annotations

import math

import numpy as np

D = 128
B = 16
SCALE_LO, SCALE_HI = 2.0 ** -40, 2.0 ** 40


def _e4m3_value(c: int) -> float:
    sign, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
    if (c & 0x7F) == 0x7F:
        return math.nan
    return sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


E4M3 = np.array([_e4m3_value(c) for c in range(256)])
_UP = E4M3[:127]                       # 0 .. 448, increasing
_MID = (_UP[:-1] + _UP[1:]) / 2        # exact


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code (ties to the even code), magnitudes beyond 448 and infinities 448, NaN 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    with np.errstate(invalid="ignore"):
        lo = np.searchsorted(_MID, a, side="left")      # first code whose upper midpoint is >= a
    tie = (lo < 126) & (a == _MID[np.minimum(lo, 125)])
    code = lo + (tie & (lo % 2 == 1))                    # a tie goes up from an odd code
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def bf16_round(x: np.ndarray) -> np.ndarray:
    """float64 -> nearest bf16 value (ties to even), as float64.  Normal range only."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    r = np.ldexp(np.round(np.ldexp(m, 8)), e - 8)        # 8 significant bits; np.round ties to even
    return np.where(np.isfinite(x), r, x)


def wanted_scale(x: np.ndarray) -> float:
    a = np.abs(x[np.isfinite(x)])
    top = float(a.max()) if a.size else 0.0
    s = SCALE_LO
    while s < SCALE_HI and top > 448.0 * s:
        s *= 2
    return s


def frequencies(R, theta, kind="none", factor=1.0, original=0.0, low=0.0, high=0.0):
    i = np.arange(R // 2, dtype=np.float64)
    w = theta ** (-2 * i / R)
    if kind == "linear":
        return w / factor
    if kind == "ntk":
        return (theta * factor ** (R / (R - 2))) ** (-2 * i / R)
    if kind == "yarn":
        d = [R * math.log(original / (2 * math.pi * t)) / (2 * math.log(theta)) for t in (high, low)]
        a, b = (min(max(v, 0), R - 1) for v in (math.floor(d[0]), math.ceil(d[1])))
        r = np.clip((i - a) / ((b - a) or 0.001), 0, 1)
        return w / factor * r + w * (1 - r)
    if kind == "banded":
        m = np.clip((original * w / (2 * math.pi) - low) / (high - low), 0, 1)
        return w / factor * (1 - m) + w * m
    return w


def rotate(x, cs, layout):
    """x [T, H, 128], cs [T, R] (cos | sin): the rotated dims in float64, not rounded."""
    half = cs.shape[1] // 2
    c, s = cs[:, None, :half].astype(np.float64), cs[:, None, half:].astype(np.float64)
    y = np.array(x, np.float64)
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    p, q = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = p * c - q * s, q * c + p * s
    return y


def store_block(codes, scales, rows):
    """One (block, KV head), K or V: codes [16, 128] uint8, its scale, rows {slot: values [128]}."""
    want = wanted_scale(np.concatenate([np.ravel(v) for v in rows.values()]))
    old = scales
    now = want if 0 in rows or not old > want else old
    codes = codes.copy()
    if 0 not in rows and now != old:
        for r in range(B):
            if r not in rows:
                codes[r] = e4m3_encode(E4M3[codes[r]] * (old / now))
    for r, v in rows.items():
        codes[r] = e4m3_encode(np.asarray(v, np.float64) / now)
    return codes, now


def store(cache, scale, x, slots):
    """cache [nb, Hkv, 16, 128] uint8 and scale [nb, Hkv] updated by rows x [T, Hkv, 128] (bf16
    values); a negative slot stores nothing."""
    cache, scale = cache.copy(), scale.copy()
    by_block: dict[int, dict[int, int]] = {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            by_block.setdefault(int(slot) // B, {})[int(slot) % B] = t
    for blk, rows in by_block.items():
        for g in range(cache.shape[1]):
            cache[blk, g], scale[blk, g] = store_block(cache[blk, g], float(scale[blk, g]),
                                                       {o: x[t, g] for o, t in rows.items()})
    return cache, scale


def attention(q, k_codes, v_codes, kv_scale, block_tables, n, scale, first=None):
    """One sequence: q [R, Hq, 128] rows at positions first .. first + R - 1 (None: one row that sees
    all n tokens).  Returns (out, A): out [R, Hq, 128]; A, times 2^-9, bounds what weights rounded
    to f16 lose: the softmax-weighted mean of |V| (2^-11 of each weight), and for weights that are
    f16 subnormals 2^-25 of an absolute error each, where the largest p_t v_t is held at 2^7 or
    more: 2^-32 max_t(p_t v_t) sum_t |code_t|."""
    R, Hq, _ = q.shape
    Hkv = k_codes.shape[1]
    G = Hq // Hkv
    ids = block_tables[: (n + B - 1) // B]
    out, mag = np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    if n == 0:
        return out, mag
    for g in range(Hkv):
        K, C = (np.concatenate([E4M3[c[b, g]] * (float(kv_scale[b, g, 0]) if c is k_codes else 1.0) for b in ids])[:n]
                for c in (k_codes, v_codes))
        vs = np.repeat(kv_scale[ids, g, 1].astype(np.float64), B)[:n]
        V = C * vs[:, None]
        x = np.einsum("rhd,td->rht", q[:, g * G:(g + 1) * G].astype(np.float64), K) * scale
        if first is not None:
            x = np.where(np.arange(n)[None, None, :] <= first + np.arange(R)[:, None, None], x, -np.inf)
        p = np.exp(x - x.max(axis=-1, keepdims=True))
        p /= p.sum(axis=-1, keepdims=True)
        out[:, g * G:(g + 1) * G] = p @ V
        mag[:, g * G:(g + 1) * G] = p @ np.abs(V) + 2.0 ** -23 * (p * vs).max(axis=-1)[..., None] * np.abs(C).sum(axis=0)
    return out, mag


def plan(cached, new, tables, free, num_free, num_blocks, T):
    """pa_plan_step, sequence after sequence.  Returns a dict and the set of flags raised."""
    S, width = tables.shape
    flags = set()
    tables = tables.copy()
    F = int(num_free)
    if not 0 <= F <= len(free):
        flags.add("block")
        F = min(max(F, 0), len(free))
    ctx, granted = np.zeros(S, np.int32), np.zeros(S, np.int32)
    starts, pos, slots = np.zeros(S + 1, np.int32), np.zeros(T, np.int32), np.full(T, -1, np.int64)
    row, asked, taken = 0, 0, 0
    for s in range(S):
        c, n = int(cached[s]), int(new[s])
        starts[s] = min(row, T)
        first = row
        if 0 <= n <= T:
            row += n
        ok = 0 <= n <= T and c >= 0 and c + n <= width * B and row <= T
        if not ok:
            flags.add("len")
            continue
        old = -(-c // B)
        need = -(-(c + n) // B) - old
        before, asked = asked, asked + need
        if need and asked > F:
            flags.add("pool")
            continue
        granted[s], ctx[s] = 1, c + n
        for j in range(need):
            i = int(free[F - 1 - (before + j)])
            tables[s, old + j] = i if 0 <= i < num_blocks else -1
            if not 0 <= i < num_blocks:
                flags.add("block")
        taken += need
        for i in range(n):
            p = c + i
            b = int(tables[s, p // B])
            pos[first + i] = p
            if 0 <= b < num_blocks:
                slots[first + i] = b * B + p % B
            else:
                flags.add("block")
    starts[S] = min(row, T)
    return dict(context_lens=ctx, q_start=starts, positions=pos, slot_mapping=slots, granted=granted,
                tables=tables, num_free=F - taken), flags
