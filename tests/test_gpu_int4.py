"""The 4-bit cache on the GPU against the 64-bit reference of int4_ref.

Tolerances, from the arithmetic:
- Stores and reads: bit for bit.  What is quantised is the rotated row rounded to fp32 and to bf16.
- Decode: the fp32 output rounds to bf16 (2^-8 |out|).  P rounds to f16 (2^-11 of each weight, and 2^-25 of an
  absolute error where it is subnormal, with the largest p_t s_t held at 2^7 or more: together 2^-11 A with the A
  below), and the exponents' fp32 error is a few 2^-20 at the scores used here: within 2^-10 A.  The sums over codes
  and over zero points are apart, and C = 15 sum p s bounds either.  An instruction adds 16 products to an
  accumulator in fp32: the accumulator loses 2^-23 of C in each of n / 16 + 8 steps.  Each of the 17 numbers is cut
  at 2^-24 of the largest of them, and there a code operand c 2^-21, below the normal f16 range, counts as the
  number below 2^-13 that its exponent field allows: 17 2^-24 2^-13 p_max, which is 17 2^-16 p_max s in units of
  elements.  The instructions' p_max add up to sum p at most: 17 2^-16 / 15 C.  (A first form of this bound counted
  one rounding an instruction and none for the field.)
- Prefill: the same output rounding, and P in bf16 (2^-8 of each weight): 2^-8 |out| + 2^-8 (1 + 2^-6) A.
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import int4_ref as R
import serving_ref as S
from paged_kv_cache_244_gb300 import _build

pytestmark = pytest.mark.gpu
B, D = 16, 128


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    _build.build()
    from paged_kv_cache_244_gb300 import binding
    binding.get_device_status()
    return binding


def clean(pa, want=0):
    rc, flags = pa.get_device_status()
    assert flags == want, (rc, hex(flags))


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    return up(np.asarray(a, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.detach().view(torch.int16).cpu().numpy()


def table_of(P, Rr, theta=1e4):
    a = np.arange(P)[:, None] * S.frequencies(Rr, theta)[None, :]
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def normal(rng, *shape, spread=0.0):
    x = rng.standard_normal(shape)
    if spread:
        x = x * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    return S.bf16_round(x)


def turned(x, cs, layout):
    """The rotated rows as bf16 (by way of fp32)."""
    return S.bf16_round(S.rotate(x, cs, layout).astype(np.float32))


class Pool:
    """A cache of random records with shuffled tables; slots past the contexts hold NaN scales."""

    def __init__(self, rng, lens, kv, spread=0.0, extra=3, canary=True):
        need = [(n + B - 1) // B for n in lens]
        self.nb = sum(need) + extra
        perm = rng.permutation(self.nb)[: sum(need)]
        self.tables = np.full((len(lens), max(max(need), 1)), 1 << 30, np.int32)   # past the context: never read
        at = 0
        for s, k in enumerate(need):
            self.tables[s, :k] = perm[at:at + k]
            at += k
        self.lens = np.array(lens, np.int32)
        self.cache = R.random_records(rng, (self.nb, kv), spread)
        if canary:
            for s, n in enumerate(lens):
                if n % B:
                    rec = self.cache[self.tables[s, n // B]]
                    rec[:, R.K_SCALES + 8 * (n % B):R.V_SCALES] = 0xFF
                    rec[:, R.V_SCALES + 2 * (n % B):] = 0xFF

    def dev(self):
        return up(self.cache)

    def attention(self, s, q, scale, first=None):
        return R.attention(q, self.cache, self.tables[s], int(self.lens[s]), scale, first)


def close(got, ref, what="", steps=0, prefill=False):
    out, mag, sums = ref
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all(), what
    w = 2.0 ** -8 * (1 + 2.0 ** -6) * mag if prefill else 2.0 ** -10 * mag + ((steps + 8) * 2.0 ** -23 + 17 / 15 * 2.0 ** -16) * sums
    err, bound = np.abs(got - out), 2.0 ** -8 * np.abs(out) + w + 1e-30
    assert (err <= bound).all(), (what, float((err / bound).max()))


# ---- reading back -------------------------------------------------------------------------

@pytest.mark.parametrize("kv,lens,first", [(2, [1], [0]), (1, [17, 0, 5], [0, 3, 15]), (8, [100, 33, 16, 250], [16, 31, 1, 0]),
                                           (3, [1, 1, 1], [15, 16, 17])])
def test_read_gives_the_elements(pa, kv, lens, first):
    rng = np.random.default_rng(3)
    p = Pool(rng, [f + n for f, n in zip(first, lens)], kv, spread=4.0, canary=False)
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(starts[-1]) + 2                                    # two rows behind the last sequence
    k = torch.full((rows, kv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    got = pa.read_kv_int4(p.dev(), up(starts), up(np.array(first, np.int32)), up(p.tables), max(max(lens), 1), k_out=k, v_out=v)
    assert got[0] is k and got[1] is v
    for s, n in enumerate(lens):
        K, V = (x.swapaxes(1, 2).reshape(-1, kv, D) for x in R.unpack(p.cache[p.tables[s, : (first[s] + n + B - 1) // B]]))
        a, b = starts[s], starts[s + 1]
        assert np.array_equal(f64(k[a:b]), K[first[s]:first[s] + n]) and np.array_equal(f64(v[a:b]), V[first[s]:first[s] + n])
    assert (f64(k[-2:]) == 7.0).all() and (f64(v[-2:]) == 7.0).all()
    clean(pa)
    k2, v2 = pa.read_kv_int4(p.dev(), up(starts), None, up(p.tables), max(max(lens), 1), num_rows=rows)
    assert np.array_equal(f64(k2[0]), R.unpack(p.cache[p.tables[0, 0]])[0][:, 0])
    clean(pa)


def test_read_skips_what_is_out_of_range(pa):
    rng = np.random.default_rng(4)
    p = Pool(rng, [40, 40, 40, 40, 40, 40], 2, canary=False)
    p.tables[0, 1] = p.nb
    p.tables[1, 2] = -1
    starts = np.array([0, 40, 80, 90, 100, 140, 200], np.int32)   # the last sequence reaches past the 180 rows
    first = np.array([0, 0, -1, 39, 0, 0], np.int32)              # 3: tokens past the table
    k, v = (torch.full((180, 2, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pa.read_kv_int4(p.dev(), up(starts), up(first), up(p.tables), 40, k_out=k, v_out=v)
    clean(pa, pa.PA_FLAG_BLOCK_ID_OOB | pa.PA_FLAG_CONTEXT_LEN_OOB)
    k, v = f64(k), f64(v)
    for s, rows in ((0, [*range(16), *range(32, 40)]), (1, range(32)), (4, range(40))):
        K = R.unpack(p.cache[np.clip(p.tables[s, :3], 0, p.nb - 1)])[0].swapaxes(1, 2).reshape(-1, 2, D)
        want = np.full((40, 2, D), 7.0)
        want[list(rows)] = K[list(rows)]
        assert np.array_equal(k[starts[s]:starts[s] + 40], want), s
    assert (k[80:100] == 7.0).all() and (k[140:] == 7.0).all() and (v[80:100] == 7.0).all()


# ---- the store ----------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Rr,T,hq,kv", [(128, 37, 12, 2), (64, 1, 8, 8), (16, 50, 5, 1), (96, 19, 9, 3), (112, 330, 4, 4),
                                        (48, 9, 64, 8), (80, 70, 28, 4), (32, 3, 7, 7), (128, 3, 1, 1), (16, 2600, 3, 3)])
def test_store_bit_for_bit(pa, layout, Rr, T, hq, kv):
    rng = np.random.default_rng(Rr + T)
    nb = (T + B - 1) // B + 3
    slots = rng.permutation(nb * B)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    pos = rng.integers(0, 500, T).astype(np.int32)
    cs = table_of(500, Rr)
    q, k, v = normal(rng, T, hq, D), normal(rng, T, kv, D, spread=2.0), normal(rng, T, kv, D, spread=2.0)
    k[..., 3] *= 16
    before = R.random_records(rng, (nb, kv))
    cache, q_dev = up(before), bf16(q)
    q_out = torch.empty_like(q_dev)
    got = pa.rope_kv_store_int4(q_dev, bf16(k), bf16(v), up(pos), up(cs), up(slots), cache, layout=layout, q_out=q_out)
    assert got is q_out and np.array_equal(f64(q_dev), q)
    qr = S.rotate(q, cs[pos], layout)
    assert (np.abs(f64(q_out) - qr) <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -20 * np.abs(qr) + 1e-30).all()
    kr, want = turned(k, cs[pos], layout), before.copy()
    for t, slot in enumerate(slots):
        for g in range(kv):
            if slot >= 0:
                R.put_row(want[slot // B, g], int(slot % B), kr[t, g], v[t, g])
    assert np.array_equal(cache.cpu().numpy(), want)
    clean(pa)
    # in place, and as the bf16 store rotates
    kb, vb = (torch.zeros((nb, kv, B, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q2 = bf16(q)
    pa.rope_kv_store_form(q2, bf16(k), bf16(v), up(pos), up(cs), up(slots), kb, vb, layout=layout)
    pa.rope_kv_store_int4(q_dev, bf16(k), bf16(v), up(pos), up(cs), up(slots), cache, layout=layout)
    assert np.array_equal(bits(q_dev), bits(q2)) and np.array_equal(bits(q_out), bits(q2))
    assert np.array_equal(cache.cpu().numpy(), want)
    clean(pa)


def test_store_of_extreme_rows(pa):
    rng = np.random.default_rng(8)
    rows = np.zeros((12, 1, D))
    rows[1] = 3e38 * np.sign(rng.standard_normal((1, D)))
    rows[2, 0, 5] = 1e-38
    rows[3, 0, :40] = -1.0
    rows[4, 0, 9], rows[4, 0, 64:] = math.inf, rng.standard_normal(64)
    rows[5, 0, 9], rows[5, 0, 70], rows[5, 0, 71] = -math.inf, math.nan, 2.0
    rows[6] = 1.0
    rows[7] = -1.0
    rows[8, 0] = np.arange(D) / 8 - 8
    rows[9] = rng.standard_normal((1, D)) * 2.0 ** -45
    rows[10] = rng.standard_normal((1, D)) * 2.0 ** 47
    rows[11, 0, 0], rows[11, 0, 127] = math.nan, math.inf
    x = S.bf16_round(rows.astype(np.float32).astype(np.float64))
    x = f64(bf16(x))
    cs = np.concatenate([np.ones((1, 64)), np.zeros((1, 64))], axis=1).astype(np.float32)
    cache = pa.int4_cache(1, 1)
    q = torch.zeros((12, 1, D), dtype=torch.bfloat16, device="cuda")
    pa.rope_kv_store_int4(q, bf16(x[::-1]), bf16(x), torch.zeros(12, dtype=torch.int32, device="cuda"), up(cs), up(np.arange(12)), cache)
    want = np.zeros((1, 1, R.RECORD), np.uint8)
    with np.errstate(invalid="ignore"):
        k = turned(x[::-1], cs[np.zeros(12, int)], "half")      # by no angle: a value stays, inf * 0 is NaN in its partner
    for t in range(12):
        R.put_row(want[0, 0], t, k[t, 0], x[t, 0])
    got = cache.cpu().numpy()
    scales = slice(R.K_SCALES, R.RECORD)
    assert np.array_equal(got[0, 0, scales].view(np.uint16), want[0, 0, scales].view(np.uint16))
    gk, gv = R.unpack(got[0, 0])
    wk, wv = R.unpack(want[0, 0])
    assert np.array_equal(gk, wk, equal_nan=True) and np.array_equal(gv, wv, equal_nan=True)
    clean(pa)


def test_a_rotated_infinity_is_the_same_in_every_row(pa):
    """An infinity stays one under a rotation, and its partner becomes NaN (a difference with an infinite product), however
    near the other values of the row come to a border of their rounding."""
    rng = np.random.default_rng(10)
    n = 8192
    k = normal(rng, n, 1, D)
    k[:, 0, 9] = math.inf
    cs = table_of(n, 128)                                  # row 0 turns by nothing: inf * 0
    pos = 1 + np.arange(n, dtype=np.int32) % (n - 1)
    cache = pa.int4_cache(n // B, 1)
    q = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    args = (bf16(k), bf16(k), up(pos), up(cs), up(np.arange(n)))
    pa.rope_kv_store_int4(q, *args, cache)
    got, _ = pa.read_kv_int4(cache, up(np.array([0, n], np.int32)), None, up(np.arange(n // B, dtype=np.int32)[None]), n, n)
    got = f64(got)[:, 0]
    assert np.isfinite(got[:, :64]).all()                  # dim 9 reads as an end of its range
    assert np.isnan(got[:, 64:96]).all()                   # the dims of its partner, 73
    assert np.isfinite(got[:, 96:]).all()
    # the fused step stores the same bytes
    stored, step, one = pa.int4_cache(n, 1), pa.int4_cache(n, 1), up(cs[7:8])
    pa.rope_kv_store_int4(q, bf16(k), bf16(k), torch.zeros_like(up(pos)), one, up(B * np.arange(n)), stored)
    pa.decode_step_int4(q, bf16(k), bf16(k), one, step, up(np.arange(n, dtype=np.int32)[:, None]), up(np.ones(n, np.int32)), B, 0.1)
    assert torch.equal(step, stored)
    clean(pa)


def test_store_skips_bad_positions_and_slots(pa):
    rng = np.random.default_rng(9)
    q, k, v = normal(rng, 5, 6, D), normal(rng, 5, 2, D), normal(rng, 5, 2, D)
    cs = table_of(10, 128)
    before = R.random_records(rng, (2, 2))
    cache, out = up(before), torch.zeros((5, 6, D), dtype=torch.bfloat16, device="cuda")
    pos, slots = np.array([0, 10, -1, 4, 5], np.int32), np.array([0, 1, 2, 32, -5])
    pa.rope_kv_store_int4(bf16(q), bf16(k), bf16(v), up(pos), up(cs), up(slots), cache, q_out=out)
    clean(pa, pa.PA_FLAG_POSITION_OOB | pa.PA_FLAG_SLOT_OOB)
    want = before.copy()
    for g in range(2):
        R.put_row(want[0, g], 0, turned(k, cs[np.clip(pos, 0, 9)], "half")[0, g], v[0, g])
    assert np.array_equal(cache.cpu().numpy(), want)
    assert np.array_equal(f64(out[1:3]), q[1:3])          # unrotated
    assert not np.array_equal(f64(out[3:]), q[3:])        # rotated, though not stored


# ---- decode -------------------------------------------------------------------------------

@pytest.mark.parametrize("hq,kv,lens,P", [
    (12, 2, [1], 0), (12, 2, [2048], 0), (5, 1, [0, 1, 15, 16, 17, 31, 33], 0), (8, 8, [100, 0, 0, 7, 64], 0),
    (64, 8, [65, 129, 700], 0), (9, 3, [300, 1, 40], 16), (28, 4, [513, 512, 511], 64), (16, 2, [5000, 3], 512),
    (7, 7, [49], 0), (32, 8, [1000] * 20, 0),
])
@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_decode(pa, hq, kv, lens, P, spread):
    rng = np.random.default_rng(len(lens) + hq)
    p = Pool(rng, lens, kv, spread)
    q = normal(rng, len(lens), hq, D, spread=0.5)
    mx = max(max(lens), 1)
    scale = 0.25 * D ** -0.5 if spread else D ** -0.5
    got = pa.decode_int4(bf16(q), p.dev(), up(p.tables), up(p.lens), mx, scale, partition_tokens=P)
    again = pa.decode_int4(bf16(q), p.dev(), up(p.tables), up(p.lens), mx, scale, partition_tokens=P)
    assert np.array_equal(bits(got), bits(again))
    for s, n in enumerate(lens):
        close(got[s:s + 1], p.attention(s, q[s:s + 1], scale), (s, n), steps=n // 16 + 1)
        if n == 0:
            assert (f64(got[s]) == 0).all()
    clean(pa)


@pytest.mark.parametrize("qmag,exponent,scale", [(1.0, 36, 1.0), (2.0 ** 100, -3, 1.0), (3e38, 36, 1.0), (1e-38, -40, 1e-3),
                                                 (2.0 ** -126, 30, D ** -0.5)])
def test_decode_and_prefill_of_far_magnitudes_are_finite_and_right(pa, qmag, exponent, scale):
    """Scores far past anything a softmax tells apart (one key has all the weight), or all alike.  The reference's
    score differences are either past 2^10 or below 2^-12 here, so the weights are known to 2^-10."""
    rng = np.random.default_rng(5)
    lens = [70, 33]
    p = Pool(rng, lens, 2)
    p.cache = R.random_records(rng, p.cache.shape[:2], 0.0, exponent)
    q = S.bf16_round(np.sign(normal(rng, 2, 6, D)) * min(qmag, 3e38))
    qd = bf16(q)
    q = f64(qd)
    got = pa.decode_int4(qd, p.dev(), up(p.tables), up(p.lens), 70, scale)
    pre = pa.prefill_int4(qd, up(np.array([0, 1, 2], np.int32)), p.dev(), up(p.tables), up(p.lens), 1, 70, scale)
    for s in range(2):
        ref = p.attention(s, q[s:s + 1], scale)
        for o in (got, pre):
            o = f64(o[s:s + 1])
            assert np.isfinite(o).all()
            err = np.abs(o - ref[0])
            assert (err <= 2.0 ** -6 * (np.abs(ref[0]) + ref[1])).all(), float((err / ref[1]).max())
    clean(pa)


def test_decode_nan_and_infinity(pa):
    rng = np.random.default_rng(6)
    lens = [40, 40, 40, 40]
    p = Pool(rng, lens, 2)
    q = normal(rng, 4, 4, D)
    p.cache[p.tables[0, 1], 0, R.K_SCALES + 8 * 3 + 2:R.K_SCALES + 8 * 3 + 4] = (0xC0, 0x7F)   # K of token 19, dims 32-63
    p.cache[p.tables[1, 2], 1, R.V_SCALES + 2 * 7:R.V_SCALES + 2 * 8] = (0xC0, 0x7F)           # V of token 39
    q[2, 1, 5] = math.inf
    q[3, 2, 9] = math.nan
    got = f64(pa.decode_int4(bf16(q), p.dev(), up(p.tables), up(p.lens), 40, 0.1))
    nan = np.zeros((4, 4), bool)
    nan[0, :2] = nan[1, 2:] = nan[2, 1] = nan[3, 2] = True
    assert (np.isnan(got).all(axis=-1) == nan).all() and (np.isfinite(got).all(axis=-1) == ~nan).all()
    clean(pa)


def test_decode_out_of_range_blocks_and_lengths(pa):
    rng = np.random.default_rng(7)
    p = Pool(rng, [64, 64, 32, 20], 2)
    q = normal(rng, 4, 6, D)
    tables = p.tables.copy()
    tables[0, 1] = p.nb
    tables[1, 3] = -3
    tables[2, :2] = 1 << 20
    got = pa.decode_int4(bf16(q), p.dev(), up(tables), up(np.array([64, 64, 32, -5], np.int32)), 64, 0.1)
    clean(pa, pa.PA_FLAG_BLOCK_ID_OOB | pa.PA_FLAG_CONTEXT_LEN_OOB)
    for s, keep in ((0, [0, 2, 3]), (1, [0, 1, 2])):
        close(got[s:s + 1], R.attention(q[s:s + 1], p.cache, p.tables[s, keep], 48, 0.1), s, steps=4)
    assert (f64(got[2:]) == 0).all()
    out = pa.prefill_int4(bf16(q[:1]), up(np.array([0, 1], np.int32)), p.dev(), up(tables[:1]), up(p.lens[:1]), 1, 64, 0.1)
    clean(pa, pa.PA_FLAG_BLOCK_ID_OOB)
    close(out, R.attention(q[:1], p.cache, p.tables[0, [0, 2, 3]], 48, 0.1), prefill=True)


# ---- the fused step -----------------------------------------------------------------------

@pytest.mark.parametrize("layout,Rr", [("half", 128), ("half", 48), ("half", 96), ("interleaved", 128), ("interleaved", 80)])
@pytest.mark.parametrize("hq,kv,lens", [(12, 2, [1, 16, 17, 0, 300]), (8, 8, [33]), (64, 8, [5, 6, 7, 130]), (7, 7, [1] * 9)])
def test_step_is_store_then_decode(pa, layout, Rr, hq, kv, lens):
    rng = np.random.default_rng(Rr + hq)
    p = Pool(rng, lens, kv)
    n = len(lens)
    q, k, v = bf16(normal(rng, n, hq, D)), bf16(normal(rng, n, kv, D, spread=1.0)), bf16(normal(rng, n, kv, D, spread=1.0))
    cs = up(table_of(310, Rr))
    c1, c2 = p.dev(), p.dev()
    pos = np.maximum(p.lens - 1, 0)
    slots = np.where(p.lens > 0, p.tables[np.arange(n), pos // B].astype(np.int64) * B + pos % B, -1)
    q0 = q.clone()
    out = pa.decode_step_int4(q, k, v, cs, c1, up(p.tables), up(p.lens), max(lens), 0.1, layout=layout)
    turned_q = pa.rope_kv_store_int4(q, k, v, up(pos.astype(np.int32)), cs, up(slots), c2, layout=layout, q_out=torch.empty_like(q))
    ref = pa.decode_int4(turned_q, c2, up(p.tables), up(p.lens), max(lens), 0.1)
    assert torch.equal(q, q0) and torch.equal(c1, c2)
    assert np.array_equal(bits(out), bits(ref))
    clean(pa)
    # a step behind another kernel of the stream, its tables written long before
    c3, tables, ctx = p.dev(), up(p.tables), up(p.lens)
    torch.cuda.synchronize()
    busy = torch.randn((2048, 2048), device="cuda")
    for _ in range(3):
        busy = busy @ busy
    early = pa.decode_step_int4(q, k, v, cs, c3, tables, ctx, max(lens), 0.1, layout=layout, early_metadata=True)
    assert np.array_equal(bits(early), bits(out)) and torch.equal(c3, c1)


def test_step_position_past_the_table(pa):
    rng = np.random.default_rng(12)
    p = Pool(rng, [20, 5], 2)
    q, k, v = bf16(normal(rng, 2, 4, D)), bf16(normal(rng, 2, 2, D)), bf16(normal(rng, 2, 2, D))
    cache = p.dev()
    out = pa.decode_step_int4(q, k, v, up(table_of(10, 128)), cache, up(p.tables), up(p.lens), 20, 0.1)
    clean(pa, pa.PA_FLAG_POSITION_OOB)
    ref = pa.decode_int4(q, p.dev(), up(p.tables), up(p.lens), 20, 0.1)
    assert np.array_equal(bits(out[0]), bits(ref[0]))               # unrotated, nothing stored
    assert np.array_equal(cache[p.tables[0, 1]].cpu().numpy(), p.cache[p.tables[0, 1]])


# ---- prefill ------------------------------------------------------------------------------

@pytest.mark.parametrize("hq,kv,new,cached", [
    (12, 2, [1], [0]), (12, 2, [40, 1, 130], [0, 100, 7]), (5, 1, [26, 25, 27], [0, 1, 900]), (8, 8, [200], [56]),
    (64, 8, [16, 17, 3], [1, 0, 30]), (9, 3, [43, 0, 5], [9, 40, 11]), (28, 4, [5, 5], [1500, 700]), (7, 7, [300], [0]),
    (12, 2, [21], [4000]), (32, 8, [1, 2, 3], [640, 639, 5]),
])
def test_prefill(pa, hq, kv, new, cached):
    rng = np.random.default_rng(sum(new) + hq)
    lens = [a + b for a, b in zip(new, cached)]
    p = Pool(rng, lens, kv, spread=0.5)
    T = sum(new)
    q = normal(rng, T, hq, D, spread=0.5)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out = torch.full((T + 1, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (up(starts), p.dev(), up(p.tables), up(p.lens), max(max(new), 1), max(lens), 0.1)
    got = pa.prefill_int4(torch.cat((bf16(q), out[:1])), *args, out=out)
    for s, n in enumerate(new):
        if n:
            rows = slice(starts[s], starts[s] + n)
            close(got[rows], p.attention(s, q[rows], 0.1, first=cached[s]), s, prefill=True)
    assert (f64(out[T]) == 7.0).all()
    clean(pa)
    # a bound of the contexts far above them changes how the keys are spread, not the result's meaning
    loose = pa.prefill_int4(bf16(q), up(starts), p.dev(), up(np.pad(p.tables, ((0, 0), (0, 2000)))), up(p.lens), max(max(new), 1),
                            max(lens) + 30000, 0.1)
    for s, n in enumerate(new):
        if n:
            rows = slice(starts[s], starts[s] + n)
            close(loose[rows], p.attention(s, q[rows], 0.1, first=cached[s]), s, prefill=True)


@pytest.mark.parametrize("cached", [30, 1000])
def test_prefill_nan_reaches_the_queries_that_see_it(pa, cached):
    rng = np.random.default_rng(13)
    new, n = 60, cached + 60
    p = Pool(rng, [n, n, n], 2)
    at = cached + 21
    blk = p.tables[:, at // B]
    p.cache[blk[0], 0, R.V_SCALES + 2 * (at % B):R.V_SCALES + 2 * (at % B) + 2] = (0xC0, 0x7F)
    p.cache[blk[1], 1, R.K_SCALES + 8 * (at % B):R.K_SCALES + 8 * (at % B) + 2] = (0xC0, 0x7F)
    q = normal(rng, 3 * new, 6, D)
    q[2 * new + 5, 3, 7] = math.nan
    got = f64(pa.prefill_int4(bf16(q), up(np.arange(4, dtype=np.int32) * new), p.dev(), up(p.tables), up(p.lens), new, n, 0.1))
    nan = np.zeros((3, new, 6), bool)
    nan[0, 21:, :3] = nan[1, 21:, 3:] = nan[2, 5, 3] = True
    got = got.reshape(3, new, 6, D)
    assert (np.isnan(got).all(axis=-1) == nan).all() and (np.isfinite(got).all(axis=-1) == ~nan).all()
    clean(pa)


def test_prefill_skips_bad_sequences(pa):
    rng = np.random.default_rng(14)
    p = Pool(rng, [40, 40, 40], 2)
    q = normal(rng, 30, 4, D)
    out = torch.full((30, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pa.prefill_int4(bf16(q), up(np.array([0, 10, 20, 31], np.int32)), p.dev(), up(p.tables), up(np.array([40, 5, 40], np.int32)),
                    20, 48, 0.1, out=out)
    clean(pa, pa.PA_FLAG_CONTEXT_LEN_OOB)
    close(out[:10], p.attention(0, q[:10], 0.1, first=30), prefill=True)
    assert (f64(out[10:]) == 7.0).all()


def test_prefill_under_jitter(pa):
    rng = np.random.default_rng(15)
    new, cached = [150, 9], [77, 900]
    p = Pool(rng, [a + b for a, b in zip(new, cached)], 2)
    q = bf16(normal(rng, 159, 12, D))
    starts = up(np.array([0, 150, 159], np.int32))

    def both():
        return [bits(pa.prefill_int4(*a)) for a in (
            (q, starts, p.dev(), up(p.tables), up(p.lens), 150, 909, 0.1),
            (q[150:].contiguous(), up(np.array([0, 9], np.int32)), p.dev(), up(p.tables[1:]), up(p.lens[1:]), 9, 909, 0.1))]
    want = both()
    try:
        for seed in range(6):
            torch.cuda.synchronize()
            pa.set_timing_jitter(20000, seed)
            got = both()
            assert all(np.array_equal(a, b) for a, b in zip(got, want)), seed
    finally:
        torch.cuda.synchronize()
        pa.set_timing_jitter(0)
    clean(pa)


# ---- together -----------------------------------------------------------------------------

def test_serving_loop_captured_and_replayed(pa):
    """Prompts stored, prefilled, then steps replayed from one graph, every table built on the GPU; the
    rows read back at the end are what the stores' definition gives."""
    rng = np.random.default_rng(20)
    S_, hq, kv, steps = 3, 12, 2, 20
    new = [37, 5, 16]
    nb, mb = 24, 8
    i32 = dict(dtype=torch.int32, device="cuda")
    cs = table_of(128, 128)
    cs_d = up(cs)
    tables, free = torch.full((S_, mb), -1, **i32), torch.randperm(nb, device="cuda").to(torch.int32)
    num_free, cache = torch.full((1,), nb, **i32), pa.int4_cache(nb, kv)
    T = sum(new)
    k0, v0 = normal(rng, T, kv, D), normal(rng, T, kv, D)
    p = pa.plan_step(torch.zeros(S_, **i32), torch.tensor(new, **i32), tables, free, num_free, nb, T)
    q = bf16(normal(rng, T, hq, D))
    pa.rope_kv_store_int4(q, bf16(k0), bf16(v0), p.positions, cs_d, p.slot_mapping, cache)
    pre = pa.prefill_int4(q, p.q_start, cache, tables, p.context_lens, max(new), mb * B, 0.09)
    lens, one = p.context_lens.clone(), torch.ones(S_, **i32)
    qs, ks, vs = (torch.empty((S_, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, kv, kv))
    ws = pa.decode_workspace_int4(qs, cache, mb * B)
    out, plan = torch.empty_like(qs), pa.step_plan(S_, S_)

    def step():
        pa.plan_step(lens, one, tables, free, num_free, nb, S_, plan=plan)
        pa.decode_step_int4(qs, ks, vs, cs_d, cache, tables, plan.context_lens, mb * B, 0.09, workspace=ws, out=out)
        lens.copy_(plan.context_lens)

    all_k, all_v = normal(rng, steps, S_, kv, D), normal(rng, steps, S_, kv, D)
    all_q = normal(rng, steps, S_, hq, D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    outs = []
    for i in range(steps):
        qs.copy_(bf16(all_q[i])), ks.copy_(bf16(all_k[i])), vs.copy_(bf16(all_v[i]))
        if i == 0:
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        elif i == 1:
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        else:
            graph.replay()
        outs.append(out.clone())
    clean(pa)
    starts = np.concatenate([[0], np.cumsum(np.array(new) + steps)]).astype(np.int32)
    k, v = pa.read_kv_int4(cache, up(starts), None, tables, mb * B, num_rows=int(starts[-1]))
    host = cache.cpu().numpy()
    tab = tables.cpu().numpy()
    at = np.concatenate([[0], np.cumsum(new)])
    for s in range(S_):
        n = new[s] + steps
        rows_k = np.concatenate([k0[at[s]:at[s + 1]], all_k[:, s]])
        rows_v = np.concatenate([v0[at[s]:at[s + 1]], all_v[:, s]])
        kr = turned(rows_k, cs[:n], "half")
        for i in range(n):
            for g in range(kv):
                rec = np.zeros(R.RECORD, np.uint8)
                R.put_row(rec, 0, kr[i, g], rows_v[i, g])
                wk, wv = R.unpack(rec)
                assert np.array_equal(f64(k[starts[s] + i, g]), wk[0]) and np.array_equal(f64(v[starts[s] + i, g]), wv[0])
        qr = S.bf16_round(S.rotate(all_q[:, s], cs[new[s]:n], "half"))
        for i in (0, 1, 7, steps - 1):
            # q rotated in fp32 may be a bf16 step from the rotation in 64 bits: 2^-8 of each element, which moves
            # scores of size x by 2^-8 x at most and here by far less than 2^-7 in all
            ref = R.attention(qr[i:i + 1], host, tab[s], new[s] + i + 1, 0.09)
            assert (np.abs(f64(outs[i][s:s + 1]) - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -6 * ref[1] + 1e-30).all()
        q_p = f64(q[at[s]:at[s + 1]])
        close(pre[at[s]:at[s + 1]], R.attention(q_p, host, tab[s], new[s], 0.09, first=0), s, prefill=True)


def test_streams_and_concurrent_calls(pa):
    """Two calls at once on two streams, each with its own workspace, and outputs allocated for the stream."""
    rng = np.random.default_rng(21)
    pools = [Pool(rng, [900, 40, 3], 4) for _ in range(2)]
    qs = [bf16(normal(rng, 3, 28, D)) for _ in range(2)]
    args = [(q, p.dev(), up(p.tables), up(p.lens), 900, 0.1) for q, p in zip(qs, pools)]
    want = [bits(pa.decode_int4(*a)) for a in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [pa.decode_int4(*a, stream=st) for a, st in zip(args, streams)]
        torch.cuda.synchronize()
        assert all(np.array_equal(bits(g), w) for g, w in zip(got, want))
    clean(pa)


def test_offsets_past_32_bits(pa):
    """A pool of over 4 GiB, the context in its last blocks."""
    rng = np.random.default_rng(22)
    kv, nb = 8, 250_000
    cache = torch.empty((nb, kv, R.RECORD), dtype=torch.uint8, device="cuda")
    n = 50
    tables = np.array([[nb - 1, nb - 7, nb - 3, nb - 2]], np.int32)
    rec = R.random_records(rng, (4, kv))
    cache[up(tables[0].astype(np.int64))] = up(rec)
    q = normal(rng, 1, 16, D)
    ref = R.attention(q, rec, np.arange(4), n, 0.1)
    lens, tab = up(np.array([n], np.int32)), up(tables)
    close(pa.decode_int4(bf16(q), cache, tab, lens, n, 0.1), ref, steps=4)
    close(pa.prefill_int4(bf16(q), up(np.array([0, 1], np.int32)), cache, tab, lens, 1, n, 0.1), ref, prefill=True)
    k, v = pa.read_kv_int4(cache, up(np.array([0, n], np.int32)), None, tab, n, num_rows=n)
    assert np.array_equal(f64(k), R.unpack(rec)[0].swapaxes(1, 2).reshape(-1, kv, D)[:n])
    x = normal(rng, 1, kv, D)
    cs = np.concatenate([np.ones((1, 64)), np.zeros((1, 64))], axis=1).astype(np.float32)
    pa.rope_kv_store_int4(bf16(normal(rng, 1, 8, D)), bf16(x), bf16(x), torch.zeros(1, dtype=torch.int32, device="cuda"), up(cs),
                          up(np.array([(nb - 2) * B + 5])), cache)
    for g in range(kv):
        R.put_row(rec[3, g], 5, x[0, g], x[0, g])
    assert np.array_equal(cache[nb - 2].cpu().numpy(), rec[3])
    clean(pa)


def test_long_context_sums(pa):
    """A context of 40,000 tokens with nearly even weights: sums of codes and of zero points are far larger than what
    is left of them."""
    rng = np.random.default_rng(23)
    n = 40_000
    p = Pool(rng, [n], 1)
    q = normal(rng, 1, 8, D) * 0.05
    q = f64(bf16(q))
    ref = p.attention(0, q, D ** -0.5)
    # a warp's range of the even split has some 1.4 blocks here and the pieces are joined in fp32; with a partition
    # for the whole context a piece is what a range holds all the same
    close(pa.decode_int4(bf16(q), p.dev(), up(p.tables), up(p.lens), n, D ** -0.5), ref, steps=64)


# ---- at the limits ------------------------------------------------------------------------

@pytest.mark.parametrize("step", [False, True])
def test_most_sequences_of_a_call(pa, step):
    """8192 sequences: their block-count prefix leaves fewer stages and warps; most contexts are a few tokens or none."""
    rng = np.random.default_rng(30)
    n = 8192
    lens = rng.integers(1 if step else 0, 12, n)
    lens[[5, 4000, 8191]] = [300, 65, 17]
    p = Pool(rng, lens.tolist(), 1)
    q = normal(rng, n, 8, D)
    cache = p.dev()
    if step:
        k, v = normal(rng, n, 1, D), normal(rng, n, 1, D)
        cs = table_of(310, 64)
        got = pa.decode_step_int4(bf16(q), bf16(k), bf16(v), up(cs), cache, up(p.tables), up(p.lens), 300, 0.1)
        pos = (p.lens - 1).astype(np.int32)
        slots = p.tables[np.arange(n), pos // B].astype(np.int64) * B + pos % B
        other = p.dev()
        qr = pa.rope_kv_store_int4(bf16(q), bf16(k), bf16(v), up(pos), up(cs), up(slots), other)
        assert torch.equal(cache, other)
        q, p.cache = f64(qr), cache.cpu().numpy()
        assert np.array_equal(bits(got), bits(pa.decode_int4(qr, cache, up(p.tables), up(p.lens), 300, 0.1)))
    else:
        got = pa.decode_int4(bf16(q), cache, up(p.tables), up(p.lens), 300, 0.1)
    for s in [0, 1, 5, 4000, 8190, 8191, *rng.integers(0, n, 60)]:
        close(got[s:s + 1], p.attention(s, q[s:s + 1], 0.1), s, steps=int(lens[s]) // 16 + 1)
    clean(pa)


def test_many_heads(pa):
    rng = np.random.default_rng(31)
    lens, kv = [40, 17], 257
    p = Pool(rng, lens, kv)
    q = normal(rng, 2, kv, D)
    got = pa.decode_int4(bf16(q), p.dev(), up(p.tables), up(p.lens), 40, 0.1)
    pre = pa.prefill_int4(bf16(q), up(np.array([0, 1, 2], np.int32)), p.dev(), up(p.tables), up(p.lens), 1, 40, 0.1)
    for s in range(2):
        ref = p.attention(s, q[s:s + 1], 0.1)
        close(got[s:s + 1], ref, s, steps=4)
        close(pre[s:s + 1], ref, s, prefill=True)
    clean(pa)


def test_read_of_thousands_of_sequences(pa):
    rng = np.random.default_rng(32)
    n = 5000
    rows = rng.integers(0, 3, n)
    rows[77] = 200
    first = rng.integers(0, 30, n)
    p = Pool(rng, (first + rows).tolist(), 2, canary=False)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    k, v = pa.read_kv_int4(p.dev(), up(starts), up(first.astype(np.int32)), up(p.tables), 200, num_rows=int(starts[-1]))
    seq = np.repeat(np.arange(n), rows)
    at = np.arange(starts[-1]) - starts[seq] + first[seq]
    K, V = (x[np.arange(len(at)), :, at % B] for x in R.unpack(p.cache[p.tables[seq, at // B]]))
    assert np.array_equal(f64(k), K) and np.array_equal(f64(v), V)
    clean(pa)


def test_a_layer_chain_with_early_metadata(pa):
    """The steps of many layers, each started while the one before it finishes, give what they give one by one."""
    rng = np.random.default_rng(33)
    lens, layers = [5, 300, 64, 33] * 8, 12
    pools = [Pool(rng, lens, 2) for _ in range(layers)]
    q, k, v = (bf16(normal(rng, layers, len(lens), h, D)) for h in (12, 2, 2))
    cs = up(table_of(310, 128))
    tabs, ctx = [up(p.tables) for p in pools], up(pools[0].lens)
    ws = pa.decode_workspace_int4(q[0], pools[0].dev(), 300)

    def chain(early):
        caches = [p.dev() for p in pools]
        outs = [torch.empty_like(q[0]) for _ in range(layers)]
        torch.cuda.synchronize()
        for i in range(layers):
            pa.decode_step_int4(q[i], k[i], v[i], cs, caches[i], tabs[i], ctx, 300, 0.1, workspace=ws, out=outs[i], early_metadata=early)
        torch.cuda.synchronize()
        return outs, caches
    (o1, c1), (o2, c2) = chain(False), chain(True)
    assert all(torch.equal(a, b) for a, b in zip(o1 + c1, o2 + c2))
    clean(pa)


def test_two_graphs_in_turn_share_a_workspace(pa):
    rng = np.random.default_rng(34)
    pools = [Pool(rng, lens, 4) for lens in ([700, 20], [33, 5, 900])]
    ws = torch.empty(1 << 22, device="cuda")
    calls = []
    for p in pools:
        q = bf16(normal(rng, len(p.lens), 28, D))
        calls.append((q, p.dev(), up(p.tables), up(p.lens), int(p.lens.max()), 0.1))
    want = [bits(pa.decode_int4(*c)) for c in calls]
    outs, graphs = [torch.empty_like(c[0]) for c in calls], []
    for c, o in zip(calls, outs):
        pa.decode_int4(*c, workspace=ws, out=o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.decode_int4(*c, workspace=ws, out=o)
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        assert all(np.array_equal(bits(o), w) for o, w in zip(outs, want))
    clean(pa)


def test_the_binding_refuses_wrong_tensors(pa):
    rng = np.random.default_rng(35)
    p = Pool(rng, [20, 20], 2)
    q, cache, t, n = bf16(normal(rng, 2, 4, D)), p.dev(), up(p.tables), up(p.lens)
    starts = up(np.array([0, 1, 2], np.int32))
    for bad in (cache[..., :2000].contiguous(), cache[0], cache.to(torch.int8), cache.transpose(0, 1), cache.cpu()):
        with pytest.raises((ValueError, pa.PaError)):
            pa.decode_int4(q, bad, t, n, 20, 0.1)
        with pytest.raises((ValueError, pa.PaError)):
            pa.prefill_int4(q, starts, bad, t, n, 1, 20, 0.1)
        with pytest.raises((ValueError, pa.PaError)):
            pa.read_kv_int4(bad, starts, None, t, 20, k_out=q[:, :2].contiguous(), v_out=q[:, 2:].contiguous())
    for args in ((q.half(), cache, t, n), (q[:1], cache, t, n), (q, cache, t.long(), n), (q, cache, t, n[:1]), (q[..., :64].contiguous(), cache, t, n)):
        with pytest.raises((ValueError, pa.PaError)):
            pa.decode_int4(*args, 20, 0.1)
    with pytest.raises((ValueError, pa.PaError)):
        pa.read_kv_int4(cache, starts, n[:1], t, 20, num_rows=2)
    with pytest.raises((ValueError, pa.PaError)):
        pa.rope_kv_store_int4(q, q, q, n, up(table_of(30, 128)), up(np.zeros(2, np.int64)), cache)   # k of 4 KV heads
    with pytest.raises(pa.PaError) as e:
        pa.decode_int4(q, cache, t, n, 20, -1.0)
    assert e.value.code == pa.PA_ERR_RANGE
    with pytest.raises(pa.PaError) as e:
        pa.decode_int4(q, cache, t, n, 20, 0.1, workspace=torch.empty(8, device="cuda"))
    assert e.value.code == pa.PA_ERR_WORKSPACE
    assert pa.decode_int4(q[:0], cache, t[:0], n[:0], 20, 0.1).shape == (0, 4, D)
    clean(pa)


def test_a_call_on_a_stream_of_its_own_with_what_it_allocates(pa):
    rng = np.random.default_rng(36)
    p = Pool(rng, [900, 40], 2)
    q = bf16(normal(rng, 2, 12, D))
    args = (p.dev(), up(p.tables), up(p.lens), 900, 0.1)
    want = bits(pa.decode_int4(q, *args))
    rows = up(np.array([0, 1, 2], np.int32))
    want_p = bits(pa.prefill_int4(q, rows, *args[:3], 1, 900, 0.1))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        a = pa.decode_int4(q, *args, stream=st)
        b = pa.prefill_int4(q, rows, *args[:3], 1, 900, 0.1, stream=st)
        k, v = pa.read_kv_int4(args[0], up(np.array([0, 900, 940], np.int32)), None, args[1], 900, num_rows=940, stream=st)
        torch.cuda.current_stream().wait_stream(st)
        assert np.array_equal(bits(a), want) and np.array_equal(bits(b), want_p)
    clean(pa)
