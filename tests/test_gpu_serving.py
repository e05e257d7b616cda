"""RoPE tables and forms, block-scaled E4M3 caches and step plans on the GPU, against the 64-bit
references of serving_ref.

Tolerances, from the arithmetic:
- A bf16 result of an fp32 value within a few ulps of the exact one: half a bf16 step, 2^-8 of the
  value, plus 2^-20 of it for the fp32 part.
- Table entries: the fraction of a turn carries two fp32 roundings (2^-23 of at most one half turn,
  pi 2^-23 in the angle), sincospif at most 2 ulps (2^-22 of 1), the magnitude one more (2^-24).
- Attention: the fp32 output rounds to bf16 (2^-8 |out|); P rounds to f16 (2^-11 of each weight, and
  2^-25 where it is subnormal), and the exponents' fp32 error is a few 2^-20 at the scores used
  here: together within 2^-9 of the A that the reference gives with the result.
- Codes, scales and plans: bit for bit (codes from the rotated k as bf16, which the bf16 store gives).
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import serving_ref as R
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
    a = np.arange(P)[:, None] * R.frequencies(Rr, theta)[None, :]
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def normal(rng, *shape, spread=0.0):
    x = rng.standard_normal(shape)
    if spread:
        x = x * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    return R.bf16_round(x)


class Pool:
    """A block-scaled cache with random codes, scales of many magnitudes and shuffled tables."""

    def __init__(self, rng, lens, kv, spread=1.0, extra=3, canary=True):
        need = [(n + B - 1) // B for n in lens]
        self.nb = sum(need) + extra
        perm = rng.permutation(self.nb)[: sum(need)]
        self.tables = np.full((len(lens), max(max(need), 1)), 1 << 30, np.int32)   # past the context: never read
        at = 0
        for s, k in enumerate(need):
            self.tables[s, :k] = perm[at:at + k]
            at += k
        self.lens = np.array(lens, np.int32)
        x = rng.standard_normal((2, self.nb, kv, B, D))
        e = np.round(spread * 3 * rng.standard_normal((2, self.nb, kv)))
        self.scale = np.ldexp(2.0 ** -7, e.astype(int)).transpose(1, 2, 0).astype(np.float32).copy()
        self.k, self.v = (R.e4m3_encode(x[i] * 100.0) for i in range(2))
        if canary:                                        # slots past the context hold NaN codes
            for s, n in enumerate(lens):
                if n % B:
                    self.k[self.tables[s, n // B], :, n % B:] = 0x7F
                    self.v[self.tables[s, n // B], :, n % B:] = 0xFF

    def dev(self):
        return up(self.k), up(self.v), up(self.scale)

    def attention(self, s, q, scale, first=None):
        return R.attention(q, self.k, self.v, self.scale, self.tables[s], int(self.lens[s]), scale, first)


def close(got, ref, mag, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    err, bound = np.abs(got - ref), 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * mag + 1e-30
    assert np.isfinite(got).all(), what
    assert (err <= bound).all(), (what, float((err / bound).max()))


# ---- tables -------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["none", "linear", "ntk", "yarn", "banded"])
@pytest.mark.parametrize("Rr,P,theta", [(16, 1, 1e4), (128, 4099, 1e6), (96, 131072, 5e5), (48, 777, 1e4), (64, 300001, 1e4)])
def test_rope_table(pa, kind, Rr, P, theta):
    kw = dict(factor=7.5, original=2048.0, low=1.0, high=32.0 if kind == "yarn" else 4.0)
    w = R.frequencies(Rr, theta, kind, **kw)
    m = 0.1 * math.log(7.5) + 1 if kind == "yarn" else 1.0
    got = pa.rope_table(P, Rr, theta, scaling=kind, factor=7.5, original_max_pos=2048, low=kw["low"], high=kw["high"])
    rows = np.unique(np.concatenate([np.arange(min(P, 500)), np.random.default_rng(1).integers(0, P, 500), [P - 1]]))
    a = rows[:, None].astype(np.float64) * w[None, :]
    # the angle itself is a product in 64 bits: 2^-52 of it
    ref = np.concatenate([np.cos(a), np.sin(a)], axis=1) * m
    tol = m * ((math.pi + 2) * 2.0 ** -23 + 2.0 ** -24) + 2.0 ** -50 * P
    assert np.abs(f64(got[up(rows)]) - ref).max() <= tol
    clean(pa)


def test_rope_table_small_angles_keep_relative_accuracy_and_magnitude(pa):
    t = f64(pa.rope_table(9, 128, 1e6, scaling="yarn", factor=4.0, original_max_pos=4096, low=1.0, high=32.0, magnitude=1.25))
    w = R.frequencies(128, 1e6, "yarn", 4.0, 4096.0, 1.0, 32.0)
    ref = np.sin(np.arange(9)[:, None] * w[None, :]) * 1.25
    assert (np.abs(t[:, 64:] - ref) <= 2.0 ** -20 * np.abs(ref)).all()
    assert np.array_equal(t[0], np.r_[np.full(64, 1.25), np.zeros(64)])


# ---- the store with a form ----------------------------------------------------------------

@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Rr,T,hq,kv", [(128, 37, 12, 2), (64, 1, 8, 8), (16, 130, 5, 1), (96, 19, 9, 3), (112, 2500, 4, 4),
                                        (48, 9, 64, 8)])
def test_form_store(pa, layout, Rr, T, hq, kv):
    rng = np.random.default_rng(Rr + T)
    nb, P = T // 8 + 4, 300
    q, k, v = normal(rng, T, hq, D), normal(rng, T, kv, D), normal(rng, T, kv, D)
    cs = table_of(P, Rr)
    pos = rng.integers(0, P, T).astype(np.int32)
    slots = rng.permutation(nb * B)[:T].astype(np.int64)
    slots[rng.random(T) < 0.2] = -1
    qd, out = bf16(q), torch.full((T, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.full((nb, kv, B, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = pa.rope_kv_store_form(qd, bf16(k), bf16(v), up(pos), up(cs), up(slots), kc, vc, layout=layout, q_out=out)
    assert got is out and np.array_equal(f64(qd), q)
    ref_q, ref_k = R.rotate(q, cs[pos], layout), R.rotate(k, cs[pos], layout)
    tol = 2.0 ** -8 + 2.0 ** -20
    assert (np.abs(f64(out) - ref_q) <= tol * np.abs(ref_q)).all()
    at = slots >= 0
    kg, vg = f64(kc), f64(vc)
    blk, off = slots[at] // B, slots[at] % B
    assert (np.abs(kg[blk, :, off] - ref_k[at]) <= tol * np.abs(ref_k[at])).all()
    assert np.array_equal(vg[blk, :, off], v[at])
    untouched = np.ones((nb, B), bool)
    untouched[blk, off] = False
    assert np.isnan(kg.transpose(0, 2, 1, 3)[untouched]).all() and np.isnan(vg.transpose(0, 2, 1, 3)[untouched]).all()
    # in place, the same bits
    pa.rope_kv_store_form(qd, bf16(k), bf16(v), up(pos), up(cs), up(slots), kc, vc, layout=layout)
    assert np.array_equal(bits(qd), bits(out))
    clean(pa)


def test_form_store_of_whole_heads_equals_the_plain_store(pa):
    rng = np.random.default_rng(5)
    T, nb = 61, 9
    q, k, v = bf16(normal(rng, T, 12, D)), bf16(normal(rng, T, 2, D)), bf16(normal(rng, T, 2, D))
    pos, slots, cs = up(np.arange(T, dtype=np.int32)), up(rng.permutation(nb * B)[:T].astype(np.int64)), up(table_of(T, 128))
    caches = [torch.zeros((nb, 2, B, D), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    out = torch.empty_like(q)
    pa.rope_kv_store_form(q, k, v, pos, cs, slots, caches[0], caches[1], q_out=out)
    pa.rope_kv_store(q, k, v, pos, cs, slots, caches[2], caches[3])
    assert np.array_equal(bits(out), bits(q))
    assert np.array_equal(bits(caches[0]), bits(caches[2])) and np.array_equal(bits(caches[1]), bits(caches[3]))


@pytest.mark.parametrize("block", [False, True])
def test_store_skips_what_is_out_of_range(pa, block):
    rng = np.random.default_rng(6)
    T, nb = 6, 2
    q, k, v = (bf16(normal(rng, T, h, D)) for h in (4, 2, 2))
    pos, slots = np.array([0, -1, 10, 3, 4, 5], np.int32), np.array([0, 1, 2, 32, -5, 5], np.int64)
    out = torch.zeros_like(q)
    cs = table_of(10, 64)
    if block:
        kc, vc = (torch.full((nb, 2, B, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        sc = torch.full((nb, 2, 2), 3.0, device="cuda")
        pa.rope_kv_store_fp8_block(q, k, v, up(pos), up(cs), up(slots), kc, vc, sc, q_out=out)
        written = (kc != 0x7F).any(dim=3)[:, 0].cpu().numpy()
        assert (f64(sc)[1] == 3.0).all() and (f64(sc)[0] < 1.0).all()
    else:
        kc, vc = (torch.full((nb, 2, B, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pa.rope_kv_store_form(q, k, v, up(pos), up(cs), up(slots), kc, vc, q_out=out)
        written = (~kc.isnan()).any(dim=3)[:, 0].cpu().numpy()
    assert np.argwhere(written).tolist() == [[0, 0], [0, 5]]
    ref = R.rotate(f64(q), cs[np.clip(pos, 0, 9)], "half")
    bad = (pos < 0) | (pos >= 10)
    assert np.array_equal(f64(out)[bad], f64(q)[bad])                # left unrotated
    assert (np.abs(f64(out) - ref)[~bad] <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref)[~bad]).all()
    clean(pa, pa.PA_FLAG_SLOT_OOB | pa.PA_FLAG_POSITION_OOB)


# ---- the block-scaled store ---------------------------------------------------------------

def rotated(pa, q, k, pos, cs, layout):
    """k as the bf16 store leaves it (checked on its own above), for the codes to come from."""
    T, kv = k.shape[0], k.shape[1]
    kc = torch.zeros(((T + B - 1) // B, kv, B, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    out = torch.empty_like(q)
    pa.rope_kv_store_form(q, k, k, pos, cs, torch.arange(T, device="cuda"), kc, vc, layout=layout, q_out=out)
    return out, f64(kc.permute(0, 2, 1, 3).reshape(-1, kv, D)[:T])


def check_block_store(pa, pool, q, k, v, pos, slots, cs, layout="half"):
    kc, vc, sc = pool.dev()
    qd, kd, vd = bf16(q), bf16(k), bf16(v)
    out = torch.empty_like(qd)
    ref_q, kr = rotated(pa, qd, kd, up(pos), up(cs), layout)
    pa.rope_kv_store_fp8_block(qd, kd, vd, up(pos), up(cs), up(slots), kc, vc, sc, layout=layout, q_out=out)
    assert np.array_equal(bits(out), bits(ref_q))
    want_k, sk = R.store(pool.k, pool.scale[..., 0].copy(), kr, slots)
    want_v, sv = R.store(pool.v, pool.scale[..., 1].copy(), f64(vd), slots)
    assert np.array_equal(sc.cpu().numpy(), np.stack([sk, sv], axis=2).astype(np.float32))
    for got, want in ((kc, want_k), (vc, want_v)):
        got = got.cpu().numpy()
        same = (got == want) | (((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F))     # NaN of either sign
        assert same.all(), np.argwhere(~same)[:5]
    return kc, vc, sc


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lens,hq,kv,Rr", [
    ([(0, 1)], 4, 4, 128), ([(5, 1), (16, 1), (31, 1), (0, 1)], 12, 2, 128), ([(3, 50), (0, 33), (16, 16), (30, 3)], 8, 1, 48),
    ([(7, 700), (0, 900)], 5, 1, 96), ([(i % 40, 1 + i % 3) for i in range(400)], 6, 3, 64)])
def test_block_store(pa, layout, lens, hq, kv, Rr):
    rng = np.random.default_rng(len(lens) * 7 + Rr)
    pool = Pool(rng, [c + n for c, n in lens], kv)
    T = sum(n for _, n in lens)
    pos = np.concatenate([np.arange(c, c + n) for c, n in lens]).astype(np.int32)
    seq = np.repeat(np.arange(len(lens)), [n for _, n in lens])
    slots = pool.tables[seq, pos // B].astype(np.int64) * B + pos % B
    k, v = normal(rng, T, kv, D, spread=1.5), normal(rng, T, kv, D, spread=1.5)
    check_block_store(pa, pool, normal(rng, T, hq, D), k, v, pos, slots, table_of(1000, Rr), layout)
    clean(pa)


def test_block_store_with_padding_rows_between(pa):
    rng = np.random.default_rng(8)
    pool = Pool(rng, [200], 2)
    T = 600
    slots = np.full(T, -1, np.int64)
    t = 3
    for p in range(20, 180):                        # up to 15 padding rows between the rows of a block
        slots[t] = pool.tables[0, p // B] * B + p % B
        t += 1 + (rng.integers(0, 6) if p % 16 else 15)
        if p % 37 == 0:
            t += 9
        if t >= T:
            break
    pos = rng.integers(0, 200, T).astype(np.int32)
    check_block_store(pa, pool, normal(rng, T, 4, D), normal(rng, T, 2, D), normal(rng, T, 2, D), pos, slots,
                      table_of(200, 128))
    clean(pa)


def test_block_store_of_extreme_values(pa):
    rng = np.random.default_rng(9)
    pool = Pool(rng, [16 * 8], 1, canary=False)
    rows = np.zeros((8, 1, D))
    rows[0] = 0.0
    rows[1] = R.bf16_round(rng.standard_normal(D)) * 2.0 ** -60
    rows[2] = R.bf16_round(rng.standard_normal(D)) * 2.0 ** 100
    rows[3, 0, :3] = [np.inf, -np.inf, 1.0]
    rows[4, 0, :3] = [np.nan, 2.0, -3.0]
    rows[5] = 448.0
    rows[6] = 450.0
    rows[7, 0, 5] = -2.0 ** 49
    cs = np.concatenate([np.ones((1, 64)), np.zeros((1, 64))], axis=1).astype(np.float32)   # angle 0: k as it is
    for off in (0, 3):                               # beginning a block, and growing (or keeping) its scale
        slots = pool.tables[0].astype(np.int64) * B + off
        kc, vc, sc = pool.dev()
        x = bf16(rows)
        pa.rope_kv_store_fp8_block(bf16(np.zeros((8, 1, D))), x, x, up(np.zeros(8, np.int32)), up(cs), up(slots), kc, vc, sc)
        for j, (got, held) in enumerate(((kc, pool.k), (vc, pool.v))):
            want, s = R.store(held, pool.scale[..., j].copy(), rows, slots)
            assert np.array_equal(sc.cpu().numpy()[..., j], s.astype(np.float32))
            got = got.cpu().numpy()
            blk = pool.tables[0]
            if j == 0:      # x cos - y sin of an infinity or a NaN is NaN beside a zero sine: rows 3, 4 only for V
                keep = np.ones(8, bool)
                keep[[3, 4]] = False
                blk = blk[keep]
            a, b = got[blk], want[blk]
            assert ((a == b) | (((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F)) | (((a | b) & 0x7F) == 0)).all()
    clean(pa)


def test_block_store_token_by_token_equals_the_reference(pa):
    """Appending with growing and shrinking magnitudes: scales only grow inside a block."""
    rng = np.random.default_rng(10)
    pool = Pool(rng, [40], 2)
    kc, vc, sc = pool.dev()
    cs = up(table_of(40, 128))
    k_ref, v_ref, s_ref = pool.k, pool.v, pool.scale.copy()
    for p in range(5, 40):
        k, v = (bf16(normal(rng, 1, 2, D) * 2.0 ** int(rng.integers(-9, 9))) for _ in range(2))
        pos, slot = np.array([p], np.int32), np.array([int(pool.tables[0, p // B]) * B + p % B], np.int64)
        q = bf16(np.zeros((1, 4, D)))
        _, kr = rotated(pa, q, k, up(pos), cs, "half")
        pa.rope_kv_store_fp8_block(q, k, v, up(pos), cs, up(slot), kc, vc, sc)
        k_ref, sk = R.store(k_ref, s_ref[..., 0].copy(), kr, slot)
        v_ref, sv = R.store(v_ref, s_ref[..., 1].copy(), f64(v), slot)
        s_ref = np.stack([sk, sv], axis=2).astype(np.float32)
    assert np.array_equal(sc.cpu().numpy(), s_ref)
    for got, want in ((kc, k_ref), (vc, v_ref)):
        got = got.cpu().numpy()
        assert ((got == want) | (((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F))).all()


# ---- decode -------------------------------------------------------------------------------

EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 255, 256, 257, 1000]


@pytest.mark.parametrize("hq,kv", [(12, 2), (8, 8), (64, 8), (5, 1), (9, 3)])
@pytest.mark.parametrize("P", [0, 16, 256])
def test_decode(pa, hq, kv, P):
    rng = np.random.default_rng(hq + P)
    pool = Pool(rng, EDGES, kv)
    q = normal(rng, len(EDGES), hq, D)
    kc, vc, sc = pool.dev()
    out = pa.decode_fp8_block(bf16(q), kc, vc, sc, up(pool.tables), up(pool.lens), 1000, D ** -0.5, partition_tokens=P)
    for s in range(len(EDGES)):
        ref, mag = pool.attention(s, q[s:s + 1], D ** -0.5)
        close(out[s:s + 1], ref, mag, (s, EDGES[s]))
    clean(pa)


@pytest.mark.parametrize("S,n", [(1, 1), (1, 5000), (300, 70), (2, 40000)])
def test_decode_sizes(pa, S, n):
    rng = np.random.default_rng(S)
    lens = [int(x) for x in rng.integers(max(1, n // 3), n + 1, S)]
    pool = Pool(rng, lens, 2)
    q = normal(rng, S, 12, D)
    kc, vc, sc = pool.dev()
    out = pa.decode_fp8_block(bf16(q), kc, vc, sc, up(pool.tables), up(pool.lens), max(lens), D ** -0.5)
    for s in range(0, S, max(1, S // 12)):
        ref, mag = pool.attention(s, q[s:s + 1], D ** -0.5)
        close(out[s:s + 1], ref, mag, s)
    clean(pa)


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("S,hq,kv", [(3, 12, 2), (40, 12, 2), (64, 10, 2), (700, 8, 1)])
def test_decode_one_long_sequence_among_short_ones(pa, S, hq, kv, P):
    """Hundreds of pieces in one sequence and one in the others, in each form of the merge."""
    rng = np.random.default_rng(S + P)
    lens = [6000] + [int(x) for x in rng.integers(0, 40, S - 1)]
    pool = Pool(rng, lens, kv)
    q = normal(rng, S, hq, D)
    out = pa.decode_fp8_block(bf16(q), *pool.dev(), up(pool.tables), up(pool.lens), 6000, D ** -0.5, partition_tokens=P)
    for s in range(0, S, max(1, S // 12)):
        ref, mag = pool.attention(s, q[s:s + 1], D ** -0.5)
        close(out[s:s + 1], ref, mag, s)
    assert not f64(out[torch.from_numpy(np.array(lens) == 0).cuda()]).any()
    clean(pa)


def test_decode_scales_far_apart_and_of_any_value(pa):
    """Blocks whose V scale is 2^-40 (zeros) carry most of the weight; scales that are no powers of
    two; K scales that make scores large."""
    rng = np.random.default_rng(11)
    pool = Pool(rng, [200, 350], 2)
    q = normal(rng, 2, 12, D)
    pool.scale[:] = rng.uniform(2.0 ** -9, 2.0 ** -6, pool.scale.shape)
    sink = pool.tables[:, 0]
    pool.v[sink] = 0
    pool.scale[sink, :, 1] = 2.0 ** -40
    pool.k[sink, :, 0] = R.e4m3_encode(20 * q[:, ::6][:, :2])      # the first token scores high
    pool.scale[sink, :, 0] = 2.0 ** -4
    pool.scale[pool.tables[0, 3], :, 1] = 2.0 ** 40
    kc, vc, sc = pool.dev()
    out = pa.decode_fp8_block(bf16(q), kc, vc, sc, up(pool.tables), up(pool.lens), 350, D ** -0.5)
    for s in range(2):
        ref, mag = pool.attention(s, q[s:s + 1], D ** -0.5)
        close(out[s:s + 1], ref, mag, s)
    clean(pa)


def test_decode_bad_blocks_and_lengths_are_skipped(pa):
    rng = np.random.default_rng(12)
    pool = Pool(rng, [64, 64], 2, canary=False)
    tables = pool.tables.copy()
    tables[0, 1], tables[1, 2] = -3, pool.nb
    q = normal(rng, 2, 4, D)
    kc, vc, sc = pool.dev()
    out = pa.decode_fp8_block(bf16(q), kc, vc, sc, up(tables), up(pool.lens), 64, D ** -0.5)
    keep = [[0, 2, 3], [0, 1, 3]]
    for s in range(2):
        ref, mag = R.attention(q[s:s + 1], pool.k, pool.v, pool.scale, tables[s][keep[s]], 48, D ** -0.5)
        close(out[s:s + 1], ref, mag, s)
    clean(pa, pa.PA_FLAG_BLOCK_ID_OOB)
    pa.decode_fp8_block(bf16(q), kc, vc, sc, up(pool.tables), up(np.array([64, 65], np.int32)), 64, D ** -0.5)
    clean(pa, pa.PA_FLAG_CONTEXT_LEN_OOB)


def test_decode_is_reproducible_and_leaves_other_streams_alone(pa):
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(1, 3000, 40)]
    pool = Pool(rng, lens, 2)
    q = bf16(normal(rng, 40, 12, D))
    kc, vc, sc = pool.dev()
    args = (q, kc, vc, sc, up(pool.tables), up(pool.lens), max(lens), D ** -0.5)
    first = pa.decode_fp8_block(*args)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    second = pa.decode_fp8_block(*args, stream=st)
    st.synchronize()
    assert np.array_equal(bits(first), bits(second))


def test_two_streams_at_once_and_two_graphs_over_one_workspace(pa):
    """Calls in flight together on streams of their own, and two captured graphs that share a workspace
    and are replayed in turn: the bits of a lone call."""
    rng = np.random.default_rng(14)
    jobs = []
    for S, hq, kv, n in ((40, 12, 2, 2500), (3, 28, 4, 6000)):
        lens = [int(x) for x in rng.integers(n // 2, n, S)]
        pool = Pool(rng, lens, kv)
        q = bf16(normal(rng, S, hq, D))
        args = (*pool.dev(), up(pool.tables), up(pool.lens))
        jobs.append((q, args, max(lens), up(np.arange(S + 1, dtype=np.int32))))
    ws = max((pa.decode_workspace(q, a[0], n) for q, a, n, _ in jobs), key=lambda t: t.numel())

    def decode(job, out, **kw):
        q, a, n, _ = job
        return pa.decode_fp8_block(q, *a, n, D ** -0.5, out=out, **kw)

    def prefill(job, out, **kw):
        q, a, n, starts = job
        return pa.prefill_fp8_block(q, starts, *a, 1, n, D ** -0.5, out=out, **kw)

    alone = [[bits(call(job, torch.empty_like(job[0]))) for call in (decode, prefill)] for job in jobs]
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [torch.empty_like(job[0]) for job in jobs for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            (prefill if i % 2 else decode)(jobs[i // 2], outs[i], stream=st)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert np.array_equal(bits(o), alone[i // 2][i % 2]), i
    graphs = []
    for job, out in zip(jobs, outs[::2]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            decode(job, out, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for i, g in enumerate(graphs):
            outs[2 * i].zero_()
            g.replay()
            assert np.array_equal(bits(outs[2 * i]), alone[i][0])
    clean(pa)


def test_many_sequences(pa):
    """The most sequences a call takes: their prefix leaves fewer stages, and so fewer warps, to a CTA."""
    rng = np.random.default_rng(40)
    S = 8192
    lens = [int(x) for x in rng.integers(0, 40, S)]
    pool = Pool(rng, lens, 1)
    q = normal(rng, S, 8, D)
    args = (*pool.dev(), up(pool.tables), up(pool.lens), 40, D ** -0.5)
    out = pa.decode_fp8_block(bf16(q), *args)
    for s in list(range(0, S, 401)) + [S - 1]:
        ref, mag = pool.attention(s, q[s:s + 1], D ** -0.5)
        close(out[s:s + 1], ref, mag, s)
    assert not f64(out[torch.from_numpy(np.array(lens) == 0).cuda()]).any()
    clean(pa)


def test_a_cache_past_four_gigabytes(pa):
    """Tiles and scales whose offsets do not fit 32 bits: the store, the decode and the prefill at the far end."""
    rng = np.random.default_rng(41)
    kv, nb = 8, 290_000                                   # 4.75 GB of codes each for K and V
    kc, vc = (torch.empty((nb, kv, B, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.empty((nb, kv, 2), device="cuda")
    table = np.array([[nb - 1, 3, nb - 7]], np.int32)
    T = 40
    q, k, v = (bf16(normal(rng, T, h, D)) for h in (16, kv, kv))
    pos = np.arange(T, dtype=np.int32)
    slots = table[0, pos // B].astype(np.int64) * B + pos % B
    q2 = pa.rope_kv_store_fp8_block(q, k, v, up(pos), up(table_of(64, 128)), up(slots), kc, vc, sc, q_out=torch.empty_like(q))
    blocks = torch.from_numpy(table[0].astype(np.int64)).cuda()
    small = [t[blocks].cpu().numpy() for t in (kc, vc, sc)]
    args = (kc, vc, sc, up(table), up(np.array([T], np.int32)))
    out = pa.prefill_fp8_block(q2, up(np.array([0, T], np.int32)), *args, T, T, D ** -0.5)
    ref, mag = R.attention(f64(q2), *small, np.arange(3), T, D ** -0.5, 0)
    close(out, ref, mag)
    one = pa.decode_fp8_block(q2[-1:].contiguous(), *args, T, D ** -0.5)
    close(one, ref[-1:], mag[-1:])
    clean(pa)


def test_a_query_that_is_not_finite_spoils_its_own_head_only(pa):
    rng = np.random.default_rng(42)
    pool = Pool(rng, [300, 40], 2)
    q = normal(rng, 2, 12, D)
    q[0, 3, 5], q[1, 7, 9] = np.inf, np.nan
    out = pa.decode_fp8_block(bf16(q), *pool.dev(), up(pool.tables), up(pool.lens), 300, D ** -0.5)
    pre = pa.prefill_fp8_block(bf16(q), up(np.array([0, 1, 2], np.int32)), *pool.dev(), up(pool.tables), up(pool.lens), 1, 300,
                               D ** -0.5)
    bad = {(0, 3), (1, 7)}
    for s in range(2):
        clean_q = np.where(np.isfinite(q[s:s + 1]), q[s:s + 1], 0.0)
        ref, mag = pool.attention(s, clean_q, D ** -0.5)
        for h in range(12):
            for o in (out, pre):
                if (s, h) in bad:
                    assert np.isnan(f64(o[s, h])).all()
                else:
                    close(f64(o[s, h]), ref[0, h], mag[0, h], (s, h))
    clean(pa)


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 15, 2.0 ** 60])
def test_queries_of_any_magnitude(pa, size):
    """A power of two on q and its inverse on the softmax scale: the same attention, whatever f16 or
    E4M3 could hold."""
    rng = np.random.default_rng(43)
    pool = Pool(rng, [200], 1)
    q = normal(rng, 1, 8, D)
    out = pa.decode_fp8_block(bf16(q * size), *pool.dev(), up(pool.tables), up(pool.lens), 200, D ** -0.5 / size)
    pre = pa.prefill_fp8_block(bf16(q * size), up(np.array([0, 1], np.int32)), *pool.dev(), up(pool.tables), up(pool.lens), 1,
                               200, D ** -0.5 / size)
    ref, mag = pool.attention(0, q, D ** -0.5)
    close(out, ref, mag)
    close(pre, ref, mag)
    clean(pa)


def test_shapes_that_do_not_fit_are_refused(pa):
    e = dict(device="cuda")
    bf = dict(dtype=torch.bfloat16, **e)
    q, k = torch.zeros((4, 12, D), **bf), torch.zeros((4, 2, D), **bf)
    kc, vc = (torch.zeros((4, 2, B, D), dtype=torch.uint8, **e) for _ in range(2))
    sc, cs = torch.ones((4, 2, 2), **e), torch.zeros((8, 64), **e)
    i32, i64, bt = (torch.zeros(s, dtype=t, **e) for s, t in ((4, torch.int32), (4, torch.int64), ((4, 2), torch.int32)))
    ws = torch.zeros(1 << 16, **e)
    qs = torch.zeros(5, dtype=torch.int32, **e)
    nf, plan = i32[:1].contiguous(), pa.step_plan(4, 5)
    store = dict(q=q, k=k, v=k, positions=i32, cos_sin=cs, slot_mapping=i64, k_cache=kc, v_cache=vc, kv_scale=sc)
    dec = dict(q=q, k_cache=kc, v_cache=vc, kv_scale=sc, block_tables=bt, context_lens=i32, max_context_len=16, scale=0.1,
               workspace=ws)
    step = dict(dec, k=k, v=k, cos_sin=cs)
    pre = dict(q=q, q_start=qs, k_cache=kc, v_cache=vc, kv_scale=sc, block_tables=bt, context_lens=i32, max_query_len=4,
               max_context_len=16, scale=0.1)
    pl = dict(cached_lens=i32, new_lens=i32, block_tables=bt, free_blocks=i32, num_free=nf, num_blocks=4, num_tokens=5,
              plan=plan)
    wide = torch.zeros((4, 2, 2 * D), **bf)[:, :, ::2]
    for call, good, bad in (
            (pa.rope_kv_store_fp8_block, store, dict(k=k[:3], v=q, positions=i32[:3], slot_mapping=i64[:3], cos_sin=cs[0],
                                                     k_cache=kc[:3], kv_scale=sc[:3], q_out=q[:3], q=q[0])),
            (pa.decode_fp8_block, dec, dict(q=q[:3], block_tables=bt[0], context_lens=i32[:2], out=q[:1], kv_scale=sc[:, :1])),
            (pa.decode_step_fp8_block, step, dict(k=k[:3], v=q, cos_sin=cs[0], out=q[:3], v_cache=vc[:2])),
            (pa.prefill_fp8_block, pre, dict(q_start=qs[:4], block_tables=bt[:3], context_lens=i32[:3], out=q[:3])),
            (pa.plan_step, pl, dict(new_lens=i32[:3], block_tables=bt[:3], num_free=i32[:2], num_tokens=6, free_blocks=bt))):
        for name, value in bad.items():
            with pytest.raises(ValueError):
                call(**dict(good, **{name: value}))
    with pytest.raises(ValueError, match="contiguous"):
        pa.rope_kv_store_fp8_block(**dict(store, k=wide))
    with pytest.raises(pa.PaError):                       # what the library refuses
        pa.decode_fp8_block(**dict(dec, max_context_len=33))
    clean(pa)


def test_nothing_to_do(pa):
    e = dict(device="cuda")
    kc, vc = (torch.zeros((2, 1, B, D), dtype=torch.uint8, **e) for _ in range(2))
    sc, cs = torch.ones((2, 1, 2), **e), torch.zeros((4, 64), **e)
    q, k = torch.zeros((0, 4, D), dtype=torch.bfloat16, **e), torch.zeros((0, 1, D), dtype=torch.bfloat16, **e)
    i32, i64 = torch.zeros(0, dtype=torch.int32, **e), torch.zeros(0, dtype=torch.int64, **e)
    bt = torch.zeros((0, 2), dtype=torch.int32, **e)
    assert pa.decode_fp8_block(q, kc, vc, sc, bt, i32, 16, 0.1).shape == q.shape
    assert pa.decode_step_fp8_block(q, k, k, cs, kc, vc, sc, bt, i32, 16, 0.1).shape == q.shape
    assert pa.rope_kv_store_fp8_block(q, k, k, i32, cs, i64, kc, vc, sc) is q
    assert pa.prefill_fp8_block(q, torch.zeros(1, dtype=torch.int32, **e), kc, vc, sc, bt, i32, 1, 16, 0.1).shape == q.shape
    clean(pa)


# ---- the fused step -----------------------------------------------------------------------

@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("layout,Rr", [("half", 128), ("half", 96), ("half", 48), ("interleaved", 128), ("interleaved", 16)])
def test_step_equals_store_then_decode(pa, layout, Rr, early):
    rng = np.random.default_rng(Rr)
    lens = [1, 2, 16, 17, 33, 100, 999, 0, 48, 64, 65]
    pool = Pool(rng, lens, 2)
    S = len(lens)
    q, k, v = bf16(normal(rng, S, 12, D)), bf16(normal(rng, S, 2, D, spread=2.0)), bf16(normal(rng, S, 2, D, spread=2.0))
    cs, bt, ctx = up(table_of(1000, Rr)), up(pool.tables), up(pool.lens)
    a, b = pool.dev(), pool.dev()
    out = pa.decode_step_fp8_block(q, k, v, cs, *a, bt, ctx, 999, D ** -0.5, layout=layout, early_metadata=early)
    pos = np.maximum(pool.lens - 1, 0)
    slots = np.where(pool.lens > 0, pool.tables[np.arange(S), pos // B].astype(np.int64) * B + pos % B, -1)
    q2 = torch.empty_like(q)
    pa.rope_kv_store_fp8_block(q, k, v, up(pos.astype(np.int32)), cs, up(slots), *b, layout=layout, q_out=q2)
    two = pa.decode_fp8_block(q2, *b, bt, ctx, 999, D ** -0.5)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert np.array_equal(bits(out), bits(two))
    # and against the reference over the caches as stored
    pool.k, pool.v, pool.scale = (t.cpu().numpy() for t in a)
    qr = f64(q2)
    for s in range(S):
        ref, mag = pool.attention(s, qr[s:s + 1], D ** -0.5)
        close(out[s:s + 1], ref, mag, s)
    clean(pa)


@pytest.mark.parametrize("S,hq,kv,P", [(200, 8, 1, 0), (200, 16, 4, 0), (40, 21, 3, 32), (1500, 5, 1, 0), (6, 64, 8, 0)])
def test_step_cuts_sequences_as_the_decode_does(pa, S, hq, kv, P):
    """Stages of another size, the same pieces: the bits of store and decode for any group and batch."""
    rng = np.random.default_rng(S + hq)
    lens = [int(x) for x in rng.integers(0, 60000 // S, S)]
    pool = Pool(rng, lens, kv)
    q, k, v = (bf16(normal(rng, S, h, D)) for h in (hq, kv, kv))
    n = max(lens)
    cs, bt, ctx = up(table_of(n, 64)), up(pool.tables), up(pool.lens)
    a, b = pool.dev(), pool.dev()
    out = pa.decode_step_fp8_block(q, k, v, cs, *a, bt, ctx, n, D ** -0.5, partition_tokens=P)
    pos = np.maximum(pool.lens - 1, 0)
    slots = np.where(pool.lens > 0, pool.tables[np.arange(S), pos // B].astype(np.int64) * B + pos % B, -1)
    q2 = torch.empty_like(q)
    pa.rope_kv_store_fp8_block(q, k, v, up(pos.astype(np.int32)), cs, up(slots), *b, q_out=q2)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert np.array_equal(bits(out), bits(pa.decode_fp8_block(q2, *b, bt, ctx, n, D ** -0.5, partition_tokens=P)))
    clean(pa)


def test_step_without_a_row_of_the_table_stores_nothing(pa):
    rng = np.random.default_rng(14)
    pool = Pool(rng, [20, 40], 2, canary=False)
    q, k, v = (bf16(normal(rng, 2, h, D)) for h in (4, 2, 2))
    kc, vc, sc = pool.dev()
    out = pa.decode_step_fp8_block(q, k, v, up(table_of(30, 64)), kc, vc, sc, up(pool.tables), up(pool.lens), 40, D ** -0.5)
    blk = int(pool.tables[1, 2])
    assert np.array_equal(kc.cpu().numpy()[blk], pool.k[blk]) and np.array_equal(sc.cpu().numpy()[blk], pool.scale[blk])
    ref, mag = pool.attention(1, f64(q)[1:], D ** -0.5)
    close(out[1:], ref, mag)
    clean(pa, pa.PA_FLAG_POSITION_OOB)


# ---- prefill ------------------------------------------------------------------------------

def check_prefill(pa, rng, lens, new, hq, kv, spread=1.0, pool=None, max_new=None):
    pool = pool or Pool(rng, lens, kv, spread=spread)
    T = sum(new)
    q = normal(rng, T, hq, D)
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    kc, vc, sc = pool.dev()
    out = torch.full((T, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = pa.prefill_fp8_block(bf16(q), up(qs), kc, vc, sc, up(pool.tables), up(pool.lens), max_new or max(max(new), 1),
                               max(lens), D ** -0.5, out=out)
    assert got is out
    for s in range(len(lens)):
        if new[s]:
            ref, mag = pool.attention(s, q[qs[s]:qs[s + 1]], D ** -0.5, lens[s] - new[s])
            close(out[qs[s]:qs[s + 1]], ref, mag, s)
    clean(pa)
    return pool, out


@pytest.mark.parametrize("hq,kv", [(12, 2), (8, 8), (64, 8), (5, 1), (9, 3), (7, 1)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([17, 64, 65, 128], [17, 64, 65, 128]), ([300, 33, 200], [41, 1, 7]),
                                      ([16, 15, 500, 48], [0, 15, 130, 48])])
def test_prefill(pa, hq, kv, lens, new):
    check_prefill(pa, np.random.default_rng(hq + sum(new)), lens, new, hq, kv)


@pytest.mark.parametrize("lens,new", [([3000], [700]), ([9000, 40], [3, 40]), ([1200] * 9, [100] * 9)])
def test_prefill_long(pa, lens, new):
    check_prefill(pa, np.random.default_rng(len(lens)), lens, new, 12, 2)


@pytest.mark.parametrize("lens,new,hq,kv", [
    ([10812, 9000, 1, 4097], [1, 1, 1, 1], 28, 4), ([2000], [1], 8, 8), ([700, 130, 64, 900], [20, 130, 3, 40], 5, 1),
    ([5000], [64], 12, 2), ([1537, 1536, 1535], [16, 17, 15], 64, 8), ([20000, 17], [5, 17], 2, 1)])
def test_prefill_split_over_the_keys(pa, lens, new, hq, kv):
    """Few tiles over long contexts: a tile's keys are shared out over a cluster; sequences much
    shorter than the longest leave most of its CTAs without keys."""
    pool, out = check_prefill(pa, np.random.default_rng(sum(lens)), lens, new, hq, kv)
    q = bf16(normal(np.random.default_rng(1), sum(new), hq, D))
    args = (q, up(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), *pool.dev(), up(pool.tables), up(pool.lens),
            max(new), max(lens), D ** -0.5)
    assert np.array_equal(bits(pa.prefill_fp8_block(*args)), bits(pa.prefill_fp8_block(*args)))


@pytest.mark.parametrize("lens,new,hq,kv,seed,max_ns", [
    ([2048, 700, 1500], [2048, 300, 64], 12, 2, 1, 3000), ([9000, 777, 4100], [150, 40, 300], 12, 2, 2, 8000),
    ([10812, 9000, 1, 4097], [1, 1, 1, 1], 28, 4, 3, 8000), ([1200] * 9, [100] * 9, 8, 8, 4, 500)])
def test_prefill_under_timing_jitter_gives_the_same_bits(pa, lens, new, hq, kv, seed, max_ns):
    """Sleeps at every stage of every role: orders of arrival that undisturbed runs rarely take."""
    rng = np.random.default_rng(seed)
    pool = Pool(rng, lens, kv)
    q = bf16(normal(rng, sum(new), hq, D))
    args = (q, up(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), *pool.dev(), up(pool.tables), up(pool.lens),
            max(new), max(lens), D ** -0.5)
    want = bits(pa.prefill_fp8_block(*args))
    torch.cuda.synchronize()
    pa.set_timing_jitter(max_ns, seed)
    try:
        got = bits(pa.prefill_fp8_block(*args))
        torch.cuda.synchronize()
    finally:
        pa.set_timing_jitter(0)
    clean(pa)
    assert np.array_equal(got, want)


def test_prefill_bound_larger_than_needed_and_scales_far_apart(pa):
    rng = np.random.default_rng(30)
    pool = Pool(rng, [200, 350], 2)
    pool.scale[:] = rng.uniform(2.0 ** -9, 2.0 ** -6, pool.scale.shape)
    sink = pool.tables[:, 0]
    pool.v[sink] = 0
    pool.scale[sink, :, 1] = 2.0 ** -40
    pool.scale[sink, :, 0] = 2.0 ** -3
    pool.scale[pool.tables[0, 3], :, 1] = 2.0 ** 40
    check_prefill(pa, rng, [200, 350], [90, 350], 12, 2, pool=pool, max_new=350)


def test_prefill_is_the_decode_for_single_tokens(pa):
    rng = np.random.default_rng(31)
    lens = [1, 16, 17, 700]
    pool = Pool(rng, lens, 2)
    q = bf16(normal(rng, 4, 12, D))
    args = (*pool.dev(), up(pool.tables), up(pool.lens))
    one = pa.prefill_fp8_block(q, up(np.arange(5, dtype=np.int32)), *args, 1, 700, D ** -0.5)
    two = pa.decode_fp8_block(q, *args, 700, D ** -0.5)
    assert (np.abs(f64(one) - f64(two)) <= 2.0 ** -6 * np.abs(f64(two)) + 2.0 ** -9 * np.abs(f64(two)).max()).all()


def test_prefill_bad_blocks_and_sequences(pa):
    rng = np.random.default_rng(32)
    pool = Pool(rng, [200, 64, 40], 2, canary=False)
    tables = pool.tables.copy()
    tables[0, 1], tables[0, 4] = -3, pool.nb
    tables[2, :3] = -1
    q = normal(rng, 30 + 10 + 4, 12, D)
    qs = np.array([0, 30, 40, 44], np.int32)
    kc, vc, sc = pool.dev()
    out = pa.prefill_fp8_block(bf16(q), up(qs), kc, vc, sc, up(tables), up(pool.lens), 30, 200, D ** -0.5)
    keep = [b for b in range(13) if b not in (1, 4)]
    k, v = pool.k[tables[0, keep]], pool.v[tables[0, keep]]
    ref, mag = R.attention(q[:30], k, v, pool.scale[tables[0, keep]], np.arange(len(keep)), 200 - 32, D ** -0.5, 200 - 32 - 30)
    close(out[:30], ref, mag)
    ref, mag = pool.attention(1, q[30:40], D ** -0.5, 54)
    close(out[30:40], ref, mag)
    assert (f64(out[40:]) == 0).all()                                       # every block out of range
    clean(pa, pa.PA_FLAG_BLOCK_ID_OOB)
    # a sequence whose lengths are out of order is skipped, the others are not
    out.fill_(7.0)
    pa.prefill_fp8_block(bf16(q), up(qs), kc, vc, sc, up(pool.tables), up(np.array([200, 9, 40], np.int32)), 30, 200,
                         D ** -0.5, out=out)
    assert (f64(out[30:40]) == 7).all()
    ref, mag = pool.attention(0, q[:30], D ** -0.5, 170)
    close(out[:30], ref, mag)
    clean(pa, pa.PA_FLAG_CONTEXT_LEN_OOB)


def test_prefill_rows_past_the_last_sequence_stay(pa):
    rng = np.random.default_rng(33)
    pool = Pool(rng, [40], 2)
    q = bf16(normal(rng, 24, 4, D))
    out = torch.full_like(q, 5.0)
    pa.prefill_fp8_block(q, up(np.array([0, 20], np.int32)), *pool.dev(), up(pool.tables), up(pool.lens), 20, 40, D ** -0.5,
                         out=out)
    assert (f64(out[20:]) == 5).all() and not (f64(out[:20]) == 5).all()
    clean(pa)


# ---- plans --------------------------------------------------------------------------------

FLAG = {"block": 1, "len": 2, "pool": 0x20}


def check_plan(pa, cached, new, tables, free, num_free, num_blocks, T, in_place=False):
    ref, flags = R.plan(cached, new, tables, free, num_free, num_blocks, T)
    bt = up(tables)
    nf = up(np.array([num_free], np.int32))
    nfo = nf if in_place else torch.full((1,), -77, dtype=torch.int32, device="cuda")
    p = pa.step_plan(len(cached), T)
    for t in p:
        t.fill_(-99)
    got = pa.plan_step(up(np.array(cached, np.int32)), up(np.array(new, np.int32)), bt, up(np.array(free, np.int32)), nf,
                       num_blocks, T, num_free_out=None if in_place else nfo, plan=p)
    torch.cuda.synchronize()
    for name in p._fields:
        assert np.array_equal(getattr(got, name).cpu().numpy(), ref[name]), name
    assert np.array_equal(bt.cpu().numpy(), ref["tables"]) and int(nfo[0]) == ref["num_free"]
    clean(pa, sum(FLAG[f] for f in flags))


def random_plan(rng, S, cached, new, short=False, pad=0):
    c, n = rng.integers(0, cached + 1, S), rng.integers(0, new + 1, S)
    have = -(-c // B)
    need = -(-(c + n) // B) - have
    width = max(1, int((have + need).max())) if S else 1
    free = max(1, int(need.sum()) * 2 // 3) if short else int(need.sum()) + 5
    nb = int(have.sum()) + free
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((S, width), -1, np.int32)
    at = 0
    for s in range(S):
        tables[s, :have[s]] = perm[at:at + have[s]]
        at += have[s]
    return c, n, tables, perm[at:], free, nb, int(n.sum()) + pad


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,cached,new,short,pad", [(1, 0, 1, False, 0), (1, 100, 40, False, 3), (33, 50, 1, False, 7), (256, 4000, 2, True, 1),
                                                    (64, 500, 300, True, 0), (700, 30, 60, False, 5), (1500, 20, 5, True, 2),
                                                    (8192, 40, 3, False, 9), (300, 64, 2400, False, 6), (2000, 64, 380, True, 1)])
def test_plan(pa, S, cached, new, short, pad, in_place):
    check_plan(pa, *random_plan(np.random.default_rng(S + new), S, cached, new, short, pad), in_place=in_place)


def test_plan_of_nothing(pa):
    for S, T in ((0, 0), (0, 5), (3, 0), (3, 4)):
        check_plan(pa, [7] * S, [0] * S, np.full((S, 2), 1, np.int32), [0, 1], 2, 4, T)


def test_plan_errors_are_refused_one_by_one(pa):
    t = np.array([[0, -1, -1], [1, 99, -1], [2, 3, -1], [4, -1, -1], [-1] * 3, [5, -1, -1]], np.int32)
    free = [10, 11, 12, 77, -4, 13]
    for cached, new, T in (([16, 20, 32, 3, -1, 16], [1, 3, 1, 40, 4, 2], 60),     # a bad id, a bad length, ids out of the pool
                           ([16, 16, 32, 16, 0, 16], [1, -2, 1, 17, 16, 1], 20),   # a negative count, rows past the end
                           ([16, 16, 32, 16, 0, 16], [1, 2**31 - 1, 1, 1, 1, 1], 9),
                           ([2**31 - 1, 16, 32, 16, 0, 16], [5, 1, 1, 1, 1, 1], 12)):
        for F in (6, 3, 0, -2, 9):
            check_plan(pa, cached, new, t, free, F, 20, T)


# ---- a serving loop -----------------------------------------------------------------------

def test_a_serving_loop_of_plan_store_attention(pa):
    """Prompts and their continuation: plan -> store -> prefill, then captured steps of plan ->
    fused step, replayed; everything against the reference over the caches as they stand."""
    rng = np.random.default_rng(20)
    S, hq, kv, nb, width = 5, 12, 2, 60, 12
    scale = D ** -0.5
    cs = pa.rope_table(256, 64, 1e4, scaling="linear", factor=2.0)
    tables = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    free, nf = up(rng.permutation(nb).astype(np.int32)), up(np.array([nb], np.int32))
    kc, vc = (torch.full((nb, kv, B, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.full((nb, kv, 2), float("nan"), device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    for new in ([17, 40, 1, 64, 30], [30, 1, 25, 3, 0]):                 # two chunks of prompts
        n = up(np.array(new, np.int32))
        T = sum(new)
        p = pa.plan_step(lens, n, tables, free, nf, nb, T)
        q, k, v = (bf16(normal(rng, T, h, D)) for h in (hq, kv, kv))
        pa.rope_kv_store_fp8_block(q, k, v, p.positions, cs, p.slot_mapping, kc, vc, sc, layout="interleaved")
        out = pa.prefill_fp8_block(q, p.q_start, kc, vc, sc, tables, p.context_lens, max(new), width * B, scale)
        ref_k, ref_v, ref_s, bt = kc.cpu().numpy(), vc.cpu().numpy(), sc.cpu().numpy(), tables.cpu().numpy()
        ctx, qs = p.context_lens.tolist(), p.q_start.tolist()
        for s in range(S):
            if new[s]:
                ref, mag = R.attention(f64(q[qs[s]:qs[s + 1]]), ref_k, ref_v, ref_s, bt[s], ctx[s], scale, ctx[s] - new[s])
                close(out[qs[s]:qs[s + 1]], ref, mag, s)
        lens.copy_(p.context_lens)
    clean(pa)
    # decode steps, captured once: lengths, tables and the free list live on the GPU
    one = torch.ones(S, dtype=torch.int32, device="cuda")
    plan = pa.step_plan(S, S)
    q, k, v = (torch.zeros((S, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, kv, kv))
    out = torch.empty_like(q)
    ws = pa.decode_workspace(q, kc, width * B)

    def step():
        pa.plan_step(lens, one, tables, free, nf, nb, S, plan=plan)
        pa.decode_step_fp8_block(q, k, v, cs, kc, vc, sc, tables, plan.context_lens, width * B, scale, layout="interleaved",
                                 workspace=ws, out=out)
        lens.copy_(plan.context_lens)

    state = [t.clone() for t in (lens, tables, nf, kc, vc, sc)]
    step()                                                               # warm, then back to where it was
    for t, x in zip((lens, tables, nf, kc, vc, sc), state):
        t.copy_(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        for t in (q, k, v):
            t.copy_(bf16(normal(rng, *t.shape)))
        before = lens.tolist()
        graph.replay()
        assert lens.tolist() == [n + 1 for n in before]
        q2 = torch.empty_like(q)
        junk = [t.clone() for t in (kc, vc, sc)]
        pos = lens - 1
        pa.rope_kv_store_fp8_block(q, k, v, pos, cs, torch.full((S,), -1, dtype=torch.int64, device="cuda"), *junk,
                                   layout="interleaved", q_out=q2)
        rk, rv, rs, bt = kc.cpu().numpy(), vc.cpu().numpy(), sc.cpu().numpy(), tables.cpu().numpy()
        for s in range(S):
            ref, mag = R.attention(f64(q2[s:s + 1]), rk, rv, rs, bt[s], before[s] + 1, scale)
            close(out[s:s + 1], ref, mag, (i, s))
    used = sum(-(-n // B) for n in lens.tolist())
    assert int(nf[0]) == nb - used
    held = sorted(int(b) for s, n in enumerate(lens.tolist()) for b in tables[s, : -(-n // B)].tolist())
    assert sorted(held + free[: int(nf[0])].tolist()) == list(range(nb))    # every block once
    clean(pa)
