"""The 4-bit cache's attention where test_gpu_int4 does not go: slots that nothing was stored in, scores far from zero, warps that go
through many blocks, small elements of q, bounds near 2^31.

Tolerances are those of test_gpu_int4 (`close`), derived there.  Scores here are exact in fp32 where they are large: q has
powers of two and small multiples of 1/2 in two dims, K small integers, and the softmax scale is the number whose product
with log2 e rounds to 1, so that a rounding of the score itself is in no bound.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import int4_ref as R
import serving_ref as S
from test_gpu_int4 import B, D, Pool, bf16, bits, clean, close, f64, normal, pa, table_of, up  # noqa: F401

pytestmark = pytest.mark.gpu


def unit_scale() -> float:
    """The fp32 number whose fp32 product with log2 e is 1."""
    x = np.float32(np.log(2.0))
    for c in (x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(1))):
        if np.float32(c) * np.float32(1.4426950408889634) == np.float32(1.0):
            return float(c)
    raise AssertionError


# ---- slots that nothing was stored in ------------------------------------------------------

def test_slots_never_stored_read_as_zeros(pa):
    """A cleared cache holds zeros: a token within the context whose slot nothing was stored in counts with a score and a
    value of 0, in every call."""
    rng = np.random.default_rng(40)
    lens, kv, hq = [40, 16, 1, 700, 33], 2, 12
    p = Pool(rng, lens, kv, canary=False)
    p.cache[:] = 0
    cs = np.concatenate([np.ones((1, 64)), np.zeros((1, 64))], axis=1).astype(np.float32)
    cache, slots = up(p.cache), []
    for s, n in enumerate(lens):                            # sequence 1 has nothing stored, the others a part
        for t in range(n):
            if s != 1 and rng.random() < 0.6:
                slots.append(p.tables[s, t // B] * B + t % B)
    T = len(slots)
    rows = normal(rng, 2, T, kv, D, spread=1.0)
    pa.rope_kv_store_int4(bf16(normal(rng, T, hq, D)), bf16(rows[0]), bf16(rows[1]), torch.zeros(T, dtype=torch.int32, device="cuda"),
                          up(cs), up(np.array(slots, np.int64)), cache)
    p.cache = cache.cpu().numpy()
    q = normal(rng, len(lens), hq, D)
    starts = up(np.arange(len(lens) + 1, dtype=np.int32))
    dec = pa.decode_int4(bf16(q), cache, up(p.tables), up(p.lens), 700, 0.1)
    pre = pa.prefill_int4(bf16(q), starts, cache, up(p.tables), up(p.lens), 1, 700, 0.1)
    for s, n in enumerate(lens):
        ref = p.attention(s, q[s:s + 1], 0.1)
        close(pre[s:s + 1], ref, ("prefill", s), prefill=True)
        close(dec[s:s + 1], ref, ("decode", s), steps=n // 16 + 1)
    k, v = pa.read_kv_int4(cache, up(np.array([0, 16], np.int32)), None, up(p.tables[1:2]), 16, num_rows=16)
    assert (f64(k) == 0).all() and (f64(v) == 0).all()
    clean(pa)


@pytest.mark.parametrize("exponent", [-40, -3, 40])
def test_slots_never_stored_beside_scales_of_any_size(pa, exponent):
    """Even weights: what is stored is thinned out by the slots that are not, whatever its scale."""
    rng = np.random.default_rng(41)
    n = 90
    p = Pool(rng, [n], 1, canary=False)
    p.cache = R.random_records(rng, p.cache.shape[:2], 0.0, exponent)
    words = p.cache[..., R.K_SCALES:].view(np.uint16)
    if exponent == 40:
        words &= 0xFF8F                                     # no mantissa bits: 2^40 is the largest scale
    empty = rng.random((p.nb, B)) < 0.5
    for t in range(B):
        for ch in range(16):
            for at in (R.k_word(t, ch), R.v_word(t, ch)):
                p.cache[empty[:, t], :, at:at + 4] = 0
        p.cache[empty[:, t], :, R.K_SCALES + 8 * t:R.K_SCALES + 8 * t + 8] = 0
        p.cache[empty[:, t], :, R.V_SCALES + 2 * t:R.V_SCALES + 2 * t + 2] = 0
    q = np.zeros((1, 8, D))
    ref = p.attention(0, q, 0.1)
    close(pa.decode_int4(bf16(q), p.dev(), up(p.tables), up(p.lens), n, 0.1), ref, "decode", steps=8)
    close(pa.prefill_int4(bf16(q), up(np.array([0, 1], np.int32)), p.dev(), up(p.tables), up(p.lens), 1, n, 0.1), ref, "prefill",
          prefill=True)
    clean(pa)


def test_step_past_the_table_into_a_cleared_cache(pa):
    """A position without a cos/sin row stores nothing and still attends over its slot, here one of zeros."""
    rng = np.random.default_rng(42)
    lens, kv, hq = [20, 5, 700], 2, 4
    p = Pool(rng, lens, kv, canary=False)
    for s, n in enumerate(lens):
        p.cache[p.tables[s, (n - 1) // B]] = 0              # the blocks of the new tokens
    q, k, v = normal(rng, 3, hq, D), normal(rng, 3, kv, D), normal(rng, 3, kv, D)
    cs = table_of(10, 128)
    cache = p.dev()
    out = pa.decode_step_int4(bf16(q), bf16(k), bf16(v), up(cs), cache, up(p.tables), up(p.lens), 700, 0.1)
    clean(pa, pa.PA_FLAG_POSITION_OOB)
    for s in (0, 2):                                        # unrotated, nothing stored
        close(out[s:s + 1], p.attention(s, q[s:s + 1], 0.1), s, steps=lens[s] // 16 + 1)
        assert not cache[p.tables[s, (lens[s] - 1) // B]].any()
    p.cache = cache.cpu().numpy()
    # rotated as the store rotates, which may be a bf16 step from 64 bits: the test is that the row is a number
    assert np.isfinite(f64(out[1])).all()


# ---- scores far from zero ------------------------------------------------------------------

CUTS = [[70, 33, 1], [2000, 900]]                           # whole pieces, and split ones


@pytest.mark.parametrize("lens", CUTS)
@pytest.mark.parametrize("size", [1.0, 2.0 ** 11, 2.0 ** 16, 2.0 ** 24, 2.0 ** 60, 3e38])
@pytest.mark.parametrize("sign", [1, -1])
def test_tied_scores_of_any_size(pa, lens, size, sign):
    """Keys that are all alike weigh the same however large their score is, and the scales of V decide nothing."""
    rng = np.random.default_rng(43)
    kv, hq = 2, 6
    p = Pool(rng, lens, kv)
    row = rng.integers(0, 256, 64, dtype=np.uint8)
    words = np.array([0x3F80, 0x3FB5, 0x3F17, 0x3FC9], np.uint16).view(np.uint8)
    for t in range(B):
        live = p.cache[..., R.V_SCALES + 2 * t + 1] != 0xFF  # canaries stay
        p.cache[live, 64 * t:64 * t + 64] = row
        p.cache[live, R.K_SCALES + 8 * t:R.K_SCALES + 8 * t + 8] = words
        e = rng.integers(-6, 7, live.sum()) + 127
        word = (e << 7 | rng.integers(0, 8, live.sum()) << 4 | rng.integers(3, 13, live.sum())).astype(np.uint16)
        p.cache[live, R.V_SCALES + 2 * t:R.V_SCALES + 2 * t + 2] = word[:, None].view(np.uint8)
    q = sign * size * np.abs(np.sign(normal(rng, len(lens), hq, D)))
    args = (p.dev(), up(p.tables), up(p.lens))
    dec = pa.decode_int4(bf16(q), *args, max(lens), 1.0)
    pre = pa.prefill_int4(bf16(q), up(np.arange(len(lens) + 1, dtype=np.int32)), *args, 1, max(lens), 1.0)
    for s, n in enumerate(lens):
        ref = p.attention(s, np.zeros((1, hq, D)), 1.0)     # even weights
        close(dec[s:s + 1], ref, ("decode", s), steps=n // 16 + 1)
        close(pre[s:s + 1], ref, ("prefill", s), prefill=True)
    clean(pa)


def levels(cache, ids, kv, level):
    """K of the blocks `ids` [n] (tokens in order): dim 0 is level [16 n], dim 32 is 15, in units; dims 1 - 31 and 33 - 63 as the
    codes are."""
    one = torch.tensor([0x80, 0x3F], dtype=torch.uint8, device=cache.device)       # s = 1, z = 0
    level = level.view(-1, B).to(torch.uint8)
    for t in range(B):
        a = cache[ids, :, 64 * t]
        cache[ids, :, 64 * t] = (a & 0xF0) | level[:, t, None]
        b = cache[ids, :, 64 * t + 4]
        cache[ids, :, 64 * t + 4] = b | 0x0F
        cache[ids, :, R.K_SCALES + 8 * t:R.K_SCALES + 8 * t + 2] = one
        cache[ids, :, R.K_SCALES + 8 * t + 2:R.K_SCALES + 8 * t + 4] = one


def random_cache(seed, nb, kv):
    """Random records, made on the GPU: elements of K and V of a few units of 2^-3, V of scales over 2^-6 .. 2^0."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cache = torch.randint(0, 256, (nb, kv, R.RECORD), dtype=torch.uint8, device="cuda", generator=gen)

    def some(lo, hi, n):
        return torch.randint(lo, hi, (nb, kv, n), device="cuda", generator=gen)

    n = (R.RECORD - R.K_SCALES) // 2
    word = (some(121, 128, n) << 7 | some(0, 8, n) << 4 | some(3, 13, n)).to(torch.int16)
    cache[..., R.K_SCALES:] = word.view(torch.uint8)
    return cache


def rising(n, period):
    """Levels 0 to 3 of a period: a quarter, a quarter, half but one token, one token.  A level's tokens together weigh
    less than the one behind them, by 16.5 in the exponent, yet as many as they are they show."""
    at = torch.arange(n) % period
    lv = (at >= period // 4).int() + (at >= period // 2).int() + (at == period - 1).int()
    return lv.cuda()


@pytest.mark.parametrize("base", [0.0, 66.0, -66.0, 2.0 ** 8, -(2.0 ** 8), 2.0 ** 16, -(2.0 ** 16)])
@pytest.mark.parametrize("seqs,n,kv", [(64, 4096, 8), (3, 300, 2), (1, 5000, 1)])
def test_maxima_that_rise_within_a_warp(pa, base, seqs, n, kv):
    """The running maximum rises by 16.5 up to three times a period of 312 tokens or of the whole context, over scores of 0 or of
    15 `base`; from 66 the last rise passes 2^10.  64 sequences of 4096 tokens: a warp goes through some 78 blocks, 39 jobs."""
    hq, nb = 2 * kv, seqs * ((n + B - 1) // B) + 3
    mb = (n + B - 1) // B
    cache = random_cache(44, nb, kv)
    gen = torch.Generator(device="cuda").manual_seed(45)
    tables = torch.randperm(nb, device="cuda", generator=gen)[: seqs * mb].view(seqs, mb)
    for s in range(seqs):
        levels(cache, tables[s], kv, rising(mb * B, 312 if s % 2 else n))
    q = np.zeros((seqs, hq, D))
    q[:, ::2, 0], q[:, 1::2, 0] = 16.5, -16.5               # odd heads see the maximum first
    q[:, :, 32] = base
    scale = unit_scale()
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    t32 = tables.to(torch.int32)
    dec = pa.decode_int4(bf16(q), cache, t32, lens, n, scale)
    pre = pa.prefill_int4(bf16(q), torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), cache, t32, lens, 1, n, scale)
    for s in sorted({0, 1, seqs // 2, seqs - 1} & set(range(seqs))):
        own = cache[tables[s]].cpu().numpy()
        ref = R.attention(q[s:s + 1], own, np.arange(mb), n, scale)
        close(dec[s:s + 1], ref, ("decode", s), steps=n // 16 + 1)
        close(pre[s:s + 1], ref, ("prefill", s), prefill=True)
    clean(pa)


@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("seqs,n,kv", [(32, 4096, 8), (3, 300, 2), (1, 5000, 1)])
def test_near_and_far_heads_side_by_side(pa, down, seqs, n, kv):
    """Heads of one group whose scores pass 2^10 on either side, at different tokens or never; levels that rise, or fall."""
    group, mb = np.array([700.0, -700.0, 0.5, -16.5, 400.0, 2.0 ** 30, -(2.0 ** 30)]), (n + B - 1) // B
    hq, nb = len(group) * kv, seqs * mb + 3
    cache = random_cache(50, nb, kv)
    tables = torch.randperm(nb, device="cuda", generator=torch.Generator(device="cuda").manual_seed(51))[: seqs * mb].view(seqs, mb)
    for s in range(seqs):
        lv = rising(mb * B, 312 if s % 2 else n)
        levels(cache, tables[s], kv, 3 - lv if down else lv)
    q = np.zeros((seqs, hq, D))
    q[:, :, 0] = np.tile(group, kv)
    lens, t32 = torch.full((seqs,), n, dtype=torch.int32, device="cuda"), tables.to(torch.int32)
    scale = unit_scale()
    assert np.array_equal(f64(bf16(group)), S.bf16_round(group))
    q = f64(bf16(q))
    dec = pa.decode_int4(bf16(q), cache, t32, lens, n, scale)
    pre = pa.prefill_int4(bf16(q), torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), cache, t32, lens, 1, n, scale)
    for s in sorted({0, 1, seqs - 1} & set(range(seqs))):
        ref = R.attention(q[s:s + 1], cache[tables[s]].cpu().numpy(), np.arange(mb), n, scale)
        close(dec[s:s + 1], ref, ("decode", s), steps=n // 16 + 1)
        close(pre[s:s + 1], ref, ("prefill", s), prefill=True)
    clean(pa)


@pytest.mark.parametrize("lens", CUTS)
@pytest.mark.parametrize("size", [2.0 ** 7, 2.0 ** 12, 2.0 ** 70])
def test_the_step_is_store_then_decode_for_far_scores(pa, lens, size):
    rng = np.random.default_rng(55)
    kv, hq, n = 2, 14, len(lens)
    p = Pool(rng, lens, kv)
    q, k, v = bf16(size * normal(rng, n, hq, D)), bf16(normal(rng, n, kv, D)), bf16(normal(rng, n, kv, D))
    cs, c1, c2 = up(table_of(max(lens), 64)), p.dev(), p.dev()
    pos = (p.lens - 1).astype(np.int32)
    slots = p.tables[np.arange(n), pos // B].astype(np.int64) * B + pos % B
    out = pa.decode_step_int4(q, k, v, cs, c1, up(p.tables), up(p.lens), max(lens), 1.0)
    qr = pa.rope_kv_store_int4(q, k, v, up(pos), cs, up(slots), c2, q_out=torch.empty_like(q))
    assert torch.equal(c1, c2)
    assert np.array_equal(bits(out), bits(pa.decode_int4(qr, c2, up(p.tables), up(p.lens), max(lens), 1.0)))
    assert np.isfinite(f64(out)).all()
    clean(pa)


# ---- many blocks of a warp -----------------------------------------------------------------

@pytest.mark.parametrize("step", [False, True])
def test_warps_that_go_through_many_blocks(pa, step):
    """64 sequences of up to 4096 tokens, 8 KV heads, nearly even weights: some 70 blocks a warp, so its ring goes round several
    times and its sums of codes and of zero points are far larger than what is left of them."""
    rng = np.random.default_rng(46)
    seqs, kv, hq, n = 64, 8, 16, 4096
    lens = rng.integers(n - 600, n + 1, seqs).astype(np.int32)
    mb = n // B
    nb = seqs * mb + 3
    cache = random_cache(47, nb, kv)
    tables = torch.from_numpy(rng.permutation(nb)[: seqs * mb].reshape(seqs, mb)).cuda()
    t32, q = tables.to(torch.int32), normal(rng, seqs, hq, D) * 2.0 ** -6
    if step:
        cs = table_of(n, 64)
        k, v = bf16(normal(rng, seqs, kv, D)), bf16(normal(rng, seqs, kv, D))
        slots = np.take_along_axis(tables.cpu().numpy(), (lens[:, None] - 1) // B, 1)[:, 0].astype(np.int64) * B + (lens - 1) % B
        other = cache.clone()
        got = pa.decode_step_int4(bf16(q), k, v, up(cs), cache, t32, up(lens), n, D ** -0.5)
        qr = pa.rope_kv_store_int4(bf16(q), k, v, up(lens - 1), up(cs), up(slots), other)
        assert torch.equal(cache, other)
        assert np.array_equal(bits(got), bits(pa.decode_int4(qr, cache, t32, up(lens), n, D ** -0.5)))
        q = f64(qr)
    else:
        got = pa.decode_int4(bf16(q), cache, t32, up(lens), n, D ** -0.5)
    for s in (0, 17, 40, 63):
        ref = R.attention(q[s:s + 1], cache[tables[s]].cpu().numpy(), np.arange(mb), int(lens[s]), D ** -0.5)
        close(got[s:s + 1], ref, s, steps=int(lens[s]) // 16 + 1)
    clean(pa)


def test_hand_overs_while_the_gpu_is_busy(pa):
    """Feeder and consumers hand stages over in whatever order the memory gives records: the bits stay what they are alone, while
    copies and other calls come and go on two more streams."""
    rng = np.random.default_rng(52)
    seqs, kv, hq, n = 48, 8, 32, 3000
    mb = (n + B - 1) // B
    nb = seqs * mb + 3
    cache, lens = random_cache(53, nb, kv), up(rng.integers(1, n + 1, seqs).astype(np.int32))
    t32 = torch.from_numpy(rng.permutation(nb)[: seqs * mb].reshape(seqs, mb).astype(np.int32)).cuda()
    q, starts = bf16(normal(rng, seqs, hq, D)), torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    k, v, cs = bf16(normal(rng, seqs, kv, D)), bf16(normal(rng, seqs, kv, D)), up(table_of(n, 128))
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    other = torch.empty_like(big)
    want = bits(pa.decode_int4(q, cache, t32, lens, n, 0.1))
    c1 = cache.clone()
    want_step = bits(pa.decode_step_int4(q, k, v, cs, c1, t32, lens, n, 0.1))
    mine, copies, calls = (torch.cuda.Stream() for _ in range(3))
    got = []
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(copies):
            other[: (i + 1) << 23].copy_(big[: (i + 1) << 23])
        pa.prefill_int4(q, starts, cache, t32, lens, 1, n, 0.1, stream=calls)
        got.append((pa.decode_int4(q, cache, t32, lens, n, 0.1, stream=mine),
                    pa.decode_step_int4(q, k, v, cs, c1, t32, lens, n, 0.1, stream=mine)))
    torch.cuda.synchronize()
    for a, b in got:
        assert np.array_equal(bits(a), want) and np.array_equal(bits(b), want_step)
    clean(pa)


# ---- small elements of q -------------------------------------------------------------------

@pytest.mark.parametrize("lens", CUTS)
def test_elements_of_q_down_to_a_24th_power_count(pa, lens):
    """The decode's q is f16 after a power of two for each head: elements down to 2^-24 of the head's largest are exact, and here
    keys make up for them, dim by dim of a word."""
    rng = np.random.default_rng(54)
    kv, hq = 2, 16
    p = Pool(rng, lens, kv)
    for t in range(B):
        live = p.cache[..., R.V_SCALES + 2 * t + 1] != 0xFF  # canaries stay
        n = live.sum()
        for g, e in ((0, -6), (1, 17), (2, -6), (3, 17)):
            word = ((e + 127) << 7 | rng.integers(0, 8, n) << 4 | rng.integers(3, 13, n)).astype(np.uint16)
            at = R.K_SCALES + 8 * t + 2 * g
            p.cache[live, at:at + 2] = word[:, None].view(np.uint8)
    q = np.zeros((len(lens), hq, D))
    q[..., 0], q[..., 70] = 1.0, -0.75
    for h in range(hq):                                     # the eight dims of a word, in groups 1 and 3
        q[:, h, (32 if h < 8 else 104) + h % 8] = 2.0 ** -24 * (1 + h / 128)
    args = (p.dev(), up(p.tables), up(p.lens))
    dec = pa.decode_int4(bf16(q), *args, max(lens), 1.0)
    pre = pa.prefill_int4(bf16(q), up(np.arange(len(lens) + 1, dtype=np.int32)), *args, 1, max(lens), 1.0)
    for s, n in enumerate(lens):
        ref = p.attention(s, q[s:s + 1], 1.0)
        close(dec[s:s + 1], ref, ("decode", s), steps=n // 16 + 1)
        close(pre[s:s + 1], ref, ("prefill", s), prefill=True)
    clean(pa)


# ---- bounds near 2^31 ----------------------------------------------------------------------

@pytest.mark.parametrize("hq", [1, 3])
def test_prefill_with_the_loosest_bounds(pa, hq):
    """A block table as wide as lengths of 32 bits allow, and both bounds at its end: tiles and stages round up without an overflow."""
    rng = np.random.default_rng(48)
    p = Pool(rng, [40], 1)
    q = normal(rng, 5, hq, D)
    wide, most = 1 << 27, 2 ** 31 - 1
    tables = torch.full((1, wide), -1, dtype=torch.int32, device="cuda")
    tables[0, : p.tables.shape[1]] = up(p.tables[0])
    starts = up(np.array([0, 5], np.int32))
    got = pa.prefill_int4(bf16(q), starts, p.dev(), tables, up(p.lens), most, most, 0.1)
    close(got, p.attention(0, q, 0.1, first=35), prefill=True)
    kb, vb = (bf16(np.nan_to_num(x)) for x in R.unpack(p.cache))      # the same elements in a bf16 cache
    got = pa.prefill(bf16(q), starts, kb, vb, tables, up(p.lens), most, most, 0.1)
    close(got, p.attention(0, q, 0.1, first=35), prefill=True)
    k8, v8 = (torch.zeros(kb.shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = torch.ones((p.nb, 1, 2), device="cuda")
    assert not pa.prefill_fp8_block(bf16(q), starts, k8, v8, scales, tables, up(p.lens), most, most, 0.1).any()
    clean(pa)
