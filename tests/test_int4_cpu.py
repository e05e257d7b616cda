"""The 4-bit cache without a GPU: the reference's own properties, and what the host refuses before a launch."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import int4_ref as R
import serving_ref as S
from paged_kv_cache_244_gb300 import _build


def test_every_element_is_a_bf16_value_and_every_word_reads_back():
    rng = np.random.default_rng(1)
    for _ in range(300):
        x = S.bf16_round(rng.standard_normal(128) * 2.0 ** rng.integers(-12, 12) + rng.choice([0.0, 3.0, -50.0]))
        rec = np.zeros(R.RECORD, np.uint8)
        t = int(rng.integers(0, 16))
        R.put_row(rec, t, x, x[::-1])
        k, v = (a[t] for a in R.unpack(rec))
        assert np.array_equal(k, S.bf16_round(k)) and np.array_equal(v, S.bf16_round(v))
        for got, want, groups in ((k, x, 4), (v, x[::-1], 1)):
            for g in range(groups):
                i = slice(g * 128 // groups, (g + 1) * 128 // groups)
                codes, s, z = R.quantise(want[i])
                assert np.array_equal(got[i], s * (codes - z))
                assert (np.abs(got[i] - want[i]) <= s / 2).all()
                assert s <= 1.125 * (max(0, want[i].max()) - min(0, want[i].min())) / 15


def test_a_quotient_is_a_tie_or_clear_of_one():
    """What lets 1 / s be off by 2^-20: a bf16 value over a scale is k + 1/2 exactly, or 2^-10 of itself away."""
    x = np.arange(128, 256, dtype=np.float64)
    for m in range(8, 16):
        for e in range(-1, 9):                           # x / s from 2^-2 to 2^6
            y = x / (m * 2.0 ** e)
            far = np.abs(y - np.floor(y) - 0.5) / y
            assert ((far == 0) | (far >= 2.0 ** -10)).all()


@pytest.mark.parametrize("x,s,z", [
    ([0.0] * 32, 2.0 ** -40, 0),
    ([1.5] + [0.0] * 31, 0.1015625, 0),                  # 1.5 / 15 = 0.1 between 0.1015625 and 0.09375
    ([-15.0, 0.0], 1.0, 15),
    ([7.5, -7.5], 1.0, 8),
    ([15.0 * 2.0 ** 41, 0.0], 2.0 ** 40, 0),
    ([-(2.0 ** 60), 1.0], 2.0 ** 40, 15),
    ([math.inf, -1.0, 14.0], 1.0, 1),
])
def test_scales_and_zero_points(x, s, z):
    codes, s2, z2 = R.quantise(np.array(x))
    assert (s2, z2) == (s, z)
    assert all(0 <= c <= 15 for c in codes)
    if math.isinf(x[0]):
        assert codes[0] == 15


A = 1 << 20     # a pointer that nothing reads
BAD = A + 8


@pytest.fixture(scope="module")
def pa():
    _build.build()
    from paged_kv_cache_244_gb300 import binding
    binding.lib()
    return binding


def dims(pa, hq=12, hkv=2, d=128, b=16):
    return ctypes.byref(pa.pa_dims(hq, hkv, d, b))


def test_store_refusals(pa):
    def call(d=None, rope=None, T=3, q=A, q_out=A, k=A, v=A, pos=A, cs=A, max_pos=64, slots=A, cache=A, nb=16):
        return pa.lib().pa_rope_kv_store_int4(d or dims(pa), rope, T, q, q_out, k, v, pos, cs, max_pos, slots, cache, nb, None)

    assert call(T=0) == pa.PA_OK and call(T=-1) == pa.PA_ERR_RANGE
    assert call(d=dims(pa, d=64)) == pa.PA_ERR_SHAPE and call(d=dims(pa, hq=18)) == pa.PA_ERR_SHAPE
    for bad in ((24, 0), (0, 0), (144, 0), (64, 2)):
        assert call(rope=ctypes.byref(pa.pa_rope(*bad))) == pa.PA_ERR_SHAPE
    for name in ("q", "q_out", "k", "v", "pos", "cs", "slots", "cache"):
        assert call(**{name: None}) == pa.PA_ERR_NULL, name
        assert call(**{name: BAD}) == pa.PA_ERR_ALIGN, name
    assert call(max_pos=0) == pa.PA_ERR_RANGE and call(nb=0) == pa.PA_ERR_RANGE


def test_read_refusals(pa):
    def call(d=None, S=2, rows=9, starts=A, first=A, max_rows=20, cache=A, nb=16, bt=A, mb=4, k=A, v=A):
        return pa.lib().pa_read_kv_int4(d or dims(pa), S, rows, starts, first, max_rows, cache, nb, bt, mb, k, v, None)

    assert call(S=0) == pa.PA_OK and call(rows=0) == pa.PA_OK
    assert call(d=dims(pa, b=32)) == pa.PA_ERR_SHAPE
    for kw in (dict(S=-1), dict(S=65536), dict(rows=-1), dict(max_rows=0), dict(max_rows=65), dict(nb=0), dict(mb=0),
               dict(mb=2 ** 27)):
        assert call(**kw) == pa.PA_ERR_RANGE, kw
    # pairs of records are one launch dimension: 2^31 - 1 at most
    assert call(d=dims(pa, 1024, 1024), mb=2 ** 27 - 1, max_rows=2 ** 31 - 16) == pa.PA_ERR_RANGE
    for name in ("starts", "cache", "bt", "k", "v"):
        assert call(**{name: None}) == pa.PA_ERR_NULL, name
    for name in ("starts", "first", "cache", "bt", "k", "v"):
        assert call(**{name: BAD}) == pa.PA_ERR_ALIGN, name


def test_decode_and_step_refusals(pa):
    def decode(d=None, S=2, q=A, cache=A, nb=16, bt=A, mb=4, ctx=A, mc=40, scale=0.1, P=0, ws=A, wsb=1 << 30, out=A):
        return pa.lib().pa_decode_int4(d or dims(pa), S, q, cache, nb, bt, mb, ctx, mc, scale, P, ws, wsb, out, None)

    def step(d=None, rope=None, S=2, q=A, k=A, v=A, cs=A, max_pos=64, cache=A, nb=16, bt=A, mb=4, ctx=A, mc=40, scale=0.1,
             P=0, ws=A, wsb=1 << 30, out=A, flags=0):
        return pa.lib().pa_decode_step_int4(d or dims(pa), rope, S, q, k, v, cs, max_pos, cache, nb, bt, mb, ctx, mc, scale,
                                            P, ws, wsb, out, flags, None)

    for call, names in ((decode, ("q", "cache", "bt", "ctx", "out")), (step, ("q", "k", "v", "cs", "cache", "bt", "ctx", "out"))):
        assert call(S=0) == pa.PA_OK
        assert call(d=dims(pa, d=64)) == pa.PA_ERR_SHAPE
        for kw in (dict(S=-1), dict(S=8193), dict(nb=0), dict(mc=0), dict(mc=65), dict(scale=0.0), dict(scale=math.nan),
                   dict(P=24), dict(nb=2 ** 27)):
            assert call(**kw) == pa.PA_ERR_RANGE, kw
        assert call(ws=None) == pa.PA_ERR_WORKSPACE and call(wsb=64) == pa.PA_ERR_WORKSPACE
        for name in names:
            assert call(**{name: None}) == pa.PA_ERR_NULL, name
            assert call(**{name: BAD}) == pa.PA_ERR_ALIGN, name
        assert call(ws=BAD) == pa.PA_ERR_ALIGN
    assert step(flags=2) == pa.PA_ERR_RANGE and step(max_pos=0) == pa.PA_ERR_RANGE
    assert step(rope=ctypes.byref(pa.pa_rope(20, 0))) == pa.PA_ERR_SHAPE


def test_prefill_refusals(pa):
    def call(d=None, S=2, T=40, q=A, qs=A, mq=32, cache=A, nb=16, bt=A, mb=4, ctx=A, mc=64, scale=0.1, out=A):
        return pa.lib().pa_prefill_int4(d or dims(pa), S, T, q, qs, mq, cache, nb, bt, mb, ctx, mc, scale, out, None)

    assert call(S=0) == pa.PA_OK and call(T=0) == pa.PA_OK
    for kw in (dict(S=-1), dict(T=-1), dict(mq=0), dict(mq=65), dict(mc=65), dict(S=40000), dict(scale=-1.0), dict(nb=0)):
        assert call(**kw) == pa.PA_ERR_RANGE, kw
    for name in ("q", "qs", "cache", "bt", "ctx", "out"):
        assert call(**{name: None}) == pa.PA_ERR_NULL, name
        assert call(**{name: BAD}) == pa.PA_ERR_ALIGN, name


def test_the_binding_refuses_what_is_not_a_cache_on_this_device(pa):
    import torch
    q = torch.zeros((2, 12, 128), dtype=torch.bfloat16)
    cache = pa.int4_cache(4, 2, device="cpu")
    assert cache.shape == (4, 2, pa.INT4_RECORD_BYTES)
    i32 = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError)):
        pa.decode_int4(q, cache, i32, i32[:, 0].contiguous(), 40, 0.1)
    with pytest.raises(ValueError, match="layout"):
        pa.rope_kv_store_int4(q, q, q, i32, i32, i32, cache, layout="thirds")
    with pytest.raises(ValueError, match="num_rows"):
        pa.read_kv_int4(cache, i32[0], None, i32, 4)
