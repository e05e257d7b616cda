"""The 4-bit cache's attention where test_gpu_int4 does not go: slots that nothing was stored in.

Tolerances are those of test_gpu_int4 (`close`), derived there.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import int4_ref as R
from test_gpu_int4 import B, D, Pool, bf16, bits, clean, close, f64, normal, pa, table_of, turned, up  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- slots that nothing was stored in ------------------------------------------------------

def test_slots_never_stored_read_as_zeros(pa):
    """A cleared cache holds zeros: a token within the context whose slot nothing was stored in counts with a score and a
    value of 0, in every call."""
    rng = np.random.default_rng(40)
    lens, kv, hq = [40, 16, 1, 700, 33], 2, 12
    p = Pool(rng, lens, kv, canary=False)
    p.cache[:] = 0
    T, cs = 0, np.concatenate([np.ones((1, 64)), np.zeros((1, 64))], axis=1).astype(np.float32)
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
