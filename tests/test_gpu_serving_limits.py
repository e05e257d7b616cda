"""The block-scaled attention where its arithmetic runs out: factors and scores at the ends of fp32, queries below
its normal range.

Tolerances are those of test_gpu_serving (`close`): half a bf16 step of the result, 2^-8, and 2^-9 of the A that
the reference gives for weights held in f16.  Scores beyond 2^24 carry an fp32 rounding of their own, up to half
a step of the score: the tests that use them check on the reference that the largest score leads by more than
its step times 64, so that the weights are 0 and 1 whatever the rounding.
"""

from __future__ import annotations

import numpy as np
import pytest

import serving_ref as R
from test_gpu_serving import B, D, Pool, bf16, clean, close, normal, pa, up  # noqa: F401

pytestmark = pytest.mark.gpu


def both(pa, pool, q, lens, new, scale, want=0):
    """Prefill of the last `new` rows of each sequence and decode of its last row, against the reference."""
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    qd = q if hasattr(q, "is_cuda") else bf16(q)
    q64 = qd.cpu().double().numpy()
    args = (*pool.dev(), up(pool.tables), up(pool.lens))
    pre = pa.prefill_fp8_block(qd, up(qs), *args, max(new), max(lens), scale)
    dec = pa.decode_fp8_block(qd[up(qs[1:].astype(np.int64) - 1)], *args, max(lens), scale)
    clean(pa, want)
    for s, (n, m) in enumerate(zip(lens, new)):
        ref, mag = pool.attention(s, q64[qs[s]:qs[s + 1]], scale, n - m)
        close(dec[s:s + 1], ref[-1:], mag[-1:], ("decode", s))
        close(pre[qs[s]:qs[s + 1]], ref, mag, ("prefill", s))


CUTS = [([70, 33, 1], [70, 5, 1]), ([2000, 900], [3, 20])]     # whole tiles, and keys split over a cluster


@pytest.mark.parametrize("lens,new", CUTS)
@pytest.mark.parametrize("size", [2.0 ** -95, 2.0 ** -105, 2.0 ** -122])
def test_small_queries_over_blocks_of_the_least_scale(pa, lens, new, size):
    """scale * K scale * the power of two of q is below fp32's range, beside masked keys."""
    rng = np.random.default_rng(1)
    pool = Pool(rng, lens, 2)
    for s in range(len(lens)):
        pool.k[pool.tables[s, : (lens[s] + B - 1) // B : 2]] = 0
        pool.scale[pool.tables[s, : (lens[s] + B - 1) // B : 2], :, 0] = 2.0 ** -40
    both(pa, pool, normal(rng, sum(new), 12, D) * size, lens, new, D ** -0.5)


@pytest.mark.parametrize("lens,new", CUTS)
def test_softmax_scale_and_query_far_apart(pa, lens, new):
    """The power of two of q and the softmax scale cancel; with the K scale alone the latter leaves fp32's range."""
    rng = np.random.default_rng(2)
    for k_scale in (2.0 ** -40, 2.0 ** 34):
        pool = Pool(rng, lens, 2)
        pool.scale[..., 0] = k_scale
        size = 2.0 ** 118 if k_scale < 1 else 2.0 ** -110
        both(pa, pool, normal(rng, sum(new), 12, D) * size, lens, new, D ** -0.5 / size / k_scale * 2.0 ** -7)


@pytest.mark.parametrize("lens,new", CUTS)
def test_large_factors_over_scores_of_zero(pa, lens, new):
    """scale * K scale * the power of two of q is above fp32's range where q . K is 0."""
    rng = np.random.default_rng(3)
    pool = Pool(rng, lens, 2)
    pool.k[..., :64] = 0
    pool.scale[..., 0] = 2.0 ** 40
    q = normal(rng, sum(new), 12, D) * 2.0 ** 120
    q[..., 64:] = 0
    for s, n in enumerate(lens):                                # the slots past the context hold NaN still
        if n % B:
            pool.k[pool.tables[s, n // B], :, n % B:] = 0x7F
    both(pa, pool, q, lens, new, D ** -0.5)


@pytest.mark.parametrize("lens,new", CUTS)
@pytest.mark.parametrize("k_scale", [2.0 ** 14, 2.0 ** 21, 2.0 ** 40])
def test_large_scores(pa, lens, new, k_scale):
    """Scores of 2^24 and more: the step between neighbouring fp32 values passes what a weight can hold."""
    rng = np.random.default_rng(4)
    pool = Pool(rng, lens, 2)
    pool.scale[..., 0] = k_scale
    q = R.bf16_round(normal(rng, sum(new), 4, D))
    qs = np.concatenate([[0], np.cumsum(new)])
    for s, (n, m) in enumerate(zip(lens, new)):                 # the largest score leads clearly, or keys are one
        ids = pool.tables[s][: (n + B - 1) // B]
        for g in range(2):
            K = np.concatenate([R.E4M3[pool.k[b, g]] for b in ids])[:n] * k_scale
            x = np.einsum("rhd,td->rht", q[qs[s]:qs[s + 1], 2 * g:2 * g + 2], K) * D ** -0.5 * np.log2(np.e)
            x = np.where(np.arange(n) <= n - m + np.arange(m)[:, None, None], x, -np.inf)
            top = np.sort(x, axis=-1)
            if n > 1:
                assert (np.isinf(top[..., -2]) | (top[..., -1] - top[..., -2] > 64 * 2.0 ** -23 * np.abs(top[..., -1]))).all()
    both(pa, pool, q, lens, new, D ** -0.5)


@pytest.mark.parametrize("lens,new", CUTS)
def test_queries_below_the_normal_range(pa, lens, new):
    rng = np.random.default_rng(5)
    pool = Pool(rng, lens, 2)
    codes = rng.integers(-100, 101, (sum(new), 12, D))          # multiples of 2^-133, the least bf16
    q = up((np.abs(codes) | np.where(codes < 0, 0x8000, 0)).astype(np.uint16).view(np.int16)).view(bf16(np.zeros(1)).dtype)
    assert np.array_equal(q.cpu().double().numpy(), codes * 2.0 ** -133)
    both(pa, pool, q, lens, new, D ** -0.5 * 2.0 ** 127)


@pytest.mark.parametrize("hq,kv", [(12, 2), (8, 8), (8, 1)])
@pytest.mark.parametrize("lens,new", CUTS + [([130, 260], [130, 130])])
def test_nan_in_a_later_token_leaves_earlier_queries_alone(pa, lens, new, hq, kv):
    """A NaN in K spoils the rows that see its token, one in V their dim of it; the rows before it have none."""
    rng = np.random.default_rng(6)
    pool = Pool(rng, lens, kv)
    q = normal(rng, sum(new), hq, D)
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = pool.k.copy(), pool.v.copy()
    hit = []
    for s, (n, m) in enumerate(zip(lens, new)):
        for i in range(6):
            t, g, d = int(rng.integers(n - m, n)), int(rng.integers(kv)), int(rng.integers(D))
            which = "k" if i == 0 else "v"
            (k if which == "k" else v)[pool.tables[s, t // B], g, t % B, d] = 0x7F if i % 2 else 0xFF
            hit.append((s, t, g, d, which))
    args = (up(k), up(v), up(pool.scale), up(pool.tables), up(pool.lens))
    out = pa.prefill_fp8_block(bf16(q), up(qs), *args, max(new), max(lens), D ** -0.5).cpu().double().numpy()
    clean(pa)
    for s, (n, m) in enumerate(zip(lens, new)):
        wrong = [h for h in hit if h[0] == s]
        for _, t, g, d, which in wrong:                          # codes of zero for the rows that do not see them
            (pool.k if which == "k" else pool.v)[pool.tables[s, t // B], g, t % B, d] = 0
        ref, mag = pool.attention(s, q[qs[s]:qs[s + 1]], D ** -0.5, n - m)
        nan = np.zeros(ref.shape, bool)
        G = hq // kv
        for _, t, g, d, which in wrong:
            heads, dims = slice(g * G, (g + 1) * G), slice(None) if which == "k" else d
            nan[max(t - (n - m), 0):, heads, dims] = True
        got = out[qs[s]:qs[s + 1]]
        assert np.array_equal(np.isnan(got), nan), (s, np.argwhere(np.isnan(got) != nan)[:4])
        close(np.where(nan, 0.0, got), np.where(nan, 0.0, ref), mag, s)


@pytest.mark.parametrize("lens,new", CUTS)
def test_rows_of_very_different_factors_side_by_side(pa, lens, new):
    """Heads and rows of one tile, and blocks of one stage, on both sides of where an exponent takes two steps."""
    rng = np.random.default_rng(7)
    pool = Pool(rng, lens, 2)
    pool.scale[..., 0] = 2.0 ** rng.integers(-12, 25, pool.scale.shape[:2])
    q = R.bf16_round(normal(rng, sum(new), 12, D) * 2.0 ** rng.integers(-45, 3, (sum(new), 12, 1)))
    qs = np.concatenate([[0], np.cumsum(new)])
    args = (*pool.dev(), up(pool.tables), up(pool.lens))
    pre = pa.prefill_fp8_block(bf16(q), up(qs.astype(np.int32)), *args, max(new), max(lens), D ** -0.5).cpu().double().numpy()
    dec = pa.decode_fp8_block(bf16(q[qs[1:] - 1]), *args, max(lens), D ** -0.5).cpu().double().numpy()
    clean(pa)
    assert np.isfinite(pre).all() and np.isfinite(dec).all()
    checked = 0
    for s, (n, m) in enumerate(zip(lens, new)):
        rows = q[qs[s]:qs[s + 1]]
        ref, mag = pool.attention(s, rows, D ** -0.5, n - m)
        top = pool.scale[pool.tables[s][: (n + B - 1) // B], :, 0].max(axis=0).repeat(6)
        # a score is off by 2^-17 of sum |q| 448 k at most: rows where that is below 2^-12 are compared
        small = np.abs(rows).max(axis=2) * D * 448 * top * D ** -0.5 * 2.0 ** -17 < 2.0 ** -12
        checked += small.sum()
        close(np.where(small[..., None], pre[qs[s]:qs[s + 1]], 0.0), np.where(small[..., None], ref, 0.0), mag, ("prefill", s))
        close(np.where(small[-1:, :, None], dec[s:s + 1], 0.0), np.where(small[-1:, :, None], ref[-1:], 0.0), mag[-1:], ("decode", s))
    assert checked > 12
