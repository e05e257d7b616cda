"""The references of the serving operators against independent facts, and the refusals of the
serving entry points that need no device (the library checks them before touching one)."""

import ctypes

import numpy as np
import pytest
import torch

import serving_ref as R
from paged_kv_cache_244_gb300 import _build


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_244_gb300 import binding
    _build.build()
    binding.lib()
    return binding


def test_e4m3_codes_agree_with_torch():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * np.exp(4 * rng.standard_normal(20000)), R.E4M3[:127], R._MID,
                        -R._MID, [0.0, -0.0, 1e30, -1e30]]).astype(np.float32)
    t = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_encode(x), t)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.E4M3, every, equal_nan=True)
    assert R.e4m3_encode(np.array([np.nan, np.inf, -np.inf])).tolist() == [0x7F, 0x7E, 0xFE]


def test_bf16_rounding_agrees_with_torch():
    x = np.random.default_rng(2).standard_normal(10000).astype(np.float32)
    assert np.array_equal(R.bf16_round(x), torch.from_numpy(x).to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("a,s", [(448.0, 1.0), (448.5, 2.0), (449.0, 2.0), (224.0, 0.5), (0.0, 2.0 ** -40), (1e-30, 2.0 ** -40),
                                 (1e30, 2.0 ** 40), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7)])
def test_wanted_scale(a, s):
    assert R.wanted_scale(np.array([a, -a / 2, 0.0, np.inf, np.nan])) == s


def test_recoding_by_powers_of_two_is_exact_above_the_subnormals():
    codes = np.arange(0x7F, dtype=np.uint8)
    for k in range(1, 15):
        again = R.e4m3_encode(R.E4M3[codes] * 2.0 ** -k)
        kept = R.E4M3[codes] * 2.0 ** -k >= 2.0 ** -6
        assert np.array_equal(R.E4M3[again][kept], (R.E4M3[codes] * 2.0 ** -k)[kept])
        assert (np.abs(R.E4M3[again] - R.E4M3[codes] * 2.0 ** -k) <= 2.0 ** -10).all()


def test_rotation_keeps_the_norm_and_the_layouts_are_permutations():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 3, 128))
    for Rr in (16, 48, 96, 128):
        w = R.frequencies(Rr, 1e4)
        a = np.arange(5)[:, None] * w[None, :]
        cs = np.concatenate([np.cos(a), np.sin(a)], axis=1)
        h, i = R.rotate(x, cs, "half"), R.rotate(x, cs, "interleaved")
        assert np.allclose((h ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(h[..., Rr:], x[..., Rr:])
        order = np.concatenate([np.arange(0, Rr, 2), np.arange(1, Rr, 2), np.arange(Rr, 128)])
        assert np.allclose(R.rotate(x[..., order], cs, "half"), i[..., order])


def test_a_short_pool_refuses_in_order():
    got, flags = R.plan([0, 16, 5], [17, 1, 3], np.full((3, 4), -1, np.int32), np.arange(10, 13, dtype=np.int32), 2, 20, 25)
    # 2 blocks for the first, then none for the second; the third's token continue no block
    assert got["granted"].tolist() == [1, 0, 1] and flags == {"pool", "block"}
    assert got["tables"][0, :2].tolist() == [11, 10] and got["num_free"] == 0
    assert got["q_start"].tolist() == [0, 17, 18, 21] and got["context_lens"].tolist() == [17, 0, 8]


def test_instruction_descriptors_of_the_8_bit_and_f16_products(tmp_path):
    """The PTX ISA's bit positions written out: accumulator f32 at 4, A format at 7, B format at 10,
    majors at 15 and 16, N / 8 at 17, M / 16 at 24; E4M3 is 0 in kind::f8f6f4, f16 0 in kind::f16."""
    import shutil
    import subprocess
    from pathlib import Path
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "d.cpp", tmp_path / "d"
    src.write_text('#include <cstdio>\n#include "umma_desc.h"\nint main() { printf("%u %u %u", pa::umma_idesc_e4m3(128, 64), '
                   'pa::umma_idesc_f16(128, 128, false, true), pa::umma_idesc_f16(64, 16, true, false)); }\n')
    inc = Path(__file__).resolve().parents[1] / "paged_kv_cache_244_gb300" / "csrc"
    subprocess.run([cxx, "-std=c++17", f"-I{inc}", str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [1 << 4 | 8 << 17 | 8 << 24, 1 << 4 | 1 << 16 | 16 << 17 | 8 << 24, 1 << 4 | 1 << 15 | 2 << 17 | 4 << 24]


# ---- refusals ---------------------------------------------------------------------------

A = 0x10000          # an aligned address that is never read: every call below is refused first


def dims(pa, hq=12, hkv=2, d=128, b=16):
    return ctypes.byref(pa.pa_dims(hq, hkv, d, b))


def form_args(pa, **k):
    a = dict(d=dims(pa), rope=ctypes.byref(pa.pa_rope(128, 0)), T=4, q=A, qo=A, k=A, v=A, pos=A, cs=A, mp=10, sl=A, kc=A,
             vc=A, nb=4)
    a.update(k)
    return a


def call_form(pa, **k):
    a = form_args(pa, **k)
    return pa.lib().pa_rope_kv_store_form(a["d"], a["rope"], a["T"], a["q"], a["qo"], a["k"], a["v"], a["pos"], a["cs"],
                                          a["mp"], a["sl"], a["kc"], a["vc"], a["nb"], None)


def call_block(pa, sc=A, **k):
    a = form_args(pa, **k)
    return pa.lib().pa_rope_kv_store_fp8_block(a["d"], a["rope"], a["T"], a["q"], a["qo"], a["k"], a["v"], a["pos"], a["cs"],
                                               a["mp"], a["sl"], a["kc"], a["vc"], sc, a["nb"], None)


@pytest.mark.parametrize("call", [call_form, call_block])
def test_store_refusals(pa, call):
    for R_, layout in ((0, 0), (8, 0), (24, 0), (144, 0), (-16, 0), (64, 2), (64, -1)):
        assert call(pa, rope=ctypes.byref(pa.pa_rope(R_, layout))) == pa.PA_ERR_SHAPE
    assert call(pa, d=None) == pa.PA_ERR_NULL
    assert call(pa, d=dims(pa, d=64)) == pa.PA_ERR_SHAPE
    assert call(pa, d=dims(pa, hq=9, hkv=2)) == pa.PA_ERR_SHAPE
    assert call(pa, T=-1) == pa.PA_ERR_RANGE
    assert call(pa, T=0) == pa.PA_OK
    for name in ("q", "qo", "k", "v", "pos", "cs", "sl", "kc", "vc"):
        assert call(pa, **{name: None}) == pa.PA_ERR_NULL, name
        assert call(pa, **{name: A + 8}) == pa.PA_ERR_ALIGN, name
    assert call(pa, mp=0) == pa.PA_ERR_RANGE and call(pa, nb=0) == pa.PA_ERR_RANGE
    if call is call_block:
        assert call(pa, sc=None) == pa.PA_ERR_NULL and call(pa, sc=A + 8) == pa.PA_ERR_ALIGN


def test_table_refusals(pa):
    def call(R_=64, n=10, out=A, **k):
        a = dict(theta=1e4, factor=2.0, original_max_pos=4096.0, low=1.0, high=32.0, magnitude=0.0, kind=3)
        a.update(k)
        return pa.lib().pa_rope_table(ctypes.byref(pa.pa_rope_scaling(**a)), R_, n, out, None)
    assert pa.lib().pa_rope_table(None, 64, 10, A, None) == pa.PA_ERR_NULL
    assert call(out=None) == pa.PA_ERR_NULL and call(out=A + 4) == pa.PA_ERR_ALIGN
    for R_ in (0, 8, 40, 144):
        assert call(R_=R_) == pa.PA_ERR_SHAPE
    assert call(n=0) == pa.PA_ERR_RANGE
    nan, inf = float("nan"), float("inf")
    for bad in (dict(theta=1.0), dict(theta=nan), dict(theta=inf), dict(factor=0.5), dict(factor=nan), dict(factor=inf),
                dict(original_max_pos=0.0), dict(low=0.0), dict(high=1.0), dict(high=inf), dict(low=nan),
                dict(magnitude=-1.0), dict(magnitude=nan), dict(magnitude=1e300), dict(kind=5), dict(kind=-1), dict(kind=4, original_max_pos=nan)):
        assert call(**bad) == pa.PA_ERR_RANGE, bad


def test_attention_refusals(pa):
    L = pa.lib()

    def decode(sc=A, d=None, S=2, q=A, kc=A, nb=4, mb=4, ctx=A, mc=64, ws=A, wb=1 << 30, P=0, scale=0.1):
        return L.pa_decode_fp8_block(d or dims(pa), S, q, kc, A, sc, nb, A, mb, ctx, mc, scale, P, ws, wb, A, None)

    def step(rope=None, sc=A, k=A, cs=A, flags=0, S=2, mp=10):
        return L.pa_decode_step_fp8_block(dims(pa), rope, S, A, k, A, cs, mp, A, A, sc, 4, A, 4, A, 64, 0.1, 0, A, 1 << 30, A,
                                          flags, None)

    def prefill(sc=A, S=2, T=4, mq=4, q=A, mc=64):
        return L.pa_prefill_fp8_block(dims(pa), S, T, q, A, mq, A, A, sc, 4, A, 4, A, mc, 0.1, A, None)

    assert decode(sc=None) == pa.PA_ERR_NULL and decode(sc=A + 8) == pa.PA_ERR_ALIGN
    assert decode(q=None) == pa.PA_ERR_NULL and decode(q=A + 8) == pa.PA_ERR_ALIGN
    assert decode(mc=65) == pa.PA_ERR_RANGE and decode(P=8) == pa.PA_ERR_RANGE and decode(nb=0) == pa.PA_ERR_RANGE
    assert decode(scale=0.0) == pa.PA_ERR_RANGE and decode(scale=float("nan")) == pa.PA_ERR_RANGE
    assert decode(wb=16) == pa.PA_ERR_WORKSPACE and decode(ws=None) == pa.PA_ERR_WORKSPACE
    assert decode(S=8193) == pa.PA_ERR_RANGE and decode(S=0) == pa.PA_OK
    assert decode(d=dims(pa, hq=18, hkv=2)) == pa.PA_ERR_SHAPE
    assert step(sc=None) == pa.PA_ERR_NULL and step(k=None) == pa.PA_ERR_NULL and step(cs=None) == pa.PA_ERR_NULL
    assert step(rope=ctypes.byref(pa.pa_rope(40, 0))) == pa.PA_ERR_SHAPE
    assert step(flags=2) == pa.PA_ERR_RANGE and step(mp=0) == pa.PA_ERR_RANGE and step(S=0) == pa.PA_OK
    assert prefill(sc=None) == pa.PA_ERR_NULL and prefill(sc=A + 8) == pa.PA_ERR_ALIGN and prefill(q=None) == pa.PA_ERR_NULL
    assert prefill(mq=65) == pa.PA_ERR_RANGE and prefill(mc=100) == pa.PA_ERR_RANGE
    assert prefill(S=0) == pa.PA_OK and prefill(T=0) == pa.PA_OK


def test_plan_refusals(pa):
    def call(**k):
        a = dict(d=dims(pa), S=3, c=A, n=A, bt=A, mb=4, fb=A, cap=8, nf=A, nfo=A, nb=8, T=5, cx=A + 64, qs=A, ps=A, sl=A, gr=A)
        a.update(k)
        return pa.lib().pa_plan_step(a["d"], a["S"], a["c"], a["n"], a["bt"], a["mb"], a["fb"], a["cap"], a["nf"], a["nfo"],
                                     a["nb"], a["T"], a["cx"], a["qs"], a["ps"], a["sl"], a["gr"], None)
    for bad in (dict(S=-1), dict(S=8193), dict(T=-1), dict(T=2 ** 31 - 1), dict(cap=-1), dict(nb=0), dict(mb=0), dict(mb=1 << 27), dict(cx=A)):
        assert call(**bad) == pa.PA_ERR_RANGE, bad
    for name in ("c", "n", "bt", "fb", "nf", "nfo", "cx", "qs", "ps", "sl", "gr"):
        assert call(**{name: None}) == pa.PA_ERR_NULL, name
        assert call(**{name: A + 2}) == pa.PA_ERR_ALIGN, name
    assert call(ps=A + 4) == pa.PA_ERR_ALIGN and call(sl=A + 8) == pa.PA_ERR_ALIGN
    assert call(d=dims(pa, b=32)) == pa.PA_ERR_SHAPE and call(d=None) == pa.PA_ERR_NULL


def test_binding_refuses_wrong_tensors(pa):
    q, k = torch.zeros(4, 12, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    kc, sc = torch.zeros(4, 2, 16, 128, dtype=torch.uint8), torch.ones(4, 2, 2)
    i32, i64, cs = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), torch.zeros(8, 64)
    bt = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="scaling"):
        pa.rope_table(16, 64, scaling="cubic")
    with pytest.raises(ValueError, match="layout"):
        pa.rope_kv_store_fp8_block(q, k, k, i32, cs, i64, kc, kc, sc, layout="thirds")
    # tensors of another type, and tensors that are not on the GPU, are named
    with pytest.raises(ValueError, match="q must be BFloat16, got Float"):
        pa.rope_kv_store_fp8_block(q.float(), k, k, i32, cs, i64, kc, kc, sc)
    for call in (lambda: pa.rope_kv_store_fp8_block(q, k, k, i32, cs, i64, kc, kc, sc),
                 lambda: pa.rope_kv_store_form(q, k, k, i32, cs, i64, kc, kc),
                 lambda: pa.decode_fp8_block(q, kc, kc, sc, bt, i32, 16, 0.1, workspace=torch.zeros(8)),
                 lambda: pa.decode_step_fp8_block(q, k, k, cs, kc, kc, sc, bt, i32, 16, 0.1, workspace=torch.zeros(8)),
                 lambda: pa.prefill_fp8_block(q, torch.zeros(5, dtype=torch.int32), kc, kc, sc, bt, i32, 4, 16, 0.1),
                 lambda: pa.plan_step(i32, i32, bt, i32, i32[:1], 4, 5),
                 lambda: pa.rope_table(4, 64, out=torch.zeros(4, 64))):
        with pytest.raises(ValueError, match="must be a CUDA tensor on the current device"):
            call()
    p = pa.step_plan(2, 5, "cpu")
    with pytest.raises(ValueError, match="cached_lens must be a tensor"):
        pa.plan_step([0, 1], i32, bt, i32, i32[:1], 4, 5, plan=p)
    assert p.q_start.shape == (3,) and p.slot_mapping.dtype == torch.int64
