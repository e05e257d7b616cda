"""Bounds of the serving calls that are refused on the host; nothing here reaches a device."""

from __future__ import annotations

import ctypes

import pytest

from paged_kv_cache_244_gb300 import _build

A = 1 << 20     # a pointer that nothing reads


@pytest.fixture(scope="module")
def pa():
    _build.build()
    from paged_kv_cache_244_gb300 import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("capacity", [2 ** 31 - 1, 2 ** 30 + 1])
def test_a_free_list_past_what_the_sums_can_count_is_refused(pa, capacity):
    """Sums of needs are clamped to 2^31 - 1: a free list of that many would grant entries past its end, and
    indexes that step by a grid of threads would pass 31 bits."""
    d = pa.pa_dims(12, 2, 128, 16)
    got = pa.lib().pa_plan_step(ctypes.byref(d), 3, A, A, A, 4, A, capacity, A, A, 8, 5, A + 64, A, A, A, A, None)
    assert got == pa.PA_ERR_RANGE
