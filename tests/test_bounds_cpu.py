"""Host bounds at the end of 32 bits: what the calls refuse, without a GPU."""

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


@pytest.mark.parametrize("bound", [2 ** 31 - 15, 2 ** 31 - 1])
@pytest.mark.parametrize("partition", [0, 512])
def test_decode_refuses_lengths_that_do_not_round_up_in_32_bits(pa, bound, partition):
    """A bound past 2^31 - 16 has no whole number of blocks in an int: no workspace size, and no call."""
    d = ctypes.byref(pa.pa_dims(4, 1, 128, 16))
    L = pa.lib()
    assert L.pa_decode_partition_tokens(d, 2, bound, partition) == pa.PA_ERR_RANGE
    assert L.pa_decode_workspace_size(d, 2, bound, partition) == 0
    args = (A, 16, A, 1 << 27, A, bound, 0.1, partition, A, 1 << 62, A)
    assert L.pa_decode_int4(d, 2, A, *args, None) == pa.PA_ERR_RANGE
    assert L.pa_decode(d, 2, A, A, *args, None) == pa.PA_ERR_RANGE


def test_decode_takes_the_largest_bound_that_does(pa):
    d = ctypes.byref(pa.pa_dims(4, 1, 128, 16))
    L, bound = pa.lib(), 2 ** 31 - 16
    assert L.pa_decode_partition_tokens(d, 2, bound, 512) == 512
    rows = 2048 * 4                                         # split evenly: a slot for each warp's range, and one a segment
    assert L.pa_decode_workspace_size(d, 2, bound, 0) == (rows + 2 * 4) * 130 * 4
