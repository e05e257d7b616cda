"""The aligned forms of collective instructions want the whole warp at the instruction, wherever its lanes come from: checked on
the source, as lanes that came apart mostly meet again by themselves."""

from __future__ import annotations

import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "paged_kv_cache_244_gb300" / "csrc"


def code(name: str) -> str:
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


@pytest.mark.parametrize("function", ["tmem_alloc", "cluster_sync", "named_barrier"])
def test_block_wide_forms_gather_their_warps(function):
    source = code("pa_device.cuh")
    body = source[source.index(f"void {function}("):]
    assert body.index("__syncwarp();") < body.index("asm volatile(")


@pytest.mark.parametrize("name", ["paged_decode.cu", "paged_decode_block.cu", "paged_decode_int4.cu"])
def test_lanes_that_mark_a_gap_are_waited_for(name):
    """A few lanes mark the skipped slot; matrix instructions and transposing loads follow."""
    source = code(name)
    store = source[source.index("if ((fl & kGap) && lane < G)"):]
    assert re.match(r"if \(\(fl & kGap\) && lane < G\)\s*a\.ws_ml\[[^;]*;\s*__syncwarp\(\);", store)
