"""Orders that the block-scaled prefill's MMA warp has to keep, checked on its source: what breaks them is a
race in tensor memory, which no run shows for certain."""

from __future__ import annotations

import re
from pathlib import Path

SOURCE = Path(__file__).resolve().parents[1] / "paged_kv_cache_244_gb300" / "csrc" / "paged_prefill_block.cu"


def mma_loop() -> str:
    """The MMA warp's loop over the stages, without comments."""
    text = re.sub(r"//[^\n]*", "", SOURCE.read_text())
    warp = text[text.index("warp == 5"):]
    loop = warp[warp.index("j < nst && !failed; ++j) {\n        const int st"):]
    return loop[: loop.index("if (lane == 0)")]


def test_scores_are_written_over_p_only_after_p_v_is_done():
    """S_{j+2} takes the columns of P_j.  MMAs of other accumulators, shapes or kinds are not ordered by their
    issue, so a wait for the commit behind P_j V_j lies between the two."""
    loop = mma_loop()
    pv = loop.index("umma_bf16_tmem_a(")
    commit = loop.index("umma_commit(hdr + kVFree + 8 * st)", pv)
    wait = loop.index("wait_all(hdr + kVFree + 8 * st, (j / kBpVRing) & 1)", commit)
    fence = loop.index("tc_fence_after()", wait)
    assert loop.index("issue_s(j + 2)") > fence
    assert loop.count("issue_s(") == 1
