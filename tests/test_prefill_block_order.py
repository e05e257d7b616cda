"""Orders that the prefill kernels' MMA warps have to keep, checked on their source: what breaks them is a
race in tensor memory, which no run shows for certain."""

from __future__ import annotations

import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "paged_kv_cache_244_gb300" / "csrc"


def source(name: str) -> str:
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


def mma_loop() -> str:
    """The block-scaled prefill's MMA warp, its loop over the stages."""
    text = source("paged_prefill_block.cu")
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


@pytest.mark.parametrize("name,done", [("paged_prefill_block.cu", "kDone"), ("paged_prefill.cu", "kBarDone")])
def test_the_thread_that_issued_the_mmas_commits_the_last_of_them(name, done):
    """A commit follows the operations of its own thread, and which lane elect.sync names is not said."""
    assert re.findall(r"if \(([^;{}]*)\) umma_commit\(hdr \+ " + done + r"\)", source(name)) == ["elect_one()"]
    assert source(name).count(f"umma_commit(hdr + {done})") == 1
