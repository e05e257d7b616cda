"""Orders that the MMA warp of the 4-bit cache's prefill has to keep, checked on its source: what breaks them is a
race in tensor memory, which no run shows for certain."""

from __future__ import annotations

import re
from pathlib import Path

SOURCE = Path(__file__).resolve().parents[1] / "paged_kv_cache_244_gb300" / "csrc" / "paged_prefill_int4.cu"


def text() -> str:
    return re.sub(r"//[^\n]*", "", SOURCE.read_text())


def mma_loop() -> str:
    warp = text()
    warp = warp[warp.index("if (warp == 4) {"):]
    loop = warp[warp.index("for (int j = 0; j < nst && !failed; ++j) {\n        const int st"):]
    return loop[: loop.index("if (lane == 0)")]


def test_scores_are_written_over_p_only_after_p_v_is_done():
    """S_{j+2} takes the columns of P_j, and MMAs of other accumulators or shapes are not ordered by their issue: a wait for
    the commit behind P_j V_j lies between the two."""
    loop = mma_loop()
    pv = loop.index("umma_bf16_tmem_a(")
    commit = loop.index("umma_commit(hdr + kVFree + 8 * st)", pv)
    wait = loop.index("wait_all(hdr + kVFree + 8 * st, (j / kIpRing) & 1)", commit)
    fence = loop.index("tc_fence_after()", wait)
    assert loop.index("issue_s(j + 2)") > fence
    assert loop.count("issue_s(") == 1


def test_p_v_begins_after_p_and_v_are_there():
    loop = mma_loop()
    assert loop.index("wait_all(hdr + kPFull + 8 * (j & 1), (j >> 1) & 1)") < loop.index("umma_bf16_tmem_a(")
    before = text()
    before = before[: before.index("for (int j = 0; j < nst && !failed; ++j) {\n        const int st")]
    assert "if (nst > 0 && !failed) failed = !v_there(0);" in before       # V_0, and V_{j+1} at the end of stage j
    assert loop.rindex("failed = !v_there(j + 1);") > loop.index("issue_s(j + 2)")


def test_converters_write_a_stage_only_after_its_readers_are_done():
    warp = text()
    warp = warp[warp.index("if (warp >= 8) {"): warp.index("} else if (warp >= 4) {")]
    for bar, first_store in (("kKFree", "ops + (c >> 1) * kIpHalf"), ("kVFree", "ops + 1024 * h + (((v_chunk + c)")):
        wait = warp.index(f"mbar_wait_parked(hdr + {bar} + 8 * st, ((j / kIpRing) - 1) & 1)")
        store = warp.index(first_store)
        arrive = warp.index(f"mbar_arrive(hdr + {bar.replace('Free', 'Full')} + 8 * st)")
        assert wait < store < warp.rindex("fence_proxy_async_smem()", 0, arrive) < arrive


def test_the_thread_that_issued_the_mmas_commits_the_last_of_them():
    """A commit follows the operations of its own thread, and which lane elect.sync names is not said."""
    source = text()
    assert re.findall(r"if \(([^;{}]*)\) umma_commit\(hdr \+ kDone\)", source) == ["elect_one()"]
    assert source.count("umma_commit(hdr + kDone)") == 1


def test_barriers_of_the_header_do_not_overlap():
    """Offsets from the ring's length: 8 bytes a slot, one after another, within the header."""
    source = text()
    ring = int(re.search(r"kIpRing = (\d+);", source).group(1))
    env = {"kIpRing": ring}
    at = {}
    for name, expr in re.findall(r"constexpr int (k\w+) = ([^;]+);", source):
        if name in ("kKFull", "kKFree", "kVFull", "kVFree", "kSFull", "kPFull", "kDone", "kQReady", "kTmemAt", "kIpHeader"):
            env[name] = at[name] = eval(expr, {}, env)                       # noqa: S307
    slots = [("kKFull", ring), ("kKFree", ring), ("kVFull", ring), ("kVFree", ring), ("kSFull", 2), ("kPFull", 2), ("kDone", 1),
             ("kQReady", 1)]
    taken = [at[n] + 8 * i for n, k in slots for i in range(k)]
    assert len(set(taken)) == len(taken) and max(taken) + 8 <= at["kTmemAt"] and at["kTmemAt"] + 4 <= at["kIpHeader"]
