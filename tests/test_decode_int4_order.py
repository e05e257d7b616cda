"""What the feeder and the consumers of the 4-bit cache's decode have to keep, checked on their source: what breaks it is a
hang or a race in shared memory, which no run shows for certain."""

from __future__ import annotations

import re
from pathlib import Path

SOURCE = Path(__file__).resolve().parents[1] / "paged_kv_cache_244_gb300" / "csrc" / "paged_decode_int4.cu"


def text() -> str:
    return re.sub(r"//[^\n]*", "", SOURCE.read_text())


def feeder() -> str:
    source = text()
    loop = source[source.index("while (__any_sync(kFullMask, rel < len)) {"):]
    return loop[: loop.index("return;")]


def test_the_feeders_lanes_leave_their_loop_together():
    """The loop's votes name the whole warp, so what ends it is one vote for all lanes, not what each has read by itself."""
    exits = re.findall(r"if \(([^;{}]*(?:\([^;{}]*\))?)\) (?:break;|\{\s*if \(lane == 0\)[^}]*break;)", feeder())
    assert len(exits) == 2 and feeder().count("break;") == 2
    assert all(e.startswith("__any_sync(kFullMask, ") for e in exits), exits


def test_a_stage_is_filled_only_after_its_consumer_has_released_it():
    loop = feeder()
    release = loop.index("if (ready && fills >= n_st) ready = mbar_test(bar + 8, phase);")
    assert release < loop.index("make_int4(seg") < loop.index("mbar_arrive_expect_tx(bar, bytes)") < loop.index("bulk_copy_g2s(")


def test_a_consumer_releases_a_stage_behind_its_fence():
    source = text()
    loop = source[source.index("left -= consume(at);"):]
    assert loop.index("fence_proxy_async_smem();") < loop.index("__syncwarp();") < loop.index("if (lane == 0) mbar_arrive(bar + 8);")


def test_copies_in_flight_land_before_the_feeder_leaves():
    source = text()
    drain = "for (int k = max(0, fills - n_st); k < fills; ++k) mbar_wait_bounded(full_bars + 16 * (k % n_st), (k / n_st) & 1);"
    assert drain in source
    assert source.index(drain) < source.index("return;", source.index("while (__any_sync(kFullMask, rel < len)) {"))


def test_every_call_has_the_same_consumers():
    """11 warps at the limits of a call (8192 sequences, 8 heads a group), so none have fewer: the count is a constant."""
    source = text()
    number = {k: int(v) for k, v in re.findall(r"constexpr int (kDiConsumers|kDiMaxRing) = (\d+);", source)}
    smem = eval(re.search(r"kDiSmemMax = ([\d* ]+);", source).group(1))          # noqa: S307
    fixed = number["kDiConsumers"] * number["kDiMaxRing"] * 16 + 16 + (8193 * 4 + 15) // 16 * 16 + 8192
    stage = 32 + 2 * 2208 + 8 * 256 + 512 + 2 * 256
    assert (smem - fixed) // stage >= 2 * number["kDiConsumers"]
    assert re.search(r"static_assert\(\(kDiSmemMax - kDiPrefixOff - prefix_bytes\(kMaxDecodeSeqs\)\) / di_stage\(8, true\) >= 2 \* kDiConsumers", source)
    launch = source[source.index("cudaError_t launch_decode_int4("):]
    assert "warps = min(" not in launch and "static_cast<int>(ctas) * kDiConsumers" in launch
