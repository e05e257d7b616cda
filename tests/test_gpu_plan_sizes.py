"""pa_plan_step about the sizes where its shared memory needs the opt-in: the sums of S sequences take 9 S + 24
bytes beside the kernel's own 256 (512 with CTAs of 1,024 threads), and 48 KiB of both together go without.
Each case runs in a process of its own: a device stays opted in once a call has asked for it."""

from __future__ import annotations

import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
TESTS = Path(__file__).resolve().parent

PROGRAM = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
import numpy as np
import test_gpu_serving as H
from paged_kv_cache_244_gb300 import binding
for in_place in ({first}, {second}):
    case = H.random_plan(np.random.default_rng({seqs}), {seqs}, 40, {new}, pad=3)
    assert (case[-1] > 311296) == ({new} > 100), case[-1]
    H.check_plan(binding, *case, in_place=in_place)
print("equal")
"""


@pytest.mark.parametrize("seqs,new,in_place", [(5430, 3, False), (5431, 3, False), (5440, 3, True), (5458, 3, False), (5459, 3, True),
                                               (5401, 130, False), (5402, 130, False), (5440, 130, True), (5459, 130, False)])
def test_plan_in_a_fresh_process(seqs, new, in_place):
    text = PROGRAM.format(tests=str(TESTS), root=str(TESTS.parent), seqs=seqs, new=new, first=in_place, second=not in_place)
    r = subprocess.run([sys.executable, "-c", text], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stdout + r.stderr[-2000:]
