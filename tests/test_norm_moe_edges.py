"""Edges of the layer norm and of the experts' step."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from test_norm_moe import cuda  # noqa: F401 (a fixture)

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------- the experts' general path launches
# A launch may use 48 KB of shared memory, static and dynamic together, unless
# its limit was raised.  These steps' tables need between what the static arrays
# leave of that and 32 KB, in a process that has made no larger call.
FIRST_GENERAL_CALLS = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import associative_algebra_block_b200 as aal
from test_norm_moe import Moe
for n, shape in enumerate({shapes!r}):
    m = Moe(*shape[:-1], seed=n, pad=shape[-1])
    if {captured!r}:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            m.run()
        g.replay()
    else:
        m.run()
    assert aal.aal_get_device_status() == aal.AAL_OK
    assert aal.aal_last_path() == aal.AAL_PATH_GENERAL
    m.check()
"""


def _general_tables(B, E, k):
    """Dynamic shared memory of the general gate/up and down kernels."""
    slots = B * k
    used = min(slots, E)
    passes = min(slots, used + slots // 8)
    up = 16 * passes + 4 * ((2 + (B + 31) // 32) * E + 4 * slots + B)
    up = (up + 15) // 16 * 16
    return up, up + B * 32 * 4


# each process: a step of every form of the kernels (fp32 vectors, fp32 and bf16 by elements)
GENERAL_BANDS = {
    "up and down": [(3, 2048, 8, 32, 24, "Q", 1, "f32", 0), (3, 2048, 8, 34, 22, "Q", 2, "f32", 1),
                    (3, 2048, 8, 33, 17, "Q", 1, "bf16", 0)],
    "down": [(80, 128, 8, 32, 48, "Q", 2, "f32", 0), (90, 24, 8, 30, 26, "Q", 2, "f32", 1),
             (110, 16, 4, 40, 24, "Q", 2, "bf16", 0)],
    "down alone, few experts": [(128, 8, 3, 64, 32, "Q", 1, "f32", 0), (121, 8, 3, 45, 27, "Q", 3, "f32", 0),
                                (128, 8, 3, 40, 24, "Q", 2, "bf16", 0)],
    "up": [(120, 128, 8, 32, 24, "Q", 1, "f32", 0), (128, 128, 8, 27, 33, "Q", 3, "f32", 0),
           (116, 128, 8, 66, 34, "Q", 2, "bf16", 1)],
}


@gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("band", GENERAL_BANDS)
def test_general_experts_launch_as_the_first_calls_of_a_process(cuda, band, captured):
    shapes = GENERAL_BANDS[band]
    for B, E, k, *_ in shapes:
        sizes = _general_tables(B, E, k)
        assert any(22272 < s <= 32768 for s in sizes), sizes
    script = FIRST_GENERAL_CALLS.format(root=ROOT, tests=os.path.join(ROOT, "tests"), shapes=shapes, captured=captured)
    done = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
