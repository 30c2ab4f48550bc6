"""CPU: the form that the gated product chooses, as DG_PRINT_CONFIGS names it, is within a tenth of the
best form measured (us in a graph, weights from HBM, MI355X). The choice is the host's alone and is
printed before the first HIP call, so a process without a GPU and fake addresses do."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
assert torch.cuda.device_count() == 0, "fake addresses: no GPU may be visible"
import fp8_block_scaled_dg_amd as dg
F = 0x10000
for shape in sys.argv[2:]:
    M, I, K = map(int, shape.split("x"))
    assert dg.lib.dg_fp8_gemm_nt_gated_fp8(F, F, F, F, 0, F, 0, F, None, 0, 2, None, M, I, K, None) != 0
"""

# (M, I, K): {(rows of a tile, K splits; (0, 1): the tile kernel): us}
MEASURED = {
    (1, 2048, 7168): {(0, 1): 25.4, (16, 1): 37.9, (16, 2): 23.3, (16, 3): 18.9, (16, 4): 15.5, (16, 5): 14.7, (16, 6): 13.7,
                      (16, 7): 12.8, (16, 10): 13.1, (16, 14): 13.6},
    (16, 2048, 7168): {(0, 1): 26.9, (16, 1): 39.4, (16, 2): 24.4, (16, 3): 19.7, (16, 4): 16.3, (16, 5): 15.4, (16, 6): 14.4,
                       (16, 7): 13.6, (16, 10): 13.6, (16, 14): 14.0, (32, 14): 15.7},
    (64, 2048, 7168): {(0, 1): 28.2, (16, 1): 37.7, (16, 2): 23.6, (16, 4): 16.3, (32, 1): 40.2, (32, 4): 17.3, (32, 7): 15.6,
                       (64, 1): 46.3, (64, 4): 21.2, (64, 7): 19.5, (64, 10): 21.4, (64, 14): 23.8},
    (64, 8192, 8192): {(0, 1): 48.4, (16, 1): 47.7, (32, 1): 50.8, (32, 2): 38.8, (64, 1): 55.2, (64, 2): 40.6, (64, 3): 32.2,
                       (64, 4): 31.7},
    (1, 1024, 4096): {(0, 1): 19.1, (16, 1): 22.6, (16, 4): 10.9, (16, 6): 10.0, (16, 8): 9.1, (16, 16): 9.9},
    (1000, 2048, 7168): {(0, 1): 46.3, (64, 1): 43.9},
    (2048, 2816, 4096): {(0, 1): 67.3, (64, 1): 76.0},
}


@pytest.fixture(scope="module")
def chosen():
    env = dict(os.environ, DG_PRINT_CONFIGS="1", HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    env.pop("DG_FORCE_CONFIG", None)
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT, *("x".join(map(str, s)) for s in MEASURED)],
                       env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = {}
    for line in r.stderr.splitlines():
        m = re.match(r"\[dg\] dense M=(\d+) N=(\d+) K=(\d+) G=1 -> (\w+) \(gated(?:, (\d+) K splits)?\)", line)
        if m:
            M, N, K = map(int, m.group(1, 2, 3))
            rows = 0 if m.group(4).startswith("pipe") else int(m.group(4).removeprefix("gated_m"))
            out[M, N // 2, K] = rows, int(m.group(5) or 1)
    return out


@pytest.mark.parametrize("shape", list(MEASURED))
def test_choice_is_near_the_best_form(chosen, shape):
    times = MEASURED[shape]
    assert chosen[shape] in times, chosen[shape]
    assert times[chosen[shape]] <= 1.1 * min(times.values()), chosen[shape]


def test_one_row_takes_no_more_splits_than_pay(chosen):
    assert chosen[1, 2048, 7168] == chosen[16, 2048, 7168] == (16, 7)
