"""CPU: the kernel that the fused-epilogue calls choose, as DG_PRINT_CONFIGS names it. The
choice is the host's alone and is printed before the first HIP call, so a process without a
GPU and fake addresses do; the launch that follows fails with a status."""
import os
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
    M, N, K = map(int, shape.split("x"))
    print("bf16", shape, flush=True)
    assert dg.lib.dg_fp8_gemm_nt_bias_act(F, F, F, F, 0, F, None, 0, 0, None, None, M, N, K, None) != 0
    if N % 128 == 0:
        assert dg.lib.dg_fp8_gemm_nt_bias_act_fp8(F, F, F, F, 0, F, 0, F, None, 0, 0, None, M, N, K, None) != 0
"""


def choices(shapes):
    """{(M, N, K, fp8?): configuration}."""
    env = dict(os.environ, DG_PRINT_CONFIGS="1", HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    env.pop("DG_FORCE_CONFIG", None)
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT, *("x".join(map(str, s)) for s in shapes)],
                       env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = {}
    for line in r.stderr.splitlines():
        if line.startswith("[dg] dense"):
            f = line.split()
            size = tuple(int(t.split("=")[1]) for t in f[2:5])
            out[size + ("FP8" in line,)] = f[7]
    return out


# the streamed form adds two splits of 33 to 64 rows: a B that wants more is not streamed
SPLIT = [(64, 7168, 18432), (64, 5120, 25600), (64, 4096, 24576), (64, 10240, 10496), (48, 5504, 18432),
         (33, 4096, 28672), (40, 8192, 14336), (64, 10880, 9856)]
STREAM = [(64, 12288, 8192), (64, 16384, 7168), (64, 18432, 7168), (33, 24576, 4224), (32, 7168, 18432),
          (16, 5504, 18432), (1, 4096, 28672)]


def test_large_b_is_streamed_unless_it_wants_more_splits():
    got = choices(SPLIT + STREAM)
    want = {s + (fp8,): name for sizes, name in ((SPLIT, "ring_n128"), (STREAM, "ring_n128_wide"))
            for s in sizes for fp8 in (False, True)}
    assert got == want


@pytest.mark.parametrize("M", [33, 64])
def test_no_step_at_the_size_of_a_large_b(M):
    # either side of 96 MB, FP8 output: the same kernel for the same number of column tiles
    got = choices([(M, 4096, 24448), (M, 4096, 24576), (M, 5376, 18432), (M, 5504, 18432)])
    assert {v for k, v in got.items() if k[3]} == {"ring_n128"}


def test_more_tiles_than_a_launch_holds_threads_for():
    # the ring kernel launches a workgroup of 512 threads per tile, fewer than 2^32 in all
    got = choices([(1 << 30, 16, 128), ((1 << 29) + 640, 256, 128), (1 << 20, 16, 128)])
    assert got[(1 << 30, 16, 128, False)] == "pipe128x256"
    assert got[((1 << 29) + 640, 256, 128, False)] == got[((1 << 29) + 640, 256, 128, True)] == "pipe128x256"
    assert got[(1 << 20, 16, 128, False)].startswith("ring")
