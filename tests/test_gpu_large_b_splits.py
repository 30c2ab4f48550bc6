"""GPU: products of a large B (over 96 MB) with few column tiles and a long K, which the
default choice splits three to eight ways: bf16 output bit for bit, FP8 output against the
oracle quantizer's bytes."""
import numpy as np
import pytest
import torch

import oracle
from tests import gpu_util as gu
from tests.test_gpu_epilogue import BF, dg, operands, pack, small_values
from tests.test_gpu_norm import Fp8Out

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(64, 7168, 18432), (48, 5504, 18432), (33, 4096, 28672), (64, 8320, 12800),
                                   (64, 10880, 9856), (37, 5120, 25600)])
def test_bitwise(M, N, K):
    A, B, sfA, sfB, r = operands(M, N, K, M + N + K)
    bias, residual = small_values(1, N, BF), small_values(2, (M, N), BF)
    a, b, sb = gu.codes(A), gu.codes(B), gu.dev(sfB)
    z = r + bias.double().numpy()
    c = z + residual.double().numpy()
    assert np.array_equal(c.astype(np.float32), c), "the case is meant to be exact in fp32"
    rc, rs = oracle.quantize_blocks(z.astype(np.float32), 1, 128)
    for sa in (gu.dev(sfA), pack(sfA)):
        out = gu.Guarded((M, N), 5)
        fp8 = Fp8Out(M, N, sa.dtype is torch.int32)
        gu.announce(f"large B, split K: M={M} N={N} K={K} {sa.dtype}")
        for _ in range(2):  # the second call finds the arrival counters of the first
            out.out.zero_()
            dg().fp8_gemm_nt_bias_act(a, b, out.out, sa, sb, bias=bias.cuda(), residual=residual.cuda())
            torch.cuda.synchronize()
            assert out.guards_intact() and np.array_equal(out.result(), oracle.bf16_rne(c))
        dg().fp8_gemm_nt_bias_act_fp8(a, b, sa, sb, bias=bias.cuda(), codes=fp8.codes, sf=fp8.sf)
        codes, sf = fp8.result()
        assert np.array_equal(rs, sf) and np.array_equal(rc, codes)
