"""GPU: dropout's gradient with bias gradients in two launches over several strips of 1024 columns:
whole and ragged last strips, ragged last row groups, partial sums of every strip."""
import numpy as np
import pytest
import torch

from tests import _block64 as blk
from tests import _ops64 as ops
from tests import gpu_util as gu
from tests.test_gpu_dropout import OFFSET, SEED, rng_state
from tests.test_gpu_norm import BF, F32, Fp8Out, hidden

pytestmark = pytest.mark.gpu


# one launch sums up to 640 rows and 3 * 2^21 values: all of these take two
@pytest.mark.parametrize("M,K", [(1000, 2048), (700, 1152), (641, 1920), (700, 16384), (500, 16512), (2100, 3200)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_partials_of_several_strips(M, K, dtype):
    import fp8_block_scaled_dg_amd as dg
    dy = hidden(M * K, M, K, dtype)
    for p, packed, sub in ((0.1, True, 3), (0.0, False, 0)):
        out = Fp8Out(M, K, packed)
        db = torch.full((K + 8,), 5.0, device="cuda")
        gu.announce(f"dropout backward {dtype} M={M} K={K} p={p}")
        dg.dropout_backward_fp8(dy.cuda(), p, rng_state(), sub, codes=out.codes, sf=out.sf, dbias=db[4:K + 4])
        codes, sf = out.result()
        assert torch.all(db[:4] == 5) and torch.all(db[-4:] == 5)
        q = blk.dropout(dy.double().numpy(), p, SEED, OFFSET, sub)
        assert not (codes[q == 0] & 0x7F).any(), "dropped elements"
        dq = 2 * ops.U * np.abs(q) * (blk.threshold(p) > 0) + 1e-300
        blk.check_fp8(q, dq, codes, sf, f"{M}x{K} p={p}")
        err = np.abs(db[4:K + 4].double().cpu().numpy() - q.sum(0))
        assert np.all(err <= blk.COL * np.abs(q).sum(0) + dq.sum(0) + 1e-45)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_launches_give_one_launchs_sums(dtype):
    # whole numbers: exact in every order, so both ways have one possible answer
    import fp8_block_scaled_dg_amd as dg
    K = 2304
    dy = torch.randint(-8, 9, (1500, K), generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    _, _, db = dg.dropout_backward_fp8(dy, 0.0, None)
    parts = [dg.dropout_backward_fp8(dy[i:i + 500].contiguous(), 0.0, None)[2] for i in (0, 500, 1000)]
    torch.cuda.synchronize()
    assert torch.equal(db, sum(parts)) and torch.equal(db, dy.double().sum(0).float())
