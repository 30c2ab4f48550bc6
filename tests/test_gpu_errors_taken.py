"""GPU: a workspace that cannot be had is reported by the call's status, and no error of it stays in
the thread: whoever asks for the last error next (torch after each of its launches) would be
told of it as its own. The product asks for a K-contiguous copy of 2^52 bytes, which the host
refuses before anything is launched."""
import numpy as np
import pytest
import torch

from tests import _block64 as blk
from tests.test_gpu_pending_error import runtime

pytestmark = pytest.mark.gpu
FAKE = 0x10000


def test_refused_workspace_leaves_no_error():
    import fp8_block_scaled_dg_amd as m
    hip = runtime()
    x, rng = torch.ones(4096, device="cuda"), torch.tensor([1, 2], device="cuda")
    torch.cuda.synchronize()
    assert hip.hipPeekAtLastError() == 0
    M, K = (1 << 30) - 1, 1 << 22  # A stored [K][M], M odd: read through a copy
    status = m.lib.dg_fp8_gemm_tn(FAKE, FAKE, FAKE, FAKE, FAKE, M, 16, K, None)
    assert m.lib.dg_status_string(status) == b"DG_ERR_LAUNCH" and b"hipMalloc" in m.lib.dg_last_error_detail()
    assert hip.hipPeekAtLastError() == 0
    # what follows is not told of it either
    m.dropout_add(x, 0.5, rng, out=x)
    y = x + 1
    assert np.array_equal(y.cpu().numpy(), np.where(blk.kept(0, 4096, 0.5, 1, 2), 3.0, 1.0))
