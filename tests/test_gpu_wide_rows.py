"""GPU: the epilogue's backward on rows of 2^29 columns and more, whose column sums do not fit
one launch (fewer than 2^32 threads, 8 a column)."""
import pytest
import torch

from tests import gpu_util as gu
from tests.test_gpu_norm import BF, dg

pytestmark = pytest.mark.gpu
N = (1 << 29) + 1152


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.synchronize()
    dg().release_workspaces()  # the partial sums: a row of N floats
    torch.cuda.empty_cache()


def test_column_sums_of_wide_rows():
    g = torch.Generator(device="cuda").manual_seed(1)
    dc = torch.randn(2, N, generator=g, device="cuda", dtype=BF)
    db = torch.full((N + 8,), 7.0, device="cuda")
    gu.announce(f"act backward M=2 N={N}")
    codes, sf, _ = dg().bias_act_backward_fp8(dc, dbias=db[4:N + 4])
    torch.cuda.synchronize()
    assert torch.equal(db[4:N + 4], dc[0].float() + dc[1].float())
    assert torch.all(db[:4] == 7) and torch.all(db[N + 4:] == 7)
    end = dc[:, N - 1024:].contiguous()
    c0, s0, d0 = dg().bias_act_backward_fp8(end)
    torch.cuda.synchronize()
    assert torch.equal(codes[:, N - 1024:].view(torch.uint8), c0.view(torch.uint8))
    assert torch.equal(sf[:, -8:], s0) and torch.equal(db[N + 4 - 1024:N + 4], d0)


def test_no_rows_write_zeros():
    db = torch.full((N + 8,), 7.0, device="cuda")
    gu.announce(f"act backward M=0 N={N}")
    dg().bias_act_backward_fp8(torch.zeros(0, N, dtype=BF, device="cuda"), dbias=db[4:N + 4])
    torch.cuda.synchronize()
    assert not db[4:N + 4].any() and torch.all(db[:4] == 7) and torch.all(db[N + 4:] == 7)
