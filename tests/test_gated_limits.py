"""CPU: the gated product refuses what none of its kernels can address. The tile kernel's 32-bit
offsets reach an up row from its gate row while (I + 256) K < 2^31, and a launch of the ring kernel
holds fewer than 2^23 tiles of 64 rows by 128 columns. No kernel is launched without a GPU, so a
size that is taken ends at the missing device."""
import pytest
import torch

FAKE = 0x10000

# the addresses are no GPU memory: only where no kernel can be launched
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")


def gated(M, I, K):
    import fp8_block_scaled_dg_amd as m
    f = FAKE
    status = m.lib.dg_fp8_gemm_nt_gated_fp8(f, f, f, f, 0, f, 0, f, f, 1, 2, f, M, I, K, None)
    return m.lib.dg_status_string(status).decode(), m.lib.dg_last_error_detail().decode()


@pytest.mark.parametrize("M,I,K", [(1 << 20, 65536, 32768), ((1 << 20) - 63, 65536, 32768), (1 << 18, 1 << 18, 1 << 13),
                                   (1 << 30, 1 << 19, 1 << 22), (1 << 30, 65536, 32768)])
def test_out_of_every_kernels_reach(M, I, K):
    status, detail = gated(M, I, K)
    assert status == "DG_ERR_UNSUPPORTED_SHAPE" and "2^31" in detail, detail


@pytest.mark.parametrize("M,I,K", [
    ((1 << 20) - 64, 65536, 32768),  # one row of tiles fewer: the ring kernel
    (1 << 20, 65536, 32512),         # the tile kernel reaches every up row
    (1 << 20, 65536 - 384, 32768), (1, 131072, 16384), (4096, 18432, 7168)])
def test_within_reach(M, I, K):
    assert gated(M, I, K)[0] in ("DG_ERR_NO_DEVICE", "DG_ERR_LAUNCH")


@pytest.mark.parametrize("config", ["pipe128x256", "gated_m16", "gated_m32", "gated_m64"])
def test_a_forced_kernel_refuses_too(config, monkeypatch):
    monkeypatch.setenv("DG_FORCE_CONFIG", config)
    assert gated(1 << 20, 65536, 32768)[0] == "DG_ERR_UNSUPPORTED_SHAPE"
