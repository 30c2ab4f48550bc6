"""GPU: dropout (dg_dropout_add) and its gradient with an FP8 output (dg_dropout_backward_fp8)
against the definition in 64 bits (tests/_block64.py). The mask has to agree element by element:
x is chosen nonzero, so that every zero of an output without a residual is a dropped element."""
import numpy as np
import pytest
import torch

from tests import _block64 as blk
from tests import _ops64 as ops
from tests import gpu_util as gu
from tests.test_gpu_norm import BF, F32, Fp8Out, hidden
from tests.test_gpu_quant import GuardedBytes

pytestmark = pytest.mark.gpu
SEED, OFFSET = -0x123456789ABCDEF, (1 << 63) - 5


def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def rng_state(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def nonzero(seed, n, dtype):
    x = torch.randn(n, generator=torch.Generator().manual_seed(seed)).to(dtype)
    return torch.where(x == 0, torch.ones((), dtype=dtype), x)


def close(got, want, slack, dtype):
    """Within the fp32 roundings `slack` and the output's own rounding."""
    own = ops.bf16_slack(np.abs(want) + slack) if dtype == BF else ops.U * np.abs(want) + 2.0 ** -149
    return np.all(np.abs(got - want) <= slack + own)


@pytest.mark.parametrize("n", [1, 3, 7, 8, 9, 255, 256, 257, 511, 512, 513, 4097, 1 << 16, 1234567])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_add(n, dtype):
    x, r = nonzero(n, n, dtype), nonzero(n + 1, n, dtype)
    for p, res, sub in ((0.1, False, 0), (0.5, True, 1 << 40), (2.0 ** -16, True, -1), (1 - 2.0 ** -16, False, 9),
                        (0.0, True, 0)):
        out = GuardedBytes(n * x.element_size(), 5)
        o = out.view(dtype, (n,))
        gu.announce(f"dropout {dtype} n={n} p={p} residual={res}")
        got = dg().dropout_add(x.cuda(), p, rng_state(), sub, residual=r.cuda() if res else None, out=o)
        torch.cuda.synchronize()
        assert got is o and out.guards_intact()
        want = blk.dropout(x.double().numpy(), p, SEED, OFFSET, sub)
        slack = 2 * ops.U * np.abs(want) * (blk.threshold(p) > 0)
        if res:
            want = want + r.double().numpy()
            slack = slack + ops.U * np.abs(want)
        else:
            assert np.array_equal(o.float().cpu().numpy() == 0, want == 0), "mask"
        assert close(o.double().cpu().numpy(), want, slack, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_add_in_place_and_shapes(dtype):
    x, r = nonzero(1, 3003, dtype).cuda().view(3, 7, 11, 13), nonzero(2, 3003, dtype).cuda().view(3, 7, 11, 13)
    want = dg().dropout_add(x, 0.3, rng_state(), 4, residual=r)
    for which in ("x", "r"):
        a, b = x.clone(), r.clone()
        out = a if which == "x" else b
        assert dg().dropout_add(a, 0.3, rng_state(), 4, residual=b, out=out) is out
        torch.cuda.synchronize()
        assert torch.equal(out, want) and want.shape == x.shape
    empty = dg().dropout_add(x[:0], 0.3, rng_state())
    assert empty.shape == (0, 7, 11, 13)


def test_dropout_drops_what_is_not_finite():
    x = torch.full((4096,), float("nan"))
    x[::2] = float("inf")
    got = dg().dropout_add(x.cuda(), 0.5, rng_state()).cpu().numpy()
    keep = blk.kept(0, 4096, 0.5, SEED, OFFSET)
    assert np.all(got[~keep] == 0)
    assert np.all(np.isnan(got[1::2][keep[1::2]])) and np.all(got[::2][keep[::2]] == np.inf)


def test_dropout_past_32_bit_indexes():
    n = (1 << 32) + 4096 + 5
    x = torch.ones(n, dtype=BF, device="cuda")
    gu.announce(f"dropout n={n}")
    out = dg().dropout_add(x, 0.25, rng_state())
    torch.cuda.synchronize()
    for first, count in ((0, 4096), ((1 << 31) - 512, 2048), (1 << 32, 4096 + 5)):
        assert np.array_equal(out[first:first + count].float().cpu().numpy() != 0,
                              blk.kept(first, count, 0.25, SEED, OFFSET)), first
    for M, K in (((1 << 32) // 8192 + 1, 8192),):
        y = x[:M * K] if M * K <= n else torch.ones(M * K, dtype=BF, device="cuda")
        codes, _, _ = dg().dropout_backward_fp8(y.view(M, K), 0.25, rng_state(), need_dbias=False)
        torch.cuda.synchronize()
        last = codes[-1].view(torch.uint8).cpu().numpy()
        assert np.array_equal(last != 0, blk.kept((M - 1) * K, K, 0.25, SEED, OFFSET))


@pytest.mark.parametrize("M,K", [(1, 128), (1, 18432), (3, 384), (5, 1024), (130, 2048), (257, 1152), (4100, 256),
                                 (64, 7168), (130, 12288)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_backward(M, K, dtype):
    dy = hidden(M * K, M, K, dtype)
    for p, packed, sub in ((0.1, False, 3), (0.6, True, 0), (0.0, False, 0)):
        out = Fp8Out(M, K, packed)
        db = torch.full((K + 8,), 5.0, device="cuda")
        gu.announce(f"dropout backward {dtype} M={M} K={K} p={p}")
        dg().dropout_backward_fp8(dy.cuda(), p, rng_state(), sub, codes=out.codes, sf=out.sf, dbias=db[4:K + 4])
        codes, sf = out.result()
        assert torch.all(db[:4] == 5) and torch.all(db[-4:] == 5)
        q = blk.dropout(dy.double().numpy(), p, SEED, OFFSET, sub)
        assert not (codes[q == 0] & 0x7F).any(), "dropped elements"
        dq = 2 * ops.U * np.abs(q) * (blk.threshold(p) > 0) + 1e-300
        blk.check_fp8(q, dq, codes, sf, f"{M}x{K} p={p}")
        err = np.abs(db[4:K + 4].double().cpu().numpy() - q.sum(0))
        assert np.all(err <= blk.COL * np.abs(q).sum(0) + dq.sum(0) + 1e-45)


def test_dropout_backward_forms_agree_with_the_forward_mask():
    dy = hidden(1, 300, 1152, BF).cuda()
    c0, s0, db = dg().dropout_backward_fp8(dy, 0.2, rng_state(), 11)
    c1, s1, none = dg().dropout_backward_fp8(dy, 0.2, rng_state(), 11, need_dbias=False, ue8m0=True)
    y = dg().dropout_add(dy.float(), 0.2, rng_state(), 11)
    c2, s2 = dg().quantize_fp8_1x128(y)
    torch.cuda.synchronize()
    assert none is None and db.shape == (1152,)
    assert torch.equal(c0.view(torch.uint8), c1.view(torch.uint8))
    # -0 of a dropped negative value and the quantizer's 0 differ in sign only
    assert torch.equal(c0.view(torch.uint8) & 0x7F, c2.view(torch.uint8) & 0x7F) and torch.equal(s0, s2)
    e = torch.zeros(0, 256, device="cuda")
    c, _, db = dg().dropout_backward_fp8(e, 0.2, rng_state(), dbias=torch.full((256,), 9.0, device="cuda"))
    torch.cuda.synchronize()
    assert c.shape == (0, 256) and not db.any()


def test_dropout_device_state_is_read_when_the_kernel_runs():
    x, state = torch.ones(10000, device="cuda"), rng_state(5, 0)
    a = dg().dropout_add(x, 0.5, state)
    state[1] += 1
    b = dg().dropout_add(x, 0.5, state)
    c = dg().dropout_add(x, 0.5, rng_state(5, 0), 1)
    torch.cuda.synchronize()
    assert not torch.equal(a, b) and torch.equal(b, c)
    assert np.array_equal(a.cpu().numpy() != 0, blk.kept(0, 10000, 0.5, 5, 0))


def test_binding_refuses_other_states():
    x = torch.ones(16, device="cuda")
    with pytest.raises(TypeError, match="rng must be torch.int64"):
        dg().dropout_add(x, 0.1, torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="rng has shape"):
        dg().dropout_add(x, 0.1, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="rng must be a GPU tensor"):
        dg().dropout_add(x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous"):
        dg().dropout_add(torch.ones(4, 4, device="cuda").t(), 0.1, rng_state())
    with pytest.raises(dg().DGError, match="16-byte aligned"):
        dg().dropout_add(torch.ones(17, device="cuda")[1:], 0.1, rng_state())
    with pytest.raises(dg().DGError, match="dropout_p"):
        dg().dropout_add(x, 1.0, rng_state())
    with pytest.raises(dg().DGError, match="NULL rng"):
        dg().dropout_add(x, 0.1, None)
