"""GPU: hipStreamPerThread is one handle for another stream in every thread, so that its calls of
several threads may run at once: each thread has buffers of its own there. Gradients of two launches
(partial sums, then their sum), of whole numbers, which have one answer in every order."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
PER_THREAD = ctypes.c_void_p(2)  # hipStreamPerThread


def test_threads_on_their_own_streams():
    import fp8_block_scaled_dg_amd as m
    K, n = 1024, 4
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    data = []
    for i in range(n):
        M = 2000 + 500 * i  # two launches each
        dy = torch.randint(-8, 9, (M, K), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda()
        h = torch.randint(-8, 9, (M, K), generator=torch.Generator().manual_seed(9 + i)).to(torch.bfloat16).cuda()
        mean, rstd = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
        out = [(torch.empty_like(h), torch.zeros(K, device="cuda"), torch.zeros(K, device="cuda")) for _ in range(20)]
        data.append((dy, h, mean, rstd, out, (dy.double() * h.double()).sum(0).float(), dy.double().sum(0).float()))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(n)

    def run(i):
        dy, h, mean, rstd, out, _, _ = data[i]
        start.wait()
        for dx, dw, db in out:
            s = m.lib.dg_layernorm_backward(dy.data_ptr(), None, h.data_ptr(), m.DTYPE_BF16, w.data_ptr(), m.DTYPE_BF16,
                                            mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr(),
                                            h.shape[0], K, PER_THREAD)
            if s:
                failed.append(m.lib.dg_last_error_detail())

    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for *_, out, dw, db in data:
        for _, a, b in out:
            assert torch.equal(a, dw) and torch.equal(b, db)
    m.release_workspaces()
