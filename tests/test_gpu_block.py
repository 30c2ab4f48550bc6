"""GPU: layer norm, gated product and dropout together, as a stack of feed-forward layers uses them
(examples/prenorm_gated.py): both passes against fp32 torch, in a captured graph, on two streams
at once; the two ways their arguments are checked; and products past 32-bit offsets.

Distances in the 2-norm. An e4m3fn rounding is at most 2^-4, uniform within half a step: 0.036. One
layer's forward pass quantizes the norm (through gate and up, each 0.036, the gate's by at most
1.05 of it for a smooth activation of a unit normal: 0.052 together) and the gated values: 0.063.
Its backward pass quantizes two gradients, and sees the first forward one in up and in the
activation's slope (at most 1.7 x 0.036 together): 0.079, of which the norm's backward takes two
projections off. Through two layers the second's input is 0.063 off, its result sqrt(2 x 0.063^2
+ 0.063^2) = 0.109 and its slopes 1.7 x 0.109: 0.19. The tolerances are half as much again."""
import importlib.util
import os
import threading

import pytest
import torch

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FORWARD, BACKWARD = {1: 0.095, 2: 0.165}, {1: 0.12, 2: 0.29}


def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "prenorm_gated.py")
    spec = importlib.util.spec_from_file_location("prenorm_gated", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def inputs(tokens, hidden, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(tokens, hidden, generator=g).to(BF).cuda() for _ in range(2)]


@pytest.mark.parametrize("tokens,hidden,ffn,layers,activation,p", [
    (1, 512, 1024, 1, "silu", 0.25), (7, 384, 640, 1, "gelu", 0.0), (64, 2048, 1024, 2, "silu", 0.1),
    (257, 1152, 2048, 1, "gelu_tanh", 0.25), (1000, 1024, 1408, 2, "gelu", 0.1)])
def test_stack_matches_fp32(tokens, hidden, ffn, layers, activation, p):
    ex = example()
    model = ex.PreNormGated(hidden, ffn, layers, activation, p, seed=tokens)
    gu.announce(f"stack {tokens} x {hidden} x {ffn} x {layers} {activation} p={p}")
    far = ex.compare(model, *inputs(tokens, hidden, tokens))
    torch.cuda.synchronize()
    for name, d in far.items():
        assert d <= (FORWARD if name == "out" else BACKWARD)[layers], far
    # the sum of the dropped gradient itself, in fp32
    assert far[f"db2[{layers - 1}]"] <= 2.0 ** -20, far


def step(model, x, dout):
    out, saved = model.forward(x)
    dx, grads = model.backward(dout, saved)
    return [out, dx] + [g[k] for g in grads for k in g]


def test_training_graph_draws_new_masks():
    ex = example()
    model = ex.PreNormGated(512, 1024, 2, "silu", 0.3, seed=5)
    for tokens in (300, 700):  # column sums in the same launch, and in a second one
        x, dout = inputs(tokens, 512, 6)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(model, x, dout)  # sizes the stream's workspace
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step(model, x, dout)
        before = None
        for r in range(3):
            x2, dout2 = inputs(tokens, 512, 10 + r // 2)
            x.copy_(x2), dout.copy_(dout2)
            model.rng.copy_(torch.tensor([7, 2 ** 40 + 16 * r]))
            want = step(model, x2, dout2)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), r
            if r == 1:  # the first replay's inputs, other masks
                assert not torch.equal(got[0], before)
            before = got[0].clone()


def test_two_streams_at_once():
    ex = example()
    models = [ex.PreNormGated(1024, 1408, 2, "gelu", 0.2, seed=s) for s in (1, 2)]
    data = [inputs(t, 1024, t) for t in (48, 600)]
    want = [step(m, *d) for m, d in zip(models, data)]
    torch.cuda.synchronize()
    got, errors = [[], []], []
    streams = [torch.cuda.Stream() for _ in models]

    def run(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(5):
                    got[i].append(step(models[i], *data[i]))
        except Exception as e:  # a failure here would be lost with the thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i in range(2):
        assert len(got[i]) == 5
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_threads_on_one_stream():
    # gradients of two launches (partial sums, then their sum) and a product that splits K: all of
    # them use the stream's one buffer of partials
    m = dg()
    stream = torch.cuda.Stream()
    K = 1024
    w = torch.ones(K, dtype=BF, device="cuda")
    data, want = [], []
    for i, M in enumerate((900, 1500)):
        h, dy = inputs(M, K, 20 + i)
        data.append((dy, h, w, torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")))
        want.append(m.layernorm_backward(*data[i]))
    a, b = signs(5, 64, 7168), signs(6, 2112, 7168)
    sa, sb, c0 = torch.ones(64, 56, device="cuda"), torch.ones(17, 56, device="cuda"), \
        torch.empty(64, 2112, dtype=BF, device="cuda")
    m.fp8_gemm_nt(a, b, c0, sa, sb)
    torch.cuda.synchronize()
    got, errors = [[], [], []], []

    def run(i):
        try:
            with torch.cuda.stream(stream):
                for _ in range(100):
                    if i < 2:
                        got[i].append(m.layernorm_backward(*data[i]))
                    else:
                        c = torch.empty_like(c0)
                        m.fp8_gemm_nt(a, b, c, sa, sb)
                        got[i].append(c)
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i in range(2):
        assert len(got[i]) == 100
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(g, want[i])), i
    assert len(got[2]) == 100 and all(torch.equal(c, c0) for c in got[2])


def test_python_checks_and_native_ones_pass_the_same_calls(monkeypatch):
    m = dg()
    ex = example()
    model = ex.PreNormGated(640, 384, 2, "gelu_tanh", 0.1, seed=3)
    x, dout = inputs(33, 640, 4)
    want = step(model, x, dout)

    class Never:
        def __getattr__(self, name):
            return lambda *args: None

    monkeypatch.setattr(m, "_marshal", Never())
    got = step(model, x, dout)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_whole_numbers_for_fractions():
    m = dg()
    x, _ = inputs(5, 256, 1)
    w, rng = torch.ones(256, dtype=BF, device="cuda"), torch.tensor([1, 2], device="cuda")
    assert torch.equal(m.dropout_add(x, 0, None), x)
    a, sa = m.layernorm_fp8_1x128(x, w, eps=1, dropout_p=0, rng=rng)
    b, sb = m.layernorm_fp8_1x128(x, w, eps=1.0)
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(sa, sb)


def signs(seed, n, K):
    """+1 and -1, e4m3fn [n, K]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (n, K), dtype=torch.uint8, device="cuda", generator=g)
    return c.bitwise_and_(0x80).bitwise_or_(0x38).view(torch.float8_e4m3fn)


def same(got, part, rows, cols):
    (codes, sf, pre), (c, s, q) = got, part
    I, Is = codes.shape[1], c.shape[1]
    assert torch.equal(codes.view(torch.uint8)[rows, cols], c.view(torch.uint8))
    assert torch.equal(sf[rows, cols.start // 128:cols.stop // 128], s)
    assert torch.equal(pre[rows, cols], q[:, :Is])
    assert torch.equal(pre[rows, I + cols.start:I + cols.stop], q[:, Is:])


def gated(a, b):
    """Scales of one: sums of K signs, exact in every order."""
    M, (N, K) = a.shape[0], b.shape
    pre = torch.empty(M, N, dtype=BF, device="cuda")
    gu.announce(f"gated M={M} I={N // 2} K={K}")
    codes, sf = dg().fp8_gemm_nt_gated_fp8(a, b, torch.ones(M, K // 128, device="cuda"),
                                           torch.ones(N // 128, K // 128, device="cuda"), activation="silu", pre=pre)
    return codes, sf, pre


def test_gated_weights_past_32_bit_offsets():
    # gate and up rows 2^31 bytes apart: out of the tile kernel's reach, the ring kernel's runs
    I, K = 131072, 16384
    b = signs(1, 2 * I, K)
    for M in (3, 70):
        a = signs(2, M, K)
        got = gated(a, b)
        for n0 in (0, I // 2, I - 256):
            part = gated(a, torch.cat([b.view(torch.uint8)[s:s + 256] for s in (n0, I + n0)]).view(torch.float8_e4m3fn))
            same(got, part, slice(0, M), slice(n0, n0 + 256))


@pytest.mark.parametrize("config", ["", "gated_m64"])
def test_gated_rows_past_32_bit_offsets(config, monkeypatch):
    monkeypatch.setenv("DG_FORCE_CONFIG", config)
    M, I, K = 270007, 256, 16384
    a, b = signs(3, M, K), signs(4, 2 * I, K)
    got = gated(a, b)
    for rows in (slice(0, 100), slice(131040, 131140), slice(262100, 262200), slice(M - 100, M)):
        same(got, gated(a[rows], b), rows, slice(0, I))
