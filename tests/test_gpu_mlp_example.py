"""The pre-norm MLP example: the fused calls together, against fp32 torch.

An e4m3fn rounding has a relative error of at most 2^-4, uniform within half a step, so its
2-norm error is at most 2^-4 / sqrt(3) = 0.036. Two activations are quantized in the forward
pass (0.051 together; the activation's slope is at most 1.13 and raises the first to 0.041),
and two gradients in the backward pass, which also sees the first forward one through the
activation's slope: four at 0.041, in quadrature 0.082, doubled because a gelu value can move
by more than its argument's relative error and the norm's backward subtracts two parts."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
FORWARD, BACKWARD = 0.09, 0.165


def example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "prenorm_mlp.py")
    spec = importlib.util.spec_from_file_location("prenorm_mlp", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def inputs(tokens, hidden, seed):
    rng = torch.Generator().manual_seed(seed)
    return [torch.randn(tokens, hidden, generator=rng).to(torch.bfloat16).cuda() for _ in range(3)]


@pytest.mark.parametrize("tokens,hidden,ffn,activation", [
    (1, 512, 1024, "silu"), (7, 256, 640, "relu"), (64, 2048, 1024, "gelu"),
    (257, 1152, 2048, "gelu_tanh"), (1000, 1024, 2048, "gelu")])
def test_mlp_matches_fp32(tokens, hidden, ffn, activation):
    ex = example()
    mlp = ex.PreNormMLP(hidden, ffn, activation, seed=tokens)
    far = ex.compare(mlp, *inputs(tokens, hidden, tokens))
    torch.cuda.synchronize()
    for name, d in far.items():
        assert d <= (FORWARD if name == "mlp(h)" else BACKWARD), far
    assert far["db2"] <= 2.0 ** -20  # the sum of dy itself, in fp32


def test_mlp_training_graph_replays():
    ex = example()
    mlp = ex.PreNormMLP(512, 1024, "gelu", seed=5)
    x, r, dy = inputs(300, 512, 6)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        mlp.backward(dy, mlp.forward(x, r)[1])  # sizes the stream's workspace
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y, saved = mlp.forward(x, r)
        dx, grads = mlp.backward(dy, saved)
    for seed in range(3):
        x2, r2, dy2 = inputs(300, 512, 10 + seed)
        x.copy_(x2), r.copy_(r2), dy.copy_(dy2)
        y0, s0 = mlp.forward(x2, r2)
        dx0, g0 = mlp.backward(dy2, s0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(dx, dx0)
        assert all(torch.equal(grads[k], g0[k]) for k in grads)
