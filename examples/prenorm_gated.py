"""A stack of pre-norm gated feed-forward layers with dropout on FP8 weights, forward and backward,
out of the library's calls. With y_0 = x and h_0 = 0, layer l = 1 .. L:

    h_l = h_(l-1) + dropout(y_(l-1))
    y_l = W2 (act(Wg n + bg) * (Wu n + bu)) + b2,   n = layernorm(h_l)

and the result is h_L + dropout(y_L).

Forward, three launches a layer: the layer norm drops, adds and writes the FP8 operand of the
gate and up projections (one product of the stacked weights [Wg; Wu], whose epilogue adds the
biases, gates and writes W2's FP8 operand), then W2's product with its bias. Backward, five calls: dropout's
gradient as W2's FP8 operand with b2's gradient, the product by W2, the gate's backward with its bias
gradients, the product by [Wg; Wu], the layer norm's backward, which adds the residual stream's
gradient. Masks are drawn again from rng = (seed, offset) on the GPU; the L + 1 places that drop use
subsequences 0 .. L, and a mask depends on offset + subsequence, so that advance() counts the offset
up by L + 1 after a step (captured with it, each replay draws new masks). The projections stay
frozen: their gradients contract over tokens, along which the FP8 gradients have no scale blocks.

    python examples/prenorm_gated.py [--tokens 4096] [--hidden 2048] [--ffn 7168] [--layers 2]
                                     [--activation silu] [--dropout 0.1]

prints the time of both passes and how far their results lie from fp32 torch with the same
(dequantized) weights and masks. --tokens 1 is a decoding step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fp8_block_scaled_dg_amd as dg  # noqa: E402
from prenorm_mlp import BF, dequantize_weight, distance, quantize_weight, seconds  # noqa: E402


class Layer:
    def __init__(self, hidden, ffn, rand):
        self.norm, self.shift = (1 + 0.1 * rand(hidden)).to(BF), (0.1 * rand(hidden)).to(BF)
        self.b1, self.b2 = 0.1 * rand(2 * ffn), (0.1 * rand(hidden)).to(BF)
        self.w1, self.sf1 = quantize_weight(rand(2 * ffn, hidden) * hidden ** -0.5)
        self.w2, self.sf2 = quantize_weight(rand(hidden, ffn) * ffn ** -0.5)
        # the backward products contract over the weights' rows: their scales transposed
        self.sf1_t, self.sf2_t = self.sf1.t().contiguous(), self.sf2.t().contiguous()


class PreNormGated:
    def __init__(self, hidden, ffn, layers=2, activation="silu", dropout=0.1, eps=1e-5, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.activation, self.p, self.eps, self.ffn = activation, dropout, eps, ffn
        self.layers = [Layer(hidden, ffn, lambda *shape: torch.randn(shape, generator=gen, device=device))
                       for _ in range(layers)]
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device=device)

    def advance(self):
        """The next step's masks: none of them is one of this step's."""
        self.rng[1].add_(len(self.layers) + 1)

    def forward(self, x, train=True):
        """x bf16 [tokens, hidden] -> (result, what backward needs)."""
        tokens, device, p = x.shape[0], x.device, self.p if train else 0.0
        y, h_before, saved = x, None, []
        for i, w in enumerate(self.layers):
            h = torch.empty_like(x)
            mean, rstd = (torch.empty(tokens, device=device) if train else None for _ in range(2))
            pre = torch.empty(tokens, 2 * self.ffn, dtype=BF, device=device) if train else None
            n, n_sf = dg.layernorm_fp8_1x128(y, w.norm, w.shift, self.eps, residual=h_before, h=h, mean=mean,
                                             rstd=rstd, dropout_p=p, rng=self.rng, subsequence=i)
            u, u_sf = dg.fp8_gemm_nt_gated_fp8(n, w.w1, n_sf, w.sf1, bias=w.b1, activation=self.activation, pre=pre)
            y, h_before = torch.empty_like(x), h
            dg.fp8_gemm_nt_bias_act(u, w.w2, y, u_sf, w.sf2, bias=w.b2)
            saved.append((h, mean, rstd, pre))
        return dg.dropout_add(y, p, self.rng, len(self.layers), residual=h_before), saved

    def backward(self, dout, saved):
        """dout bf16 -> (gradient of x, gradients of each layer's norm, shift, b1 and b2)."""
        dh, grads = dout, []
        for i in reversed(range(len(self.layers))):
            w, (h, mean, rstd, pre) = self.layers[i], saved[i]
            g2, g2_sf, db2 = dg.dropout_backward_fp8(dh, self.p, self.rng, i + 1)
            du = torch.empty(h.shape[0], self.ffn, dtype=BF, device=h.device)
            dg.fp8_gemm_nn(g2, w.w2, du, g2_sf, w.sf2_t)
            g1, g1_sf, db1 = dg.gated_backward_fp8(du, pre, self.activation)
            dn = torch.empty_like(h)
            dg.fp8_gemm_nn(g1, w.w1, dn, g1_sf, w.sf1_t)
            dh, dnorm, dshift = dg.layernorm_backward(dn, h, w.norm, mean, rstd, dh=dh)
            grads.insert(0, dict(norm=dnorm, shift=dshift, b1=db1, b2=db2))
        return dg.dropout_add(dh, self.p, self.rng, 0), grads


def reference(model, x, dout):
    """The same stack in fp32 torch with autograd and the library's masks: (result, gradient of x,
    gradients, gradient of the residual stream at the bottom)."""
    act = {None: lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[model.activation]
    ones = torch.ones_like(x, dtype=torch.float32)
    params = [{k: getattr(w, k).float().requires_grad_() for k in ("norm", "shift", "b1", "b2")} for w in model.layers]
    x = x.float().requires_grad_()
    y, h = x, 0
    for i, (w, p) in enumerate(zip(model.layers, params)):
        h = h + y * dg.dropout_add(ones, model.p, model.rng, i)
        n = torch.nn.functional.layer_norm(h, h.shape[1:], p["norm"], p["shift"], model.eps)
        z = n @ dequantize_weight(w.w1, w.sf1).t() + p["b1"]
        u = act(z[:, :model.ffn]) * z[:, model.ffn:]
        y = u @ dequantize_weight(w.w2, w.sf2).t() + p["b2"]
    out = h + y * dg.dropout_add(ones, model.p, model.rng, len(params))
    out.backward(dout.float())
    return out.detach(), x.grad, [{k: t.grad for k, t in p.items()} for p in params]


def compare(model, x, dout):
    """Relative distances of both passes from the fp32 reference; the result and dx without what
    the residual stream carries, which would hide the layers' own part."""
    out, saved = model.forward(x)
    dx, grads = model.backward(dout, saved)
    out_ref, dx_ref, grads_ref = reference(model, x, dout)
    first = dg.dropout_add(x.float(), model.p, model.rng, 0)
    carried = dg.dropout_add(dout.float(), model.p, model.rng, 0)
    far = {"out": distance(out.float() - first, out_ref - first), "dx": distance(dx.float() - carried, dx_ref - carried)}
    far.update({f"d{k}[{i}]": distance(g[k], r[k]) for i, (g, r) in enumerate(zip(grads, grads_ref)) for k in g})
    return far


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=7168)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--activation", choices=[a for a in dg.ACTIVATIONS if a], default="silu")
    ap.add_argument("--dropout", type=float, default=0.1)
    a = ap.parse_args()
    model = PreNormGated(a.hidden, a.ffn, a.layers, a.activation, a.dropout)
    x, dout = (torch.randn(a.tokens, a.hidden, device="cuda").to(BF) for _ in range(2))
    for name, d in compare(model, x, dout).items():
        print(f"{name:9s} {d:.4f} from fp32 torch")
    model.advance()
    saved = model.forward(x)[1]
    flops = 6 * a.tokens * a.hidden * a.ffn * a.layers
    for name, f in (("forward", lambda: model.forward(x)), ("inference", lambda: model.forward(x, train=False)),
                    ("backward", lambda: model.backward(dout, saved))):
        s = seconds(f)
        print(f"{name:9s} {s * 1e6:8.1f} us  {flops / s * 1e-12:7.1f} TFLOP/s")


if __name__ == "__main__":
    main()
