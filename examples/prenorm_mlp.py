"""A pre-norm MLP block on FP8 weights, forward and backward, out of the library's calls.

    h = x + residual;  y = h + W2 act(W1 norm(h) + b1) + b2

Forward, three launches: the norm writes W1's FP8 operand, W1's epilogue adds the bias,
applies the activation and writes W2's FP8 operand, W2's epilogue adds bias and residual.
Backward, per layer: the epilogue's backward writes the gradient as an FP8 operand and the
bias gradient, fp8_gemm_nn multiplies it by the weights as they are stored, and the norm's
backward adds the gradient of the residual stream. W1 and W2 stay frozen: their gradients
contract over tokens, along which the FP8 gradient has no scale blocks.

    python examples/prenorm_mlp.py [--tokens 4096] [--hidden 2048] [--ffn 7168] [--activation gelu]

prints the time of both passes and how far their results lie from fp32 torch with the same
(dequantized) weights. --tokens 1 is a decoding step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import fp8_block_scaled_dg_amd as dg  # noqa: E402

BLOCK = 128
BF = torch.bfloat16


def quantize_weight(w):
    """w [N, K] fp32 (multiples of 128) -> (e4m3fn codes, fp32 scale per 128x128 block)."""
    n, k = w.shape
    blocks = w.reshape(n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    sf = torch.exp2(torch.ceil(torch.log2(blocks.abs().amax(dim=(1, 3)).clamp_min(1e-30) / 448)))
    codes = (blocks / sf[:, None, :, None]).reshape(n, k).to(torch.float8_e4m3fn)
    return codes, sf.contiguous()


def dequantize_weight(codes, sf):
    return codes.float() * sf.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)


class PreNormMLP:
    def __init__(self, hidden, ffn, activation="gelu", eps=1e-6, seed=0, device="cuda"):
        rng = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=rng, device=device)  # noqa: E731
        self.activation, self.eps, self.hidden, self.ffn = activation, eps, hidden, ffn
        self.norm = (1 + 0.1 * rand(hidden)).to(BF)
        self.b1, self.b2 = 0.1 * rand(ffn), 0.1 * rand(hidden)
        self.w1, self.sf1 = quantize_weight(rand(ffn, hidden) * hidden ** -0.5)
        self.w2, self.sf2 = quantize_weight(rand(hidden, ffn) * ffn ** -0.5)
        # the backward products contract over the weights' rows: their scales transposed
        self.sf1_t, self.sf2_t = self.sf1.t().contiguous(), self.sf2.t().contiguous()

    def forward(self, x, residual=None, train=True):
        """x, residual bf16 [tokens, hidden] -> (y, what backward needs)."""
        tokens, device = x.shape[0], x.device
        h = torch.empty_like(x)
        rstd = torch.empty(tokens, device=device) if train else None
        pre = torch.empty(tokens, self.ffn, dtype=BF, device=device) if train else None
        n, n_sf = dg.rmsnorm_fp8_1x128(x, self.norm, self.eps, residual=residual, h=h, rstd=rstd)
        u, u_sf = dg.fp8_gemm_nt_bias_act_fp8(n, self.w1, n_sf, self.sf1, bias=self.b1,
                                              activation=self.activation, pre=pre)
        y = torch.empty_like(x)
        dg.fp8_gemm_nt_bias_act(u, self.w2, y, u_sf, self.sf2, bias=self.b2, residual=h)
        return y, (h, rstd, pre)

    def backward(self, dy, saved):
        """dy bf16 -> (gradient of x and of residual, gradients of norm, b1 and b2)."""
        h, rstd, pre = saved
        g2, g2_sf, db2 = dg.bias_act_backward_fp8(dy)
        du = torch.empty_like(pre)
        dg.fp8_gemm_nn(g2, self.w2, du, g2_sf, self.sf2_t)
        g1, g1_sf, db1 = dg.bias_act_backward_fp8(du, pre, self.activation)
        dn = torch.empty_like(h)
        dg.fp8_gemm_nn(g1, self.w1, dn, g1_sf, self.sf1_t)
        dx, dnorm = dg.rmsnorm_backward(dn, h, self.norm, rstd, dh=dy, dx=dn)
        return dx, dict(norm=dnorm, b1=db1, b2=db2)


def reference(mlp, x, residual, dy):
    """The same block in fp32 torch with autograd: (y, dx, gradients)."""
    act = {None: lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu,
           "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[mlp.activation]
    p = {k: getattr(mlp, k).float().requires_grad_() for k in ("norm", "b1", "b2")}
    h = (x.float() + residual.float()).requires_grad_()
    n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + mlp.eps) * p["norm"]
    u = act(n @ dequantize_weight(mlp.w1, mlp.sf1).t() + p["b1"])
    y = h + u @ dequantize_weight(mlp.w2, mlp.sf2).t() + p["b2"]
    y.backward(dy.float())
    return y.detach(), h.grad, {k: t.grad for k, t in p.items()}


def distance(got, want):
    """Relative distance in the 2-norm."""
    return float((got.float() - want.float()).norm() / want.float().norm())


def compare(mlp, x, residual, dy):
    """Relative distances of both passes from the fp32 reference. y and dx without what the
    residual stream adds, which would hide the MLP's own part."""
    y, saved = mlp.forward(x, residual)
    dx, grads = mlp.backward(dy, saved)
    y_ref, dx_ref, grads_ref = reference(mlp, x, residual, dy)
    h = x.float() + residual.float()
    out = {"mlp(h)": distance(y.float() - h, y_ref - h),
           "dx - dy": distance(dx.float() - dy.float(), dx_ref - dy.float())}
    out.update({"d" + k: distance(grads[k], grads_ref[k]) for k in grads})
    return out


def seconds(f, repeats=50):
    for _ in range(5):
        f()
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(repeats):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / repeats / 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=7168)
    ap.add_argument("--activation", choices=[a for a in dg.ACTIVATIONS if a], default="gelu")
    a = ap.parse_args()
    mlp = PreNormMLP(a.hidden, a.ffn, a.activation)
    x, residual, dy = (torch.randn(a.tokens, a.hidden, device="cuda").to(BF) for _ in range(3))
    for name, d in compare(mlp, x, residual, dy).items():
        print(f"{name:8s} {d:.4f} from fp32 torch")
    saved = mlp.forward(x, residual)[1]
    flops = 4 * a.tokens * a.hidden * a.ffn
    for name, f in (("forward", lambda: mlp.forward(x, residual)), ("inference", lambda: mlp.forward(x, residual, train=False)),
                    ("backward", lambda: mlp.backward(dy, saved))):
        s = seconds(f)
        print(f"{name:9s} {s * 1e6:8.1f} us  {flops / s * 1e-12:7.1f} TFLOP/s")


if __name__ == "__main__":
    main()
