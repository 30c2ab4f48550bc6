"""Cases of the operators around the FP8 block-scaled GEMM: the RMS norm that writes the
GEMM's A operand, the GEMM with bias, activation and residual in its epilogue (bf16 or FP8
output), and their backward passes.

``own`` false: plain torch operations in 32 bits. ``own`` true: the library's calls.
Scales of FP8 outputs are taken in the packed UE8M0 form; a case returns the codes as the
float8 values they are and each scale byte as the power of two it stands for.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # the norm before a projection while one sequence decodes: latency alone
        dict(name="norm 1 token", op="norm", M=1, K=7168, dtype="bf16", residual=True),
        # a small model's odd batch with its residual stream in fp32
        dict(name="norm 257 fp32", op="norm", M=257, K=2048, dtype="fp32", residual=False),
        # prefill of 4096 tokens
        dict(name="norm prefill", op="norm", M=4096, K=7168, dtype="bf16", residual=True),
        # training step of a small model, odd batch, fp32 stream
        dict(name="norm grad 1000 fp32", op="norm_grad", M=1000, K=2048, dtype="fp32", residual=False),
        # training step at the prefill width, gradient of the residual stream added
        dict(name="norm grad 4096", op="norm_grad", M=4096, K=7168, dtype="bf16", residual=True),
        # output projection of a 64-sequence decode step, added to the residual stream
        dict(name="gemm 64 residual", op="gemm", M=64, N=2112, K=7168, act="none", residual=True,
             pre=False, packed=False),
        # one token through a wide, shallow projection
        dict(name="gemm 1 token silu", op="gemm", M=1, N=32768, K=512, act="silu", residual=False,
             pre=False, packed=True),
        # down projection of a prefill MLP: the largest product
        dict(name="gemm prefill residual", op="gemm", M=4096, N=7168, K=18432, act="none",
             residual=True, pre=False, packed=True),
        # up projection of a decode step, quantized for the down projection
        dict(name="gemm fp8 64 gelu", op="gemm_fp8", M=64, N=18432, K=7168, act="gelu", pre=False,
             packed=True),
        # up projection of a training batch of odd size: keeps the pre-activation
        dict(name="gemm fp8 1000 silu pre", op="gemm_fp8", M=1000, N=4096, K=7168, act="silu",
             pre=True, packed=False),
        # gradient through a small MLP's activation
        dict(name="act grad 130 silu", op="act_grad", M=130, N=2048, act="silu"),
        # gradient through the prefill MLP's activation
        dict(name="act grad 4096 gelu", op="act_grad", M=4096, N=18432, act="gelu"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "gemm", "gemm_fp8", "act_grad"))
    M = _log(rng, 1, 4096)
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("norm", "norm_grad"):
        return dict(op=op, M=M, K=_log(rng, 512, 18432, BLOCK), dtype=rng.choice(("bf16", "fp32")),
                    residual=flag())
    if op == "act_grad":
        return dict(op=op, M=M, N=_log(rng, 512, 18432, BLOCK), act=rng.choice(ACTS[1:]))
    K = _log(rng, 512, 18432, BLOCK)
    most = 4096 * 7168 * 18432 // (M * K)
    if op == "gemm":
        N = _log(rng, 256, min(32768, most // 16 * 16), 16)
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(ACTS), residual=flag(), pre=flag(),
                    packed=flag())
    N = _log(rng, 256, min(32768, most // BLOCK * BLOCK), BLOCK)
    return dict(op=op, M=M, N=N, K=K, act=rng.choice(ACTS), pre=flag(), packed=flag())


def work(case):
    M = case["M"]
    if case["op"] in ("norm", "norm_grad"):
        K, e = case["K"], 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "norm":  # x (and residual, sum), codes, scales, weight, 1/rms
            per = e * (3 if case["residual"] else 1) + 1 + 1 / BLOCK
            return {"bytes": M * K * per + 2 * K + 4 * M, "flops": 6 * M * K}
        per = e * (4 if case["residual"] else 3)  # dy, h, dx (and dh)
        return {"bytes": M * K * per + 6 * K + 4 * M, "flops": 10 * M * K}
    N = case["N"]
    if case["op"] == "act_grad":  # dc, pre, codes, scales, dbias
        return {"bytes": M * N * (5 + 1 / BLOCK) + 4 * N, "flops": 12 * M * N}
    K = case["K"]
    KB, NB = K // BLOCK, -(-N // BLOCK)
    read = M * K + N * K + M * KB * (1 if case["packed"] else 4) + 4 * NB * KB + 2 * N
    out = M * N * (2 if case["op"] == "gemm" else 1 + 1 / BLOCK)
    out += 2 * M * N * (bool(case.get("residual")) + bool(case["pre"]))
    return {"bytes": read + out, "flops": 2 * M * N * K}


# ---------------------------------------------------------------- inputs

def _hidden(M, K, g, dtype):
    """Hidden states: normal values, a few channels far larger than the rest."""
    x = torch.randn(M, K, device="cuda", generator=g)
    wide = torch.rand(K, device="cuda", generator=g) < 0.01
    return (x * torch.where(wide, 12.0, 1.0)).to(dtype)


def _activations(M, K, g, packed):
    """e4m3fn codes [M, K] and power-of-two 1x128 scales, fp32 or packed bytes in int32 words."""
    codes, e = _quantize(torch.randn(M, K, device="cuda", generator=g))
    KB = K // BLOCK
    if not packed:
        return codes, torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    words = torch.zeros(M, -(-KB // 4) * 4, dtype=torch.uint8, device="cuda")
    words[:, :KB] = (e + 127).to(torch.uint8)
    return codes, words.view(torch.int32)


def _weights(N, K, g):
    """e4m3fn codes [N, K] of normal weights and their fp32 scales per 128x128 block."""
    NB, KB = -(-N // BLOCK), K // BLOCK
    w = torch.zeros(NB * BLOCK, K, device="cuda")
    w[:N] = torch.randn(N, K, device="cuda", generator=g) * (1.0 / math.sqrt(K))
    w = w.view(NB, BLOCK, KB, BLOCK)
    sf = w.abs().amax((1, 3)) / 448
    codes = (w / sf[:, None, :, None]).to(torch.float8_e4m3fn).view(NB * BLOCK, K)[:N]
    return codes.contiguous(), sf.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, M = case["op"], case["M"]
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    s = dict(case)

    def fp8_out(cols):  # an FP8 output and its packed scales, as a user's program keeps them
        CB = cols // BLOCK
        s["codes"] = new(M, cols, dtype=torch.float8_e4m3fn)
        s["sf"] = new(M, -(-CB // 4), dtype=torch.int32)
        s["sf_values"] = s["sf"].view(torch.uint8)[:, :CB].view(torch.float8_e8m0fnu)

    if op in ("norm", "norm_grad"):
        K, dt = case["K"], DTYPES[case["dtype"]]
        s["w"] = (1 + 0.1 * torch.randn(K, device="cuda", generator=g)).to(torch.bfloat16)
        s["x"] = _hidden(M, K, g, dt)
        s["r"] = _hidden(M, K, g, dt) if case["residual"] else None
        if op == "norm":
            s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["rstd"] = new(M, dtype=torch.float32)
            fp8_out(K)
        else:  # x is the stored sum, r the gradient that comes along the residual stream
            s["dy"] = torch.randn(M, K, device="cuda", generator=g).to(dt)
            if case["residual"]:
                s["r"] = torch.randn(M, K, device="cuda", generator=g).to(dt)
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = new(K, dtype=torch.float32)
        return s
    N = case["N"]
    if op == "act_grad":
        s["dc"] = torch.randn(M, N, device="cuda", generator=g).to(torch.bfloat16)
        s["pre"] = (1.5 * torch.randn(M, N, device="cuda", generator=g)).to(torch.bfloat16)
        s["dbias"] = new(N, dtype=torch.float32)
        fp8_out(N)
        return s
    s["a"], s["a_sf"] = _activations(M, case["K"], g, case["packed"])
    s["b"], s["b_sf"] = _weights(N, case["K"], g)
    s["bias"] = (0.5 * torch.randn(N, device="cuda", generator=g)).to(torch.bfloat16)
    s["pre_out"] = new(M, N, dtype=torch.bfloat16) if case["pre"] else None
    if op == "gemm":
        s["r"] = _hidden(M, N, g, torch.bfloat16) if case["residual"] else None
        s["c"] = new(M, N, dtype=torch.bfloat16)
    else:
        fp8_out(N)
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits

def _quantize(y):
    """codes and exponents of y [M, K]: per 1x128 block the least e with amax <= 448 * 2^e."""
    M, K = y.shape
    b = y.view(M, K // BLOCK, BLOCK)
    amax = b.abs().amax(-1)
    f, x = torch.frexp(amax)
    e = torch.where(amax > 0, x - 9 + (f > 0.875), 0).clamp(min=-127)
    return torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).view(M, K), e


def _fp8_values(y):
    codes, e = _quantize(y)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return x


def _act_slope(x, act):
    if act == "relu":
        return (x > 0).float()
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def _plain_norm(s):
    t = s["x"].float()
    if s["r"] is not None:
        t = t + s["r"].float()
    rstd = torch.rsqrt(t.square().mean(1) + EPS)
    codes, sf = _fp8_values(t * rstd[:, None] * s["w"].float())
    out = {"codes": codes, "sf": sf, "rstd": rstd}
    if s["r"] is not None:
        out["h"] = t.to(s["x"].dtype)
    return out


def _plain_norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = s["x"].float() * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0)}


def _plain_gemm(s):
    M, K = s["a"].shape
    N = s["b"].shape[0]
    sf = s["a_sf"]
    if s["packed"]:
        sf = torch.ldexp(torch.ones((), device="cuda"), sf.view(torch.uint8)[:, :K // BLOCK].int() - 127)
    a = (s["a"].float().view(M, -1, BLOCK) * sf[..., None]).view(M, K)
    b = s["b"].float().view(N, -1, BLOCK) * s["b_sf"].repeat_interleave(BLOCK, 0)[:N, :, None]
    pre = a @ b.view(N, K).t() + s["bias"].float()
    v = _act(pre, s["act"])
    out = {"pre": pre.to(torch.bfloat16)} if s["pre"] else {}
    if s["op"] == "gemm":
        out["c"] = (v if s["r"] is None else v + s["r"].float()).to(torch.bfloat16)
    else:
        out["codes"], out["sf"] = _fp8_values(v)
    return out


def _plain_act_grad(s):
    p = s["dc"].float() * _act_slope(s["pre"].float(), s["act"])
    codes, sf = _fp8_values(p)
    return {"codes": codes, "sf": sf, "dbias": p.sum(0)}


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "gemm": _plain_gemm,
                "gemm_fp8": _plain_gemm, "act_grad": _plain_act_grad}[op](s)
    import fp8_block_scaled_dg_amd as dg
    if op == "norm":
        dg.rmsnorm_fp8_1x128(s["x"], s["w"], EPS, residual=s["r"], h=s["h"], rstd=s["rstd"],
                             codes=s["codes"], sf=s["sf"])
        out = {"codes": s["codes"], "sf": s["sf_values"], "rstd": s["rstd"]}
        if s["h"] is not None:
            out["h"] = s["h"]
        return out
    if op == "norm_grad":
        dg.rmsnorm_backward(s["dy"], s["x"], s["w"], s["rstd"], dh=s["r"], dx=s["dx"],
                            dweight=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "act_grad":
        dg.bias_act_backward_fp8(s["dc"], s["pre"], s["act"], codes=s["codes"], sf=s["sf"],
                                 dbias=s["dbias"])
        return {"codes": s["codes"], "sf": s["sf_values"], "dbias": s["dbias"]}
    out = {"pre": s["pre_out"]} if s["pre"] else {}
    if op == "gemm":
        dg.fp8_gemm_nt_bias_act(s["a"], s["b"], s["c"], s["a_sf"], s["b_sf"], bias=s["bias"],
                                activation=s["act"], residual=s["r"], pre=s["pre_out"])
        out["c"] = s["c"]
    else:
        dg.fp8_gemm_nt_bias_act_fp8(s["a"], s["b"], s["a_sf"], s["b_sf"], bias=s["bias"],
                                    activation=s["act"], pre=s["pre_out"], codes=s["codes"],
                                    sf=s["sf"])
        out["codes"], out["sf"] = s["codes"], s["sf_values"]
    return out


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_codes(y):
    """What the codes stand for before their one rounding: y / 2^e. The scale itself is a
    choice between neighbouring powers of two, which a block whose largest value lies within
    rounding of 448 * 2^e may take either way: it has no exact value to be held to."""
    top = y.unflatten(1, (-1, BLOCK)).abs().amax(-1)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 448.0) / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    return y / torch.exp2(e).repeat_interleave(BLOCK, 1)


def _exact_act(z, act):
    sigmoid = lambda t: torch.special.expit(t)  # noqa: E731
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
        return z * sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return z


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "norm":
        t = s["x"].to(d) + (s["r"].to(d) if s["r"] is not None else 0)
        rstd = ((t * t).sum(1) / t.shape[1] + EPS) ** -0.5
        out = {"codes": _exact_codes(t * s["w"].to(d) * rstd.unsqueeze(1)), "sf": None, "rstd": rstd}
        if s["r"] is not None:
            out["h"] = t
        return out
    if op == "norm_grad":
        # the derivative of y_k = w_k h_k rstd with rstd = (mean h^2 + eps)^(-1/2), as stored
        h, dy, w, q = s["x"].to(d), s["dy"].to(d), s["w"].to(d), s["rstd"].to(d).unsqueeze(1)
        along = (w * dy * h).sum(1, keepdim=True) / h.shape[1]
        dx = q * w * dy - q ** 3 * h * along + (s["r"].to(d) if s["r"] is not None else 0)
        return {"dx": dx, "dw": (dy * h * q).sum(0)}
    if op == "act_grad":
        z = s["pre"].to(d).requires_grad_()
        p, = torch.autograd.grad(_exact_act(z, case["act"]), z, s["dc"].to(d))
        return {"codes": _exact_codes(p), "sf": None, "dbias": p.sum(0)}
    K = case["K"]
    sf = s["a_sf"]
    if case["packed"]:
        sf = torch.exp2(sf.view(torch.uint8).to(d)[:, :K // BLOCK] - 127)
    a = s["a"].to(d) * sf.to(d).repeat_interleave(BLOCK, 1)
    b = s["b"].to(d) * s["b_sf"].to(d).repeat_interleave(BLOCK, 0)[:case["N"]].repeat_interleave(BLOCK, 1)
    z = a.matmul(b.t().contiguous()) + s["bias"].to(d)
    out = {"pre": z} if case["pre"] else {}
    v = _exact_act(z, case["act"])
    if op == "gemm":
        out["c"] = v if s["r"] is None else v + s["r"].to(d)
    else:
        out["codes"], out["sf"] = _exact_codes(v), None
    return out
