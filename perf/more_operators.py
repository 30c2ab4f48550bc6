"""Cases of a transformer block's further operators around the FP8 block-scaled GEMM: the
layer norm that writes the GEMM's A operand (of residual + dropout(x) where asked), the gated
feed-forward product (both projections, activation and product, FP8 output), dropout from a
counter-based generator, and their backward passes.

``own`` false: plain torch operations in 32 bits. ``own`` true: the library's calls.
Scales of FP8 outputs are taken in the packed UE8M0 form; a case returns the codes as the
float8 values they are and each scale byte as the power of two it stands for.

Dropout. Element i of a tensor (row-major) is kept where 16 random bits reach
threshold = round(65536 p), and then multiplied by 65536 / (65536 - threshold). The bits are
half i % 2 of word (i % 8) / 2 of Philox 4x32 with 7 rounds, key = the seed's two words,
counter = the two words of i / 8 and the two words of offset + subsequence; the seed and the
offset are a tensor of two int64.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ("relu", "silu", "gelu", "gelu_tanh")
LARGEST = 4096 * 18432 * 7168  # rows x hidden columns x K of the largest gated product


def listed():
    return [
        # the norm before a projection while one sequence decodes: latency alone
        dict(name="norm 1 token", op="norm", M=1, K=7168, dtype="bf16", residual=True, bias=True, p=0.0),
        # training step of 4096 tokens: residual dropout of the block before joins the norm
        dict(name="norm 4096 dropout", op="norm", M=4096, K=7168, dtype="bf16", residual=True, bias=True,
             p=0.1),
        # training step of a small model, odd batch, fp32 stream
        dict(name="norm grad 257 fp32", op="norm_grad", M=257, K=2048, dtype="fp32", residual=False),
        # training step at the prefill width, gradient of the residual stream added
        dict(name="norm grad 4096", op="norm_grad", M=4096, K=7168, dtype="bf16", residual=True),
        # one token through a small expert's gate and up projections
        dict(name="gated 1 token", op="gated", M=1, I=2048, K=7168, act="silu", bias=False, pre=False,
             packed=True),
        # decode step of 64 sequences through a wide feed-forward: bound by the weights
        dict(name="gated 64", op="gated", M=64, I=18432, K=7168, act="silu", bias=False, pre=False,
             packed=True),
        # training batch of odd size: keeps the pre-activations
        dict(name="gated 1000 pre", op="gated", M=1000, I=2048, K=7168, act="gelu_tanh", bias=True,
             pre=True, packed=False),
        # training step of 4096 tokens, the largest product
        dict(name="gated 4096 pre", op="gated", M=4096, I=18432, K=7168, act="silu", bias=True, pre=True,
             packed=True),
        # gradient through a small block's gate, odd batch
        dict(name="gated grad 130", op="gated_grad", M=130, I=2048, act="gelu"),
        # gradient through the wide gate
        dict(name="gated grad 4096", op="gated_grad", M=4096, I=18432, act="silu"),
        # residual dropout at the end of a block
        dict(name="dropout 4096", op="dropout", M=4096, K=7168, dtype="bf16", residual=True, p=0.1),
        # its gradient, odd batch, fp32 stream, as the operand of the projection's backward
        dict(name="dropout grad 1000 fp32", op="dropout_grad", M=1000, K=2048, dtype="fp32", p=0.1),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "gated", "gated", "gated_grad", "dropout", "dropout_grad"))
    M = _log(rng, 1, 4096)
    flag = lambda: rng.random() < 0.5  # noqa: E731
    dtype, p = rng.choice(("bf16", "fp32")), rng.choice((0.05, 0.1, 0.2, 0.5))
    if op == "norm":
        return dict(op=op, M=M, K=_log(rng, 512, 18432, BLOCK), dtype=dtype, residual=flag(), bias=flag(),
                    p=p if flag() else 0.0)
    if op == "norm_grad":
        return dict(op=op, M=M, K=_log(rng, 512, 18432, BLOCK), dtype=dtype, residual=flag())
    if op == "gated_grad":
        return dict(op=op, M=M, I=_log(rng, 256, 18432, BLOCK), act=rng.choice(ACTS))
    if op == "dropout":  # any width: odd ones leave a tail
        return dict(op=op, M=M, K=_log(rng, 500, 18432), dtype=dtype, residual=flag(), p=p)
    if op == "dropout_grad":
        return dict(op=op, M=M, K=_log(rng, 512, 18432, BLOCK), dtype=dtype, p=p)
    K = _log(rng, 512, 18432, BLOCK)
    most = min(18432, LARGEST // (M * K) // BLOCK * BLOCK)
    return dict(op=op, M=M, I=_log(rng, 256, most, BLOCK), K=K, act=rng.choice(ACTS), bias=flag(),
                pre=flag(), packed=flag())


def work(case):
    M, op = case["M"], case["op"]
    if op in ("gated", "gated_grad"):
        I = case["I"]
        if op == "gated_grad":  # dh, pre, codes, scales, dbias
            return {"bytes": M * I * (2 + 4 + 2 + 2 / BLOCK) + 8 * I, "flops": 16 * M * I}
        K = case["K"]
        KB = K // BLOCK
        read = M * K + 2 * I * K + M * KB * (1 if case["packed"] else 4) + 8 * I // BLOCK * KB
        read += 4 * I if case["bias"] else 0
        out = M * I * (1 + 1 / BLOCK) + (4 * M * I if case["pre"] else 0)
        return {"bytes": read + out, "flops": 4 * M * I * K}
    K, e = case["K"], 2 if case["dtype"] == "bf16" else 4
    drop = 20 if case.get("p") else 0  # integer operations of the generator, about, per value
    if op == "norm":  # x (and residual, sum), codes, scales, weight, bias, mean, 1/deviation
        per = e * (1 + case["residual"] + (case["residual"] or case["p"] > 0)) + 1 + 1 / BLOCK
        return {"bytes": M * K * per + 4 * K + 8 * M, "flops": (9 + drop) * M * K}
    if op == "norm_grad":  # dy, h, dx (and dh); weight, dweight, dbias, mean, 1/deviation
        return {"bytes": M * K * e * (4 if case["residual"] else 3) + 10 * K + 8 * M, "flops": 12 * M * K}
    if op == "dropout":
        return {"bytes": M * K * e * (3 if case["residual"] else 2), "flops": (2 + drop) * M * K}
    return {"bytes": M * K * (e + 1 + 1 / BLOCK) + 4 * K, "flops": (4 + drop) * M * K}


# ---------------------------------------------------------------- inputs

def _hidden(M, K, g, dtype):
    """Hidden states: normal values about a row's mean, a few channels far larger than the rest."""
    x = torch.randn(M, K, device="cuda", generator=g) + torch.randn(M, 1, device="cuda", generator=g)
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
    w = torch.randn(N, K, device="cuda", generator=g) * (1.0 / math.sqrt(K))
    w = w.view(N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    sf = w.abs().amax((1, 3)) / 448
    codes = (w / sf[:, None, :, None]).to(torch.float8_e4m3fn).view(N, K)
    return codes.contiguous(), sf.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, M = case["op"], case["M"]
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    s = dict(case)
    # the generator's seed and the offset that a training loop counts up
    s["rng"] = torch.randint(0, 1 << 62, (2,), device="cuda", generator=g)

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
            s["b"] = (0.1 * torch.randn(K, device="cuda", generator=g)).to(torch.bfloat16) if case["bias"] else None
            s["h"] = torch.empty_like(s["x"]) if case["residual"] or case["p"] > 0 else None
            s["mean"], s["rstd"] = new(M, dtype=torch.float32), new(M, dtype=torch.float32)
            fp8_out(K)
        else:  # x is the stored sum, r the gradient that comes along the residual stream
            s["dy"] = torch.randn(M, K, device="cuda", generator=g).to(dt)
            if case["residual"]:
                s["r"] = torch.randn(M, K, device="cuda", generator=g).to(dt)
            t = s["x"].float()
            s["mean"] = t.mean(1)
            s["rstd"] = torch.rsqrt((t - s["mean"][:, None]).square().mean(1) + EPS)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"], s["db"] = new(K, dtype=torch.float32), new(K, dtype=torch.float32)
        return s
    if op == "dropout":
        dt = DTYPES[case["dtype"]]
        s["x"] = _hidden(M, case["K"], g, dt)
        s["r"] = _hidden(M, case["K"], g, dt) if case["residual"] else None
        s["out"] = torch.empty_like(s["x"])
        return s
    if op == "dropout_grad":
        s["dy"] = torch.randn(M, case["K"], device="cuda", generator=g).to(DTYPES[case["dtype"]])
        s["dbias"] = new(case["K"], dtype=torch.float32)
        fp8_out(case["K"])
        return s
    I = case["I"]
    if op == "gated_grad":
        s["dh"] = torch.randn(M, I, device="cuda", generator=g).to(torch.bfloat16)
        s["pre"] = (1.5 * torch.randn(M, 2 * I, device="cuda", generator=g)).to(torch.bfloat16)
        s["dbias"] = new(2 * I, dtype=torch.float32)
        fp8_out(2 * I)
        return s
    s["a"], s["a_sf"] = _activations(M, case["K"], g, case["packed"])
    s["b"], s["b_sf"] = _weights(2 * I, case["K"], g)
    s["bias"] = (0.5 * torch.randn(2 * I, device="cuda", generator=g)).to(torch.bfloat16) if case["bias"] else None
    s["pre_out"] = new(M, 2 * I, dtype=torch.bfloat16) if case["pre"] else None
    fp8_out(I)
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


def _keep(shape, p, rng):
    """Truth values [shape] of the elements that dropout keeps: the generator in int64, whose
    products of two 32-bit words wrap without loss of bits."""
    n, low = math.prod(shape), 0xFFFFFFFF
    i = torch.arange(-(-n // 8), dtype=torch.int64, device=rng.device)
    word = lambda v, k: (v >> (32 * k)) & low  # noqa: E731
    c = [word(i, 0), word(i, 1), word(rng[1], 0).expand_as(i), word(rng[1], 1).expand_as(i)]
    k0, k1 = word(rng[0], 0), word(rng[0], 1)
    for _ in range(7):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [word(b, 1) ^ c[1] ^ k0, word(b, 0), word(a, 1) ^ c[3] ^ k1, word(a, 0)]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    bits = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], -1).view(-1)[:n]
    return (bits >= int(p * 65536 + 0.5)).view(shape)


def _dropped(x, s):
    """dropout of x in fp32"""
    if s["p"] == 0:
        return x
    scale = 65536 / (65536 - int(s["p"] * 65536 + 0.5))
    return torch.where(_keep(x.shape, s["p"], s["rng"]), x * scale, 0.0)


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


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
    t = _dropped(s["x"].float(), s)
    if s["r"] is not None:
        t = t + s["r"].float()
    mean = t.mean(1)
    d = t - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(1) + EPS)
    y = d * rstd[:, None] * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    codes, sf = _fp8_values(y)
    out = {"codes": codes, "sf": sf, "mean": mean, "rstd": rstd}
    if s["h"] is not None:
        out["h"] = t.to(s["x"].dtype)
    return out


def _plain_norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _plain_gated(s):
    M, K = s["a"].shape
    N = s["b"].shape[0]
    sf = s["a_sf"]
    if s["packed"]:
        sf = torch.ldexp(torch.ones((), device="cuda"), sf.view(torch.uint8)[:, :K // BLOCK].int() - 127)
    a = (s["a"].float().view(M, -1, BLOCK) * sf[..., None]).view(M, K)
    b = s["b"].float().view(N, -1, BLOCK) * s["b_sf"].repeat_interleave(BLOCK, 0)[:, :, None]
    z = a @ b.view(N, K).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    codes, sf = _fp8_values(_act(z[:, :N // 2], s["act"]) * z[:, N // 2:])
    out = {"codes": codes, "sf": sf}
    if s["pre"]:
        out["pre"] = z.to(torch.bfloat16)
    return out


def _plain_gated_grad(s):
    I = s["I"]
    dh, gate, up = s["dh"].float(), s["pre"][:, :I].float(), s["pre"][:, I:].float()
    d = torch.cat([dh * up * _act_slope(gate, s["act"]), dh * _act(gate, s["act"])], 1)
    codes, sf = _fp8_values(d)
    return {"codes": codes, "sf": sf, "dbias": d.sum(0)}


def _plain_dropout(s):
    y = _dropped(s["x"].float(), s)
    return {"out": (y if s["r"] is None else y + s["r"].float()).to(s["x"].dtype)}


def _plain_dropout_grad(s):
    d = _dropped(s["dy"].float(), s)
    codes, sf = _fp8_values(d)
    return {"codes": codes, "sf": sf, "dbias": d.sum(0)}


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "gated": _plain_gated,
                "gated_grad": _plain_gated_grad, "dropout": _plain_dropout,
                "dropout_grad": _plain_dropout_grad}[op](s)
    import fp8_block_scaled_dg_amd as dg
    if op == "norm":
        dg.layernorm_fp8_1x128(s["x"], s["w"], s["b"], EPS, residual=s["r"], dropout_p=s["p"], rng=s["rng"],
                               h=s["h"], mean=s["mean"], rstd=s["rstd"], codes=s["codes"], sf=s["sf"])
        out = {"codes": s["codes"], "sf": s["sf_values"], "mean": s["mean"], "rstd": s["rstd"]}
        if s["h"] is not None:
            out["h"] = s["h"]
        return out
    if op == "norm_grad":
        dg.layernorm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], dh=s["r"], dx=s["dx"],
                              dweight=s["dw"], dbias=s["db"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "dropout":
        dg.dropout_add(s["x"], s["p"], s["rng"], residual=s["r"], out=s["out"])
        return {"out": s["out"]}
    out = {"codes": s["codes"], "sf": s["sf_values"]}
    if op == "gated":
        dg.fp8_gemm_nt_gated_fp8(s["a"], s["b"], s["a_sf"], s["b_sf"], bias=s["bias"], activation=s["act"],
                                 pre=s["pre_out"], codes=s["codes"], sf=s["sf"])
        if s["pre"]:
            out["pre"] = s["pre_out"]
        return out
    if op == "gated_grad":
        dg.gated_backward_fp8(s["dh"], s["pre"], s["act"], codes=s["codes"], sf=s["sf"], dbias=s["dbias"])
    else:
        dg.dropout_backward_fp8(s["dy"], s["p"], s["rng"], codes=s["codes"], sf=s["sf"], dbias=s["dbias"])
    out["dbias"] = s["dbias"]
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


def _exact_dropout(x, p, rng):
    """x with dropout, the generator in numpy's unsigned integers."""
    if p == 0:
        return x
    seed, offset = (int(v) for v in rng.cpu())
    n, u = x.numel(), np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    group = np.arange((n + 7) // 8, dtype=u)
    x0, x1 = group & low, group >> half
    x2, x3 = np.full_like(group, offset & 0xFFFFFFFF), np.full_like(group, offset >> 32 & 0xFFFFFFFF)
    for j in range(7):
        key0 = u((seed + j * 0x9E3779B9) & 0xFFFFFFFF)
        key1 = u(((seed >> 32) + j * 0xBB67AE85) & 0xFFFFFFFF)
        even, odd = u(0xD2511F53) * x0, u(0xCD9E8D57) * x2
        x0, x1, x2, x3 = (odd >> half) ^ x1 ^ key0, odd & low, (even >> half) ^ x3 ^ key1, even & low
    words = np.stack((x0, x1, x2, x3), 1).astype("<u4")
    threshold = int(p * 65536 + 0.5)
    kept = words.view("<u2").reshape(-1)[:n] >= threshold
    mask = torch.from_numpy(kept).to(x.device).view(x.shape).to(x.dtype)
    return x * mask * 65536 / (65536 - threshold)


def _exact_act(z, act):
    sigmoid = lambda t: torch.special.expit(t)  # noqa: E731
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    # (1 + tanh u) / 2 = sigmoid(2 u)
    return z * sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "norm":
        t = _exact_dropout(s["x"].to(d), case["p"], s["rng"]) + (s["r"].to(d) if s["r"] is not None else 0)
        var, mean = torch.var_mean(t, 1, correction=0, keepdim=True)
        y = (t - mean) * (var + EPS) ** -0.5 * s["w"].to(d) + (s["b"].to(d) if s["b"] is not None else 0)
        out = {"codes": _exact_codes(y), "sf": None, "mean": mean[:, 0], "rstd": (var[:, 0] + EPS) ** -0.5}
        if s["h"] is not None:
            out["h"] = t
        return out
    if op == "norm_grad":
        # the derivative of y = w xh + b with xh = (h - mean) q for the stored mean and q = rstd, which
        # move with h: dmean = dh / K, dq = -q^3 (h - mean) dh / K
        h, dy, w, q = s["x"].to(d), s["dy"].to(d), s["w"].to(d), s["rstd"].to(d).unsqueeze(1)
        c = h - s["mean"].to(d).unsqueeze(1)
        along = (w * dy * c).sum(1, keepdim=True) / h.shape[1]
        dx = q * (w * dy) - q * (w * dy).sum(1, keepdim=True) / h.shape[1] - q ** 3 * c * along
        dx = dx + (s["r"].to(d) if s["r"] is not None else 0)
        return {"dx": dx, "dw": (dy * c * q).sum(0), "db": dy.sum(0)}
    if op == "dropout":
        t = _exact_dropout(s["x"].to(d), case["p"], s["rng"])
        return {"out": t if s["r"] is None else t + s["r"].to(d)}
    if op == "dropout_grad":
        t = _exact_dropout(s["dy"].to(d), case["p"], s["rng"])
        return {"codes": _exact_codes(t), "sf": None, "dbias": t.sum(0)}
    I = case["I"]
    if op == "gated_grad":
        z = s["pre"].to(d).requires_grad_()
        p, = torch.autograd.grad(_exact_act(z[:, :I], case["act"]) * z[:, I:], z, s["dh"].to(d))
        return {"codes": _exact_codes(p), "sf": None, "dbias": p.sum(0)}
    K = case["K"]
    sf = s["a_sf"]
    if case["packed"]:
        sf = torch.exp2(sf.view(torch.uint8).to(d)[:, :K // BLOCK] - 127)
    a = s["a"].to(d) * sf.to(d).repeat_interleave(BLOCK, 1)
    b = s["b"].to(d) * s["b_sf"].to(d).repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
    z = a.matmul(b.t().contiguous())
    if s["bias"] is not None:
        z = z + s["bias"].to(d)
    out = {"codes": _exact_codes(_exact_act(z[:, :I], case["act"]) * z[:, I:]), "sf": None}
    if case["pre"]:
        out["pre"] = z
    return out
