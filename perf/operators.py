"""Cases of the layer norm, its backward pass, row quantisation and the 8-bit
integer product, with their plain forms.

`own` false: elementary torch operations.  `own` true: the calls a user makes.
A case names its operator in "op":

  ln        layer_norm: rows x [M][D] -> y, mean, rstd
  ln_int8   layer_norm_int8 -> int8 rows and scales, read back in 16 bits
  ln_bwd    layer_norm_bwd: dy, x, mean, rstd -> dx, dweight, dbias
  quant     quantize_rows, read back by dequantize_rows
  linear    int8_linear: [M][K] x [N][K] int8 with a scale per token and channel
  gated     int8_gated: u * ReLU(g) of two such products

"gap" is the distance between the rows of x beyond their length (the FFN's
rows carry the gate bias in a last column that the norm leaves alone).
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # The norm before a decode step of 16 sequences.
        {"name": "ln_decode", "op": "ln", "M": 16, "D": 2048, "gap": 0, "x": "bf16", "y": "bf16"},
        # A training batch's fp32 residual stream into the FFN's bf16 rows.
        {"name": "ln_train", "op": "ln", "M": 16384, "D": 2560, "gap": 0, "x": "f32", "y": "bf16"},
        # Rows with the gate bias in their last column: 1535 of 1536 columns are normalised.
        {"name": "ln_bias_column", "op": "ln", "M": 2047, "D": 1535, "gap": 1, "x": "bf16", "y": "bf16"},
        # A prompt's rows normalised straight into the int8 product's operand.
        {"name": "ln_int8_prompt", "op": "ln_int8", "M": 8192, "D": 2048, "gap": 0, "x": "bf16", "y": "bf16"},
        # A short fine-tuning batch.
        {"name": "ln_bwd_small", "op": "ln_bwd", "M": 64, "D": 256, "gap": 0, "x": "bf16", "y": "bf16"},
        # The norm's gradient behind the sparse FFN's fp32 dx, whole training batch.
        {"name": "ln_bwd_train", "op": "ln_bwd", "M": 16384, "D": 2560, "gap": 0, "x": "f32", "y": "f32"},
        # Odd width, contiguous rows (no row but the first is aligned).
        {"name": "ln_bwd_odd", "op": "ln_bwd", "M": 4099, "D": 2047, "gap": 0, "x": "f16", "y": "f16"},
        # The hidden rows between the two products of an int8 FFN.
        {"name": "quant_hidden", "op": "quant", "M": 8192, "D": 5632, "gap": 0, "x": "bf16", "y": "bf16"},
        # A few fp32 rows of odd length.
        {"name": "quant_odd", "op": "quant", "M": 37, "D": 4093, "gap": 0, "x": "f32", "y": "f32"},
        # Decode: 16 tokens against an up projection.
        {"name": "linear_decode", "op": "linear", "M": 16, "K": 2048, "N": 8192, "y": "bf16", "bias": False},
        # Down projection of a ragged mid-size batch, fp32 out, with a bias.
        {"name": "linear_ragged", "op": "linear", "M": 1000, "K": 4093, "N": 1535, "y": "f32", "bias": True},
        # Gate and up products of the largest workload's FFN.
        {"name": "gated_prefill", "op": "gated", "M": 16384, "K": 2560, "N": 10240, "y": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ln_int8", "ln_bwd", "quant", "linear", "gated"])
    if op in ("linear", "gated"):
        most = 16384 * 2560 * 10240 * (2 if op == "linear" else 1)
        while True:
            M, K, N = _log_int(rng, 1, 16384), _log_int(rng, 32, 10240), _log_int(rng, 32, 10240)
            if rng.random() < 0.6:  # widths are usually whole multiples
                K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
            if M * K * N <= most:
                break
        case = {"op": op, "M": M, "K": K, "N": N, "y": rng.choice(["bf16", "bf16", "f16", "f32"])}
        if op == "linear":
            case["bias"] = rng.random() < 0.5
        return case
    M, D = _log_int(rng, 1, 16384), _log_int(rng, 16, 8192 if op != "quant" else 16384)
    if rng.random() < 0.5:
        D = max(16, D // 16 * 16)
    while M * D > 16384 * 2560:
        M = max(1, M // 2)
    x = rng.choice(["f32", "bf16", "f16"])
    y = x if op == "quant" else ("bf16" if op == "ln_int8" else rng.choice([x, "f32" if x != "f32" else "bf16"]))
    return {"op": op, "M": M, "D": D, "gap": rng.choice([0, 0, 1, 8]), "x": x, "y": y}


def _rows(M, D, gap, dtype, g):
    """Activations: a scale per row, a few channels far above the rest, an offset."""
    x = torch.randn((M, D + gap), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((M, 1), generator=g, device="cuda"))
    x *= torch.where(torch.rand((1, D + gap), generator=g, device="cuda") < 0.005, 8.0, 1.0)
    x += 0.1
    return x.to(dtype)[:, :D]


def _int8_rows(R, K, g):
    """int8 rows in storage whose row stride is a multiple of 16, and their scales."""
    q = torch.randn((R, (K + 15) // 16 * 16), generator=g, device="cuda").mul_(36).round_().clamp_(-127, 127)
    return q.to(torch.int8)[:, :K], torch.exp(0.3 * torch.randn(R, generator=g, device="cuda")) * 0.01


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    op, M = case["op"], case["M"]
    if op in ("linear", "gated"):
        K, N = case["K"], case["N"]
        s["xq"], s["xs"] = _int8_rows(M, K, g)
        s["wq"], s["ws"] = _int8_rows(N, K, g)
        if op == "gated":
            s["uq"], s["us"] = _int8_rows(N, K, g)
        s["bias"] = torch.randn(N, generator=g, device="cuda") if case.get("bias") else None
        return s
    D = case["D"]
    s["x"] = _rows(M, D, case["gap"], TYPES[case["x"]], g)
    if op == "quant":
        return s
    s["w"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
    s["b"] = 0.2 * torch.randn(D, generator=g, device="cuda")
    if op == "ln_bwd":
        s["dy"] = torch.randn((M, D + case["gap"]), generator=g, device="cuda").to(TYPES[case["y"]])[:, :D]
        x = s["x"].double()
        s["mean"] = x.mean(1).float()
        s["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
    return s


def _plain_norm(x, w, b):
    x = x.float()
    mean = x.sum(1, keepdim=True) / x.shape[1]
    c = x - mean
    rstd = 1 / ((c * c).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt()
    return c * rstd * w + b, mean[:, 0], rstd[:, 0]


def _plain_quant(x):
    """(q, scale): q is the integer nearest to 127 x / max|x|, ties to even."""
    amax = x.abs().amax(1, keepdim=True).float()
    q = (x.double() * 127 / amax.double().clamp_min(1e-300)).round().float()
    return q, amax / 127


def _plain_product(xq, xs, wq, ws):
    return (xq.float() @ wq.float().t()) * xs[:, None] * ws


def run(s):
    c = s["case"]
    op, y = c["op"], TYPES[c["y"]]
    if own:
        from activation_sparse_gated_tma_b200 import twell as tw
        if op == "ln":
            return tw.layer_norm(s["x"], s["w"], s["b"], EPS, out_dtype=y, stats=True)
        if op == "ln_int8":
            q, scale = tw.layer_norm_int8(s["x"], s["w"], s["b"], EPS)
            return tw.dequantize_rows(q, scale, out_dtype=y), scale
        if op == "ln_bwd":
            return tw.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
        if op == "quant":
            q, scale = tw.quantize_rows(s["x"])
            return tw.dequantize_rows(q, scale, out_dtype=y), scale
        if op == "linear":
            return tw.int8_linear(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"], out_dtype=y)
        return tw.int8_gated(s["xq"], s["xs"], s["wq"], s["ws"], s["uq"], s["us"], out_dtype=y)
    if op == "ln":
        v, mean, rstd = _plain_norm(s["x"], s["w"], s["b"])
        return v.to(y), mean, rstd
    if op == "ln_int8":
        q, scale = _plain_quant(_plain_norm(s["x"], s["w"], s["b"])[0])
        return (q * scale).to(y), scale[:, 0]
    if op == "ln_bwd":
        dy, mean, rstd = s["dy"].float(), s["mean"][:, None], s["rstd"][:, None]
        xh = (s["x"].float() - mean) * rstd
        gr = dy * s["w"]
        dx = rstd * (gr - (gr.sum(1, keepdim=True) + xh * (gr * xh).sum(1, keepdim=True)) / c["D"])
        return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    if op == "quant":
        q, scale = _plain_quant(s["x"])
        return (q * scale).to(y), scale[:, 0]
    v = _plain_product(s["xq"], s["xs"], s["wq"], s["ws"])
    if op == "gated":
        v = v.clamp_min(0) * _plain_product(s["xq"], s["xs"], s["uq"], s["us"])
    elif s["bias"] is not None:
        v = v + s["bias"]
    return v.to(y)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op in ("linear", "gated"):
        def product(wq, ws):
            return torch.einsum("mk,nk->mn", s["xq"].to(f64), wq.to(f64)) * torch.outer(s["xs"].to(f64), ws.to(f64))
        v = product(s["wq"], s["ws"])
        if op == "gated":
            return torch.where(v > 0, v, 0) * product(s["uq"], s["us"])
        return v if s["bias"] is None else v + s["bias"].to(f64)

    def quantised(v):
        top = v.abs().max(dim=1, keepdim=True).values
        steps = torch.where(top > 0, v / top * 127, 0)
        return steps.round() * (top / 127), top[:, 0] / 127

    x = s["x"].to(f64)
    if op == "quant":
        top = x.abs().max(dim=1, keepdim=True).values
        return (x * 127 / torch.where(top > 0, top, 1)).round() * (top / 127), top[:, 0] / 127
    if op == "ln_bwd":
        dy, w = s["dy"].to(f64), s["w"].to(f64)
        mean, rstd = s["mean"].to(f64).unsqueeze(1), s["rstd"].to(f64).unsqueeze(1)
        hat = (x - mean) * rstd
        along = torch.mean(dy * w * hat, dim=1, keepdim=True)
        level = torch.mean(dy * w, dim=1, keepdim=True)
        return (dy * w - level - hat * along) * rstd, torch.einsum("md,md->d", dy, hat), dy.sum(dim=0)
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    rstd = torch.rsqrt(var + EPS)
    v = torch.addcmul(s["b"].to(f64), (x - mean) * rstd, s["w"].to(f64))
    return quantised(v) if op == "ln_int8" else (v, mean[:, 0], rstd[:, 0])


def work(case):
    op, M = case["op"], case["M"]
    if op in ("linear", "gated"):
        K, N, n = case["K"], case["N"], 2 if op == "gated" else 1
        return {"bytes": M * K + n * N * K + M * N * SIZE[case["y"]] + 4 * (M + n * N) + (4 * N if case.get("bias") else 0),
                "flops": 2 * n * M * N * K}
    D = case["D"]
    x, y = M * D * SIZE[case["x"]], M * D * SIZE[case["y"]]
    if op == "ln":
        return {"bytes": x + y + 8 * M + 8 * D, "flops": 8 * M * D}
    if op == "ln_int8":
        return {"bytes": x + M * D + y + 4 * M + 8 * D, "flops": 11 * M * D}
    if op == "ln_bwd":
        return {"bytes": 2 * x + y + 8 * M + 12 * D, "flops": 15 * M * D}
    return {"bytes": x + M * D + y + 4 * M, "flops": 4 * M * D}
