"""Cases and plain forms of the operators on 8-bit activations.

Four operators, in the order in which a block of a transformer runs them:

  norm   root-mean-square norm of x + residual, output in 8 bits with a scale per row, or dense
  quant  rows of activations in 8 bits with a scale per row
  silu   silu(a) * b, output in 8 bits with a scale per row, or dense
  gemm   y = sx[m] sw[n] sum_k xq[m, k] wq[n, k] (+ bias[n]) for one or several weights over the same rows

"q8" is int8 (largest code 127), "f8" is float8_e4m3fn (largest value 448). Codes come back as the whole numbers
(int8) or the values (float8_e4m3fn) that they are in units of the row's scale, which comes back beside them.
A code is the nearest one to 127 p / max|p| (448 p / max|p|), ties to even, so the norm's own factor cancels; the plain
form takes it in 64 bits, because a quotient next to a rounding border would go either way in 32.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
TOP = {"q8": 127.0, "f8": 448.0}
EPS = 1e-6


def listed():
    return [
        # one token of the d_model 512 model between two blocks
        dict(name="norm_token_512", op="norm", M=1, K=512, dtype="fp32", out="q8", residual=True, pad=0),
        # a prefill batch of a wider model in bf16
        dict(name="norm_2048x4096_bf16", op="norm", M=2048, K=4096, dtype="bf16", out="q8", residual=True, pad=0),
        # the large batch of the d_model 512 model, E4M3 rows
        dict(name="norm_65536x512_f8", op="norm", M=65536, K=512, dtype="fp32", out="f8", residual=True, pad=0),
        # attention's output before wo: odd width, fp16, rows inside a wider buffer
        dict(name="quant_1000x1023_fp16", op="quant", M=1000, K=1023, dtype="fp16", out="q8", pad=9),
        dict(name="quant_16384x8192_f8", op="quant", M=16384, K=8192, dtype="bf16", out="f8", pad=0),
        # the gated product of the d_ff 2048 model's golden batch (5 x 16 rows)
        dict(name="silu_80x2048", op="silu", M=80, K=2048, dtype="fp32", out="q8", fused=False),
        # a long prefill; a and b are the halves of one fused projection's output
        dict(name="silu_8192x8192_f8", op="silu", M=8192, K=8192, dtype="bf16", out="f8", fused=True),
        # one token through a wide projection: the weights are all there is to read
        dict(name="gemm_1x8192x8192", op="gemm", M=1, N=8192, K=8192, fmt="q8", y="bf16", bias=False, count=1),
        # wq, wk, wv, wg of one d_model 512 block at the golden batch
        dict(name="gemm_80x512x512_by_4", op="gemm", M=80, N=512, K=512, fmt="q8", y="fp32", bias=False, count=4),
        # nothing is a multiple of anything
        dict(name="gemm_1111x1000x1030_f8", op="gemm", M=1111, N=1000, K=1030, fmt="f8", y="fp32", bias=True, count=1),
        # w1 at the large batch, fp32 output with its bias
        dict(name="gemm_65536x2048x512", op="gemm", M=65536, N=2048, K=512, fmt="q8", y="fp32", bias=True, count=1),
        # a prefill of a wide model in E4M3
        dict(name="gemm_8192x8192x8192_f8", op="gemm", M=8192, N=8192, K=8192, fmt="f8", y="bf16", bias=False, count=1),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm; every third one rounded to a multiple of 64 where it is large."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v > 256 and rng.random() < 1 / 3:
        v -= v % 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["norm", "quant", "silu", "gemm", "gemm"])
    if op == "gemm":
        K = _spread(rng, 16, 8192)
        N = _spread(rng, 16, 8192)
        M = _spread(rng, 1, max(1, min(65536, 8192 ** 3 // (N * K), 2 ** 27 // N)))
        count = rng.choice([1, 1, 2, 4]) if M * N * K <= 2 ** 33 else 1
        return dict(op=op, M=M, N=N, K=K, fmt=rng.choice(["q8", "f8"]), y=rng.choice(["fp32", "bf16", "fp16"]),
                    bias=rng.random() < 0.5, count=count)
    K = _spread(rng, 16, 16384)
    M = _spread(rng, 1, min(65536, 2 ** 25 // K))
    c = dict(op=op, M=M, K=K, dtype=rng.choice(["fp32", "bf16", "fp16"]))
    if op == "quant":
        return dict(c, out=rng.choice(["q8", "f8"]), pad=rng.choice([0, 0, 8, 3]))
    c["out"] = rng.choice(["q8", "q8", "f8", "f8", "same", "fp32"])
    if op == "silu":
        return dict(c, fused=rng.random() < 0.5)
    return dict(c, residual=rng.random() < 0.7, pad=rng.choice([0, 0, 8, 3]))


def _out_dtype(case):
    return DTYPES[case["dtype"]] if case["out"] == "same" else torch.float32


def _rows(g, M, K, dtype, pad=0):
    """Rows as they run through a model: a few channels far larger than the others, token norms that vary."""
    x = torch.randn(M, K + pad, generator=g, device="cuda")
    channel = torch.rand(K + pad, generator=g, device="cuda")
    x *= torch.where(channel > 0.99, 20.0, 1.0)
    x *= torch.exp(torch.randn(M, 1, generator=g, device="cuda") * 0.5)
    return x.to(dtype)[:, :K]


def _as_codes(p, fmt):
    """Codes and scales of rows p for the inputs of the matrix product."""
    top = p.abs().amax(1, keepdim=True)
    t = p * (TOP[fmt] / top)
    codes = t.round().to(torch.int8) if fmt == "q8" else t.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (top[:, 0] / TOP[fmt])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, K, op = case["M"], case["K"], case["op"]
    s = dict(case=case)
    if op == "gemm":
        N, fmt, y = case["N"], case["fmt"], DTYPES[case["y"]]
        s["x"], s["sx"] = _as_codes(_rows(g, M, K, torch.float32), fmt)
        s["w"] = []
        for _ in range(case["count"]):
            w = torch.randn(N, K, generator=g, device="cuda") * 0.02
            if fmt == "q8":
                payload, scale = _as_codes(w, fmt)
            else:
                payload, scale = w.to(torch.float8_e4m3fn).view(torch.uint8), None
            bias = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
            s["w"].append((payload, scale, bias, torch.empty(M, N, dtype=y, device="cuda")))
        return s
    T = DTYPES[case["dtype"]]
    if op == "silu":
        if case["fused"]:
            ab = _rows(g, M, 2 * K, T)
            s["a"], s["b"] = ab[:, :K], ab[:, K:]
        else:
            s["a"], s["b"] = _rows(g, M, K, T), _rows(g, M, K, T)
    else:
        s["x"] = _rows(g, M, K, T, case["pad"])
    if op == "norm":
        s["weight"] = 1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")
        s["residual"] = s["sum"] = None
        if case["residual"]:
            s["residual"] = _rows(g, M, K, T)
            s["sum"] = torch.empty(M, K, dtype=T, device="cuda")
    if case["out"] in TOP:
        s["out"] = (torch.empty(M, K, dtype=torch.int8 if case["out"] == "q8" else torch.uint8, device="cuda"),
                    torch.empty(M, dtype=torch.float32, device="cuda"))
    else:
        s["out"] = torch.empty(M, K, dtype=_out_dtype(case), device="cuda")
    return s


# ---- plain forms ----

def _plain_codes(p, r, fmt):
    """p [M, K] in 64 bits, r [M, 1] or 1: codes of p and the scale of r p, by row."""
    top = p.abs().amax(1, keepdim=True)
    scale = (top * r / TOP[fmt]).float()
    fine = torch.isfinite(scale)
    t = torch.where(fine & (top > 0), TOP[fmt] * p / top, 0.0)
    codes = t.round().to(torch.int8) if fmt == "q8" else t.float().to(torch.float8_e4m3fn)
    return {"codes": codes, "scale": torch.where(fine, scale, math.nan)[:, 0]}


def _plain_norm(s):
    case, x, w = s["case"], s["x"], s["weight"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    d = h.double()
    r = 1.0 / (d.square().mean(1, keepdim=True) + EPS).sqrt()
    if case["out"] in TOP:
        out = _plain_codes(d * w.double(), r, case["out"])
    else:
        out = {"y": (h.float() * r.float() * w).to(_out_dtype(case))}
    if s["residual"] is not None:
        out["sum"] = h
    return out


def _plain_silu(s):
    case = s["case"]
    if case["out"] in TOP:
        a = s["a"].double()
        return _plain_codes(a / (1.0 + torch.exp(-a)) * s["b"].double(), 1.0, case["out"])
    a = s["a"].float()
    return {"y": (a / (1.0 + torch.exp(-a)) * s["b"].float()).to(_out_dtype(case))}


def _plain_gemm(s):
    q8, ys = s["case"]["fmt"] == "q8", []
    x = (s["x"] if q8 else s["x"].view(torch.float8_e4m3fn)).float()
    for payload, scale, bias, y in s["w"]:
        w = (payload if q8 else payload.view(torch.float8_e4m3fn)).float()
        v = (x @ w.t()) * s["sx"][:, None]
        if scale is not None:
            v = v * scale
        if bias is not None:
            v = v + bias
        ys.append(v.to(y.dtype))
    return ys


# ---- the framework's calls ----

def _own_out(rtq, s):
    return rtq.A8Rows(*s["out"]) if s["case"]["out"] in TOP else s["out"]


def _own_codes(case, out):
    if case["out"] not in TOP:
        return {"y": out}
    return {"codes": out.codes if case["out"] == "q8" else out.codes.view(torch.float8_e4m3fn), "scale": out.scale}


def _own_run(s):
    import weight_only_quantized_rtq_amd as rtq
    case = s["case"]
    op = case["op"]
    fmt = case.get("out") if case.get("out") in TOP else None
    if op == "norm":
        out = _own_out(rtq, s)
        rtq.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], fmt=fmt, out=out, sum_out=s["sum"])
        out = _own_codes(case, out)
        if s["sum"] is not None:
            out["sum"] = s["sum"]
        return out
    if op == "quant":
        return _own_codes(case, rtq.quantize_rows(s["x"], fmt, out=_own_out(rtq, s)))
    if op == "silu":
        return _own_codes(case, rtq.silu_mul(s["a"], s["b"], fmt=fmt, out=_own_out(rtq, s)))
    x = rtq.A8Rows(s["x"], s["sx"])
    weights = [rtq.F8Weight(p) if scale is None else rtq.Q8Weight(p, scale) for p, scale, _, _ in s["w"]]
    if len(weights) == 1:
        return [rtq.gemm_a8(x, weights[0], y=s["w"][0][3], bias=s["w"][0][2])]
    rtq.project_a8([rtq.Projection(w, x, y, bias) for w, (_, _, bias, y) in zip(weights, s["w"])])
    return [y for _, _, _, y in s["w"]]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "quant":
        return _plain_codes(state["x"].double(), 1.0, state["case"]["out"])
    if op == "silu":
        return _plain_silu(state)
    return _plain_gemm(state)


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "gemm":
        N, n = case["N"], case["count"]
        size = SIZE[case["y"]]
        per = N * K + M * N * size + (4 * N if case["fmt"] == "q8" else 0) + (4 * N if case["bias"] else 0)
        return {"bytes": M * K + 4 * M + n * per, "flops": 2 * n * M * N * K}
    T = SIZE[case["dtype"]]
    out = M * K + 4 * M if case["out"] in TOP else M * K * (T if case["out"] == "same" else 4)
    if case["op"] == "quant":
        return {"bytes": M * K * T + out, "flops": 3 * M * K}
    if case["op"] == "silu":
        return {"bytes": 2 * M * K * T + out, "flops": 8 * M * K}
    return {"bytes": M * K * T * (3 if case["residual"] else 1) + 4 * K + out, "flops": 7 * M * K}


# ---- the definitions in 64 bits ----

def _exact_e4m3(t):
    """The nearest value with four significant bits and exponents of -6 and up, ties to even."""
    step = torch.exp2(torch.frexp(t).exponent.clamp(min=-5).double() - 4.0)
    return (t / step).round() * step


def _exact_rows(y, fmt):
    """Row values y in 64 bits; int8 codes are whole numbers and have no error of their own."""
    top = torch.linalg.vector_norm(y, ord=math.inf, dim=1)
    scale = top / TOP[fmt]
    if fmt == "q8":
        return {"codes": None, "scale": scale}
    return {"codes": _exact_e4m3(torch.where(top[:, None] > 0, y * TOP[fmt] / top[:, None], y)), "scale": scale}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        value = (lambda c: c.double()) if case["fmt"] == "q8" else (lambda c: c.view(torch.float8_e4m3fn).to(torch.float64))
        x = value(s["x"]) * s["sx"].double()[:, None]
        ys = []
        for payload, scale, bias, _ in s["w"]:
            w = value(payload) if scale is None else value(payload) * scale.double()[:, None]
            y = torch.mm(x, w.t())
            ys.append(y if bias is None else y + bias.double())
        return ys
    if op == "quant":
        return _exact_rows(s["x"].to(torch.float64), case["out"])
    if op == "silu":
        a, b = s["a"].to(torch.float64), s["b"].to(torch.float64)
        y = a * b * torch.sigmoid(a)
        return _exact_rows(y, case["out"]) if case["out"] in TOP else {"y": y}
    h = s["x"].to(torch.float64)
    out = {}
    if s["residual"] is not None:
        out["sum"] = h + s["residual"].to(torch.float64)
        h = out["sum"].to(s["x"].dtype).to(torch.float64)
    y = h * torch.rsqrt(torch.sum(h * h, 1, keepdim=True) / case["K"] + EPS) * s["weight"].to(torch.float64)
    out.update(_exact_rows(y, case["out"]) if case["out"] in TOP else {"y": y})
    return out
