"""Cases of the 8-bit row operators: RMSNorm with residual -> 8-bit rows with a scale each, SiLU(gate)*up -> the
same, and the product of 8-bit integer rows and weights with a scale for each token and channel.

`run` computes an operator in plain torch operations, or, with `own`, by the framework's entry points."""
import math

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
OUT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
TINY = 2.0 ** -100  # a row whose products are all below this counts as zero
EXP_FLOOR = -87.0   # silu below this gate value counts as zero (its exponential leaves fp32's range)


def listed():
    return [
        # one new token between two layers of a decoding model
        {"name": "norm_1x6144_res_int8", "op": "norm", "rows": 1, "cols": 6144, "residual": True, "type": "int8"},
        # a ragged batch of new tokens, first layer (no residual yet)
        {"name": "norm_127x5120_e4m3", "op": "norm", "rows": 127, "cols": 5120, "residual": False, "type": "e4m3"},
        # one image's or prompt's tokens at this repository's wide model width
        {"name": "norm_4608x6144_res_int8", "op": "norm", "rows": 4608, "cols": 6144, "residual": True, "type": "int8"},
        # a long prompt batch
        {"name": "norm_16384x8192_res_e4m3", "op": "norm", "rows": 16384, "cols": 8192, "residual": True, "type": "e4m3"},
        # gate and up of one new token
        {"name": "silu_1x18432_int8", "op": "silu", "rows": 1, "cols": 18432, "type": "int8"},
        # gate and up of a ragged batch, odd multiple of eight columns
        {"name": "silu_333x5640_e4m3", "op": "silu", "rows": 333, "cols": 5640, "type": "e4m3"},
        # gate and up of a whole prompt at this repository's MLP width
        {"name": "silu_4608x18432_int8", "op": "silu", "rows": 4608, "cols": 18432, "type": "int8"},
        # decoding: one token through an attention output projection
        {"name": "mm_1x6144x6144", "op": "mm", "m": 1, "n": 6144, "k": 6144, "out": "bf16", "bias": False},
        # decoding: a small batch through the gate/up projection
        {"name": "mm_16x36864x6144", "op": "mm", "m": 16, "n": 36864, "k": 6144, "out": "bf16", "bias": False},
        # a ragged batch, biased fp32 output (logits of a small, odd vocabulary)
        {"name": "mm_201x10007x4096_fp32", "op": "mm", "m": 201, "n": 10007, "k": 4096, "out": "fp32", "bias": True},
        # a prompt through the gate/up projection
        {"name": "mm_4608x36864x6144", "op": "mm", "m": 4608, "n": 36864, "k": 6144, "out": "bf16", "bias": False},
        # a prompt through the down projection (long sums)
        {"name": "mm_4608x6144x18432", "op": "mm", "m": 4608, "n": 6144, "k": 18432, "out": "bf16", "bias": True},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "silu", "mm", "mm"])
    if op == "norm":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": _log_int(rng, 64, 8192, 8),
                "residual": rng.random() < 0.7, "type": rng.choice(["int8", "e4m3"])}
    if op == "silu":
        return {"op": op, "rows": _log_int(rng, 1, 4608), "cols": _log_int(rng, 64, 18432, 8),
                "type": rng.choice(["int8", "e4m3"])}
    return {"op": op, "m": _log_int(rng, 1, 4608), "n": _log_int(rng, 64, 12288), "k": _log_int(rng, 256, 18432, 16),
            "out": rng.choice(["bf16", "bf16", "fp32"]), "bias": rng.random() < 0.3}


def _rows(g, rows, cols):
    """Activations as a residual stream has them: normal, one channel in a hundred twenty times as large."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.rand(cols, generator=g, device="cuda") < 0.01
    return torch.where(loud, x * 20, x)


def _codes(g, rows, cols):
    """int8 codes and fp32 scales of normal rows."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    s = x.abs().amax(1) / 127
    return (x / s[:, None]).round_().to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        s["x"] = _rows(g, case["rows"], case["cols"]).bfloat16()
        s["r"] = _rows(g, case["rows"], case["cols"]).bfloat16() if case["residual"] else None
        s["w"] = (1 + 0.1 * torch.randn(case["cols"], generator=g, device="cuda")).bfloat16()
    elif case["op"] == "silu":
        gu = torch.randn(case["rows"], 2 * case["cols"], generator=g, device="cuda").mul_(1.5).bfloat16()
        s["gate"], s["up"] = gu[:, :case["cols"]], gu[:, case["cols"]:]
    else:
        s["a"], sa = _codes(g, case["m"], case["k"])
        s["w"], sw = _codes(g, case["n"], case["k"])
        s["sa"], s["sw"] = sa, sw * 0.02
        s["b"] = torch.randn(case["n"], generator=g, device="cuda").bfloat16() if case["bias"] else None
    return s


def _quantise(p, top, kind):
    """Codes of exact products p (fp32) with row maxima top: the ratio is rounded once for int8, and for e4m3 to
    fp32 and then to the code."""
    inv = torch.where(top >= TINY, QMAX[kind] / top, torch.zeros_like(top))
    if kind == "int8":
        return (p.double() * inv.double()).round_().to(torch.int8)  # 64 bits: ratios next to a half
    return (p * inv).to(torch.float8_e4m3fn)


def _plain(s):
    if s["op"] == "norm":
        h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).bfloat16()
        hf = h.float()
        p = hf * s["w"].float()
        top = p.abs().amax(1, keepdim=True)
        rstd = 1 / torch.sqrt(hf.square().mean(1, keepdim=True) + EPS)
        scale = torch.where(top >= TINY, top * rstd / QMAX[s["type"]], torch.zeros_like(top))
        q = _quantise(p, top, s["type"])
        return {"q": q, "scale": scale[:, 0]} if s["r"] is None else {"h": h, "q": q, "scale": scale[:, 0]}
    if s["op"] == "silu":
        g = s["gate"].double()  # 64 bits: values next to a bf16 border
        a = torch.where(g < EXP_FLOOR, torch.zeros_like(g), g / (1 + torch.exp(-g))).float().bfloat16()
        p = a.float() * s["up"].float()
        top = p.abs().amax(1, keepdim=True)
        scale = torch.where(top >= TINY, top / QMAX[s["type"]], torch.zeros_like(top))
        return {"q": _quantise(p, top, s["type"]), "scale": scale[:, 0]}
    out = s["a"].float() @ s["w"].float().t() * s["sw"] * s["sa"][:, None]
    if s["b"] is not None:
        out = out + s["b"].float()
    return out.to(OUT[s["out"]])


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp8_quant_row_gb300 as fq

    if s["op"] == "norm":
        got = fq.rms_norm_quant(s["x"], s["w"], residual=s["r"], dtype=DTYPE[s["type"]], eps=EPS)
        return dict(zip(("q", "scale") if s["r"] is None else ("h", "q", "scale"), got))
    if s["op"] == "silu":
        q, scale = fq.silu_mul_quant(s["gate"], s["up"], dtype=DTYPE[s["type"]])
        return {"q": q, "scale": scale}
    return fq.int8_matmul(s["a"], s["sa"], s["w"], s["sw"], bias=s["b"], out_dtype=OUT[s["out"]])


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (7 if case["residual"] else 3) + 2 * case["cols"] + 4 * case["rows"], "flops": 6 * n}
    if case["op"] == "silu":
        n = case["rows"] * case["cols"]
        return {"bytes": 5 * n + 4 * case["rows"], "flops": 10 * n}
    m, n, k = case["m"], case["n"], case["k"]
    size = 2 if case["out"] == "bf16" else 4
    return {"bytes": m * k + n * k + size * m * n + 4 * (m + n) + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits. Codes of int8 rows are whole numbers and have no 64-bit
    value of their own: None."""
    s = prepare(case, seed)
    if case["op"] == "mm":
        acc = torch.matmul(s["a"].double(), s["w"].double().t())
        acc *= s["sa"].double().unsqueeze(1) * s["sw"].double().unsqueeze(0)
        return acc if s["b"] is None else acc.add_(s["b"].double())
    qmax = 127 if case["type"] == "int8" else 448
    got = {}
    if case["op"] == "norm":
        if s["r"] is None:
            h = s["x"].double()
        else:
            got["h"] = s["x"].double() + s["r"].double()
            h = got["h"].bfloat16().double()
        v = h * s["w"].double()
        size = torch.linalg.vector_norm(v, ord=math.inf, dim=1)
        got["scale"] = size / torch.sqrt(torch.linalg.vector_norm(h, dim=1).square() / case["cols"] + EPS) / qmax
    else:
        v = s["gate"].double()
        v = (v * torch.sigmoid(v)).bfloat16().double() * s["up"].double()
        size = torch.linalg.vector_norm(v, ord=math.inf, dim=1)
        got["scale"] = size / qmax
    got["q"] = None
    if case["type"] == "e4m3":  # four significant bits, steps of 2^-9 below 2^-6, by arithmetic on the values
        t = v * (qmax / size).unsqueeze(1)
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
        got["q"] = (torch.round(t / step) * step).clamp(-448, 448)
    return got
