"""Cases of the paged key/value cache: per-head norm and rotation of q and k, the write of k and v into the cache's
pages (bf16, or 8-bit rows with a scale each), reading sequences back, and the attention of one new token over them.

`run` computes an operator in plain torch operations, or, with `own`, by the framework's entry points."""
import math

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "int8": 1, "e4m3": 1}
EPS = 1e-6
TINY = 2.0 ** -100  # a row whose values are all below this counts as zero


def listed():
    return [
        # q and k of one new token, half-split rotation, grouped heads
        {"name": "rope_1_32x8x128", "op": "rope", "tokens": 1, "heads": 32, "kv": 8, "dim": 128, "norm": True, "inter": False,
         "rot": 128, "axes": 1},
        # an image's tokens at this repository's 24 heads: interleaved rotation over time, height and width
        {"name": "rope_4352_24x24x128_axes", "op": "rope", "tokens": 4352, "heads": 24, "kv": 24, "dim": 128, "norm": True,
         "inter": True, "rot": 128, "axes": 3},
        # one new token into an e4m3 cache
        {"name": "write_1_32x8x128_e4m3", "op": "write", "tokens": 1, "heads": 32, "kv": 8, "dim": 128, "norm": True,
         "inter": False, "rot": 128, "axes": 1, "type": "e4m3", "page": 16, "pages": 64},
        # a long prompt into an e4m3 cache, a quarter of each head rotated
        {"name": "write_8192_48x8x128_e4m3", "op": "write", "tokens": 8192, "heads": 48, "kv": 8, "dim": 128, "norm": True,
         "inter": False, "rot": 32, "axes": 1, "type": "e4m3", "page": 64, "pages": 160},
        # a prompt's next chunk into an int8 cache, and the whole sequence read back for a dense attention
        {"name": "chunk_777_of_5000_32x4x128_int8", "op": "chunk", "tokens": 777, "heads": 32, "kv": 4, "dim": 128, "norm": False,
         "inter": False, "rot": 128, "axes": 1, "type": "int8", "page": 32, "low": 5000, "high": 5000, "batch": 1},
        # three short sequences read back
        {"name": "read_3_upto100_8x64_bf16", "op": "read", "batch": 3, "low": 1, "high": 100, "kv": 8, "dim": 64, "type": "bf16",
         "page": 16},
        # ragged long sequences read back
        {"name": "read_16_upto16384_8x128_e4m3", "op": "read", "batch": 16, "low": 100, "high": 16384, "kv": 8, "dim": 128,
         "type": "e4m3", "page": 64},
        # the start of one conversation
        {"name": "attn_1_57_32x8x128_bf16", "op": "attn", "batch": 1, "low": 57, "high": 57, "heads": 32, "kv": 8, "dim": 128,
         "type": "bf16", "page": 16, "window": 0, "lse": False},
        # one long document, few rows: split over its length
        {"name": "attn_1_131072_64x8x128_int8", "op": "attn", "batch": 1, "low": 131072, "high": 131072, "heads": 64, "kv": 8,
         "dim": 128, "type": "int8", "page": 64, "window": 0, "lse": True},
        # a served batch of ragged lengths
        {"name": "attn_64_upto8192_32x8x128_e4m3", "op": "attn", "batch": 64, "low": 3, "high": 8192, "heads": 32, "kv": 8,
         "dim": 128, "type": "e4m3", "page": 32, "window": 0, "lse": False},
        # a batch at this repository's 24 heads, each with its own keys, unquantised
        {"name": "attn_32_upto4096_24x24x128_bf16", "op": "attn", "batch": 32, "low": 500, "high": 4096, "heads": 24, "kv": 24,
         "dim": 128, "type": "bf16", "page": 64, "window": 0, "lse": False},
        # a decoding step's two calls together: the new tokens of a batch into the cache, then their attention
        {"name": "step_33_upto2000_32x8x128_e4m3", "op": "step", "batch": 33, "low": 1, "high": 2000, "heads": 32, "kv": 8,
         "dim": 128, "norm": True, "inter": False, "rot": 128, "axes": 1, "type": "e4m3", "page": 16, "window": 0},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["rope", "write", "chunk", "read", "attn", "attn", "attn", "step"])
    kv = rng.choice([1, 2, 4, 5, 8, 16, 24])
    group = rng.choice([1, 1, 2, 3, 4, 6, 8, 12, 16])
    c = {"op": op, "kv": kv, "dim": rng.choice([64, 128, 128, 128, 256]), "page": rng.choice([16, 32, 48, 64, 128])}
    if op != "read":
        c["heads"] = kv * group
    if op in ("rope", "write", "chunk", "step"):
        c["norm"], c["inter"] = rng.random() < 0.6, rng.random() < 0.4
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, c["dim"] // 4])
        c["axes"] = rng.choice([1, 1, 2, 3])
    if op != "rope":
        c["type"] = rng.choice(["bf16", "e4m3"] if op in ("write", "step") else ["bf16", "int8", "e4m3"])
    width = c["kv"] * c["dim"]
    if op in ("rope", "write"):
        most = min(16384, 50_000_000 // ((c["heads"] + 2 * kv) * c["dim"]))
        c["tokens"] = _log_int(rng, 1, most)
        if op == "write":
            c["pages"] = -(-c["tokens"] // c["page"]) + rng.randint(1, 30)
        return c
    total = _log_int(rng, 200, min(131072, 300_000_000 // (2 * width) // 2))  # about so many tokens in all
    c["batch"] = 1 if op == "chunk" else min(256, _log_int(rng, 1, max(2, total // 4)))
    high = max(2, int(2 * total / c["batch"] / 1.1)) if c["batch"] > 1 else total
    c["low"], c["high"] = (high if c["batch"] == 1 else max(1, high // 10)), high
    if op == "chunk":
        c["tokens"] = _log_int(rng, 1, min(high, 20_000_000 // (c["heads"] * c["dim"])))
    if op in ("attn", "step"):
        c["window"] = 0 if rng.random() < 0.75 else _log_int(rng, 1, high)
    if op == "attn":
        c["lse"] = rng.random() < 0.5
    return c


def _lengths(case):
    """Lengths spread evenly over the range: their sum does not depend on the seed."""
    n = case["batch"]
    return [round(case["low"] + (case["high"] - case["low"]) * i / max(1, n - 1)) for i in range(n)]


def _rotary(case):
    """Frequencies of the rotated pairs, and each pair's axis: an axis has its own run of frequencies."""
    pairs, axes = case["rot"] // 2, case["axes"]
    sizes = [pairs] if axes == 1 else [pairs // 8, pairs - pairs // 8] if axes == 2 else [pairs // 8, (pairs - pairs // 8) // 2]
    sizes += [pairs - sum(sizes)] if axes == 3 else []
    freq = [10000.0 ** (-i / n) for n in sizes for i in range(n)]
    axis = [a for a, n in enumerate(sizes) for _ in range(n)]
    return (torch.tensor(freq, dtype=torch.float64, device="cuda"), torch.tensor(axis, dtype=torch.int32, device="cuda"))


def _projection(s, case, tokens, g):
    """The packed product of q, k and v of some tokens, as views, with what their norm and rotation take."""
    h, kv, d = case["heads"], case["kv"], case["dim"]
    x = torch.randn(tokens, (h + 2 * kv) * d, generator=g, device="cuda")
    x *= (0.5 + torch.rand((h + 2 * kv) * d, generator=g, device="cuda"))
    x = x.bfloat16()
    s["q"] = x[:, :h * d].view(tokens, h, d)
    s["k"] = x[:, h * d:(h + kv) * d].view(tokens, kv, d)
    s["v"] = x[:, (h + kv) * d:].view(tokens, kv, d)
    s["wq"] = s["wk"] = None
    if case["norm"]:
        s["wq"], s["wk"] = ((1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2))
    s["freq"], s["axis"] = _rotary(case)


def _cache(s, case, pages, g):
    """A cache in use: normal rows at their scales (bf16: the rows)."""
    shape = (pages, case["kv"], case["page"], case["dim"])
    for name in ("k", "v"):
        if case["type"] == "int8":
            s["c" + name] = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
        else:
            x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
            s["c" + name] = x if case["type"] == "bf16" else (x * 100).clamp_(-448, 448).to(DTYPE["e4m3"])
        s["s" + name] = None
        if case["type"] != "bf16":
            r = torch.rand(shape[:3], generator=g, device="cuda") + 0.5
            s["s" + name] = r * (1.0 / 64 if case["type"] == "int8" else 1.0 / 100)


def _tables(s, case, g):
    """Pages of the sequences, scattered over the pool, and their lengths in a shuffled order."""
    lengths = torch.tensor(_lengths(case), device="cuda")
    lengths = lengths[torch.randperm(len(lengths), generator=g, device="cuda")]
    width = max(1, -(-case["high"] // case["page"]))
    pages = case["batch"] * width
    s["table"] = torch.randperm(pages, generator=g, device="cuda").view(case["batch"], width).to(torch.int32)
    s["lengths"] = lengths.to(torch.int32)
    return pages


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "rope":
        _projection(s, case, case["tokens"], g)
        if case["axes"] == 1:  # the tokens of a text, or one far into it
            first = torch.randint(0, 100000, (1, 1), generator=g, device="cuda")
            s["pos"] = first + torch.arange(case["tokens"], device="cuda")
        else:
            s["pos"] = torch.randint(-64, 2000, (case["axes"], case["tokens"]), generator=g, device="cuda")
        return s
    if op == "write":
        _projection(s, case, case["tokens"], g)
        _cache(s, case, case["pages"], g)
        s["slots"] = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:case["tokens"]]
        s["pos"] = torch.randint(0, 100000, (case["axes"], case["tokens"]), generator=g, device="cuda")
        return s
    _cache(s, case, _tables(s, case, g), g)
    if op in ("chunk", "read"):
        s["rows"] = sum(_lengths(case))
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), s["lengths"].cumsum(0)])
    if op == "chunk":  # the last tokens of the sequence are new
        _projection(s, case, case["tokens"], g)
        t = torch.arange(case["high"] - case["tokens"], case["high"], device="cuda")
        s["pos"] = t.expand(case["axes"], -1).contiguous()
        s["slots"] = s["table"][0, t // case["page"]].long() * case["page"] + t % case["page"]
    elif op == "step":  # each sequence's last token is new
        _projection(s, case, case["batch"], g)
        t = s["lengths"].long() - 1
        s["pos"] = t.expand(case["axes"], -1).contiguous()
        page = s["table"].gather(1, (t // case["page"]).unsqueeze(1))[:, 0]
        s["slots"] = page.long() * case["page"] + t % case["page"]
        s["qa"] = None
    elif op == "attn":
        q = torch.randn(case["batch"], case["heads"], case["dim"], generator=g, device="cuda")
        s["qa"] = (q * 1.5).bfloat16()
    return s


def _norm_rope(s, x, w):
    """fp32 values of x after its norm and rotation; the angles in 64 bits."""
    x = x.float()
    if w is not None:
        x = x * (1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)) * w.float()
    angle = (s["pos"].view(s["axes"], -1)[s["axis"].long()].double() * s["freq"][:, None]).t().unsqueeze(1)
    cos, sin = angle.cos().float(), angle.sin().float()
    r, rest = x[..., :s["rot"]], x[..., s["rot"]:]
    if s["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :s["rot"] // 2], r[..., s["rot"] // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _put(s, name, x):
    """Rows x [tokens, heads, dim] in fp32 to the cache's slots."""
    page, at = s["slots"] // s["page"], s["slots"] % s["page"]
    if s["type"] == "bf16":
        s["c" + name][page, :, at] = x.bfloat16()
        return
    top = x.abs().amax(-1, keepdim=True)
    inv = torch.where(top >= TINY, QMAX[s["type"]] * (1 / top), torch.zeros_like(top))
    if s["type"] == "int8":
        code = (x.double() * inv.double()).round().to(torch.int8)  # 64 bits: ratios next to a half
    else:
        code = (x * inv).to(DTYPE["e4m3"])
    s["c" + name].view(torch.uint8)[page, :, at] = code.view(torch.uint8)
    s["s" + name][page, :, at] = torch.where(top >= TINY, top / QMAX[s["type"]], torch.zeros_like(top))[..., 0]


def _got(s, name):
    """All sequences' cached rows in fp32, padded: [batch, heads, width * page, dim]."""
    t = s["table"].long()
    x = s["c" + name].view(torch.uint8)[t].view(DTYPE[s["type"]]) if s["type"] == "e4m3" else s["c" + name][t]
    x = x.float()
    if s["type"] != "bf16":
        x = x * s["s" + name][t].unsqueeze(-1)
    return x.transpose(1, 2).flatten(2, 3)


def _inside(s, width):
    at = torch.arange(width, device="cuda")
    n = s["lengths"].long()[:, None]
    first = n - s["window"] if s.get("window") else torch.zeros_like(n)
    return (at < n) & (at >= first)


def _attend(s, q):
    k, v = _got(s, "k"), _got(s, "v")
    inside = _inside(s, k.shape[2])[:, None, None]
    b, h, d = q.shape
    x = torch.matmul(q.float().view(b, s["kv"], -1, d), k.transpose(2, 3)) * d ** -0.5
    x = x.masked_fill(~inside, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.view(b, h, d).bfloat16(), (top + torch.log(total)).view(b, h)


def _state_of(s):
    got = {"ck": s["ck"], "cv": s["cv"]}
    if s["type"] != "bf16":
        got["sk"], got["sv"] = s["sk"], s["sv"]
    return got


def _read(s):
    rows = _inside({**s, "window": 0}, s["table"].shape[1] * s["page"])
    return {n: _got(s, n).transpose(1, 2)[rows].bfloat16() for n in ("k", "v")}


def _plain(s):
    op = s["op"]
    if op == "rope":
        return {"q": _norm_rope(s, s["q"], s["wq"]).bfloat16(), "k": _norm_rope(s, s["k"], s["wk"]).bfloat16()}
    got = {}
    if op in ("write", "chunk", "step"):
        q = got["q"] = _norm_rope(s, s["q"], s["wq"]).bfloat16()
        _put(s, "k", _norm_rope(s, s["k"], s["wk"]))
        _put(s, "v", s["v"].float())
    if op == "write":
        got.update(_state_of(s))
    elif op in ("chunk", "read"):
        got.update(_read(s))
    elif op == "step":
        got["o"] = _attend(s, q)[0]
        got.update(_state_of(s))
    else:
        got["o"], lse = _attend(s, s["qa"])
        if s["lse"]:
            got["lse"] = lse
    return got


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp8_quant_row_gb300 as fq

    op = s["op"]
    if op == "rope":
        q, k = fq.qk_norm_rope(s["q"], s["k"], s["freq"], s["pos"], axis=s["axis"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                               interleaved=s["inter"])
        return {"q": q, "k": k}
    cache = fq.PagedCache(s["ck"], s["cv"], s["sk"], s["sv"])
    got = {}
    if op in ("write", "chunk", "step"):
        q = got["q"] = fq.cache_write(s["k"], s["v"], cache, s["slots"], q=s["q"], inv_freq=s["freq"], positions=s["pos"],
                                      axis=s["axis"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=s["inter"])
    if op == "write":
        got.update(_state_of(s))
    elif op in ("chunk", "read"):
        got["k"], got["v"] = fq.cache_read(cache, s["table"], s["offsets"], s["rows"])
    elif op == "step":
        got["o"] = fq.paged_attention(q, cache, s["table"], s["lengths"], window=s["window"])
        got.update(_state_of(s))
    elif s["lse"]:
        got["o"], got["lse"] = fq.paged_attention(s["qa"], cache, s["table"], s["lengths"], window=s["window"], return_lse=True)
    else:
        got["o"] = fq.paged_attention(s["qa"], cache, s["table"], s["lengths"], window=s["window"])
    return got


def work(case):
    op, kv, d = case["op"], case["kv"], case["dim"]
    row = d * BYTES[case["type"]] + (0 if case["type"] == "bf16" else 4) if op != "rope" else 2 * d  # of k or v, as stored
    if op in ("rope", "write", "chunk", "step"):
        t = case["batch"] if op == "step" else case["tokens"]
        h = case["heads"]
        size = t * (4 * h * d + 2 * kv * d + kv * row + (0 if op == "rope" else 2 * kv * d + kv * row))
        size += t * 8 * case["axes"] + case["rot"] * 6 + (0 if op == "rope" else 8 * t)
        flops = t * (h + kv) * d * (8 if case["norm"] else 4)
        if op in ("rope", "write"):
            return {"bytes": size, "flops": flops}
    else:
        size = flops = 0
    lengths = _lengths(case)
    if case.get("window"):
        lengths = [min(n, case["window"]) for n in lengths]
    n, pages = sum(lengths), sum(-(-x // case["page"]) for x in lengths)
    size += 2 * n * kv * row + 4 * pages
    if op in ("chunk", "read"):
        return {"bytes": size + 4 * n * kv * d, "flops": flops + 2 * n * kv * d}
    b, h = case["batch"], case["heads"]
    size += b * h * d * (2 if op == "step" else 4) + 4 * b + (4 * b * h if case.get("lse") else 0)
    return {"bytes": size, "flops": flops + 4 * n * h * d}


def _turned(s, x, w):
    """Norm and rotation in 64 bits, pairs as complex numbers."""
    x = x.double()
    if w is not None:
        n = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        x = x * w.double() / torch.sqrt(n * n / s["dim"] + EPS)
    where = s["pos"].reshape(s["axes"], -1).t().double()  # [tokens, axes]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), where[:, s["axis"].long()] * s["freq"])[:, None]
    half = s["rot"] // 2
    y = x.clone()
    if s["inter"]:
        z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:2], half, 2).contiguous()) * turn
        y[..., :2 * half] = torch.view_as_real(z).reshape(*x.shape[:2], 2 * half)
    else:
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def _stored(kind, x):
    """Codes, as numbers, and scales of 64-bit rows."""
    size = torch.linalg.vector_norm(x, ord=math.inf, dim=-1)
    t = x * (QMAX[kind] / size).unsqueeze(-1)
    step = torch.ones_like(t)
    if kind == "e4m3":  # four significant bits, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(t / step) * step).clamp(-QMAX[kind], QMAX[kind]), size / QMAX[kind]


def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    op, kind = case["op"], case.get("type")
    got, pool = {}, {}
    if op != "rope":
        for n in ("k", "v"):
            scale = None if kind == "bf16" else s["s" + n].double()
            pool[n] = [s["c" + n].double(), scale]
    if op in ("rope", "write", "chunk", "step"):
        q, k = _turned(s, s["q"], s["wq"]), _turned(s, s["k"], s["wk"])
        got["q"] = q
        if op == "rope":
            return {"q": q, "k": k}
        page, at = s["slots"] // case["page"], s["slots"] % case["page"]
        for n, x in (("k", k), ("v", s["v"].double())):
            if kind == "bf16":
                pool[n][0][page, :, at] = x if op == "write" else x.bfloat16().double()
            else:
                pool[n][0][page, :, at], pool[n][1][page, :, at] = _stored(kind, x)
        if op != "chunk":
            got.update(ck=pool["k"][0], cv=pool["v"][0])
            if kind != "bf16":
                got.update(sk=pool["k"][1], sv=pool["v"][1])
        if op == "write":
            return got
        q = q.bfloat16().double()  # (as the attention takes it)
    else:
        q = s["qa"].double() if op == "attn" else None
    out, lse, ks, vs = [], [], [], []
    for i, n in enumerate(s["lengths"].tolist()):
        first = max(0, n - case["window"]) if case.get("window") else 0
        t = torch.arange(first, n, device="cuda")
        page, at = s["table"][i].long()[t // case["page"]], t % case["page"]
        k, v = (pool[x][0][page, :, at] * (1 if kind == "bf16" else pool[x][1][page, :, at].unsqueeze(-1)) for x in ("k", "v"))
        if q is None or op == "chunk":
            ks.append(k)
            vs.append(v)
            continue
        qi = q[i].view(case["kv"], -1, case["dim"])
        x = torch.einsum("hgd,thd->hgt", qi, k) / math.sqrt(case["dim"])
        lse.append(torch.logsumexp(x, -1).flatten())
        out.append(torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v).reshape(case["heads"], -1))
    if op in ("chunk", "read"):
        return {**got, "k": torch.cat(ks), "v": torch.cat(vs)}
    got["o"] = torch.stack(out)
    if case.get("lse"):
        got["lse"] = torch.stack(lse)
    return got
