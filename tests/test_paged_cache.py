"""qk_norm_rope, cache_write, cache_read and paged_attention: against plain 64-bit implementations
(GPU), and their refusals (host only)."""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import pytest
import torch

import fp8_quant_row_gb300 as fq
from fp8_quant_row_gb300 import _capi

OK, NULL, ALIGN, SHAPE, UNSUPPORTED, ALIAS, CUDA, VALUE = range(8)
A = 1 << 32  # fake device addresses, never dereferenced
gpu = pytest.mark.gpu
E4M3, BF16, INT8 = torch.float8_e4m3fn, torch.bfloat16, torch.int8
TYPES = [BF16, INT8, E4M3]
QMAX = {INT8: 127.0, E4M3: 448.0}
TINY = 2.0 ** -100
EPS = 1e-6


def ids(v):
    return str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None


@pytest.fixture(scope="module")
def L():
    fq.build()
    return _capi.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(BF16)


# ------------------------------------------------------------------------------------------
# plain forms, 64 bits
# ------------------------------------------------------------------------------------------

def plain_heads(x, w, inv_freq=None, positions=None, axis=None, interleaved=False, eps=EPS):
    """(value, size): the normed and rotated heads, and |a| + |b| of each value's pair."""
    n = x.double()
    if w is not None:
        n = n * w.double() / torch.sqrt(n.square().mean(-1, keepdim=True) + eps)
    if inv_freq is None:
        return n, n.abs()
    pos = positions.view(-1, x.shape[0]).double()
    axis = torch.zeros(len(inv_freq), dtype=torch.int32, device=x.device) if axis is None else axis
    t = (pos[axis.long()] * inv_freq[:, None]).t()[:, None]
    p = len(inv_freq)
    y, size = n.clone(), n.abs()
    at = (slice(0, 2 * p, 2), slice(1, 2 * p, 2)) if interleaved else (slice(0, p), slice(p, 2 * p))
    a, b = n[..., at[0]], n[..., at[1]]
    y[..., at[0]], y[..., at[1]] = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    for s in at:
        size[..., s] = a.abs() + b.abs()
    return y, size


# fp32 chain of a value before its last rounding: the sum of squares takes a square through at most
# 16 fused additions in a lane and 4 of lanes, halved by the root (10 units of 2^-24), the root, its
# two products and the mean with eps 4 more; cos and sin are off by the turn's last place, its
# conversion, the series and its roundings, 5 units; product and fused sum 2; 1 for second-order terms
# and 2 for the 64-bit form's own angles at positions up to 2^20: 24 units of |a| + |b|.
CHAIN = 24 * 2.0 ** -24


def near_bf16(got, y, size):
    d = (got.double() - y).abs()
    assert bool((d <= 2.0 ** -8 * (y.abs() + CHAIN * size) + CHAIN * size).all()), float((d / size.clamp_min(1e-30)).max())


def near_codes(code, scale, y, size):
    """Codes times scales within half a step (of the value's own code for e4m3): inv times scale is one
    but for three roundings, e4m3 rounds the product to fp32 first (2^-22 of the value in all)."""
    kind = code.dtype
    got = code.double() * scale.double()[..., None]
    s = scale.double()[..., None]
    half = 0.5 * s if kind == INT8 else torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s)
    err = CHAIN * size * (1 if kind == INT8 else 1 + 2.0 ** -4)
    tol = half * (1 + 2.0 ** -20) + err + 2.0 ** -22 * y.abs()
    assert bool(((got - y).abs() <= tol).all()), float(((got - y).abs() / s).max())
    # the scale: the row's largest value, off as the chain
    top = y.abs().amax(-1)
    worst = (CHAIN * size).amax(-1) + 2.0 ** -23 * top
    assert bool(((scale.double() * QMAX[kind] - top).abs() <= worst).all())


def exact_codes(x, kind):
    """Codes and scales of bf16 rows as they are, bit for bit."""
    p = x.double()
    top = p.abs().amax(-1, keepdim=True)
    ok = torch.isfinite(p).all(-1, keepdim=True) & (top >= TINY)
    inv = torch.where(ok, top.float().reciprocal() * QMAX[kind], 0.0)
    t = torch.where(ok, p, 0.0) * inv.double()
    code = t.round().to(INT8) if kind == INT8 else t.float().to(E4M3)
    scale = torch.where(ok, top / QMAX[kind], 0.0).float()
    return code, torch.where(torch.isfinite(p).all(-1, keepdim=True), scale, float("nan"))[..., 0]


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return torch.equal(bits(a), bits(b))


# ------------------------------------------------------------------------------------------
# qk_norm_rope
# ------------------------------------------------------------------------------------------

ROTATIONS = [None, ("halves", 1), ("pairs", 1), ("pairs", 0.5), ("halves", 0.5), ("halves", 0.25),
             ("halves", 0.75), ("odd", 1)]


def rotary(dim, how, tokens, axes, seed):
    if how is None:
        return {}
    kind, part = how
    pairs = int(dim * part) // 2
    if kind == "odd":  # interleaved, an odd number of pairs
        pairs, kind = dim // 2 - 5, "pairs"
    f = torch.tensor([10000.0 ** (-i / pairs) for i in range(pairs)], dtype=torch.float64, device="cuda")
    axis = torch.randint(0, axes, (pairs,), generator=gen(seed), device="cuda", dtype=torch.int32)
    pos = torch.randint(-100, 1 << 20, (axes, tokens), generator=gen(seed + 1), device="cuda")
    return dict(inv_freq=f, positions=pos if axes > 1 else pos[0].int(), axis=axis if axes > 1 else None,
                interleaved=kind == "pairs")


@gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("how", ROTATIONS, ids=str)
@pytest.mark.parametrize("tokens,heads,kv,axes", [(1, 32, 8, 1), (5, 3, 1, 3), (333, 24, 24, 2)])
@pytest.mark.parametrize("norm", [False, True])
def test_qk_norm_rope(dim, how, tokens, heads, kv, axes, norm):
    qkv = normal((tokens, (heads + 2 * kv) * dim), 1, 3.0)  # a packed product
    q, k = qkv[:, :heads * dim].view(tokens, heads, dim), qkv[:, heads * dim:(heads + kv) * dim].view(tokens, kv, dim)
    r = rotary(dim, how, tokens, axes, 2)
    wq, wk = ((1 + 0.2 * normal((dim,), s).float()).to(BF16) if norm else None for s in (3, 4))
    got = fq.qk_norm_rope(q, k, q_weight=wq, k_weight=wk, eps=1e-5, **r)
    for g, x, w in zip(got, (q, k), (wq, wk)):
        assert g.shape == x.shape and g.is_contiguous()
        near_bf16(g, *plain_heads(x, w, eps=1e-5, **r))
        if how is not None and r["inv_freq"].numel() * 2 < dim and not norm:  # the rest passes
            assert same(g[..., 2 * r["inv_freq"].numel():], x[..., 2 * r["inv_freq"].numel():])


@gpu
def test_qk_norm_rope_in_place_streams_and_guards():
    from tests.gpu_util import Guarded
    t, h, kv, d = 37, 5, 3, 128
    q, k = normal((t, h, d), 1), normal((t, kv, d), 2)
    r = rotary(d, ("halves", 0.5), t, 1, 3)
    w = normal((d,), 4)
    want = fq.qk_norm_rope(q, k, q_weight=w, k_weight=w, **r)
    gq, gk = Guarded((t, h, d), BF16), Guarded((t, kv, d), BF16)
    got = fq.qk_norm_rope(q, k, q_weight=w, k_weight=w, q_out=gq.tensor, k_out=gk.tensor, **r)
    assert all(same(a, b) for a, b in zip(got, want)) and gq.intact() and gk.intact()
    packed = torch.cat([q.view(t, -1), k.view(t, -1)], 1)
    qv, kk = packed[:, :h * d].view(t, h, d), packed[:, h * d:].view(t, kv, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fq.qk_norm_rope(qv, kk, q_weight=w, k_weight=w, q_out=qv, k_out=kk, stream=s, **r)
    torch.cuda.current_stream().wait_stream(s)
    assert got[0] is qv and same(qv, want[0]) and same(kk, want[1])
    q0, k0 = fq.qk_norm_rope(q[:0], k[:0], q_weight=w)
    assert q0.shape == (0, h, d) and k0.shape == (0, kv, d)


def turned(x, freq, pos):
    """cos and sin of freq * pos, reduced exactly."""
    tau = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    t = Fraction(freq) * pos
    t = float(t - tau * round(t / tau))
    return math.cos(t), math.sin(t)


@gpu
@pytest.mark.parametrize("pos", [0, 1, -1, 4097, 2 ** 24 + 1, -2 ** 31, 2 ** 31 - 1, 2 ** 40 + 12345])
def test_far_positions(pos):
    """The step is the double's to 2^-54 turns at most (product and rounding: 2^-53 of itself each), so
    at position p an angle is off by at most |p| 2^-52 turns beside the chain's."""
    d = 128
    f = torch.tensor([10000.0 ** (-i / 64) for i in range(64)], dtype=torch.float64, device="cuda")
    q = torch.zeros(1, 1, d, dtype=BF16, device="cuda")
    q[..., :64] = 1.0
    p = torch.tensor([pos], device="cuda")
    want = torch.zeros(d, dtype=torch.float64)
    for i, x in enumerate(f.tolist()):
        want[i], want[64 + i] = turned(1.0, x, pos)
    got, _ = fq.qk_norm_rope(q, q, f, p)
    err = (got[0, 0].double().cpu() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + CHAIN + abs(pos) * 2.0 ** -52 * 2 * math.pi).all())
    if -2 ** 31 <= pos < 2 ** 31:
        assert same(fq.qk_norm_rope(q, q, f, p.int())[0], got)


@gpu
def test_rotation_keeps_what_is_not_finite_apart():
    """Values that are not rotated pass as they are, beside rotated ones that are not finite."""
    q = normal((2, 3, 128), 1)
    q[0, 0, 100] = float("inf")
    q[1, 2, 127] = float("nan")
    f, _ = fq.rotary_axes((32,))
    p = torch.tensor([7, 9], device="cuda")
    for inter in (False, True):
        got, _ = fq.qk_norm_rope(q, q, f, p, interleaved=inter)
        # (a NaN's payload is not a value: conversions to bf16 give one NaN)
        assert torch.equal(torch.isnan(got), torch.isnan(q)) and torch.isfinite(got[..., :32]).all()
        assert same(got[..., 32:].nan_to_num(7.0), q[..., 32:].nan_to_num(7.0))


@gpu
def test_rotary_axes_is_the_table_of_qkv_epilogue():
    """The rotation over three axes is the one that qkv_epilogue takes as a stored table: norm and
    rotation agree to a rounding of the normed value (2^-8 of each of the pair) and their own."""
    t, h = 50, 24
    f, axis = fq.rotary_axes((16, 56, 56))
    pos = torch.randint(-30, 60, (3, t), generator=gen(1), device="cuda")
    x = normal((t, 3 * h * 128), 2)
    q, k, v = (x[:, i * h * 128:(i + 1) * h * 128] for i in range(3))
    wq, wk = ((1 + 0.2 * normal((128,), s).float()).to(BF16) for s in (3, 4))
    angle = (pos[axis.long()].double() * f[:, None]).t()
    table = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    st = dict(q=q, k=k, v=v, q_weight=wq, k_weight=wk, cos_sin=table, eps=1e-6)
    empty = dict(st, q=q[:0], k=k[:0], v=v[:0])
    jq, jk, _ = fq.qkv_epilogue(empty, st, h)
    got = fq.qk_norm_rope(q.view(t, h, 128), k.view(t, h, 128), f, pos, axis=axis, q_weight=wq,
                          k_weight=wk, interleaved=True)
    for g, j, s, w in zip(got, (jq, jk), (q, k), (wq, wk)):
        y, size = plain_heads(s.view(t, h, 128), w, f, pos, axis, True)
        assert bool(((g.double() - j.double()).abs() <= 2 * 2.0 ** -8 * y.abs() + 2.0 ** -8 * size + CHAIN * size).all())


# ------------------------------------------------------------------------------------------
# cache_write, cache_read
# ------------------------------------------------------------------------------------------

def clone(cache):
    return fq.PagedCache(*(None if t is None else t.clone() for t in cache))


def garbage(pages, page, heads, dim, dtype, joint=False):
    """A cache full of bytes that no test should meet: NaN everywhere (int8: -128). joint: k and v the
    halves of one array."""
    shape = (pages, 2, heads, page, dim)
    raw = torch.full(shape, 0x80 if dtype == INT8 else 0x7F if dtype == E4M3 else 0, dtype=torch.uint8, device="cuda").view(dtype) \
        if dtype != BF16 else torch.full(shape, float("nan"), dtype=BF16, device="cuda")
    sc = None if dtype == BF16 else torch.full(shape[:4], float("nan"), device="cuda")
    k, v = raw[:, 0], raw[:, 1]
    if not joint:
        k, v = k.contiguous(), v.contiguous()
    if sc is None:
        return fq.PagedCache(k, v)
    return fq.PagedCache(k, v, sc[:, 0] if joint else sc[:, 0].contiguous(), sc[:, 1] if joint else sc[:, 1].contiguous())


def rows_of(cache, slots):
    """(k, v, k_scale, v_scale) of the slots' rows: [tokens, heads, ...]."""
    page = cache.k.shape[2]
    return [None if t is None else
            (t.view(torch.uint8) if t.dtype == E4M3 else t)[slots // page, :, slots % page].view(t.dtype)
            for t in cache]


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("how,norm", [(None, False), (("halves", 1), True), (("pairs", 1), False), (("halves", 0.25), True)], ids=str)
@pytest.mark.parametrize("tokens,heads,kv,page", [(1, 8, 2, 16), (77, 6, 3, 48), (600, 16, 1, 128)])
def test_cache_write(dtype, dim, how, norm, tokens, heads, kv, page):
    x = normal((tokens, (heads + 2 * kv) * dim), 1, 2.0)
    q, k, v = (x[:, a * dim:b * dim].view(tokens, b - a, dim) for a, b in
               ((0, heads), (heads, heads + kv), (heads + kv, heads + 2 * kv)))
    pages = tokens // page + 3
    cache = garbage(pages, page, kv, dim, dtype, joint=tokens == 77)
    before = clone(cache)
    slots = torch.randperm(pages * page, generator=gen(5), device="cuda")[:tokens]
    stored = torch.ones(tokens, dtype=torch.bool, device="cuda")
    if tokens > 1:
        slots[3], stored[3] = -1, False  # a padded token
    r = rotary(dim, how, tokens, 1, 6)
    w = (1 + 0.2 * normal((dim,), 7).float()).to(BF16) if norm else None
    got = fq.cache_write(k, v, cache, slots, q=q, q_weight=w, k_weight=w, **r)
    near_bf16(got, *plain_heads(q, w, **r))
    ks, vs = plain_heads(k, w, **r), plain_heads(v, None)
    at = slots[stored]
    gk, gv, sk, sv = rows_of(cache, at)
    if dtype == BF16:
        near_bf16(gk, ks[0][stored], ks[1][stored])
        assert same(gv, v[stored])
    else:
        near_codes(gk, sk, ks[0][stored], ks[1][stored])
        code, scale = exact_codes(v[stored], dtype)
        assert same(gv, code) and same(sv, scale)
        if how is None and not norm:
            code, scale = exact_codes(k[stored], dtype)
            assert same(gk, code) and same(sk, scale)
    # nothing else has changed
    for t, b in zip(cache, before):
        if t is not None:
            t, b = (u.view(torch.uint8) if u.dtype == E4M3 else u.view(torch.int16 if u.dtype == BF16 else torch.int32 if u.dtype == torch.float32 else INT8) for u in (t, b))
            t, b = t.clone(), b.clone()
            for u in (t, b):
                u[at // page, :, at % page] = 0
            assert torch.equal(t, b)
    # k and v alone give the same rows
    again = clone(before) if tokens != 77 else fq.PagedCache(*(None if t is None else t.clone(memory_format=torch.contiguous_format) for t in before))
    assert fq.cache_write(k, v, again, slots, k_weight=w, **r) is None
    for a, b in zip(rows_of(cache, at), rows_of(again, at)):
        assert a is None or same(a, b)
    assert fq.device_error() == 0


@gpu
@pytest.mark.parametrize("dtype", [INT8, E4M3], ids=ids)
def test_cache_write_special_rows(dtype):
    """Rows of zeros, of tiny values, with a NaN or an infinity, and halves of a step."""
    k = normal((8, 2, 64), 1)
    k[0] = 0
    k[1, 0, 5] = float("nan")
    k[2, 1, 63] = float("-inf")
    k[3] = 2.0 ** -110
    k[4] = 2.0 ** -90
    k[5] = (torch.arange(64, device="cuda") - 31.5).to(BF16)
    k[5, :, 0] = 127.0
    k[6] = -0.0
    cache = fq.paged_cache(1, 16, 2, 64, dtype=dtype)
    slots = torch.arange(8, device="cuda")
    fq.cache_write(k, k, cache, slots)
    code, scale = exact_codes(k, dtype)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c, s = c[0, :, :8].transpose(0, 1), s[0, :, :8].t()
        assert torch.equal(c.float(), code.float())
        assert torch.equal(torch.isnan(s), torch.isnan(scale)) and torch.equal(s.nan_to_num(7.0), scale.nan_to_num(7.0))
    assert torch.isnan(scale[1, 0]) and torch.isnan(scale[2, 1]) and not torch.isnan(scale[1, 1])


@gpu
def test_slots_past_the_cache_are_left_out():
    cache = fq.paged_cache(2, 16, 1, 64)
    k = normal((4, 1, 64), 1)
    fq.cache_write(k, k, cache, torch.tensor([0, 32, 1 << 50, -5], device="cuda"))
    assert fq.device_error() == 2 and fq.device_error() == 0
    assert bool(cache.k[0, 0, 0].any()) and not cache.k.view(-1)[64:].any()


def scattered(batch, width, pages, seed):
    """A page table of distinct pages in a random order."""
    assert batch * width <= pages
    return torch.randperm(pages, generator=gen(seed), device="cuda")[:batch * width].view(batch, width).int()


def filled(cache, table, lengths, seed, scale=1.0):
    """Fills the sequences' rows through cache_write: (k, v) [sum of lengths, heads, dim] as stored, in
    64 bits, and the offsets."""
    pages, heads, page, dim = cache.k.shape
    at = [torch.arange(n, device="cuda") for n in lengths]
    slots = torch.cat([table[b].long()[t // page] * page + t % page for b, t in enumerate(at)])
    n = len(slots)
    k, v = normal((n, heads, dim), seed, scale), normal((n, heads, dim), seed + 1)
    k *= 0.25 + torch.rand(n, heads, 1, generator=gen(seed + 2), device="cuda").to(BF16)
    v *= 10.0 ** torch.randint(-2, 2, (n, heads, 1), generator=gen(seed + 3), device="cuda").to(BF16)
    if n:
        fq.cache_write(k, v, cache, slots)
    gk, gv, sk, sv = rows_of(cache, slots)
    k64, v64 = gk.double(), gv.double()
    if sk is not None:
        k64, v64 = k64 * sk.double()[..., None], v64 * sv.double()[..., None]
    offsets = torch.tensor([0] + list(lengths), device="cuda").cumsum(0)
    return k64, v64, offsets


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim,heads,page", [(64, 1, 16), (128, 8, 48), (256, 3, 1024), (128, 5, 64)])
@pytest.mark.parametrize("lengths", [[1], [0, 0], [3, 0, 100, 1, 64, 0], [1000, 17]], ids=str)
def test_cache_read(dtype, dim, heads, page, lengths):
    from tests.gpu_util import Guarded
    width = -(-max(lengths + [1]) // page)
    cache = garbage(len(lengths) * width + 2, page, heads, dim, dtype)
    table = scattered(len(lengths), width, len(cache.k), 1)
    k64, v64, offsets = filled(cache, table, lengths, 2)
    n, more = sum(lengths), 9
    gk, gv = (Guarded((n + more, heads, dim), BF16) for _ in range(2))
    gk.tensor.fill_(7.0), gv.tensor.fill_(7.0)
    wide = torch.full((len(lengths), width + 3), -7, dtype=torch.int32, device="cuda")
    wide[:, :width] = table
    got = fq.cache_read(cache, wide[:, :width], offsets, n + more, k=gk.tensor, v=gv.tensor)
    for g, w, r in zip(got, (gk, gv), (k64, v64)):
        assert g is w.tensor and w.intact()
        # the code's product with its scale is rounded to fp32, then to bf16
        assert same(g[:n], r.float().to(BF16)) and bool((g[n:] == 7).all())
    got = fq.cache_read(cache, table, offsets, n)
    assert same(got[0], gk.tensor[:n]) and same(got[1], gv.tensor[:n])
    if n > 1:  # offsets that begin later, and past the rows
        gk.tensor.fill_(7.0)
        fq.cache_read(cache, table, offsets + 2, n + 1, k=gk.tensor[:n + 1], v=gv.tensor[:n + 1])
        assert bool((gk.tensor[:2] == 7).all()) and same(gk.tensor[2:n + 1], got[0][:n - 1])
    assert fq.device_error() == 0


@gpu
def test_bad_pages_are_left_out():
    """A page outside the cache: its tokens read as zeros and count for nothing in attention."""
    heads, dim, page = 2, 128, 16
    for dtype in TYPES:
        cache = fq.paged_cache(8, page, heads, dim, dtype=dtype)
        table = scattered(1, 8, 8, 3)
        k64, v64, offsets = filled(cache, table, [128], 4)
        for bad in (-1, 8, -2 ** 31, 2 ** 31 - 1):
            broken = table.clone()
            broken[0, 3] = bad
            k, v = fq.cache_read(cache, broken, offsets, 128)
            assert fq.device_error() == 2
            assert not k[48:64].any() and same(k[64:], k64[64:].float().to(BF16)) and not v[48:64].any()
            q = normal((1, 4, dim), 5)
            o = fq.paged_attention(q, cache, broken, torch.tensor([128], dtype=torch.int32, device="cuda"))
            assert fq.device_error() == 2
            keep = torch.cat([torch.arange(48), torch.arange(64, 128)]).cuda()
            check_attention(o[0], None, q[0], k64[keep], v64[keep], dim ** -0.5, dtype)
        short = fq.cache_read(cache, table[:, :2], offsets, 128)[0]  # past the table's width
        assert fq.device_error() == 2 and not short[32:].any()


# ------------------------------------------------------------------------------------------
# paged_attention
# ------------------------------------------------------------------------------------------

def check_attention(o, lse, q, k, v, scale, dtype):
    """One sequence: q [heads, dim], k, v [n, kv heads, dim] in 64 bits.

    A logit is a sum of exact products in fp32: dim / 16 matrix steps, in each 17 terms whose alignment
    and rounding cost at most 2^-21 of the sum of their magnitudes (m), and four roundings of the
    logit. It enters a weight by a difference with the maximum (rounded at the size of either) and the
    exponential (2^-22). A weight is rounded to fp16 (2^-11) or two bf16 (2^-16); products with v as above,
    a tile of 16 tokens a step, of n / 16 at most; the maximum's and sum's rescaling 2^-20 more.
    fp16 weights (p times the value's scale) lie on a grid of 2^-24 where the largest is 2^8 at least:
    each is off by up to 2^-33 of the largest, and codes are at most QMAX, so a row's largest value
    times its p bounds what a weight's unit moves."""
    heads, dim = q.shape
    if len(k) == 0:
        assert not o.any() and (lse is None or bool((lse == -math.inf).all()))
        return
    qs = q.double().view(k.shape[1], -1, dim)
    s = torch.einsum("hgd,thd->hgt", qs, k) * scale
    m = torch.einsum("hgd,thd->hgt", qs.abs(), k.abs()) * abs(scale)
    e = (dim / 16 * 2.0 ** -21 * m + 2.0 ** -21 * (s.abs() + s.abs().amax(-1, keepdim=True) + 1)).amax(-1, keepdim=True)
    p = torch.softmax(s, -1)
    want = torch.einsum("hgt,thd->hgd", p, v).reshape(heads, dim)
    size = torch.einsum("hgt,thd->hgd", p, v.abs()).reshape(heads, dim)
    rel = 2 * e + (2.0 ** -16 if dtype == BF16 else 2.0 ** -11) + len(k) / 16 * 2.0 ** -21 + 2.0 ** -20
    tol = 2.0 ** -8 * want.abs() + 1.01 * (rel.reshape(heads, 1) * size)
    if dtype != BF16:
        largest = (p * v.abs().amax(-1).t()[:, None]).amax(-1).reshape(heads, 1)
        tol = tol + len(k) * 2.0 ** -33 * largest
    err = (o.double() - want).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), float(err.max()))
    if lse is not None:
        ref = torch.logsumexp(s, -1).reshape(heads)
        bound = e.reshape(heads) + len(k) / 16 * 2.0 ** -21 + 2.0 ** -22 * (ref.abs() + 1)
        assert bool(((lse.double() - ref).abs() <= bound).all()), float((lse.double() - ref).abs().max())


def attention_case(dtype, dim, heads, kv, page, lengths, window=0, seed=1, joint=False, scale=None, q_scale=1.5):
    width = -(-max(max(lengths), 1) // page)
    cache = garbage(len(lengths) * width + 1, page, kv, dim, dtype, joint)
    table = scattered(len(lengths), width, len(cache.k), seed)
    k, v, offsets = filled(cache, table, lengths, seed + 1)
    # entries of pages outside the range are not read
    t = torch.arange(width, device="cuda")
    n = torch.tensor(lengths, device="cuda")[:, None]
    first = (n - window).clamp_min(0) if window else torch.zeros_like(n)
    table = torch.where((t * page < n) & ((t + 1) * page > first), table, -1)
    packed = normal((len(lengths), heads + 3, dim), seed + 9, q_scale)
    q = packed[:, :heads]
    lens = n[:, 0].int()
    o, lse = fq.paged_attention(q, cache, table, lens, window=window, scale=scale, return_lse=True)
    assert o.shape == q.shape and lse.shape == q.shape[:2]
    for b, (x, y) in enumerate(zip(offsets[:-1].tolist(), offsets[1:].tolist())):
        x = max(x, y - window) if window else x
        check_attention(o[b], lse[b], q[b], k[x:y], v[x:y], dim ** -0.5 if scale is None else scale, dtype)
    assert fq.device_error() == 0
    return q, cache, table, lens, o, lse


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim,heads,kv", [(64, 8, 2), (128, 8, 8), (128, 32, 4), (256, 10, 5), (64, 1, 1), (128, 20, 1), (64, 48, 4),
                                          (256, 12, 1), (128, 40, 2)])
@pytest.mark.parametrize("page,lengths", [(16, [1]), (48, [0, 5, 16, 17, 300, 48, 0]), (64, [2000, 31])], ids=str)
def test_paged_attention(dtype, dim, heads, kv, page, lengths):
    attention_case(dtype, dim, heads, kv, page, lengths)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("lengths", [[1] * 200, [0] * 7, [20] * 700 + [3000], [40000], [40000, 1, 0, 9000], list(range(0, 600, 7)),
                                     [15, 16, 17, 127, 128, 129, 143, 144, 145] * 4, [0] * 40 + [700] + [0] * 40 + [5000, 0]],
                         ids=["ones", "none", "one-long", "long", "longs", "ragged", "edges", "gaps"])
@pytest.mark.parametrize("heads,kv", [(8, 2), (3, 3), (12, 1)])
def test_paged_attention_splits(dtype, lengths, heads, kv):
    attention_case(dtype, 128 if kv > 1 else 64, heads, kv, 32, lengths)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("batch,high,heads,kv", [(40, 20000, 8, 4), (90, 6000, 8, 8), (19, 20000, 80, 8)],
                         ids=["some", "many", "wide"])
def test_paged_attention_much_work(dtype, batch, high, heads, kv):
    """Enough tiles for a second round of CTAs with smaller shares: fewer and more segments than CTAs,
    lengths of zero among them, the longest first and last, and twice the same bits."""
    lengths = [round(high * (i * 7 % batch) / (batch - 1)) for i in range(batch)]
    lengths[1], lengths[batch // 2], lengths[-1] = 0, 0, high
    q, cache, table, lens, o, lse = attention_case(dtype, 64, heads, kv, 64, lengths)
    again = fq.paged_attention(q, cache, table, lens, return_lse=True)
    assert same(again[0], o) and same(again[1], lse)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim,batch,high,heads,kv", [(64, 100, 4000, 8, 8), (128, 100, 4000, 8, 8), (256, 50, 8000, 8, 4),
                                                     (128, 100, 1000, 96, 8), (64, 100, 1000, 30, 3), (64, 400, 300, 2, 2)], ids=str)
def test_paged_attention_many_segments(dtype, dim, batch, high, heads, kv):
    """Many segments over several CTAs each: both forms of the join, with small last shares and without."""
    attention_case(dtype, dim, heads, kv, 64, [high * i // (batch - 1) for i in range(batch)])


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("window", [1, 15, 16, 100, 1000, 10 ** 6])
def test_paged_attention_window(dtype, window):
    attention_case(dtype, 128, 8, 2, 16, [1, 15, 16, 17, 101, 0, 1500, 20000], window=window, joint=True)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("scale,q_scale", [(1.0, 1.0), (0.01, 30.0), (-0.1, 1.0), (0.0, 1.0), (3.0, 1e-3), (1e-6, 1e6), (1e9, 1e-9)])
def test_paged_attention_scales(dtype, scale, q_scale):
    """Sharp and flat softmaxes, queries far from one."""
    attention_case(dtype, 128, 16, 2, 16, [700, 9, 3000], scale=scale, q_scale=q_scale)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("page", [16, 80, 176, 512, 1024])
def test_paged_attention_page_sizes(dtype, page):
    """Pages of 1, 5, 11, 32 and 64 tiles, more of them in a sequence than a warp looks up at once."""
    attention_case(dtype, 64, 4, 2, page, [40 * page, 33 * page + 1, 32 * page, page - 1, 5], joint=page == 80)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim", [64, 256])
def test_no_pages_no_sequences(dtype, dim):
    """Caches without a page, tables without a column, batches without a sequence."""
    empty, some = fq.paged_cache(0, 16, 2, dim, dtype=dtype), fq.paged_cache(3, 16, 2, dim, dtype=dtype)
    q = normal((5, 4, dim), 1)
    lens = torch.tensor([0, 7, -3, 10 ** 9, 1], dtype=torch.int32, device="cuda")
    none = torch.zeros(5, 0, dtype=torch.int32, device="cuda")
    for cache, table in ((empty, none), (some, none), (empty, torch.zeros(5, 40, dtype=torch.int32, device="cuda"))):
        o, lse = fq.paged_attention(q, cache, table, lens, return_lse=True)
        assert not o.any() and bool((lse == -math.inf).all())
    assert fq.paged_attention(q[:0], some, none[:0], lens[:0]).shape == (0, 4, dim)
    k, v = fq.cache_read(empty, none, torch.zeros(6, dtype=torch.int64, device="cuda"), 0)
    assert k.shape == (0, 2, dim)
    assert fq.cache_write(q[:0, :2], q[:0, :2], some, torch.zeros(0, dtype=torch.int64, device="cuda"), q=q[:0]).shape == (0, 4, dim)
    assert not some.k.view(torch.uint8).any()
    # lengths beyond the table count as its pages' tokens
    k64, v64, _ = filled(some, torch.tensor([[0, 2, 1]], dtype=torch.int32, device="cuda"), [48], 2)
    o = fq.paged_attention(q[:1], some, torch.tensor([[0, 2, 1]], dtype=torch.int32, device="cuda"), lens[3:4])
    check_attention(o[0], None, q[0], k64, v64, dim ** -0.5, dtype)
    assert fq.device_error() == 0


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("power", [-130, -100, 120])
def test_paged_attention_far_queries(dtype, power):
    """Queries near the ends of bf16's range, with a scale that brings the logits back (in fp32)."""
    q_scale = 2.0 ** power
    q = (normal((1, 8, 128), 1).float() * q_scale).to(BF16)
    cache = fq.paged_cache(8, 16, 2, 128, dtype=dtype)
    table = scattered(1, 8, 8, 1)
    k64, v64, _ = filled(cache, table, [100], 2)
    scale = 2.0 ** min(-power, 120) * 0.1
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    o, lse = fq.paged_attention(q, cache, table, lens, scale=scale, return_lse=True)
    check_attention(o[0], lse[0], q[0], k64, v64, scale, dtype)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_paged_attention_heads_of_unlike_size(dtype):
    """Query heads of one block that differ by 2^30, rising logits (the maximum is raised again and
    again), and values whose scales rise and fall by 2^40."""
    n, page = 1500, 16
    cache = fq.paged_cache(n // page + 1, page, 1, 64, dtype=dtype)
    t = torch.arange(n, device="cuda")
    k = normal((n, 1, 64), 1) * (0.2 + t[:, None, None] / 100).to(BF16)
    v = normal((n, 1, 64), 2) * (2.0 ** (20 * torch.sin(t / 50.0))).to(BF16)[:, None, None]
    fq.cache_write(k, v, cache, t)
    gk, gv, sk, sv = rows_of(cache, t)
    k64, v64 = gk.double(), gv.double()
    if sk is not None:
        k64, v64 = k64 * sk.double()[..., None], v64 * sv.double()[..., None]
    q = normal((1, 8, 64), 3)
    q[0, ::2] *= 2.0 ** -30
    table = torch.arange(len(cache.k), device="cuda").int()[None]
    for order in (1, -1):  # rising and falling
        if order < 0:
            fq.cache_write(k, v, cache, n - 1 - t)
        o, lse = fq.paged_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), return_lse=True)
        check_attention(o[0], lse[0], q[0], k64, v64, 0.125, dtype)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_paged_attention_special_values(dtype):
    """A NaN in a key or value of one sequence reaches that sequence's head and no other; infinite
    logits behave as in a softmax."""
    lengths = [50, 50, 900, 900]
    q, cache, table, lens, o, _ = attention_case(dtype, 128, 4, 2, 16, lengths)
    for b, what in ((0, "k"), (2, "v")):
        k = normal((1, 2, 128), 1)
        k[0, 1, 3] = float("nan")
        t = 20
        slot = table[b, t // 16].long() * 16 + t % 16
        fine = normal((1, 2, 128), 2)
        fq.cache_write(k if what == "k" else fine, k if what == "v" else fine, cache, slot[None])
    got = fq.paged_attention(q, cache, table, lens)
    nan = torch.isnan(got).any(-1)
    whole = torch.isnan(got).all(-1)  # (a bf16 value's NaN stays in its column, a scale's is the row's)
    assert torch.equal(nan[:2], whole[:2]) and (dtype == BF16 or torch.equal(nan, whole))
    if dtype == BF16:
        assert torch.isnan(got[2]).sum(-1).tolist() == [0, 0, 1, 1] and torch.isnan(got[2, 2:, 3]).all()
    assert nan.tolist() == [[False, False, True, True], [False] * 4, [False, False, True, True], [False] * 4]
    assert same(got[1], o[1]) and same(got[3], o[3])


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_paged_attention_repeats_captured_and_on_other_streams(dtype):
    """The same bits again, on other streams at once, and from a graph whose lengths, tables and
    queries change between replays."""
    lengths = [3000, 0, 17, 800, 5000]
    q, cache, table, lens, o, lse = attention_case(dtype, 128, 16, 4, 64, lengths)
    table = table.clamp_min(0)
    want = [fq.paged_attention(q, cache, table, lens, return_lse=True) for _ in range(3)]
    assert all(same(x, o) and same(y, lse) for x, y in want)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [fq.paged_attention(q, cache, table, lens, stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    assert all(same(x, o) for x in got)
    qs, ts, ls = q.clone(), table.clone(), lens.clone()
    outs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=s):
        outs.append(fq.paged_attention(qs, cache, ts, ls))
    with torch.cuda.graph(g2, stream=s):
        outs.append(fq.paged_attention(qs, cache, ts, ls))
    for n in ([1, 2, 3, 4, 5], [0] * 5, lengths, [5000, 0, 0, 0, 1], lengths):
        ls.copy_(torch.tensor(n, dtype=torch.int32))
        ls.copy_(torch.minimum(ls, lens))
        want = fq.paged_attention(qs, cache, ts, ls)
        g1.replay(), g2.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want) and same(outs[1], want)
    assert same(outs[0], o)


@gpu
def test_threads_at_once():
    """Several Python threads, each on a stream of its own, writing to caches of their own and attending:
    the results of one after the other."""
    import threading

    def one(i):
        dtype = TYPES[i % 3]
        lengths = [100 + 900 * i, 17, 0, 2000]
        cache = fq.paged_cache(300, 16, 2, 128, dtype=dtype)
        pages = torch.arange(300, device="cuda").int()
        table = pages[:280].view(4, 70) if i < 2 else pages[:290].view(2, 145)
        lengths = lengths[-len(table):]
        lengths = [min(n, table.shape[1] * 16) for n in lengths]
        filled(cache, table, lengths, i)
        q = normal((len(lengths), 16, 128), 50 + i)
        lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        return [fq.paged_attention(q, cache, table, lens) for _ in range(10)]

    want = [one(i) for i in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got[i] = one(i)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert all(same(x, a[0]) for x in a + b)
    assert fq.device_error() == 0


@gpu
def test_captured_writes():
    """cache_write and cache_read in a graph: new inputs, slots and positions at each replay."""
    d, h, kv, t = 128, 4, 2, 33
    cache = fq.paged_cache(8, 16, kv, d)
    f, _ = fq.rotary_axes((d,))
    q, k, v = normal((t, h, d), 1), normal((t, kv, d), 2), normal((t, kv, d), 3)
    slots, pos = torch.arange(t, device="cuda"), torch.arange(t, device="cuda")
    table = torch.arange(8, device="cuda").int()[None]
    off = torch.tensor([0, 128], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qo = fq.cache_write(k, v, cache, slots, q=q, inv_freq=f, positions=pos)
        ko, vo = fq.cache_read(cache, table, off, 128)
    for i in range(3):
        k.copy_(normal((t, kv, d), 10 + i)), q.copy_(normal((t, h, d), 20 + i))
        slots.copy_(torch.randperm(128, generator=gen(i), device="cuda")[:t]), pos.add_(1000 * i)
        g.replay()
        again = fq.PagedCache(*(x.clone() for x in cache))
        want = fq.cache_write(k, v, again, slots, q=q, inv_freq=f, positions=pos)
        assert same(want, qo) and same(again.k, cache.k) and same(again.k_scale, cache.k_scale)
        for x, y in zip(fq.cache_read(again, table, off, 128), (ko, vo)):
            assert same(x, y)


@gpu
def test_offsets_beyond_32_bits():
    """A cache of 9 GB of keys: bytes, values and scales past 2^32."""
    for dtype, pages in ((INT8, 1 << 16), (BF16, 1 << 15)):
        page, heads, dim = 64, 8, 256
        k = torch.empty(pages, heads, page, dim, dtype=dtype, device="cuda")
        cache = fq.PagedCache(k, torch.empty_like(k), *((None, None) if dtype == BF16 else
                              (torch.empty(pages, heads, page, device="cuda") for _ in range(2))))
        table = torch.arange(pages - 5, pages, device="cuda").int().flip(0)[None].contiguous()
        k64, v64, offsets = filled(cache, table, [300], 1)
        q = normal((1, 16, dim), 2)
        o = fq.paged_attention(q, cache, table, torch.tensor([300], dtype=torch.int32, device="cuda"))
        check_attention(o[0], None, q[0], k64, v64, dim ** -0.5, dtype)
        assert same(fq.cache_read(cache, table, offsets, 300)[0], k64.float().to(BF16))
        del k, cache


@gpu
def test_a_decoding_run():
    """Prompt, then token by token: packed int8 projection, cache_write with norm and rotation,
    paged_attention, norm to 8-bit rows, int8 output projection. Each step's attention is the dense
    one over what cache_read gives back, and a captured step gives the same bits."""
    hidden, heads, kv, dim, page, steps = 512, 8, 2, 64, 16, 21
    lens0 = [5, 40, 1]
    width = 5
    cache = fq.paged_cache(16, page, kv, dim)
    table = scattered(3, width, 16, 1)
    f, _ = fq.rotary_axes((dim,))
    wn, wq, wk, wo = ((1 + 0.1 * normal((n,), s).float()).to(BF16) for n, s in ((hidden, 2), (dim, 3), (dim, 4), (heads * dim, 5)))

    def weights(n, k, seed):
        w = torch.randint(-127, 128, (n, k), generator=gen(seed), device="cuda", dtype=INT8)
        return w, torch.rand(n, generator=gen(seed + 1), device="cuda") * 1e-3

    w_qkv, s_qkv = weights((heads + 2 * kv) * dim, hidden, 6)
    w_out, s_out = weights(hidden, heads * dim, 8)

    def project(x, slots, positions):
        q8, s = fq.rms_norm_quant(x, wn)
        qkv = fq.int8_matmul(q8, s, w_qkv, s_qkv)
        q, k, v = (qkv[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, heads), (heads, heads + kv), (heads + kv, heads + 2 * kv)))
        return fq.cache_write(k, v, cache, slots, q=q, inv_freq=f, positions=positions, q_weight=wq, k_weight=wk)

    def step(x, slots, lens):
        q = project(x, slots, lens - 1)
        o = fq.paged_attention(q, cache, table, lens)
        q8, s = fq.rms_norm_quant(o.flatten(1), wo)
        return q, o, fq.int8_matmul(q8, s, w_out, s_out)

    at = [(b, t) for b, n in enumerate(lens0) for t in range(n)]
    place = lambda b, t: int(table[b, t // page]) * page + t % page  # noqa: E731
    project(normal((len(at), hidden), 9), torch.tensor([place(*p) for p in at], device="cuda"), torch.tensor([t for _, t in at], device="cuda"))
    x = normal((3, hidden), 10)
    lens = torch.tensor(lens0, dtype=torch.int32, device="cuda")
    xs, ss, ls = x.clone(), torch.zeros(3, dtype=torch.int64, device="cuda"), lens.clone()
    graph = None
    for i in range(steps):
        lens = lens + 1
        slots = torch.tensor([place(b, int(n) - 1) for b, n in enumerate(lens)], device="cuda")
        q, o, y = step(x, slots, lens)
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)])
        rows = int(offsets[-1])
        k, v = fq.cache_read(cache, table, offsets, rows)
        for b in range(3):
            a, z = int(offsets[b]), int(offsets[b + 1])
            # what is read back is rounded to bf16 (2^-8), what attention reads is not
            kk, vv = k[a:z].double(), v[a:z].double()
            s = torch.einsum("hgd,thd->hgt", q[b].double().view(kv, -1, dim), kk) * dim ** -0.5
            m = torch.einsum("hgd,thd->hgt", q[b].double().abs().view(kv, -1, dim), kk.abs()) * dim ** -0.5
            p = torch.softmax(s, -1)
            want = torch.einsum("hgt,thd->hgd", p, vv).reshape(heads, dim)
            size = torch.einsum("hgt,thd->hgd", p, vv.abs()).reshape(heads, dim)
            rel = (2 * 2.0 ** -8 * m.amax(-1) + 2.0 ** -8 + 2.0 ** -10).exp().sub(1).reshape(heads, 1)
            assert bool(((o[b].double() - want).abs() <= 2.0 ** -8 * want.abs() + rel * size).all())
        assert bool(torch.isfinite(y).all())
        xs.copy_(x), ss.copy_(slots), ls.copy_(lens)
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                captured = step(xs, ss, ls)
        graph.replay()
        assert all(same(a, b) for a, b in zip(captured, (q, o, y)))
        x = (x.float() + y.float()).to(BF16)
    assert fq.device_error() == 0


# ------------------------------------------------------------------------------------------
# refusals (no GPU)
# ------------------------------------------------------------------------------------------

def c_cache(**kw):
    c = dict(k=A, v=2 * A, k_scale=3 * A, v_scale=4 * A, k_stride=8 * 64 * 128, v_stride=8 * 64 * 128,
             k_scale_stride=8 * 64, v_scale_stride=8 * 64, pages=100, page_size=64, heads=8, head_dim=128, type=0)
    c.update(kw)
    return _capi.PagedCacheView(*(c[n] for n, _ in _capi.PagedCacheView._fields_))


def c_rotary(**kw):
    r = dict(inv_freq=20 * A, axis=21 * A, positions=22 * A, position_stride=1000, position_bytes=8, axes=3, pairs=64, interleaved=0)
    r.update(kw)
    return _capi.Rotary(*(r[n] for n, _ in _capi.Rotary._fields_))


BAD_CACHES = [(dict(type=3), VALUE), (dict(type=-1), VALUE), (dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE),
              (dict(page_size=24), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=2048), SHAPE), (dict(heads=0), SHAPE),
              (dict(heads=4097), SHAPE), (dict(pages=-1), SHAPE), (dict(k_stride=8 * 64 * 128 - 16), SHAPE),
              (dict(v_stride=8 * 64 * 128 + 8), SHAPE), (dict(k_scale_stride=511), SHAPE), (dict(k=None), NULL),
              (dict(v_scale=None), NULL), (dict(v=2 * A + 8), ALIGN), (dict(k_scale=3 * A + 2), ALIGN)]


@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=str)
def test_caches_refused(L, bad, status):
    if bad.get("heads") == 0:
        pass
    c = c_cache(**bad)
    w = L.fp8q_cache_write(c, 10 * A, None, 0, None, 0, 11 * A, 1024, 12 * A, 1024, None, None, 1e-6, None, 4, 0, None)
    r = L.fp8q_cache_read(13 * A, 14 * A, c, 15 * A, 10, 10, 16 * A, 2, 5, None)
    q_heads = 32 if bad.get("heads", 8) == 8 else 4097
    a = L.fp8q_paged_attention(13 * A, None, 17 * A, 1 << 20, c, 15 * A, 10, 10, 16 * A, 2, q_heads, 1.0, 0, 18 * A, 1 << 30, None)
    for got in (r, a):
        assert got == status or (bad.get("heads") == 0 and got == SHAPE)
    assert w == status or ("head_dim" in bad and w == SHAPE)


def test_qk_norm_rope_refusals(L):
    def call(qo=A, qo_ld=4096, ko=2 * A, ko_ld=1024, q=3 * A, q_ld=6144, k=3 * A + 8192, k_ld=6144, wq=5 * A, wk=6 * A, eps=1e-6,
             rot=None, tokens=1000, h=32, kv=8, d=128):
        return L.fp8q_qk_norm_rope(qo, qo_ld, ko, ko_ld, q, q_ld, k, k_ld, wq, wk, eps, rot, tokens, h, kv, d, None)

    for bad in (dict(tokens=-1), dict(h=0), dict(kv=0), dict(h=5000), dict(d=96), dict(d=0), dict(q_ld=4088), dict(k_ld=1000),
                dict(q_ld=6148), dict(qo_ld=4000), dict(ko_ld=1028), dict(rot=c_rotary(pairs=0)), dict(rot=c_rotary(pairs=65)),
                dict(rot=c_rotary(pairs=20)), dict(rot=c_rotary(axes=0)), dict(rot=c_rotary(position_stride=999))):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rot=c_rotary(position_bytes=2))):
        assert call(**bad) == VALUE, bad
    for bad in (dict(qo=None), dict(ko=None), dict(q=None), dict(k=None), dict(rot=c_rotary(inv_freq=None)), dict(rot=c_rotary(positions=None))):
        assert call(**bad) == NULL, bad
    for bad in (dict(qo=A + 8), dict(q=3 * A + 2), dict(wq=5 * A + 4), dict(rot=c_rotary(inv_freq=20 * A + 4)),
                dict(rot=c_rotary(positions=22 * A + 4)), dict(rot=c_rotary(axis=21 * A + 2))):
        assert call(**bad) == ALIGN, bad
    for bad in (dict(ko=A), dict(ko=A + 4096 * 2000 - 16), dict(qo=3 * A, qo_ld=4096), dict(qo=3 * A + 16, qo_ld=6144),
                dict(qo=3 * A + 8192 - 16, qo_ld=6144), dict(ko=3 * A + 2 * 4096 - 16, ko_ld=6144), dict(ko=5 * A), dict(ko=20 * A, rot=c_rotary()),
                dict(qo=22 * A + 64, rot=c_rotary()), dict(qo=21 * A, rot=c_rotary())):
        assert call(**bad) == ALIAS, bad
    assert call(tokens=0, qo=None, q=None) == OK
    # in place, in the columns of a packed product: not refused for that (no device here)
    here = call(qo=3 * A, qo_ld=6144, ko=3 * A + 8192, ko_ld=6144)
    assert here in (OK, UNSUPPORTED, CUDA)


def test_cache_write_refusals(L):
    def call(c=None, slots=10 * A, qo=11 * A, qo_ld=4096, q=12 * A, q_ld=6144, k=12 * A + 8192, k_ld=6144, v=12 * A + 10240, v_ld=6144,
             wq=None, wk=None, eps=1e-6, rot=None, tokens=1000, h=32):
        return L.fp8q_cache_write(c_cache() if c is None else c, slots, qo, qo_ld, q, q_ld, k, k_ld, v, v_ld, wq, wk, eps, rot, tokens, h, None)

    assert L.fp8q_cache_write(None, 10 * A, None, 0, None, 0, A, 1024, A, 1024, None, None, 1e-6, None, 1, 0, None) == NULL
    for bad in (dict(tokens=-1), dict(h=-1), dict(h=4097), dict(k_ld=1016), dict(v_ld=1020), dict(q_ld=4000), dict(rot=c_rotary(pairs=65))):
        assert call(**bad) == SHAPE, bad
    assert call(wk=30 * A, eps=0.0) == VALUE
    for bad in (dict(slots=None), dict(q=None), dict(qo=None), dict(k=None), dict(v=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(slots=10 * A + 4), dict(k=12 * A + 4), dict(wk=30 * A + 8)):
        assert call(**bad) == ALIGN, bad
    for bad in (dict(qo=A), dict(qo=2 * A + 512), dict(qo=4 * A), dict(slots=A), dict(k=A), dict(v=2 * A), dict(qo=10 * A),
                dict(c=c_cache(v=A)), dict(c=c_cache(v_scale=A)), dict(c=c_cache(k_scale=10 * A)), dict(wk=A), dict(rot=c_rotary(positions=A)),
                dict(c=c_cache(v=A + 65536 - 64, k_stride=131072, v_stride=131072))):
        assert call(**bad) == ALIAS, bad
    joint = c_cache(v=A + 65536, k_stride=131072, v_stride=131072, v_scale=3 * A + 2048, k_scale_stride=1024, v_scale_stride=1024)
    assert call(c=joint) in (OK, UNSUPPORTED, CUDA)
    assert call(tokens=0, k=None, v=None, slots=None, q=None, qo=None) == OK


def test_cache_read_refusals(L):
    def call(k=10 * A, v=11 * A, c=None, table=12 * A, ld=10, width=10, offsets=13 * A, batch=4, rows=1000):
        return L.fp8q_cache_read(k, v, c_cache() if c is None else c, table, ld, width, offsets, batch, rows, None)

    for bad in (dict(rows=-1), dict(batch=-1), dict(width=-1), dict(ld=9)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(table=None), dict(offsets=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(k=10 * A + 8), dict(table=12 * A + 2), dict(offsets=13 * A + 4)):
        assert call(**bad) == ALIGN, bad
    for bad in (dict(v=10 * A + 1024), dict(k=A), dict(v=4 * A), dict(k=12 * A), dict(v=13 * A)):
        assert call(**bad) == ALIAS, bad
    assert call(rows=0, k=None, v=None) == OK and call(batch=0) == OK


def test_paged_attention_refusals(L):
    def call(out=10 * A, lse=11 * A, q=12 * A, q_ld=4096, c=None, table=13 * A, ld=10, width=10, lengths=14 * A, batch=4, h=32, scale=0.1,
             window=0, ws=15 * A, size=1 << 30):
        return L.fp8q_paged_attention(out, lse, q, q_ld, c_cache() if c is None else c, table, ld, width, lengths, batch, h, scale, window, ws, size, None)

    for bad in (dict(batch=-1), dict(h=0), dict(h=33), dict(width=-1), dict(width=1 << 24, ld=1 << 24), dict(ld=9), dict(q_ld=4088), dict(q_ld=4100)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1)):
        assert call(**bad) == VALUE, bad
    for bad in (dict(out=None), dict(q=None), dict(table=None), dict(lengths=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(out=10 * A + 8), dict(lse=11 * A + 2), dict(q=12 * A + 8), dict(table=13 * A + 1), dict(lengths=14 * A + 2), dict(ws=15 * A + 4)):
        assert call(**bad) == ALIGN, bad
    for bad in (dict(lse=10 * A), dict(out=12 * A), dict(out=A), dict(lse=3 * A), dict(ws=10 * A), dict(ws=2 * A), dict(out=13 * A), dict(lse=14 * A), dict(ws=12 * A)):
        assert call(**bad) == ALIAS, bad
    assert call(batch=0, out=None, q=None) == OK
    assert L.fp8q_paged_attention_workspace(None, 1, 32, 10) == -1
    assert L.fp8q_paged_attention_workspace(c_cache(), 1, 33, 10) == -1
    assert L.fp8q_paged_attention_workspace(c_cache(head_dim=100), 1, 32, 10) == -1


def test_bindings_refuse_what_is_not_on_a_gpu():
    fq.build()
    x = torch.zeros(4, 2, 64, dtype=BF16)
    cache = fq.paged_cache(1, 16, 2, 64, device="cpu")
    assert cache.k.dtype == INT8 and cache.k_scale.shape == (1, 2, 16)
    assert fq.paged_cache(1, 16, 2, 64, dtype=BF16, device="cpu").k_scale is None
    for f in (lambda: fq.qk_norm_rope(x, x), lambda: fq.cache_write(x, x, cache, torch.zeros(4, dtype=torch.int64)),
              lambda: fq.cache_read(cache, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), 1),
              lambda: fq.paged_attention(x, cache, torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)),
              lambda: fq.qk_norm_rope(1, x), lambda: fq.paged_cache(1, 16, 2, 64, dtype=torch.float16, device="cpu")):
        with pytest.raises(TypeError):
            f()
    for bad in ((1, 24, 2, 64), (1, 16, 2, 96), (1, 0, 2, 64), (1, 2048, 1, 64)):
        with pytest.raises(ValueError):
            fq.paged_cache(*bad, device="cpu")
    for bad in ((), (3,), (0,), (16, -2)):
        with pytest.raises(ValueError):
            fq.rotary_axes(bad, device="cpu")


from tests.test_launch_shapes import fake  # noqa: E402,F401


def test_attention_launches(fake):  # noqa: F811
    """Seen through the stand-in for the runtime: a join only where a sequence may have more tiles than a
    CTA has warps, as many CTAs as are resident, twice as many where there may be much work."""
    got = fake("""
    class Cache(ctypes.Structure):
        _fields_ = [(n, P) for n in ("k", "v", "ks", "vs")] + [(n, I64) for n in ("a", "b", "c", "d", "pages", "page", "heads", "dim")] + [("type", ctypes.c_int)]
    L.fp8q_paged_attention_workspace.restype = I64
    def call(batch, width, heads, kv, dim=128, type=1, page=16):
        n = kv * page
        c = Cache(1 << 40, 2 << 40, 3 << 40, 4 << 40, n * dim, n * dim, n, n, 1000, page, kv, dim, type)
        before = F.fake_launches()
        size = L.fp8q_paged_attention_workspace(ctypes.byref(c), I64(batch), I64(heads), I64(width))
        st = L.fp8q_paged_attention(P(5 << 40), None, P(6 << 40), I64(heads * dim), ctypes.byref(c), P(7 << 40), I64(width), I64(width),
                                    P(8 << 40), I64(batch), I64(heads), ctypes.c_float(1), I64(0), P(9 << 40), I64(size), None)
        n = F.fake_launches() - before
        l = F.fake_launch_at(before)
        return [st, n, l.grid, l.block, size > 0]
    print(json.dumps([call(1, 8, 32, 8), call(1, 9, 32, 8), call(2, 1, 32, 8), call(64, 512, 32, 8), call(1, 8192, 32, 8),
                      call(64, 512, 128, 8), call(64, 512, 128, 8, type=2), call(1, 4, 32, 8, dim=256, type=2), call(1, 5, 32, 8, dim=256, type=2),
                      call(4096, 65528, 4096, 8), call(4096, 65529, 4096, 8), call(0, 8, 32, 8)]))
    """)
    assert got[-1][:2] == [0, 0]  # no sequences: no launch
    assert got[-3][:2] == [0, 2] and got[-2][:2] == [SHAPE, 0]  # 2^40 tiles of heads, and more
    assert got[:-3] == [[0, 1, 64, 256, False], [0, 2, 72, 256, True], [0, 1, 16, 256, False], [0, 2, 608, 256, True],
                   [0, 2, 304, 256, True], [0, 2, 152, 256, True], [0, 2, 304, 256, True], [0, 1, 32, 128, False], [0, 2, 40, 128, True]]


def test_rotary_axes():
    f, axis = fq.rotary_axes((4, 6), theta=100.0, device="cpu")
    assert f.dtype == torch.float64 and axis.tolist() == [0, 0, 1, 1, 1]
    assert f.tolist() == pytest.approx([1.0, 0.1, 1.0, 100 ** (-1 / 3), 100 ** (-2 / 3)], rel=1e-15)


@gpu
def test_bindings_refuse_wrong_tensors():
    t, h, kv, d = 4, 8, 2, 64
    q, k = normal((t, h, d), 1), normal((t, kv, d), 2)
    f, axis = fq.rotary_axes((d,))
    p = torch.arange(t, device="cuda")
    cache, bf = fq.paged_cache(3, 16, kv, d), fq.paged_cache(3, 16, kv, d, dtype=BF16)
    slots = torch.arange(t, device="cuda")
    table, lens = torch.zeros(t, 2, dtype=torch.int32, device="cuda"), torch.ones(t, dtype=torch.int32, device="cuda")
    off = torch.zeros(t + 1, dtype=torch.int64, device="cuda")
    bad = [
        lambda: fq.qk_norm_rope(q.float(), k), lambda: fq.qk_norm_rope(q[0], k), lambda: fq.qk_norm_rope(q[:3], k),
        lambda: fq.qk_norm_rope(q.transpose(0, 1), k), lambda: fq.qk_norm_rope(q[..., ::2], k[..., ::2]),
        lambda: fq.qk_norm_rope(q, k, f), lambda: fq.qk_norm_rope(q, k, None, p), lambda: fq.qk_norm_rope(q, k, f.float(), p),
        lambda: fq.qk_norm_rope(q, k, f, p[:3]), lambda: fq.qk_norm_rope(q, k, f, p.float()),
        lambda: fq.qk_norm_rope(q, k, f, torch.stack([p, p])), lambda: fq.qk_norm_rope(q, k, f, p, axis=axis[:5]),
        lambda: fq.qk_norm_rope(q, k, f, p, axis=axis.long()), lambda: fq.qk_norm_rope(q, k, q_weight=q[0, 0, :32]),
        lambda: fq.qk_norm_rope(q, k, q_weight=torch.ones(d, device="cuda")), lambda: fq.qk_norm_rope(q, k, q_out=k),
        lambda: fq.qk_norm_rope(q, k.cpu()),
        lambda: fq.cache_write(k, k[:3], cache, slots), lambda: fq.cache_write(q, q, cache, slots), lambda: fq.cache_write(k, k, cache, slots.int()),
        lambda: fq.cache_write(k, k, cache, slots[:2]), lambda: fq.cache_write(k, k, cache, slots, q_out=q),
        lambda: fq.cache_write(k, k, cache, slots, q_weight=q[0, 0]), lambda: fq.cache_write(k, k, cache, slots, q=q[:2]),
        lambda: fq.cache_write(k, k, cache._replace(v=bf.v), slots), lambda: fq.cache_write(k, k, cache._replace(k_scale=None), slots),
        lambda: fq.cache_write(k, k, bf._replace(k_scale=cache.k_scale), slots), lambda: fq.cache_write(k, k, cache._replace(k=cache.k.transpose(1, 2)), slots),
        lambda: fq.cache_write(k, k, cache._replace(k_scale=cache.k_scale.double()), slots),
        lambda: fq.cache_read(cache, table.long(), off, 3), lambda: fq.cache_read(cache, table, off.int(), 3), lambda: fq.cache_read(cache, table, off, -1),
        lambda: fq.cache_read(cache, table, off[:3], 3), lambda: fq.cache_read(cache, table, off, 3, k=k[:2]),
        lambda: fq.paged_attention(q[:, :7], cache, table, lens), lambda: fq.paged_attention(q, cache, table, lens.long()),
        lambda: fq.paged_attention(q, cache, table[:2], lens), lambda: fq.paged_attention(q, cache, table, lens[:2]),
        lambda: fq.paged_attention(q, cache, table, lens, lse=torch.empty(t, h, device="cuda")),
        lambda: fq.paged_attention(q, cache, table, lens, out=q.float()), lambda: fq.paged_attention(q.half(), cache, table, lens),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, fq.Fp8qError)):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(fq.Fp8qError):  # an output over an input
        fq.paged_attention(q, cache, table, lens, out=q)
    with pytest.raises(fq.Fp8qError):
        fq.paged_attention(q, cache, table, lens, window=-1)
    with pytest.raises(fq.Fp8qError):
        fq.qk_norm_rope(q, k, q_weight=q[0, 0], eps=0.0)
    with pytest.raises((fq.Fp8qError, TypeError)):
        fq.qk_norm_rope(q.view(t, h * d // 32, 32), k.view(t, kv * d // 32, 32))
