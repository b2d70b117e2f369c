"""rms_norm_quant, silu_mul_quant and int8_matmul: against plain 64-bit implementations (GPU), and
their refusals (host only)."""
from __future__ import annotations

import pytest
import torch

import fp8_quant_row_gb300 as fq

OK, NULL, ALIGN, SHAPE, UNSUPPORTED, ALIAS, CUDA, VALUE = range(8)
A = 1 << 24  # fake device addresses, never dereferenced
gpu = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -100


@pytest.fixture(scope="module")
def L():
    fq.build()
    return fq._capi.lib()


# ------------------------------------------------------------------------------------------
# plain forms, 64 bits
# ------------------------------------------------------------------------------------------

def codes(p, dtype):
    """(codes, row maximum) of float64 products p, which are exact: int8 rounds the product with
    the fp32 inverse once, e4m3 takes it through fp32."""
    top = p.abs().amax(-1, keepdim=True)
    ok = torch.isfinite(p).all(-1, keepdim=True) & (top >= TINY)
    qmax = 127.0 if dtype == torch.int8 else 448.0
    inv = torch.where(ok, top.float().reciprocal() * qmax, 0.0)  # each step rounded to fp32
    t = torch.where(ok, p, 0.0) * inv.double()  # 16 x 24 bits: exact in 64
    if dtype == torch.int8:
        q = t.round()
        assert q.abs().max() <= 127
        return q.to(torch.int8), torch.where(ok, top, 0.0)[..., 0]
    return t.float().to(E4M3), torch.where(ok, top, 0.0)[..., 0]


def plain_rms(x, w, r, dtype, eps):
    h = x if r is None else (x.float() + r.float()).bfloat16()
    h64 = h.double()
    p = h64 * w.double()
    q, top = codes(p, dtype)
    scale = top / torch.sqrt(h64.square().mean(-1) + eps) / (127.0 if dtype == torch.int8 else 448.0)
    return h, q, torch.where(torch.isfinite(p).all(-1) & (h64.square().sum(-1) < 3.4e38), scale,
                             float("nan"))


def plain_silu(g, u, dtype):
    s = torch.where(g.double() < -87, 0.0, g.double() / (1 + torch.exp(-g.double())))
    p = s.float().bfloat16().double() * u.double()
    q, top = codes(p, dtype)
    return q, torch.where(torch.isfinite(p).all(-1), top / (127.0 if dtype == torch.int8 else 448.0),
                          float("nan"))


def same_codes(q, ref):
    return torch.equal(q.view(torch.uint8) if q.dtype == E4M3 else q,
                       ref.view(torch.uint8) if q.dtype == E4M3 else ref)


def close_scale(s, ref, cols):
    """fp32 chain: the sum of cols squares takes each through at most cols / 8 + 18 additions (runs
    in a thread, then lanes and warps), each off by at most 2^-24; the square root halves that;
    five more roundings."""
    bad = torch.isnan(ref)
    assert torch.equal(torch.isnan(s), bad)
    d = (s.double() - ref).abs()[~bad]
    assert bool((d <= ((cols / 8 + 18) / 2 + 5) * 2.0 ** -24 * ref.abs()[~bad]).all()), float(d.max())


def normal(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()


def int8(shape, seed, lo=-127, hi=128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int8)


def f32(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(n, generator=g, device="cuda") + 0.5


# ------------------------------------------------------------------------------------------
# rms_norm_quant
# ------------------------------------------------------------------------------------------

NORM_SHAPES = [(1, 8), (3, 16), (2, 248), (5, 1000), (1, 6144), (127, 5120), (300, 2056),
               (1000, 6144), (700, 8192), (9, 12288), (5, 24576), (3, 32768), (4000, 64), (1000, 248),
               (306, 8200), (400, 12288), (310, 32768), (3001, 1024)]


@gpu
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [torch.int8, E4M3])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_quant(rows, cols, dtype, residual):
    x, w = normal((rows, cols), 1, 2.0), (1 + 0.2 * normal((cols,), 2).float()).bfloat16()
    x[:, cols // 2] *= 20
    r = normal((rows, cols), 3) if residual else None
    got = fq.rms_norm_quant(x, w, residual=r, dtype=dtype, eps=1e-5)
    h, q, s = got if residual else (x, *got)
    hr, qr, sr = plain_rms(x, w, r, dtype, 1e-5)
    assert torch.equal(h, hr)
    assert same_codes(q, qr)
    close_scale(s, sr, cols)


@gpu
@pytest.mark.parametrize("dtype", [torch.int8, E4M3])
def test_rms_norm_quant_ties(dtype):
    """Maxima of 127 * 2^e (448 * 2^e): the other values lie on halves of a step."""
    cols = 512
    x = (torch.arange(cols, device="cuda") - cols // 2).float()[None].repeat(6, 1) / 2
    x = x.clamp(-127, 127)
    x *= torch.tensor([1, 2, 0.5, 2.0 ** 20, 2.0 ** -30, 3.5], device="cuda")[:, None]
    x = x.bfloat16()
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    q, s = fq.rms_norm_quant(x, w, dtype=dtype)
    _, qr, sr = plain_rms(x, w, None, dtype, 1e-6)
    assert same_codes(q, qr)
    close_scale(s, sr, cols)


@gpu
@pytest.mark.parametrize("cols", [64, 2056, 6144, 32768])
@pytest.mark.parametrize("dtype", [torch.int8, E4M3])
def test_rms_norm_quant_special_rows(cols, dtype):
    x, w = normal((9, cols), 5), torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, cols - 1] = float("inf")
    x[3] = -0.0
    x[4] = 2.0 ** -110
    x[5, 7] = 2.0 ** 70     # its square leaves fp32
    x[6] = 2.0 ** -90
    x[7, 0] = float("-inf")
    q, s = fq.rms_norm_quant(x, w, dtype=dtype)
    _, qr, sr = plain_rms(x, w, None, dtype, 1e-6)
    assert torch.equal(q.float(), qr.float())
    close_scale(s, sr, cols)
    assert torch.isnan(s).tolist() == [False, True, True, False, False, True, False, True, False]
    assert s[0] == 0 and s[3] == 0 and s[4] == 0 and not q[1].float().any()


@gpu
def test_rms_norm_quant_in_place_and_guards():
    from tests.gpu_util import Guarded
    rows, cols = 37, 1032
    x, w, r = normal((rows, cols), 1), normal((cols,), 2), normal((rows, cols), 3)
    want = fq.rms_norm_quant(x, w, residual=r)
    gh, gq = Guarded((rows, cols), torch.bfloat16), Guarded((rows, cols), torch.int8)
    gs = Guarded((rows,), torch.float32)
    gh.tensor.copy_(r)
    got = fq.rms_norm_quant(x, w, residual=gh.tensor, residual_out=gh.tensor, q=gq.tensor,
                            scale=gs.tensor)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert gh.intact() and gq.intact() and gs.intact()


def scatter(x, kinds):
    """Puts each kind of row at several places among normal ones: the first and last rows, and
    rows far apart, so that the same threads go from a special row to a normal one and back. kinds:
    functions that change a row in place. Returns the kind of each row, -1 for normal ones."""
    rows, kind = x.shape[0], torch.full((x.shape[0],), -1, device="cuda")
    g = torch.Generator().manual_seed(rows)
    places = torch.randperm(rows, generator=g)[:8 * len(kinds)].tolist()
    for i, r in enumerate(places + [0, rows - 1]):
        kinds[i % len(kinds)](x[r])
        kind[r] = i % len(kinds)
    return kind


# widths and row counts of each kernel that goes from row to row: rows of a warp, of a CTA in
# registers, in shared memory (with 256, 512 and 1024 threads)
@gpu
@pytest.mark.parametrize("rows,cols", [(5000, 64), (5000, 1000), (2000, 2056), (1500, 8192),
                                       (1600, 8200), (1500, 12288), (700, 32768)])
@pytest.mark.parametrize("dtype", [torch.int8, E4M3])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_quant_special_rows_among_many(rows, cols, dtype, residual):
    x, w = normal((rows, cols), 5), torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    r = normal((rows, cols), 6) if residual else None

    def put(value, at=slice(None)):
        def change(row):
            row[at] = value
        return change

    kind = scatter(x, [put(0.0), put(float("nan"), 3), put(float("inf"), cols - 1), put(-0.0),
                       put(2.0 ** -110), put(2.0 ** 70, 7), put(2.0 ** -90),
                       put(float("-inf"), 0)])
    if residual:
        r[kind >= 0] = 0
    got = fq.rms_norm_quant(x, w, residual=r, dtype=dtype)
    h, q, s = got if residual else (x, *got)
    hr, qr, sr = plain_rms(x, w, r, dtype, 1e-6)
    assert torch.equal(h.nan_to_num(7.0), hr.nan_to_num(7.0))
    assert torch.equal(q.float(), qr.float())
    close_scale(s, sr, cols)
    nan = torch.isnan(s)
    assert torch.equal(nan, (kind == 1) | (kind == 2) | (kind == 5) | (kind == 7))
    assert not s[(kind == 0) | (kind == 3) | (kind == 4)].any()


@gpu
@pytest.mark.parametrize("cols", [64, 248, 2056, 6144, 8192, 12288, 32768])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_quant_scales_close(cols, residual):
    """A chunk's eight squares go through four roundings at most, and the carried sum of the chunks
    is rounded once, as are the mean and the addition of eps: 7 * 2^-24, halved by the square root.
    The root, its product with the maximum and the quotient are rounded once each: 6.5 * 2^-24 in
    all, and 7 covers the products of these and the carried errors' own roundings (2^-44)."""
    rows = 700
    x, w = normal((rows, cols), 1, 2.0), (1 + 0.2 * normal((cols,), 2).float()).bfloat16()
    x[:, cols // 2] *= 20
    r = normal((rows, cols), 3) if residual else None
    few = [fq.rms_norm_quant(x[i:i + 7], w, residual=None if r is None else r[i:i + 7])[-1]
           for i in range(0, rows, 7)]
    many = fq.rms_norm_quant(x, w, residual=r)[-1]
    _, _, ref = plain_rms(x, w, r, torch.int8, 1e-6)
    for s in (torch.cat(few), many):
        assert bool(((s.double() - ref).abs() <= 7 * 2.0 ** -24 * ref).all())
    # A sum within about 2^-44 of a border of fp32 may go either way, one row in 2^19.
    assert torch.equal(torch.cat(few), many)


# ------------------------------------------------------------------------------------------
# silu_mul_quant
# ------------------------------------------------------------------------------------------

@gpu
def test_silu_of_every_bf16_gate():
    """One row per gate value: p = s is the row's maximum, so the scale gives s, and the codes of
    the two rows' halves its sign. Every finite bf16 gate with |silu| of at least 2^-100."""
    g = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    gate = g[:, None].repeat(1, 8)
    up = torch.ones_like(gate)
    q, s = fq.silu_mul_quant(gate, up)
    g64 = g.double()
    want = torch.where(g64 < -87, 0.0, g64 / (1 + torch.exp(-g64))).float().bfloat16()
    finite = torch.isfinite(want) & torch.isfinite(g64)
    big = finite & (want.float().abs() >= TINY)
    assert bool(big.sum() > 30000)
    top = want.double().abs()
    assert torch.equal(s[big], (top[big] / 127).float())  # divided in 64 bits
    assert torch.equal(q[big][:, 0], (127 * torch.sign(want[big].double())).to(torch.int8))
    small = finite & ~big
    assert not s[small].any() and not q[small].any()
    assert bool(torch.isnan(s[~finite & ~(g64 == float("-inf"))]).all())


SILU_SHAPES = [(1, 8), (3, 24), (5, 1000), (1, 18432), (333, 5640), (700, 2048), (40, 18432),
               (9, 40000), (2, 1 << 20), (3000, 128), (400, 12288),
               (310, 12160), (400, 8192), (1000, 520), (330, 58000), (306, 65536)]


@gpu
@pytest.mark.parametrize("rows,cols", SILU_SHAPES)
@pytest.mark.parametrize("dtype", [torch.int8, E4M3])
@pytest.mark.parametrize("layout", ["packed", "apart"])
def test_silu_mul_quant(rows, cols, dtype, layout):
    gu = normal((rows, 2 * cols), 4, 3.0)
    g, u = gu[:, :cols], gu[:, cols:]
    if layout == "apart":
        g, u = g.contiguous(), u.contiguous()
    q, s = fq.silu_mul_quant(g, u, dtype=dtype)
    qr, sr = plain_silu(g, u, dtype)
    assert same_codes(q, qr)
    close_scale(s, sr, 8)


@gpu
@pytest.mark.parametrize("cols", [64, 1000, 18432, 40000])
@pytest.mark.parametrize("dtype", [torch.int8, E4M3])
def test_silu_mul_quant_special_rows(cols, dtype):
    g, u = normal((7, cols), 5), normal((7, cols), 6)
    g[0] = 0
    g[1, 3] = float("nan")
    u[2, cols - 1] = float("inf")
    g[3] = -1000.0
    u[4] = 0
    g[5, 5] = 1000.0
    q, s = fq.silu_mul_quant(g, u, dtype=dtype)
    qr, sr = plain_silu(g, u, dtype)
    assert torch.equal(q.float(), qr.float())
    close_scale(s, sr, 8)
    assert torch.isnan(s).tolist() == [False, True, True, False, False, False, False]


# the same kernels, and rows wider than shared memory, read twice
@gpu
@pytest.mark.parametrize("rows,cols", [(5000, 64), (5000, 760), (2000, 2056), (1500, 6144),
                                       (1600, 8200), (1500, 18432), (700, 40000), (700, 57856),
                                       (700, 57864)])
@pytest.mark.parametrize("dtype", [torch.int8, E4M3])
def test_silu_mul_quant_special_rows_among_many(rows, cols, dtype):
    gu = normal((rows, 2 * cols), 5)

    def put(half, value, at=slice(None)):
        def change(row):
            row[half * cols:(half + 1) * cols][at] = value
        return change

    kind = scatter(gu, [put(0, 0.0), put(0, float("nan"), 3), put(1, float("inf"), cols - 1),
                        put(0, -1000.0), put(1, 0.0), put(0, 1000.0, 5), put(1, 2.0 ** -120),
                        put(0, float("inf"), 9)])
    gu[kind == 7, cols + 9] = 0.0  # infinity times zero
    g, u = gu[:, :cols], gu[:, cols:]
    q, s = fq.silu_mul_quant(g, u, dtype=dtype)
    qr, sr = plain_silu(g, u, dtype)
    assert torch.equal(q.float(), qr.float())
    close_scale(s, sr, 8)
    assert torch.equal(torch.isnan(s), (kind == 1) | (kind == 2) | (kind == 7))
    assert not s[(kind == 0) | (kind == 3) | (kind == 4) | (kind == 6)].any()


# ------------------------------------------------------------------------------------------
# int8_matmul
# ------------------------------------------------------------------------------------------

def plain_matmul(a, sa, w, sw, bias, dtype):
    out = (a.double() @ w.double().t()) * sw.double() * sa.double()[:, None]
    return out if bias is None else out + bias.double()


def check_matmul(m, n, k, dtype, bias, seed=0, lda=None, lo=-127, hi=128):
    full = int8((m, lda or k), seed + 1, lo, hi)
    a, w = full[:, :k], int8((n, k), seed + 2, lo, hi)
    sa, sw = f32(m, seed + 3) * 0.01, f32(n, seed + 4) * 0.01
    b = normal((n,), seed + 5) if bias else None
    out = fq.int8_matmul(a, sa, w, sw, bias=b, out_dtype=dtype)
    ref = plain_matmul(a, sa, w, sw, b, dtype)
    assert out.shape == (m, n) and out.dtype == dtype
    # |acc| rounded to fp32 (at most k / 1024 + 1 times), two factors and the sum with the bias
    # rounded to fp32, then the output's own half step
    mag = ref.abs() + (b.double().abs() if bias else 0)
    worst = (a.double().abs() @ w.double().abs().t()) * sw.double() * sa.double()[:, None]
    tol = 3 * 2.0 ** -24 * mag + torch.where(worst / (sw.double() * sa.double()[:, None]) > 2 ** 24,
                                             (k / 1024 + 1) * 2.0 ** -24 * worst, 0.0)
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    d = (out.double() - ref).abs()
    assert bool((d <= tol).all()), (float(d.max()), int((d > tol).sum()))
    assert fq.device_error() == 0


MM_SHAPES = [(1, 1, 16), (1, 7, 16), (1, 64, 48), (2, 129, 64), (3, 1000, 4096), (1, 6144, 6144),
             (4, 333, 2064), (5, 2050, 1040), (8, 4096, 1024), (9, 127, 18432), (16, 5120, 5120),
             (17, 640, 512), (31, 1023, 272), (33, 257, 1056), (64, 6144, 2048), (65, 384, 640),
             (100, 1111, 3088), (128, 128, 64), (129, 255, 96), (200, 10007, 256), (256, 2048, 2064),
             (257, 513, 2096), (300, 4100, 1024), (511, 300, 4096), (1000, 1024, 1040),
             (2049, 777, 528), (12, 64, 16), (40, 65, 16), (90, 64, 16), (300, 64, 16),
             # several tiles a CTA, several drains a tile
             (20, 30000, 1104), (60, 25000, 2064), (120, 41000, 1040), (2500, 9000, 2064)]


@gpu
@pytest.mark.parametrize("m,n,k", MM_SHAPES)
@pytest.mark.parametrize("dtype,bias", [(torch.bfloat16, False), (torch.float32, True)])
def test_int8_matmul(m, n, k, dtype, bias):
    check_matmul(m, n, k, dtype, bias)


@gpu
@pytest.mark.parametrize("m", [1, 6, 20, 48, 100, 260])
def test_int8_matmul_strided_rows(m):
    check_matmul(m, 200, 160, torch.float32, True, lda=1024)


@gpu
@pytest.mark.parametrize("m", [1, 5, 16, 40, 130, 300])
@pytest.mark.parametrize("sign", [1, -1])
def test_int8_matmul_largest_sums(m, sign):
    """All products 2^14 (a = -128): sums of up to 2^24 * k / 1024, of which each multiple of
    2^14 is an fp32 value."""
    n, k = 160, 18432
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128 * sign if sign == 1 else 127, dtype=torch.int8, device="cuda")
    one = torch.ones(max(m, n), device="cuda")
    out = fq.int8_matmul(a, one[:m], w, one[:n], out_dtype=torch.float32)
    assert torch.equal(out, torch.full_like(out, float(k * -128 * int(w[0, 0]))))


@gpu
@pytest.mark.parametrize("m", [1, 3, 16, 33, 64, 200])
@pytest.mark.parametrize("n,k", [(515, 1024), (96, 1040), (130, 2048), (1, 64)])
def test_int8_matmul_exact_integers(m, n, k):
    """Scales of one and |sums| below 2^24: the fp32 output is the integer."""
    a, w = int8((m, k), 7, -100, 101), int8((n, k), 8, -100, 101)
    one = torch.ones(max(m, n), device="cuda")
    out = fq.int8_matmul(a, one[:m], w, one[:n], out_dtype=torch.float32)
    assert torch.equal(out.double(), a.double() @ w.double().t())


@gpu
@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_int8_matmul_guards_and_nan_scales(m):
    from tests.gpu_util import Guarded
    n, k = 333, 272
    a, w = int8((m, k), 1), int8((n, k), 2)
    sa, sw = f32(m, 3), f32(n, 4)
    sa[0] = float("nan")
    sw[5] = float("inf")
    g = Guarded((m, n), torch.bfloat16)
    fq.int8_matmul(a, sa, w, sw, out=g.tensor)
    assert g.intact()
    assert bool(torch.isnan(g.tensor[0]).all())
    rest = g.tensor[1:].clone()
    assert not torch.isfinite(rest[:, 5]).any()
    rest[:, 5] = 0
    assert bool(torch.isfinite(rest).all())


@gpu
@pytest.mark.parametrize("m", [2, 12, 30, 70, 140])
def test_int8_matmul_unaligned_vectors(m):
    """The output, the scales and the bias start at any of their elements."""
    n, k = 259, 144
    a, w = int8((m, k), 1), int8((n, k), 2)
    sa, sw, b = f32(m + 1, 3)[1:], f32(n + 3, 4)[3:], normal((n + 1,), 5)[1:]
    buf = torch.zeros(m * n + 1, dtype=torch.bfloat16, device="cuda")
    out = buf[1:].view(m, n)
    fq.int8_matmul(a, sa, w, sw, bias=b, out=out)
    assert torch.equal(out, fq.int8_matmul(a, sa.clone(), w, sw.clone(), bias=b.clone()))
    assert buf[0] == 0


@gpu
def test_int8_matmul_batch_of_one_equals_rows():
    """A token's result does not depend on which other tokens are there beyond the sums' order:
    exact sums make it the same for every kernel."""
    a, w = int8((300, 768), 1, -50, 51), int8((640, 768), 2, -50, 51)
    sa, sw = f32(300, 3), f32(640, 4)
    full = fq.int8_matmul(a, sa, w, sw, out_dtype=torch.float32)
    for m in (1, 8, 9, 16, 17, 33, 65, 129, 200):
        assert torch.equal(full[:m], fq.int8_matmul(a[:m], sa[:m], w, sw, out_dtype=torch.float32))


# ------------------------------------------------------------------------------------------
# offsets beyond 32 bits
# ------------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("m", [1, 16, 40, 128, 300])
def test_int8_matmul_large_weights(m):
    n, k = 140000, 32768  # 4.6 GB
    w = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    w[-40:] = int8((40, k), 1)
    w[:24] = int8((24, k), 2)
    a, sa, sw = int8((m, k), 3), f32(m, 4), f32(n, 5)
    out = fq.int8_matmul(a, sa, w, sw)
    for part in (slice(0, 24), slice(n - 40, n)):
        ref = plain_matmul(a, sa, w[part], sw[part], None, None)
        assert float(((out[:, part].double() - ref).abs() / ref.abs().clamp_min(1)).max()) < 2.0 ** -7
    assert not out[:, 24:-40].any()


@gpu
def test_int8_matmul_large_output():
    m, n, k = 70000, 32768, 64  # 2.3e9 values
    a, w, sa, sw = int8((m, k), 1), int8((n, k), 2), f32(m, 3), f32(n, 4)
    out = fq.int8_matmul(a, sa, w, sw)
    for r in (slice(0, 3), slice(65534, 65540), slice(m - 3, m)):
        ref = plain_matmul(a[r], sa[r], w, sw, None, None)
        assert bool(((out[r].double() - ref).abs() <= 2.0 ** -8 * 1.001 * ref.abs()).all())


@gpu
def test_rows_beyond_four_gigabytes():
    rows, cols = 300000, 8192  # 4.9 GB of bf16
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[:] = normal((1, cols), 1)
    tail = normal((5, cols), 2)
    x[-5:] = tail
    w = normal((cols,), 3)
    q, s = fq.rms_norm_quant(x, w)
    want = fq.rms_norm_quant(tail, w)
    assert torch.equal(q[-5:], want[0]) and torch.equal(s[-5:], want[1])
    assert bool((q[:-5] == q[0]).all()) and bool((s[:-5] == s[0]).all())
    q, s = fq.silu_mul_quant(x[:, :4096], x[:, 4096:])
    want = fq.silu_mul_quant(tail[:, :4096], tail[:, 4096:])
    assert torch.equal(q[-5:], want[0]) and torch.equal(s[-5:], want[1])
    assert bool((q[:-5] == q[0]).all())


# ------------------------------------------------------------------------------------------
# as they are used together
# ------------------------------------------------------------------------------------------

def mlp_block(x, r, w):
    """One MLP block: norm -> gate/up product -> gated activation -> down product."""
    h, q, s = fq.rms_norm_quant(x, w["norm"], residual=r)
    gu = fq.int8_matmul(q, s, w["gu"], w["gu_s"])
    f = gu.shape[-1] // 2
    q2, s2 = fq.silu_mul_quant(gu[..., :f], gu[..., f:])
    return h, fq.int8_matmul(q2, s2, w["down"], w["down_s"])


def block_weights(d, f):
    return {"norm": (1 + 0.1 * normal((d,), 1).float()).bfloat16(), "gu": int8((2 * f, d), 2),
            "gu_s": f32(2 * f, 3) * 0.0003, "down": int8((d, f), 4), "down_s": f32(d, 5) * 0.0003}


@gpu
@pytest.mark.parametrize("shape", [(1,), (2, 7), (130,), (1, 300)])
def test_mlp_block(shape):
    d, f = 512, 1376
    w = block_weights(d, f)
    x, r = normal((*shape, d), 6), normal((*shape, d), 7)
    h, y = mlp_block(x, r, w)
    x2, r2 = x.view(-1, d), r.view(-1, d)
    hr, q, s = plain_rms(x2, w["norm"], r2, torch.int8, 1e-6)
    gu = plain_matmul(q, s, w["gu"], w["gu_s"], None, torch.bfloat16)
    a = torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
    yr = a @ (w["down"].double() * w["down_s"].double()[:, None]).t()
    assert torch.equal(h.view(-1, d), hr)
    assert y.shape == (*shape, d)
    # gate, up and the activation rounded to bf16 (2^-9 rms each at most 2^-8) and the activation
    # to steps of max / 127 (error of half a step at most; its rms under max / 254), all averaged
    # over f products of independent sign: the relative 2-norm stays under the sum of the parts
    rel = float((y.view(-1, d).double() - yr).norm() / yr.norm())
    step = float((a.abs().amax(1) / 254 / a.square().mean(1).sqrt()).max())
    assert rel < 3 * 2.0 ** -8 + step + 2.0 ** -8, (rel, step)


@gpu
@pytest.mark.parametrize("rows", [1, 16, 200])
def test_graph_capture_and_streams(rows):
    d, f = 512, 768
    w = block_weights(d, f)
    x, r = normal((rows, d), 6), normal((rows, d), 7)
    want = mlp_block(x, r, w)
    g = torch.cuda.CUDAGraph()
    xs, rs = x.clone(), r.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mlp_block(xs, rs, w)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        got = mlp_block(xs, rs, w)
    for seed in (20, 21):
        x2, r2 = normal((rows, d), seed), normal((rows, d), seed + 5)
        xs.copy_(x2), rs.copy_(r2)
        g.replay()
        for a, b in zip(got, mlp_block(x2, r2, w)):
            assert torch.equal(a, b)
    s.wait_stream(torch.cuda.current_stream())
    h, q, sc = fq.rms_norm_quant(x, w["norm"], residual=r, stream=s)
    gu = fq.int8_matmul(q, sc, w["gu"], w["gu_s"], stream=s)
    q2, s2 = fq.silu_mul_quant(gu[:, :f], gu[:, f:], stream=s)
    y = fq.int8_matmul(q2, s2, w["down"], w["down_s"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    assert fq.device_error() == 0


@gpu
def test_first_calls_of_a_process_captured():
    """Nothing has run before the capture: the launch caches fill during it."""
    code = """
import torch, fp8_quant_row_gb300 as fq
torch.cuda.init()
x = torch.randn(40, 1024, device="cuda").bfloat16(); w = torch.ones(1024, device="cuda").bfloat16()
W = torch.randint(-127, 128, (2048, 1024), device="cuda", dtype=torch.int8); sw = torch.rand(2048, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = []
    for m in (1, 12, 40):
        q, s = fq.rms_norm_quant(x[:m], w)
        y = fq.int8_matmul(q, s, W, sw)
        outs.append((m, y, *fq.silu_mul_quant(y[:, :1024], y[:, 1024:])))
g.replay(); torch.cuda.synchronize()
for m, y, q2, s2 in outs:
    q, s = fq.rms_norm_quant(x[:m], w)
    assert torch.equal(y, fq.int8_matmul(q, s, W, sw))
    a, b = fq.silu_mul_quant(y[:, :1024], y[:, 1024:])
    assert torch.equal(a, q2) and torch.equal(b, s2)
print("fine")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0 and "fine" in out.stdout, out.stderr[-2000:]


@gpu
@pytest.mark.parametrize("m", [1, 8, 16, 40, 200])
def test_reused_buffers_back_to_back(m):
    """Each product reads rows that the call just before it wrote over others, on kernels that may
    begin while the one before still runs."""
    d = 1024
    w, wq, sw = normal((d,), 1), int8((512, d), 2), f32(512, 3)
    xs = [normal((m, d), 100 + i) for i in range(40)]
    q, s = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    torch.cuda.synchronize()
    outs = []
    for x in xs:
        fq.rms_norm_quant(x, w, q=q, scale=s)
        outs.append(fq.int8_matmul(q, s, wq, sw))
    torch.cuda.synchronize()
    for x, out in zip(xs, outs):
        q, s = fq.rms_norm_quant(x, w)
        torch.cuda.synchronize()
        assert torch.equal(out, fq.int8_matmul(q, s, wq, sw))


@gpu
def test_two_streams_at_once():
    w = block_weights(1024, 2048)
    xs = [normal((m, 1024), 30 + m) for m in (1, 24, 150, 600)]
    rs = [normal(x.shape, 60) for x in xs]
    want = [mlp_block(x, r, w) for x, r in zip(xs, rs)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[] for _ in xs]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mlp_block(xs[i], rs[i], w))
    torch.cuda.synchronize()
    for i, runs in enumerate(got):
        for h, y in runs:
            assert torch.equal(h, want[i][0]) and torch.equal(y, want[i][1])
    assert fq.device_error() == 0


@gpu
@pytest.mark.parametrize("m", [8, 24, 64, 128, 300, 2000])
def test_int8_matmul_beside_copies(m):
    """Its tiles come late and out of order while another stream copies. Sums of small integers are
    exact, so every run gives the same values."""
    n, k = 6144, 6144
    a, w = int8((m, k), 1, -4, 5), int8((n, k), 2, -4, 5)
    sa, sw = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    want = (a.double() @ w.double().t()).float()
    src = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    dst, side = torch.empty_like(src), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(12):
        with torch.cuda.stream(side):
            for _ in range(4):
                dst.copy_(src)
        for _ in range(4):
            outs.append(fq.int8_matmul(a, sa, w, sw, out_dtype=torch.float32))
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    assert all(torch.equal(out, want) for out in outs)


@gpu
@pytest.mark.parametrize("m", [1025, 1200, 2049])
@pytest.mark.parametrize("n,k", [(200, 16), (256, 128), (300, 400), (700, 640), (513, 1040)])
def test_int8_matmul_short_pairs_back_to_back(m, n, k):
    """Products of a few stages on pairs of CTAs, each followed at once by the next and by one on
    single CTAs: the last arrivals of one lie close to the first barriers of the next, whose shared
    memory is the same. Sums of small integers are exact."""
    a, w = int8((m, k), 1, -4, 5), int8((n, k), 2, -4, 5)
    one = torch.ones(max(m, n), device="cuda")
    want = (a.double() @ w.double().t()).float()
    outs = []
    torch.cuda.synchronize()
    for _ in range(40):
        outs.append(fq.int8_matmul(a, one[:m], w, one[:n], out_dtype=torch.float32))
        outs.append(fq.int8_matmul(a[:40], one[:40], w, one[:n], out_dtype=torch.float32))
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    assert all(torch.equal(out, want[:len(out)]) for out in outs)


@gpu
@pytest.mark.parametrize("m,n", [(24, 640), (64, 640), (128, 640), (1030, 300), (2050, 1000)])
@pytest.mark.parametrize("k", [1024, 1152, 4112, 18432])
def test_int8_matmul_many_drains(m, n, k):
    """Several drains of a tile, one of them of a single stage, in every tile shape. Sums of small
    integers are exact."""
    a, w = int8((m, k), 1, -4, 5), int8((n, k), 2, -4, 5)
    one = torch.ones(max(m, n), device="cuda")
    want = (a.double() @ w.double().t()).float()
    outs = [fq.int8_matmul(a, one[:m], w, one[:n], out_dtype=torch.float32) for _ in range(10)]
    assert fq.device_error() == 0
    assert all(torch.equal(out, want) for out in outs)


@gpu
def test_other_threads_run_during_a_call(tmp_path):
    """A launch waits on the host while the stream's queue is full, an allocation for the device:
    other Python threads go on. Stood in for by entry points that sleep and launch nothing."""
    import ctypes
    import subprocess
    import threading
    import time
    src, so = tmp_path / "slow.c", str(tmp_path / "slow.so")
    src.write_text("#include <unistd.h>\nint slow(void) { return usleep(300000); }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", so], check=True)
    slow = ctypes.cast(ctypes.CDLL(so).slow, ctypes.c_void_p).value
    native, lib = fq._native(), fq._capi.lib()
    real = [ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in
            ("fp8q_rms_norm_quant", "fp8q_silu_mul_quant", "fp8q_int8_matmul")]
    x, w = normal((4, 512), 1), torch.ones(512, dtype=torch.bfloat16, device="cuda")
    q, s4, s1 = int8((4, 512), 2), f32(4, 3), f32(4, 4)
    turns, done = [0], threading.Event()

    def other():
        while not done.wait(0.002):
            turns[0] += 1

    native.init(slow, slow, slow, fq._capi.check)
    thread = threading.Thread(target=other)
    try:
        thread.start()
        for call in (lambda: fq.rms_norm_quant(x, w), lambda: fq.silu_mul_quant(x, x),
                     lambda: fq.int8_matmul(q, s4, q, s1)):
            before, t0 = turns[0], time.monotonic()
            call()
            after = turns[0]
            assert time.monotonic() - t0 >= 0.29
            assert after - before >= 10  # of about 140
    finally:
        done.set()
        thread.join()
        native.init(*real, fq._capi.check)
    assert fq.rms_norm_quant(x, w)[0].abs().max() == 127


@gpu
def test_calls_from_several_threads():
    """Each thread on its own stream, all through the same launch caches."""
    import threading
    w = block_weights(512, 1376)
    xs = [normal((m, 512), 40 + m) for m in (2, 20, 90, 330, 1100)]
    want = [mlp_block(x, x, w) for x in xs]
    torch.cuda.synchronize()
    got, failed = [[] for _ in xs], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got[i].append(mlp_block(xs[i], xs[i], w))
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i, runs in enumerate(got):
        assert len(runs) == 30
        for h, y in runs:
            assert torch.equal(h, want[i][0]) and torch.equal(y, want[i][1])
    assert fq.device_error() == 0


@gpu
def test_single_rows_without_a_row_dimension():
    d, f = 512, 1376
    w = block_weights(d, f)
    x, r = normal((d,), 6), normal((d,), 7)
    h, q, s = fq.rms_norm_quant(x, w["norm"], residual=r)
    assert h.shape == q.shape == (d,) and s.shape == ()
    gu = fq.int8_matmul(q, s, w["gu"], w["gu_s"])
    q2, s2 = fq.silu_mul_quant(gu[:f], gu[f:])
    assert gu.shape == (2 * f,) and q2.shape == (f,) and s2.shape == ()
    hr, y = mlp_block(x[None], r[None], w)
    assert torch.equal(h, hr[0])
    assert torch.equal(fq.int8_matmul(q2, s2, w["down"], w["down_s"]), y[0])


@gpu
def test_empty_calls():
    x = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    q, s = fq.rms_norm_quant(x, w)
    assert q.shape == (0, 512) and s.shape == (0,)
    q, s = fq.silu_mul_quant(x, x)
    assert q.shape == (0, 512) and s.shape == (0,)
    out = fq.int8_matmul(q, s, int8((8, 512), 1), f32(8, 2))
    assert out.shape == (0, 8)


@gpu
def test_gpu_refusals_leave_outputs_alone():
    x = normal((4, 512), 1)
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    q = torch.full((4, 512), 77, dtype=torch.int8, device="cuda")
    with pytest.raises(TypeError):
        fq.rms_norm_quant(x, w[:504].contiguous(), q=q)
    with pytest.raises(TypeError):
        fq.rms_norm_quant(x, w, q=q, dtype=E4M3)
    with pytest.raises(TypeError):
        fq.rms_norm_quant(x, w, q=q, residual_out=x.clone())
    with pytest.raises(fq.Fp8qError):
        fq.rms_norm_quant(x, w, residual=x.clone(), residual_out=x, q=q)
    with pytest.raises(fq.Fp8qError):
        fq.rms_norm_quant(x, w, eps=-1.0, q=q)
    with pytest.raises(TypeError):
        fq.silu_mul_quant(x, x[:, :504], q=q)
    with pytest.raises(TypeError):
        fq.silu_mul_quant(x.t(), x.t())
    wq, s4 = int8((8, 512), 1), f32(4, 2)
    with pytest.raises(TypeError):
        fq.int8_matmul(q, s4[:3], wq, f32(8, 3))
    with pytest.raises(TypeError):
        fq.int8_matmul(q, s4, wq[:, :496], f32(8, 3))
    with pytest.raises(fq.Fp8qError):
        fq.int8_matmul(q[:, :504], s4, int8((8, 504), 1), f32(8, 3))
    torch.cuda.synchronize()
    assert bool((q == 77).all())


# ------------------------------------------------------------------------------------------
# refusals, host only
# ------------------------------------------------------------------------------------------

def test_rms_argument_checks(L):
    def call(ro=A, q=2 * A, s=3 * A, x=4 * A, r=5 * A, w=6 * A, t=0, rows=4, cols=512, eps=1e-6):
        return L.fp8q_rms_norm_quant(ro, q, s, x, r, w, t, rows, cols, eps, None)
    assert call(rows=-1) == SHAPE
    assert call(rows=1 << 62) == SHAPE
    for cols in (0, 4, 100, 32776):
        assert call(cols=cols) == SHAPE
    assert call(eps=-1.0) == VALUE and call(eps=float("nan")) == VALUE
    assert call(t=2) == VALUE and call(t=-1) == VALUE
    assert call(rows=0, q=None, x=None) == OK
    for n in ("q", "s", "x", "w"):
        assert call(**{n: None}) == NULL
    assert call(ro=None) == NULL and call(r=None) == NULL  # both or neither
    for n, v in (("q", 2 * A + 8), ("s", 3 * A + 2), ("x", 4 * A + 2), ("w", 6 * A + 8),
                 ("ro", A + 4), ("r", 5 * A + 8)):
        assert call(**{n: v}) == ALIGN, n
    assert call(ro=4 * A) == ALIAS           # h over x
    assert call(ro=5 * A + 64) == ALIAS      # partly over the residual
    assert call(q=A + 64) == ALIAS
    assert call(s=2 * A + 64) == ALIAS
    assert call(q=4 * A) == ALIAS
    assert call(s=6 * A) == ALIAS
    assert call(ro=5 * A, q=5 * A) == ALIAS  # in place, but q over it


def test_silu_argument_checks(L):
    def call(q=A, s=2 * A, g=3 * A, u=4 * A, ld=512, t=0, rows=4, cols=512):
        return L.fp8q_silu_mul_quant(q, s, g, u, ld, t, rows, cols, None)
    for cols in (0, 12, (1 << 20) + 8):
        assert call(cols=cols, ld=1 << 21) == SHAPE
    assert call(ld=504) == SHAPE and call(ld=516) == SHAPE and call(ld=1 << 31) == SHAPE
    assert call(rows=-1) == SHAPE and call(rows=1 << 60) == SHAPE
    assert call(t=5) == VALUE
    assert call(rows=0, g=None) == OK
    for n in ("q", "s", "g", "u"):
        assert call(**{n: None}) == NULL
    for n, v in (("q", A + 8), ("s", 2 * A + 1), ("g", 3 * A + 2), ("u", 4 * A + 8)):
        assert call(**{n: v}) == ALIGN
    assert call(q=3 * A) == ALIAS and call(s=4 * A) == ALIAS and call(s=A + 2044) == ALIAS
    assert call(q=3 * A + 3 * 2048, ld=1024) == ALIAS  # inside the last strided row


def test_matmul_argument_checks(L):
    def call(o=A, a=2 * A, lda=512, sa=3 * A, w=4 * A, sw=5 * A, b=6 * A, t=0, m=4, n=8, k=512):
        return L.fp8q_int8_matmul(o, a, lda, sa, w, sw, b, t, m, n, k, None)
    assert call(m=-1) == SHAPE and call(n=0) == SHAPE and call(m=1 << 31) == SHAPE
    for k in (0, 8, 500, 131072):
        assert call(k=k, lda=1 << 20) == SHAPE
    assert call(lda=496) == SHAPE and call(lda=520) == SHAPE and call(lda=1 << 31) == SHAPE
    assert call(t=2) == VALUE
    assert call(m=0, o=None) == OK
    for name in ("o", "a", "sa", "w", "sw"):
        assert call(**{name: None}) == NULL
    for name, v in (("o", A + 1), ("a", 2 * A + 8), ("sa", 3 * A + 2), ("w", 4 * A + 4),
                    ("sw", 5 * A + 1), ("b", 6 * A + 1)):
        assert call(**{name: v}) == ALIGN
    assert call(o=A + 2, t=1) == ALIGN
    for v in (2 * A, 3 * A, 4 * A, 5 * A, 6 * A):
        assert call(o=v) == ALIAS


def test_binding_fails_loudly_without_the_native_module(monkeypatch, tmp_path):
    monkeypatch.setattr(fq, "NATIVE", str(tmp_path / "missing.so"))
    monkeypatch.setattr(fq, "_native_module", None)
    with pytest.raises(RuntimeError, match="missing"):
        fq.rms_norm_quant(None, None)


def test_native_module_is_rebuilt_for_a_change(monkeypatch):
    import os
    from fp8_quant_row_gb300 import _build
    _build.build()
    assert _build.native_up_to_date()
    built, real = os.path.getmtime(_build.NATIVE), os.path.getmtime
    monkeypatch.setattr(os.path, "getmtime",
                        lambda p: built + 1.0 if p == _build.NATIVE_SOURCE else real(p))
    assert not _build.native_up_to_date()
    monkeypatch.setattr(os.path, "getmtime", real)
    monkeypatch.setattr(_build, "_native_stamp", lambda: "another torch")
    assert not _build.native_up_to_date()


def test_binding_refuses_what_is_no_tensor():
    fq.build()
    x = torch.zeros(4, 512, dtype=torch.bfloat16)
    for bad in (None, 3, "x", [1.0]):
        with pytest.raises(TypeError):
            fq.rms_norm_quant(bad, x)
        with pytest.raises(TypeError):
            fq.silu_mul_quant(x, bad)
        with pytest.raises(TypeError):
            fq.int8_matmul(x, bad, x, x)
    with pytest.raises(TypeError):
        fq.rms_norm_quant(x, x, eps="small")


def test_binding_refuses_cpu_tensors_and_types():
    fq.build()
    x = torch.zeros(4, 512, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fq.rms_norm_quant(x, x[0])
    with pytest.raises(TypeError):
        fq.rms_norm_quant(x, x[0], dtype=torch.uint8)
    with pytest.raises(TypeError):
        fq.silu_mul_quant(x, x)
    with pytest.raises(TypeError):
        fq.silu_mul_quant(x, x, dtype=torch.bfloat16)
    q = torch.zeros(4, 512, dtype=torch.int8)
    with pytest.raises(TypeError):
        fq.int8_matmul(q, torch.ones(4), q, torch.ones(4))
    with pytest.raises(TypeError):
        fq.int8_matmul(q, torch.ones(4), q, torch.ones(4), out_dtype=torch.float16)
