"""The paged cache's attention at the ends of its numbers: values, queries and logits near the ends of
fp32's range, infinities, tables much wider than the sequences, caches that are refused."""
from __future__ import annotations

import math

import pytest
import torch

import fp8_quant_row_gb300 as fq
from tests.test_paged_cache import (A, ALIGN, BAD_CACHES, BF16, L, NULL, OK, TYPES, VALUE, c_cache,  # noqa: F401
                                    check_attention, garbage, gpu, ids, normal, rows_of, scattered)

# (sequences, tokens): each sequence a warp's, a CTA's, shared by CTAs and joined. The number of tiles
# leaves the remainder 0 by 3.
WHERE = {"warp": (400, 48), "cta": (1, 336), "join": (1, 20016)}
where = pytest.mark.parametrize("shape", WHERE.values(), ids=WHERE)
types = pytest.mark.parametrize("dtype", TYPES, ids=ids)


def attend(dtype, k, v, q, batch, scale=None):
    """Writes k, v [batch * n, heads, dim] and attends: (out, log-sum, k and v as stored, in 64 bits)."""
    n, heads, dim, page = len(k) // batch, k.shape[1], k.shape[2], 16
    width = -(-n // page)
    cache = garbage(batch * width, page, heads, dim, dtype)
    table = scattered(batch, width, batch * width, 7)
    t = torch.arange(n, device="cuda")
    slots = (table[:, t // page].long() * page + t % page).flatten()
    fq.cache_write(k, v, cache, slots)
    gk, gv, sk, sv = rows_of(cache, slots)
    k64, v64 = gk.double(), gv.double()
    if sk is not None:
        k64, v64 = k64 * sk.double()[..., None], v64 * sv.double()[..., None]
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    o, lse = fq.paged_attention(q, cache, table, lens, scale=scale, return_lse=True)
    assert fq.device_error() == 0
    return o, lse, k64, v64


def check_all(o, lse, q, k64, v64, scale, dtype, some=5):
    n = len(k64) // len(q)
    for b in list(range(len(q)))[::-(-len(q) // some)]:
        check_attention(o[b], lse[b], q[b], k64[b * n:(b + 1) * n], v64[b * n:(b + 1) * n], scale, dtype)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())


def check_mean(o, lse, v, logit, size_of_logit):
    """One sequence whose weights are all the same, v [n, kv heads, dim] those tokens' values. A weight
    times its value's scale is rounded to fp16 (2^-11; on a grid of 2^-33 of the largest), sums of n / 16
    steps to 2^-21 each. The logit is a sum of 64 products in four steps of 2^-21 of their magnitudes' sum,
    the log-sum rounded a few times at its size."""
    n, kv, dim = v.shape
    want = v.mean(0).repeat_interleave(len(o) // kv, 0)
    size = v.abs().mean(0).repeat_interleave(len(o) // kv, 0)
    largest = v.abs().amax((0, 2)).repeat_interleave(len(o) // kv, 0)[:, None]
    tol = 2.0 ** -8 * want.abs() + 1.01 * ((2.0 ** -11 + n / 16 * 2.0 ** -21 + 2.0 ** -20) * size + 2.0 ** -33 * largest)
    err = (o.double() - want).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), float(err.max()))
    ref = logit + math.log(n)
    assert bool(((lse.double() - ref).abs() <= 4 * 2.0 ** -21 * size_of_logit + 2.0 ** -20 * abs(ref)).all()), (lse.tolist(), ref)


@gpu
@types
@where
def test_rising_logits_over_rows_of_zeros(dtype, shape):
    """Tiles of large values, of zeros and of ordinary ones in turn, each tile's logits 130 powers of two
    above the last one's: what came before counts for nothing, whatever the factors of its weights. (Weights
    below 2^-94 of the largest may count as zero: 2^-130 of values of 2^40 here.)"""
    batch, n = shape
    tile = (torch.arange(n, device="cuda") // 16).repeat(batch)
    k = torch.zeros(batch * n, 2, 64, dtype=BF16, device="cuda")
    k[..., 0] = (90.0 * tile)[:, None].to(BF16)
    v = normal((batch * n, 2, 64), 1) * torch.tensor([2.0 ** 40, 0.0, 1.0], device="cuda")[tile % 3][:, None, None].to(BF16)
    q = normal((batch, 4, 64), 2)
    q[..., 0] = 1.0
    check_all(*(x := attend(dtype, k, v, q, batch, 1.0))[:2], q, *x[2:], 1.0, dtype)


@gpu
@types
@where
@pytest.mark.parametrize("power", [108, 120, 124])
def test_large_values(dtype, shape, power):
    """Values up to the end of bf16's range, ordinary ones beside them."""
    batch, n = shape
    k, q = normal((batch * n, 2, 64), 1), normal((batch, 4, 64), 2, 1.5)
    v = normal((batch * n, 2, 64), 3) * torch.where(torch.arange(batch * n, device="cuda") % 5 < 3, 2.0 ** power, 1.0)[:, None, None].to(BF16)
    check_all(*(x := attend(dtype, k, v, q, batch))[:2], q, *x[2:], 0.125, dtype)


@gpu
@types
@where
def test_small_values(dtype, shape):
    """Values of 2^-98, little above what 8-bit rows take for zeros (2^-100)."""
    batch, n = shape
    k, q = normal((batch * n, 2, 64), 1), normal((batch, 4, 64), 2, 1.5)
    v = (normal((batch * n, 2, 64), 3).float() * 2.0 ** -98).to(BF16)
    check_all(*(x := attend(dtype, k, v, q, batch))[:2], q, *x[2:], 0.125, dtype)


@gpu
@types
@where
def test_small_weights_of_large_values(dtype, shape):
    """A token whose weight is 2^-95 of the others', with values so large that it makes the output."""
    batch, n = shape
    first = torch.arange(batch * n, device="cuda") % n == 0
    k = torch.zeros(batch * n, 2, 64, dtype=BF16, device="cuda")
    k[..., 0] = torch.where(first, 0.0, 66.0)[:, None].to(BF16)
    v = (normal((batch * n, 2, 64), 1).float() * torch.where(first, 2.0 ** 110, 2.0 ** -40)[:, None, None]).to(BF16)
    q = torch.zeros(batch, 4, 64, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    check_all(*(x := attend(dtype, k, v, q, batch, 1.0))[:2], q, *x[2:], 1.0, dtype)


@gpu
@types
@where
def test_the_largest_values(dtype, shape):
    """All values bf16's largest: their mean is no larger."""
    batch, n = shape
    v = torch.full((batch * n, 2, 64), torch.finfo(BF16).max, dtype=BF16, device="cuda")
    k, q = normal((batch * n, 2, 64), 1), normal((batch, 2, 64), 2)
    o, _, _, _ = attend(dtype, k, v, q, batch)
    # fp16 weights 2^-11, sums at most n / 16 2^-21: less than the half step (2^-9) to either side
    assert bool((o == torch.finfo(BF16).max).all())


@gpu
@types
@where
@pytest.mark.parametrize("logit", [-1e31, -1e37, -1e38])
def test_low_logits(dtype, shape, logit):
    """Every logit far below zero, every other token's twice as far: the mean of the rest's values."""
    batch, n = shape
    even = torch.arange(batch * n, device="cuda") % 2 == 0
    k = torch.zeros(batch * n, 2, 64, dtype=BF16, device="cuda")
    k[..., 0] = torch.where(even, logit, 2 * logit)[:, None].to(BF16)
    v = normal((batch * n, 2, 64), 1)
    q = torch.zeros(batch, 4, 64, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    o, lse, k64, v64 = attend(dtype, k, v, q, batch, 1.0)
    for b in range(0, batch, 90):
        at = torch.arange(b * n, (b + 1) * n, 2, device="cuda")
        check_mean(o[b], lse[b], v64[at], float(k64[0, 0, 0]), abs(float(k64[0, 0, 0])))


@gpu
@types
@where
@pytest.mark.parametrize("power", [100, 118, 124])
def test_far_queries_on_small_keys(dtype, shape, power):
    """Queries near the end of bf16's range over keys of 2^-90 (alike, so that all weights are): the
    logits are within fp32, and so is the way to them."""
    batch, n = shape
    k = (normal((1, 2, 64), 1).float() * 2.0 ** -90).to(BF16).repeat(batch * n, 1, 1)
    v = normal((batch * n, 2, 64), 2)
    one = (normal((1, 4, 64), 3).float() * 2.0 ** power).to(BF16)
    q = one.repeat(batch, 1, 1)
    o, lse, k64, v64 = attend(dtype, k, v, q, batch)
    s, m = (torch.einsum("hgd,hd->hg", x.view(2, 2, 64), y).flatten() / 8 for x, y in
            ((one[0].double(), k64[0]), (one[0].double().abs(), k64[0].abs())))
    for b in range(0, batch, 90):
        for h in range(4):
            check_mean(o[b, h:h + 1], lse[b, h:h + 1], v64[b * n:(b + 1) * n, h // 2:h // 2 + 1], float(s[h]), float(m[h]))


@gpu
@types
def test_the_log_sum_of_one_token(dtype):
    """One token's log-sum is its logit, which the product gives exactly here (one value): a product with the scale,
    one by log2(e) and its own back (2^-24 each, and the constants' 2^-25), the scale of 8-bit keys (2^-24, and
    the factor's): 2^-21 of it in all, whatever its size."""
    n = 2000
    k = torch.zeros(n, 1, 64, dtype=BF16, device="cuda")
    k[:, 0, 0] = torch.linspace(0.01, 9, n, device="cuda").to(BF16)
    v = normal((n, 1, 64), 1)
    q = torch.zeros(n, 1, 64, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    o, lse, k64, v64 = attend(dtype, k, v, q, n, 0.37)
    want = k64[:, 0, 0] * 0.37
    assert bool(((lse[:, 0].double() - want).abs() <= 2.0 ** -21 * want).all()), float(((lse[:, 0].double() - want).abs() / want).max())
    assert bool(((o[:, 0].double() - v64[:, 0]).abs() <= (2.0 ** -8 + 2.0 ** -10) * v64[:, 0].abs()).all())


@gpu
@types
def test_infinite_logits(dtype):
    """-infinity is a weight of zero (nothing but that: zeros, and a log-sum of -infinity), +infinity a
    NaN in its head and in no other."""
    n, dim, kv = 300, 64, 3
    k, v = normal((n, kv, dim), 1), normal((n, kv, dim), 2)
    k[..., 0] = k[..., 0].abs() + 1
    q = normal((1, 6, dim), 3)
    q[..., 0] = 1.0
    inf = float("inf")
    if dtype == BF16:  # (8-bit rows with an infinity have the scale NaN)
        gone = torch.arange(n, device="cuda") % 7 == 2
        k[gone, 0, 0], k[5, 1, 0] = -inf, inf
        o, lse, k64, v64 = attend(dtype, k, v, q, 1)
        rest = ~gone
        check_attention(o[0, :2], lse[0, :2], q[0, :2], k64[rest, :1], v64[rest, :1], dim ** -0.5, dtype)
        assert bool(torch.isnan(o[0, 2:4]).all()) and bool(torch.isnan(lse[0, 2:4]).all())
        check_attention(o[0, 4:], lse[0, 4:], q[0, 4:], k64[:, 2:], v64[:, 2:], dim ** -0.5, dtype)
        k[gone, 0, 0], k[5, 1, 0] = 1.0, 1.0
    q[0, 0, 0], q[0, 3, 0] = -inf, inf
    o, lse, k64, v64 = attend(dtype, k, v, q, 1)
    assert not o[0, 0].any() and float(lse[0, 0]) == -inf
    assert bool(torch.isnan(o[0, 3]).all()) and bool(torch.isnan(lse[0, 3]))
    for h in (1, 2, 4, 5):
        c = slice(h // 2, h // 2 + 1)
        check_attention(o[0, h:h + 1], lse[0, h:h + 1], q[0, h:h + 1], k64[:, c], v64[:, c], dim ** -0.5, dtype)


@gpu
@types
@pytest.mark.parametrize("lengths,window", [([5, 0, 130, 17], 0), ([1] * 60, 0), ([3000, 2, 900], 0), ([3000, 2, 900], 40)], ids=str)
def test_wide_tables(dtype, lengths, window):
    """A table for much longer sequences (whose entries are no pages): the same answers as from one that
    is as wide as the longest."""
    page, kv, dim = 16, 2, 128
    width = -(-max(lengths) // page)
    cache = garbage(len(lengths) * width, page, kv, dim, dtype)
    table = scattered(len(lengths), width, len(lengths) * width, 1)
    slots = torch.cat([table[b].long()[(t := torch.arange(n, device="cuda")) // page] * page + t % page for b, n in enumerate(lengths)])
    k, v = normal((len(slots), kv, dim), 2), normal((len(slots), kv, dim), 3)
    fq.cache_write(k, v, cache, slots)
    gk, gv, sk, sv = rows_of(cache, slots)
    k64, v64 = (g.double() if s is None else g.double() * s.double()[..., None] for g, s in ((gk, sk), (gv, sv)))
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q = normal((len(lengths), 8, dim), 4)
    for wide in (1, 16, 300):
        t = torch.full((len(lengths), wide * width), -1, dtype=torch.int32, device="cuda")
        t[:, :width] = table
        o, lse = fq.paged_attention(q, cache, t, lens, window=window, return_lse=True)
        end = 0
        for b, n in enumerate(lengths):
            first, end = end + (max(0, n - window) if window else 0), end + n
            check_attention(o[b], lse[b], q[b], k64[first:end], v64[first:end], dim ** -0.5, dtype)
    assert fq.device_error() == 0


@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=str)
def test_a_refused_cache_is_refused_by_every_call(L, bad, status):
    """The status of the cache's own fault, from each entry point (rows and heads as the sound cache's)."""
    c = c_cache(**bad)
    assert L.fp8q_cache_write(c, 10 * A, None, 0, None, 0, 11 * A, 1024, 12 * A, 1024, None, None, 1e-6, None, 4, 0, None) == status
    assert L.fp8q_cache_read(13 * A, 14 * A, c, 15 * A, 10, 10, 16 * A, 2, 5, None) == status
    assert L.fp8q_paged_attention(13 * A, None, 17 * A, 1 << 20, c, 15 * A, 10, 10, 16 * A, 2, 32, 1.0, 0, 18 * A, 1 << 30, None) == status
    if status not in (NULL, ALIGN):
        assert L.fp8q_paged_attention_workspace(c, 2, 32, 10) == -1


@pytest.mark.parametrize("scale,status", [(3e38, VALUE), (-3e38, VALUE), (math.inf, VALUE), (math.nan, VALUE), (2.0 ** 127, OK), (-1e38, OK)])
def test_scales_refused(L, scale, status):
    """A scale that is beyond fp32 in log2 units (times 1.44) would make every logit a NaN or infinite.
    (No sequences: nothing is launched.)"""
    assert L.fp8q_paged_attention(13 * A, None, 17 * A, 4096, c_cache(), 15 * A, 10, 10, 16 * A, 0, 32, scale, 0, 18 * A, 1 << 30, None) == status
