"""Test helpers for prompt attention and the 8-bit cache: paged pools laid
out from logical sequences, both operators' formulas in 64 bits on the CPU,
and the error that the kernels' number formats allow.

The bounds count roundings.  Rounding to a type is off by at most half a
step, u = finfo.eps / 2 of the value: 2^-8 for bf16, 2^-24 for fp32.  An
output row is out = out_scale * sum_t p_t c_t / sum_t p_t, so with

  e  the largest absolute error of a score of that row (in nats), and
  r  the relative rounding of a probability before the output product,

|error| <= u_bf16 |out| + A (r + 2 e + 2^-18) with A = out_scale sum p |c| /
sum p: the output's own rounding, the rounded numerator, the weights' error
in numerator and denominator, and 2^-18 for what stays in fp32 (the sums, the
exponential to 2^-22, the normalisation).  A score is a sum of K = d_c + d_r
products in fp32, so e <= K 2^-24 S with S = scale sum |q| |c|, plus 2^-22 |s|
for the scaling by log2(e) and the subtraction of the maximum.
"""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 16


def paged(lens, page, rng, slack=3, max_pages=None):
    """(block_table [N, max_pages] with -1 in unused places, pages in the pool)."""
    counts = [-(-n // page) for n in lens]
    total = sum(counts) + slack
    order = rng.permutation(total)
    table = np.full((len(lens), max_pages or max(max(counts), 1)), -1, dtype=np.int32)
    k = 0
    for n, c in enumerate(counts):
        table[n, :c] = order[k:k + c]
        k += c
    return torch.from_numpy(table), total


def put(pool, table, n, values, start=0):
    """Writes values [q, ...] to sequence n's positions from `start` on."""
    P = pool.shape[1]
    for i in range(values.shape[0]):
        t = start + i
        pool[int(table[n, t // P]), t % P] = values[i]


def rows(pool, table, n, length):
    """Sequence n's first `length` rows of a pool, in order."""
    P = pool.shape[1]
    pages = table[n, :-(-length // P)].long()
    return pool[pages].flatten(0, 1)[:length]


def attend(q_lat, q_rope, lat, kr, scale, out_scale, past, r_prob, q_err=0.0, sigma=None):
    """(out, tolerance) [q, H, B, d_c] in 64 bits of the queries of one
    sequence, the i-th at position past + i, over latents lat [L, B, d_c] and
    keys kr [L, d_r].  q_err: the absolute error of a query value.  sigma
    [L, B]: the scales of an 8-bit cache, whose kernel rounds the products
    p_t sigma_t, to r_prob of their value or 2^-24 of the largest."""
    q, qr, c, k = q_lat.double(), q_rope.double(), lat.double(), kr.double()
    L, K = c.shape[0], c.shape[2] + k.shape[1]
    s = (torch.einsum("qhbk,lbk->qhbl", q, c) + torch.einsum("qhr,lr->qhl", qr, k)[:, :, None]) * scale
    S = (torch.einsum("qhbk,lbk->qhbl", q.abs(), c.abs()) + torch.einsum("qhr,lr->qhl", qr.abs(), k.abs())[:, :, None]) * abs(scale)
    later = torch.arange(L)[None] > past + torch.arange(q.shape[0])[:, None]
    s = s.masked_fill(later[:, None, None], -math.inf)
    p = torch.softmax(s, -1)
    seen = (~later)[:, None, None]
    e = (S * seen).amax(-1) * K * 2.0 ** -24 + s.masked_fill(~seen, 0).abs().amax(-1) * 2.0 ** -22
    if q_err:
        e = e + abs(scale) * q_err * (c.abs().sum(-1).T[None, None] * seen).amax(-1)
    out = torch.einsum("qhbl,lbk->qhbk", p, c) * out_scale
    A = torch.einsum("qhbl,lbk->qhbk", p, c.abs()) * abs(out_scale)
    tol = 2.0 ** -8 * out.abs() + A * (r_prob + 2 * e[..., None] + 2.0 ** -18)
    if sigma is not None:
        sig = sigma.double()
        codes = (c / sig[..., None]).abs().sum(0)  # [B, d_c]
        tol = tol + abs(out_scale) * 2.0 ** -24 * (p * sig.T[None, None]).amax(-1)[..., None] * codes[None, None]
    return out, tol


def within(got, out, tol, what=""):
    got = got.double().cpu()
    over = (got - out).abs() - tol
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} values past their bound, by up to {worst:.3e}"


# ----------------------------------------------------------------- the 8-bit cache
def scale_of(values):
    """The scale of one block and branch from its new values (any shape)."""
    v = np.abs(np.asarray(values, dtype=np.float64))
    v = v[np.isfinite(v)]
    amax = float(v.max()) if v.size else 0.0
    s = 2.0 ** -40
    while amax > 448.0 * s:
        s *= 2.0
    return s


def e4m3(x):
    """float64 -> the nearest e4m3 (ties to even, infinities to +-448), as a
    float8 tensor; by the format's definition: steps of 2^(e-3), e >= -6."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.clip(np.where(np.isnan(x), 0.0, x), -448.0, 448.0)
    e = np.floor(np.log2(np.maximum(np.abs(fin), 2.0 ** -30)))
    step = 2.0 ** (np.maximum(e, -6.0) - 3.0)
    y = np.clip(np.rint(fin / step) * step, -448.0, 448.0)
    y = np.where(np.isnan(x), np.nan, y)
    return torch.from_numpy(y).float().to(torch.float8_e4m3fn)  # exact: y is an e4m3 value


def append(cache, scale, rope, table, c_new, kr_new, cu, lens, base):
    """mlra_append_fp8 on CPU copies, block by block: cache float64 values of
    the codes [pages, P, B, d_c], scale float64 [pages, P/16, B], rope float64
    (unrounded keys)."""
    P, d_r = cache.shape[1], kr_new.shape[1]
    for n, L in enumerate(lens):
        q = int(cu[n + 1] - cu[n])
        begin = L - q
        x = c_new[int(cu[n]):int(cu[n + 1])].double().numpy()
        k = kr_new[int(cu[n]):int(cu[n + 1])].double().numpy()
        for p0 in range(begin // BLOCK * BLOCK, L if q else 0, BLOCK):
            lo, hi = max(begin, p0), min(L, p0 + BLOCK)
            page, s0 = int(table[n, p0 // P]), p0 % P
            for b in range(cache.shape[2]):
                old = float(scale[page, s0 // BLOCK, b])
                new = scale_of(x[lo - begin:hi - begin, b])
                if lo > p0 and old >= new:
                    new = old
                if lo > p0:
                    kept = cache[page, s0:s0 + lo - p0, b].numpy() * (old / new)
                    cache[page, s0:s0 + lo - p0, b] = e4m3(kept).double()
                scale[page, s0 // BLOCK, b] = new
                cache[page, s0 + lo - p0:s0 + hi - p0, b] = e4m3(x[lo - begin:hi - begin, b] / new).double()
        for i in range(q):
            t = begin + i
            a = t * base ** (-2.0 * np.arange(d_r // 2) / d_r)
            y = np.empty(d_r)
            y[0::2] = k[i, 0::2] * np.cos(a) - k[i, 1::2] * np.sin(a)
            y[1::2] = k[i, 0::2] * np.sin(a) + k[i, 1::2] * np.cos(a)
            rope[int(table[n, t // P]), t % P] = torch.from_numpy(y)


def quantised(x):
    """(codes float8 [pages, P, B, d_c], scale fp32 [pages, P/16, B]) of a
    bf16 pool, block by block as the append would write whole blocks."""
    pages, P, B, d_c = x.shape
    v = x.double().view(pages, P // BLOCK, BLOCK, B, d_c)
    amax = v.abs().amax((2, 4)).clamp(min=448.0 * 2.0 ** -40)
    s = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
    codes = e4m3((v / s[:, :, None, :, None]).numpy()).view(pages, P, B, d_c)
    return codes, s.float()


def values(codes, scale):
    """float64 latents that the codes and scales stand for."""
    return codes.double() * scale.double().repeat_interleave(BLOCK, 1)[..., None]
