"""The 8-bit decode over a long tail of small, equal weights behind one large
one, in a single CTA's range: what three e5m2 parts leave of such a weight.

A weight w = p sigma / 2^M is rounded to fp16 and then to 2^-21, the step of
the third part's smallest values: off by at most 2^-22 + 2^-25 wherever that is
more than R_PROB of it.  The largest weight of a range of n tokens, 2^13 <= n <=
2^18, is n 2^-11 or more, so the errors of its weights add up to at most 1.125
2^-11 of that one: 1.125 2^-29 for each of 2^18 tokens."""
import math

import pytest
import torch

from branch_latent_kv_b200 import binding as b
from tests.test_fp8_cache import R_PROB


@pytest.mark.gpu
@pytest.mark.parametrize("below", [22.3, 24.5])
def test_a_flat_tail_far_below_a_token_of_no_value(below):
    """One token scores 2^below times the weight of each of 2^18 others and its
    latents are zero, as those of a token that only collects weight are: the
    output is the tail's alone.  160 sequences read the same pages, so that no
    range is shorter than most of a sequence."""
    N, H, L, P, d_c, d_r = 160, 5, 1 << 18, 64, 128, 32
    pages = L // P
    g = torch.Generator().manual_seed(60)
    codes = torch.randn(d_c, generator=g).to(torch.float8_e4m3fn)
    lat = codes.view(torch.uint8)[None].expand(L, d_c).clone()
    lat[77] = 0
    keys = torch.zeros(L, d_r)
    scale, out_scale = 0.125, 0.5
    keys[77, 0] = below * math.log(2.0) / (16.0 * scale)
    keys = keys.to(torch.bfloat16)
    q = torch.zeros(N, H, 1, d_c, dtype=torch.bfloat16)
    qr = torch.zeros(N, H, d_r, dtype=torch.bfloat16)
    qr[..., 0] = 16.0
    got = b.mlra_decode_fp8(q.cuda(), qr.cuda(), lat.view(pages, P, 1, d_c).cuda().view(torch.float8_e4m3fn),
                            torch.full((pages, P // 16, 1), 0.25, device="cuda"), keys.view(pages, P, d_r).cuda(),
                            torch.arange(pages, dtype=torch.int32)[None].expand(N, pages).contiguous().cuda(),
                            torch.full((N,), L, dtype=torch.int32, device="cuda"), scale, out_scale).double().cpu()
    assert b.mlra_read_device_error() == 0
    ratio = math.exp(-16.0 * scale * float(keys[77, 0]))  # of the tail's weights to the large one
    tail = (L - 1) * ratio / (1.0 + (L - 1) * ratio)
    want = (out_scale * 0.25 * tail * codes.double())[None, None, None].expand(N, H, 1, d_c)
    # the weights; the score's fp32 arithmetic and the sums (2^-18 each); the output's rounding
    rel = R_PROB + 1.125 * 2.0 ** -29 / ratio + 2.0 ** -17 + 2.0 ** -22 * 2 * below + 2.0 ** -8
    worst = float(((got - want).abs() / want.abs().clamp(min=1e-30)).max())
    assert worst <= rel, (worst, rel)


@pytest.mark.gpu
@pytest.mark.parametrize("log2", range(20, 34))
def test_scores_so_large_that_the_reference_is_rounded(log2):
    """Scores of 2^log2 in log2 units, where fp32 steps by 2^(log2 - 23): the
    reference, a little below the largest, rounds to it or to a step below."""
    N, H, L, P, d_c, d_r = 3, 16, 300, 64, 128, 64
    pages = -(-L // P)
    g = torch.Generator().manual_seed(61)
    codes = torch.randn(pages, P, 1, d_c, generator=g).to(torch.float8_e4m3fn)
    keys = torch.zeros(pages, P, d_r)
    keys.view(-1, d_r)[:, 0] = 1.0
    q = torch.zeros(N, H, 1, d_c, dtype=torch.bfloat16)
    qr = torch.zeros(N, H, d_r)
    qr[..., 0] = 2.0 ** log2 * (1.0 + torch.arange(H) / 16.0)
    got = b.mlra_decode_fp8(q.cuda(), qr.to(torch.bfloat16).cuda(), codes.cuda(), torch.full((pages, P // 16, 1), 0.5, device="cuda"), keys.to(torch.bfloat16).cuda(),
                            torch.arange(pages, dtype=torch.int32)[None].expand(N, pages).contiguous().cuda(),
                            torch.full((N,), L, dtype=torch.int32, device="cuda"), math.log(2.0), 1.0).double().cpu()
    assert b.mlra_read_device_error() == 0
    # every token scores the same: the mean of the latents
    c = codes.double().view(-1, d_c)[:L] * 0.5
    want, size = c.mean(0), c.abs().mean(0)
    tol = 2.0 ** -8 * want.abs() + size * (R_PROB + 2.0 ** -17)
    assert bool(((got - want).abs() <= tol).all())
