"""Prompt attention of a few new tokens in each of many sequences: every
sequence has row blocks of its own, however few rows they hold.  Split calls
with more clusters than the device holds at once, calls that are not split,
and a served batch that goes from prompts over draft tokens to the 8-bit
cache."""
import math

import numpy as np
import pytest
import torch

from branch_latent_kv_b200 import binding as b
from tests import latent_ref as ref
from tests.test_prefill import SHAPES, _case, _check, _gpu


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c", SHAPES)
def test_short_runs_of_many_sequences(branches, d_c):
    """48 sequences with 1 to 3 new tokens behind up to 4000 cached ones."""
    rng = np.random.default_rng(70)
    new, past = rng.integers(1, 4, 48).tolist(), rng.integers(0, 4001, 48).tolist()
    _check(_case(70, 16, branches, d_c, 64, 64, new, past), f"B={branches} d_c={d_c}")


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c,new", [
    (4, 64, [1, 11, 6]), (4, 128, [11, 6, 1]), (1, 128, [1, 11] * 7), (2, 128, [1, 11] * 3 + [6]),
    (2, 256, [1, 5] * 3), (1, 256, [5, 1] * 7), (1, 512, [1, 5] * 8)])
def test_more_split_clusters_than_the_device_holds(branches, d_c, new):
    """40 heads: an average run fills most of a block, the longer ones take
    two.  By the average the blocks, split in as many parts as there are, fit
    the device at once (15 clusters of 8 CTAs); there are half as many again."""
    rng = np.random.default_rng(71)
    past = (4200 - np.array(new) - rng.integers(0, 2, len(new)) * rng.integers(0, 4100, len(new))).tolist()
    past[-1] = 4200
    _check(_case(71, 40, branches, d_c, 64, 64, new, past), f"B={branches} d_c={d_c}")


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c", [(4, 64), (4, 128), (1, 512)])
def test_single_tokens_of_many_sequences_are_not_split(branches, d_c):
    """A row's bits depend on its sequence alone as long as its block's tokens
    are not divided.  With one new token in each of N sequences there are N
    blocks for each branch: once they fill the device, a call of 40 times as
    many must give the same bits, and it is not split by any count."""
    n = 160 // branches
    c = _case(72, 16, branches, d_c, 64, 64, [1] * n, [4100 - 7 * i for i in range(n)])
    out = _check(c, f"B={branches} d_c={d_c}")
    many = {k: c[k].repeat((40,) + (1,) * (c[k].dim() - 1)) for k in ("q_lat", "q_rope", "block_table", "seqlens")}
    many["cu_seqlens"] = torch.arange(40 * n + 1, dtype=torch.int32)
    got = b.mlra_prefill(**_gpu({**c, **many}))
    assert torch.equal(got, out.repeat(40, 1, 1, 1))


def _rotated(x, pos, base=10000.0):
    """Rotary pairs of x [T, ..., d_r] at positions pos [T], in 64 bits."""
    d = x.shape[-1]
    angle = pos.double()[:, None] * base ** (torch.arange(0, d, 2).double() * (-1.0 / d))
    angle = angle.view(len(pos), *[1] * (x.dim() - 2), d // 2)
    a, z = x.double().view(*x.shape[:-1], d // 2, 2).unbind(-1)
    return torch.stack((a * angle.cos() - z * angle.sin(), a * angle.sin() + z * angle.cos()), -1).view(x.shape)


@pytest.mark.gpu
def test_prompts_drafts_and_steps_of_a_served_batch():
    """Prompts, then two rounds of draft tokens: mlra_prepare with the packed
    tokens as its batch writes the bf16 pool and makes the queries,
    mlra_prefill attends, mlra_append_fp8 writes the same tokens to the 8-bit
    pool; at the end mlra_decode and mlra_decode_fp8 of the last tokens.  Each
    against its formula over the pools' own values."""
    H, B, d_c, d_r, d_h, P, N = 16, 4, 128, 64, 128, 64, 5
    g = torch.Generator().manual_seed(73)

    def normal(*shape, fan=1.0):
        return (torch.randn(*shape, generator=g) / math.sqrt(fan)).to(torch.bfloat16)
    rounds = [[70, 1, 300, 33, 128], [3, 1, 7, 2, 5], [1, 4, 2, 6, 3]]
    total = [sum(r[n] for r in rounds) for n in range(N)]
    table, pages = ref.paged(total, P, np.random.default_rng(73))
    lat = torch.full((pages, P, B, d_c), float("nan"), dtype=torch.bfloat16, device="cuda")
    rope = torch.full((pages, P, d_r), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool8 = (torch.full((pages, P, B, d_c), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
             torch.full((pages, P // 16, B), float("nan"), device="cuda"), torch.full_like(rope, float("nan")))
    w_uk = normal(B, H, d_h, d_c, fan=d_h).cuda()
    scale, out_scale, tb = (d_c + d_r) ** -0.5, B ** -0.5, table.cuda()
    lens = [0] * N
    for k, new in enumerate(rounds):
        T = sum(new)
        lens = [x + q for x, q in zip(lens, new)]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        of = torch.repeat_interleave(torch.arange(N), torch.tensor(new))     # each token's sequence
        upto = torch.cat([torch.arange(L - q + 1, L + 1) for q, L in zip(new, lens)]).int()  # its length with it
        q_c, q_r, c_new, kr_new = normal(T, H, d_h), normal(T, H, d_r), normal(T, B, d_c, fan=d_c), normal(T, d_r, fan=d_r)
        q_lat, q_rope = b.mlra_prepare(q_c.cuda(), q_r.cuda(), w_uk, c_new.cuda(), kr_new.cuda(), upto.cuda(), table[of].contiguous().cuda(), lat, rope)
        got = b.mlra_prefill(q_lat, q_rope, lat, rope, tb, torch.tensor(lens, dtype=torch.int32).cuda(), cu.cuda(), scale, out_scale)
        b.mlra_append_fp8(c_new.cuda(), kr_new.cuda(), cu.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), tb, *pool8)
        # the pre-step: keys and queries turned to their positions, one bf16 rounding
        for turned, x in ((q_rope, q_r), (torch.cat([ref.rows(rope.cpu(), table, n, L)[L - q:] for n, (q, L) in enumerate(zip(new, lens))]), kr_new)):
            want = _rotated(x, upto - 1)
            assert bool(((turned.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * 2 * float(x.abs().max())).all())
        for n, L in enumerate(lens):
            lo, hi = int(cu[n]), int(cu[n + 1])
            o, tol = ref.attend(q_lat[lo:hi].cpu(), q_rope[lo:hi].cpu(), ref.rows(lat.cpu(), table, n, L), ref.rows(rope.cpu(), table, n, L),
                                scale, out_scale, L - (hi - lo), 2.0 ** -8)
            ref.within(got[lo:hi], o, tol, f"round {k}, sequence {n}")
    last = (cu[1:] - 1).long().cuda()
    step = (q_lat[last].contiguous(), q_rope[last].contiguous())
    seqlens = torch.tensor(lens, dtype=torch.int32).cuda()
    full = b.mlra_decode(*step, lat, rope, tb, seqlens, scale, out_scale)
    small = b.mlra_decode_fp8(*step, *pool8, tb, seqlens, scale, out_scale)
    assert b.mlra_read_device_error() == b.MLRA_OK
    values = ref.values(pool8[0].cpu(), pool8[1].cpu())
    sigma = pool8[1].cpu().repeat_interleave(16, 1)
    for n, L in enumerate(lens):
        q, qr = step[0][n:n + 1].cpu(), step[1][n:n + 1].cpu()
        o, tol = ref.attend(q, qr, ref.rows(lat.cpu(), table, n, L), ref.rows(rope.cpu(), table, n, L), scale, out_scale, L - 1, 2.0 ** -8)
        ref.within(full[n:n + 1], o, tol, f"mlra_decode, sequence {n}")
        o, tol = ref.attend(q, qr, ref.rows(values, table, n, L), ref.rows(pool8[2].cpu(), table, n, L), scale, out_scale, L - 1,
                            2.0 ** -9 + 2.0 ** -11, float(q.abs().max()) * 2.0 ** -10 / 224, ref.rows(sigma, table, n, L))
        ref.within(small[n:n + 1], o, tol, f"mlra_decode_fp8, sequence {n}")


@pytest.mark.gpu
@pytest.mark.parametrize("log2", [18, 23, 26, 30, 32, 35, 60])
@pytest.mark.parametrize("branches,d_c,new,past", [(4, 128, 150, 30), (2, 256, 150, 30), (1, 512, 150, 30), (2, 128, 3, 5000)])
def test_scores_so_large_that_fp32_steps_by_more_than_one(branches, d_c, new, past, log2):
    """Every token of a row scores the same, about 2^log2: each row is the mean
    of the latents it sees, whatever the maximum is rounded to."""
    H, P, d_r = 16, 64, 64
    c = _case(74, H, branches, d_c, d_r, P, [new], [past], poison=False)
    c["q_lat"] = torch.zeros_like(c["q_lat"])
    c["q_rope"] = torch.zeros_like(c["q_rope"])
    c["q_rope"][..., 0] = (2.0 ** log2 * (1.0 + torch.arange(new * H) % 128 / 128.0)).view(new, H).to(torch.bfloat16)
    c["rope_cache"] = torch.zeros_like(c["rope_cache"])
    c["rope_cache"][..., 0] = 1.0
    for scale in (0.1, -0.3):
        c["scale"] = scale
        status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        got = b.mlra_prefill(**_gpu(c), device_status=status)
        assert int(status.item()) == 0
        lat = ref.rows(c["latent_cache"], c["block_table"], 0, new + past).double()
        seen = torch.arange(past + 1, past + new + 1).double()[:, None, None]
        mean, size = (x.cumsum(0)[past:] / seen * c["out_scale"] for x in (lat, lat.abs()))
        # equal weights: their rounding to bf16 is one factor, 2^-8 at most
        tol = 2.0 ** -8 * mean.abs() + size * (2.0 ** -8 + 2.0 ** -17)
        ref.within(got, mean[:, None].expand(got.shape), tol[:, None].expand(got.shape), f"scale {scale}")
