"""The 8-bit cache: mlra_append_fp8 (codes and scales exactly, keys within a
bf16 rounding) and mlra_decode_fp8 (against its formula in 64 bits over the
values the cache stands for), at ragged and block-crossing runs, scales that
grow, non-finite values, poisoned slots, every supported shape, errors,
streams and graphs, and a run of both as a serving loop makes it.

Bounds: a key is rounded once to bf16 (2^-8 of it) from fp32 products with an
angle good to 2^-21 (2^-20 of |x0| + |x1| in all).  In the decode the products
p sigma are rounded to fp16 (2^-11) and split into three e5m2 parts, the last
rounded (2^-9 in all); a query value is split into two e4m3 parts of one scale
for the sequence: off by at most half the smallest e4m3 step, 2^-10, of a unit
that is at most 1/224 of the largest query value."""
import ctypes
import math

import numpy as np
import pytest
import torch

from branch_latent_kv_b200 import binding as b
from branch_latent_kv_b200 import DecodeStep
from tests import latent_ref as ref

R_PROB = 2.0 ** -9 + 2.0 ** -11
SHAPES = [(2, 64), (4, 64), (1, 128), (2, 128), (4, 128), (1, 256), (2, 256), (1, 512)]
F8 = torch.float8_e4m3fn


def _bytes(t):
    return t.view(torch.uint8)


# ----------------------------------------------------------------- append
def _pools(pages, P, B, d_c, d_r, seed):
    """A pool full of arbitrary codes (never NaN), scales and keys."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 127, (pages, P, B, d_c), generator=g, dtype=torch.uint8).view(F8)
    scale = torch.exp2(torch.randint(-12, 4, (pages, P // 16, B), generator=g).float())
    return codes, scale, torch.randn(pages, P, d_r, generator=g).to(torch.bfloat16)


def _append_gpu(pool, table, c_new, kr_new, cu, lens, base=10000.0, status=None):
    b.mlra_append_fp8(c_new.cuda(), kr_new.cuda(), cu.cuda(), lens.cuda(), table.cuda(), *pool, rope_base=base, device_status=status)


def _compare(pool, want, kr_mag, what):
    codes, scale, rope = (t.cpu() for t in pool)
    w_codes, w_scale, w_rope, touched = want
    assert torch.equal(scale.double(), w_scale), f"{what}: scales"
    a, e = codes.double(), w_codes
    same = (a == e) | (a.isnan() & e.isnan())
    assert bool(same.all()), f"{what}: {int((~same).sum())} codes differ"
    err = (rope.double() - w_rope).abs()
    tol = 2.0 ** -8 * w_rope.abs() + 2.0 ** -20 * kr_mag
    tol[~touched] = 0.0
    assert bool((err <= tol).all()), f"{what}: keys"


def _run_append(pool_gpu, state, table, c_new, kr_new, new, lens, what, base=10000.0):
    """One append on the GPU pool and on the CPU statement's state; compared."""
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    lens_t = torch.tensor(lens, dtype=torch.int32)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    _append_gpu(pool_gpu, table, c_new, kr_new, cu, lens_t, base, status)
    assert int(status.item()) == 0
    codes, scale, rope, touched = state
    ref.append(codes, scale, rope, table, c_new, kr_new, cu, lens, base)
    for n, L in enumerate(lens):
        for t in range(L - new[n], L):
            touched[int(table[n, t // codes.shape[1]]), t % codes.shape[1]] = True
    _compare(pool_gpu, state, float(kr_new.float().abs().max()) * 2 if kr_new.numel() else 0.0, what)


def _state(pool):
    return pool[0].double(), pool[1].double(), pool[2].double(), torch.zeros(pool[0].shape[:2], dtype=torch.bool)


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c", SHAPES + [(3, 64), (8, 64)])
@pytest.mark.parametrize("page,d_r", [(16, 64), (64, 32), (128, 64), (48, 6)])
def test_append_in_runs(branches, d_c, page, d_r):
    """Three appends to five sequences: whole prompts and nothing, then runs
    that start and end inside blocks and pages, then single tokens."""
    rng = np.random.default_rng(1)
    g = torch.Generator().manual_seed(1)
    runs = [[5, 0, 16, 100, 31], [11, 40, 1, 0, 3], [1, 1, 1, 1, 1]]
    total = [sum(r[n] for r in runs) for n in range(5)]
    table, pages = ref.paged(total, page, rng)
    pool = _pools(pages, page, branches, d_c, d_r, 2)
    state, gpu = _state(pool), [t.cuda() for t in pool]
    lens = [0] * 5
    for k, new in enumerate(runs):
        lens = [x + y for x, y in zip(lens, new)]
        T = sum(new)
        size = torch.exp2(torch.randint(-9, 9, (T, branches, 1), generator=g).float())
        c_new = (torch.randn(T, branches, d_c, generator=g) * size).to(torch.bfloat16)
        kr_new = torch.randn(T, d_r, generator=g).to(torch.bfloat16)
        _run_append(gpu, state, table, c_new, kr_new, new, lens, f"run {k}")


@pytest.mark.gpu
def test_append_values_at_the_borders():
    """Zeros, the smallest and largest bf16 values, ties between e4m3 values,
    values on and next to 448 sigma, infinities and NaN, in blocks of their own."""
    P, d_c = 16, 64
    rows = []
    for special in ([0.0], [1e-40, 3e-39], [3.3e38, -3.3e38], [448.0, 1.0], [450.0, 1.0], [-448.0, 9.0], [float("inf"), 3.0], [float("nan"), 0.01],
                    [float("nan")] * 2, [float("-inf")] * 3, [1.0625, 17.0, 2.125, 18.0, 19.0, 0.0009765625], [2.0 ** -40, 2.0 ** -50, 448 * 2.0 ** -40]):
        row = torch.zeros(16, 1, d_c)
        row.view(-1)[:len(special)] = torch.tensor(special)
        rows.append(row)
    c_new = torch.cat(rows).to(torch.bfloat16)
    T = c_new.shape[0]
    table, pages = ref.paged([T], P, np.random.default_rng(2))
    pool = _pools(pages, P, 1, d_c, 32, 3)
    state, gpu = _state(pool), [t.cuda() for t in pool]
    _run_append(gpu, state, table, c_new, torch.randn(T, 32).to(torch.bfloat16), [T], [T], "borders")


@pytest.mark.gpu
def test_append_grows_a_blocks_scale_and_keeps_the_rest():
    """Tokens one at a time whose size jumps up and down: each jump up rounds
    the block's earlier rows again, nothing else changes."""
    P, B, d_c, d_r = 32, 2, 128, 64
    table, pages = ref.paged([40], P, np.random.default_rng(3))
    pool = _pools(pages, P, B, d_c, d_r, 4)
    state, gpu = _state(pool), [t.cuda() for t in pool]
    g = torch.Generator().manual_seed(4)
    grown = 0
    for i in range(40):
        size = 2.0 ** [0, -3, 4, 4, 9, -20, 12, 0][i % 8]
        c_new = (torch.randn(1, B, d_c, generator=g) * size).to(torch.bfloat16)
        before = state[1].clone()
        _run_append(gpu, state, table, c_new, torch.randn(1, d_r, generator=g).to(torch.bfloat16), [1], [i + 1], f"token {i}")
        grown += int(i % 16 != 0 and bool((state[1] > before).any()))
    assert grown >= 5


@pytest.mark.gpu
def test_append_at_a_far_position():
    """A key two million positions in keeps its phase."""
    P, L = 128, 2_000_001
    table = torch.zeros(1, -(-L // P), dtype=torch.int32)
    table[0, -1] = 1
    pool = _pools(3, P, 1, 64, 64, 5)
    codes, scale, rope, touched = _state(pool)
    gpu = [t.cuda() for t in pool]
    _run_append(gpu, (codes, scale, rope, touched), table, torch.randn(1, 1, 64).to(torch.bfloat16), torch.randn(1, 64).to(torch.bfloat16), [1], [L], "far")


@pytest.mark.gpu
def test_append_reports_bad_runs_and_writes_nothing_for_them():
    P, B, d_c, d_r = 64, 4, 128, 64
    table, pages = ref.paged([100, 100, 100], P, np.random.default_rng(6))
    pool = _pools(pages, P, B, d_c, d_r, 6)
    c_new, kr_new = torch.randn(30, B, d_c).to(torch.bfloat16), torch.randn(30, d_r).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    S, I = b.MLRA_ERR_DEVICE_BAD_SEQLEN, b.MLRA_ERR_DEVICE_BAD_INDEX
    for cu, lens, page, code, written in [([0, 10, 20, 30], [50, 9, 50], None, S, (0, 2)), ([0, 10, 20, 30], [50, 129, 50], None, S, (0, 2)),
                                          ([0, 10, 20, 30], [50, -1, 50], None, S, (0, 2)), ([0, 10, 5, 30], [50, 50, 50], None, S, None),
                                          ([0, 10, 20, 31], [50, 50, 50], None, S, (0, 1)), ([-4, 10, 20, 30], [50, 50, 50], None, S, (1, 2)),
                                          ([0, 10, 20, 30], [50, 50, 50], -1, I, (0, 2)), ([0, 10, 20, 30], [50, 50, 50], pages, I, (0, 2))]:
        gpu = [t.cuda() for t in pool]
        tb = table.clone()
        if page is not None:
            tb[1, 0] = page
        _append_gpu(gpu, tb, c_new, kr_new, torch.tensor(cu, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32), status=status)
        assert int(status.item()) == code, (cu, lens, page)
        if written is None:
            continue
        changed = torch.zeros(pages, P, dtype=torch.bool)
        changed |= (gpu[2].cpu() != pool[2]).any(-1)
        want = torch.zeros_like(changed)
        for n in written:
            for t in range(lens[n] - 10, lens[n]):
                want[int(table[n, t // P]), t % P] = True
        assert torch.equal(changed, want), (cu, lens, page)
        rows_changed = (_bytes(gpu[0]).cpu() != _bytes(pool[0])).flatten(2).any(-1)
        blocks = want.view(pages, -1, 16).any(-1)
        assert not bool((rows_changed & ~blocks.repeat_interleave(16, 1)).any())
    gpu = [t.cuda() for t in pool]
    b.mlra_append_fp8(c_new[:0].cuda(), kr_new[:0].cuda(), torch.zeros(4, dtype=torch.int32).cuda(), torch.tensor([50, 0, 3], dtype=torch.int32).cuda(),
                      table.cuda(), *gpu, device_status=status)
    assert int(status.item()) == 0 and torch.equal(_bytes(gpu[0]).cpu(), _bytes(pool[0]))


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 31, 33, 1100])
def test_append_of_many_sequences(batch):
    """The search of a block's sequence: batches around and past 32^2, runs of
    0 to 40 tokens."""
    rng = np.random.default_rng(batch)
    new = rng.integers(0, 41 if batch < 100 else 3, batch).tolist()
    past = rng.integers(0, 20, batch).tolist()
    lens = [max(p, 0) + q for p, q in zip(past, new)]
    table, pages = ref.paged([max(x, 1) for x in lens], 16, rng)
    pool = _pools(pages, 16, 1, 64, 32, 7)
    state, gpu = _state(pool), [t.cuda() for t in pool]
    T = sum(new)
    _run_append(gpu, state, table, torch.randn(T, 1, 64).to(torch.bfloat16), torch.randn(T, 32).to(torch.bfloat16), new, lens, f"{batch} sequences")


# ----------------------------------------------------------------- decode
def _decode_case(seed, H, B, d_c, d_r, P, lens, std=2.0, spread=1.0, poison=True):
    """CPU tensors of one step; token sizes 2^(spread * normal); unused slots NaN."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    table, pages = ref.paged(lens, P, rng)
    lat = torch.zeros(pages, P, B, d_c, dtype=torch.bfloat16)
    rope = torch.full((pages, P, d_r), float("nan") if poison else 0.0, dtype=torch.bfloat16)
    used = torch.zeros(pages, P, dtype=torch.bool)
    scale = (d_c + d_r) ** -0.5
    gain = std / (scale * math.sqrt(1.0 / d_c + 1.0 / d_r))
    for n, L in enumerate(lens):
        size = torch.exp2(spread * torch.randn(L, B, 1, generator=g))
        ref.put(lat, table, n, (torch.randn(L, B, d_c, generator=g) * size * d_c ** -0.5).to(torch.bfloat16))
        ref.put(rope, table, n, (torch.randn(L, d_r, generator=g) * d_r ** -0.5).to(torch.bfloat16))
        ref.put(used, table, n, torch.ones(L, dtype=torch.bool))
    codes, sigma = ref.quantised(lat)
    if poison:
        _bytes(codes)[~used] = 0x7f
        sigma[~used.view(pages, -1, 16).any(-1)] = float("nan")
    N = len(lens)
    q = (torch.randn(N, H, B, d_c, generator=g) * gain * d_c ** -0.5).to(torch.bfloat16)
    qr = (torch.randn(N, H, d_r, generator=g) * gain * d_r ** -0.5).to(torch.bfloat16)
    return dict(q_lat=q, q_rope=qr, latent_cache=codes, latent_scale=sigma, rope_cache=rope, block_table=table,
                seqlens=torch.tensor(lens, dtype=torch.int32), scale=scale, out_scale=B ** -0.5)


def _gpu(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def _expect(c):
    out = torch.zeros(c["q_lat"].shape, dtype=torch.float64)
    tol = torch.zeros_like(out)
    per_token = c["latent_scale"].repeat_interleave(16, 1)
    lat = ref.values(c["latent_cache"], c["latent_scale"])
    for n, L in enumerate(c["seqlens"].tolist()):
        q_err = float(c["q_lat"][n].float().abs().max()) * 2.0 ** -10 / 224
        o, t = ref.attend(c["q_lat"][n:n + 1], c["q_rope"][n:n + 1], ref.rows(lat, c["block_table"], n, L), ref.rows(c["rope_cache"], c["block_table"], n, L),
                          c["scale"], c["out_scale"], L - 1, R_PROB, q_err, ref.rows(per_token, c["block_table"], n, L))
        out[n], tol[n] = o[0], t[0]
    return out, tol


def _check(c, what=""):
    g = _gpu(c)
    got = b.mlra_decode_fp8(**g)
    torch.cuda.synchronize()
    assert b.mlra_read_device_error() == 0
    ref.within(got, *_expect(c), what)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c", SHAPES)
@pytest.mark.parametrize("d_r,page", [(32, 16), (64, 64), (64, 128), (32, 32)])
def test_every_shape_on_ragged_lengths(branches, d_c, d_r, page):
    _check(_decode_case(20, 12, branches, d_c, d_r, page, [1000, 1, 640, 129, 2047]), f"B={branches} d_c={d_c} d_r={d_r} P={page}")


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 5, 16, 17, 40, 128])
@pytest.mark.parametrize("branches,d_c", [(4, 128), (2, 64), (1, 512)])
def test_head_counts(heads, branches, d_c):
    _check(_decode_case(21, heads, branches, d_c, 64, 32, [513, 33, 3000]), f"H={heads}")


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1], [2, 15, 16, 17], [127, 128, 129], [1] * 300, [20000], [255, 4096, 1, 8191]])
def test_lengths(lens):
    _check(_decode_case(22, 16, 4, 128, 64, 64, lens), f"{lens[:4]}")


@pytest.mark.gpu
@pytest.mark.parametrize("std,spread", [(0.0, 0.0), (0.5, 6.0), (8.0, 1.0), (4.0, 10.0)])
@pytest.mark.parametrize("branches,d_c", [(4, 128), (4, 64), (1, 256)])
def test_score_and_scale_spreads(std, spread, branches, d_c):
    """Flat and peaked scores; scales that differ by up to 2^60 in a sequence."""
    _check(_decode_case(23, 16, branches, d_c, 64, 64, [1500, 300, 17], std=std, spread=spread), f"std={std} spread={spread}")


@pytest.mark.gpu
def test_a_sink_token_and_a_flat_tail():
    """One token scored far above a long flat tail: the tail's small weights
    add up to as much as the sink's."""
    c = _decode_case(24, 16, 4, 128, 64, 64, [16000], std=0.1, spread=0.0)
    k = torch.zeros(64)
    k[0] = 1.0
    c["q_rope"] = torch.zeros_like(c["q_rope"])
    c["q_rope"][..., 0] = 64.0
    ref.put(c["rope_cache"], c["block_table"], 0, (k * math.log(16000.0) / (64.0 * c["scale"])).to(torch.bfloat16)[None], start=40)
    _check(c)


@pytest.mark.gpu
def test_scores_that_keep_growing():
    """Every tile raises the running maximum by more than the lazy rescale
    lets stand; then every tile lowers it."""
    for sign in (1.0, -1.0):
        c = _decode_case(25, 8, 4, 128, 64, 64, [1300], std=1.0)
        k = torch.nn.functional.normalize(c["q_rope"][0].float().mean(0), dim=0)
        c["q_rope"] = (k * 40).to(torch.bfloat16).expand_as(c["q_rope"]).contiguous()
        ref.put(c["rope_cache"], c["block_table"], 0, (torch.linspace(-sign, sign, 1300)[:, None] * k * 60).to(torch.bfloat16))
        _check(c, f"sign {sign}")


@pytest.mark.gpu
def test_scales_that_are_no_powers_of_two():
    c = _decode_case(26, 16, 4, 128, 64, 64, [700, 90], poison=False)
    c["latent_scale"] = c["latent_scale"] * (1 + torch.rand(c["latent_scale"].shape, generator=torch.Generator().manual_seed(1)))
    _check(c)


@pytest.mark.gpu
def test_length_one_is_the_latent():
    c = _decode_case(27, 16, 4, 128, 64, 64, [1, 1, 1], std=20.0)
    got = b.mlra_decode_fp8(**_gpu(c)).cpu()
    lat = ref.values(c["latent_cache"], c["latent_scale"])
    for n in range(3):
        want = (lat[int(c["block_table"][n, 0]), 0] * c["out_scale"]).to(torch.bfloat16)
        assert torch.equal(got[n], want[None].expand_as(got[n]))


@pytest.mark.gpu
def test_a_query_that_is_not_finite_stays_in_its_head():
    c = _decode_case(33, 20, 4, 128, 64, 64, [700, 5000, 30])
    out, tol = _expect(c)
    c["q_lat"][0, 3, 1, 5] = float("nan")
    c["q_lat"][1, 18, 0, 127] = float("inf")
    c["q_lat"][1, 2, 3, 0] = -float("inf")
    c["q_rope"][2, 7, 9] = float("nan")
    got = b.mlra_decode_fp8(**_gpu(c)).double().cpu()
    lost = torch.zeros(got.shape[:3], dtype=torch.bool)
    for at in ((0, 3, 1), (1, 18, 0), (1, 2, 3)):
        lost[at] = True
    lost[2, 7] = True
    assert bool(got[lost].isnan().all())
    ref.within(got[~lost], out[~lost], tol[~lost])


@pytest.mark.gpu
def test_page_order_and_repeats_give_the_same_bits():
    c = _decode_case(28, 16, 4, 128, 64, 64, [3000, 1, 640, 129, 2049])
    perm = torch.randperm(c["latent_cache"].shape[0], generator=torch.Generator().manual_seed(2))
    inv = torch.argsort(perm)
    d = {**c, "latent_cache": _bytes(c["latent_cache"])[inv].view(F8), "latent_scale": c["latent_scale"][inv], "rope_cache": c["rope_cache"][inv],
         "block_table": torch.where(c["block_table"] >= 0, perm[c["block_table"].clamp(min=0).long()].int(), -1).to(torch.int32)}
    one = b.mlra_decode_fp8(**_gpu(c))
    assert torch.equal(one, b.mlra_decode_fp8(**_gpu(d)))
    assert torch.equal(one, b.mlra_decode_fp8(**_gpu(c)))


@pytest.mark.gpu
def test_bad_sequences_are_reported_and_zeroed():
    c = _decode_case(29, 40, 4, 128, 64, 64, [300, 5000, 70])
    out, tol = _expect(c)
    limit = 64 * c["block_table"].shape[1]
    for lens, page, code in [((300, 0, 70), None, b.MLRA_ERR_DEVICE_BAD_SEQLEN), ((300, limit + 1, 70), None, b.MLRA_ERR_DEVICE_BAD_SEQLEN),
                             ((300, -3, 70), None, b.MLRA_ERR_DEVICE_BAD_SEQLEN), ((300, 5000, 70), -1, b.MLRA_ERR_DEVICE_BAD_INDEX),
                             ((300, 5000, 70), c["latent_cache"].shape[0], b.MLRA_ERR_DEVICE_BAD_INDEX)]:
        d = {**c, "seqlens": torch.tensor(lens, dtype=torch.int32), "block_table": c["block_table"].clone()}
        if page is not None:
            d["block_table"][1, 50] = page
        got = b.mlra_decode_fp8(**_gpu(d))
        assert b.mlra_read_device_error() == code
        assert b.mlra_read_device_error() == 0
        assert bool((got[1] == 0).all())
        ref.within(got[[0, 2]], out[[0, 2]], tol[[0, 2]])


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[300, 1, 512, 77], [512] * 3, [100] * 160])
@pytest.mark.parametrize("branches,d_c", [(4, 128), (2, 64), (1, 512)])
def test_short_contexts(lens, branches, d_c):
    """Block tables of at most four tiles: a CTA for each sequence and head
    tile (and, with 160 sequences, the split kernel)."""
    c = _decode_case(36, 20, branches, d_c, 64, 64, lens)
    _check(c, f"{lens[:4]}")
    d = {**c, "seqlens": c["seqlens"].clone(), "block_table": c["block_table"].clone()}
    d["seqlens"][0] = 0
    got = b.mlra_decode_fp8(**_gpu(d))
    assert b.mlra_read_device_error() == b.MLRA_ERR_DEVICE_BAD_SEQLEN
    out, tol = _expect(c)
    assert bool((got[0] == 0).all())
    ref.within(got[1:], out[1:], tol[1:])
    d["seqlens"][0] = c["seqlens"][0]
    d["block_table"][1, 0] = -5
    got = b.mlra_decode_fp8(**_gpu(d))
    assert b.mlra_read_device_error() == b.MLRA_ERR_DEVICE_BAD_INDEX
    assert bool((got[1] == 0).all())
    keep = [0] + list(range(2, len(lens)))
    ref.within(got[keep], out[keep], tol[keep])


@pytest.mark.gpu
def test_streams_graphs_and_workspaces():
    """Calls on two streams at once, two captured graphs replayed at once and
    an eager call between: none shares a workspace with another."""
    c = _decode_case(30, 16, 4, 128, 64, 64, [4000, 900, 17, 2500])
    d = _decode_case(31, 16, 4, 128, 64, 64, [100, 6000, 3000, 1])
    gc, gd = _gpu(c), _gpu(d)
    want_c, want_d = b.mlra_decode_fp8(**gc), b.mlra_decode_fp8(**gd)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    graphs, outs = [], []
    for g in (gc, gd):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(b.mlra_decode_fp8(**g))
        graphs.append(graph)
    for _ in range(5):
        with torch.cuda.stream(s1):
            one = b.mlra_decode_fp8(**gc)
            graphs[0].replay()
        with torch.cuda.stream(s2):
            two = b.mlra_decode_fp8(**gd)
            graphs[1].replay()
        three = b.mlra_decode_fp8(**gc)
    torch.cuda.synchronize()
    assert torch.equal(one, want_c) and torch.equal(two, want_d) and torch.equal(three, want_c)
    assert torch.equal(outs[0], want_c) and torch.equal(outs[1], want_d)
    ws = torch.zeros(b.mlra_decode_workspace_bytes(b.mlra_dims(4, 16, 4, 128, 64, 64, gc["block_table"].shape[1], gc["latent_cache"].shape[0])),
                     dtype=torch.uint8, device="cuda")
    by_arg = b.mlra_decode_fp8(**gc, workspace=ws, stream=s1)
    torch.cuda.synchronize()
    assert torch.equal(by_arg, want_c)
    assert torch.equal(b.mlra_decode_fp8(**gc, workspace=ws), want_c)
    with pytest.raises(b.MlraError):
        b.mlra_decode_fp8(**gc, workspace=ws[:4096])
    # the workspace serves mlra_decode too (same layout, counters left at zero)
    lat = ref.values(c["latent_cache"], c["latent_scale"].nan_to_num(1.0)).to(torch.bfloat16).cuda()
    full = b.mlra_decode(gc["q_lat"], gc["q_rope"], lat, gc["rope_cache"], gc["block_table"], gc["seqlens"], c["scale"], c["out_scale"], workspace=ws)
    out, tol = _expect(c)
    ref.within(full, out, tol + 2.0 ** -7 * out.abs().amax(-1, keepdim=True), "mlra_decode over the same values")


@pytest.mark.gpu
def test_pool_past_32_bit_offsets():
    """Pages behind 2^32 bytes of latents, written by the append and read by
    the decode."""
    P, B, d_c, d_r, L = 64, 4, 128, 64, 200
    pages = (1 << 32) // (P * B * d_c) + 50
    codes = torch.empty(pages, P, B, d_c, dtype=torch.uint8, device="cuda").view(F8)
    scale = torch.empty(pages, P // 16, B, device="cuda")
    rope = torch.empty(pages, P, d_r, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1, pages - 40, pages - 3, pages - 2]], dtype=torch.int32)
    g = torch.Generator().manual_seed(32)
    c_new, kr = torch.randn(L, B, d_c, generator=g).to(torch.bfloat16), torch.randn(L, d_r, generator=g).to(torch.bfloat16)
    _append_gpu((codes, scale, rope), table, c_new, kr, torch.tensor([0, L], dtype=torch.int32), torch.tensor([L], dtype=torch.int32))
    near = pages - 64
    c = dict(q_lat=(torch.randn(1, 8, B, d_c, generator=g)).to(torch.bfloat16), q_rope=torch.randn(1, 8, d_r, generator=g).to(torch.bfloat16),
             latent_cache=_bytes(codes)[near:].cpu().view(F8), latent_scale=scale[near:].cpu(), rope_cache=rope[near:].cpu(), block_table=table - near,
             seqlens=torch.tensor([L], dtype=torch.int32), scale=0.05, out_scale=0.5)
    state = (torch.zeros(64, P, B, d_c, dtype=torch.float64), torch.zeros(64, P // 16, B, dtype=torch.float64), torch.zeros(64, P, d_r, dtype=torch.float64))
    ref.append(*state, c["block_table"], c_new, kr, torch.tensor([0, L]), [L], 10000.0)
    assert torch.equal(ref.rows(c["latent_cache"].double(), c["block_table"], 0, L), ref.rows(state[0], c["block_table"], 0, L))
    got = b.mlra_decode_fp8(c["q_lat"].cuda(), c["q_rope"].cuda(), codes, scale, rope, table.cuda(), c["seqlens"].cuda(), 0.05, 0.5)
    ref.within(got, *_expect(c))


@pytest.mark.gpu
def test_serving_loop():
    """A served batch: prompts by the pre-step and mlra_prefill over a bf16
    pool, moved to the 8-bit cache by one append, then decode steps, each an
    append of one token and mlra_decode_fp8, the last through DecodeStep with
    the up-projection.  Checked against the formulas over the cache's values."""
    H, B, d_c, d_r, d_h, P = 16, 4, 128, 64, 64, 64
    prompts, steps = [70, 1, 33], 4
    N = len(prompts)
    g = torch.Generator().manual_seed(33)

    def normal(*shape, fan=1.0):
        return (torch.randn(*shape, generator=g) / math.sqrt(fan)).to(torch.bfloat16)
    rng = np.random.default_rng(33)
    table, pages = ref.paged([n + steps for n in prompts], P, rng)
    pool = _pools(pages, P, B, d_c, d_r, 33)
    state, gpu = _state(pool), [t.cuda() for t in pool]
    T = sum(prompts)
    _run_append(gpu, state, table, normal(T, B, d_c, fan=d_c), normal(T, d_r), prompts, prompts, "prompts")
    scale, out_scale, tb = (d_c + d_r) ** -0.5, B ** -0.5, table.cuda()
    lens = list(prompts)
    for k in range(steps):
        lens = [n + 1 for n in lens]
        _run_append(gpu, state, table, normal(N, B, d_c, fan=d_c), normal(N, d_r), [1] * N, lens, f"step {k}")
        c = dict(q_lat=normal(N, H, B, d_c), q_rope=normal(N, H, d_r), latent_cache=gpu[0].cpu(), latent_scale=gpu[1].cpu(), rope_cache=gpu[2].cpu(),
                 block_table=table, seqlens=torch.tensor(lens, dtype=torch.int32), scale=scale, out_scale=out_scale)
        got = b.mlra_decode_fp8(c["q_lat"].cuda(), c["q_rope"].cuda(), *gpu, tb, c["seqlens"].cuda(), scale, out_scale)
        ref.within(got, *_expect(c), f"step {k}")
    w_uv = normal(B, d_c, H * d_h, fan=B * d_c).cuda()
    args = (c["q_lat"].cuda(), c["q_rope"].cuda(), gpu[0], gpu[2], tb, c["seqlens"].cuda(), scale, out_scale)
    step = DecodeStep(*args, latent_scale=gpu[1], w_uv=w_uv)
    y = step()
    torch.cuda.synchronize()
    assert torch.equal(step.out, got)
    assert torch.equal(y, b.mlra_up_proj(got, w_uv))
    plain = DecodeStep(*args, latent_scale=gpu[1])
    assert torch.equal(plain(), got)


# ----------------------------------------------------------------- refusals
@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    c = _gpu(_decode_case(34, 4, 2, 64, 32, 16, [30]))
    for change in (dict(latent_cache=_bytes(c["latent_cache"])), dict(latent_scale=c["latent_scale"].half()), dict(latent_scale=c["latent_scale"][:, :, :1]),
                   dict(seqlens=c["seqlens"].cpu()), dict(q_rope=c["q_rope"].float()), dict(block_table=c["block_table"].long()),
                   dict(workspace=torch.zeros(1 << 24, dtype=torch.uint8))):
        with pytest.raises((TypeError, ValueError)):
            b.mlra_decode_fp8(**{**c, **change})
    with pytest.raises((TypeError, ValueError)):
        DecodeStep(c["q_lat"], c["q_rope"], c["latent_cache"], c["rope_cache"], c["block_table"], c["seqlens"], 0.1, 0.5)


def test_binding_refuses_host_tensors():
    c = _decode_case(35, 4, 2, 64, 32, 16, [30])
    with pytest.raises(ValueError, match="CUDA"):
        b.mlra_decode_fp8(**c)
    with pytest.raises(ValueError, match="CUDA"):
        b.mlra_append_fp8(torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 32, dtype=torch.bfloat16), torch.tensor([0, 1], dtype=torch.int32),
                          c["seqlens"], c["block_table"], c["latent_cache"], c["latent_scale"], c["rope_cache"])


def _dims(kw):
    base = dict(batch=2, heads=16, branches=4, d_c=128, d_r=64, page_size=64, max_pages_per_seq=8, num_pages=32)
    return b.mlra_dims(*[kw.get(k, base[k]) for k, _ in b.mlra_dims._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), b.MLRA_ERR_INVALID_ARG), (dict(d_c=96), b.MLRA_ERR_UNSUPPORTED), (dict(d_c=32), b.MLRA_ERR_UNSUPPORTED),
    (dict(d_c=1024), b.MLRA_ERR_UNSUPPORTED), (dict(branches=9), b.MLRA_ERR_UNSUPPORTED), (dict(d_r=33), b.MLRA_ERR_UNSUPPORTED),
    (dict(d_r=66), b.MLRA_ERR_UNSUPPORTED), (dict(page_size=8), b.MLRA_ERR_UNSUPPORTED), (dict(tokens=-1), b.MLRA_ERR_INVALID_ARG),
    *[(dict(ptr=i), b.MLRA_ERR_INVALID_ARG) for i in range(8)], (dict(base=1.0), b.MLRA_ERR_INVALID_ARG), (dict(base=float("nan")), b.MLRA_ERR_INVALID_ARG),
    (dict(status=3), b.MLRA_ERR_INVALID_ARG), (dict(num_pages=2 ** 30), b.MLRA_ERR_INVALID_ARG),
])
def test_append_refuses_before_any_cuda_call(kw, code):
    ok = 1 << 20
    p = [ok + 8 if kw.get("ptr") == i else ok for i in range(8)]
    st = b.library().mlra_append_fp8(ctypes.byref(_dims(kw)), kw.get("tokens", 4), *p[:5], kw.get("base", 10000.0), *p[5:], ok + kw.get("status", 0), None)
    assert st == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), b.MLRA_ERR_INVALID_ARG), (dict(heads=129), b.MLRA_ERR_UNSUPPORTED), (dict(heads=128, batch=8192), b.MLRA_ERR_UNSUPPORTED),
    (dict(d_c=96), b.MLRA_ERR_UNSUPPORTED), (dict(branches=8), b.MLRA_ERR_UNSUPPORTED), (dict(d_r=48), b.MLRA_ERR_UNSUPPORTED),
    (dict(page_size=8), b.MLRA_ERR_UNSUPPORTED), (dict(page_size=96), b.MLRA_ERR_UNSUPPORTED), *[(dict(ptr=i), b.MLRA_ERR_INVALID_ARG) for i in range(8)],
    (dict(scale=float("nan")), b.MLRA_ERR_INVALID_ARG), (dict(ws=0), b.MLRA_ERR_WORKSPACE), (dict(ws=(1 << 20) + 16), b.MLRA_ERR_WORKSPACE),
])
def test_decode_refuses_before_any_cuda_call(kw, code):
    ok = 1 << 20
    p = [ok + 8 if kw.get("ptr") == i else ok for i in range(8)]
    st = b.library().mlra_decode_fp8(ctypes.byref(_dims(kw)), *p[:7], kw.get("scale", 0.1), 0.5, p[7], kw.get("ws", ok) or None, 1 << 30, None)
    assert st == code
