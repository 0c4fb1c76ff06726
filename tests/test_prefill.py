"""Prompt attention (mlra_prefill) against its formula in 64 bits: packed
ragged sequences, chunks behind cached tokens, every supported shape, poisoned
slots behind the sequences, refusals and device-detected errors, streams,
graphs, and the path prompt -> pre-step -> prompt attention -> decode.

The probabilities enter the output product as bf16 (half a step: 2^-8)."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from branch_latent_kv_b200 import binding as b
from tests import latent_ref as ref

R_PROB = 2.0 ** -8
SHAPES = [(2, 64), (4, 64), (1, 128), (2, 128), (4, 128), (1, 256), (2, 256), (1, 512)]


def _case(seed, H, B, d_c, d_r, P, new, past, std=2.0, poison=True):
    """CPU tensors of one packed call; scores of standard deviation `std`."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    lens = [q + p for q, p in zip(new, past)]
    table, pages = ref.paged(lens, P, rng)
    scale = (d_c + d_r) ** -0.5
    gain = std / (scale * math.sqrt(1.0 / d_c + 1.0 / d_r))

    def normal(*shape, f):
        return (torch.randn(*shape, generator=g) * f).to(torch.bfloat16)
    fill = float("nan") if poison else 0.0
    lat = torch.full((pages, P, B, d_c), fill, dtype=torch.bfloat16)
    rope = torch.full((pages, P, d_r), fill, dtype=torch.bfloat16)
    for n, L in enumerate(lens):
        ref.put(lat, table, n, normal(L, B, d_c, f=d_c ** -0.5))
        ref.put(rope, table, n, normal(L, d_r, f=d_r ** -0.5))
    T = sum(new)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return dict(q_lat=normal(T, H, B, d_c, f=gain * d_c ** -0.5), q_rope=normal(T, H, d_r, f=gain * d_r ** -0.5),
                latent_cache=lat, rope_cache=rope, block_table=table, seqlens=torch.tensor(lens, dtype=torch.int32),
                cu_seqlens=cu, scale=scale, out_scale=B ** -0.5)


def _gpu(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def _expect(c, only=None):
    """(out, tolerance) of every row, sequence by sequence."""
    out = torch.zeros(c["q_lat"].shape, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for n, L in enumerate(c["seqlens"].tolist()):
        lo, hi = int(c["cu_seqlens"][n]), int(c["cu_seqlens"][n + 1])
        if hi == lo or (only is not None and n not in only):
            continue
        out[lo:hi], tol[lo:hi] = ref.attend(c["q_lat"][lo:hi], c["q_rope"][lo:hi], ref.rows(c["latent_cache"], c["block_table"], n, L),
                                            ref.rows(c["rope_cache"], c["block_table"], n, L), c["scale"], c["out_scale"], L - (hi - lo), R_PROB)
    return out, tol


def _check(c, what="", **kw):
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = b.mlra_prefill(**_gpu(c), device_status=status, **kw)
    assert int(status.item()) == 0
    ref.within(got, *_expect(c), what)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c", SHAPES)
@pytest.mark.parametrize("d_r,page", [(32, 16), (64, 64), (64, 128)])
def test_every_shape_on_ragged_prompts(branches, d_c, d_r, page):
    c = _case(1, 12, branches, d_c, d_r, page, [1, 130, 0, 33, 257], [0, 0, 5, 100, 3])
    _check(c, f"B={branches} d_c={d_c} d_r={d_r} P={page}")


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 3, 16, 17, 40, 128])
def test_head_counts(heads):
    c = _case(2, heads, 4, 128, 64, 32, [70, 1, 19], [0, 200, 61])
    _check(c, f"H={heads}")


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c,heads", [(4, 128, 16), (2, 256, 16), (1, 512, 5), (4, 64, 16)])
@pytest.mark.parametrize("new,past", [([1], [0]), ([2], [0]), ([127], [0]), ([128], [0]), ([129], [1]), ([600], [0]),
                                      ([1], [1000]), ([5], [1019]), ([64, 64], [64, 0])])
def test_lengths_around_the_tiles(new, past, branches, d_c, heads):
    c = _case(3, heads, branches, d_c, 64, 64, new, past)
    _check(c, f"new={new} past={past}")


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c", SHAPES)
@pytest.mark.parametrize("heads,new,past", [(16, [3], [5000]), (1, [300], [3000]), (5, [1, 2], [2100, 40]), (16, [40, 0, 7], [1500, 9, 2600])])
def test_few_rows_over_long_contexts(branches, d_c, heads, new, past):
    """Row blocks that leave most SMs idle: their tokens are split over
    clusters; parts without tiles, and parts that some rows see nothing of."""
    c = _case(17, heads, branches, d_c, 64, 64, new, past)
    _check(c, f"H={heads} new={new} past={past}")


@pytest.mark.gpu
def test_chunks_split_for_the_last_wave():
    """More row blocks than SMs, contexts several times the chunks: two parts
    each; against the same call's rows one sequence at a time."""
    c = _case(18, 16, 4, 64, 32, 64, [160] * 4, [900, 700, 800, 1100], poison=False)
    got = _check(c)
    for n in range(4):
        lo, hi = int(c["cu_seqlens"][n]), int(c["cu_seqlens"][n + 1])
        d = {**c, "q_lat": c["q_lat"][lo:hi].contiguous(), "q_rope": c["q_rope"][lo:hi].contiguous(), "block_table": c["block_table"][n:n + 1].contiguous(),
             "seqlens": c["seqlens"][n:n + 1].clone(), "cu_seqlens": torch.tensor([0, hi - lo], dtype=torch.int32)}
        ref.within(b.mlra_prefill(**_gpu(d)), got[lo:hi].double().cpu(), 2.0 ** -6 * got[lo:hi].double().abs().cpu() + 2.0 ** -8 * float(got.abs().max()))


@pytest.mark.gpu
def test_bad_page_behind_a_split():
    """A page outside the pool in one part's tokens empties every part's rows."""
    c = _case(19, 8, 4, 128, 64, 64, [4, 3], [4000, 20])
    out, tol = _expect(c)
    c["block_table"][0, 10] = -7
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = b.mlra_prefill(**_gpu(c), device_status=status)
    assert int(status.item()) == b.MLRA_ERR_DEVICE_BAD_INDEX
    assert bool((got[:4] == 0).all())
    ref.within(got[4:], out[4:], tol[4:])


@pytest.mark.gpu
def test_zero_and_negative_scales():
    for scale in (0.0, -0.05):
        c = _case(20, 8, 2, 128, 64, 64, [130], [70])
        c["scale"] = scale
        _check(c, f"scale {scale}")


@pytest.mark.gpu
def test_long_prompt_of_the_benchmark_shape():
    c = _case(4, 16, 4, 128, 64, 64, [1200], [300])
    _check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("d_c,branches", [(128, 4), (256, 2), (512, 1)])
def test_large_scores_rescale(d_c, branches):
    """Scores that keep growing along the sequence: every tile raises the
    running maximum far past what the lazy rescale lets stand."""
    c = _case(5, 8, branches, d_c, 64, 64, [300], [300], std=1.0)
    for n in range(1):
        L = int(c["seqlens"][n])
        ramp = torch.linspace(0.5, 12.0, L)[:, None]
        k = c["q_rope"][:, 0].float().mean(0)
        ref.put(c["rope_cache"], c["block_table"], n, (ramp * (k / k.norm()) * 3).to(torch.bfloat16))
    c["q_rope"] = (c["q_rope"][:, :1].float().mean(0, keepdim=True).expand_as(c["q_rope"]) * 30).to(torch.bfloat16).contiguous()
    _check(c)


@pytest.mark.gpu
def test_first_token_attends_to_itself_only():
    """A prompt's first row is its own latent times out_scale, bit for bit."""
    c = _case(6, 16, 4, 128, 64, 64, [200, 3], [0, 0])
    got = b.mlra_prefill(**_gpu(c)).cpu()
    for n in range(2):
        want = (ref.rows(c["latent_cache"], c["block_table"], n, 1)[0].float() * c["out_scale"]).to(torch.bfloat16)
        row = got[int(c["cu_seqlens"][n])]
        assert torch.equal(row, want[None].expand_as(row))


@pytest.mark.gpu
def test_page_order_and_company_do_not_change_a_sequence():
    """The same sequence alone, in other pages and packed behind others gives
    the same bits when it starts at the same row of the tile walk."""
    c = _case(7, 16, 4, 128, 64, 64, [300], [50])
    d = {**c, "latent_cache": c["latent_cache"].clone(), "rope_cache": c["rope_cache"].clone(), "block_table": c["block_table"].clone()}
    used = c["block_table"][0].clone()
    d["block_table"][0] = used.flip(0)
    d["latent_cache"][used.flip(0).long()] = c["latent_cache"][used.long()]
    d["rope_cache"][used.flip(0).long()] = c["rope_cache"][used.long()]
    one, two = b.mlra_prefill(**_gpu(c)), b.mlra_prefill(**_gpu(d))
    assert torch.equal(one, two)
    assert torch.equal(one, b.mlra_prefill(**_gpu(c)))
    lead = _case(8, 16, 4, 128, 64, 64, [40], [0])
    P = 64
    table = torch.full((2, c["block_table"].shape[1]), -1, dtype=torch.int32)
    table[0, :1] = lead["block_table"][0, :1] + c["latent_cache"].shape[0]
    table[1] = c["block_table"][0]
    both = dict(q_lat=torch.cat([lead["q_lat"], c["q_lat"]]), q_rope=torch.cat([lead["q_rope"], c["q_rope"]]),
                latent_cache=torch.cat([c["latent_cache"], lead["latent_cache"]]), rope_cache=torch.cat([c["rope_cache"], lead["rope_cache"]]),
                block_table=table, seqlens=torch.tensor([40, 350], dtype=torch.int32), cu_seqlens=torch.tensor([0, 40, 340], dtype=torch.int32),
                scale=c["scale"], out_scale=c["out_scale"])
    assert P == c["latent_cache"].shape[1]
    got = b.mlra_prefill(**_gpu(both))
    assert torch.equal(got[40:], one)


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c", [(4, 128), (2, 256), (1, 512)])
def test_a_query_that_is_not_finite_stays_in_its_row(branches, d_c):
    c = _case(24, 8, branches, d_c, 64, 64, [70, 33], [100, 0])
    out, tol = _expect(c)
    last = branches - 1
    c["q_lat"][5, 3, last, 7] = float("nan")
    c["q_lat"][69, 0, 0, d_c - 1] = float("inf")
    c["q_rope"][71, 7, 1] = float("nan")
    got = b.mlra_prefill(**_gpu(c)).double().cpu()
    lost = torch.zeros(got.shape[:3], dtype=torch.bool)
    lost[5, 3, last] = lost[69, 0, 0] = True
    lost[71, 7] = True
    assert bool(got[lost].isnan().all())
    ref.within(got[~lost], out[~lost], tol[~lost])


@pytest.mark.gpu
def test_rows_of_no_sequence_stay():
    c = _case(9, 16, 2, 128, 64, 64, [50, 20], [0, 0])
    T = 70
    pad = {**c, "q_lat": torch.cat([c["q_lat"][:7], c["q_lat"], c["q_lat"][:9]]), "q_rope": torch.cat([c["q_rope"][:7], c["q_rope"], c["q_rope"][:9]]),
           "cu_seqlens": c["cu_seqlens"] + 7}
    out = torch.full_like(pad["q_lat"], 7.0).cuda()
    got = b.mlra_prefill(**_gpu(pad), out=out)
    assert got is out and bool((out[:7] == 7).all()) and bool((out[7 + T:] == 7).all())
    ref.within(out[7:7 + T], *_expect(c))


@pytest.mark.gpu
def test_bad_sequences_are_reported_and_zeroed():
    c = _case(10, 16, 4, 128, 64, 64, [40, 100, 30], [0, 300, 10])
    out, tol = _expect(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    too_long = 64 * c["block_table"].shape[1] + 1
    for lens, page, code in [((40, 0, 40), None, b.MLRA_ERR_DEVICE_BAD_SEQLEN), ((40, 99, 40), None, b.MLRA_ERR_DEVICE_BAD_SEQLEN),
                             ((40, too_long, 40), None, b.MLRA_ERR_DEVICE_BAD_SEQLEN), ((40, -5, 40), None, b.MLRA_ERR_DEVICE_BAD_SEQLEN),
                             ((40, 400, 40), -1, b.MLRA_ERR_DEVICE_BAD_INDEX), ((40, 400, 40), c["latent_cache"].shape[0], b.MLRA_ERR_DEVICE_BAD_INDEX)]:
        d = {**c, "seqlens": torch.tensor(lens, dtype=torch.int32), "block_table": c["block_table"].clone()}
        if page is not None:
            d["block_table"][1, 3] = page
        got = b.mlra_prefill(**_gpu(d), out=torch.full_like(c["q_lat"], 5.0).cuda(), device_status=status)
        assert int(status.item()) == code, (lens, page)
        assert bool((got[40:140] == 0).all())
        for lo, hi in ((0, 40), (140, 170)):
            ref.within(got[lo:hi], out[lo:hi], tol[lo:hi])
    for cu in ([0, 40, 20, 170], [0, 40, 140, 171], [-1, 40, 140, 170]):
        d = {**c, "cu_seqlens": torch.tensor(cu, dtype=torch.int32)}
        b.mlra_prefill(**_gpu(d), device_status=status)
        assert int(status.item()) == b.MLRA_ERR_DEVICE_BAD_SEQLEN, cu
    b.mlra_prefill(**_gpu(c), device_status=status)
    assert int(status.item()) == 0  # each call reports its own


@pytest.mark.gpu
@pytest.mark.parametrize("branches,d_c,heads", [(4, 64, 16), (1, 128, 40), (4, 128, 16), (2, 256, 16), (1, 512, 16)])
def test_more_row_blocks_than_the_gpu_holds(branches, d_c, heads):
    """Several row blocks one after the other on each SM, of any length, empty
    sequences and bad ones among them."""
    rng = np.random.default_rng(40)
    new = [int(q) for q in rng.integers(0, 41, 150)] + [500, 1, 333]
    past = [int(p) for p in rng.integers(1, 260, len(new))]
    c = _case(41, heads, branches, d_c, 64, 32, new, past)
    short, torn = (n for n in (20, 90) if new[n] > 0)
    want, tol = _expect(c)
    for n in (short, torn):
        lo, hi = int(c["cu_seqlens"][n]), int(c["cu_seqlens"][n + 1])
        want[lo:hi], tol[lo:hi] = 0, 0
    c["seqlens"][short] = new[short] - 1
    c["block_table"][torn, 0] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = b.mlra_prefill(**_gpu(c), out=torch.full_like(c["q_lat"], 3.0).cuda(), device_status=status)
    assert int(status.item()) in (b.MLRA_ERR_DEVICE_BAD_SEQLEN, b.MLRA_ERR_DEVICE_BAD_INDEX)
    ref.within(got, want, tol)
    again = b.mlra_prefill(**_gpu(c))
    assert torch.equal(again, got)


@pytest.mark.gpu
def test_output_of_a_call_on_another_stream():
    """The output's memory is not what the current stream still works on."""
    c = _gpu(_case(44, 16, 4, 128, 64, 64, [300], [0]))
    want = b.mlra_prefill(**c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    held = torch.empty_like(want)
    keep = torch.zeros_like(want)
    place = held.data_ptr()
    torch.cuda._sleep(20_000_000)
    held.fill_(5.0)  # queued behind the pause, on memory that is free for this stream now
    keep.copy_(held)
    del held
    got = b.mlra_prefill(**c, stream=side)
    assert got.data_ptr() != place
    side.synchronize()
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((keep == 5).all())


@pytest.mark.gpu
def test_two_calls_at_once():
    """Calls on two streams that share the GPU's SMs: the results of each alone."""
    one = _gpu(_case(42, 16, 4, 128, 64, 64, [700, 300], [0, 200]))
    two = _gpu(_case(43, 16, 4, 64, 32, 32, [600, 90, 400], [10, 0, 77]))
    want = [b.mlra_prefill(**one), b.mlra_prefill(**two)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(w) for _ in range(4)] for w in want]
    torch.cuda.synchronize()
    for i in range(4):
        for c, s, o in zip((one, two), streams, outs):
            b.mlra_prefill(**c, out=o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


FIRST_CALL = """
import torch
from branch_latent_kv_b200 import binding as b
torch.manual_seed(0)
new = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
q, qr, lat, rope = new(70, 8, 2, 128), new(70, 8, 64), new(3, 64, 2, 128), new(3, 64, 64)
lat8, sig = torch.zeros(3, 64, 2, 128, device="cuda", dtype=torch.float8_e4m3fn), torch.ones(3, 4, 2, device="cuda")
table, lens, cu = i32(2, 0).view(1, 2), i32(70), i32(0, 70)
graph = torch.cuda.CUDAGraph()
def calls():
    x = b.mlra_prefill(q, qr, lat, rope, table, lens, cu, 0.1, 1.0)
    b.mlra_append_fp8(lat[:1].view(64, 2, 128)[:6], rope[0, :6], i6, lens, table, lat8, sig, rope8)
    return x, b.mlra_decode_fp8(q[:1], qr[:1], lat8, sig, rope8, table, lens, 0.1, 1.0)
i6, rope8 = i32(0, 6), torch.zeros(3, 64, 64, device="cuda", dtype=torch.bfloat16)
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
want = calls()
assert all(torch.equal(x, y) for x, y in zip(got, want)) and bool(got[0].isfinite().all())
print("the same")
"""


@pytest.mark.gpu
def test_first_calls_of_a_process_are_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "the same" in run.stdout, run.stderr[-2000:]


@pytest.mark.gpu
def test_nothing_to_do():
    c = _gpu(_case(11, 16, 4, 128, 64, 64, [4], [0]))
    c["q_lat"], c["q_rope"] = c["q_lat"][:0], c["q_rope"][:0]
    c["cu_seqlens"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert b.mlra_prefill(**c).shape == (0, 16, 4, 128)


@pytest.mark.gpu
def test_other_stream_and_graph_replay():
    c = _case(12, 16, 4, 128, 64, 64, [90, 200], [0, 17])
    g = _gpu(c)
    want = b.mlra_prefill(**g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        on_side = b.mlra_prefill(**g)
    by_arg = b.mlra_prefill(**g, out=torch.empty_like(want), stream=side)
    side.synchronize()
    assert torch.equal(on_side, want) and torch.equal(by_arg, want)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.mlra_prefill(**g, device_status=status)
    for _ in range(3):
        out.zero_()
        graph.replay()
    assert torch.equal(out, want) and int(status.item()) == 0
    # new lengths in the same buffers: the captured call follows them
    g["cu_seqlens"].copy_(torch.tensor([0, 1, 290], dtype=torch.int32))
    g["seqlens"].copy_(torch.tensor([90, 217], dtype=torch.int32))
    graph.replay()
    assert int(status.item()) == b.MLRA_ERR_DEVICE_BAD_SEQLEN  # 289 new tokens of 217
    assert bool((out[1:] == 0).all()) and bool((out[0] != 0).any())


@pytest.mark.gpu
def test_pool_past_32_bit_offsets():
    """Pages at the far end of a pool of more than 2^32 values."""
    c = _case(13, 8, 4, 128, 64, 64, [70], [30], poison=False)
    far = (1 << 32) // (64 * 512) + 40  # pages; the pool holds 2^32 + values
    lat = torch.empty(far, 64, 4, 128, dtype=torch.bfloat16, device="cuda")
    rope = torch.empty(far, 64, 64, dtype=torch.bfloat16, device="cuda")
    k = c["latent_cache"].shape[0]
    lat[-k:], rope[-k:] = c["latent_cache"].cuda(), c["rope_cache"].cuda()
    g = _gpu(c)
    g.update(latent_cache=lat, rope_cache=rope, block_table=torch.where(g["block_table"] >= 0, g["block_table"] + (far - k), -1).to(torch.int32))
    ref.within(b.mlra_prefill(**g), *_expect(c))


@pytest.mark.gpu
def test_prompt_then_decode():
    """A served sequence: its prompt through the pre-step and the prompt
    attention, the next token through the pre-step and mlra_decode.  The
    prompt's last row also is what mlra_decode gives for that token."""
    H, B, d_c, d_r, d_h, P, L = 16, 4, 128, 64, 128, 64, 150
    g = torch.Generator().manual_seed(14)

    def normal(*shape, fan):
        return (torch.randn(*shape, generator=g) / math.sqrt(fan)).to(torch.bfloat16).cuda()
    w_uk = normal(B, H, d_h, d_c, fan=d_h)
    q_c, q_r, c_new, kr = normal(L + 1, H, d_h, fan=d_h), normal(L + 1, H, d_r, fan=1), normal(L + 1, B, d_c, fan=d_c), normal(L + 1, d_r, fan=1)
    lat, rope = torch.zeros(4, P, B, d_c, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, P, d_r, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    # the prompt's tokens are a batch of the pre-step, each at its own position
    q_lat, q_rope = b.mlra_prepare(q_c[:L].contiguous(), q_r[:L].contiguous(), w_uk, c_new[:L].contiguous(), kr[:L].contiguous(),
                                   torch.arange(1, L + 1, dtype=torch.int32, device="cuda"), table.expand(L, 3).contiguous(), lat, rope)
    scale, out_scale = (d_c + d_r) ** -0.5, B ** -0.5
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    out = b.mlra_prefill(q_lat, q_rope, lat, rope, table, lens, cu, scale, out_scale)
    want, tol = ref.attend(q_lat.cpu(), q_rope.cpu(), ref.rows(lat.cpu(), table.cpu(), 0, L), ref.rows(rope.cpu(), table.cpu(), 0, L),
                           scale, out_scale, 0, R_PROB)
    ref.within(out, want, tol)
    last = b.mlra_decode(q_lat[-1:].contiguous(), q_rope[-1:].contiguous(), lat, rope, table, lens, scale, out_scale)
    ref.within(last, want[-1:], tol[-1:], "the prompt's last token by mlra_decode")
    lens2 = torch.tensor([L + 1], dtype=torch.int32, device="cuda")
    q2, qr2 = b.mlra_prepare(q_c[L:].contiguous(), q_r[L:].contiguous(), w_uk, c_new[L:].contiguous(), kr[L:].contiguous(), lens2, table, lat, rope)
    nxt = b.mlra_decode(q2, qr2, lat, rope, table, lens2, scale, out_scale)
    by_prompt = b.mlra_prefill(q2, qr2, lat, rope, table, lens2, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), scale, out_scale)
    w2, t2 = ref.attend(q2.cpu(), qr2.cpu(), ref.rows(lat.cpu(), table.cpu(), 0, L + 1), ref.rows(rope.cpu(), table.cpu(), 0, L + 1),
                        scale, out_scale, L, R_PROB)
    ref.within(nxt, w2, t2, "decode after the prompt")
    ref.within(by_prompt, w2, t2, "one token by mlra_prefill")


# ----------------------------------------------------------------- on the host
def test_binding_refuses_wrong_arguments():
    c = _case(15, 4, 2, 64, 32, 16, [3], [2])
    with pytest.raises(ValueError, match="CUDA"):
        b.mlra_prefill(**c)
    with pytest.raises(TypeError):
        b.mlra_prefill(**{**c, "q_lat": 3})
    with pytest.raises(ValueError, match="dimensions"):
        b.mlra_prefill(**{**c, "q_lat": c["q_lat"][0]})


@pytest.mark.gpu
@pytest.mark.parametrize("change", [dict(q_lat=torch.float16), dict(seqlens=torch.int64), dict(cu_seqlens="short"), dict(q_rope="strided"),
                                    dict(rope_cache="cpu"), dict(block_table="long")])
def test_binding_refuses_wrong_tensors(change):
    c = _gpu(_case(16, 4, 2, 64, 32, 16, [3], [2]))
    (name, how), = change.items()
    if isinstance(how, torch.dtype):
        c[name] = c[name].to(how)
    elif how == "short":
        c[name] = c[name][:1]
    elif how == "long":
        c[name] = torch.cat([c[name], c[name]])
    elif how == "cpu":
        c[name] = c[name].cpu()
    else:
        c[name] = c[name].transpose(0, 1)
    with pytest.raises((TypeError, ValueError)):
        b.mlra_prefill(**c)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), b.MLRA_ERR_INVALID_ARG), (dict(heads=129), b.MLRA_ERR_UNSUPPORTED), (dict(d_c=96), b.MLRA_ERR_UNSUPPORTED),
    (dict(branches=3), b.MLRA_ERR_UNSUPPORTED), (dict(d_r=48), b.MLRA_ERR_UNSUPPORTED), (dict(page_size=8), b.MLRA_ERR_UNSUPPORTED),
    (dict(page_size=48), b.MLRA_ERR_UNSUPPORTED), (dict(tokens=-1), b.MLRA_ERR_INVALID_ARG), (dict(tokens=2 ** 27), b.MLRA_ERR_INVALID_ARG),
    (dict(ptr=0), b.MLRA_ERR_INVALID_ARG), (dict(ptr=6), b.MLRA_ERR_INVALID_ARG), (dict(scale=float("nan")), b.MLRA_ERR_INVALID_ARG),
    (dict(status=2), b.MLRA_ERR_INVALID_ARG), (dict(out=8), b.MLRA_ERR_INVALID_ARG),
])
def test_entry_refuses_before_any_cuda_call(kw, code):
    import ctypes
    base = dict(batch=2, heads=16, branches=4, d_c=128, d_r=64, page_size=64, max_pages_per_seq=8, num_pages=32)
    dims = b.mlra_dims(*[kw.get(k, base[k]) for k, _ in b.mlra_dims._fields_])
    ok = 1 << 20  # never dereferenced
    p = [ok + 4 if kw.get("ptr") == i else ok for i in range(7)]
    st = b.library().mlra_prefill(ctypes.byref(dims), kw.get("tokens", 8), *p, kw.get("scale", 0.1), 0.5, ok + kw.get("out", 0),
                                  ok + kw.get("status", 0), None)
    assert st == code
