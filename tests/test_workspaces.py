"""Default workspaces: decode calls of both caches on different streams, in
captured graphs and of growing sizes share none."""
import pytest
import torch

from branch_latent_kv_b200 import binding as b
from tests import latent_ref as ref
from tests.test_fp8_cache import _decode_case, _gpu


def _case(seed, lens, heads=16):
    """One step over both caches: (arguments of mlra_decode, of mlra_decode_fp8)."""
    c = _decode_case(seed, heads, 4, 128, 64, 64, lens, poison=False)
    lat = ref.values(c["latent_cache"], c["latent_scale"]).to(torch.bfloat16)
    g8 = _gpu(c)
    g16 = {k: v for k, v in g8.items() if k != "latent_scale"}
    return {**g16, "latent_cache": lat.cuda()}, g8


def _dims(g):
    return b.decode_dims(g["q_lat"], g["q_rope"], g["latent_cache"], g["block_table"])


@pytest.mark.gpu
def test_each_stream_and_each_capture_has_its_own():
    g16, _ = _case(50, [300, 20])
    dims, dev = _dims(g16), g16["q_lat"].device
    seen = [b.workspace_for(dims, dev)]
    side = torch.cuda.Stream()
    seen.append(b.workspace_for(dims, dev, side))
    with torch.cuda.stream(side):
        assert b.workspace_for(dims, dev).data_ptr() == seen[1].data_ptr()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            seen.append(b.workspace_for(dims, dev))
            again = b.workspace_for(dims, dev)  # one for the whole capture
            pad = torch.zeros(1, device=dev)    # (a graph of something)
        assert again.data_ptr() == seen[-1].data_ptr() and pad.numel() == 1
    assert b.workspace_for(dims, dev).data_ptr() == seen[0].data_ptr()
    spans = sorted((w.data_ptr(), w.data_ptr() + w.numel()) for w in seen)
    assert all(x[1] <= y[0] for x, y in zip(spans, spans[1:])), spans


@pytest.mark.gpu
def test_both_decodes_at_once_on_streams_and_in_graphs():
    """mlra_decode on a side stream, replays of a captured one and of a
    captured mlra_decode_fp8, and mlra_decode_fp8 on the default stream, all
    at once and without a workspace, with larger calls in between."""
    g16, g8 = _case(51, [4000, 900, 17, 2500])
    h16, h8 = _case(52, [100, 6000, 3000, 1])
    big16, big8 = _case(53, [700, 20, 1, 3000, 64, 128] * 4, heads=40)
    torch.cuda.synchronize()
    b._ws_cache.clear()
    graphs, outs = [], []
    for call, args in ((b.mlra_decode, g16), (b.mlra_decode_fp8, h8)):  # the first calls that need a workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(**args))
        graphs.append(graph)
    want16, want8 = b.mlra_decode(**h16), b.mlra_decode_fp8(**g8)
    torch.cuda.synchronize()
    s1, s2, s3 = (torch.cuda.Stream() for _ in range(3))
    got16, got8, large = [], [], []
    for i in range(6):
        with torch.cuda.stream(s1):
            got16.append(b.mlra_decode(**h16))
            if i == 2:
                large.append(b.mlra_decode(**big16))
        with torch.cuda.stream(s2):
            graphs[0].replay()
        with torch.cuda.stream(s3):
            graphs[1].replay()
        got8.append(b.mlra_decode_fp8(**g8))
        if i == 3:
            large.append(b.mlra_decode_fp8(**big8))
    torch.cuda.synchronize()
    assert b.mlra_read_device_error() == b.MLRA_OK
    assert all(torch.equal(x, want16) for x in got16) and all(torch.equal(x, want8) for x in got8)
    assert torch.equal(outs[0], b.mlra_decode(**g16)) and torch.equal(outs[1], b.mlra_decode_fp8(**h8))
    assert torch.equal(large[0], b.mlra_decode(**big16)) and torch.equal(large[1], b.mlra_decode_fp8(**big8))


@pytest.mark.gpu
def test_errors_of_other_streams_are_found():
    g16, g8 = _case(54, [300, 900])
    bad = torch.tensor([300, 0], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    for call, args in ((b.mlra_decode, g16), (b.mlra_decode_fp8, g8)):
        call(**{**args, "seqlens": bad}, stream=side, out=torch.empty_like(g16["q_lat"]))
        side.synchronize()
        assert b.mlra_read_device_error() == b.MLRA_ERR_DEVICE_BAD_SEQLEN
        assert b.mlra_read_device_error() == b.MLRA_OK
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(**{**args, "seqlens": bad})
        graph.replay()
        assert b.mlra_read_device_error() == b.MLRA_ERR_DEVICE_BAD_SEQLEN
        assert b.mlra_read_device_error() == b.MLRA_OK


@pytest.mark.gpu
def test_an_output_made_for_another_stream_is_not_the_current_ones_memory():
    """A call on a stream of the caller's must not write memory that was given
    back on the current stream, where work that uses it may still be queued."""
    N, H, B, d_c, d_r, d_h = 3, 16, 4, 128, 64, 128
    g16, _ = _case(55, [300, 20, 4])
    w_uv = torch.randn(B, d_c, H * d_h, device="cuda").to(torch.bfloat16)
    w_uk = torch.randn(B, H, d_h, d_c, device="cuda").to(torch.bfloat16)
    new = [torch.randn(*s, device="cuda").to(torch.bfloat16) for s in ((N, H, d_h), (N, H, d_r), (N, B, d_c), (N, d_r))]
    out = b.mlra_decode(**g16)
    y = b.mlra_up_proj(out, w_uv)
    side = torch.cuda.Stream()
    for call, shapes in (
            (lambda: b.mlra_decode(**g16, stream=side), [out.shape]),
            (lambda: b.mlra_decode_up_proj(**g16, w_uv=w_uv, stream=side), [out.shape, y.shape]),
            (lambda: b.mlra_up_proj(out, w_uv, stream=side), [y.shape]),
            (lambda: b.mlra_prepare(new[0], new[1], w_uk, new[2], new[3], g16["seqlens"], g16["block_table"], g16["latent_cache"],
                                    g16["rope_cache"], stream=side), [out.shape, (N, H, d_r)])):
        torch.cuda.synchronize()
        freed = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in shapes]
        held = {t.data_ptr() for t in freed}
        del freed
        got = call()
        side.synchronize()
        got = got if isinstance(got, tuple) else (got,)
        assert [tuple(t.shape) for t in got] == [tuple(s) for s in shapes]
        assert not held & {t.data_ptr() for t in got}
