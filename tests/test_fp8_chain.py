"""Appends and decode steps launched one behind the other, in a stream and in
a captured graph, read what the call before them wrote: the same bits as with
the device waited for after each call."""
import pytest
import torch

from branch_latent_kv_b200 import binding as b


@pytest.mark.gpu
@pytest.mark.parametrize("N,B,d_c,P,past", [(16, 4, 128, 64, 0), (64, 4, 128, 64, 400), (32, 2, 64, 16, 3), (24, 4, 128, 128, 2000)])
def test_steps_behind_one_another(N, B, d_c, P, past):
    """Tokens of growing size, by another factor in each branch: almost every
    append raises scales, whose neighbours in memory other warps raise."""
    H, d_r, steps = 16, 64, 24
    g = torch.Generator(device="cuda").manual_seed(80)

    def normal(*shape, f=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * f).to(torch.bfloat16)
    per = -(-(past + steps) // P)
    table = torch.randperm(N * per, generator=g, device="cuda").view(N, per).int()
    start = (torch.zeros(N * per, P, B, d_c, dtype=torch.uint8, device="cuda"), torch.full((N * per, P // 16, B), 2.0 ** -12, device="cuda"),
             torch.zeros(N * per, P, d_r, dtype=torch.bfloat16, device="cuda"))
    pool = tuple(t.clone() for t in start)
    cache = (pool[0].view(torch.float8_e4m3fn), pool[1], pool[2])
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    lens = [torch.full((N,), past + i + 1, dtype=torch.int32, device="cuda") for i in range(steps)]
    c_new = [(normal(N, B, d_c) * torch.exp2(i % 16 / 1.5 + 3 * torch.rand(N, B, 1, generator=g, device="cuda"))).to(torch.bfloat16) for i in range(steps)]
    kr_new = [normal(N, d_r) for _ in range(steps)]
    q, qr = normal(N, H, B, d_c, f=0.05), normal(N, H, d_r, f=0.1)
    outs = [torch.empty_like(q) for _ in range(steps)]

    def run(wait):
        for i in range(steps):
            b.mlra_append_fp8(c_new[i], kr_new[i], cu, lens[i], table, *cache)
            wait()
            b.mlra_decode_fp8(q, qr, *cache, table, lens[i], 0.1, 0.5, out=outs[i])
            wait()

    def again():
        for t, s in zip(pool, start):
            t.copy_(s)
    run(torch.cuda.synchronize)
    want, state = [o.clone() for o in outs], [t.clone() for t in pool]
    assert all(bool(torch.isfinite(o).all()) for o in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lambda: None)
    for replay in [graph.replay] * 5 + [lambda: run(lambda: None)] * 5:
        again()
        replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert all(torch.equal(t, s) for t, s in zip(pool, state))
    assert b.mlra_read_device_error() == b.MLRA_OK
