"""The 8-bit decode's accuracy is each head's and branch's own: queries whose
sizes differ by far between heads, between branches, and in single values.

Bounds as in test_fp8_cache.py, with the query error of every head and branch
taken from its own largest value: two e4m3 parts are off by at most half the
smallest step, 2^-10, of a unit that is at most 1/224 of that value."""
import pytest
import torch

from branch_latent_kv_b200 import binding as b
from tests import latent_ref as ref
from tests.test_fp8_cache import R_PROB, SHAPES, _decode_case, _gpu


def _expect(c):
    out = torch.zeros(c["q_lat"].shape, dtype=torch.float64)
    tol = torch.zeros_like(out)
    per_token = c["latent_scale"].repeat_interleave(16, 1)
    lat = ref.values(c["latent_cache"], c["latent_scale"])
    N, H, B, _ = c["q_lat"].shape
    for n, L in enumerate(c["seqlens"].tolist()):
        rows, keys, sigma = (ref.rows(t, c["block_table"], n, L) for t in (lat, c["rope_cache"], per_token))
        for h in range(H):
            for br in range(B):
                q = c["q_lat"][n:n + 1, h:h + 1, br:br + 1]
                o, t = ref.attend(q, c["q_rope"][n:n + 1, h:h + 1], rows[:, br:br + 1], keys, c["scale"], c["out_scale"], L - 1, R_PROB,
                                  float(q.float().abs().max()) * 2.0 ** -10 / 224, sigma[:, br:br + 1])
                out[n, h, br], tol[n, h, br] = o[0, 0, 0], t[0, 0, 0]
    return out, tol


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["head", "branch", "value"])
@pytest.mark.parametrize("log2", [12, 60])
@pytest.mark.parametrize("branches,d_c", SHAPES)
def test_large_queries_of_one_head_or_branch_cost_the_others_nothing(branches, d_c, log2, where):
    """One head, one branch, or one value of a head and branch 2^log2 times
    the size of the rest; two head tiles, split and whole sequences."""
    c = _decode_case(41, 18, branches, d_c, 64, 64, [700, 129, 2500], std=2.0)
    big = torch.ones(c["q_lat"].shape)
    if where == "head":
        big[:, 3] = 2.0 ** log2
    elif where == "branch":
        big[:, :, branches - 1] = 2.0 ** log2
    else:
        big[:, 17, 0, d_c - 1] = 2.0 ** log2
    c["q_lat"] = (c["q_lat"].float() * big).to(torch.bfloat16)
    got = b.mlra_decode_fp8(**_gpu(c))
    assert b.mlra_read_device_error() == 0
    ref.within(got, *_expect(c), f"{where} 2^{log2}")
