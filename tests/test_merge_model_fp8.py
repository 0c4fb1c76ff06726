"""The split merge's counter protocol over the 8-bit decode's plan, whose
charge for a range change (12 or 20 units) is more than a tile's cost: windows
can lie in a charge and own no tile."""
import random

import pytest

from tests import plan_model
from tests import test_merge_model as model

CHARGES = [12, 20]


@pytest.fixture(params=CHARGES)
def charge(request, monkeypatch):
    monkeypatch.setattr(plan_model, "SEQ_COST", request.param)
    return request.param


@pytest.mark.parametrize("ctas", [3, 7, 16, 148])
def test_counters_are_exact_and_reset_between_launches(ctas, charge):
    rng = random.Random(ctas)
    for seed in range(40):
        assert model.run(model._launches(rng, ctas), ctas, seed) == "ok", seed


@pytest.mark.parametrize("ctas", [3, 7, 16, 148])
def test_what_the_kernel_takes_from_the_plan(ctas, charge):
    """No CTA has more than two split sequences; a sequence's splits are the
    CTAs from its first tile's owner to its last's without a gap; and the owner
    of the last tile merges it exactly if the next sequence's first tile is
    another CTA's (how the kernel decides it)."""
    rng = random.Random(200 + ctas)
    gaps = 0
    for _ in range(120):
        for seqlens in model._launches(rng, ctas):
            multi, arrivals, merges, groups = model.structure(seqlens, ctas)
            assert max(len(v) for v in arrivals.values()) <= 2, seqlens
            tiles = [plan_model.seq_tiles(L, model.P, model.MAXP) for L in seqlens]
            total = sum(plan_model.TILE_COST * t + charge for t in tiles if t)
            chunk = plan_model.TILE_COST * max(-(-total // (ctas * plan_model.TILE_COST)), 1)
            owned = {c for _, _, c in plan_model.owners(seqlens, model.P, model.MAXP, ctas)}
            gaps += len(set(range(min(ctas, -(-total // chunk)))) - owned)
            cum = 0
            for n, t in enumerate(tiles):
                if not t:
                    continue
                c0, c1 = cum // chunk, (cum + (t - 1) * plan_model.TILE_COST) // chunk
                after = cum + t * plan_model.TILE_COST + charge
                later = any(tiles[n + 1:])
                if c1 > c0:
                    assert multi[n] == list(range(c0, c1 + 1))
                    member = not later or after // chunk != c1
                    assert groups[n] == list(range(c0, c1 + (1 if member else 0)))
                cum = after
    assert gaps > 0  # windows without a tile were among them
