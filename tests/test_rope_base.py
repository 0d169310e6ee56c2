"""RopeTable refuses bases that give no frequencies (no GPU)."""

import pytest

import decode_attention_kv_cache_gb300 as kvc


@pytest.mark.parametrize("base", [0, -1e4, float("inf"), float("nan")])
@pytest.mark.parametrize("rot", [64, 2])
def test_bases_that_are_none(base, rot):
    with pytest.raises(ValueError):
        kvc.RopeTable(rot, base, device="cpu")
    assert kvc.RopeTable(2, base, inv_freq=[1.0], device="cpu").c.n_pairs == 1      # where it is not used
