"""RopeTable's fixed-point frequencies against rational arithmetic, and its refusals (no GPU)."""

from fractions import Fraction

import pytest
import torch

import decode_attention_kv_cache_gb300 as kvc

PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798, 10 ** 101)


def test_turns_are_the_nearest_fractions():
    for rot, base in ((128, 1e4), (64, 1e6), (2, 7.0), (256, 5e5)):
        t = kvc.RopeTable(rot, base, device="cpu").turns.tolist()
        for i, x in enumerate(t):
            want = Fraction(base ** (-2.0 * i / rot)) / (2 * PI) * 2 ** 64
            assert abs(x % 2 ** 64 - want % 2 ** 64) <= Fraction(1, 2) + Fraction(1, 2 ** 40), (rot, i)
    f = [0.0, -0.5, 1e-30, 3e5, 6.283185307179586, -1e-12, 1e300]
    for x, v in zip(kvc.RopeTable(14, style="pairs", inv_freq=f, device="cpu").turns.tolist(), f):
        if v == 1e300:
            continue    # more turns than 2^64 / (2 pi) is known to
        off = (Fraction(x) - Fraction(v) / (2 * PI) * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, v


def test_refusals():
    for kw in (dict(rot=3), dict(rot=-2), dict(rot=8, style="thirds"), dict(rot=8, inv_freq=[1.0] * 3),
               dict(rot=4, inv_freq=[1.0, float("nan")]), dict(rot=2, inv_freq=[float("inf")])):
        with pytest.raises(ValueError):
            kvc.RopeTable(device="cpu", **kw)
    assert kvc.RopeTable(0, device="cpu").c.n_pairs == 0


def test_free_pages():
    f = kvc.FreePages(5, [3, 1], device="cpu")
    assert f.ring.tolist()[:2] == [3, 1] and f.state.tolist() == [0, 2, 0] and f.free() == (2, 0)
    assert kvc.FreePages(3, device="cpu").ring.tolist() == [0, 1, 2]
    assert kvc.FreePages(3, torch.empty(0, dtype=torch.int32), device="cpu").free() == (0, 0)
    for bad in (dict(n_pages=0), dict(n_pages=2, pages=[0, 1, 1]), dict(n_pages=3, pages=torch.zeros(2)),
                dict(n_pages=3, pages=torch.zeros(1, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            kvc.FreePages(device="cpu", **bad)
