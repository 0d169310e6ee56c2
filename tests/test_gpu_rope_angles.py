"""The angles of qk_norm_rope by themselves: a head of ones in front of zeros gives cosines and sines, without another rounding.

The fraction of a turn is exact but for its cut to 32 bits (2^-32 of a turn, and half of 2^-64 for each position); what is
left of it beside the nearest quarter of a turn is rounded to float32 (2^-24 of itself), and sine and cosine are off by a unit in
the last place at most: 2^-23 of themselves, the rounded angle by 2^-24 more (x cos x <= sin x, x sin x <= cos x up to an
eighth of a turn)."""

import math
from fractions import Fraction

import pytest
import torch

from paged_util import i32

pytestmark = pytest.mark.gpu
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798, 10 ** 101)


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def turned(freq, pos):
    """Cosine and sine of freq * pos, each to a float64's last bits: the angle beside the nearest quarter of a turn is exact."""
    t = Fraction(freq) * pos / (2 * PI) * 4
    quarter = math.floor(t + Fraction(1, 2))
    x = float((t - quarter) * PI / 2)
    c, s = math.cos(x), math.sin(x)
    return ((c, s), (-s, c), (-c, -s), (s, -c))[quarter % 4]


@pytest.mark.parametrize("style,d", [("half", 64), ("pairs", 64), ("half", 96)])
def test_cosines_and_sines(kvc, style, d):
    rot = 64
    pos = [0, 1, 2, 3, 7, 100, 1023, 4096, 58300, 131071, 10 ** 6 + 1, 2 ** 31 - 1, -1, -77, -2 ** 31]
    # near quarters and halves of a turn from either side, and ordinary ones
    freq = [math.pi * f * (1 + e) for f in (0.25, 0.5, 0.75, 1.0, 1.5) for e in (0.0, 1e-3, -1e-4, 1e-6)]
    freq += [1e4 ** (-i / 6) for i in range(12)]
    rope = kvc.RopeTable(rot, style=style, inv_freq=freq)
    x = torch.zeros(len(pos), 1, d, device="cuda")
    first = list(range(32)) if style == "half" else list(range(0, 64, 2))
    second = list(range(32, 64)) if style == "half" else list(range(1, 64, 2))
    x[..., first] = 1.0
    out, _ = kvc.qk_norm_rope(x, x, i32(pos), rope)
    out = out[:, 0].double().cpu()
    for r, p in enumerate(pos):
        cut = 2 * math.pi * (2.0 ** -32 + abs(p) * 2.0 ** -65)
        for i, f in enumerate(freq):
            for got, want in zip((out[r, first[i]].item(), out[r, second[i]].item()), turned(f, p)):
                assert abs(got - want) <= cut * 1.01 + abs(want) * (2.0 ** -23 + 2.0 ** -24) * 1.01, (p, f, got, want)
