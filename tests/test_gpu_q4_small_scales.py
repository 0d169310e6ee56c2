"""decode_attn_paged over q4_0 where V's scales differ by many powers of two: keys whose scales lie far below the greatest one of
their block count as kvc.h says."""

import pytest
import torch

from paged_util import TYPES, i32
from pool4_close import attend_close, check_close
from pool4_util import codes4, make_pool4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("below", [12, 17, 20, 24, 26])
@pytest.mark.parametrize("hq", [6, 24])
@pytest.mark.parametrize("heavy", [False, True])
def test_keys_far_below_the_greatest_scale_count(kvc, dtype, below, hq, heavy):
    # one key has a scale of 2^13, all others scales of 2^(13 - below); its codes are zero (heavy), or its weight is next to
    # nothing; other scores are small, so that weights are alike
    hkv, d, n = 2, 64, 3000
    cache, pages, slots = make_pool4(kvc, [n], 16, hkv, d, "head_major", layers=1)
    at = torch.tensor(slots[0], device="cuda")
    cache.codes(1).fill_(0xBB)                                   # codes of 3
    cache.codes(1)[:, 0, at[::2]] = 0x99                         # and of 1
    cache.scales(1).fill_(2.0 ** (13 - below))
    big = at[n // 3]
    cache.codes(1)[:, 0, big], cache.scales(1)[:, 0, big] = 0x88 if heavy else 0xB9, 2.0 ** 13
    cache.scales(0).mul_(0.05)
    q = torch.randn(1, hq, d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").abs().half().to(TYPES[dtype])
    if not heavy:                                                # a score of -50 or so
        cache.codes(0)[:, 0, big], cache.scales(0)[:, 0, big] = 0x00, 1.0
    out = kvc.decode_attn_paged(cache, 0, pages, q)
    (k, dk), (v, dv) = (codes4(cache, 0, kv, slots[0]) for kv in (0, 1))
    want, dev, rest, _, _ = attend_close(q, k, dk, v, dv, roundings=2 if dtype == "bf16" else 1)
    assert (dev < want.abs() * 0.02).all()                       # the bound is worth something
    check_close(out, want, dev, rest)
