"""decode_attn_paged over f16 and q8_0 pools with scores far past 2^27, where a reference's rounding is more than any numerator's
exponent: all weight goes to the key that is greatest, and to two alike in equal parts."""

import pytest
import torch

from paged_util import TYPES, make_pool, pool_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


@pytest.mark.parametrize("cache_type", ["f16", "q8_0"])
@pytest.mark.parametrize("hq,d", [(4, 64), (12, 128)])       # up to 8 query heads to a group, and more
@pytest.mark.parametrize("held", [[500], [20000]])           # whole, and in many runs
@pytest.mark.parametrize("great", [300.0, 5000.0, 60000.0])
def test_a_great_score_takes_all_the_weight(kvc, cache_type, hq, d, held, great):
    cache, pages, slots = make_pool(kvc, held, 16, 1, d, cache_type, "head_major", layers=1)
    at = torch.tensor(slots[0], device="cuda")
    if cache_type == "q8_0":                                 # scores of 2^26 to 2^42
        cache.codes(0).fill_(40)
        cache.scales(0).fill_(great)
    else:
        cache.codes(0).fill_(great / 2)
    v = pool_values(cache, 0, 1, slots[0])[:, 0]
    win = [7, held[0] * 3 // 4]
    for dtype, q in (("f32", 49999.0), ("bf16", 40000.0), ("f16", 65504.0)):
        q = torch.full((1, hq, d), q, device="cuda").to(TYPES[dtype])
        for n in (1, 2):
            for w in win:
                cache.codes(0)[0, 0, at[w]] = 40 if cache_type == "q8_0" else great / 2
            for w in win[:n]:
                cache.codes(0)[0, 0, at[w]] = 120 if cache_type == "q8_0" else great
            lse = torch.empty(1, hq, device="cuda")
            out = kvc.decode_attn_paged(cache, 0, pages, q, lse=lse)
            want = v[win[:n]].mean(0)
            # numerators that are powers of two; fp16 values; the output's own rounding, and the last division's
            limit = v[win[:n]].abs().amax(0) * 2.0 ** -11 + want.abs() * torch.finfo(out.dtype).eps / 2 * 1.01 + 2.0 ** -24
            assert ((out[0].double() - want).abs() <= limit).all(), (dtype, n)
            k = pool_values(cache, 0, 0, slots[0])[win[0], 0]
            score = (q[0, 0].half().double() * k).sum() / d ** 0.5
            assert ((lse[0].double() / score - 1).abs() <= 2.0 ** -20).all()
    assert kvc.kvc_device_status() == 0
