"""decode_attn_paged over q4_0 with queries of any magnitude: each head has a power of two of its own, and scores of a few units
come from queries and scales that are far from one, so that a wrong power, or a query lost in it, shows."""

import pytest
import torch

from paged_util import TYPES, i32
from pool4_util import codes4, make_pool4, verify4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def normal(shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").half().float()


def spread(kvc, cache, slots, q, head):
    """The weights are far from even: the greatest of a head's is many times the mean."""
    k, dk = codes4(cache, 0, 0, slots)
    k = k * dk.repeat_interleave(32, -1)
    g = q.shape[1] // k.shape[1]
    p = torch.softmax(k[:, head // g] @ q[0, head].double() / q.shape[2] ** 0.5, 0)
    return p.max().item() * p.numel()


@pytest.mark.parametrize("e", [-17, -14, -8, 8, 13, 18, 22])
@pytest.mark.parametrize("hq,d", [(6, 64), (24, 128)])
def test_scores_of_a_few_units(kvc, e, hq, d):
    # queries of 2^e over scales of 2^-e, in fp16's normal range as long as they can be
    cache, pages, slots = make_pool4(kvc, [400, 20], 16, 2, d, "layer_major", layers=1)
    cache.scales(0).mul_(2.0 ** -max(e, -16))
    q = normal((2, hq, d), 8) * 2.0 ** e
    assert all(spread(kvc, cache, slots[0], q, h) > 2 for h in range(hq))
    verify4(kvc, cache, 0, pages, slots, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq", [8, 26])
def test_heads_of_a_group_with_magnitudes_of_their_own(kvc, dtype, hq):
    # head h has values in one block of 32 only, where the keys' scales are as small as its queries are large
    d, e = 128, [-12, -4, 5, 11]
    cache, pages, slots = make_pool4(kvc, [300, 77], 16, 2, d, "head_major", layers=1)
    for b in range(4):
        cache.scales(0)[..., b].mul_(2.0 ** -e[b])
    q = torch.zeros(2, hq, d, device="cuda")
    x = normal((2, hq, 32), 5)
    for h in range(hq):
        b = (h * 3 + h // 4) % 4
        q[:, h, 32 * b:32 * b + 32] = x[:, h] * 2.0 ** (e[b] + 1)
    q = q.to(TYPES[dtype])
    assert all(spread(kvc, cache, slots[0], q, h) > 2 for h in range(hq))
    verify4(kvc, cache, 0, pages, slots, q)


@pytest.mark.parametrize("e", [90, 60, 30])
def test_a_great_query_picks_its_key(kvc, e):
    # scores of 2^(e - 10) and more: all weight goes to the one key that is greatest
    cache, pages, slots = make_pool4(kvc, [500], 16, 1, 64, "head_major", layers=1)
    at = torch.tensor(slots[0], device="cuda")
    cache.codes(0).fill_(0x99)                      # codes of 1
    cache.scales(0).fill_(2.0 ** -8)
    q = torch.zeros(1, 4, 64, device="cuda")
    win = [3, 250, 499, 16]
    for h, w in enumerate(win):                     # value 8 h alone, the greatest at position w
        cache.codes(0)[0, 0, at[w], 4 * h] = 0x9B   # its first nibble (value 8 h of the head): a code of 3
        q[0, h, 8 * h] = 2.0 ** e
    k, dk = codes4(cache, 0, 0, slots[0])
    for h, w in enumerate(win):
        col = k[:, 0, 8 * h]
        assert col[w] == 3 and (col.sum() - 3) == len(slots[0]) - 1
    out = kvc.decode_attn_paged(cache, 0, pages, q)
    v, dv = codes4(cache, 0, 1, slots[0])
    v = (v * dv.repeat_interleave(32, -1))[:, 0]
    for h, w in enumerate(win):                     # one rounding of a numerator times a scale
        assert ((out[0, h].double() - v[w]).abs() <= v[w].abs() * 2.0 ** -10).all(), h


@pytest.mark.parametrize("e", [-90, -60])
def test_a_small_query_weighs_all_keys_alike(kvc, e):
    cache, pages, slots = make_pool4(kvc, [500], 16, 1, 64, "head_major", layers=1)
    q = normal((1, 4, 64), 2) * 2.0 ** e
    verify4(kvc, cache, 0, pages, slots, q)
