"""q8_0 blocks whose scale lies in float32's subnormal range: every call that stores them stores the oracle's bytes.

The scale is zero in fp16, so no value depends on these codes; the cache's bytes and the state's do.  1 / d overflows
below d = 2^-128, and a subnormal d can be so coarse that x / d passes 127.
"""

import numpy as np
import pytest
import torch

from oracle import q8_0
from paged_util import TYPES, i32, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def rows(n, hkv, d, dtype, seed):
    rng = np.random.default_rng(seed)
    amax = np.ldexp(rng.uniform(1, 2, (n, hkv, d // 32, 1)), rng.integers(-149, -118, (n, hkv, d // 32, 1)))
    x = amax * rng.uniform(-1, 1, (n, hkv, d // 32, 32))
    x[..., 3:5] = 0
    x[..., 7] = amax[..., 0]
    x[0, 0] = 0
    return torch.from_numpy(x.astype(np.float32).reshape(n, hkv, d)).to(TYPES[dtype])


def expect(cache, kv, x, at):
    """The codes and scales of rows x [n][H][D] at positions `at` of a head-major cache of one layer."""
    d, q = q8_0.quantize_blocks(x.float().cpu().numpy())
    codes, scales = cache.codes(kv)[:, 0, at], cache.scales(kv)[:, 0, at]
    assert torch.equal(codes.transpose(0, 1).cpu(), torch.from_numpy(q))
    assert torch.equal(scales.transpose(0, 1).cpu().view(torch.int16), torch.from_numpy(d.view(np.int16)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_call_stores_the_oracles_bytes(kvc, dtype):
    hq, hkv, d, n = 10, 2, 128, 300
    k, v = rows(n, hkv, d, dtype, 1).cuda(), rows(n, hkv, d, dtype, 2).cuda()
    q = torch.randn(n, hq, d, device="cuda").to(TYPES[dtype])
    new = lambda: kvc.KVCache(1, 512, hkv, d, "q8_0", "head_major")
    whole = slice(0, n)

    plain = new()
    kvc.kv_cache_append(plain, 0, 0, k, v)
    paged = new()
    pages = kvc.PageTable(torch.arange(8, dtype=torch.int32, device="cuda")[None], i32([n]), 64)
    kvc.kv_paged_append(paged, 0, pages, starts([n]), k, v)
    step = new()
    out = kvc.prefill_step(step, 0, 0, q[:250], k[:250], v[:250])
    assert (out == 0).all()
    for p in range(250, 260):
        assert (kvc.decode_step(step, 0, p, q[p], k[p], v[p]) == 0).all()
    kvc.kv_cache_append_batch([step], 0, [260], k[260:261], v[260:261])
    for cache, at in ((plain, whole), (paged, whole), (step, slice(0, 261))):
        expect(cache, 0, k[at], at)
        expect(cache, 1, v[at], at)
    assert torch.equal(kvc.kv_state_get(plain, n), kvc.kv_state_get(paged, n))


def test_ordinary_blocks_beside_tiny_ones(kvc):
    # a tiny block next to ordinary ones, and values of both signs on either side of the limits
    hkv, d, n = 4, 128, 64
    x = torch.randn(n, hkv, d)
    x[::2, :, 32:64] = rows(n // 2, hkv, 32, "f32", 3)
    x[1, 0, :32] = 2.0 ** -121 * torch.linspace(-1, 1, 32)
    x[1, 1, :32] = 2.0 ** -120.99 * torch.linspace(-1, 1, 32)
    cache = kvc.KVCache(1, n, hkv, d, "q8_0", "head_major")
    kvc.kv_cache_append(cache, 0, 0, x.cuda(), x.flip(0).contiguous().cuda())
    expect(cache, 0, x, slice(0, n))
    expect(cache, 1, x.flip(0), slice(0, n))
