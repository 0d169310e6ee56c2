"""Keys far below a row's greatest score: each weighs almost nothing, but a long context has many of them.

One key scores zero and has the value zero; all others score 17.5 less (25.2 powers of two) and have the value v, so
out = v T / (1 + T) with T = (n - 1) exp(-17.5): nothing but the small weights shows.  A numerator 2^-25.2 of the
greatest is below half of fp16's least number, and 2^-18.2 (the greatest being 2^7) is within 2^-25 of an fp16 number,
2^-6.7 of itself.  (Where the zero-scoring key is not in the same part of the row, the numerators are closer.)  Beside that:
the other roundings, 2^-9 at most together.
"""

import pytest
import torch

from paged_util import TYPES, half_step, make_pool, pool_values, starts

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -6.7 + 2.0 ** -9


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def put(cache, kv, at, x):
    """x [dim] at the pool positions `at` of every head and layer."""
    codes, scales = cache.codes(kv), cache.scales(kv)
    if scales is None:
        codes[:, :, at] = x.to(codes.dtype)
        return
    d = (x.unflatten(-1, (-1, 32)).abs().amax(-1) / 127).half()
    q = (x.unflatten(-1, (-1, 32)) / d.float().clamp(min=1e-6)[..., None]).round().flatten(-2)
    codes[:, :, at] = q.to(codes.dtype)
    scales[:, :, at] = d


@pytest.mark.parametrize("held", [[16], [64, 3, 130], [5000]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cache_type,d", [("f16", 64), ("f16", 128), ("q8_0", 64), ("q8_0", 128)])
@pytest.mark.parametrize("hq", [2, 12])
def test_decode(kvc, cache_type, d, dtype, held, hq):
    cache, pages, slots = make_pool(kvc, held, 16, 1, d, cache_type, "head_major", layers=1)
    tail = torch.zeros(d, device="cuda")
    tail[0] = -17.5 * d ** 0.5 / 8
    ones = torch.ones(d, device="cuda")
    for sl in slots:
        at = torch.tensor(sl, device="cuda")
        for kv, x in ((0, tail), (1, ones)):
            put(cache, kv, at, x)
            put(cache, kv, at[:1], x * 0)
    q = torch.zeros(len(held), hq, d, dtype=TYPES[dtype], device="cuda")
    q[..., 0] = 8
    out = kvc.decode_attn_paged(cache, 0, pages, q)
    for i, sl in enumerate(slots):
        k, v = (pool_values(cache, 0, kv, sl)[:, 0] for kv in (0, 1))
        s = (k @ q[i, 0].double()) / d ** 0.5
        p = torch.exp(s - s.max())
        want = (p @ v) / p.sum()
        assert want.min() > 0.9 * (len(sl) - 1) * 2.4e-8
        assert ((out[i].double() - want).abs() <= want * (STEP + half_step(out.dtype))).all()
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("f16", 128), ("bf16", 64)])
def test_packed(kvc, dtype, d):
    # enough sequences that the CTAs' runs leave most of them whole; one row each, over all keys
    n, n_seq, t = 2500, 320, TYPES[dtype]
    k = torch.zeros(n_seq, n, 1, d, device="cuda", dtype=t)
    v = torch.full((n_seq, n, 1, d), 1024.0, device="cuda", dtype=t)
    c = {64: 17.5, 128: 24.75}[d]
    k[:, 1:, :, 0] = -c
    v[:, 0] = 0
    q = torch.zeros(n_seq, 4, d, device="cuda", dtype=t)
    q[..., 0] = 8
    out = kvc.attn_packed(q, k.flatten(0, 1), v.flatten(0, 1), starts([1] * n_seq), starts([n] * n_seq))
    T = torch.exp(torch.tensor(-8 * c / d ** 0.5, dtype=torch.float64)) * (n - 1)
    want = 1024 * (T / (1 + T)).item()
    assert ((out.double() - want).abs() <= want * (STEP + 2 * half_step(t))).all()
    assert kvc.kvc_device_status() == 0
