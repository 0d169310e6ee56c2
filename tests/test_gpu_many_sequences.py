"""The paged and packed calls at their limit of 65,535 sequences: each is a copy of one of a few dozen, whose outputs are
known in 64 bits."""

import numpy as np
import pytest
import torch

from paged_util import attend64, half_step, i32, inputs, make_pool, pool_values, starts

pytestmark = pytest.mark.gpu

N, KINDS = 65535, 40


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def close(got, want, bound):
    limit = bound * 1.01 + want.abs() * half_step(got.dtype) * 1.01 + 2.0 ** -25
    assert ((got.double() - want).abs() <= limit).all()


@pytest.mark.parametrize("cache_type", ["q8_0", "f16"])
def test_paged(kvc, cache_type):
    rng = np.random.default_rng(5)
    held = [int(x) for x in rng.integers(0, 45, KINDS)]
    held[:3] = [0, 1, 45]
    cache, pages, slots = make_pool(kvc, held, 16, 2, 64, cache_type, "layer_major", layers=1)
    kind = torch.from_numpy(rng.integers(0, KINDS, N)).cuda()
    many = kvc.PageTable(pages.table[kind].contiguous(), pages.lengths[kind].contiguous(), 16)
    q = inputs((KINDS, 4, 64), torch.bfloat16, 3)
    out = kvc.decode_attn_paged(cache, 0, many, q[kind].contiguous())
    want = torch.zeros(KINDS, 4, 64, dtype=torch.float64, device="cuda")
    bound = want.clone()
    for i, sl in enumerate(slots):
        k, v = (pool_values(cache, 0, kv, sl) for kv in (0, 1))
        o, _, b, _ = attend64(q[i:i + 1], k, v, i32([len(sl)]), v_step=2.0 ** -11)
        want[i], bound[i] = o[0], b[0]
    close(out, want[kind], bound[kind])
    # the last row of each, read from the pool; sequences without positions have none
    rows = (many.lengths > 0).int()
    at = torch.cat([i32([0]), rows.cumsum(0).int()])
    n = int(rows.sum())
    k, _ = kvc.kv_paged_read(cache, 0, many, at, n, dtype=torch.float32)
    last = torch.zeros(KINDS, 2, 64, dtype=torch.float64, device="cuda")
    for i, sl in enumerate(slots):
        if sl:
            last[i] = pool_values(cache, 0, 0, sl[-1:])[0]
    assert torch.equal(k.double(), last[kind[rows.bool()]])
    assert kvc.kvc_device_status() == 0


def test_packed(kvc):
    rng = np.random.default_rng(6)
    nk = rng.integers(0, 12, KINDS)
    nq = np.minimum(rng.integers(0, 5, KINDS), nk)
    nq[0], nk[0], nk[1], nq[1] = 2, 0, 300, 3
    q, k, v = (inputs((KINDS, r, h, 64), torch.float16, s) for r, h, s in ((5, 4, 1), (300, 2, 2), (300, 2, 3)))
    kind = rng.integers(0, KINDS, N)
    kind[kind == 1] = 2
    kind[[0, 1000, N - 1]] = 1
    rows = lambda n: (torch.from_numpy(np.repeat(kind, n[kind])).cuda(),
                      torch.from_numpy(np.concatenate([np.arange(n[i]) for i in kind])).cuda())
    (qi, qr), (ki, kr) = rows(nq), rows(nk)
    out = kvc.attn_packed(q[qi, qr], k[ki, kr], v[ki, kr], starts(nq[kind]), starts(nk[kind]))
    want = torch.zeros(KINDS, 5, 4, 64, dtype=torch.float64, device="cuda")
    bound = want.clone()
    for i in range(KINDS):
        r = int(nq[i])
        o, _, b, _ = attend64(q[i, :r], k[i, :nk[i]], v[i, :nk[i]], torch.arange(r, device="cuda") + int(nk[i]) - r,
                              p_step=half_step(q.dtype))
        want[i, :r], bound[i, :r] = o, b
    close(out, want[qi, qr], bound[qi, qr])
    assert kvc.kvc_device_status() == 0
