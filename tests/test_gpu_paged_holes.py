"""decode_attn_paged over tables with many holes: tiles without any key (whose slot of the ring nothing is copied to),
tiles with some, and short ends, in turn, so that a slot's counts change with every use."""

import numpy as np
import pytest
import torch

from paged_util import attend64, check, check_lse, inputs, make_pool, pool_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("cache_type", ["f16", "q8_0"])
def test_tiles_without_keys_between_others(kvc, cache_type, page):
    rng = np.random.default_rng(page)
    held = [6000, 4500, 777, 130, 64, 1] * 4
    cache, pages, slots = make_pool(kvc, held, page, 2, 128, cache_type, "head_major", seed=page, layers=1)
    table = pages.table.cpu().numpy()
    run = max(64 // page, 1)
    for i, h in enumerate(held):
        for a in range(0, -(-h // page), run):     # whole tiles let go, and single pages
            if rng.random() < 0.5:
                table[i, a:a + run] = -1
        table[i][rng.random(table.shape[1]) < 0.2] = -1
        slots[i] = [s if table[i, p // page] >= 0 else -1 for p, s in enumerate(slots[i])]
    pages.table.copy_(torch.from_numpy(table))
    q = inputs((len(held), 10, 128), torch.bfloat16, 3)
    lse = torch.empty(len(held), 10, device="cuda")
    out = kvc.decode_attn_paged(cache, 0, pages, q, lse=lse)
    for i, sl in enumerate(slots):
        sl = [s for s in sl if s >= 0]
        k, v = (pool_values(cache, 0, kv, sl) for kv in (0, 1))
        o, l, b, lb = attend64(q[i:i + 1], k, v, torch.full((1,), len(sl), device="cuda"), v_step=2.0 ** -11)
        check(out[i], o[0], b[0], "seq %d" % i)
        check_lse(lse[i], l[0], lb[0], "seq %d" % i)
    for _ in range(20):
        assert torch.equal(kvc.decode_attn_paged(cache, 0, pages, q), out)
    assert kvc.kvc_device_status() == 0
