"""q8_0 codes of bf16 and fp16 values on pages: every pair of mantissas (a block's greatest, a value), at every distance of
their exponents at which the code is not zero, against IEEE division."""

import pytest
import torch

from paged_util import TYPES, i32, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


@pytest.mark.parametrize("dtype,bits", [("bf16", 8), ("f16", 11)])
@pytest.mark.parametrize("scale", [2.0 ** -9, 1.0])
def test_every_pair_of_mantissas(kvc, dtype, bits, scale):
    m = torch.arange(2 ** (bits - 1), 2 ** bits, device="cuda", dtype=torch.float32)
    n = m.numel()
    at = [m / 2 ** s for s in range(9)]
    values = torch.cat(at)                                       # 9 n values, of which a block takes those up to its greatest
    pad = -values.numel() % 31
    values = torch.cat([values, values[:pad]]).view(-1, 31)      # 31 to a block beside the greatest
    for first in range(0, n, 128):
        a = m[first:first + 128]
        x = torch.minimum(values[None], a[:, None, None])        # [amax][block][31]
        x = torch.cat([a[:, None, None].expand(-1, x.shape[1], 1), x], -1) * scale
        x[..., 1::2] *= -1
        x = x.reshape(-1, 32)
        rows = -(-x.shape[0] // 8)
        x = torch.cat([x, x[:rows * 8 - x.shape[0]]]).view(rows, 2, 128)
        t = x.to(TYPES[dtype])
        assert torch.equal(t.float(), x)                         # exactly representable
        page = 16
        n_pages = -(-rows // page)
        cache = kvc.KVCache(1, n_pages * page, 2, 128, "q8_0", "layer_major")
        pages = kvc.PageTable(torch.arange(n_pages, dtype=torch.int32, device="cuda")[None], i32([rows]), page)
        kvc.kv_paged_append(cache, 0, pages, starts([rows]), t, -t)
        b = x.view(rows, 2, 4, 32)
        d = b.abs().amax(-1)
        d = d / torch.full_like(d, 127.0)                        # (by a plain number torch would multiply by its reciprocal)
        y = (b / d[..., None]).double()
        q = (torch.sign(y) * torch.floor(y.abs() + 0.5)).view(rows, 2, 128).to(torch.int8)
        assert torch.equal(cache.codes(0)[0, :rows], q) and torch.equal(cache.codes(1)[0, :rows], -q)
        assert torch.equal(cache.scales(0)[0, :rows], d.half()) and torch.equal(cache.scales(1)[0, :rows], d.half())
