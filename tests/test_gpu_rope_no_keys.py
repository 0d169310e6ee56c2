"""qk_norm_rope of queries alone: no key heads."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


@pytest.mark.parametrize("rows", [9, 3000])
@pytest.mark.parametrize("d,rot", [(64, 64), (96, 48)])      # both kernels
def test_no_key_heads(kvc, rows, d, rot):
    x = torch.randn(rows, 3, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    pos, rope = torch.arange(rows, device="cuda", dtype=torch.int32), kvc.RopeTable(rot)
    w = 1 + 0.1 * torch.arange(d, device="cuda", dtype=torch.float32) / d
    a, b = kvc.qk_norm_rope(x, torch.empty(rows, 0, d, device="cuda"), pos, rope, w)
    c, _ = kvc.qk_norm_rope(x, x[:, :1], pos, rope, w, w)
    assert b.shape == (rows, 0, d) and torch.equal(a, c)
    got, none = kvc.qk_norm_rope(x, x[:, :0], pos, rope, w, q_out=x)      # in place
    assert got is x and none.numel() == 0 and torch.equal(x, c)
