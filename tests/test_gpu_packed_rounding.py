"""attn_packed: what the rounding of the softmax numerators adds to that of the output, over many rows.

With h half a step of the type just above a power of two, rounding a number of mantissa x (1 to 2) errs by h / x at most and
h / (x sqrt 3) in the mean square, relative to the number.  Over mantissas evenly spread in their logarithm the mean square
of 1 / x is 3 / (8 ln 2) = 0.541.  An output is a sum of values with rounded weights, and the values are independent: the
relative mean square of the numerators' part is theirs, 0.541 h^2 / 3 where their mantissas are spread, or 1 / x^2 h^2 / 3 of
the greatest where it is most of the sum.  Beside the output's own 0.541 h^2 / 3 this gives errors of at most sqrt(2) = 1.41
times the output's rounding if the greatest numerator is not near the lower end of a power of two (x >= 1.36), and of
sqrt(1 + 1 / 0.541) = 1.69 if it is.  In rows of one key the output's rounding is nothing, which can only raise the ratio.
"""

import pytest
import torch

from paged_util import TYPES, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,many,d", [(2, 3000, 64), (3, 2000, 128), (8, 800, 64), (40, 100, 128), (92, 60, 64), (500, 6, 128)])
def test_few_keys(kvc, dtype, n, many, d):
    t, g = TYPES[dtype], torch.Generator(device="cuda").manual_seed(n)
    q, k, v = (torch.randn(many, n, h, d, generator=g, device="cuda").to(t) for h in (8, 2, 2))
    out = kvc.attn_packed(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), starts([n] * many)).view(many, n, 8, d)
    kk, vv = (x.double().repeat_interleave(4, 2) for x in (k, v))
    s = torch.einsum("brhd,bnhd->bhrn", q.double(), kk) / d ** 0.5
    s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -float("inf"))
    want = torch.einsum("bhrn,bnhd->brhd", torch.softmax(s, -1), vv)
    err = (out.double() - want).norm() / (want.to(t).double() - want).norm()
    assert err < 1.45, err.item()
