"""attn_packed over long prefixes with values that name their key: a piece of V left out, taken twice or put in another's
place changes an output by a quarter or more, where the bound is the roundings of one number.

V is one in the dimension that belongs to the key's piece of 128 (piece mod D) and zero elsewhere.
  Equal weights (q = 0): out is count / keys.  All numerators are the same number, one that both types hold exactly but
    for the exponential's 2^-22, so that what errs beside it is 1 / l and the product (2^-24 each), the sum l of n numbers
    ((n / 8 + 32) 2^-23; the products' sums are whole multiples of one number and exact) and the output's rounding.
  Weights e^0 to e^3 by piece (whole-number scores in one dimension): with V >= 0 the numerators' rounding, half a step
    of the type, bounds the relative error; exponents 2^-17, sums (n / 8 + 32) 2^-23 twice, the output's rounding.
"""

import pytest
import torch

from paged_util import TYPES, half_step, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


@pytest.mark.parametrize("weights", ["equal", "by piece"])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("qn,kn", [([16], [30000]), ([600], [9001]), ([1], [20011]), ([1, 300, 128], [257, 5000, 12345]),
                                   ([4500], [4500])])
def test_every_piece_counts_once(kvc, qn, kn, dtype, d, weights):
    t, hq, hkv = TYPES[dtype], 10, 2
    q = torch.zeros(sum(qn), hq, d, dtype=t, device="cuda")
    k = torch.zeros(sum(kn), hkv, d, dtype=t, device="cuda")
    piece = torch.cat([torch.arange(n, device="cuda") // 128 for n in kn])
    v = torch.nn.functional.one_hot(piece % d, d)[:, None].expand(-1, hkv, -1).to(t).contiguous()
    step = 2.0 ** -21
    if weights != "equal":
        q[..., 0] = 8
        k[..., 0] = (piece % 7 % 4)[:, None].to(t)
        step = half_step(t) + 2.0 ** -17 + 2.0 ** -21
    out = kvc.attn_packed(q, k, v, starts(qn), starts(kn))
    a = b = 0
    for nq, nk in zip(qn, kn):
        r = torch.unique(torch.linspace(0, nq - 1, 40, device="cuda").long())
        s = k[b:b + nk, 0, 0].double()[None, :] * float(q[a, 0, 0]) / d ** 0.5
        seen = torch.arange(nk, device="cuda")[None, :] <= (r + nk - nq)[:, None]
        p = torch.exp(s) * seen
        want = ((p @ v[b:b + nk, 0].double()) / p.sum(-1, keepdim=True))[:, None]
        bound = want * (step + half_step(t) + 2 * (nk / 8 + 32) * 2.0 ** -23)
        got = out[a:a + nq][r].double()
        assert ((got - want).abs() <= bound * 1.01 + 2.0 ** -25).all(), (nq, nk)
        a, b = a + nq, b + nk
    assert kvc.kvc_device_status() == 0
