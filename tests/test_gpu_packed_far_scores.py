"""attn_packed where a row's scores lie far from zero and close together, on inputs whose products and sums are exact.

Two dimensions of q and k are in use: one carries a product of integers that is the same for all keys near a row's
end, the other small integers that set the keys apart.  All products are whole numbers below 2^24, so the scores are
exact in float32 whatever the order of the sums, and what is left to err is counted here:
  numerators rounded to the inputs' type, half a step each: p_step = eps / 2;
  exponents: s times fl(log2 e / sqrt(D)) less the reference, one rounding, at most 64 units: 2^-24 x 64, and the
    constant's own rounding, 2^-24 of the scores' spread; with an exponential good to 2^-22 together below 2^-17;
  sums of n numerators and of n products, in chains of n / 8 + 32 steps: (n / 8 + 32) 2^-23 each;
  the output's own rounding.
Numerators more than 24 powers of two below the greatest may round to nothing: n 2^-25 of the greatest |v|.
A reference that missed the row's maximum by more than the type's range allows would show as zeros or infinities.
"""

import pytest
import torch

from paged_util import TYPES, half_step, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def verify(q, k, v, lens, out, lse):
    t, d = q.dtype, q.shape[2]
    a = 0
    for n in lens:
        g = q.shape[1] // k.shape[1]
        kk, vv = (x[a:a + n].double().repeat_interleave(g, 1) for x in (k, v))
        s = torch.einsum("rhd,nhd->rhn", q[a:a + n].double(), kk) / d ** 0.5
        late = torch.arange(n, device="cuda")[None, :] > torch.arange(n, device="cuda")[:, None]
        s = s.masked_fill(late[:, None, :], -float("inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1)
        want = torch.einsum("rhn,nhd->rhd", p, vv) / l[..., None]
        A = torch.einsum("rhn,nhd->rhd", p, vv.abs()) / l[..., None]
        bound = A * (half_step(t) + 2.0 ** -17 + 2 * (n / 8 + 32) * 2.0 ** -23) + n * 2.0 ** -25 * vv.abs().amax()
        assert (bound.amax() < 0.02 * A.amax()).all()      # the bound tells a wrong row from a right one
        got = out[a:a + n].double()
        assert torch.isfinite(got).all()
        worst = ((got - want).abs() / (bound * 1.01 + want.abs() * half_step(t) * 1.01)).max().item()
        assert worst <= 1.0, worst
        ref = m[..., 0] + torch.log(l)
        err = (lse[a:a + n].double() - ref).abs()
        assert (err <= ref.abs() * 2.0 ** -22 + 2.0 ** -16).all(), err.max().item()
        a += n


def integers(shape, lo, hi, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device="cuda").float()


def products(size):
    """Two whole numbers with a product near `size`, the greater below 2048: exact in fp16 (and, of 8 bits, in bf16)."""
    b = 1 << max((int(size).bit_length() - 8), 0)
    return (int(size) // b) & ~1, b


LENS = [700] * 12 + [513, 64, 1]     # several blocks for each CTA, of one to three tiles


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("scaled", [900, 3000, 6000, 12000, 20000, 29000, 41000])
@pytest.mark.parametrize("dtype,d", [("f16", 64), ("f16", 128), ("bf16", 64)])
def test_rows_far_from_zero(kvc, dtype, d, scaled, sign):
    n, t = sum(LENS), TYPES[dtype]
    big, scale = products(scaled * d ** 0.5)
    q = torch.zeros(n, 4, d, device="cuda")
    k = torch.zeros(n, 2, d, device="cuda")
    q[..., 0], k[..., 0] = big, sign * scale
    q[..., 1], k[..., 1] = 8, integers((n, 2), -2, 3, 1)
    v = torch.randn(n, 2, d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(t)
    q, k = q.to(t), k.to(t)
    lse = torch.empty(n, 4, device="cuda")
    out = kvc.attn_packed(q, k, v, starts(LENS), lse=lse)
    assert kvc.kvc_device_status() == 0
    verify(q, k, v, LENS, out, lse)


@pytest.mark.parametrize("rise", [500, 2500, 6000, 20000, 41000])
@pytest.mark.parametrize("dtype,d", [("f16", 64), ("f16", 128)])
def test_rows_that_rise_in_a_later_tile(kvc, dtype, d, rise):
    # the first 300 keys of a sequence score near zero; the rows from 300 on see keys that score `rise` more
    t = TYPES[dtype]
    big, scale = products(rise * d ** 0.5)
    q = torch.zeros(sum(LENS), 4, d, device="cuda")
    k = torch.zeros(sum(LENS), 2, d, device="cuda")
    a = 0
    for n in LENS:
        k[a + 300:a + n, :, 0] = scale
        a += n
    q[..., 0] = big
    q[..., 1], k[..., 1] = 8, integers((sum(LENS), 2), -2, 3, 1)
    v = torch.randn(sum(LENS), 2, d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(t)
    q, k = q.to(t), k.to(t)
    lse = torch.empty(sum(LENS), 4, device="cuda")
    out = kvc.attn_packed(q, k, v, starts(LENS), lse=lse)
    assert kvc.kvc_device_status() == 0
    verify(q, k, v, LENS, out, lse)
