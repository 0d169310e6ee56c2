"""Helpers of the paged-cache and packed-prompt tests: pools with shuffled pages, and attention in 64 bits.

The bound of an attention output counts its roundings.  With A = sum_j p_j |v_j| (p the softmax weights):
rounding the numerators to a type of relative step eps costs at most eps/2 A, rounding the values eps/2 A, an error
ds in the scores 2 ds A, and the output's own rounding eps/2 |out|.  float32 sums of n terms, taken in chains of
n/8 + 32 steps at most, cost (n/8 + 32) 2^-23 A in the numerator and the same in the denominator.  fp16 numerators
below its normal range are off by 2^-25 each, against a denominator l of at least 1.
"""

import numpy as np
import torch

import seeded_inputs as si  # noqa: F401  (the path of the repository is set by conftest)

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(counts):
    return i32([0] + list(np.cumsum(counts)))


def inputs(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def make_pool(kvc, held, page, hkv, d, cache_type, layout, seed=0, layers=2, extra_pages=2, max_pages=None):
    """A pool of `layers` layers whose every byte is set (codes and scales of noise, so that anything read by
    mistake shows), its page table in shuffled order, and the slots of every sequence's positions."""
    used = [-(-h // page) for h in held]
    n_pages = sum(used) + extra_pages
    rng = np.random.default_rng(seed)
    order = rng.permutation(n_pages)
    width = max_pages or max(max(used), 1)
    table = np.full((len(held), width), -1, dtype=np.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    cache = kvc.KVCache(layers, n_pages * page, hkv, d, cache_type, layout)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    for kv in (0, 1):
        c = cache.codes(kv)
        if cache_type == "q8_0":
            c.copy_(torch.randint(-127, 128, c.shape, generator=g, device="cuda", dtype=torch.int8))
            s = cache.scales(kv)
            s.copy_(torch.rand(s.shape, generator=g, device="cuda") * 0.03 + 0.001)
        else:
            c.copy_(torch.randn(c.shape, generator=g, device="cuda"))
    pages = kvc.PageTable(torch.from_numpy(table).cuda(), i32(list(held)), page)
    slots = [[int(table[i, p // page]) * page + p % page for p in range(h)] for i, h in enumerate(held)]
    return cache, pages, slots


def pool_values(cache, layer, kv, slots):
    """The values the pool holds at `slots`, in 64 bits: [slot][head][value]."""
    at = torch.tensor(slots, dtype=torch.long, device="cuda")

    def pick(t):
        return t[:, layer, at].transpose(0, 1) if cache.layout == "head_major" else t[layer, at]

    x = pick(cache.codes(kv)).double()
    if cache.cache_type == "q8_0":
        x = x * pick(cache.scales(kv)).double().repeat_interleave(32, -1)
    return x


def attend64(q, k, v, last, p_step=2.0 ** -11, v_step=0.0, q_step=0.0):
    """Attention in 64 bits of rows q [r][hq][d] over k, v [n][hkv][d]; row i sees keys j <= last[i] (a tensor) .
    Returns (out, lse, bound of out without its own rounding, bound of lse)."""
    r, hq, d = q.shape
    n, hkv, _ = k.shape
    if n == 0:
        z = torch.zeros(r, hq, d, dtype=torch.float64, device=q.device)
        return z, torch.full((r, hq), -np.inf, dtype=torch.float64, device=q.device), z, z[..., 0]
    q, k, v = q.double(), k.double(), v.double()
    kk, vv = (t.repeat_interleave(hq // hkv, 1) for t in (k, v))
    s = torch.einsum("rhd,nhd->rhn", q, kk) / d ** 0.5
    unseen = (torch.arange(n, device=q.device)[None, :] > last[:, None])[:, None, :].expand_as(s)
    # scores: q rounded (q_step), products summed in float32 over d terms
    ds = torch.einsum("rhd,nhd->rhn", q.abs(), kk.abs()) / d ** 0.5 * (q_step + (d / 8 + 8) * 2.0 ** -23)
    ds = ds.masked_fill(unseen, 0).amax(-1) + 2.0 ** -21
    s = s.masked_fill(unseen, -np.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m).nan_to_num(0.0)
    l = p.sum(-1)
    none = l == 0
    safe = l.masked_fill(none, 1)
    out = torch.einsum("rhn,nhd->rhd", p, vv) / safe[..., None]
    A = torch.einsum("rhn,nhd->rhd", p, vv.abs()) / safe[..., None]
    acc = (n / 8 + 32) * 2.0 ** -23
    bound = A * (p_step + v_step + 2 * ds[..., None] + 2 * acc) + n * 2.0 ** -25 * vv.abs().amax() / safe[..., None]
    lse = torch.where(none, torch.full_like(l, -np.inf), m[..., 0] + torch.log(safe))
    return out, lse, bound, ds + acc + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -21 + 2.0 ** -20


def check(got, want, bound, what=""):
    """got (rounded to its type) against want [64 bits] within bound plus its own rounding."""
    g = got.double()
    assert g.shape == want.shape, (g.shape, want.shape)
    assert torch.isfinite(g).all(), "%s: non-finite output" % what
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    limit = bound * 1.01 + want.abs() * half_step(got.dtype) * 1.01 + tiny
    worst = ((g - want).abs() / limit.clamp(min=1e-300)).max().item() if g.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g of the bound (max abs %.3g)" % (what, worst, (g - want).abs().max().item())


def check_lse(got, want, bound, what=""):
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got) & (got < 0), inf), what
    err = (got.double() - want).masked_fill(inf, 0).abs()
    assert (err <= bound).all(), "%s: lse off by %.3g" % (what, err.max().item())
