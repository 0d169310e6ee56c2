"""Pools of q4_0 for the tests: made with every byte set, read back in 64 bits, and the bound of an attention over them.

The bound is paged_util's with what a product of nibbles (codes + 8) adds: the sums run over nibbles and the eights in them
apart, so that the roundings of a sum count magnitudes of 15 + 8 scales where the value itself may be small.  Values
are exact; a numerator times a scale is rounded to float32 and then to fp16 (2^-11 and 2^-24, paged_util's p_step),
and 2^-25 where it is below fp16's normal range, against eight times the scale."""

import numpy as np
import torch

from oracle import q4_0
from paged_util import i32, make_pool


def make_pool4(kvc, held, page, hkv, d, layout, seed=0, **kw):
    cache, pages, slots = make_pool(kvc, held, page, hkv, d, "q4_0", layout, seed=seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    for kv in (0, 1):
        c, s = cache.codes(kv), cache.scales(kv)
        c.copy_(torch.randint(0, 256, c.shape, generator=g, device="cuda", dtype=torch.uint8))
        sign = torch.randint(0, 2, s.shape, generator=g, device="cuda") * 2 - 1
        s.copy_((torch.rand(s.shape, generator=g, device="cuda") * 0.3 + 0.01) * sign)
    return cache, pages, slots


def _pick(cache, layer, t, slots):
    at = torch.tensor(slots, dtype=torch.long, device="cuda")
    return t[:, layer, at].transpose(0, 1) if cache.layout == "head_major" else t[layer, at]


def codes4(cache, layer, kv, slots):
    """Codes [slot][head][value] (float64) and scales [slot][head][block] (float64) at `slots`."""
    q = q4_0.unpack(_pick(cache, layer, cache.codes(kv), slots).contiguous().cpu().numpy())
    return torch.from_numpy(q).cuda().double(), _pick(cache, layer, cache.scales(kv), slots).double()


def pool_values4(cache, layer, kv, slots):
    q, d = codes4(cache, layer, kv, slots)
    return q * d.repeat_interleave(32, -1)


def attend4(q, k, dk, v, dv, q_step=0.0):
    """One row q [hq][d] over k, v [n][hkv][d] with scales dk, dv [n][hkv][d / 32]: out, lse, and the bounds of both."""
    hq, d = q.shape
    n, hkv, _ = k.shape
    if n == 0:
        z = torch.zeros(hq, d, dtype=torch.float64, device=q.device)
        return z, torch.full((hq,), -np.inf, dtype=torch.float64, device=q.device), z, z[..., 0]
    q = q.double()
    rep = lambda t: t.repeat_interleave(hq // hkv, 1)
    kk, vv = rep(k), rep(v)
    km, vm = (rep(t.abs().repeat_interleave(32, -1)) * 23 for t in (dk, dv))
    s = torch.einsum("hd,nhd->hn", q, kk) / d ** 0.5
    ds = torch.einsum("hd,nhd->hn", q.abs(), kk.abs()) / d ** 0.5 * q_step
    ds = ds + torch.einsum("hd,nhd->hn", q.abs(), km) / d ** 0.5 * (d / 8 + 8) * 2.0 ** -23
    ds = ds.amax(-1) + 2.0 ** -21
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1)
    out = torch.einsum("hn,nhd->hd", p, vv) / l[:, None]
    A = torch.einsum("hn,nhd->hd", p, vv.abs()) / l[:, None]
    M = torch.einsum("hn,nhd->hd", p, vm) / l[:, None]
    acc = (n / 8 + 32) * 2.0 ** -23
    bound = A * (2.0 ** -11 + 2 * ds[:, None]) + 2 * acc * M + n * 2.0 ** -25 * vv.abs().amax() / l[:, None]
    lse = m[:, 0] + torch.log(l)
    return out, lse, bound, ds + acc + lse.abs() * 2.0 ** -21 + 2.0 ** -20


def verify4(kvc, cache, layer, pages, slots, q, lse=True, **kw):
    from paged_util import check, check_lse
    n, hq = len(slots), q.shape[1]
    ls = torch.full((n, hq), 5.0, device="cuda") if lse else None
    out = kvc.decode_attn_paged(cache, layer, pages, q, lse=ls, **kw)
    q_step = 2.0 ** -11 if q.dtype == torch.float32 else 0.0
    for i, sl in enumerate(slots):
        sl = [x for x in sl if x >= 0]
        (k, dk), (v, dv) = (codes4(cache, layer, kv, sl) for kv in (0, 1))
        k, v = k * dk.repeat_interleave(32, -1), v * dv.repeat_interleave(32, -1)
        o, l, b, lb = attend4(q[i], k, dk, v, dv, q_step)
        check(out[i], o, b, "seq %d" % i)
        if lse:
            check_lse(ls[i], l, lb, "seq %d" % i)
    assert kvc.kvc_device_status() == 0
    return out, ls


__all__ = ["attend4", "codes4", "i32", "make_pool4", "pool_values4", "verify4"]
