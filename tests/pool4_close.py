"""How far decode_attn_paged over a q4_0 pool may be from 64 bits where the sums are long: roundings as the independent errors
that they are.  (pool4_util's bound adds up the worst of each, which grows with the number of keys while the output of as many
keys shrinks: past some ten thousand it would let a lost tile through.)

With weights p (the greatest 1), L = sum p, x = sum p v / L, and n keys:
  - a numerator times V's scale is rounded to fp16: 2^-11 of itself at most, uniform: 2^-11 / sqrt(3) sqrt(sum (p v)^2) / L, as
    often as `roundings` says; below fp16's normal range it is 2^-25 at most for a scale, the greatest of which is taken to 2^3 or more,
    and less for the rest: 2^-28 of the greatest scale for a code: 2^-28 / sqrt(3) sqrt(sum (p code)^2) d_max / L;
  - a score is off by ds (pool4_util's: float32 sums over nibbles and their eights; a query's rounding besides), which moves x by
    p (v - x) ds / L: ds sqrt(sum (p (v - x))^2) / L;
  - float32 sums of signed terms, 16 keys at a time, each step off by 2^-24 of the sum on average if it truncates: n / 16 2^-24
    (sqrt(sum (p v)^2) / L + |x|); the sum of weights 2^-24 sqrt(n) |x|, exponentials and the last division 2^-20 |x|;
  - sums are taken over codes + 8 and the eights apart, 128 keys at most: the key of greatest p d stays in 8 steps of both, 15 and
    8 times.  A step adds 16 products in an order of its own, and may cut each of them and each of its sums to the 24 bits of the
    greatest, 2^-23 of it: 8 (15 + 8) 32 2^-23 max(p d) / L;
  - the output's own rounding, half a step at most, uniform.
An element may be off by 6.5 of these deviations beside what does not average out; all of them together by the deviations
themselves, since each is an upper bound (a relative rounding is 0.7 of what is counted, on average)."""

import math

import torch

from paged_util import half_step


def attend_close(q, k, dk, v, dv, q_step=0.0, roundings=1):
    """Rows q [r][hq][d] over codes k, v [n][hkv][d] with scales dk, dv [n][hkv][d / 32], all float64: out, the deviation of an
    element, what does not average out, lse and its bound."""
    r, hq, d = q.shape
    n, hkv = k.shape[:2]
    g = hq // hkv
    full = lambda t: t.repeat_interleave(32, -1)
    out, dev, rest = (torch.empty(r, hq, d, dtype=torch.float64, device=q.device) for _ in range(3))
    lse, off = (torch.empty(r, hq, dtype=torch.float64, device=q.device) for _ in range(2))
    for h in range(hkv):
        rows = q[:, h * g:(h + 1) * g].reshape(-1, d).double()
        kk, vv, code = k[:, h] * full(dk[:, h]), v[:, h] * full(dv[:, h]), v[:, h]
        km, top = full(dk[:, h].abs()), full(dv[:, h].abs()).amax(0)
        step = 256 // g * g or g
        for a in range(0, rows.shape[0], step):
            z = rows[a:a + step]
            s = z @ kk.T / d ** 0.5
            ds = (z.abs() @ kk.abs().T * q_step + z.abs() @ km.T * (23 * (d / 8 + 8) * 2.0 ** -23)) / d ** 0.5
            ds = ds.amax(-1, keepdim=True) + 2.0 ** -21
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            L = p.sum(-1, keepdim=True)
            x = p @ vv / L
            p2 = p * p
            pv2 = p2 @ (vv * vv)
            spread = (pv2 - 2 * x * (p2 @ vv) + x * x * p2.sum(-1, keepdim=True)).clamp(min=0)
            var = pv2 * (roundings * 2.0 ** -22 / 3) + spread * ds * ds
            var = var + p2 @ (code * code) * top * top * (2.0 ** -56 / 3)
            most = torch.stack([(p * dv[:, h, b].abs()).amax(-1) for b in range(d // 32)], -1).repeat_interleave(32, -1) / L
            root = pv2.sqrt() / L
            to = lambda t: t.reshape(-1, g, t.shape[-1])
            at = slice(a // g, a // g + to(x).shape[0])
            out[at, h * g:(h + 1) * g] = to(x)
            dev[at, h * g:(h + 1) * g] = to(var.sqrt() / L)
            rest[at, h * g:(h + 1) * g] = to((root + x.abs()) * (n / 16 * 2.0 ** -24) + x.abs() * (n ** 0.5 * 2.0 ** -24 + 2.0 ** -20) +
                                             most * (8 * 23 * 32 * 2.0 ** -23))
            l = (m + torch.log(L))
            lse[at, h * g:(h + 1) * g] = to(l)[..., 0]
            off[at, h * g:(h + 1) * g] = to(ds + n ** 0.5 * 2.0 ** -24 + l.abs() * 2.0 ** -21 + 2.0 ** -20)[..., 0]
    return out, dev, rest, lse, off


def check_close(got, want, dev, rest, what=""):
    own = half_step(got.dtype)
    g = got.double()
    assert g.shape == want.shape and torch.isfinite(g).all(), what
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    err = (g - want).abs()
    limit = 6.5 * dev + rest + want.abs() * own * 1.001 + tiny
    worst = (err / limit.clamp(min=1e-300)).max().item()
    assert worst <= 1.0, "%s: %.3g of an element's bound (off by %.3g)" % (what, worst, err.max().item())
    mean = lambda t: math.sqrt(t.square().mean().item())
    both = (dev.square() + (want.abs() * own).square() / 3).sqrt() + rest + tiny
    assert mean(err) <= mean(both), "%s: off by %.3g, %.3g of the bound of all" % (what, mean(err), mean(err) / mean(both))
