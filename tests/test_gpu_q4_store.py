"""kv_paged_append and kv_paged_read on q4_0 pools: bytes equal to the oracle's quantiser, values read back exact to one
rounding, nothing else touched."""

import numpy as np
import pytest
import torch

from oracle import q4_0
from paged_util import TYPES, i32, inputs, starts
from pool4_util import make_pool4, pool_values4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def snapshot(cache):
    return [b.clone() for b in cache._bufs]


def expected_bufs(cache, before, layer, slots, k, v):
    """The pool's four buffers after rows k, v [n][H][D] (CPU float32) went to `slots` (-1: dropped)."""
    saved = cache._bufs
    cache._bufs = [b.clone() for b in before]
    keep = [i for i, s in enumerate(slots) if s >= 0]
    at = torch.tensor([slots[i] for i in keep], dtype=torch.long, device="cuda")
    for kv, x in ((0, k), (1, v)):
        d, q = q4_0.quantize_blocks(x[keep])
        for t, val in ((cache.codes(kv), q4_0.pack(q)), (cache.scales(kv), d)):
            val = torch.from_numpy(val).cuda()
            if cache.layout == "head_major":
                t[:, layer, at] = val.transpose(0, 1)
            else:
                t[layer, at] = val
    views, cache._bufs = cache._bufs, saved
    return views


CASES = [  # layout, dtype, heads, d, page, held, rows
    ("head_major", "bf16", 8, 128, 16, [1, 17, 300, 64], [1, 17, 300, 64]),
    ("layer_major", "f32", 2, 64, 48, [100, 0, 49, 48, 1], [3, 0, 49, 1, 1]),
    ("head_major", "f16", 3, 96, 64, [65, 128, 129], [1, 128, 2]),
    ("layer_major", "bf16", 1, 32, 128, [500], [37]),
    ("layer_major", "f16", 8, 128, 32, [2500, 3000], [2500, 3000]),
    ("head_major", "f32", 5, 256, 16, [40], [40]),
]


@pytest.mark.parametrize("layout,dtype,hkv,d,page,held,rows", CASES)
def test_append_stores_the_oracles_bytes_and_read_returns_them(kvc, layout, dtype, hkv, d, page, held, rows):
    cache, pages, slots = make_pool4(kvc, held, page, hkv, d, layout, seed=len(held) + d)
    n, pad = sum(rows), 3
    k = inputs((n + pad, hkv, d), TYPES[dtype], 5)
    v = inputs((n + pad, hkv, d), TYPES[dtype], 6, 0.3)
    k[:, 0, :32] = 0   # a block of zeros
    before = snapshot(cache)
    kvc.kv_paged_append(cache, 1, pages, starts(rows), k, v)
    mine = [s for sl, r in zip(slots, rows) for s in (sl[len(sl) - r:] if r else [])]
    f = lambda t: t[:n].float().cpu().numpy()
    want = expected_bufs(cache, before, 1, mine, f(k), f(v))
    for a, b in zip(cache._bufs, want):
        assert torch.equal(a, b)
    for out in ("f32", "bf16", "f16"):
        for shift in (0, 8):   # outputs on 32-byte boundaries and 16 bytes off them
            room = [torch.full(((n + pad) * hkv * d + 16,), 7.0, dtype=TYPES[out], device="cuda") for _ in (0, 1)]
            kk, vv = (t[shift:shift + (n + pad) * hkv * d].view(n + pad, hkv, d) for t in room)
            kvc.kv_paged_read(cache, 1, pages, starts(rows), n + pad, dtype=TYPES[out], k=kk, v=vv)
            for kv, got in ((0, kk), (1, vv)):
                assert torch.equal(got[:n], pool_values4(cache, 1, kv, mine).float().to(TYPES[out]))
                assert (got[n:] == 7).all()   # rows behind the last sequence stay as they were


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ties_near_ties_and_extreme_magnitudes(kvc, dtype):
    """Quotients at and around every half-integer, for magnitudes over the whole range, against exact arithmetic."""
    rng = np.random.default_rng(3)
    rows, hkv, d = 512, 4, 128
    lo, hi = (-14, 15) if dtype == "f16" else (-126, 18)   # a scale within fp16's range
    m = np.ldexp(rng.uniform(1, 2, (rows, hkv, 4)), rng.integers(lo, hi, (rows, hkv, 4))).astype(np.float32)
    m = torch.from_numpy(m).to(TYPES[dtype]).float().numpy()
    h = rng.integers(0, 8, (rows, hkv, 4, 32)) + 0.5
    x = (m[..., None] / np.float32(8) * h.astype(np.float32)).astype(np.float32)
    for _ in range(3):   # up to three floats to either side
        side = rng.integers(-1, 2, x.shape)
        x = np.where(side == 0, x, np.nextafter(x, np.where(side < 0, np.float32(0), np.float32(np.inf)))).astype(np.float32)
    x = np.minimum(x, m[..., None])
    x[..., 5] = m
    x *= rng.choice([-1, 1], x.shape)
    if dtype == "f32":
        x[:8] *= np.float32(2.0 ** -30)       # down into the subnormal numbers
        x[0, 0, :, :] = np.float32(1e-40)
        x[1, 0, :, :] = np.float32(1e-45) * rng.integers(-3, 4, x[1, 0].shape)
    t = torch.from_numpy(x.reshape(rows, hkv, d)).to(TYPES[dtype]).cuda()
    cache, pages, slots = make_pool4(kvc, [rows], 64, hkv, d, "head_major")
    before = snapshot(cache)
    kvc.kv_paged_append(cache, 0, pages, starts([rows]), t, t.flip(0).contiguous())
    f = lambda u: u.float().cpu().numpy()
    want = expected_bufs(cache, before, 0, slots[0], f(t), f(t.flip(0)))
    for a, b in zip(cache._bufs, want):
        assert torch.equal(a, b)


def test_blocks_that_are_not_finite_read_as_such(kvc):
    cache, pages, slots = make_pool4(kvc, [3], 16, 2, 64, "layer_major")
    k, v = inputs((3, 2, 64), torch.float32, 1), inputs((3, 2, 64), torch.float32, 2)
    k[0, 0, 3] = float("nan")
    k[1, 1, 40] = float("inf")
    v[2, 0, 0] = -float("inf")
    kvc.kv_paged_append(cache, 0, pages, starts([3]), k, v)
    kk, vv = kvc.kv_paged_read(cache, 0, pages, starts([3]), 3, dtype=torch.float32)
    bad = torch.zeros(3, 2, 64, dtype=torch.bool, device="cuda")
    bad[0, 0, :32] = bad[1, 1, 32:] = True
    assert torch.equal(~torch.isfinite(kk), bad)
    bad[:] = False
    bad[2, 0, :32] = True
    assert torch.equal(~torch.isfinite(vv), bad)


def test_holes_and_rows_before_the_start(kvc):
    held, page, hkv, d = [40, 40, 40, 10], 16, 2, 64
    cache, pages, slots = make_pool4(kvc, held, page, hkv, d, "layer_major", max_pages=3)
    pages.table[0, 1] = -1                       # a page let go
    pages.table[1, 2] = cache.n_ctx // page      # one past the pool
    pages.lengths[2] = 60                        # 12 positions past the table
    rows = [40, 40, 60, 14]                      # the last sequence has four rows too many
    for i, h in ((0, range(16, 32)), (1, range(32, 40))):
        for p in h:
            slots[i][p] = -1
    third = [int(pages.table[2, p // page]) * page + p % page for p in range(48)] + [-1] * 12
    mine = slots[0] + slots[1] + third + [-1] * 4 + slots[3]
    n = sum(rows)
    k, v = inputs((n, hkv, d), torch.float32, 3), inputs((n, hkv, d), torch.float32, 4)
    before = snapshot(cache)
    kvc.kv_paged_append(cache, 0, pages, starts(rows), k, v)
    want = expected_bufs(cache, before, 0, mine, k.cpu().numpy(), v.cpu().numpy())
    assert all(torch.equal(a, b) for a, b in zip(cache._bufs, want))
    kk, vv = kvc.kv_paged_read(cache, 0, pages, starts(rows), n, dtype=torch.float32)
    hole = torch.tensor([s < 0 for s in mine], device="cuda")
    for kv, got in ((0, kk), (1, vv)):
        ref = pool_values4(cache, 0, kv, [max(s, 0) for s in mine]).float()
        ref[hole] = 0
        assert torch.equal(got, ref)


def test_pool_past_32_bit_offsets(kvc):
    # 2^32 codes, 2^31 bytes of them, lie before the last page
    cache = kvc.KVCache(1, 1 << 20, 32, 128, "q4_0", "layer_major")
    n_pages = (1 << 20) // 64
    pages = kvc.PageTable(i32([[n_pages - 1]]), i32([50]), 64)
    x, y = inputs((50, 32, 128), torch.bfloat16, 1), inputs((50, 32, 128), torch.bfloat16, 2)
    kvc.kv_paged_append(cache, 0, pages, starts([50]), x, y)
    k, v = kvc.kv_paged_read(cache, 0, pages, starts([50]), 50, dtype=torch.float32)
    at = (n_pages - 1) * 64
    for kv, got, src in ((0, k, x), (1, v, y)):
        d, q = q4_0.quantize_blocks(src.float().cpu().numpy())
        assert np.array_equal(cache.codes(kv)[0, at:at + 50].cpu().numpy(), q4_0.pack(q))
        assert np.array_equal(got.cpu().numpy(), q4_0.dequantize_blocks(d, q))


def test_truncate_clears_the_tail(kvc):
    cache, _, _ = make_pool4(kvc, [40], 16, 2, 64, "head_major")
    want = [cache.codes(0).clone(), cache.scales(0).clone(), cache.codes(1).clone(), cache.scales(1).clone()]
    kvc.kv_cache_truncate(cache, 21)
    for t in want:
        t[:, :, 21:] = 0
    got = [cache.codes(0), cache.scales(0), cache.codes(1), cache.scales(1)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,bits", [("bf16", 8), ("f16", 11)])
@pytest.mark.parametrize("sign", [1, -1])
def test_every_pair_of_mantissas(kvc, dtype, bits, sign):
    # a block's greatest and a value, at every distance of their exponents at which the code is not zero, in exact arithmetic
    m = torch.arange(2 ** (bits - 1), 2 ** bits, device="cuda", dtype=torch.float64)
    values = torch.cat([m / 2 ** s for s in range(6)])
    values = torch.cat([values, values[:-values.numel() % 31]]).view(-1, 31)
    for first in range(0, m.numel(), 128):
        a = m[first:first + 128]
        x = torch.minimum(values[None], a[:, None, None])
        x = torch.cat([sign * a[:, None, None].expand(-1, x.shape[1], 1), x], -1)
        x[..., 2::2] *= -1
        x = x.reshape(-1, 32)
        rows = -(-x.shape[0] // 8)
        x = torch.cat([x, x[:rows * 8 - x.shape[0]]])
        t = x.view(rows, 2, 128).to(TYPES[dtype])
        assert torch.equal(t.double(), x.view(rows, 2, 128))
        n_pages = -(-rows // 16)
        cache = kvc.KVCache(1, n_pages * 16, 2, 128, "q4_0", "layer_major")
        pages = kvc.PageTable(torch.arange(n_pages, dtype=torch.int32, device="cuda")[None], i32([rows]), 16)
        kvc.kv_paged_append(cache, 0, pages, starts([rows]), t, t)
        k, v = kvc.kv_paged_read(cache, 0, pages, starts([rows]), rows, dtype=torch.float32)
        lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
        g = torch.where(-lo >= hi, lo, hi)                     # of greatest magnitude, of +m and -m the negative one
        num, den = 16 * x.abs() + g.abs(), 2 * g.abs()         # floor(num / den): the magnitude, ties away from zero
        q = torch.floor(num / den)
        q = q - (q * den > num).double() + ((q + 1) * den <= num).double()
        q = torch.minimum(q * torch.sign(x) * -torch.sign(g), torch.full_like(q, 7.0))
        want = (q * (g / -8).half().double()).float().view(rows, 2, 128)
        assert torch.equal(k, want) and torch.equal(v, want)
