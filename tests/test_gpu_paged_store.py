"""kv_paged_append and kv_paged_read: bytes equal to kv_cache_append's on the oracle's quantiser, whatever the page
size, layout, type and packing; values read back exact to one rounding; nothing else touched."""

import numpy as np
import pytest
import torch

from oracle import q8_0
from paged_util import TYPES, i32, inputs, make_pool, pool_values, starts

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
        x = x[keep]
        if cache.cache_type == "q8_0":
            d_, q = q8_0.quantize_blocks(x.reshape(-1, 32))
            parts = [(cache.codes(kv), torch.from_numpy(q.reshape(x.shape)).cuda()),
                     (cache.scales(kv), torch.from_numpy(d_.reshape(*x.shape[:2], -1)).cuda())]
        else:
            parts = [(cache.codes(kv), torch.from_numpy(x.astype(np.float16)).cuda())]
        for t, val in parts:
            if cache.layout == "head_major":
                t[:, layer, at] = val.transpose(0, 1).to(t.dtype)
            else:
                t[layer, at] = val.to(t.dtype)
    views, cache._bufs = cache._bufs, saved
    return views


CASES = [  # cache, layout, dtype, heads, d, page, held, rows
    ("q8_0", "head_major", "bf16", 8, 128, 16, [1, 17, 300, 64], [1, 17, 300, 64]),
    ("q8_0", "layer_major", "f32", 2, 64, 48, [100, 0, 49, 48, 1], [3, 0, 49, 1, 1]),
    ("q8_0", "head_major", "f16", 3, 96, 64, [65, 128, 129], [1, 128, 2]),
    ("q8_0", "layer_major", "bf16", 1, 32, 128, [500], [37]),
    ("f16", "head_major", "f32", 2, 64, 32, [33, 5, 0, 96], [33, 5, 0, 96]),
    ("f16", "layer_major", "bf16", 8, 128, 16, [1, 2, 3, 400], [1, 1, 1, 1]),
    ("f16", "head_major", "f16", 5, 128, 256, [257, 255], [130, 255]),
]


@pytest.mark.parametrize("cache_type,layout,dtype,hkv,d,page,held,rows", CASES)
def test_append_stores_the_oracles_bytes_and_read_returns_them(kvc, cache_type, layout, dtype, hkv, d, page, held, rows):
    cache, pages, slots = make_pool(kvc, held, page, hkv, d, cache_type, layout, seed=len(held) + d)
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
        kk = torch.full((n + pad, hkv, d), 7.0, dtype=TYPES[out], device="cuda")
        vv = kk.clone()
        kvc.kv_paged_read(cache, 1, pages, starts(rows), n + pad, dtype=TYPES[out], k=kk, v=vv)
        for kv, got in ((0, kk), (1, vv)):
            assert torch.equal(got[:n], pool_values(cache, 1, kv, mine).float().to(TYPES[out]))
            assert (got[n:] == 7).all()   # rows behind the last sequence stay as they were


def test_same_bytes_as_the_contiguous_append(kvc):
    # pages in order make the pool a plain cache
    hkv, d, n = 8, 128, 333
    k, v = inputs((n, hkv, d), torch.bfloat16, 1), inputs((n, hkv, d), torch.bfloat16, 2)
    a = kvc.KVCache(1, 384, hkv, d, "q8_0", "head_major")
    b = kvc.KVCache(1, 384, hkv, d, "q8_0", "head_major")
    for c in (a, b):
        for t in c._bufs:
            t.zero_()
    kvc.kv_cache_append(a, 0, 0, k, v)
    pages = kvc.PageTable(torch.arange(6, dtype=torch.int32, device="cuda")[None], i32([n]), 64)
    kvc.kv_paged_append(b, 0, pages, starts([n]), k, v)
    assert all(torch.equal(x, y) for x, y in zip(a._bufs, b._bufs))


@pytest.mark.parametrize("cache_type", ["q8_0", "f16"])
def test_strided_rows_of_a_fused_projection(kvc, cache_type):
    held = [40, 70]
    cache, pages, slots = make_pool(kvc, held, 16, 4, 64, cache_type, "head_major")
    qkv = inputs((110, 12, 64), torch.bfloat16, 9)
    k, v = qkv[:, 4:8], qkv[:, 8:]
    before = snapshot(cache)
    kvc.kv_paged_append(cache, 0, pages, starts(held), k, v)
    got = snapshot(cache)
    for b, s in zip(cache._bufs, before):
        b.copy_(s)
    kvc.kv_paged_append(cache, 0, pages, starts(held), k.contiguous(), v.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, cache._bufs))


@pytest.mark.parametrize("cache_type,layout", [("q8_0", "layer_major"), ("f16", "head_major")])
def test_holes_and_rows_before_the_start(kvc, cache_type, layout):
    held, page, hkv, d = [40, 40, 40, 10], 16, 2, 64
    cache, pages, slots = make_pool(kvc, held, page, hkv, d, cache_type, layout, max_pages=3)
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
        ref = pool_values(cache, 0, kv, [max(s, 0) for s in mine]).float()
        ref[hole] = 0
        assert torch.equal(got, ref)


def test_row_starts_that_leave_rows_to_nobody(kvc):
    # leading and trailing rows belong to no sequence; starts past the tensor are cut at its end
    cache, pages, slots = make_pool(kvc, [20, 30], 16, 2, 32, "f16", "layer_major")
    rs = i32([5, 15, 45])                        # rows 5..14 and 15..44, of which the tensor has 40
    k, v = inputs((40, 2, 32), torch.float16, 1), inputs((40, 2, 32), torch.float16, 2)
    mine = [-1] * 5 + slots[0][10:] + slots[1][:25]
    before = snapshot(cache)
    kvc.kv_paged_append(cache, 0, pages, rs, k, v)
    want = expected_bufs(cache, before, 0, mine, k.float().cpu().numpy(), v.float().cpu().numpy())
    assert all(torch.equal(a, b) for a, b in zip(cache._bufs, want))


def test_empty_calls(kvc):
    cache, pages, _ = make_pool(kvc, [20], 16, 2, 64, "q8_0", "head_major")
    before = snapshot(cache)
    none = torch.empty(0, 2, 64, device="cuda")
    kvc.kv_paged_append(cache, 0, pages, starts([0]), none, none)
    k, v = kvc.kv_paged_read(cache, 0, pages, starts([0]), 0)
    assert k.shape == (0, 2, 64)
    nobody = kvc.PageTable(torch.empty(0, 1, dtype=torch.int32, device="cuda"), i32([]), 16)
    x = inputs((4, 2, 64), torch.float32, 1)
    kvc.kv_paged_append(cache, 0, nobody, i32([0]), x, x)
    assert all(torch.equal(a, b) for a, b in zip(cache._bufs, before))


def test_captured_append_and_read_follow_new_lengths_and_pages(kvc):
    held = [18, 35]
    cache, pages, slots = make_pool(kvc, held, 16, 4, 128, "q8_0", "head_major", extra_pages=4)
    k, v = inputs((2, 4, 128), torch.bfloat16, 1), inputs((2, 4, 128), torch.bfloat16, 2)
    rs = starts([1, 1])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        kvc.kv_paged_append(cache, 0, pages, rs, k, v)
        kk, vv = kvc.kv_paged_read(cache, 0, pages, rs, 2, dtype=torch.float32)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kvc.kv_paged_append(cache, 0, pages, rs, k, v)
            kvc.kv_paged_read(cache, 0, pages, rs, 2, dtype=torch.float32, k=kk, v=vv)
    torch.cuda.synchronize()
    pages.lengths.add_(1)
    k.copy_(inputs((2, 4, 128), torch.bfloat16, 11))
    g.replay()
    torch.cuda.synchronize()
    now = [int(pages.table[i, h // 16]) * 16 + h % 16 for i, h in enumerate(held)]
    ref = pool_values(cache, 0, 0, now)
    assert torch.equal(kk, ref.float())
    d, q = q8_0.quantize_blocks(k.float().cpu().numpy().reshape(-1, 32))
    assert np.array_equal((q.astype(np.float64) * d.astype(np.float64).reshape(-1, 1)).reshape(2, 4, 128),
                          ref.cpu().numpy())


def test_pool_past_32_bit_offsets(kvc):
    # 2^31 elements lie before the last page
    cache = kvc.KVCache(1, 1 << 20, 32, 128, "q8_0", "layer_major")
    n_pages = (1 << 20) // 64
    pages = kvc.PageTable(i32([[n_pages - 1]]), i32([50]), 64)
    x, y = inputs((50, 32, 128), torch.bfloat16, 1), inputs((50, 32, 128), torch.bfloat16, 2)
    kvc.kv_paged_append(cache, 0, pages, starts([50]), x, y)
    k, v = kvc.kv_paged_read(cache, 0, pages, starts([50]), 50, dtype=torch.float32)
    at = (n_pages - 1) * 64
    for kv, got, src in ((0, k, x), (1, v, y)):
        d, q = q8_0.quantize_blocks(src.float().cpu().numpy().reshape(-1, 32))
        assert np.array_equal(cache.codes(kv)[0, at:at + 50].cpu().numpy().reshape(-1, 32), q)
        ref = (q.astype(np.float32) * d.astype(np.float32).reshape(-1, 1)).reshape(50, 32, 128)
        assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ties_near_ties_and_extreme_scales(kvc, dtype):
    """Quotients at and around every half-integer, for scales over the whole range, against IEEE division."""
    rng = np.random.default_rng(3)
    rows, hkv, d = 256, 4, 128
    lo, hi = (-14, 15) if dtype == "f16" else (-120, 120)
    amax = np.ldexp(rng.uniform(1, 2, (rows, hkv, 4)), rng.integers(lo, hi, (rows, hkv, 4))).astype(np.float32)
    amax = torch.from_numpy(amax).to(TYPES[dtype]).float().numpy()
    step = amax / np.float32(127)
    h = rng.integers(0, 127, (rows, hkv, 4, 32)) + 0.5
    x = (step[..., None] * h.astype(np.float32)).astype(np.float32)
    for _ in range(3):   # up to three floats to either side
        side = rng.integers(-1, 2, x.shape)
        x = np.where(side == 0, x, np.nextafter(x, np.where(side < 0, np.float32(0), np.float32(np.inf)))).astype(np.float32)
    x = np.minimum(x, amax[..., None])
    x[..., 5] = amax
    x *= rng.choice([-1, 1], x.shape)
    if dtype == "f32":
        x[:8] *= np.float32(2.0 ** -30)       # down into the subnormal numbers
        x[0, 0, :, :] = np.float32(1e-40)
    t = torch.from_numpy(x.reshape(rows, hkv, d)).to(TYPES[dtype]).cuda()
    cache, pages, slots = make_pool(kvc, [rows], 64, hkv, d, "q8_0", "head_major")
    before = snapshot(cache)
    kvc.kv_paged_append(cache, 0, pages, starts([rows]), t, t.flip(0).contiguous())
    f = lambda u: u.float().cpu().numpy()
    want = expected_bufs(cache, before, 0, slots[0], f(t), f(t.flip(0)))
    for a, b in zip(cache._bufs, want):
        assert torch.equal(a, b)
