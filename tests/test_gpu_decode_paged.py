"""decode_attn_paged against attention in 64 bits over the values the pool holds (paged_util has the bound)."""

import pytest
import torch

from paged_util import TYPES, attend64, check, check_lse, i32, inputs, make_pool, pool_values, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def expect(cache, layer, slots, q):
    """Per sequence (out, lse, bounds) with the roundings of fp16 products: q, the values d * q and the numerators."""
    v_step = 2.0 ** -11 if cache.cache_type == "q8_0" else 0.0
    q_step = 2.0 ** -11 if q.dtype == torch.float32 else 0.0
    for i, sl in enumerate(slots):
        sl = [x for x in sl if x >= 0]
        k, v = (pool_values(cache, layer, kv, sl) for kv in (0, 1))
        last = torch.full((1,), len(sl), device="cuda")
        o, l, b, lb = attend64(q[i:i + 1], k, v, last, v_step=v_step, q_step=q_step)
        yield o[0], l[0], b[0], lb[0]


def verify(kvc, cache, layer, pages, slots, q, **kw):
    lse = torch.full((len(slots), q.shape[1]), 5.0, device="cuda")
    out = kvc.decode_attn_paged(cache, layer, pages, q, lse=lse, **kw)
    for i, (o, l, b, lb) in enumerate(expect(cache, layer, slots, q)):
        check(out[i], o, b, "seq %d" % i)
        check_lse(lse[i], l, lb, "seq %d" % i)
    assert kvc.kvc_device_status() == 0
    return out, lse


CASES = [  # cache, layout, dtype, hq, hkv, d, page, held
    ("q8_0", "head_major", "bf16", 40, 8, 128, 16, [1, 2, 15, 16, 17, 63, 64, 65, 0, 1000]),
    ("q8_0", "layer_major", "f16", 40, 8, 128, 64, [2049, 5, 127, 129]),
    ("q8_0", "head_major", "f32", 16, 1, 128, 32, [700, 31]),
    ("q8_0", "layer_major", "bf16", 24, 2, 64, 48, [900, 0, 47, 49, 95]),
    ("q8_0", "head_major", "f16", 4, 2, 64, 16, [300]),
    ("f16", "head_major", "bf16", 40, 8, 128, 16, [5000, 1, 33]),
    ("f16", "layer_major", "f16", 9, 1, 128, 128, [640, 127, 1]),
    ("f16", "layer_major", "bf16", 8, 8, 64, 32, [65, 64, 63, 0]),
    ("f16", "head_major", "f32", 32, 2, 64, 256, [257, 4]),
    ("f16", "head_major", "bf16", 6, 2, 128, 16, [1] * 40 + [200] * 3 + [3] * 60),
]


@pytest.mark.parametrize("cache_type,layout,dtype,hq,hkv,d,page,held", CASES)
def test_matches_64_bits(kvc, cache_type, layout, dtype, hq, hkv, d, page, held):
    cache, pages, slots = make_pool(kvc, held, page, hkv, d, cache_type, layout, seed=hq + d)
    q = inputs((len(held), hq, d), TYPES[dtype], 3)
    verify(kvc, cache, 1, pages, slots, q)


@pytest.mark.parametrize("n_seq", [1, 3, 151, 400])
@pytest.mark.parametrize("cache_type", ["q8_0", "f16"])
def test_ragged_batches(kvc, cache_type, n_seq):
    held = [(i * 7919) % 1500 if i % 5 else (i * 31) % 40 for i in range(n_seq)]
    held[0] = 20000 if n_seq < 10 else 3000
    cache, pages, slots = make_pool(kvc, held, 32, 2, 128, cache_type, "layer_major", seed=n_seq, layers=1)
    q = inputs((n_seq, 10, 128), torch.bfloat16, 4)
    verify(kvc, cache, 0, pages, slots, q)


@pytest.mark.parametrize("cache_type,d", [("q8_0", 128), ("f16", 128), ("f16", 64), ("q8_0", 64)])
def test_holes_and_noise_outside_the_sequences(kvc, cache_type, d):
    held = [200, 100, 50, 300]
    cache, pages, slots = make_pool(kvc, held, 16, 2, d, cache_type, "head_major", seed=2)
    mine = {s for sl in slots for s in sl}
    other = [p for p in range(cache.n_ctx) if p not in mine]
    at = torch.tensor(other, device="cuda")
    for kv in (0, 1):   # NaN and infinity wherever no sequence holds a position
        t = cache.codes(kv) if cache_type == "f16" else cache.scales(kv)
        t[:, :, at[::2]] = float("nan")
        t[:, :, at[1::2]] = float("inf")
    pages.table[0, 3] = -1                        # holes: inside, at the front, the whole of a sequence
    pages.table[1, 0] = 1 << 30
    pages.table[2, :] = -7
    for i, h in ((0, range(48, 64)), (1, range(16)), (2, range(50))):
        for p in h:
            slots[i][p] = -1
    q = inputs((4, 10, d), torch.bfloat16, 8)
    out, lse = verify(kvc, cache, 0, pages, slots, q)
    assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()


def test_lengths_past_the_table_and_negative(kvc):
    cache, pages, slots = make_pool(kvc, [40, 40, 40], 16, 2, 128, "f16", "layer_major")
    q = inputs((3, 4, 128), torch.float16, 8)
    pages.lengths.copy_(i32([100, -5, 40]))       # the table has 48 positions
    slots[0] = [int(pages.table[0, p // 16]) * 16 + p % 16 for p in range(48)]
    slots[1] = []
    verify(kvc, cache, 1, pages, slots, q)


def test_large_scores(kvc):
    # scores up to a few hundred: the running maximum grows by more than its slack many times
    cache, pages, slots = make_pool(kvc, [1500, 700], 16, 2, 128, "f16", "head_major")
    ramp = torch.linspace(0.05, 6, cache.n_ctx, device="cuda").half()
    cache.codes(0)[:, 0].mul_(ramp[None, :, None])
    q = inputs((2, 10, 128), torch.bfloat16, 8, 4.0)
    verify(kvc, cache, 0, pages, slots, q)


def test_strided_queries_and_given_outputs(kvc):
    cache, pages, slots = make_pool(kvc, [77, 300], 16, 2, 64, "q8_0", "head_major")
    qkv = inputs((2, 14, 64), torch.bfloat16, 8)
    out = torch.empty(2, 10, 64, dtype=torch.bfloat16, device="cuda")
    scratch = kvc.paged_scratch(cache, 2, 10)
    got, _ = verify(kvc, cache, 0, pages, slots, qkv[:, :10], out=out, scratch=scratch)
    assert got is out
    again = kvc.decode_attn_paged(cache, 0, pages, qkv[:, :10].contiguous(), scratch=scratch)
    assert torch.equal(got, again)


def test_shared_pages(kvc):
    # two sequences with one prefix read the same pages
    cache, pages, slots = make_pool(kvc, [64, 64], 16, 2, 128, "q8_0", "layer_major")
    pages.table[1, :3] = pages.table[0, :3]
    slots[1][:48] = slots[0][:48]
    verify(kvc, cache, 0, pages, slots, inputs((2, 10, 128), torch.bfloat16, 1))


@pytest.mark.parametrize("cache_type", ["q8_0", "f16"])
def test_replayed_graph_follows_lengths_and_pages(kvc, cache_type):
    held = [100, 900, 3]
    cache, pages, slots = make_pool(kvc, held, 16, 2, 128, cache_type, "head_major", extra_pages=8, max_pages=64)
    q = inputs((3, 10, 128), torch.bfloat16, 1)
    out, scratch = torch.empty_like(q), kvc.paged_scratch(cache, 3, 10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kvc.decode_attn_paged(cache, 0, pages, q, out=out, scratch=scratch)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kvc.decode_attn_paged(cache, 0, pages, q, out=out, scratch=scratch)
    used = set(pages.table.flatten().tolist())
    free = [p for p in range(cache.n_ctx // 16) if p not in used]
    pages.table[2, 1:5] = i32(free[:4])
    pages.lengths.copy_(i32([7, 900, 70]))
    q.copy_(inputs((3, 10, 128), torch.bfloat16, 2))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    slots[0] = slots[0][:7]
    slots[2] = [int(pages.table[2, p // 16]) * 16 + p % 16 for p in range(70)]
    for i, (o, l, b, lb) in enumerate(expect(cache, 0, slots, q)):
        check(out[i], o, b, "seq %d" % i)


def test_two_streams_at_once(kvc):
    cache, pages, slots = make_pool(kvc, [4000, 2500, 10], 16, 2, 128, "q8_0", "head_major")
    qs = [inputs((3, 10, 128), torch.bfloat16, 20 + i) for i in range(2)]
    scratch = [kvc.paged_scratch(cache, 3, 10) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(kvc.decode_attn_paged(cache, 0, pages, qs[i], scratch=scratch[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])
        for j, (o, l, b, lb) in enumerate(expect(cache, 0, slots, qs[i])):
            check(outs[i][0][j], o, b, "stream %d seq %d" % (i, j))


def test_what_a_call_allocates_belongs_to_its_stream(kvc):
    # the side stream is busy when memory is asked for on the current one
    held = [9000, 200]
    cache, pages, _ = make_pool(kvc, held, 16, 2, 128, "f16", "head_major", seed=9)
    q = inputs((2, 10, 128), torch.bfloat16, 4)
    x, xs = inputs((3000, 10, 128), torch.bfloat16, 5), i32([0, 3000])
    want, want_x = kvc.decode_attn_paged(cache, 0, pages, q), kvc.attn_packed(x, x[:, :2], x[:, 2:4], xs)
    sizes = [kvc.paged_scratch(cache, 2, 10).nbytes, kvc.packed_scratch(3000, 1, 10, 2, 128).nbytes, q.nbytes, x.nbytes]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = kvc.decode_attn_paged(cache, 0, pages, q, stream=side)
    got_x = kvc.attn_packed(x, x[:, :2], x[:, 2:4], xs, stream=side)
    for n in sizes:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_x, want_x)


def test_pool_past_32_bit_offsets(kvc):
    cache = kvc.KVCache(1, 1 << 20, 16, 128, "f16", "head_major")    # 2^31 values, 2^32 bytes
    n_pages = (1 << 20) // 64
    table = i32([[n_pages - 1, 0, n_pages // 2]])
    pages = kvc.PageTable(table, i32([150]), 64)
    slots = [[int(table[0, p // 64]) * 64 + p % 64 for p in range(150)]]
    kvc.kv_paged_append(cache, 0, pages, starts([150]), inputs((150, 16, 128), torch.bfloat16, 1),
                        inputs((150, 16, 128), torch.bfloat16, 2))
    verify(kvc, cache, 0, pages, slots, inputs((1, 32, 128), torch.bfloat16, 3))


def test_no_sequences(kvc):
    cache, _, _ = make_pool(kvc, [20], 16, 2, 64, "q8_0", "head_major")
    nobody = kvc.PageTable(torch.empty(0, 1, dtype=torch.int32, device="cuda"), i32([]), 16)
    out = kvc.decode_attn_paged(cache, 0, nobody, torch.empty(0, 4, 64, device="cuda"))
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("cache_type", ["q8_0", "f16"])
def test_a_query_of_nan_is_nan(kvc, cache_type):
    # one inside a run, one cut into many; the other heads and sequences are what they would be
    held = [40, 30000, 333]
    cache, pages, slots = make_pool(kvc, held, 16, 2, 128, cache_type, "head_major", seed=5)
    q = inputs((3, 10, 128), torch.bfloat16, 6)
    clean = kvc.decode_attn_paged(cache, 0, pages, q)
    q[0, 3, 7] = q[1, 8] = float("nan")
    out = kvc.decode_attn_paged(cache, 0, pages, q)
    want = clean.clone()
    want[0, 3] = want[1, 8] = float("nan")
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(0.0), want.nan_to_num(0.0))


def test_keys_of_infinity_have_no_weight(kvc):
    # scores of -infinity, over whole tiles and among others, count nothing
    held = [500, 20000]
    cache, pages, slots = make_pool(kvc, held, 16, 1, 64, "f16", "head_major", seed=5, layers=1)
    q = inputs((2, 4, 64), torch.float16, 6).abs() + 0.01
    gone = [list(range(0, 200)) + [300], list(range(3000, 9000)) + [19999]]
    at = [s for sl, g in zip(slots, gone) for s in (sl[j] for j in g)]
    cache.codes(0)[:, 0, torch.tensor(at, device="cuda")] = -float("inf")
    kept = [[s for j, s in enumerate(sl) if j not in set(g)] for sl, g in zip(slots, gone)]
    lse = torch.full((2, 4), 5.0, device="cuda")
    out = kvc.decode_attn_paged(cache, 0, pages, q, lse=lse)
    for i, (o, l, b, lb) in enumerate(expect(cache, 0, kept, q)):
        check(out[i], o, b, "seq %d" % i)
        check_lse(lse[i], l, lb, "seq %d" % i)
