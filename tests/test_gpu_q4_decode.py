"""decode_attn_paged over q4_0 pools against attention in 64 bits over the values the pool holds (pool4_util has the bound)."""

import pytest
import torch

from paged_util import TYPES, i32, inputs, starts
from paged_util import check, check_lse
from pool4_util import attend4, codes4, make_pool4, verify4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


CASES = [  # layout, dtype, hq, hkv, d, page, held
    ("head_major", "bf16", 40, 8, 128, 16, [1, 2, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129, 1000]),
    ("layer_major", "f16", 40, 8, 128, 64, [2049, 5, 127, 129]),
    ("head_major", "f32", 16, 1, 128, 32, [700, 31]),
    ("layer_major", "bf16", 24, 2, 64, 48, [900, 0, 47, 49, 95]),
    ("head_major", "f16", 4, 2, 64, 16, [300]),
    ("layer_major", "f32", 8, 8, 64, 128, [257, 1, 128]),
    ("head_major", "bf16", 9, 1, 128, 256, [640, 127, 1]),
    ("head_major", "bf16", 6, 2, 128, 16, [1] * 40 + [200] * 3 + [3] * 60),
]


@pytest.mark.parametrize("layout,dtype,hq,hkv,d,page,held", CASES)
def test_matches_64_bits(kvc, layout, dtype, hq, hkv, d, page, held):
    cache, pages, slots = make_pool4(kvc, held, page, hkv, d, layout, seed=hq + d)
    verify4(kvc, cache, 1, pages, slots, inputs((len(held), hq, d), TYPES[dtype], 3))


@pytest.mark.parametrize("n_seq", [1, 3, 151, 400])
@pytest.mark.parametrize("hq", [10, 26])
def test_ragged_batches(kvc, n_seq, hq):
    held = [(i * 7919) % 1500 if i % 5 else (i * 31) % 40 for i in range(n_seq)]
    held[0] = 20000 if n_seq < 10 else 3000
    cache, pages, slots = make_pool4(kvc, held, 32, 2, 128, "layer_major", seed=n_seq, layers=1)
    verify4(kvc, cache, 0, pages, slots, inputs((n_seq, hq, 128), torch.bfloat16, 4))


@pytest.mark.parametrize("n_seq,every,hkv,d", [(5000, 41, 2, 64), (65535, 997, 1, 128), (65535, 65534, 4, 64), (3000, 1, 1, 64)])
def test_many_sequences_of_which_most_are_empty(kvc, n_seq, every, hkv, d):
    cache, _, _ = make_pool4(kvc, [1024], 16, hkv, d, "layer_major", layers=1)
    n_pages = cache.n_ctx // 16
    g = torch.Generator(device="cuda").manual_seed(n_seq + every)
    table = torch.randint(0, n_pages, (n_seq, 20), generator=g, device="cuda", dtype=torch.int32)   # shared, only read
    lengths = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    lengths[::every] = torch.randint(0, 40, lengths[::every].shape, generator=g, device="cuda", dtype=torch.int32)
    lengths[n_seq - 1] = 320
    lengths[n_seq // 2] = 319
    pages = kvc.PageTable(table, lengths, 16)
    q = inputs((n_seq, 3 * hkv, d), torch.float16, 5)
    lse = torch.full((n_seq, 3 * hkv), 5.0, device="cuda")
    out = kvc.decode_attn_paged(cache, 0, pages, q, lse=lse)
    empty = lengths == 0
    assert (out[empty] == 0).all() and (lse[empty] == -float("inf")).all()
    some = torch.nonzero(~empty)[:, 0].tolist()
    for i in some[:60] + some[-60:]:
        n = int(lengths[i])
        slots = (table[i].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()[:n].tolist()
        (k, dk), (v, dv) = (codes4(cache, 0, kv, slots) for kv in (0, 1))
        o, l, b, lb = attend4(q[i], k * dk.repeat_interleave(32, -1), dk, v * dv.repeat_interleave(32, -1), dv)
        check(out[i], o, b, "seq %d" % i)
        check_lse(lse[i], l, lb, "seq %d" % i)
    assert torch.equal(out, kvc.decode_attn_paged(cache, 0, pages, q))


@pytest.mark.parametrize("d", [128, 64])
def test_holes_and_noise_outside_the_sequences(kvc, d):
    held = [200, 100, 50, 300]
    cache, pages, slots = make_pool4(kvc, held, 16, 2, d, "head_major", seed=2)
    mine = {s for sl in slots for s in sl}
    other = torch.tensor([p for p in range(cache.n_ctx) if p not in mine], device="cuda")
    for kv in (0, 1):   # NaN and infinity wherever no sequence holds a position
        cache.scales(kv)[:, :, other[::2]] = float("nan")
        cache.scales(kv)[:, :, other[1::2]] = float("inf")
    pages.table[0, 3] = -1                        # holes: inside, at the front, the whole of a sequence
    pages.table[1, 0] = 1 << 30
    pages.table[2, :] = -7
    for i, h in ((0, range(48, 64)), (1, range(16)), (2, range(50))):
        for p in h:
            slots[i][p] = -1
    out, lse = verify4(kvc, cache, 0, pages, slots, inputs((4, 10, d), torch.bfloat16, 8))
    assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()


def test_lengths_past_the_table_and_negative(kvc):
    cache, pages, slots = make_pool4(kvc, [40, 40, 40], 16, 2, 128, "layer_major")
    pages.lengths.copy_(i32([100, -5, 40]))       # the table has 48 positions
    slots[0] = [int(pages.table[0, p // 16]) * 16 + p % 16 for p in range(48)]
    slots[1] = []
    verify4(kvc, cache, 1, pages, slots, inputs((3, 4, 128), torch.float16, 8))


def test_large_scores(kvc):
    # scores up to a few hundred: the running maximum grows by more than its slack many times
    cache, pages, slots = make_pool4(kvc, [1500, 700], 16, 2, 128, "head_major")
    ramp = torch.linspace(0.05, 3, cache.n_ctx, device="cuda").half()
    cache.scales(0)[:, 0].mul_(ramp[None, :, None])
    verify4(kvc, cache, 0, pages, slots, inputs((2, 10, 128), torch.bfloat16, 8, 4.0))


@pytest.mark.parametrize("factor", [2.0 ** -13, 2.0 ** 12])
def test_scales_of_values_far_from_one(kvc, factor):
    # the numerators times V's scales stay in fp16's normal range whatever the scales are
    cache, pages, slots = make_pool4(kvc, [5000, 90], 16, 2, 128, "head_major")
    cache.scales(1).mul_(factor)
    verify4(kvc, cache, 0, pages, slots, inputs((2, 10, 128), torch.float32, 8))


def test_scales_of_values_that_grow(kvc):
    # from 2^-14 to 2^13 along the sequence, by jumps and within tiles, and zero at first
    cache, pages, slots = make_pool4(kvc, [3000], 16, 1, 64, "head_major", seed=4)
    e = torch.linspace(-14, 13, 3000).round()
    at = torch.tensor(slots[0], device="cuda")
    s = cache.scales(1)[:, 0]
    s[:, at] = (s[:, at].float() * (2.0 ** e).cuda()[None, :, None]).half()
    s[:, at[:40]] = 0
    verify4(kvc, cache, 0, pages, slots, inputs((1, 8, 64), torch.float32, 8, 0.3))
    verify4(kvc, cache, 0, pages, slots, inputs((1, 16, 64), torch.float32, 9, 0.3))


@pytest.mark.parametrize("factor", [1e-30, 2.0 ** -20, 1e30])
def test_queries_of_any_magnitude(kvc, factor):
    # each head is scaled by a power of two: 11 bits of every query count; keys of the opposite magnitude where they can be
    cache, pages, slots = make_pool4(kvc, [400, 20], 16, 2, 64, "layer_major")
    q = inputs((2, 6, 64), torch.float32, 8)
    if factor > 1:
        for i in (0, 1):
            cache.scales(0).zero_()
        verify4(kvc, cache, 0, pages, slots, q * factor)
    else:
        verify4(kvc, cache, 0, pages, slots, q * factor)


def test_queries_past_the_range_of_fp16(kvc):
    cache, pages, slots = make_pool4(kvc, [400, 20], 16, 2, 64, "layer_major")
    cache.scales(0).mul_(2.0 ** -14)    # scores of a few units from queries of 2^18
    verify4(kvc, cache, 0, pages, slots, inputs((2, 6, 64), torch.float32, 8, 2.0 ** 18))


def test_small_weights_of_long_contexts_count(kvc):
    # one key 2^20 times as heavy as each of 60,000 others: together they weigh 6% of it
    n = 60001
    cache, pages, slots = make_pool4(kvc, [n], 64, 1, 128, "head_major", layers=1)
    at = torch.tensor(slots[0], device="cuda")
    cache.codes(0).fill_(0x99)                         # all codes +1
    cache.scales(0)[:] = 2.0 ** -10
    cache.codes(1)[:, 0, at] = 0xBB                    # all values 3 d
    cache.scales(1)[:] = 0.25
    big = at[n // 2]
    cache.codes(1)[:, 0, big] = 0x88                   # but for the heavy one: zero
    cache.scales(0)[:, 0, big] = 2.0 ** -10 * 8
    q = torch.full((1, 4, 128), 1.0, device="cuda") * (20 * 0.6931471805599453 * 128 ** 0.5 / (128 * 7 * 2.0 ** -10))
    out, _ = verify4(kvc, cache, 0, pages, slots, q)
    w = 60000 * 2.0 ** -20
    assert abs(out.double().mean().item() / (0.75 * w / (1 + w)) - 1) < 0.02   # the score's own steps: 13.9 * 2^-11


def test_strided_queries_and_given_outputs(kvc):
    cache, pages, slots = make_pool4(kvc, [77, 300], 16, 2, 64, "head_major")
    qkv = inputs((2, 14, 64), torch.bfloat16, 8)
    out, scratch = torch.empty(2, 10, 64, dtype=torch.bfloat16, device="cuda"), kvc.paged_scratch(cache, 2, 10)
    got, _ = verify4(kvc, cache, 0, pages, slots, qkv[:, :10], out=out, scratch=scratch)
    assert got is out
    assert torch.equal(got, kvc.decode_attn_paged(cache, 0, pages, qkv[:, :10].contiguous(), scratch=scratch))


def test_replayed_graph_follows_lengths_and_pages(kvc):
    held = [100, 900, 3]
    cache, pages, slots = make_pool4(kvc, held, 16, 2, 128, "head_major", extra_pages=8, max_pages=64)
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
    replayed = out.clone()
    slots[0] = slots[0][:7]
    slots[2] = [int(pages.table[2, p // 16]) * 16 + p % 16 for p in range(70)]
    again, _ = verify4(kvc, cache, 0, pages, slots, q)
    assert torch.equal(replayed, again)


def test_two_streams_at_once(kvc):
    cache, pages, slots = make_pool4(kvc, [4000, 2500, 10], 16, 2, 128, "head_major")
    qs = [inputs((3, 10, 128), torch.bfloat16, 20 + i) for i in range(2)]
    scratch = [kvc.paged_scratch(cache, 3, 10) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = [verify4(kvc, cache, 0, pages, slots, q)[0] for q in qs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(kvc.decode_attn_paged(cache, 0, pages, qs[i], scratch=scratch[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_pool_past_32_bit_offsets(kvc):
    cache = kvc.KVCache(1, 1 << 21, 32, 128, "q4_0", "head_major")    # 2^33 codes, 2^32 bytes
    n_pages = (1 << 21) // 64
    table = i32([[n_pages - 1, 0, n_pages // 2]])
    pages = kvc.PageTable(table, i32([150]), 64)
    slots = [[int(table[0, p // 64]) * 64 + p % 64 for p in range(150)]]
    kvc.kv_paged_append(cache, 0, pages, starts([150]), inputs((150, 32, 128), torch.bfloat16, 1),
                        inputs((150, 32, 128), torch.bfloat16, 2))
    verify4(kvc, cache, 0, pages, slots, inputs((1, 64, 128), torch.bfloat16, 3))


def test_a_query_of_nan_is_nan(kvc):
    # one inside a run, one cut into many; the other heads and sequences are what they would be
    cache, pages, slots = make_pool4(kvc, [40, 30000, 333], 16, 2, 128, "head_major", seed=5)
    q = inputs((3, 10, 128), torch.bfloat16, 6)
    clean = kvc.decode_attn_paged(cache, 0, pages, q)
    q[0, 3, 7] = q[1, 8] = float("nan")
    out = kvc.decode_attn_paged(cache, 0, pages, q)
    want = clean.clone()
    want[0, 3] = want[1, 8] = float("nan")
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(0.0), want.nan_to_num(0.0))


@pytest.mark.parametrize("layout", ["head_major", "layer_major"])
def test_tokens_stored_just_before(kvc, layout):
    # a step's scales lie in sectors that the step before read
    held = [33, 700, 5, 16]
    cache, pages, _ = make_pool4(kvc, held, 16, 4, 128, layout, extra_pages=12, max_pages=50)
    used = {int(p) for i, h in enumerate(held) for p in pages.table[i, :-(-h // 16)].tolist()}
    spare = [p for p in range(cache.n_ctx // 16) if p not in used]
    for i, h in enumerate(held):          # pages for 40 more tokens of each
        n = -(-h // 16)
        pages.table[i, n:n + 3] = i32(spare[3 * i:3 * i + 3])
    q = inputs((40, 4, 12, 128), torch.bfloat16, 1)
    kv = inputs((40, 2, 4, 4, 128), torch.bfloat16, 2)
    one, scratch, outs = starts([1] * 4), kvc.paged_scratch(cache, 4, 12), []
    start = pages.lengths.clone()
    for t in range(40):
        pages.lengths.add_(1)
        kvc.kv_paged_append(cache, 0, pages, one, kv[t, 0], kv[t, 1])
        outs.append(kvc.decode_attn_paged(cache, 0, pages, q[t], scratch=scratch))
    torch.cuda.synchronize()
    for t in range(40):
        pages.lengths.copy_(start + t + 1)
        torch.cuda.synchronize()
        assert torch.equal(outs[t], kvc.decode_attn_paged(cache, 0, pages, q[t])), t
        torch.cuda.synchronize()
