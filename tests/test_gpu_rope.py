"""qk_norm_rope against the formula in 64 bits, and qk_norm_rope_append against qk_norm_rope and kv_paged_append.

The bound counts roundings.  With the pair's normalised values y_a, y_b: the angle is off by at most 2 pi 2^-25 (its
conversion to float32), sine and cosine by two units in the last place, and norm, weights and sums are some 16 roundings of
2^-24, all relative to |y_a| + |y_b|; then the output's own half step."""

import math

import pytest
import torch

from paged_util import TYPES, half_step, i32, inputs, make_pool, starts
from pool4_util import make_pool4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def expect(x, pos, rot, style, weight, freq, eps):
    """The output in 64 bits, and the magnitude |y_a| + |y_b| for each value."""
    y = x.double()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    out, mag, n = y.clone(), y.abs(), rot // 2
    t = pos.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    a, b = (slice(0, n), slice(n, rot)) if style == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    out[..., a] = y[..., a] * torch.cos(t) - y[..., b] * torch.sin(t)
    out[..., b] = y[..., a] * torch.sin(t) + y[..., b] * torch.cos(t)
    mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, mag


def check(got, want, mag, what, slack=0.0):
    g = got.double()
    assert g.shape == want.shape and torch.isfinite(g).all(), what
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    limit = mag * (2 * math.pi * 2.0 ** -25 + 20 * 2.0 ** -24 + slack) + want.abs() * half_step(got.dtype) * 1.001 + tiny
    worst = ((g - want).abs() / limit.clamp(min=1e-300)).max().item() if g.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g of the bound" % (what, worst)


def freqs(rot, base):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


CASES = [  # dtype, rows, hq, hkv, d, rot, style, base, far
    ("bf16", 1, 40, 8, 128, 128, "half", 1e6, 100),
    ("bf16", 7, 40, 8, 128, 128, "half", 1e6, 60000),
    ("bf16", 3000, 40, 8, 128, 128, "half", 5e5, 3000),
    ("f16", 333, 16, 4, 64, 64, "pairs", 1e4, 5000),
    ("f32", 2000, 16, 4, 64, 32, "half", 1e4, 70000),
    ("f32", 129, 5, 1, 96, 96, "half", 1e4, 100),
    ("f32", 65, 3, 3, 96, 50, "pairs", 1e4, 100),
    ("bf16", 50, 7, 1, 256, 128, "half", 1e4, 100),
    ("f16", 1500, 2, 1, 32, 32, "pairs", 1e4, 100),
    ("f32", 90, 2, 1, 32, 0, "half", 1e4, 100),
    ("bf16", 5000, 5, 1, 64, 48, "half", 1e4, 100),
    ("f32", 700, 9, 2, 256, 256, "pairs", 1e4, 1 << 20),
]


@pytest.mark.parametrize("dtype,rows,hq,hkv,d,rot,style,base,far", CASES)
def test_matches_64_bits(kvc, dtype, rows, hq, hkv, d, rot, style, base, far):
    t = TYPES[dtype]
    q, k = inputs((rows, hq, d), t, 1), inputs((rows, hkv, d), t, 2, 3.0)
    qw, kw = ((1 + inputs((d,), torch.float32, s, 0.3)).to(t) for s in (3, 4))
    g = torch.Generator(device="cuda").manual_seed(7)
    pos = torch.randint(0, far, (rows,), generator=g, device="cuda", dtype=torch.int32)
    rope = kvc.RopeTable(rot, base, style)
    for weights in ((qw, kw), (None, kw), (None, None)):
        out = kvc.qk_norm_rope(q, k, pos, rope, *weights, eps=1e-5)
        for got, x, w in zip(out, (q, k), weights):
            check(got, *expect(x, pos, rot, style, w, freqs(rot, base), 1e-5), "%s %s" % (dtype, w is not None))


WHOLE = [  # heads that rotate whole, not at all, or in neighbours: dtype, rows, hq, hkv, d, rot, style
    ("bf16", 300, 6, 2, 256, 256, "half"),
    ("f16", 257, 11, 3, 64, 64, "half"),
    ("f32", 100, 3, 1, 128, 0, "half"),
    ("f16", 65, 1, 1, 128, 40, "pairs"),
    ("bf16", 2500, 13, 5, 128, 128, "half"),
    ("f32", 2500, 21, 1, 64, 64, "half"),
]


@pytest.mark.parametrize("dtype,rows,hq,hkv,d,rot,style", WHOLE)
def test_heads_that_rotate_whole(kvc, dtype, rows, hq, hkv, d, rot, style):
    test_matches_64_bits(kvc, dtype, rows, hq, hkv, d, rot, style, 2e4, 9000)


@pytest.mark.parametrize("dtype,d,rot", [("bf16", 128, 128), ("f32", 64, 64), ("f16", 96, 48)])
def test_weights_on_any_boundary_of_their_type(kvc, dtype, d, rot):
    t = TYPES[dtype]
    q, k = inputs((33, 5, d), t, 1), inputs((33, 2, d), t, 2)
    w = (1 + inputs((2 * d,), torch.float32, 3, 0.3)).to(t)
    pos, rope = torch.arange(33, device="cuda", dtype=torch.int32) * 7, kvc.RopeTable(rot)
    for at in (1, 3, d - 1):
        part = w[at:at + d]
        got = kvc.qk_norm_rope(q, k, pos, rope, part, part)
        want = kvc.qk_norm_rope(q, k, pos, rope, part.clone(), part.clone())
        assert all(torch.equal(a, b) for a, b in zip(got, want)), at


def test_weights_that_the_kernel_before_wrote(kvc):
    q, k = inputs((2000, 8, 128), torch.bfloat16, 1), inputs((2000, 2, 128), torch.bfloat16, 2)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos, rope = torch.arange(2000, device="cuda", dtype=torch.int32), kvc.RopeTable(128)
    one = kvc.qk_norm_rope(q, k, pos, rope, w, w)
    for x in (2.0, 0.5, 4.0, 1.0):      # powers of two: the outputs scale exactly
        w.fill_(x)
        got = kvc.qk_norm_rope(q, k, pos, rope, w, w)
        assert all(torch.equal(a, b * x) for a, b in zip(got, one)), x


def test_far_and_negative_positions(kvc):
    # reference angles by exact integers: the fraction of a turn, from 300 bits of pi
    from fractions import Fraction
    pos = [0, -1, 1, 2 ** 31 - 1, -2 ** 31, 123456789, 2 ** 24 + 1]
    rot, base = 64, 1e4
    q, k = inputs((len(pos), 2, 64), torch.float32, 1), inputs((len(pos), 1, 64), torch.float32, 2)
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798,
                  10 ** 101)
    out, _ = kvc.qk_norm_rope(q, k, i32(pos), kvc.RopeTable(rot, base))
    for r, p in enumerate(pos):
        for i, f in enumerate(freqs(rot, base)):
            turn = Fraction(f) * p / (2 * pi)
            t = float((turn - turn.__floor__()) * 2 * pi)
            a, b = q[r, :, i].double(), q[r, :, i + 32].double()
            # the fraction of a turn is kept to 2^-64 a position, and its upper 32 bits are used
            slack = (a.abs() + b.abs()) * (2 * math.pi * (abs(p) * 2.0 ** -65 + 2.0 ** -32 + 2.0 ** -25) + 8 * 2.0 ** -24)
            assert ((out[r, :, i] - (a * math.cos(t) - b * math.sin(t))).abs() <= slack).all(), (p, i)
            assert ((out[r, :, i + 32] - (a * math.sin(t) + b * math.cos(t))).abs() <= slack).all(), (p, i)


def test_given_frequencies(kvc):
    f = [0.5, 0.031, 7.0, -0.25, 1e-9, 0.0, 3.5, 0.125]
    q, k = inputs((40, 3, 32), torch.float32, 1), inputs((40, 2, 32), torch.float32, 2)
    pos = torch.arange(40, device="cuda", dtype=torch.int32) * 91
    for style in ("half", "pairs"):
        out = kvc.qk_norm_rope(q, k, pos, kvc.RopeTable(16, style=style, inv_freq=f))
        for got, x in zip(out, (q, k)):
            check(got, *expect(x, pos, 16, style, None, f, 0), style)


def test_rows_of_zeros_and_of_very_unequal_magnitudes(kvc):
    q, k = torch.zeros(5, 3, 64, device="cuda"), inputs((5, 2, 64), torch.float32, 2)
    k[0] *= 1e-18
    k[1] *= 1e15
    w = 1 + inputs((64,), torch.float32, 3, 0.1)
    pos = torch.arange(5, device="cuda", dtype=torch.int32)
    qo, ko = kvc.qk_norm_rope(q, k, pos, kvc.RopeTable(64), w, w, eps=1e-6)
    assert (qo == 0).all()
    check(ko, *expect(k, pos, 64, "half", w, freqs(64, 1e4), 1e-6), "k")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_parts_of_a_fused_projection_and_in_place(kvc, dtype):
    t = TYPES[dtype]
    for rows in (9, 1200):
        qkv = inputs((rows, 16, 64), t, 1)
        q, k = qkv[:, :10], qkv[:, 10:13]
        pos = torch.arange(rows, device="cuda", dtype=torch.int32)
        rope, w = kvc.RopeTable(64), torch.ones(64, dtype=t, device="cuda") * 1.25
        a, b = kvc.qk_norm_rope(q.contiguous(), k.contiguous(), pos, rope, w, w)
        c, d = kvc.qk_norm_rope(q, k, pos, rope, w, w)
        assert torch.equal(a, c) and torch.equal(b, d)
        rest = qkv[:, 13:].clone()
        qo, ko = kvc.qk_norm_rope(q, k, pos, rope, w, w, q_out=q, k_out=k)
        assert qo is q and ko is k
        assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(qkv[:, 13:], rest)


def pool_of(kvc, cache_type, held, page, hkv, d, layout, **kw):
    return (make_pool4(kvc, held, page, hkv, d, layout, **kw) if cache_type == "q4_0"
            else make_pool(kvc, held, page, hkv, d, cache_type, layout, **kw))


STORES = [  # cache, layout, dtype, hq, hkv, d, page, held, rows, rot, style
    ("f16", "head_major", "bf16", 40, 8, 128, 16, [1, 17, 300, 64], [1, 17, 300, 64], 128, "half"),
    ("q8_0", "layer_major", "f16", 10, 2, 64, 48, [100, 0, 49, 48, 1], [3, 0, 49, 1, 1], 32, "half"),
    ("q4_0", "layer_major", "bf16", 40, 8, 128, 32, [64, 900, 5, 31], [1, 1, 1, 1], 128, "half"),
    ("q4_0", "head_major", "f32", 5, 1, 96, 64, [65, 128, 129], [1, 128, 2], 96, "pairs"),
    ("q8_0", "head_major", "bf16", 40, 8, 128, 64, [2500, 700], [2500, 700], 128, "half"),
    ("f16", "layer_major", "f32", 3, 3, 256, 16, [500], [37], 128, "pairs"),
    ("q4_0", "head_major", "f16", 7, 2, 32, 16, [333, 1], [333, 1], 32, "half"),
    ("q8_0", "layer_major", "f32", 5, 3, 64, 32, [700, 33], [700, 1], 64, "half"),
    ("q4_0", "layer_major", "f32", 6, 2, 128, 16, [90, 2600], [3, 2600], 50, "pairs"),
    ("q4_0", "head_major", "bf16", 11, 11, 256, 64, [130, 0, 64], [130, 0, 1], 256, "half"),
    ("f16", "head_major", "f16", 1, 1, 64, 16, [1, 2, 3], [1, 2, 3], 0, "half"),
]


@pytest.mark.parametrize("cache_type,layout,dtype,hq,hkv,d,page,held,rows,rot,style", STORES)
def test_append_stores_what_the_two_calls_store(kvc, cache_type, layout, dtype, hq, hkv, d, page, held, rows, rot, style):
    t, n, pad = TYPES[dtype], sum(rows), 3
    cache, pages, slots = pool_of(kvc, cache_type, held, page, hkv, d, layout, seed=d)
    qkv = inputs((n + pad, hq + 2 * hkv, d), t, 5)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    qw, kw = ((1 + inputs((d,), torch.float32, s, 0.3)).to(t) for s in (3, 4))
    rope, rs = kvc.RopeTable(rot, 1e5, style), starts(rows)
    pos = i32([p for h, r in zip(held, rows) for p in range(h - r, h)] + [0] * pad)
    before = [b.clone() for b in cache._bufs]
    want_q, kk = kvc.qk_norm_rope(q, k, pos, rope, qw, kw)
    kvc.kv_paged_append(cache, 1, pages, rs, kk, v)
    want = [b.clone() for b in cache._bufs]
    for b, s in zip(cache._bufs, before):
        b.copy_(s)
    out = torch.full((n + pad, hq, d), 7.0, dtype=t, device="cuda")
    got = kvc.qk_norm_rope_append(cache, 1, pages, rs, q, k, v, rope, qw, kw, q_out=out)
    assert got is out and torch.equal(out[:n], want_q[:n])
    assert (out[n:] == 7).all()      # rows behind the last sequence stay as they were
    assert all(torch.equal(a, b) for a, b in zip(cache._bufs, want))


@pytest.mark.parametrize("cache_type", ["f16", "q8_0", "q4_0"])
def test_append_with_holes_and_foreign_rows(kvc, cache_type):
    held, page, hkv, d = [40, 40, 40, 10], 16, 2, 64
    cache, pages, _ = pool_of(kvc, cache_type, held, page, hkv, d, "layer_major", max_pages=3)
    pages.table[0, 1] = -1                       # a page let go
    pages.table[1, 2] = cache.n_ctx // page      # one past the pool
    pages.lengths[2] = 60                        # 12 positions past the table
    rows = [40, 40, 60, 14]                      # the last sequence has four rows too many
    rs = starts(rows) + 2                        # two rows in front belong to nobody
    n = 2 + sum(rows)
    q, k, v = (inputs((n, h, d), torch.bfloat16, s) for h, s in ((6, 1), (hkv, 2), (hkv, 3)))
    pos = i32([0, 0] + list(range(40)) * 2 + list(range(60)) + list(range(-4, 10)))
    rope, w = kvc.RopeTable(64), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    before = [b.clone() for b in cache._bufs]
    want_q, kk = kvc.qk_norm_rope(q, k, pos, rope, w, w)
    kvc.kv_paged_append(cache, 0, pages, rs, kk, v)
    want = [b.clone() for b in cache._bufs]
    for b, s in zip(cache._bufs, before):
        b.copy_(s)
    out = torch.full((n, 6, d), 7.0, dtype=torch.bfloat16, device="cuda")
    kvc.qk_norm_rope_append(cache, 0, pages, rs, q, k, v, rope, w, w, q_out=out)
    assert (out[:2] == 7).all() and torch.equal(out[2:], want_q[2:])
    assert all(torch.equal(a, b) for a, b in zip(cache._bufs, want))


def test_replayed_graph_follows_positions_and_pages(kvc):
    held = [18, 35]
    cache, pages, _ = make_pool4(kvc, held, 16, 4, 128, "head_major", extra_pages=4)
    q, k, v = (inputs((2, h, 128), torch.bfloat16, s) for h, s in ((8, 1), (4, 2), (4, 3)))
    rope, rs, w = kvc.RopeTable(128), starts([1, 1]), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        kvc.qk_norm_rope_append(cache, 0, pages, rs, q, k, v, rope, w, w, q_out=out)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kvc.qk_norm_rope_append(cache, 0, pages, rs, q, k, v, rope, w, w, q_out=out)
    torch.cuda.synchronize()
    pages.lengths.add_(1)
    q.copy_(inputs((2, 8, 128), torch.bfloat16, 11))
    g.replay()
    torch.cuda.synchronize()
    got, bufs = out.clone(), [b.clone() for b in cache._bufs]
    want, kk = kvc.qk_norm_rope(q, k, i32(held), rope, w, w)
    assert torch.equal(got, want)
    kvc.kv_paged_append(cache, 0, pages, rs, kk, v)
    assert all(torch.equal(a, b) for a, b in zip(bufs, cache._bufs))


def test_outputs_belong_to_the_given_stream(kvc):
    q, k = inputs((4000, 8, 128), torch.bfloat16, 1), inputs((4000, 2, 128), torch.bfloat16, 2)
    pos, rope = torch.arange(4000, device="cuda", dtype=torch.int32), kvc.RopeTable(128)
    want = kvc.qk_norm_rope(q, k, pos, rope)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = kvc.qk_norm_rope(q, k, pos, rope, stream=side)
    for x in want:
        torch.empty(x.nbytes, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_rows(kvc):
    none = torch.empty(0, 4, 64, device="cuda")
    a, b = kvc.qk_norm_rope(none, none[:, :1], i32([]), kvc.RopeTable(64))
    assert a.shape == (0, 4, 64) and b.shape == (0, 1, 64)
