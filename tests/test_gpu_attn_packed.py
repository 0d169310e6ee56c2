"""attn_packed against attention in 64 bits (paged_util has the bound), and the serving steps that the packed and
paged calls make up together."""

import pytest
import torch

from paged_util import (TYPES, attend64, check, check_lse, half_step, i32, inputs, make_pool, starts)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def verify(q, k, v, qn, kn, out, lse, q0=0, k0=0, rows=None):
    """Every sequence's rows (all of them, or about `rows` spread over each) against 64 bits."""
    a, b = q0, k0
    for i, (nq, nk) in enumerate(zip(qn, kn)):
        r = torch.arange(nq, device="cuda")
        if rows and nq > rows:
            r = torch.cat([torch.linspace(0, nq - 1, rows, device="cuda").long(), r[-3:]])
        o, l, bd, lb = attend64(q[a:a + nq][r], k[b:b + nk], v[b:b + nk], r + nk - nq, p_step=half_step(q.dtype))
        check(out[a:a + nq][r], o, bd, "seq %d" % i)
        check_lse(lse[a:a + nq][r], l, lb, "seq %d" % i)
        a, b = a + nq, b + nk


def run(kvc, q, k, v, qn, kn, rows=None, **kw):
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    ks = None if list(qn) == list(kn) else starts(kn)
    out = kvc.attn_packed(q, k, v, starts(qn), ks, lse=lse, **kw)
    verify(q, k, v, qn, kn, out, lse, rows=rows)
    assert kvc.kvc_device_status() == 0
    return out, lse


CASES = [  # dtype, hq, hkv, d, rows, keys
    ("bf16", 40, 8, 128, [1, 7, 128, 129, 0, 300], None),
    ("f16", 4, 2, 64, [64, 256, 1, 255, 257], None),
    ("bf16", 3, 3, 128, [127, 128, 129, 383], None),
    ("f16", 24, 3, 128, [1, 2, 3, 500], None),
    ("bf16", 14, 2, 64, [18, 19, 333], None),
    ("f16", 128, 1, 64, [5, 70], None),
    ("bf16", 66, 1, 128, [40], None),
    ("bf16", 16, 4, 128, [1, 1, 1, 1], [1, 500, 128, 1025]),        # one row each over cached keys
    ("f16", 40, 8, 128, [100, 17, 64], [612, 17, 700]),            # chunks over prefixes
    ("bf16", 8, 2, 64, [50, 20, 0, 9], [20, 0, 30, 3]),             # rows that see no key
    ("f16", 8, 8, 64, [130, 33], [2000, 4100]),
    ("bf16", 10, 2, 128, [1] * 70 + [90] + [2] * 30, None),
]


@pytest.mark.parametrize("dtype,hq,hkv,d,qn,kn", CASES)
def test_matches_64_bits(kvc, dtype, hq, hkv, d, qn, kn):
    kn = kn or qn
    t = TYPES[dtype]
    q, k, v = (inputs((n, h, d), t, s) for n, h, s in ((sum(qn), hq, 1), (sum(kn), hkv, 2), (sum(kn), hkv, 3)))
    out, lse = run(kvc, q, k, v, qn, kn)
    a = 0
    for nq, nk in zip(qn, kn):
        e = max(nq - nk, 0)
        assert (out[a:a + e] == 0).all() and (lse[a:a + e] == -float("inf")).all()
        a += nq


@pytest.mark.parametrize("dtype,hq,hkv,d,n", [("bf16", 40, 8, 128, 2900), ("f16", 16, 4, 64, 5001), ("bf16", 4, 4, 128, 4097)])
def test_long_prompts(kvc, dtype, hq, hkv, d, n):
    t = TYPES[dtype]
    q, k, v = inputs((n, hq, d), t, 1), inputs((n, hkv, d), t, 2), inputs((n, hkv, d), t, 3)
    run(kvc, q, k, v, [n], [n], rows=40)


@pytest.mark.parametrize("nq,nk", [(16, 30000), (600, 9001), (1, 20011)])
def test_few_rows_over_long_prefixes(kvc, nq, nk):
    q = inputs((nq, 10, 128), torch.bfloat16, 1)
    k, v = inputs((nk, 2, 128), torch.bfloat16, 2), inputs((nk, 2, 128), torch.bfloat16, 3)
    run(kvc, q, k, v, [nq], [nk], rows=30)


def test_large_scores(kvc):
    n = 900
    q, k, v = (inputs((n, 4, 128), torch.float16, s) for s in (1, 2, 3))
    k *= torch.linspace(0.05, 8, n, device="cuda").half()[:, None, None]
    q *= 3
    run(kvc, q, k, v, [n], [n])


@pytest.mark.parametrize("d", [64, 128])
def test_noise_outside_the_sequences_is_never_used(kvc, d):
    # rows before the first, between q and k's sequences and behind the last hold NaN; they stay as they were
    qn, kn, nan = [70, 33], [140, 33], float("nan")
    q, k, v = (inputs((n, h, d), torch.bfloat16, s) for n, h, s in ((120, 10, 1), (300, 2, 2), (300, 2, 3)))
    q[:5], q[108:] = nan, nan
    k[:11], v[:11], k[184:], v[184:] = nan, float("inf"), nan, nan
    out = torch.full_like(q, 7.0)
    lse = torch.full((120, 10), 5.0, device="cuda")
    kvc.attn_packed(q, k, v, i32([5, 75, 108]), i32([11, 151, 184]), out=out, lse=lse)
    verify(q, k, v, qn, kn, out, lse, q0=5, k0=11)
    assert (out[:5] == 7).all() and (out[108:] == 7).all() and (lse[:5] == 5).all() and (lse[108:] == 5).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_sequence_of_nan_keeps_to_itself(kvc, d):
    n = [77, 130, 200]
    q, k, v = (inputs((sum(n), h, d), torch.bfloat16, s) for h, s in ((6, 1), (2, 2), (2, 3)))
    clean = kvc.attn_packed(q, k, v, starts(n))
    for t in (q, k, v):
        t[77:207] = float("nan")
    out = kvc.attn_packed(q, k, v, starts(n))
    assert torch.equal(out[:77], clean[:77]) and torch.equal(out[207:], clean[207:])


def test_strided_parts_of_a_fused_projection(kvc):
    qn = [100, 45]
    qkv = inputs((145, 14, 64), torch.bfloat16, 1)
    q, k, v = qkv[:, :10], qkv[:, 10:12], qkv[:, 12:]
    out, _ = run(kvc, q, k, v, qn, qn)
    again, _ = run(kvc, q.contiguous(), k.contiguous(), v.contiguous(), qn, qn)
    assert torch.equal(out, again)


def test_starts_past_the_tensors_are_cut(kvc):
    q, k, v = (inputs((60, h, 64), torch.float16, s) for h, s in ((4, 1), (2, 2), (2, 3)))
    out = kvc.attn_packed(q, k, v, i32([0, 20, 90]), i32([0, 20, 90]))
    assert kvc.kvc_device_status() == 0
    o, _, b, _ = attend64(q[:20], k[:20], v[:20], torch.arange(20, device="cuda"), p_step=half_step(q.dtype))
    check(out[:20], o, b)


def test_empty_calls(kvc):
    e = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    assert kvc.attn_packed(e, e, e, i32([0, 0])).shape == (0, 4, 64)
    q = inputs((3, 4, 64), torch.float16, 1)
    lse = torch.zeros(3, 4, device="cuda")
    out = kvc.attn_packed(q, e, e, i32([0, 3]), i32([0, 0]), lse=lse)
    assert (out == 0).all() and (lse == -float("inf")).all()
    out = torch.full_like(q, 7.0)
    kvc.attn_packed(q, q, q, i32([0]), out=out)      # no sequences: no row belongs to any
    assert (out == 7).all()


def test_repeats_and_replays_give_the_same_bits(kvc):
    qn, kn = [300, 5, 700, 64], [800, 5, 700, 3000]
    q, k, v = (inputs((n, h, 128), torch.bfloat16, s) for n, h, s in ((sum(qn), 10, 1), (sum(kn), 2, 2), (sum(kn), 2, 3)))
    qs, ks = starts(qn), starts(kn)
    scratch = kvc.packed_scratch(sum(qn), 4, 10, 2, 128)
    ref = kvc.attn_packed(q, k, v, qs, ks, scratch=scratch)
    out = torch.empty_like(ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kvc.attn_packed(q, k, v, qs, ks, out=out, scratch=scratch)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    # other sequences of the same tensors, without a new capture
    qn, kn = [64, 1000, 5, 0], [64, 1500, 500, 100]
    qs.copy_(starts(qn)); ks.copy_(starts(kn))
    out.fill_(7)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    lse = torch.empty(q.shape[:2], device="cuda")
    assert torch.equal(kvc.attn_packed(q, k, v, qs, ks, out=torch.full_like(out, 7.0), lse=lse), out)
    verify(q, k, v, qn, kn, out, lse)


@pytest.mark.parametrize("cache_type,layout,dtype", [("q8_0", "head_major", "bf16"), ("f16", "layer_major", "f16")])
def test_a_serving_run(kvc, cache_type, layout, dtype):
    """Prompts packed into the pool, a second chunk over the cached prefix, then decode steps; every output against
    64-bit attention over what the pool holds."""
    from paged_util import pool_values
    hq, hkv, d, t = 10, 2, 128, TYPES[dtype]
    first, second = [130, 40, 257], [64, 0, 33]
    held = [a + b + 4 for a, b in zip(first, second)]
    cache, pages, slots = make_pool(kvc, held, 32, hkv, d, cache_type, layout, seed=1)
    seqs = lambda n, s: [inputs((n, h, d), t, s + i) for i, h in enumerate((hq, hkv, hkv))]
    have = [0, 0, 0]
    for rows, seed in ((first, 10), (second, 20)):
        q, k, v = seqs(sum(rows), seed)
        have = [a + b for a, b in zip(have, rows)]
        pages.lengths.copy_(i32(have))
        kvc.kv_paged_append(cache, 0, pages, starts(rows), k, v)
        kk, vv = kvc.kv_paged_read(cache, 0, pages, starts(have), sum(have), dtype=t)
        lse = torch.empty(sum(rows), hq, device="cuda")
        out = kvc.attn_packed(q, kk, vv, starts(rows), starts(have), lse=lse)
        verify(q, kk, vv, rows, have, out, lse)
    for step in range(4):
        q, k, v = seqs(3, 100 + 10 * step)
        have = [h + 1 for h in have]
        pages.lengths.copy_(i32(have))
        kvc.kv_paged_append(cache, 0, pages, starts([1, 1, 1]), k, v)
        out = kvc.decode_attn_paged(cache, 0, pages, q)
        for i in range(3):
            K, V = (pool_values(cache, 0, kv, slots[i][:have[i]]) for kv in (0, 1))
            o, _, b, _ = attend64(q[i:i + 1], K, V, i32([have[i]]), v_step=2.0 ** -11)
            check(out[i], o[0], b[0], "step %d seq %d" % (step, i))
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("dtype,sign,size", [("bf16", -1, 100), ("bf16", 1, 100), ("f16", -1, 200), ("f16", 1, 200)])
def test_scores_far_from_zero(kvc, dtype, sign, size):
    # all scores of a row lie near sign * size^2 * sqrt(128) (113,000 or 450,000) and differ by a few units
    n, t = 700, TYPES[dtype]
    q = torch.full((n, 4, 128), float(size), device="cuda").to(t)
    k = torch.full((n, 2, 128), float(sign * size), device="cuda").to(t)
    k[:, :, 0] += (inputs((n, 2), torch.float32, 2) * 0.25 * size).to(t)
    v = inputs((n, 2, 128), t, 3)
    run(kvc, q, k, v, [n], [n])


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan"), 3e38])
def test_calls_with_infinities_end(kvc, bad):
    # a key of infinities, of NaN or of the largest numbers: the rows that see it hold anything, the others what they would
    n = [300, 700, 130]
    q, k, v = (inputs((sum(n), h, 128), torch.bfloat16, s) for h, s in ((10, 1), (2, 2), (2, 3)))
    clean = kvc.attn_packed(q, k, v, starts(n))
    k[700] = bad
    q[800, :5] = bad
    out = kvc.attn_packed(q, k, v, starts(n))
    assert kvc.kvc_device_status() == 0
    assert torch.equal(out[:700], clean[:700]) and torch.equal(out[1000:], clean[1000:])


def test_a_row_of_nan_is_nan(kvc):
    # whole or cut: the long prompt's blocks are shared among the CTAs
    for n in (40, 9000):
        q, k, v = (inputs((n, h, 128), torch.bfloat16, s) for h, s in ((4, 1), (1, 2), (1, 3)))
        q[n - 1, 2] = float("nan")
        out = kvc.attn_packed(q, k, v, starts([n]))
        bad = torch.isnan(out)
        assert bad[n - 1, 2].all() and int(bad.sum()) == 128
