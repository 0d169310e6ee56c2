"""Refusals of the q4_0 type where it is none, of kv_pages_advance, qk_norm_rope and qk_norm_rope_append, and the
sizes of q4_0 pools: nothing here reaches a GPU."""

import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def kvc():
    from decode_attention_kv_cache_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    import decode_attention_kv_cache_gb300 as m
    return m


FAKE = 1 << 20   # an aligned address that nothing reads: every call here fails its checks or has nothing to do


def pool(kvc, **kw):
    d = dict(n_layer=2, n_ctx=512, n_head_kv=2, head_dim=64, cache_type="q4_0", layout="head_major")
    d.update(kw)
    c = kvc.kvc_cache()
    desc = kvc.make_desc(*d.values())
    assert kvc.lib.kvc_cache_init(ctypes.byref(c), ctypes.byref(desc), FAKE, FAKE, FAKE, FAKE) == 0
    return c


def pages(kvc, **kw):
    p = dict(table=FAKE, len=FAKE, n_seq=3, max_pages=8, page_size=16)
    p.update(kw)
    return kvc.kvc_pages(*p.values())


def test_q4_0_sizes(kvc):
    d = kvc.make_desc(64, 32768, 8, 128, "q4_0", "head_major")
    n = 64 * 32768 * 8 * 128
    assert kvc.cache_bytes(d) == (n // 2, n // 16, n // 2, n // 16)
    b = ctypes.c_size_t()
    assert kvc.lib.kvc_paged_scratch_bytes(ctypes.byref(d), 3, 40, ctypes.byref(b)) == 0 and b.value > 0
    bad = kvc.make_desc(1, 16, 2, 48, "q4_0")
    s = [ctypes.c_size_t() for _ in range(4)]
    assert kvc.lib.kvc_cache_bytes(ctypes.byref(bad), *[ctypes.byref(x) for x in s]) == kvc.KVC_EINVAL
    c = kvc.kvc_cache()
    ok = kvc.make_desc(1, 16, 2, 64, "q4_0")
    assert kvc.lib.kvc_cache_init(ctypes.byref(c), ctypes.byref(ok), FAKE, None, FAKE, FAKE) == kvc.KVC_EINVAL
    assert kvc.lib.kvc_cache_init(ctypes.byref(c), ctypes.byref(ok), FAKE, FAKE, FAKE, FAKE + 8) == kvc.KVC_EINVAL


def test_calls_on_contiguous_caches_refuse_q4_0(kvc):
    c, L, E = pool(kvc), kvc.lib, kvc.KVC_EINVAL
    d = ctypes.byref(c.d)
    b = ctypes.c_size_t()
    one, n = (ctypes.c_int32 * 1)(0), ctypes.c_int32()
    big = 1 << 40
    assert L.kvc_scratch_bytes(d, 4, ctypes.byref(b)) == E
    assert L.kvc_prefill_scratch_bytes(d, 4, 64, ctypes.byref(b)) == E
    assert L.kv_state_size(d, 5) == 0
    r = ctypes.byref(c)
    assert L.kv_cache_append(r, 0, 0, 1, FAKE, FAKE, 1, None) == E
    assert L.kv_cache_append_batch(r, 1, 0, one, FAKE, FAKE, 1, None) == E
    assert L.prefill_chunk_attn(r, 0, 0, 1, FAKE, 1, 4, FAKE, FAKE, big, None) == E
    assert L.prefill_step(r, 0, 0, 1, FAKE, FAKE, FAKE, 1, 4, FAKE, FAKE, big, 0, None) == E
    assert L.decode_attn(r, 0, 0, FAKE, 1, 4, FAKE, FAKE, big, None) == E
    assert L.decode_step(r, 0, 0, FAKE, FAKE, FAKE, 1, 4, FAKE, FAKE, big, None) == E
    assert L.decode_attn_batch(r, 1, 0, one, FAKE, 1, 4, FAKE, FAKE, big, None) == E
    assert L.decode_step_batch(r, 1, 0, one, FAKE, FAKE, FAKE, 1, 4, FAKE, FAKE, big, None) == E
    assert L.kv_state_get(r, 1, FAKE, big, None) == E
    assert L.kv_state_set(r, FAKE, big, ctypes.byref(n), None) == E
    assert L.kv_state_get_heads(r, 0, 2, 1, FAKE, big, None) == E
    assert L.kv_state_set_heads(r, 0, FAKE, big, ctypes.byref(n), None) == E
    lib = ctypes.CDLL(kvc.LIB_PATH)
    f = lib.decode_attn_noalloc
    f.argtypes = [ctypes.c_void_p] + [ctypes.c_int32] * 2 + [ctypes.c_void_p] + [ctypes.c_int32] * 2 + [ctypes.c_void_p] * 2
    assert f(ctypes.addressof(c), 0, 0, FAKE, 1, 4, FAKE, None) == E
    assert L.kv_cache_truncate(r, 513, None) == kvc.KVC_ERANGE      # one that takes it
    assert L.kv_cache_truncate(r, 512, None) == 0


ADVANCE = dict(pages=None, free=None, rows=FAKE, row_start=FAKE, n_rows=4, positions=FAKE, slots=FAKE)


def advance(kvc, pages_kw=(), free_kw=(), **kw):
    a = dict(ADVANCE, **kw)
    f = dict(ring=FAKE, state=FAKE, n_pages=32)
    f.update(dict(free_kw))
    a["pages"] = ctypes.byref(pages(kvc, **dict(pages_kw))) if a["pages"] is None else None
    a["free"] = ctypes.byref(kvc.kvc_free_pages(*f.values())) if a["free"] is None else None
    return kvc.lib.kv_pages_advance(*a.values(), None)


def test_advance_refusals(kvc):
    E = kvc.KVC_EINVAL
    assert advance(kvc, pages=0) == E and advance(kvc, free=0) == E and advance(kvc, n_rows=-1) == E
    for bad in (dict(page_size=0), dict(page_size=-16), dict(page_size=24), dict(n_seq=-1), dict(n_seq=65536),
                dict(max_pages=0), dict(max_pages=(1 << 31) - 1), dict(table=0), dict(len=0), dict(len=FAKE + 2)):
        assert advance(kvc, pages_kw=bad) == E, bad
    for bad in (dict(ring=0), dict(state=0), dict(n_pages=0), dict(n_pages=-3), dict(n_pages=1 << 28), dict(ring=FAKE + 1)):
        assert advance(kvc, free_kw=bad) == E, bad
    for bad in (dict(rows=0), dict(row_start=0), dict(rows=FAKE + 2), dict(positions=FAKE + 1), dict(slots=FAKE + 3)):
        assert advance(kvc, **bad) == E, bad
    assert advance(kvc, pages_kw=dict(n_seq=0)) == 0


ROPE = dict(rope=None, q=FAKE, k=FAKE, ld_q=256, ld_k=128, dtype=1, n_rows=4, n_head_q=4, n_head_kv=2, head_dim=64, pos=FAKE,
            q_weight=FAKE, k_weight=FAKE, eps=1e-6, q_out=FAKE, k_out=FAKE, ld_qo=256, ld_ko=128)
APPEND = dict(pool=None, pages=None, layer=0, row_start=FAKE, n_rows=4, rope=None, q=FAKE, k=FAKE, v=FAKE, ld_q=256,
              ld_k=128, ld_v=128, dtype=1, n_head_q=4, q_weight=FAKE, k_weight=FAKE, eps=1e-6, q_out=FAKE, ld_qo=256)


def rotate(kvc, rope_kw=(), **kw):
    a, r = dict(ROPE, **kw), dict(turns=FAKE, n_pairs=32, style=0)
    r.update(dict(rope_kw))
    a["rope"] = ctypes.byref(kvc.kvc_rope(*r.values())) if a["rope"] is None else None
    return kvc.lib.qk_norm_rope(*a.values(), None)


def rotate_append(kvc, pool_kw=(), pages_kw=(), rope_kw=(), **kw):
    a, r = dict(APPEND, **kw), dict(turns=FAKE, n_pairs=32, style=0)
    r.update(dict(rope_kw))
    a["rope"] = ctypes.byref(kvc.kvc_rope(*r.values())) if a["rope"] is None else None
    a["pool"] = ctypes.byref(pool(kvc, **dict(pool_kw))) if a["pool"] is None else None
    a["pages"] = ctypes.byref(pages(kvc, **dict(pages_kw))) if a["pages"] is None else None
    return kvc.lib.qk_norm_rope_append(*a.values(), None)


BAD_ROPES = (dict(n_pairs=-8), dict(n_pairs=33), dict(n_pairs=40), dict(n_pairs=12), dict(style=2), dict(style=-1), dict(turns=0),
             dict(turns=FAKE + 4))


def test_rope_refusals(kvc):
    E = kvc.KVC_EINVAL
    assert rotate(kvc, rope=0) == E
    for bad in BAD_ROPES:
        assert rotate(kvc, rope_kw=bad) == E, bad
    for bad in (dict(dtype=3), dict(dtype=-1), dict(n_rows=-1), dict(n_head_q=0), dict(n_head_kv=-1), dict(head_dim=48),
                dict(head_dim=0), dict(head_dim=288, ld_q=4096, ld_k=4096, ld_qo=4096, ld_ko=4096), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(ld_q=248), dict(ld_q=260), dict(ld_k=120),
                dict(ld_qo=-256), dict(ld_ko=132), dict(q=0), dict(k=0), dict(pos=0), dict(q_out=0), dict(k_out=0),
                dict(q=FAKE + 8), dict(k=FAKE + 2), dict(q_out=FAKE + 4), dict(k_out=FAKE + 8), dict(q_weight=FAKE + 1),
                dict(k_weight=FAKE + 1, dtype=2), dict(n_head_q=65535, n_head_kv=1, ld_q=1 << 23, ld_qo=1 << 23)):
        assert rotate(kvc, **bad) == E, bad
    assert rotate(kvc, n_rows=0) == 0
    assert rotate(kvc, n_rows=0, rope_kw=dict(n_pairs=0, turns=0)) == 0
    assert rotate(kvc, n_rows=0, rope_kw=dict(n_pairs=13, style=1)) == 0


def test_rope_append_refusals(kvc):
    E = kvc.KVC_EINVAL
    f = lambda **kw: rotate_append(kvc, **kw)
    assert f(pool=0) == E and f(pages=0) == E and f(rope=0) == E
    for bad in BAD_ROPES:
        assert f(rope_kw=bad) == E, bad
    for bad in (dict(page_size=24), dict(page_size=48), dict(n_seq=65536), dict(table=0), dict(len=0)):
        assert f(pages_kw=bad) == E, bad
    for bad in (dict(layer=-1), dict(layer=2)):
        assert f(**bad) == kvc.KVC_ERANGE, bad
    for bad in (dict(dtype=3), dict(n_rows=-1), dict(n_head_q=0), dict(eps=-0.5), dict(ld_q=248), dict(ld_k=120),
                dict(ld_v=132), dict(ld_qo=252), dict(row_start=0), dict(q=0), dict(k=0), dict(v=0), dict(q_out=0),
                dict(v=FAKE + 8), dict(q_out=FAKE + 2), dict(n_head_q=65532, ld_q=1 << 23, ld_qo=1 << 23)):
        assert f(**bad) == E, bad
    assert f(pool_kw=dict(head_dim=288), ld_q=8192, ld_k=8192, ld_v=8192, ld_qo=8192) == E
    assert f(n_rows=0) == 0 and f(pages_kw=dict(n_seq=0)) == 0


def test_binding_refuses_tensors_it_cannot_pass(kvc):
    x, rope = torch.zeros(4, 2, 64), kvc.RopeTable(64, device="cpu")
    with pytest.raises(ValueError):
        kvc.qk_norm_rope(x, x, torch.zeros(4, dtype=torch.int32), rope)      # not on a GPU
    with pytest.raises(ValueError):
        kvc.qk_norm_rope(x[0], x, torch.zeros(4, dtype=torch.int32), rope)


def test_pools_of_4_bits_with_too_many_heads_for_decode(kvc):
    b = ctypes.c_size_t()
    for heads, want in ((65535, 0), (65536, kvc.KVC_EINVAL)):
        d = kvc.make_desc(1, 16, heads, 64, "q4_0")
        assert kvc.lib.kvc_paged_scratch_bytes(ctypes.byref(d), 1, heads, ctypes.byref(b)) == want


def test_tensors_that_calls_hold_cannot_be_replaced(kvc):
    free, rope = kvc.FreePages(4, device="cpu"), kvc.RopeTable(16, device="cpu")
    for x, names in ((free, ("ring", "state", "n_pages", "c")), (rope, ("turns", "rot", "style"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(x, name, getattr(x, name))
    free.state[1] = 2
    assert free.free() == (2, 0)
