"""Refusals of the paged and packed calls, and their size queries: nothing here reaches a GPU."""

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
    d = dict(n_layer=2, n_ctx=512, n_head_kv=2, head_dim=64, cache_type="q8_0", layout="head_major")
    d.update(kw)
    c = kvc.kvc_cache()
    desc = kvc.make_desc(*d.values())
    assert kvc.lib.kvc_cache_init(ctypes.byref(c), ctypes.byref(desc), FAKE, FAKE, FAKE, FAKE) == 0
    return c


def pages(kvc, **kw):
    p = dict(table=FAKE, len=FAKE, n_seq=3, max_pages=8, page_size=16)
    p.update(kw)
    return kvc.kvc_pages(*p.values())


APPEND = dict(pool=None, pages=None, layer=0, row_start=FAKE, n_rows=4, k=FAKE, v=FAKE, ld_k=128, ld_v=128, dtype=1)
READ = dict(pool=None, pages=None, layer=0, row_start=FAKE, n_rows=4, k=FAKE, v=FAKE, dtype=1)
DECODE = dict(pool=None, pages=None, layer=0, q=FAKE, ld_q=256, dtype=1, n_head_q=4, out=FAKE, lse=0, scratch=FAKE,
              scratch_bytes=1 << 40)
PACKED = dict(q=FAKE, k=FAKE, v=FAKE, ld_q=256, ld_k=128, ld_v=128, dtype=1, q_start=FAKE, k_start=FAKE, n_seq=3,
              n_q=9, n_k=9, n_head_q=4, n_head_kv=2, head_dim=64, out=FAKE, lse=0, scratch=FAKE, scratch_bytes=1 << 40)


def call(kvc, name, args, pool_kw=(), pages_kw=(), **kw):
    a = dict(args, **kw)
    if "pool" in a:
        a["pool"] = ctypes.byref(pool(kvc, **dict(pool_kw))) if a["pool"] is None else None
        a["pages"] = ctypes.byref(pages(kvc, **dict(pages_kw))) if a["pages"] is None else None
    return getattr(kvc.lib, name)(*a.values(), None)


PAGED = [("kv_paged_append", APPEND), ("kv_paged_read", READ), ("decode_attn_paged", DECODE)]


@pytest.mark.parametrize("name,args", PAGED)
def test_paged_refusals(kvc, name, args):
    E, R = kvc.KVC_EINVAL, kvc.KVC_ERANGE
    assert call(kvc, name, args, pool=0) == E and call(kvc, name, args, pages=0) == E
    for bad in (dict(page_size=0), dict(page_size=-16), dict(page_size=24), dict(page_size=48), dict(n_seq=-1),
                dict(n_seq=65536), dict(max_pages=0), dict(max_pages=(1 << 31) - 1), dict(table=0), dict(len=0)):
        assert call(kvc, name, args, pages_kw=bad) == E, bad
    for bad in (dict(layer=-1), dict(layer=2)):
        assert call(kvc, name, args, **bad) == R, bad
    assert call(kvc, name, args, dtype=3) == E and call(kvc, name, args, dtype=-1) == E
    for p in ("row_start", "k", "v", "q", "out", "scratch"):
        if p in args:
            assert call(kvc, name, args, **{p: 0}) == E, p
            if p != "row_start":
                assert call(kvc, name, args, **{p: FAKE + 8}) == E, p
    for ld in ("ld_k", "ld_v", "ld_q"):
        if ld in args:
            for bad in (0, -128, args[ld] - 8, args[ld] + 4, 1 << 40):
                assert call(kvc, name, args, **{ld: bad}) == E, (ld, bad)
    if "n_rows" in args:
        assert call(kvc, name, args, n_rows=-1) == E
        assert call(kvc, name, args, n_rows=0) == kvc.KVC_OK
    assert call(kvc, name, args, pages_kw=dict(n_seq=0)) == kvc.KVC_OK


def test_decode_refusals(kvc):
    f = lambda **kw: call(kvc, "decode_attn_paged", DECODE, **kw)
    for hq in (0, -2, 3, 34):
        assert f(n_head_q=hq, ld_q=4096) == kvc.KVC_EINVAL, hq
    assert f(pool_kw=dict(head_dim=96)) == kvc.KVC_EINVAL
    n = ctypes.c_size_t()
    desc = kvc.make_desc(2, 512, 2, 64, "q8_0", "head_major")
    assert kvc.lib.kvc_paged_scratch_bytes(ctypes.byref(desc), 3, 4, ctypes.byref(n)) == 0 and n.value > 0
    assert f(scratch_bytes=n.value - 1) == kvc.KVC_ENOSPC
    for bad in ((-1, 4), (65536, 4), (3, 0), (3, 3), (3, 34)):
        assert kvc.lib.kvc_paged_scratch_bytes(ctypes.byref(desc), *bad, ctypes.byref(n)) == kvc.KVC_EINVAL
    assert kvc.lib.kvc_paged_scratch_bytes(None, 3, 4, ctypes.byref(n)) == kvc.KVC_EINVAL


def test_packed_refusals(kvc):
    E = kvc.KVC_EINVAL
    f = lambda **kw: call(kvc, "attn_packed", PACKED, **kw)
    for bad in (dict(dtype=0), dict(dtype=3), dict(head_dim=32), dict(head_dim=96), dict(n_head_q=3), dict(n_head_q=0),
                dict(n_head_kv=0), dict(n_head_q=65536), dict(n_head_q=258, ld_q=258 * 64), dict(n_seq=-1), dict(n_seq=65536), dict(n_q=-1),
                dict(n_k=-1), dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(scratch=0), dict(q_start=0),
                dict(k_start=0), dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(out=FAKE + 8),
                dict(scratch=FAKE + 8), dict(ld_q=248), dict(ld_q=260), dict(ld_k=120), dict(ld_v=132), dict(ld_v=-128)):
        assert f(**bad) == E, bad
    n = ctypes.c_size_t()
    assert kvc.lib.kvc_packed_scratch_bytes(9, 3, 4, 2, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert f(scratch_bytes=n.value - 1) == kvc.KVC_ENOSPC
    assert f(n_q=0) == 0 and f(n_seq=0) == 0


def test_binding_refuses_tensors_it_cannot_pass(kvc):
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kvc.PageTable(t, torch.zeros(2, dtype=torch.int32), 16)      # not on the GPU
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kvc.attn_packed(x, x, x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvc.attn_packed(x.float(), x.float(), x.float(), torch.zeros(2, dtype=torch.int32))
