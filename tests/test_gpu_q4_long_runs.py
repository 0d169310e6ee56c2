"""decode_attn_paged over q4_0 where a warp attends to many thousands of keys by itself, and over long single contexts, against
64 bits with pool4_close's bound: sums that cancel, or a tile lost where runs meet, would show."""

import pytest
import torch

from paged_util import TYPES, i32, inputs, starts
from pool4_close import attend_close, check_close
from pool4_util import codes4, make_pool4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def shared_pool(kvc, n_seq, n, hkv, d, layout, one_sign, seed):
    """n_seq sequences over the same n keys, each with the pages in an order of its own (they are only read)."""
    page = 64
    cache = kvc.KVCache(1, n, hkv, d, "q4_0", layout)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(n, hkv, d, generator=g, device="cuda") for _ in (0, 1))
    if one_sign:
        v[..., ::32] = 2.5 + 0.5 * v[..., ::32].abs()   # the greatest of each block, as a channel that stands out is
    table = torch.stack([torch.randperm(n // page, generator=g, device="cuda") for _ in range(n_seq)]).to(torch.int32)
    pages = kvc.PageTable(table, i32([n] * n_seq), page)
    whole = kvc.PageTable(torch.arange(n // page, device="cuda", dtype=torch.int32)[None], i32([n]), page)
    kvc.kv_paged_append(cache, 0, whole, starts([n]), k, v)
    return cache, pages


RUNS = [  # dtype, hq, hkv, d, n_seq, n: as many sequences as there are runs on 152 SMs, or a multiple
    ("f32", 8, 4, 128, 456, 16384),
    ("f16", 4, 4, 128, 456, 16384),
    ("bf16", 8, 4, 128, 456, 16384),
    ("f32", 48, 4, 128, 304, 8192),     # 12 heads to a group
    ("bf16", 64, 4, 64, 304, 16384),
    ("f16", 20, 4, 64, 456, 8192),
    ("f32", 1, 1, 128, 1824, 16384),
    ("f16", 4, 4, 128, 456, 65536),
]


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("dtype,hq,hkv,d,n_seq,n", RUNS)
def test_a_warp_attends_to_whole_sequences(kvc, dtype, hq, hkv, d, n_seq, n, one_sign):
    cache, pages = shared_pool(kvc, n_seq, n, hkv, d, "layer_major", one_sign, hq + n_seq)
    q = inputs((n_seq, hq, d), torch.float16, 3).to(TYPES[dtype])   # 11 bits: nothing of a query is rounded
    lse = torch.empty(n_seq, hq, device="cuda")
    out = kvc.decode_attn_paged(cache, 0, pages, q, lse=lse)
    (k, dk), (v, dv) = (codes4(cache, 0, kv, list(range(n))) for kv in (0, 1))
    some = torch.arange(0, n_seq, max(1, n_seq * hq * n // (1 << 24)), device="cuda")
    want, dev, rest, l, off = attend_close(q[some], k, dk, v, dv, roundings=2 if dtype == "bf16" else 1)
    check_close(out[some], want, dev, rest, "out")
    assert ((lse[some].double() - l).abs() <= off).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("held", [[20000], [58300], [20011, 333, 7000, 12, 40000], [9000] * 7 + [1]])
def test_long_contexts_lose_nothing_where_runs_meet(kvc, dtype, held):
    hq, hkv, d = 10, 2, 128
    cache, pages, slots = make_pool4(kvc, held, 16, hkv, d, "layer_major", seed=len(held), layers=1)
    q = inputs((len(held), hq, d), torch.float16, 4).to(TYPES[dtype])
    out = kvc.decode_attn_paged(cache, 0, pages, q)
    for i, sl in enumerate(slots):
        (k, dk), (v, dv) = (codes4(cache, 0, kv, sl) for kv in (0, 1))
        want, dev, rest, _, _ = attend_close(q[i:i + 1], k, dk, v, dv, roundings=2 if dtype == "bf16" else 1)
        check_close(out[i:i + 1], want, dev, rest, "seq %d" % i)
    assert torch.equal(out, kvc.decode_attn_paged(cache, 0, pages, q))
