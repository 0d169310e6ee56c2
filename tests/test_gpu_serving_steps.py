"""Pages, norms with rotation, 4-bit stores and attention together, as a serving loop uses them: several scheduler
steps, each checked against the formulas in 64 bits on what the step before has left."""

import pytest
import torch

from oracle import q4_0
from paged_util import check, i32, inputs
from pool4_util import codes4, attend4
from test_gpu_rope import check as check_rope, expect, freqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


@pytest.mark.parametrize("layout,hq,hkv,d", [("layer_major", 10, 2, 128), ("head_major", 16, 4, 64)])
def test_prompts_tokens_rewinds_and_ends(kvc, layout, hq, hkv, d):
    n_seq, page, n_pages, t = 4, 16, 40, torch.bfloat16
    pool = kvc.KVCache(2, n_pages * page, hkv, d, "q4_0", layout)
    pages = kvc.PageTable(torch.full((n_seq, 16), -1, dtype=torch.int32, device="cuda"), i32([0] * n_seq), page)
    free, rope = kvc.FreePages(n_pages), kvc.RopeTable(d, 1e5)
    qw, kw = ((1 + inputs((d,), torch.float32, s, 0.3)).to(t) for s in (3, 4))
    scratch = kvc.paged_scratch(pool, n_seq, hq)
    held = {i: [] for i in range(n_seq)}         # each sequence's rotated keys and values, as rounded, in order
    steps = [[70, 0, 33, 1], [1, 90, 1, 1], [1, 1, 1, 1], [-3, 1, -2 ** 31, 1], [1, 1, 50, 1], [1, 1, 1, 1]]
    for step, rows in enumerate(steps):
        n = sum(max(r, 0) for r in rows)
        start, pos, slots = kvc.kv_pages_advance(pages, free, i32(rows), n)
        qkv = inputs((n, hq + 2 * hkv, d), t, 100 + step)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        qo = kvc.qk_norm_rope_append(pool, 1, pages, start, q, k, v, rope, qw, kw, 1e-5)
        check_rope(qo, *expect(q, pos, d, "half", qw, freqs(d, 1e5), 1e-5), "step %d queries" % step)
        _, ko = kvc.qk_norm_rope(q, k, pos, rope, qw, kw, 1e-5)
        check_rope(ko, *expect(k, pos, d, "half", kw, freqs(d, 1e5), 1e-5), "step %d keys" % step)
        for i, r in enumerate(rows):
            held[i] = held[i][:max(len(held[i]) + r, 0)] if r < 0 else held[i]
            for x in range(max(r, 0)):
                held[i].append((ko[start[i] + x].float().cpu().numpy(), v[start[i] + x].float().cpu().numpy()))
        assert pages.lengths.tolist() == [len(held[i]) for i in range(n_seq)]
        assert free.free()[1] == 0
        last = torch.empty(n_seq, hq, d, dtype=t, device="cuda")
        for i in range(n_seq):                   # a query of each sequence, whether or not it has new rows
            last[i] = qo[start[i + 1] - 1] if rows[i] > 0 else inputs((hq, d), t, 7 * step + i)
        out = kvc.decode_attn_paged(pool, 1, pages, last, scratch=scratch)
        table = pages.table.tolist()
        for i in range(n_seq):
            at = [table[i][p // page] * page + p % page for p in range(len(held[i]))]
            (kc, dk), (vc, dv) = (codes4(pool, 1, kv, at) for kv in (0, 1))
            for kv, (codes, scales) in enumerate(((kc, dk), (vc, dv))):
                for p, row in enumerate(held[i]):    # what the pages hold is what was stored, wherever it lies
                    d_h, c = q4_0.quantize_blocks(row[kv])
                    assert (codes[p].cpu().numpy() == c).all() and (scales[p].cpu().numpy() == d_h).all(), (step, i, p)
            k64, v64 = kc * dk.repeat_interleave(32, -1), vc * dv.repeat_interleave(32, -1)
            o, _, b, _ = attend4(last[i], k64, dk, v64, dv)
            check(out[i], o, b, "step %d seq %d" % (step, i))
    kvc.kv_pages_advance(pages, free, i32([-2 ** 31] * n_seq), 0)
    assert free.free() == (n_pages, 0)


def test_captured_decode_loop(kvc):
    # one graph: advance by a token, normalise, rotate and store, attend; replayed over page borders
    n_seq, page, hq, hkv, d, t = 3, 16, 8, 2, 128, torch.bfloat16
    pool = kvc.KVCache(1, 30 * page, hkv, d, "q4_0", "layer_major")
    pages = kvc.PageTable(torch.full((n_seq, 8), -1, dtype=torch.int32, device="cuda"), i32([0] * n_seq), page)
    free, rope, w = kvc.FreePages(30), kvc.RopeTable(d), torch.ones(d, dtype=t, device="cuda")
    prompt = [14, 31, 1]
    start, pos, _ = kvc.kv_pages_advance(pages, free, i32(prompt), sum(prompt))
    x = inputs((sum(prompt), hq + 2 * hkv, d), t, 1)
    kvc.qk_norm_rope_append(pool, 0, pages, start, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], rope, w, w)
    y, ones = torch.empty(n_seq, hq + 2 * hkv, d, dtype=t, device="cuda"), i32([1] * n_seq)
    scratch, out = kvc.paged_scratch(pool, n_seq, hq), torch.empty(n_seq, hq, d, dtype=t, device="cuda")

    def step():
        rs, _, _ = kvc.kv_pages_advance(pages, free, ones, n_seq)
        q = kvc.qk_norm_rope_append(pool, 0, pages, rs, y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], rope, w, w)
        kvc.decode_attn_paged(pool, 0, pages, q, out=out, scratch=scratch)
        return q

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            q = step()
    for i in range(5):
        y.copy_(inputs((n_seq, hq + 2 * hkv, d), t, 50 + i))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert pages.lengths.tolist() == [p + i + 1 for p in prompt]
        table = pages.table.tolist()
        for j in range(n_seq):
            at = [table[j][p // page] * page + p % page for p in range(prompt[j] + i + 1)]
            (kc, dk), (vc, dv) = (codes4(pool, 0, kv, at) for kv in (0, 1))
            o, _, b, _ = attend4(q[j], kc * dk.repeat_interleave(32, -1), dk, vc * dv.repeat_interleave(32, -1), dv)
            check(out[j], o, b, "replay %d seq %d" % (i, j))
    assert free.free() == (30 - sum(-(-(p + 5) // page) for p in prompt), 0)
