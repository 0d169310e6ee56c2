"""The operators of the paged cache and of packed prompts: cases, inputs, plain forms and what each pass has to move.

A serving step keeps the keys and values of many sequences in one cache whose positions are cut into pages; a
table gives each sequence its pages in order.  Prompts of different lengths lie one after another ("packed") in
one tensor, row_start giving the first row of each.  Four operators work on these:

  append  quantise (q8_0) or round (f16) new rows and store them on their sequences' pages
  read    the rows back from the pages, dequantised and packed
  decode  attention of one new token for each sequence over its pages
  packed  causal attention of packed prompts with grouped heads; each may have a cached prefix in front

`run` with own = False is the plain form in elementary torch operations; with own = True it calls the package.
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases ----------------------------------------------------------------------------------------

def listed():
    full = {"heads_q": 40, "heads_kv": 8, "head_dim": 128}
    small = {"heads_q": 16, "heads_kv": 4, "head_dim": 64}
    return [
        # a decode step of eight parallel sequences at 2k context stores one token each: pure latency
        {"name": "append_f16_step8", "op": "append", "cache": "f16", "layout": "head_major", "page": 16, "dtype": "bf16",
         "n_seq": 8, "shortest": 2048, "longest": 2176, "new": 1, "shape": 1, **full},
        # a batch of prompts of different lengths enters an f16 cache in one call
        {"name": "append_f16_prompts", "op": "append", "cache": "f16", "layout": "layer_major", "page": 64,
         "dtype": "f16", "n_seq": 6, "shortest": 700, "longest": 5000, "new": 0, "shape": 2, **full},
        # a decode step of 64 sequences into a q8_0 cache, and the stored rows read back
        {"name": "store_q8_step64", "op": "store", "cache": "q8_0", "layout": "layer_major", "page": 32, "dtype": "bf16",
         "out": "f16", "n_seq": 64, "shortest": 33, "longest": 4100, "new": 1, "shape": 3, **full},
        # packed prompts into a q8_0 cache, read back as the attention over them reads them
        {"name": "store_q8_prompts", "op": "store", "cache": "q8_0", "layout": "head_major", "page": 64, "dtype": "bf16",
         "out": "f16", "n_seq": 9, "shortest": 1023, "longest": 4100, "new": 0, "shape": 4, **full},
        # the cached context of a prompt that continues, 58,300 positions, unpacked for its attention
        {"name": "read_q8_58k", "op": "read", "cache": "q8_0", "layout": "head_major", "page": 64, "dtype": "bf16",
         "out": "bf16", "n_seq": 1, "shortest": 58300, "longest": 58300, "new": 0, "shape": 5, **full},
        # short sequences with small heads from an f16 cache of small pages
        {"name": "read_f16_short", "op": "read", "cache": "f16", "layout": "layer_major", "page": 16, "dtype": "f16",
         "out": "f32", "n_seq": 12, "shortest": 1, "longest": 700, "new": 0, "shape": 6, **small},
        # eight parallel sequences at 2k context, f16 cache
        {"name": "decode_f16_npl8", "op": "decode", "cache": "f16", "layout": "head_major", "page": 16, "dtype": "bf16",
         "n_seq": 8, "shortest": 2048, "longest": 2176, "new": 1, "shape": 7, **full},
        # one long conversation: a single token over 58,300 positions
        {"name": "decode_q8_58k", "op": "decode", "cache": "q8_0", "layout": "head_major", "page": 64, "dtype": "bf16",
         "n_seq": 1, "shortest": 58300, "longest": 58300, "new": 1, "shape": 8, **full},
        # a full serving batch, lengths from a few tokens to 16k
        {"name": "decode_q8_batch96", "op": "decode", "cache": "q8_0", "layout": "layer_major", "page": 32, "dtype": "f16",
         "n_seq": 96, "shortest": 5, "longest": 16384, "new": 1, "shape": 9, **full},
        # many short prompts at once, some of a single token
        {"name": "packed_short48", "op": "packed", "dtype": "bf16", "n_seq": 48, "shortest": 1, "longest": 513, "new": 0,
         "shape": 10, **full},
        # one long prompt, whole
        {"name": "packed_10041", "op": "packed", "dtype": "bf16", "n_seq": 1, "shortest": 10041, "longest": 10041,
         "new": 0, "shape": 11, **full},
        # 512-token chunks of four prompts over the prefixes they already have, small heads
        {"name": "packed_chunk512", "op": "packed", "dtype": "f16", "n_seq": 4, "shortest": 2500, "longest": 9000,
         "new": 512, "shape": 12, **small},
    ]


def _log_between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "store", "read", "decode", "decode", "packed", "packed"])
    hq, hkv = rng.choice([(40, 8), (40, 8), (16, 4), (10, 2), (8, 8), (4, 2), (24, 3)])
    c = {"op": op, "heads_q": hq, "heads_kv": hkv, "head_dim": rng.choice([64, 128, 128]),
         "dtype": rng.choice(["bf16", "f16"]), "shape": rng.randrange(1 << 30)}
    if op != "packed":
        c["cache"] = "f16" if op == "append" else "q8_0" if op == "store" else rng.choice(["q8_0", "f16"])
        c["layout"] = rng.choice(["head_major", "layer_major"])
        c["page"] = rng.choice([16, 32, 48, 64, 128])
    if op in ("store", "read"):
        c["out"] = rng.choice(["bf16", "f16", "f32"])
    budget = {"append": 16000, "store": 16000, "read": 50000, "decode": 200000, "packed": 8000}[op]
    c["n_seq"] = _log_between(rng, 1, 96)
    longest = _log_between(rng, 8, 16384 if op != "packed" else 6000)
    c["longest"] = max(2, min(longest, budget // c["n_seq"]))
    c["shortest"] = rng.choice([1, max(1, c["longest"] // 2), c["longest"]])
    c["new"] = 1 if op == "decode" else rng.choice([0, 1, rng.randint(1, max(1, c["longest"] // 2))])
    return c


def lengths(case):
    """(tokens held, rows of this call) of each sequence; new = 0: all of them are rows of this call."""
    rng = random.Random(case["shape"])
    held = [_log_between(rng, case["shortest"], case["longest"]) for _ in range(case["n_seq"])]
    held[rng.randrange(len(held))] = case["longest"]
    return held, [min(n, case["new"]) if case["new"] else n for n in held]


# ---- inputs ---------------------------------------------------------------------------------------

def _starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


def _keys(gen, n, hkv, d):
    """Keys of n tokens: N(0, 1), one channel in a hundred four times as large."""
    k = torch.randn(n, hkv, d, generator=gen, device="cuda")
    wide = torch.randperm(hkv * d, generator=gen, device="cuda")[: max(1, hkv * d // 100)]
    k.view(n, hkv * d)[:, wide] *= 4
    return k


def _q8(x):
    """q8_0: codes and fp16 scales of blocks of 32 values of the last axis."""
    b = x.float().unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 127.0
    r = torch.where(d > 0, b / d, torch.zeros((), device=x.device)).double()  # in 64 bits |r| + 0.5 is exact
    q = torch.sign(r) * torch.floor(r.abs() + 0.5)
    return q.to(torch.int8).flatten(-2), d.squeeze(-1).half()


def _by_token(t, layout):
    """A pool buffer as [position][head][...]."""
    return t[:, 0].transpose(0, 1) if layout == "head_major" else t[0]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    held, rows = lengths(case)
    n, hq, hkv, d = case["n_seq"], case["heads_q"], case["heads_kv"], case["head_dim"]
    dt = DT[case["dtype"]]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    s = dict(case, held=i32(held), row_start=i32(_starts(rows)), n_rows=sum(rows), longest_row=max(rows),
             longest_held=max(held))
    if case["op"] == "packed":
        s["q"] = torch.randn(sum(rows), hq, d, generator=gen, device="cuda").to(dt)
        s["k"] = _keys(gen, sum(held), hkv, d).to(dt)
        s["v"] = torch.randn(sum(held), hkv, d, generator=gen, device="cuda").to(dt)
        s["k_start"] = i32(_starts(held))
        if own:
            import decode_attention_kv_cache_gb300 as kvc
            s["scratch"] = kvc.packed_scratch(sum(rows), n, hq, hkv, d, device="cuda")
        return s
    page = case["page"]
    used = [-(-h // page) for h in held]
    n_pages = sum(used) + 3  # a few pages belong to nobody
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(n, max(used), dtype=torch.int32, device="cuda")
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    s["table"] = table
    positions = n_pages * page
    quant = case["cache"] == "q8_0"
    if own:
        import decode_attention_kv_cache_gb300 as kvc
        cache = kvc.KVCache(1, positions, hkv, d, case["cache"], case["layout"])
        s["cache"] = cache
        s["pages"] = kvc.PageTable(table, s["held"], page)
        pool = [cache.codes(0), cache.codes(1), cache.scales(0), cache.scales(1)]
        if case["op"] == "decode":
            s["scratch"] = kvc.paged_scratch(cache, n, hq)
    else:
        dims = (hkv, 1, positions) if case["layout"] == "head_major" else (1, positions, hkv)
        pool = [torch.empty(*dims, d, dtype=torch.int8 if quant else torch.float16, device="cuda") for _ in (0, 1)]
        pool += [torch.empty(*dims, d // 32, dtype=torch.float16, device="cuda") if quant else None for _ in (0, 1)]
    for kv in (0, 1):
        x = _keys(gen, positions, hkv, d) if kv == 0 else torch.randn(positions, hkv, d, generator=gen, device="cuda")
        x = x.to(dt)
        if quant:
            q, sc = _q8(x)
            _by_token(pool[kv], case["layout"]).copy_(q)
            _by_token(pool[2 + kv], case["layout"]).copy_(sc)
        else:
            _by_token(pool[kv], case["layout"]).copy_(x)
        del x
    s["pool"] = pool
    if case["op"] in ("append", "store"):
        s["k"] = _keys(gen, s["n_rows"], hkv, d).to(dt)
        s["v"] = torch.randn(s["n_rows"], hkv, d, generator=gen, device="cuda").to(dt)
    if case["op"] == "decode":
        s["q"] = torch.randn(n, hq, d, generator=gen, device="cuda").to(dt)
    return s


# ---- one pass -------------------------------------------------------------------------------------

def _slots(s):
    """The pool position of each packed row."""
    row = torch.arange(s["n_rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["row_start"], row, right=True) - 1
    pos = s["held"][seq] - s["row_start"][seq + 1] + row
    return s["table"][seq, (pos // s["page"]).long()].long() * s["page"] + pos % s["page"]


def _values(s, kv, slots):
    """What the pool holds for K (0) or V (1) at `slots`, in 32 bits: [..., head, value]."""
    x = _by_token(s["pool"][kv], s["layout"])[slots].float()
    if s["cache"] == "q8_0":
        scale = _by_token(s["pool"][2 + kv], s["layout"])[slots].float()
        x = (x.unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)
    return x


def _store(s):
    slots = _slots(s)
    for kv, x in ((0, s["k"]), (1, s["v"])):
        if s["cache"] == "q8_0":
            q, d = _q8(x)
            _by_token(s["pool"][kv], s["layout"])[slots] = q
            _by_token(s["pool"][2 + kv], s["layout"])[slots] = d
        else:
            _by_token(s["pool"][kv], s["layout"])[slots] = x.half()


def _read(s):
    slots = _slots(s)
    return tuple(_values(s, kv, slots).to(DT[s["out"]]) for kv in (0, 1))


def _weights(scores, seen):
    scores = torch.where(seen, scores, torch.full((), -math.inf, device="cuda"))
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _decode(s):
    n, hkv, d = s["n_seq"], s["heads_kv"], s["head_dim"]
    pos = torch.arange(s["longest_held"], device="cuda", dtype=torch.int32)
    pages = s["table"][:, (pos // s["page"]).long()].long()
    slots = pages * s["page"] + pos % s["page"]
    q = s["q"].float().view(n, hkv, -1, d)
    scores = torch.matmul(q, _values(s, 0, slots).permute(0, 2, 3, 1)) / math.sqrt(d)
    p = _weights(scores, (pos < s["held"][:, None])[:, None, None, :])
    out = torch.matmul(p, _values(s, 1, slots).transpose(1, 2))
    return out.reshape(n, -1, d).to(s["q"].dtype)


def _packed(s):
    n, hq, hkv, d = s["n_seq"], s["heads_q"], s["heads_kv"], s["head_dim"]
    qs, ks = s["row_start"], s["k_start"]
    nq, nk = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    i = torch.arange(s["longest_row"], device="cuda", dtype=torch.int32)
    j = torch.arange(s["longest_held"], device="cuda", dtype=torch.int32)
    # the sequences side by side, each padded to the longest with some other row
    qi = (qs[:-1, None] + i).clamp(max=s["n_rows"] - 1).long()
    kj = (ks[:-1, None] + j).clamp(max=s["k"].shape[0] - 1).long()
    q = s["q"][qi].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4)
    k = s["k"][kj].float().permute(0, 2, 3, 1).unsqueeze(2)
    v = s["v"][kj].float().permute(0, 2, 1, 3).unsqueeze(2)
    scores = torch.matmul(q, k) / math.sqrt(d)
    last = i[None, :] + (nk - nq)[:, None]          # the last key that row i sees
    p = _weights(scores, (j <= last[:, :, None])[:, None, None])
    del scores
    o = torch.matmul(p, v).permute(0, 3, 1, 2, 4).reshape(n, s["longest_row"], hq, d).to(s["q"].dtype)
    row = torch.arange(s["n_rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(qs, row, right=True) - 1
    return o[seq, (row - qs[seq]).long()]


def run(s):
    op = s["op"]
    if own:
        import decode_attention_kv_cache_gb300 as kvc
        if op == "packed":
            return kvc.attn_packed(s["q"], s["k"], s["v"], s["row_start"], s["k_start"], scratch=s["scratch"])
        if op == "decode":
            return kvc.decode_attn_paged(s["cache"], 0, s["pages"], s["q"], scratch=s["scratch"])
        if op in ("append", "store"):
            kvc.kv_paged_append(s["cache"], 0, s["pages"], s["row_start"], s["k"], s["v"])
        if op == "append":
            return s["pool"][0], s["pool"][1]
        return kvc.kv_paged_read(s["cache"], 0, s["pages"], s["row_start"], s["n_rows"], dtype=DT[s["out"]])
    if op == "packed":
        return _packed(s)
    if op == "decode":
        return _decode(s)
    if op in ("append", "store"):
        _store(s)
    if op == "append":
        return s["pool"][0], s["pool"][1]
    return _read(s)


# ---- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    held, rows = lengths(case)
    hq, hkv, d = case["heads_q"], case["heads_kv"], case["head_dim"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    row_in, row_q = hkv * d * size[case["dtype"]], hq * d * size[case["dtype"]]
    if case["op"] == "packed":
        pairs = sum(r * (h - r) + r * (r + 1) // 2 for h, r in zip(held, rows))
        return {"bytes": 2 * sum(rows) * row_q + 2 * sum(held) * row_in, "flops": 4 * hq * d * pairs}
    row_pool = hkv * (d * 2 if case["cache"] == "f16" else d + d // 32 * 2)
    if case["op"] == "decode":
        return {"bytes": 2 * sum(held) * row_pool + 2 * len(held) * row_q, "flops": 4 * hq * d * sum(held)}
    n, values = sum(rows), sum(rows) * hkv * d * 2
    if case["op"] == "append":
        return {"bytes": 2 * n * (row_in + row_pool), "flops": values}
    row_out = hkv * d * size[case["out"]]
    if case["op"] == "read":
        return {"bytes": 2 * n * (row_pool + row_out), "flops": values}
    return {"bytes": 2 * n * (row_in + 2 * row_pool + row_out), "flops": 5 * values}


# ---- the same from the definitions, in 64 bits ----------------------------------------------------

def _places(case, s):
    """For each sequence the pool positions of its tokens, in order (host)."""
    table, page = s["table"].cpu().tolist(), case["page"]
    held, rows = lengths(case)
    return [[table[i][p // page] * page + p % page for p in range(h)] for i, h in enumerate(held)], rows


def _held64(case, s, kv, places):
    at = torch.tensor(places, device="cuda", dtype=torch.long)
    pick = (lambda t: t[:, 0, at].permute(1, 0, 2)) if case["layout"] == "head_major" else (lambda t: t[0, at])
    x = pick(s["pool"][kv]).double()
    if case["cache"] == "q8_0":
        x = x * pick(s["pool"][2 + kv]).double().repeat_interleave(32, dim=-1)
    return x


def _attend64(q, k, v, first):
    """Rows q [r][g][d] over k, v [n][d]; row i sees the keys up to first + i."""
    r, g, d = q.shape
    z = torch.einsum("rgd,nd->grn", q, k) * d ** -0.5
    late = torch.arange(k.shape[0], device="cuda")[None, :] > first + torch.arange(r, device="cuda")[:, None]
    z.masked_fill_(late, -math.inf)
    return torch.einsum("grn,nd->rgd", torch.softmax(z, dim=-1), v)


def exact(case, seed):
    s = prepare(case, seed)
    held, rows = lengths(case)
    hq, hkv, d = case["heads_q"], case["heads_kv"], case["head_dim"]
    g, op = hq // hkv, case["op"]
    if op == "packed":
        out, a, b = [], 0, 0
        for h, r in zip(held, rows):
            q, k, v = s["q"][a:a + r].double(), s["k"][b:b + h].double(), s["v"][b:b + h].double()
            out.append(torch.cat([_attend64(q[:, i * g:(i + 1) * g], k[:, i], v[:, i], h - r) for i in range(hkv)], 1))
            a, b = a + r, b + h
        return torch.cat(out)
    places, _ = _places(case, s)
    if op == "decode":
        out = []
        for i, at in enumerate(places):
            q, k, v = s["q"][i:i + 1].double(), _held64(case, s, 0, at), _held64(case, s, 1, at)
            out.append(torch.cat([_attend64(q[:, j * g:(j + 1) * g], k[:, j], v[:, j], len(at)) for j in range(hkv)], 1))
        return torch.cat(out)
    mine = [p for at, r in zip(places, rows) for p in at[len(at) - r:]]
    if op == "read":
        return tuple(_held64(case, s, kv, mine) for kv in (0, 1))
    if op == "append":
        at = torch.tensor(mine, device="cuda", dtype=torch.long)
        pool = [t.double() for t in s["pool"][:2]]
        for kv, x in ((0, s["k"]), (1, s["v"])):
            if case["layout"] == "head_major":
                pool[kv][:, 0, at] = x.double().transpose(0, 1)
            else:
                pool[kv][0, at] = x.double()
        return tuple(pool)
    out = []
    for x in (s["k"], s["v"]):  # the format's own steps: amax / 127 and x / d are rounded to 32 bits, d is stored as fp16
        b = x.float().cpu().numpy().reshape(-1, 32)
        d32 = np.abs(b).max(axis=1, keepdims=True) / np.float32(127)
        y = (b / np.maximum(d32, np.float32(1e-38))).astype("f8")
        codes = np.copysign(np.floor(np.abs(y) + 0.5), y)
        out.append(torch.from_numpy(codes * d32.astype("f2").astype("f8")).reshape(-1, hkv, d))
    return tuple(out)
