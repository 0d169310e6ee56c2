"""More operators of a serving step over a paged cache: cases, inputs, plain forms and what each pass has to move.

  pages   the page table, positions and slots of the packed rows, from the sequences' new rows, on the device: lengths
          advance (or go back), pages are taken from and given back to a ring of free ones
  rope    queries and keys divided by their root mean square for each head, times a weight, then rotated by the
          row's position, in one pass
  step    the same, with the keys and values stored in the paged pool
  store   rows quantised to 4 bits (q4_0) and stored on their pages, then read back
  decode  attention of one new token of each sequence over a pool of 4 bits

q4_0: 32 values along the head share an fp16 scale d = -m / 8, m the one of greatest magnitude (of two, the negative
one); codes c = min(round(-8 x / m), 7), ties away from zero; value d c.  Eight codes are one 32-bit word: value i of
the eight lies, as c + 8, in the four bits from bit 16 (i % 2) + 4 (i / 2).

`run` with own = False is the plain form in elementary torch operations; with own = True it calls the package.
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------------

def listed():
    full = {"heads_q": 40, "heads_kv": 8, "head_dim": 128}
    small = {"heads_q": 16, "heads_kv": 4, "head_dim": 64}
    return [
        # a decode step of 64 sequences: all one token further, now and then one ends and another begins
        {"name": "pages_step64", "op": "pages", "page": 16, "n_seq": 64, "shortest": 33, "longest": 4100, "prompts": 2,
         "ends": 2, "longest_prompt": 700, "spare": 40, "shape": 1},
        # a full scheduler with many new prompts at once
        {"name": "pages_batch1024", "op": "pages", "page": 32, "n_seq": 1024, "shortest": 5, "longest": 16384,
         "prompts": 40, "ends": 60, "longest_prompt": 2048, "spare": 500, "shape": 2},
        # a decode step of 96 sequences
        {"name": "rope_step96", "op": "rope", "dtype": "bf16", "n_seq": 96, "shortest": 5, "longest": 16384, "new": 1,
         "base": 1e6, "rot": 128, "style": "half", "shape": 3, **full},
        # one long prompt, whole
        {"name": "rope_10041", "op": "rope", "dtype": "bf16", "n_seq": 1, "shortest": 10041, "longest": 10041, "new": 0,
         "base": 1e6, "rot": 128, "style": "half", "shape": 4, **full},
        # chunks of a few prompts with small heads, half of each head rotated in neighbouring pairs, 32-bit values
        {"name": "rope_f32_pairs", "op": "rope", "dtype": "f32", "n_seq": 3, "shortest": 1000, "longest": 60000,
         "new": 333, "base": 1e4, "rot": 32, "style": "pairs", "shape": 5, **small},
        # a decode step of 64 sequences into an f16 cache
        {"name": "step_f16_64", "op": "step", "cache": "f16", "layout": "head_major", "page": 16, "dtype": "bf16",
         "n_seq": 64, "shortest": 33, "longest": 4100, "new": 1, "base": 1e6, "rot": 128, "style": "half", "shape": 6,
         **full},
        # prompts of different lengths enter a q8_0 cache, and are read back for their attention
        {"name": "step_q8_prompts", "op": "step", "cache": "q8_0", "layout": "layer_major", "page": 64, "dtype": "bf16",
         "n_seq": 6, "shortest": 700, "longest": 5000, "new": 0, "base": 1e6, "rot": 128, "style": "half", "shape": 7,
         **full},
        # a decode step of 64 sequences into a cache of 4 bits, and the stored rows read back
        {"name": "store_q4_step64", "op": "store", "layout": "layer_major", "page": 32, "dtype": "bf16", "out": "f16",
         "n_seq": 64, "shortest": 33, "longest": 4100, "new": 1, "shape": 8, **full},
        # packed prompts into a cache of 4 bits, read back as the attention over them reads them
        {"name": "store_q4_prompts", "op": "store", "layout": "head_major", "page": 64, "dtype": "bf16", "out": "f16",
         "n_seq": 9, "shortest": 1023, "longest": 4100, "new": 0, "shape": 9, **full},
        # eight parallel sequences at 2k context
        {"name": "decode_q4_npl8", "op": "decode", "layout": "head_major", "page": 16, "dtype": "bf16", "n_seq": 8,
         "shortest": 2048, "longest": 2176, "new": 1, "shape": 10, **full},
        # one long conversation: a single token over 58,300 positions
        {"name": "decode_q4_58k", "op": "decode", "layout": "head_major", "page": 64, "dtype": "bf16", "n_seq": 1,
         "shortest": 58300, "longest": 58300, "new": 1, "shape": 11, **full},
        # a full serving batch, lengths from a few tokens to 16k
        {"name": "decode_q4_batch96", "op": "decode", "layout": "layer_major", "page": 32, "dtype": "f16", "n_seq": 96,
         "shortest": 5, "longest": 16384, "new": 1, "shape": 12, **full},
    ]


def _log_between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "pages", "rope", "rope", "step", "step", "store", "decode", "decode", "decode"])
    c = {"op": op, "shape": rng.randrange(1 << 30)}
    if op == "pages":
        c["page"] = rng.choice([16, 32, 48, 64, 128])
        c["n_seq"] = _log_between(rng, 1, 1024)
        c["longest"] = _log_between(rng, 8, 16384)
        c["shortest"] = rng.choice([1, max(1, c["longest"] // 2)])
        c["prompts"] = rng.randint(0, 1 + c["n_seq"] // 20)
        c["ends"] = rng.randint(0, 1 + c["n_seq"] // 16)
        c["longest_prompt"] = _log_between(rng, 1, 2048)
        c["spare"] = rng.choice([-3, 0, 7, 200])
        return c
    c["heads_q"], c["heads_kv"] = rng.choice([(40, 8), (40, 8), (16, 4), (10, 2), (8, 8), (4, 2), (24, 3)])
    c["head_dim"] = rng.choice([64, 128, 128])
    c["dtype"] = rng.choice(["bf16", "f16", "f32"] if op == "rope" else ["bf16", "f16"])
    if op in ("rope", "step"):
        c["base"] = rng.choice([1e4, 5e5, 1e6])
        c["rot"] = rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2])
        c["style"] = rng.choice(["half", "pairs"])
    if op != "rope":
        c["layout"] = rng.choice(["head_major", "layer_major"])
        c["page"] = rng.choice([16, 32, 48, 64, 128])
    if op == "step":
        c["cache"] = rng.choice(["f16", "q8_0"])
    if op == "store":
        c["out"] = rng.choice(["bf16", "f16", "f32"])
    budget = {"rope": 9000, "step": 9000, "store": 16000, "decode": 200000}[op]
    c["n_seq"] = _log_between(rng, 1, 96)
    longest = _log_between(rng, 8, 16384)
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


def schedule(case):
    """(tokens held, what the next step adds to them) of each sequence: one token, a prompt, or their end."""
    rng = random.Random(case["shape"])
    n = case["n_seq"]
    held = [_log_between(rng, case["shortest"], case["longest"]) for _ in range(n)]
    add = [1] * n
    order = rng.sample(range(n), n)
    for i in order[:case["prompts"]]:
        held[i], add[i] = 0, _log_between(rng, 1, case["longest_prompt"])
    for i in order[case["prompts"]:case["prompts"] + case["ends"]]:
        add[i] = -held[i]
    return held, add


def _used(n, page):
    return -(-n // page)


# ---- inputs ---------------------------------------------------------------------------------------

def _starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _keys(gen, n, hkv, d):
    """Keys of n tokens: N(0, 1), one channel in a hundred four times as large."""
    k = torch.randn(n, hkv, d, generator=gen, device="cuda")
    wide = torch.randperm(hkv * d, generator=gen, device="cuda")[: max(1, hkv * d // 100)]
    k.view(n, hkv * d)[:, wide] *= 4
    return k


def _q8(x):
    """q8_0: codes and fp16 scales of blocks of 32 values of the last axis."""
    b = x.float().unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=x.device)
    r = torch.where(d > 0, b / d, torch.zeros((), device=x.device)).double()  # in 64 bits |r| + 0.5 is exact
    q = torch.sign(r) * torch.floor(r.abs() + 0.5)
    return q.to(torch.int8).flatten(-2), d.squeeze(-1).half()


def _q4(x):
    """q4_0: words of eight codes and fp16 scales of blocks of 32 values of the last axis."""
    b = x.float().unflatten(-1, (-1, 32))
    hi, lo = b.amax(-1, keepdim=True), b.amin(-1, keepdim=True)
    m = torch.where(hi > -lo, hi, lo)
    r = torch.where(m != 0, b.double() * -8 / m.double(), torch.zeros((), device=x.device, dtype=torch.float64))
    c = (torch.sign(r) * torch.floor(r.abs() + 0.5)).clamp(max=7) + 8
    i = torch.arange(8, device=x.device)
    w = (c.to(torch.int64).unflatten(-1, (4, 8)) << (16 * (i % 2) + 4 * (i // 2))).sum(-1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    return w.flatten(-2), (m.squeeze(-1) / -8).half()


def _values4(w, d):
    """The values of q4_0 words and scales, in 32 bits."""
    i = torch.arange(8, device=w.device, dtype=torch.int32)
    c = (w.unsqueeze(-1) >> (16 * (i % 2) + 4 * (i // 2))) & 15
    return ((c.flatten(-2).unflatten(-1, (-1, 32)) - 8).float() * d.float().unsqueeze(-1)).flatten(-2)


def _by_token(t, layout):
    """A pool buffer as [position][head][...]."""
    return t[:, 0].transpose(0, 1) if layout == "head_major" else t[0]


def _prepare_pages(case, seed):
    held, add = schedule(case)
    page, n = case["page"], case["n_seq"]
    rng = np.random.default_rng(seed)
    most = [_used(max(h, h + a), page) for h, a in zip(held, add)]
    n_pages = max(1, sum(most) + case["spare"])
    width = max(max(most), 1)
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((n, width), -1, dtype=np.int32)
    at = 0
    for i, h in enumerate(held):
        u = min(_used(h, page), n_pages - at)
        table[i, :u] = order[at:at + u]
        at += u
    s = dict(case, table=torch.from_numpy(table).cuda(), held=_i32(held), n_pages=n_pages,
             add=_i32(add), back=_i32([-a for a in add]),
             n_rows=sum(a for a in add if a > 0), n_back=sum(-a for a in add if a < 0))
    free = torch.from_numpy(order[at:]).cuda()
    if own:
        import decode_attention_kv_cache_gb300 as kvc
        s["pages"] = kvc.PageTable(s["table"], s["held"], page)
        s["free"] = kvc.FreePages(n_pages, free)
        s["ring"], s["state"] = s["free"].ring, s["free"].state
    else:
        s["ring"] = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        s["ring"][:free.numel()] = free
        s["state"] = _i32([0, free.numel(), 0])   # where the ring begins, free pages, pages that were missing
    return s


def prepare(case, seed):
    if case["op"] == "pages":
        return _prepare_pages(case, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    held, rows = lengths(case)
    n, hq, hkv, d = case["n_seq"], case["heads_q"], case["heads_kv"], case["head_dim"]
    dt, op = DT[case["dtype"]], case["op"]
    n_rows = sum(rows)
    s = dict(case, held=_i32(held), row_start=_i32(_starts(rows)), n_rows=n_rows, longest_held=max(held))
    if op in ("rope", "step"):
        qkv = torch.randn(n_rows, hq + 2 * hkv, d, generator=gen, device="cuda")
        qkv[:, hq:hq + hkv] = _keys(gen, n_rows, hkv, d)
        qkv = qkv.to(dt)                          # a fused projection: q, k and v are parts of its rows
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt) for _ in (0, 1))
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        s["freq"] = case["base"] ** (-2 * i / case["rot"])
        if own:
            import decode_attention_kv_cache_gb300 as kvc
            s["rope"] = kvc.RopeTable(case["rot"], base=case["base"], style=case["style"])
        if op == "rope":
            seq = torch.repeat_interleave(torch.arange(n, device="cuda"), s["row_start"].diff())
            row = torch.arange(n_rows, device="cuda", dtype=torch.int32)
            s["positions"] = s["held"][seq] - s["row_start"][seq + 1] + row
            return s
    page = case["page"]
    used = [_used(h, page) for h in held]
    n_pages = sum(used) + 3  # a few pages belong to nobody
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(n, max(used), dtype=torch.int32, device="cuda")
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    s["table"] = table
    positions = n_pages * page
    kind = s["cache"] = case.get("cache", "q4_0")
    if own:
        import decode_attention_kv_cache_gb300 as kvc
        cache = s["own_cache"] = kvc.KVCache(1, positions, hkv, d, kind, case["layout"])
        s["pages"] = kvc.PageTable(table, s["held"], page)
        pool = [cache.codes(0), cache.codes(1), cache.scales(0), cache.scales(1)]
        if kind == "q4_0":
            pool[:2] = [t.view(torch.int32) for t in pool[:2]]
        if op == "decode":
            s["scratch"] = kvc.paged_scratch(cache, n, hq)
    else:
        dims = (hkv, 1, positions) if case["layout"] == "head_major" else (1, positions, hkv)
        last, t = {"f16": (d, torch.float16), "q8_0": (d, torch.int8), "q4_0": (d // 8, torch.int32)}[kind]
        pool = [torch.empty(*dims, last, dtype=t, device="cuda") for _ in (0, 1)]
        pool += [torch.empty(*dims, d // 32, dtype=torch.float16, device="cuda") if kind != "f16" else None
                 for _ in (0, 1)]
    for kv in (0, 1):
        x = _keys(gen, positions, hkv, d) if kv == 0 else torch.randn(positions, hkv, d, generator=gen, device="cuda")
        x = x.to(dt)
        if kind == "f16":
            _by_token(pool[kv], case["layout"]).copy_(x)
        else:
            for part in range(0, positions, 16384):
                q, sc = (_q8 if kind == "q8_0" else _q4)(x[part:part + 16384])
                _by_token(pool[kv], case["layout"])[part:part + 16384] = q
                _by_token(pool[2 + kv], case["layout"])[part:part + 16384] = sc
        del x
    s["pool"] = pool
    if op == "store":
        s["k"] = _keys(gen, n_rows, hkv, d).to(dt)
        s["v"] = torch.randn(n_rows, hkv, d, generator=gen, device="cuda").to(dt)
    if op == "decode":
        s["q"] = torch.randn(n, hq, d, generator=gen, device="cuda").to(dt)
    return s


# ---- one pass -------------------------------------------------------------------------------------

def _slots(s):
    """The position of each packed row in its sequence, and in the pool."""
    row = torch.arange(s["n_rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["row_start"], row, right=True) - 1
    pos = s["held"][seq] - s["row_start"][seq + 1] + row
    return pos, s["table"][seq, (pos // s["page"]).long()].long() * s["page"] + pos % s["page"]


def _values(s, kv, slots):
    """What the pool holds for K (0) or V (1) at `slots`, in 32 bits: [..., head, value]."""
    x = _by_token(s["pool"][kv], s["layout"])[slots]
    if s["cache"] == "f16":
        return x.float()
    scale = _by_token(s["pool"][2 + kv], s["layout"])[slots]
    if s["cache"] == "q4_0":
        return _values4(x, scale)
    return (x.float().unflatten(-1, (-1, 32)) * scale.float().unsqueeze(-1)).flatten(-2)


def _store(s, slots, k, v):
    for kv, x in ((0, k), (1, v)):
        if s["cache"] == "f16":
            _by_token(s["pool"][kv], s["layout"])[slots] = x.half()
        else:
            q, d = (_q8 if s["cache"] == "q8_0" else _q4)(x)
            _by_token(s["pool"][kv], s["layout"])[slots] = q
            _by_token(s["pool"][2 + kv], s["layout"])[slots] = d


def _norm_rope(s, x, weight, positions):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = positions.double()[:, None] * s["freq"]    # far positions need more than 32 bits
    c, z = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    rot = s["rot"]
    if s["style"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * c - b * z, b * c + a * z), -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * c - b * z, b * c + a * z), -1).flatten(-2)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


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


def _advance(s, add, n_rows):
    """Lengths grow by `add` (or shrink); pages come from the front of the ring and go back to its end."""
    table, held, ring, state, page = s["table"], s["held"], s["ring"], s["state"], s["page"]
    width, cap = table.shape[1], ring.numel()
    now = (held.long() + add).clamp(min=0)
    had, has = ((x + page - 1) // page for x in (held.long(), now))
    had, has = had.clamp(max=width), has.clamp(max=width)
    e = torch.arange(width, device="cuda")
    takes = ((e >= had[:, None]) & (e < has[:, None])).flatten()
    gives = ((e >= has[:, None]) & (e < had[:, None])).flatten()
    flat = table.view(-1)
    good = gives & (flat >= 0) & (flat < cap)
    head, count = state[0].long(), state[1].long()
    # the k-th entry that needs a page has the k-th of the ring; what there is not is -1
    k = torch.cumsum(takes, 0) - 1
    page_of = torch.where(k < count, ring[((head + k) % cap).clamp(min=0)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    j = torch.cumsum(good, 0) - 1
    room = good & (count + j < cap)
    # entries that give nothing write the cell that the ring has behind its end
    cells = torch.cat((ring, ring[:1]))
    cells[torch.where(room, (head + count + j) % cap, torch.full((), cap, device="cuda"))] = flat
    ring.copy_(cells[:cap])
    flat.copy_(torch.where(takes, page_of, torch.where(gives, torch.full((), -1, dtype=torch.int32, device="cuda"), flat)))
    need, back = takes.sum(), room.sum()
    taken = torch.minimum(need, count)
    state.copy_(torch.stack(((head + taken) % cap, count - taken + back, state[2] + need - taken)))
    held.copy_(now)
    start = torch.zeros(held.numel() + 1, dtype=torch.int32, device="cuda")
    start[1:] = torch.cumsum(add.clamp(min=0), 0)
    row = torch.arange(n_rows, device="cuda", dtype=torch.int32)
    seq = (torch.searchsorted(start, row, right=True) - 1).clamp(max=held.numel() - 1)
    pos = held[seq] - start[seq + 1] + row
    at = table[seq, (pos // page).clamp(0, width - 1).long()]
    slot = torch.where((at >= 0) & (pos // page < width), at * page + pos % page, torch.full((), -1, dtype=torch.int32, device="cuda"))
    return start, pos, slot


def run(s):
    op = s["op"]
    if op == "pages":
        # one scheduler step, and the way back: what grew is taken back (as rejected tokens are), what ended begins again
        if own:
            import decode_attention_kv_cache_gb300 as kvc
            there = kvc.kv_pages_advance(s["pages"], s["free"], s["add"], s["n_rows"])
            again = kvc.kv_pages_advance(s["pages"], s["free"], s["back"], s["n_back"])
        else:
            there = _advance(s, s["add"], s["n_rows"])
            again = _advance(s, s["back"], s["n_back"])
        return there, again, s["table"], s["held"], s["ring"], s["state"]
    if own:
        import decode_attention_kv_cache_gb300 as kvc
        if op == "decode":
            return kvc.decode_attn_paged(s["own_cache"], 0, s["pages"], s["q"], scratch=s["scratch"])
        if op == "rope":
            return kvc.qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"], s["q_weight"], s["k_weight"], EPS)
        if op == "store":
            kvc.kv_paged_append(s["own_cache"], 0, s["pages"], s["row_start"], s["k"], s["v"])
            return kvc.kv_paged_read(s["own_cache"], 0, s["pages"], s["row_start"], s["n_rows"], dtype=DT[s["out"]])
        q = kvc.qk_norm_rope_append(s["own_cache"], 0, s["pages"], s["row_start"], s["q"], s["k"], s["v"], s["rope"],
                                    s["q_weight"], s["k_weight"], EPS)
        if s["cache"] == "f16":
            return q, s["pool"][0], s["pool"][1]
        return q, kvc.kv_paged_read(s["own_cache"], 0, s["pages"], s["row_start"], s["n_rows"], dtype=torch.float16)
    if op == "decode":
        return _decode(s)
    if op == "rope":
        return tuple(_norm_rope(s, s[x], s[x + "_weight"], s["positions"]) for x in ("q", "k"))
    pos, slots = _slots(s)
    if op == "store":
        _store(s, slots, s["k"], s["v"])
        return tuple(_values(s, kv, slots).to(DT[s["out"]]) for kv in (0, 1))
    q, k = (_norm_rope(s, s[x], s[x + "_weight"], pos) for x in ("q", "k"))
    _store(s, slots, k, s["v"])
    if s["cache"] == "f16":
        return q, s["pool"][0], s["pool"][1]
    return q, tuple(_values(s, kv, slots).half() for kv in (0, 1))


# ---- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    if case["op"] == "pages":
        held, add = schedule(case)
        page, n = case["page"], case["n_seq"]
        moved = sum(abs(_used(h + a, page) - _used(h, page)) for h, a in zip(held, add))
        rows = sum(abs(a) for a in add)
        # each way: lengths read and written, rows read, starts written; positions and slots of the rows written; a ring
        # cell and a table entry for each page that changes hands
        return {"bytes": 2 * 4 * (4 * n + 1) + 8 * rows + 2 * 12 * moved, "flops": 2 * (4 * n + 4 * rows)}
    held, rows = lengths(case)
    hq, hkv, d = case["heads_q"], case["heads_kv"], case["head_dim"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    e, n = size[case["dtype"]], sum(rows)
    if case["op"] == "rope":
        return {"bytes": 2 * n * (hq + hkv) * d * e + 4 * n + 2 * d * e, "flops": 8 * n * (hq + hkv) * d}
    kind = case.get("cache", "q4_0")
    row_pool = hkv * {"f16": 2 * d, "q8_0": d + d // 16, "q4_0": d // 2 + d // 16}[kind]
    if case["op"] == "decode":
        return {"bytes": 2 * sum(held) * row_pool + 2 * len(held) * hq * d * e, "flops": 4 * hq * d * sum(held)}
    if case["op"] == "store":
        return {"bytes": 2 * n * (hkv * d * e + 2 * row_pool + hkv * d * size[case["out"]]), "flops": 10 * n * hkv * d}
    back = 0 if kind == "f16" else 2 * n * (row_pool + 2 * hkv * d)
    return {"bytes": 2 * n * (hq + hkv) * d * e + 2 * n * row_pool + back,
            "flops": 8 * n * (hq + 2 * hkv) * d}


# ---- the same from the definitions, in 64 bits ----------------------------------------------------

def _places(case, s):
    """For each sequence the pool positions of its tokens, in order (host)."""
    table, page = s["table"].cpu().tolist(), case["page"]
    held, rows = lengths(case)
    return [[table[i][p // page] * page + p % page for p in range(h)] for i, h in enumerate(held)], held, rows


def _held64(case, s, kv, places):
    at = torch.tensor(places, device="cuda", dtype=torch.long)
    pick = (lambda t: t[:, 0, at].permute(1, 0, 2)) if case["layout"] == "head_major" else (lambda t: t[0, at])
    w, d = pick(s["pool"][kv]), pick(s["pool"][2 + kv]).double()
    codes = torch.stack([(w >> (16 * (i & 1) + 4 * (i >> 1))) & 15 for i in range(8)], -1).flatten(-2).double() - 8
    return codes * d.repeat_interleave(32, dim=-1)


def _attend64(q, k, v):
    z = torch.einsum("gd,nd->gn", q, k) * q.shape[-1] ** -0.5
    return torch.softmax(z, dim=-1) @ v


def _turned64(x, weight, at, case):
    """The norm and rotation of rows x [row][head][value] at the host's positions `at`."""
    x = x.double()
    y = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    rot, out = case["rot"], y.clone()
    at = torch.tensor(at, dtype=torch.float64, device="cuda")[:, None]
    for i in range(rot // 2):
        p, q = (i, i + rot // 2) if case["style"] == "half" else (2 * i, 2 * i + 1)
        t = at * case["base"] ** (-2.0 * i / rot)
        out[..., p] = y[..., p] * torch.cos(t) - y[..., q] * torch.sin(t)
        out[..., q] = y[..., p] * torch.sin(t) + y[..., q] * torch.cos(t)
    return out


def _positions(held, rows):
    return [p for h, r in zip(held, rows) for p in range(h - r, h)]


def exact(case, seed):
    if case["op"] == "pages":
        return None                        # whole numbers: the plain form is the definition
    s = prepare(case, seed)
    hq, hkv, d, op = case["heads_q"], case["heads_kv"], case["head_dim"], case["op"]
    g = hq // hkv
    if op == "rope":
        held, rows = lengths(case)
        return tuple(_turned64(s[x], s[x + "_weight"], _positions(held, rows), case) for x in ("q", "k"))
    places, held, rows = _places(case, s)
    if op == "decode":
        out = []
        for i, at in enumerate(places):
            q, k, v = s["q"][i].double(), _held64(case, s, 0, at), _held64(case, s, 1, at)
            out.append(torch.cat([_attend64(q[j * g:(j + 1) * g], k[:, j], v[:, j]) for j in range(hkv)]))
        return torch.stack(out)
    if op == "step":
        # the keys are rounded to the inputs' type before they are stored, so a q8_0 pool's codes have no value here
        at = _positions(held, rows)
        q = _turned64(s["q"], s["q_weight"], at, case)
        if case["cache"] != "f16":
            return q, (None, None)
        mine = torch.tensor([p for a, r in zip(places, rows) for p in a[len(a) - r:]], device="cuda")
        pool = [t.double() for t in s["pool"][:2]]
        for kv, x in ((0, _turned64(s["k"], s["k_weight"], at, case)), (1, s["v"].double())):
            if case["layout"] == "head_major":
                pool[kv][:, 0, mine] = x.transpose(0, 1)
            else:
                pool[kv][0, mine] = x
        return q, pool[0], pool[1]
    out = []
    for x in (s["k"], s["v"]):
        b = x.double().cpu().numpy().reshape(-1, 32)
        first, last = b.min(1, keepdims=True), b.max(1, keepdims=True)
        m = np.where(last > -first, last, first)
        y = np.divide(-8 * b, m, out=np.zeros_like(b), where=m != 0)
        codes = np.minimum(np.copysign(np.floor(np.abs(y) + 0.5), y), 7)
        out.append(torch.from_numpy(codes * (m / -8).astype("f2").astype("f8")).reshape(-1, hkv, d))
    return tuple(out)
