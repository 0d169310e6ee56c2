"""Python binding of libkvc: attention over a device-resident q8_0/f16 KV cache (pools of pages: also q4_0) on GB300.

Argument marshalling only.  Every step of the path (quantise-and-append,
chunked prefill attention, split-K decode attention, state pack/unpack) runs in
the library's CUDA kernels; torch supplies device memory and the current
stream.  The functions carry the names of the C ABI in include/kvc.h.

There is no fallback: the library is loaded on first use, which raises
ImportError if libkvc.so has not been built (python -m
decode_attention_kv_cache_gb300.build); every call raises KvcError when the
library reports an error.
"""

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvc.so")

KVC_OK, KVC_EINVAL, KVC_ERANGE, KVC_ENOSPC, KVC_EFORMAT, KVC_ECUDA, KVC_EDEVICE = 0, -1, -2, -3, -4, -5, -6
CACHE_TYPES = {"f16": 0, "q8_0": 1, "q4_0": 2}
LAYOUTS = {"head_major": 0, "layer_major": 1}
# 2^128 / (2 pi)
_TURN = (10 ** 39 << 128) // (2 * 3141592653589793238462643383279502884197)


def _turns(freq):
    """The frequency in turns, modulo 1, as a fraction of 2^64: a signed 64-bit integer.  In integers, as a float's
    product with 1 / (2 pi) would lose the last bits."""
    n, d = freq.as_integer_ratio()          # d is a power of two
    shift = 64 + d.bit_length() - 1
    t = ((n * _TURN >> shift - 1) + 1 >> 1) & (1 << 64) - 1
    return t - (1 << 64) if t >> 63 else t


DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class KvcError(RuntimeError):
    def __init__(self, status, what):
        super().__init__("%s: %s (%d)" % (what, _lib().kvc_strerror(status).decode(), status))
        self.status = status


class kvc_desc(ctypes.Structure):
    _fields_ = [("n_layer", ctypes.c_int32), ("n_ctx", ctypes.c_int32), ("n_head_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("type", ctypes.c_int32), ("layout", ctypes.c_int32)]


class kvc_cache(ctypes.Structure):
    _fields_ = [("d", kvc_desc), ("k_q", ctypes.c_void_p), ("k_s", ctypes.c_void_p),
                ("v_q", ctypes.c_void_p), ("v_s", ctypes.c_void_p)]


class kvc_pages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("len", ctypes.c_void_p), ("n_seq", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class kvc_free_pages(ctypes.Structure):
    _fields_ = [("ring", ctypes.c_void_p), ("state", ctypes.c_void_p), ("n_pages", ctypes.c_int32)]


class kvc_rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("n_pairs", ctypes.c_int32), ("style", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libkvc.so is not built; run `python -m decode_attention_kv_cache_gb300.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, SZ, VP = ctypes.POINTER, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
    I64 = ctypes.c_int64
    sig = {
        "kvc_cache_bytes": (ctypes.c_int, [P(kvc_desc), P(SZ), P(SZ), P(SZ), P(SZ)]),
        "kvc_scratch_bytes": (ctypes.c_int, [P(kvc_desc), I32, P(SZ)]),
        "kv_state_size": (SZ, [P(kvc_desc), I32]),
        "kvc_cache_init": (ctypes.c_int, [P(kvc_cache), P(kvc_desc), VP, VP, VP, VP]),
        "kv_cache_append": (ctypes.c_int, [P(kvc_cache), I32, I32, I32, VP, VP, I32, VP]),
        "kvc_prefill_scratch_bytes": (ctypes.c_int, [P(kvc_desc), I32, I32, P(SZ)]),
        "prefill_chunk_attn": (ctypes.c_int, [P(kvc_cache), I32, I32, I32, VP, I32, I32, VP, VP, SZ, VP]),
        "decode_attn": (ctypes.c_int, [P(kvc_cache), I32, I32, VP, I32, I32, VP, VP, SZ, VP]),
        "prefill_step": (ctypes.c_int, [P(kvc_cache), I32, I32, I32, VP, VP, VP, I32, I32, VP, VP, SZ, I32, VP]),
        "kv_state_get": (ctypes.c_int, [P(kvc_cache), I32, VP, SZ, VP]),
        "kv_state_set": (ctypes.c_int, [P(kvc_cache), VP, SZ, P(I32), VP]),
        "kvc_strerror": (ctypes.c_char_p, [ctypes.c_int]),
        "kvc_device_status": (ctypes.c_int, [P(I32)]),
        "kvc_pipeline_chunk": (ctypes.c_int, [I32, I32, I32, ctypes.c_double, P(I32)]),
        "kv_cache_truncate": (ctypes.c_int, [P(kvc_cache), I32, VP]),
        "decode_attn_batch": (ctypes.c_int, [P(kvc_cache), I32, I32, P(I32), VP, I32, I32, VP, VP, SZ, VP]),
        "decode_step": (ctypes.c_int, [P(kvc_cache), I32, I32, VP, VP, VP, I32, I32, VP, VP, SZ, VP]),
        "decode_step_batch": (ctypes.c_int, [P(kvc_cache), I32, I32, P(I32), VP, VP, VP, I32, I32, VP, VP, SZ, VP]),
        "kv_cache_append_batch": (ctypes.c_int, [P(kvc_cache), I32, I32, P(I32), VP, VP, I32, VP]),
        "kv_state_get_heads": (ctypes.c_int, [P(kvc_cache), I32, I32, I32, VP, SZ, VP]),
        "kv_state_set_heads": (ctypes.c_int, [P(kvc_cache), I32, VP, SZ, P(I32), VP]),
        "kv_paged_append": (ctypes.c_int, [VP, VP, I32, VP, I32, VP, VP, I64, I64, I32, VP]),
        "kv_paged_read": (ctypes.c_int, [VP, VP, I32, VP, I32, VP, VP, I32, VP]),
        "kvc_paged_scratch_bytes": (ctypes.c_int, [P(kvc_desc), I32, I32, P(SZ)]),
        "decode_attn_paged": (ctypes.c_int, [VP, VP, I32, VP, I64, I32, I32, VP, VP, VP, SZ, VP]),
        "kvc_packed_scratch_bytes": (ctypes.c_int, [I32, I32, I32, I32, I32, P(SZ)]),
        "attn_packed": (ctypes.c_int, [VP, VP, VP, I64, I64, I64, I32, VP, VP, I32, I32, I32, I32, I32, I32, VP, VP,
                                       VP, SZ, VP]),
        "kv_pages_advance": (ctypes.c_int, [VP, VP, VP, VP, I32, VP, VP, VP]),
        "qk_norm_rope": (ctypes.c_int, [VP, VP, VP, I64, I64, I32, I32, I32, I32, I32, VP, VP, VP, ctypes.c_float, VP, VP,
                                        I64, I64, VP]),
        "qk_norm_rope_append": (ctypes.c_int, [VP, VP, I32, VP, I32, VP, VP, VP, VP, I64, I64, I64, I32, I32, VP, VP,
                                               ctypes.c_float, VP, I64, VP]),
        "kvc_test_arm_wait_timeout": (ctypes.c_int, [I32, ctypes.c_uint64]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


def _check(status, what):
    if status != KVC_OK:
        raise KvcError(status, what)


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t, what, dtype=None):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % what)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s" % (what, dtype))


def make_desc(n_layer, n_ctx, n_head_kv, head_dim, cache_type="q8_0", layout="head_major"):
    return kvc_desc(n_layer, n_ctx, n_head_kv, head_dim, CACHE_TYPES[cache_type], LAYOUTS[layout])


def cache_bytes(desc):
    s = [ctypes.c_size_t() for _ in range(4)]
    _check(_lib().kvc_cache_bytes(ctypes.byref(desc), *[ctypes.byref(x) for x in s]), "kvc_cache_bytes")
    return tuple(x.value for x in s)


class KVCache:
    """A cache whose four buffers are torch allocations on `device`.

    Codes/values: k_q, v_q; scales (q8_0 and q4_0): k_s, v_s.  The buffers are
    exposed as typed views in the layout of the descriptor.  "q4_0" is a type
    of pools: the calls with a PageTable take it.
    """

    def __init__(self, n_layer, n_ctx, n_head_kv, head_dim, cache_type="q8_0", layout="head_major",
                 device="cuda"):
        self.desc = make_desc(n_layer, n_ctx, n_head_kv, head_dim, cache_type, layout)
        self.n_layer, self.n_ctx, self.n_head_kv, self.head_dim = n_layer, n_ctx, n_head_kv, head_dim
        self.cache_type, self.layout = cache_type, layout
        self.device = torch.device(device)
        kq, ks, vq, vs = cache_bytes(self.desc)
        self._bufs = [torch.empty(max(n, 16), dtype=torch.uint8, device=self.device) for n in (kq, ks, vq, vs)]
        self._sizes = (kq, ks, vq, vs)
        self.c = kvc_cache()
        scales = cache_type != "f16"
        _check(_lib().kvc_cache_init(ctypes.byref(self.c), ctypes.byref(self.desc), _ptr(self._bufs[0]),
                                  _ptr(self._bufs[1]) if scales else ctypes.c_void_p(0), _ptr(self._bufs[2]),
                                  _ptr(self._bufs[3]) if scales else ctypes.c_void_p(0)), "kvc_cache_init")
        self.addr, self.cuda = ctypes.addressof(self.c), self._bufs[0].device

    def _shape(self, last):
        if self.layout == "head_major":
            return (self.n_head_kv, self.n_layer, self.n_ctx, last)
        return (self.n_layer, self.n_ctx, self.n_head_kv, last)

    def codes(self, kv):
        """K (kv=0) or V (kv=1) codes (int8; q4_0: uint8, two to a byte) or values (float16), in layout order."""
        b = self._bufs[2 * kv][: self._sizes[2 * kv]]
        if self.cache_type == "q4_0":
            return b.view(self._shape(self.head_dim // 2))
        dt = torch.int8 if self.cache_type == "q8_0" else torch.float16
        return b.view(dt).view(self._shape(self.head_dim))

    def scales(self, kv):
        if self.cache_type == "f16":
            return None
        b = self._bufs[2 * kv + 1][: self._sizes[2 * kv + 1]]
        return b.view(torch.float16).view(self._shape(self.head_dim // 32))

    def scratch_bytes(self, n_head_q):
        n = ctypes.c_size_t()
        _check(_lib().kvc_scratch_bytes(ctypes.byref(self.desc), n_head_q, ctypes.byref(n)), "kvc_scratch_bytes")
        return n.value

    def prefill_scratch_bytes(self, n_head_q, max_tokens):
        n = ctypes.c_size_t()
        _check(_lib().kvc_prefill_scratch_bytes(ctypes.byref(self.desc), n_head_q, max_tokens, ctypes.byref(n)),
               "kvc_prefill_scratch_bytes")
        return n.value

    def prefill_scratch(self, n_head_q, max_tokens):
        """A prefill scratch buffer for chunks of up to max_tokens rows (needs no initialisation)."""
        return torch.empty(max(self.prefill_scratch_bytes(n_head_q, max_tokens), 16), dtype=torch.uint8,
                           device=self.device)

    def state_size(self, n_tokens):
        return _lib().kv_state_size(ctypes.byref(self.desc), n_tokens)


def pipeline_chunk(n_tokens, cap, stages, b_over_a=1024.0):
    """Prompt chunk size for prefill over `stages` layer-split pipeline stages (host only)."""
    c = ctypes.c_int32(0)
    _check(_lib().kvc_pipeline_chunk(int(n_tokens), int(cap), int(stages), ctypes.c_double(b_over_a),
                                     ctypes.byref(c)), "kvc_pipeline_chunk")
    return c.value


def kv_cache_append(cache, layer, pos0, k, v, stream=None):
    """Quantise/round and store K, V [n, H_kv, D] at positions [pos0, pos0 + n) of `layer`."""
    _need(k, "k"); _need(v, "v", k.dtype)
    st = _lib().kv_cache_append(ctypes.byref(cache.c), layer, pos0, k.shape[0], _ptr(k), _ptr(v), DTYPES[k.dtype],
                             _stream(stream, k.device))
    _check(st, "kv_cache_append")


def prefill_chunk_attn(cache, layer, pos0, q, out=None, scratch=None, stream=None):
    """Causal attention of chunk rows q [C, H_q, D] at positions [pos0, pos0 + C); returns out [C, H_q, D] f32.

    scratch: a uint8 CUDA buffer (KVCache.prefill_scratch); one is made when None.
    """
    _need(q, "q")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if scratch is None:
        scratch = cache.prefill_scratch(q.shape[1], max(q.shape[0], 1))
    _need(out, "out", torch.float32); _need(scratch, "scratch")
    st = _lib().prefill_chunk_attn(ctypes.byref(cache.c), layer, pos0, q.shape[0], _ptr(q), DTYPES[q.dtype],
                                q.shape[1], _ptr(out), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                _stream(stream, q.device))
    _check(st, "prefill_chunk_attn")
    return out


def prefill_step(cache, layer, pos0, q, k, v, out=None, scratch=None, stream=None, copy_valid=0):
    """One prompt chunk: store k, v [C, H_kv, D] at positions [pos0, pos0 + C) (as kv_cache_append) and
    attend with q [C, H_q, D] (as prefill_chunk_attn); returns out [C, H_q, D] f32.  copy_valid: leading
    positions of the scratch's fp16 copy (q8_0) already holding this layer's values from earlier calls
    with this scratch (pos0 when the previous chunk of this layer went through it)."""
    _need(q, "q"); _need(k, "k", q.dtype); _need(v, "v", q.dtype)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if scratch is None:
        scratch = cache.prefill_scratch(q.shape[1], max(q.shape[0], 1))
    _need(out, "out", torch.float32); _need(scratch, "scratch")
    st = _lib().prefill_step(ctypes.byref(cache.c), layer, pos0, q.shape[0], _ptr(q), _ptr(k), _ptr(v), DTYPES[q.dtype],
                             q.shape[1], _ptr(out), _ptr(scratch), scratch.numel() * scratch.element_size(),
                             copy_valid, _stream(stream, q.device))
    _check(st, "prefill_step")
    return out


def decode_attn(cache, layer, pos, q, out=None, scratch=None, stream=None):
    """Attention of one query token q [H_q, D] at position pos; returns out [H_q, D] f32."""
    _need(q, "q")
    n_head_q = q.shape[0]
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if scratch is None:
        scratch = torch.empty(cache.scratch_bytes(n_head_q), dtype=torch.uint8, device=q.device)
    _need(out, "out", torch.float32); _need(scratch, "scratch")
    st = _lib().decode_attn(ctypes.byref(cache.c), layer, pos, _ptr(q), DTYPES[q.dtype], n_head_q, _ptr(out),
                         _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream, q.device))
    _check(st, "decode_attn")
    return out


def decode_step(cache, layer, pos, q, k, v, out=None, scratch=None, stream=None):
    """One decode step: store k, v [H_kv, D] at position pos (as kv_cache_append) and attend with
    q [H_q, D] over positions [0, pos] (as decode_attn); returns out [H_q, D] f32."""
    _need(q, "q"); _need(k, "k", q.dtype); _need(v, "v", q.dtype)
    n_head_q = q.shape[0]
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if scratch is None:
        scratch = torch.empty(cache.scratch_bytes(n_head_q), dtype=torch.uint8, device=q.device)
    _need(out, "out", torch.float32); _need(scratch, "scratch")
    st = _lib().decode_step(ctypes.byref(cache.c), layer, pos, _ptr(q), _ptr(k), _ptr(v), DTYPES[q.dtype], n_head_q,
                            _ptr(out), _ptr(scratch), scratch.numel() * scratch.element_size(),
                            _stream(stream, q.device))
    _check(st, "decode_step")
    return out


def decode_step_batch(caches, layer, pos, q, k, v, out=None, scratch=None, stream=None):
    """decode_step for len(caches) sequences in one call: q [n_seq][H_q][D], k and v [n_seq][H_kv][D]
    (CUDA), pos a list; returns out [n_seq][H_q][D] f32."""
    n = len(caches)
    if n != len(pos) or q.dim() != 3 or q.shape[0] != n or k.shape[0] != n or v.shape != k.shape:
        raise ValueError("one position, one query and one K/V row block per sequence")
    _need(q, "q"); _need(k, "k", q.dtype); _need(v, "v", q.dtype)
    c0 = caches[0]
    n_head_q = q.shape[1]
    if out is None:
        out = torch.empty(n, n_head_q, c0.head_dim, dtype=torch.float32, device=c0.device)
    _need(out, "out", torch.float32)
    if scratch is None:
        scratch = torch.empty(n * c0.scratch_bytes(n_head_q), dtype=torch.uint8, device=c0.device)
    _need(scratch, "scratch")
    arr = (kvc_cache * n)(*[c.c for c in caches])
    ps = (ctypes.c_int32 * n)(*[int(p) for p in pos])
    st = _lib().decode_step_batch(arr, n, layer, ps, _ptr(q), _ptr(k), _ptr(v), DTYPES[q.dtype], n_head_q, _ptr(out),
                                  _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream, c0.device))
    _check(st, "decode_step_batch")
    return out


def kv_cache_append_batch(caches, layer, pos, k, v, stream=None):
    """Append one token per sequence: row i of k and v ([n_seq][H_kv][D], CUDA) to caches[i] at pos[i]."""
    n = len(caches)
    if n != len(pos) or k.shape[0] != n or v.shape != k.shape or k.dtype != v.dtype:
        raise ValueError("one position and one K/V row block per sequence")
    _need(k, "k"); _need(v, "v")
    arr = (kvc_cache * n)(*[c.c for c in caches])
    ps = (ctypes.c_int32 * n)(*[int(p) for p in pos])
    st = _lib().kv_cache_append_batch(arr, n, layer, ps, _ptr(k), _ptr(v), DTYPES[k.dtype],
                                   _stream(stream, caches[0].device))
    _check(st, "kv_cache_append_batch")


def decode_attn_batch(caches, layer, pos, q, out=None, scratch=None, stream=None):
    """Decode one token for each of len(caches) sequences in one call: q [n_seq][n_head_q][head_dim]
    (CUDA), pos a list of positions; returns out [n_seq][n_head_q][head_dim] float32."""
    n = len(caches)
    if n != len(pos) or q.dim() != 3 or q.shape[0] != n:
        raise ValueError("one position and one query row block per sequence")
    _need(q, "q")
    c0 = caches[0]
    n_head_q = q.shape[1]
    if out is None:
        out = torch.empty(n, n_head_q, c0.head_dim, dtype=torch.float32, device=c0.device)
    _need(out, "out", torch.float32)
    if scratch is None:
        scratch = torch.empty(n * c0.scratch_bytes(n_head_q), dtype=torch.uint8, device=c0.device)
    _need(scratch, "scratch")
    arr = (kvc_cache * n)(*[c.c for c in caches])
    ps = (ctypes.c_int32 * n)(*[int(p) for p in pos])
    st = _lib().decode_attn_batch(arr, n, layer, ps, _ptr(q), DTYPES[q.dtype], n_head_q, _ptr(out), _ptr(scratch),
                               scratch.numel() * scratch.element_size(), _stream(stream, c0.device))
    _check(st, "decode_attn_batch")
    return out


def kv_state_get(cache, n_tokens, dst=None, stream=None):
    """Serialise positions [0, n_tokens) into dst (uint8 CUDA tensor); returns dst."""
    n = cache.state_size(n_tokens)
    if dst is None:
        dst = torch.empty(max(n, 16), dtype=torch.uint8, device=cache.device)
    _need(dst, "dst")
    st = _lib().kv_state_get(ctypes.byref(cache.c), n_tokens, _ptr(dst), dst.numel() * dst.element_size(),
                          _stream(stream, cache.device))
    _check(st, "kv_state_get")
    return dst[:n]


def kv_state_set(cache, src, stream=None):
    """Restore a state (uint8 CUDA tensor of exactly the state's size); returns n_tokens."""
    _need(src, "src")
    n = ctypes.c_int32(-1)
    st = _lib().kv_state_set(ctypes.byref(cache.c), _ptr(src), src.numel() * src.element_size(), ctypes.byref(n),
                          _stream(stream, cache.device))
    _check(st, "kv_state_set")
    return n.value


def kv_state_get_heads(cache, head0, n_head_total, n_tokens, dst=None, stream=None):
    """Write the part of the whole state (n_head_total kv heads) that `cache`, holding kv heads
    [head0, head0 + cache.n_head_kv), owns, plus the header, into dst; returns dst."""
    whole = make_desc(cache.n_layer, cache.n_ctx, n_head_total, cache.head_dim, cache.cache_type, cache.layout)
    n = _lib().kv_state_size(ctypes.byref(whole), n_tokens)
    if dst is None:
        dst = torch.zeros(max(n, 16), dtype=torch.uint8, device=cache.device)
    _need(dst, "dst")
    st = _lib().kv_state_get_heads(ctypes.byref(cache.c), head0, n_head_total, n_tokens, _ptr(dst),
                                dst.numel() * dst.element_size(), _stream(stream, cache.device))
    _check(st, "kv_state_get_heads")
    return dst[:n]


def kv_state_set_heads(cache, head0, src, stream=None):
    """Restore kv heads [head0, head0 + cache.n_head_kv) of a whole state into `cache`; returns n_tokens."""
    _need(src, "src")
    n = ctypes.c_int32(-1)
    st = _lib().kv_state_set_heads(ctypes.byref(cache.c), head0, _ptr(src), src.numel() * src.element_size(),
                                ctypes.byref(n), _stream(stream, cache.device))
    _check(st, "kv_state_set_heads")
    return n.value


def kv_cache_truncate(cache, n_tokens, stream=None):
    """Rewind `cache` to its first n_tokens positions (later positions cleared to zero bytes)."""
    _check(_lib().kv_cache_truncate(ctypes.byref(cache.c), int(n_tokens), _stream(stream, cache.device)),
           "kv_cache_truncate")


class PageTable:
    """The pages of n_seq sequences in a pool (a KVCache whose positions are cut into pages).

    table: int32 [n_seq][max_pages], lengths: int32 [n_seq], contiguous tensors on the pool's device.  They are
    read when a kernel runs, so both may be updated in place between calls (and between replays of a graph, which
    reads the tensors that it was captured with).  Either may also be replaced by assignment: the next call reads the
    new tensor, which has to fit the other one.  An entry outside the pool, such as -1, is a hole.
    """

    def __init__(self, table, lengths, page_size):
        self._check(table, lengths, table.shape[:1], table.device)
        page_size = int(page_size)
        c = kvc_pages(table.data_ptr(), lengths.data_ptr(), table.shape[0], table.shape[1], page_size)
        self.__dict__.update(table=table, lengths=lengths, page_size=page_size, n_seq=table.shape[0],
                             device=table.device, c=c, addr=ctypes.addressof(c))

    @staticmethod
    def _check(table, lengths, n_seq, device):
        _need(table, "table", torch.int32); _need(lengths, "lengths", torch.int32)
        if (table.dim() != 2 or table.shape[:1] != n_seq or lengths.shape != n_seq or table.device != device or
                lengths.device != device):
            raise ValueError("table must be [n_seq][max_pages] and lengths [n_seq], on one device")

    # c holds the tensors' addresses: an assignment that left it alone would have the next call read freed memory
    def __setattr__(self, name, value):
        if name == "table":
            self._check(value, self.lengths, (self.n_seq,), self.device)
            self.c.table, self.c.max_pages = value.data_ptr(), value.shape[1]
        elif name == "lengths":
            self._check(self.table, value, (self.n_seq,), self.device)
            self.c.len = value.data_ptr()
        elif name in self.__dict__:
            raise AttributeError("%s of a PageTable cannot be changed" % name)
        self.__dict__[name] = value


class _Held:
    """Attributes are set once: what a call reads holds their addresses, and one replaced would leave it freed memory."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError("%s of a %s cannot be replaced; its contents can" % (name, type(self).__name__))
        self.__dict__[name] = value


class FreePages(_Held):
    """The free pages of a pool of n_pages pages, for kv_pages_advance: ring (int32 [n_pages]), and state (int32 [3]: where
    the ring begins, how many pages it holds, how many were asked for and not there), on the device.  pages: those
    that are free at first (a sequence or int32 tensor of page numbers, each once); None: all of them, in order."""

    def __init__(self, n_pages, pages=None, device="cuda"):
        if n_pages < 1:
            raise ValueError("a pool has a page or more")
        if pages is None:
            pages = torch.arange(n_pages, dtype=torch.int32)
        elif not isinstance(pages, torch.Tensor):
            pages = torch.tensor(list(pages), dtype=torch.int32)
        if pages.dim() != 1 or pages.dtype != torch.int32 or pages.numel() > n_pages:
            raise ValueError("pages must be at most n_pages int32 page numbers")
        self.n_pages = int(n_pages)
        self.ring = torch.full((self.n_pages,), -1, dtype=torch.int32, device=device)
        self.ring[:pages.numel()] = pages.to(self.ring.device)
        self.state = torch.tensor([0, pages.numel(), 0], dtype=torch.int32).to(self.ring.device)
        self.device = self.ring.device
        self.c = kvc_free_pages(self.ring.data_ptr(), self.state.data_ptr(), self.n_pages)
        self.addr = ctypes.addressof(self.c)

    def free(self):
        """How many pages are free, and how many were asked for and not there (waits for the device)."""
        return tuple(self.state.tolist()[1:])


# The calls below are made once a layer and step with a few rows, where the host's time counts: they look at each
# attribute once and pass plain integers.  A given stream is made the current one, so that what they allocate belongs
# to it.

def _on(device):
    """The current stream of `device`, which has to be the current device."""
    index = device.index
    if torch._C._cuda_getDevice() != index:
        raise ValueError("the tensors are on %s, which is not the current device" % device)
    return torch._C._cuda_getCurrentRawStream(index)


def _packed_rows(t, what, heads, head_dim, dtype, device):
    """Distance between tokens (elements) of a [rows][heads][head_dim] tensor with contiguous heads."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim or t.dtype != dtype or t.device != device:
        raise ValueError("%s must be a %s tensor [rows][%d][%d] on %s" % (what, dtype, heads, head_dim, device))
    ld, hs, es = t.stride()
    if es != 1 or (hs != head_dim and heads != 1):
        raise ValueError("%s must have contiguous heads" % what)
    return ld if shape[0] > 1 else heads * head_dim


def _starts(t, what, n_seq, device):
    if t.shape != (n_seq + 1,) or t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor [n_seq + 1] on %s" % (what, device))
    return t.data_ptr()


def _output(t, what, shape, dtype, device, like=None):
    if t is None:
        if like is not None and like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(shape, dtype=dtype, device=device)
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor %s on %s" % (what, dtype, list(shape), device))
    return t


def _bytes(scratch, device):
    if scratch.device != device or not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous tensor on %s" % device)
    return scratch.nbytes


def _pool(cache, pages):
    if cache.cuda != pages.device:
        raise ValueError("the pool is on %s, its pages on %s" % (cache.cuda, pages.device))
    return pages.device


def kv_pages_advance(pages, free, rows, n_rows, row_start=None, positions=None, slots=None, stream=None):
    """Change the lengths of pages (a PageTable) by rows (int32 [n_seq]; negative: rewound or ended), take the pages that
    they need from free (a FreePages) and give back those that they do not: table, lengths and free are updated in
    place.  Returns (row_start [n_seq + 1], positions [n_rows], slots [n_rows]) of the packed rows that are added."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv_pages_advance(pages, free, rows, n_rows, row_start, positions, slots)
    dev, n = pages.device, pages.n_seq
    if free.device != dev or rows.shape != (n,) or rows.dtype != torch.int32 or rows.device != dev or \
            not rows.is_contiguous():
        raise ValueError("rows must be a contiguous int32 tensor [n_seq], and the free pages be, on %s" % dev)
    row_start = _output(row_start, "row_start", (n + 1,), torch.int32, dev)
    positions = _output(positions, "positions", (n_rows,), torch.int32, dev)
    slots = _output(slots, "slots", (n_rows,), torch.int32, dev, positions)
    st = _lib().kv_pages_advance(pages.addr, free.addr, rows.data_ptr(), row_start.data_ptr(), n_rows,
                                 positions.data_ptr() or None, slots.data_ptr() or None, _on(dev))
    if st:
        raise KvcError(st, "kv_pages_advance")
    if n == 0:
        row_start.zero_()
        positions.fill_(-1)
        slots.fill_(-1)
    return row_start, positions, slots


def kv_paged_append(cache, layer, pages, row_start, k, v, stream=None):
    """Store packed rows k, v [n_rows][H_kv][D]: rows [row_start[i], row_start[i + 1]) are the last positions of
    sequence i (pages.lengths counts them), quantised or rounded as kv_cache_append does."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv_paged_append(cache, layer, pages, row_start, k, v)
    dev, dtype, code = _pool(cache, pages), k.dtype, DTYPES.get(k.dtype)
    ld_k = _packed_rows(k, "k", cache.n_head_kv, cache.head_dim, dtype, dev)
    ld_v = _packed_rows(v, "v", cache.n_head_kv, cache.head_dim, dtype, dev)
    n = k.shape[0]
    if v.shape[0] != n or code is None:
        raise ValueError("k and v must have the same rows and be f32, bf16 or f16")
    st = _lib().kv_paged_append(cache.addr, pages.addr, layer, _starts(row_start, "row_start", pages.n_seq, dev), n,
                                k.data_ptr(), v.data_ptr(), ld_k, ld_v, code, _on(dev))
    if st:
        raise KvcError(st, "kv_paged_append")


def kv_paged_read(cache, layer, pages, row_start, n_rows, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """The values the pool holds for packed rows (as in kv_paged_append): k, v [n_rows][H_kv][D] in dtype."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv_paged_read(cache, layer, pages, row_start, n_rows, dtype, k, v)
    dev, code = _pool(cache, pages), DTYPES.get(dtype)
    if code is None:
        raise ValueError("dtype must be f32, bf16 or f16")
    shape = (n_rows, cache.n_head_kv, cache.head_dim)
    k = _output(k, "k", shape, dtype, dev)
    v = _output(v, "v", shape, dtype, dev, k)
    st = _lib().kv_paged_read(cache.addr, pages.addr, layer, _starts(row_start, "row_start", pages.n_seq, dev), n_rows,
                              k.data_ptr(), v.data_ptr(), code, _on(dev))
    if st:
        raise KvcError(st, "kv_paged_read")
    return k, v


def paged_scratch(cache, n_seq, n_head_q):
    """A scratch buffer for decode_attn_paged (needs no initialisation)."""
    n = ctypes.c_size_t()
    _check(_lib().kvc_paged_scratch_bytes(ctypes.byref(cache.desc), n_seq, n_head_q, ctypes.byref(n)),
           "kvc_paged_scratch_bytes")
    return torch.empty(max(n.value, 16), dtype=torch.uint8, device=cache.device)


def decode_attn_paged(cache, layer, pages, q, out=None, lse=None, scratch=None, stream=None):
    """Attention of one token q[i] [H_q][D] of each sequence over its pages.lengths[i] keys; returns out
    [n_seq][H_q][D] in q's type.  lse: None, or a float32 tensor [n_seq][H_q] to fill."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return decode_attn_paged(cache, layer, pages, q, out, lse, scratch)
    dev, n, dtype, shape = _pool(cache, pages), pages.n_seq, q.dtype, q.shape
    code = DTYPES.get(dtype)
    if len(shape) != 3 or shape[0] != n or code is None:
        raise ValueError("q must be an f32, bf16 or f16 tensor [n_seq][H_q][D]")
    hq = shape[1]
    ld = _packed_rows(q, "q", hq, cache.head_dim, dtype, dev)
    out = _output(out, "out", shape, dtype, dev, q)
    if lse is not None:
        lse = _output(lse, "lse", (n, hq), torch.float32, dev).data_ptr()
    if scratch is None:
        scratch = paged_scratch(cache, n, hq)
    st = _lib().decode_attn_paged(cache.addr, pages.addr, layer, q.data_ptr(), ld, code, hq, out.data_ptr(), lse,
                                  scratch.data_ptr(), _bytes(scratch, dev), _on(dev))
    if st:
        raise KvcError(st, "decode_attn_paged")
    return out


def packed_scratch(n_rows, n_seq, n_head_q, n_head_kv, head_dim, device="cuda"):
    """A scratch buffer for attn_packed calls of up to n_rows query rows and n_seq sequences."""
    n = ctypes.c_size_t()
    _check(_lib().kvc_packed_scratch_bytes(n_rows, n_seq, n_head_q, n_head_kv, head_dim, ctypes.byref(n)),
           "kvc_packed_scratch_bytes")
    return torch.empty(max(n.value, 16), dtype=torch.uint8, device=device)


def attn_packed(q, k, v, q_start, k_start=None, out=None, lse=None, scratch=None, stream=None):
    """Causal attention of packed prompts: q [n_q][H_q][D], k and v [n_k][H_kv][D] (bf16 or f16); sequence s has
    query rows [q_start[s], q_start[s + 1]) and keys [k_start[s], k_start[s + 1]) (q_start when None), its queries
    being its last positions.  Returns out like q, contiguous.  lse: None, or a float32 [n_q][H_q] to fill."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return attn_packed(q, k, v, q_start, k_start, out, lse, scratch)
    dev, dtype, qshape, kshape = q.device, q.dtype, q.shape, k.shape
    if len(qshape) != 3 or len(kshape) != 3 or dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q, k and v must be bf16 or f16 tensors [rows][heads][D]")
    if v.shape != kshape or dev.type != "cuda":
        raise ValueError("k and v must have the same rows, on a CUDA device")
    n_q, hq, d = qshape
    n_k, hkv = kshape[0], kshape[1]
    n_seq = q_start.shape[0] - 1
    ld_q = _packed_rows(q, "q", hq, d, dtype, dev)
    ld_k, ld_v = _packed_rows(k, "k", hkv, d, dtype, dev), _packed_rows(v, "v", hkv, d, dtype, dev)
    qs = _starts(q_start, "q_start", n_seq, dev)
    ks = qs if k_start is None else _starts(k_start, "k_start", n_seq, dev)
    out = _output(out, "out", qshape, dtype, dev, q)
    if lse is not None:
        lse = _output(lse, "lse", (n_q, hq), torch.float32, dev).data_ptr()
    if scratch is None:
        scratch = packed_scratch(n_q, n_seq, hq, hkv, d, dev)
    st = _lib().attn_packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), ld_q, ld_k, ld_v, DTYPES[dtype], qs, ks, n_seq,
                            n_q, n_k, hq, hkv, d, out.data_ptr(), lse, scratch.data_ptr(), _bytes(scratch, dev),
                            _on(dev))
    if st:
        raise KvcError(st, "attn_packed")
    return out


ROPE_STYLES = {"half": 0, "pairs": 1}


class RopeTable(_Held):
    """A rotation by position of the first `rot` values of each head: pairs (i, i + rot / 2) ("half") or (2 i, 2 i + 1)
    ("pairs"), pair i by position * base ** (-2 i / rot), or by position * inv_freq[i] where inv_freq (a sequence or
    tensor of rot / 2 frequencies in radians) is given.  The frequencies, as float64, are kept as 64-bit fractions of a
    turn on `device`: angles are exact to 2^-32 of a turn at any position, and rounded to float32 beside the nearest
    quarter of a turn (2^-28 of a turn at most).  rot = 0: no rotation.  The calls take "half" with rot a multiple of 16.
    Make it once for a model and keep it: making one works the frequencies out on the host and copies them."""

    def __init__(self, rot, base=10000.0, style="half", inv_freq=None, device="cuda"):
        if rot < 0 or rot % 2 or style not in ROPE_STYLES:
            raise ValueError('rot must be even and style "half" or "pairs"')
        if inv_freq is None and not 0 < base < math.inf:
            raise ValueError("base must be positive and finite")
        n = rot // 2
        if inv_freq is None:
            freq = [float(base) ** (-2.0 * i / rot) for i in range(n)]
        else:
            freq = [float(f) for f in inv_freq]
        if len(freq) != n or not all(math.isfinite(f) for f in freq):
            raise ValueError("inv_freq must be rot / 2 finite frequencies")
        self.turns = torch.tensor([_turns(f) for f in freq], dtype=torch.int64).to(device)
        self.rot, self.style, self.device = rot, style, self.turns.device
        self.c = kvc_rope(self.turns.data_ptr() if n else None, n, ROPE_STYLES[style])
        self.addr = ctypes.addressof(self.c)


def _weight(w, what, head_dim, dtype, device):
    if w is None:
        return None
    if w.shape != (head_dim,) or w.dtype != dtype or w.device != device or not w.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor [%d] on %s" % (what, dtype, head_dim, device))
    return w.data_ptr()


def _rows_out(t, what, like, heads, head_dim, dtype, device):
    """An output of packed rows, which may have a distance of its own between rows: (tensor, ld)."""
    if t is None:
        t = torch.empty(like.shape, dtype=dtype, device=device)
        return t, heads * head_dim
    ld = _packed_rows(t, what, heads, head_dim, dtype, device)
    if t.shape[0] != like.shape[0]:
        raise ValueError("%s must have the rows of its input" % what)
    return t, ld


def qk_norm_rope(q, k, positions, rope, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Norms and rotation of packed rows in one pass: q [rows][H_q][D], k [rows][H_kv][D] divided by their root mean
    square for each head (where a weight [D] of their type is given) times the weight, then rotated by positions
    (int32 [rows]) as rope (a RopeTable) says.  Returns (q_out, k_out); outputs may be the inputs themselves."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qk_norm_rope(q, k, positions, rope, q_weight, k_weight, eps, q_out, k_out)
    dev, dtype, code = q.device, q.dtype, DTYPES.get(q.dtype)
    if q.dim() != 3 or k.dim() != 3 or code is None or dev.type != "cuda" or rope.device != dev:
        raise ValueError("q and k must be f32, bf16 or f16 tensors [rows][heads][D] on the rope's CUDA device")
    n, hq, d = q.shape
    hkv = k.shape[1]
    ld_q, ld_k = _packed_rows(q, "q", hq, d, dtype, dev), _packed_rows(k, "k", hkv, d, dtype, dev)
    if k.shape[0] != n:
        raise ValueError("q and k must have the same rows")
    if positions.shape != (n,) or positions.dtype != torch.int32 or positions.device != dev or \
            not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 tensor [rows] on %s" % dev)
    qw, kw = _weight(q_weight, "q_weight", d, dtype, dev), _weight(k_weight, "k_weight", d, dtype, dev)
    q_out, ld_qo = _rows_out(q_out, "q_out", q, hq, d, dtype, dev)
    k_out, ld_ko = _rows_out(k_out, "k_out", k, hkv, d, dtype, dev)
    st = _lib().qk_norm_rope(rope.addr, q.data_ptr(), k.data_ptr(), ld_q, ld_k, code, n, hq, hkv, d,
                             positions.data_ptr(), qw, kw, eps, q_out.data_ptr(), k_out.data_ptr(), ld_qo, ld_ko, _on(dev))
    if st:
        raise KvcError(st, "qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_append(cache, layer, pages, row_start, q, k, v, rope, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
                        stream=None):
    """qk_norm_rope of packed rows at the positions that pages and row_start give them, and kv_paged_append of the
    resulting keys and of v, in one pass.  Returns the queries."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qk_norm_rope_append(cache, layer, pages, row_start, q, k, v, rope, q_weight, k_weight, eps, q_out)
    dev, dtype, code = _pool(cache, pages), q.dtype, DTYPES.get(q.dtype)
    if q.dim() != 3 or code is None or rope.device != dev:
        raise ValueError("q must be an f32, bf16 or f16 tensor [rows][H_q][D], the rope on its device")
    n, hq, d = q.shape[0], q.shape[1], cache.head_dim
    ld_q = _packed_rows(q, "q", hq, d, dtype, dev)
    ld_k = _packed_rows(k, "k", cache.n_head_kv, d, dtype, dev)
    ld_v = _packed_rows(v, "v", cache.n_head_kv, d, dtype, dev)
    if k.shape[0] != n or v.shape[0] != n:
        raise ValueError("q, k and v must have the same rows")
    qw, kw = _weight(q_weight, "q_weight", d, dtype, dev), _weight(k_weight, "k_weight", d, dtype, dev)
    q_out, ld_qo = _rows_out(q_out, "q_out", q, hq, d, dtype, dev)
    st = _lib().qk_norm_rope_append(cache.addr, pages.addr, layer, _starts(row_start, "row_start", pages.n_seq, dev), n,
                                    rope.addr, q.data_ptr(), k.data_ptr(), v.data_ptr(), ld_q, ld_k, ld_v, code, hq, qw, kw,
                                    eps, q_out.data_ptr(), ld_qo, _on(dev))
    if st:
        raise KvcError(st, "qk_norm_rope_append")
    return q_out


def kvc_device_status():
    """Synchronise and read/clear the device status word (non-zero: a kernel gave up a bounded wait,
    which the C call reports as KVC_EDEVICE)."""
    s = ctypes.c_int32(0)
    rc = _lib().kvc_device_status(ctypes.byref(s))
    if rc != KVC_EDEVICE:
        _check(rc, "kvc_device_status")
    return s.value


TEST_PREFILL, TEST_DECODE, TEST_PAGED, TEST_PACKED = 0, 1, 2, 3


def arm_test_wait_timeout(which, limit_ns):
    """Test hook: the next launch of the prefill (TEST_PREFILL), head_dim-128 decode (TEST_DECODE), paged decode
    (TEST_PAGED) or packed (TEST_PACKED) kernel waits on a barrier nothing arrives at, gives up after limit_ns and unwinds."""
    _check(_lib().kvc_test_arm_wait_timeout(which, limit_ns), "kvc_test_arm_wait_timeout")
