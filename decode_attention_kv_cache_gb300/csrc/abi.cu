// The C ABI (include/kvc.h): argument checks, size queries and dispatch.
//
// Every check runs before anything is launched, so a call that fails leaves
// the cache untouched and usable - the error contract of the pages' state
// switch (llama.cpp PR #58 "completion : allow the prompt to be processed
// under its own split mode", section "Memory": a mode that does not fit must
// not lose the request; llama.cpp PR #59 "llama : switch the split mode of a
// live context", section "What this adds": the call returns false and the
// caller keeps a working context).
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>

#include "kvc_internal.h"

using namespace kvc;

namespace kvc {
namespace {
std::atomic<uint64_t> g_test_stall[4];   // per kernel kind: wait limit of the armed stall, 0 = none
}  // namespace
void arm_test_stall(int which, uint64_t limit_ns) { g_test_stall[which].store(limit_ns); }
uint64_t take_test_stall(int which) { return g_test_stall[which].exchange(0); }
}  // namespace kvc

namespace {

constexpr uint32_t STATE_MAGIC = 0x3143564Bu;  // 'K' 'V' 'C' '1' little-endian
constexpr uint32_t STATE_VERSION = 1u;
constexpr size_t STATE_HEADER = 32;

// any cache: what the calls on pools of pages take
bool pool_desc_ok(const kvc_desc *d) {
    if (!d) return false;
    if (d->n_layer <= 0 || d->n_ctx <= 0 || d->n_head_kv <= 0 || d->head_dim <= 0) return false;
    if (d->head_dim % 32 != 0 || d->head_dim > 1024) return false;
    if (d->type != KVC_F16 && d->type != KVC_Q8_0 && d->type != KVC_Q4_0) return false;
    if (d->layout != KVC_HEAD_MAJOR && d->layout != KVC_LAYER_MAJOR) return false;
    return true;
}

// one that every call takes: q4_0 is a type of pools
bool desc_ok(const kvc_desc *d) { return pool_desc_ok(d) && d->type != KVC_Q4_0; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// True when p is device memory of the current device (or managed memory the runtime attributes to it).
bool on_current_device(const void *p) {
    int dev = -1;
    cudaPointerAttributes at;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();   // a failed query leaves no sticky error behind
        return false;
    }
    return (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) && at.device == dev;
}

bool pool_ok(const kvc_cache *c) {
    if (!c || !pool_desc_ok(&c->d)) return false;
    if (!c->k_q || !c->v_q || !aligned16(c->k_q) || !aligned16(c->v_q)) return false;
    if (has_scales(c->d.type) && (!c->k_s || !c->v_s || !aligned16(c->k_s) || !aligned16(c->v_s)))
        return false;
    return true;
}

bool cache_ok(const kvc_cache *c) { return pool_ok(c) && desc_ok(&c->d); }

size_t elems(const kvc_desc &d) { return (size_t)d.n_layer * d.n_ctx * d.n_head_kv * d.head_dim; }

size_t record_bytes(const kvc_desc &d) {
    return d.type == KVC_Q8_0 ? (size_t)d.n_head_kv * (d.head_dim / 32) * 34
                              : (size_t)d.n_head_kv * d.head_dim * 2;
}

bool pages_ok(const kvc_cache *c, const kvc_pages *p) {
    return p && p->n_seq >= 0 && p->n_seq <= 65535 && p->max_pages > 0 && p->page_size > 0 && p->page_size % 16 == 0 &&
           c->d.n_ctx % p->page_size == 0 && (int64_t)p->max_pages * p->page_size <= INT32_MAX;
}

// whether ld is a distance between tokens of `heads` heads of the type: no overlap, 16-byte rows
bool ld_ok(int64_t ld, int64_t heads, int64_t head_dim, int dtype) {
    return ld >= heads * head_dim && ld * dtype_bytes(dtype) % 16 == 0 && ld < ((int64_t)1 << 38);
}

bool dtype_ok(int dtype) { return dtype == KVC_IN_F32 || dtype == KVC_IN_BF16 || dtype == KVC_IN_F16; }

}  // namespace

extern "C" {

int kvc_cache_bytes(const kvc_desc *desc, size_t *k_q, size_t *k_s, size_t *v_q, size_t *v_s) {
    if (!pool_desc_ok(desc) || !k_q || !k_s || !v_q || !v_s) return KVC_EINVAL;
    const size_t n = elems(*desc);
    *k_q = *v_q = (size_t)code_bytes(desc->type, (int64_t)n);
    *k_s = *v_s = has_scales(desc->type) ? n / 32 * 2 : 0;
    return KVC_OK;
}

int kvc_scratch_bytes(const kvc_desc *desc, int32_t n_head_q, size_t *bytes) {
    if (!desc_ok(desc) || !bytes || n_head_q <= 0 || n_head_q % desc->n_head_kv) return KVC_EINVAL;
    *bytes = (size_t)n_head_q * decode_max_split() * (desc->head_dim + 2) * sizeof(float);
    return KVC_OK;
}

size_t kv_state_size(const kvc_desc *desc, int32_t n_tokens) {
    if (!desc_ok(desc) || n_tokens < 0 || n_tokens > desc->n_ctx) return 0;
    return STATE_HEADER + (size_t)desc->n_layer * n_tokens * 2 * record_bytes(*desc);
}

int kvc_cache_init(kvc_cache *out, const kvc_desc *desc, void *k_q, void *k_s, void *v_q, void *v_s) {
    if (!out || !pool_desc_ok(desc)) return KVC_EINVAL;
    kvc_cache c;
    c.d = *desc;
    c.k_q = k_q;
    c.k_s = has_scales(desc->type) ? k_s : nullptr;
    c.v_q = v_q;
    c.v_s = has_scales(desc->type) ? v_s : nullptr;
    if (!pool_ok(&c)) return KVC_EINVAL;
    *out = c;
    return KVC_OK;
}

int kv_cache_append(const kvc_cache *cache, int32_t layer, int32_t pos0, int32_t n_tokens,
                    const void *k, const void *v, int32_t dtype, kvc_stream_t stream) {
    if (!cache_ok(cache) || !dtype_ok(dtype)) return KVC_EINVAL;
    if (n_tokens < 0) return KVC_EINVAL;
    if (layer < 0 || layer >= cache->d.n_layer || pos0 < 0 || (int64_t)pos0 + n_tokens > cache->d.n_ctx)
        return KVC_ERANGE;
    if (n_tokens == 0) return KVC_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return KVC_EINVAL;
    return launch_append(*cache, layer, pos0, n_tokens, k, v, dtype, (cudaStream_t)stream);
}

int kv_cache_append_batch(const kvc_cache *caches, int32_t n_seq, int32_t layer, const int32_t *pos, const void *k,
                          const void *v, int32_t dtype, kvc_stream_t stream) {
    if (!caches || !pos || n_seq < 1 || n_seq > append_max_batch() || !dtype_ok(dtype)) return KVC_EINVAL;
    const kvc_desc &d = caches[0].d;
    for (int i = 0; i < n_seq; ++i) {
        const kvc_desc &e = caches[i].d;
        if (!cache_ok(&caches[i]) || e.n_head_kv != d.n_head_kv || e.head_dim != d.head_dim || e.type != d.type)
            return KVC_EINVAL;
    }
    for (int i = 0; i < n_seq; ++i)
        if (layer < 0 || layer >= caches[i].d.n_layer || pos[i] < 0 || pos[i] >= caches[i].d.n_ctx) return KVC_ERANGE;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return KVC_EINVAL;
    return launch_append_batch(caches, n_seq, layer, pos, k, v, dtype, (cudaStream_t)stream);
}

int kvc_prefill_scratch_bytes(const kvc_desc *desc, int32_t n_head_q, int32_t max_tokens, size_t *bytes) {
    if (!desc_ok(desc) || !bytes || n_head_q <= 0 || n_head_q % desc->n_head_kv) return KVC_EINVAL;
    if (max_tokens <= 0 || max_tokens > desc->n_ctx) return KVC_ERANGE;
    const size_t b = prefill_scratch_bytes(*desc, n_head_q, max_tokens);
    if (b == 0) return KVC_EINVAL;
    *bytes = b;
    return KVC_OK;
}

int prefill_chunk_attn(const kvc_cache *cache, int32_t layer, int32_t pos0, int32_t n_tokens,
                       const void *q, int32_t dtype, int32_t n_head_q, float *out, void *scratch,
                       size_t scratch_bytes, kvc_stream_t stream) {
    if (!cache_ok(cache) || !dtype_ok(dtype)) return KVC_EINVAL;
    if (cache->d.head_dim != 64 && cache->d.head_dim != 128) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_q % cache->d.n_head_kv || n_head_q > 65535 || n_tokens < 0) return KVC_EINVAL;
    if (layer < 0 || layer >= cache->d.n_layer || pos0 < 0 || (int64_t)pos0 + n_tokens > cache->d.n_ctx)
        return KVC_ERANGE;
    if (n_tokens == 0) return KVC_OK;
    if (!q || !out || !scratch || !aligned16(q) || !aligned16(out) || !aligned16(scratch)) return KVC_EINVAL;
    return launch_prefill(*cache, layer, pos0, n_tokens, q, dtype, n_head_q, out, scratch, scratch_bytes,
                          (cudaStream_t)stream);
}

int prefill_step(const kvc_cache *cache, int32_t layer, int32_t pos0, int32_t n_tokens, const void *q, const void *k,
                 const void *v, int32_t dtype, int32_t n_head_q, float *out, void *scratch, size_t scratch_bytes,
                 int32_t copy_valid, kvc_stream_t stream) {
    if (!cache_ok(cache) || !dtype_ok(dtype)) return KVC_EINVAL;
    if (cache->d.head_dim != 64 && cache->d.head_dim != 128) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_q % cache->d.n_head_kv || n_head_q > 65535 || n_tokens < 0) return KVC_EINVAL;
    if (layer < 0 || layer >= cache->d.n_layer || pos0 < 0 || (int64_t)pos0 + n_tokens > cache->d.n_ctx ||
        copy_valid < 0 || copy_valid > pos0)
        return KVC_ERANGE;
    if (n_tokens == 0) return KVC_OK;
    if (!q || !k || !v || !out || !scratch || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
        !aligned16(scratch))
        return KVC_EINVAL;
    return launch_prefill_step(*cache, layer, pos0, n_tokens, q, k, v, dtype, n_head_q, out, scratch, scratch_bytes,
                               copy_valid, (cudaStream_t)stream);
}

int decode_attn(const kvc_cache *cache, int32_t layer, int32_t pos, const void *q, int32_t dtype,
                int32_t n_head_q, float *out, void *scratch, size_t scratch_bytes, kvc_stream_t stream) {
    if (!cache_ok(cache) || !dtype_ok(dtype)) return KVC_EINVAL;
    if (cache->d.head_dim != 64 && cache->d.head_dim != 128) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_q % cache->d.n_head_kv || n_head_q / cache->d.n_head_kv > 16)
        return KVC_EINVAL;
    if (layer < 0 || layer >= cache->d.n_layer || pos < 0 || pos >= cache->d.n_ctx) return KVC_ERANGE;
    if (!q || !out || !scratch || !aligned16(q) || !aligned16(out) || !aligned16(scratch)) return KVC_EINVAL;
    size_t need = 0;
    kvc_scratch_bytes(&cache->d, n_head_q, &need);
    if (scratch_bytes < need) return KVC_ENOSPC;
    return launch_decode(*cache, layer, pos, q, dtype, n_head_q, out, static_cast<float *>(scratch),
                         (cudaStream_t)stream);
}

int decode_step(const kvc_cache *cache, int32_t layer, int32_t pos, const void *q, const void *k, const void *v,
                int32_t dtype, int32_t n_head_q, float *out, void *scratch, size_t scratch_bytes, kvc_stream_t stream) {
    if (!cache_ok(cache) || !dtype_ok(dtype)) return KVC_EINVAL;
    if (cache->d.head_dim != 64 && cache->d.head_dim != 128) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_q % cache->d.n_head_kv || n_head_q / cache->d.n_head_kv > 16)
        return KVC_EINVAL;
    if (layer < 0 || layer >= cache->d.n_layer || pos < 0 || pos >= cache->d.n_ctx) return KVC_ERANGE;
    if (!q || !k || !v || !out || !scratch || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
        !aligned16(scratch))
        return KVC_EINVAL;
    size_t need = 0;
    kvc_scratch_bytes(&cache->d, n_head_q, &need);
    if (scratch_bytes < need) return KVC_ENOSPC;
    return launch_decode_step(*cache, layer, pos, q, k, v, dtype, n_head_q, out, static_cast<float *>(scratch),
                              (cudaStream_t)stream);
}

int decode_step_batch(const kvc_cache *caches, int32_t n_seq, int32_t layer, const int32_t *pos, const void *q,
                      const void *k, const void *v, int32_t dtype, int32_t n_head_q, float *out, void *scratch,
                      size_t scratch_bytes, kvc_stream_t stream) {
    if (!caches || !pos || n_seq < 1 || n_seq > decode_max_batch() || !dtype_ok(dtype)) return KVC_EINVAL;
    const kvc_desc &d = caches[0].d;
    for (int i = 0; i < n_seq; ++i) {
        const kvc_desc &e = caches[i].d;
        if (!cache_ok(&caches[i]) || e.n_layer != d.n_layer || e.n_ctx != d.n_ctx || e.n_head_kv != d.n_head_kv ||
            e.head_dim != d.head_dim || e.type != d.type)
            return KVC_EINVAL;
    }
    if (d.head_dim != 64 && d.head_dim != 128) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_q % d.n_head_kv || n_head_q / d.n_head_kv > 16) return KVC_EINVAL;
    for (int i = 0; i < n_seq; ++i)
        if (layer < 0 || layer >= d.n_layer || pos[i] < 0 || pos[i] >= d.n_ctx) return KVC_ERANGE;
    if (!q || !k || !v || !out || !scratch || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
        !aligned16(scratch))
        return KVC_EINVAL;
    size_t need = 0;
    kvc_scratch_bytes(&d, n_head_q, &need);
    if (scratch_bytes / (size_t)n_seq < need) return KVC_ENOSPC;
    return launch_decode_step_batch(caches, n_seq, layer, pos, q, k, v, dtype, n_head_q, out,
                                    static_cast<float *>(scratch), need, (cudaStream_t)stream);
}

int decode_attn_noalloc(const kvc_cache *cache, int32_t layer, int32_t pos, const void *q, int32_t dtype,
                        int32_t n_head_q, float *out, kvc_stream_t stream) {
    if (!cache_ok(cache) || !dtype_ok(dtype)) return KVC_EINVAL;
    if (cache->d.head_dim != 64 && cache->d.head_dim != 128) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_q % cache->d.n_head_kv || n_head_q / cache->d.n_head_kv > 16)
        return KVC_EINVAL;
    if (layer < 0 || layer >= cache->d.n_layer || pos < 0 || pos >= cache->d.n_ctx) return KVC_ERANGE;
    if (!q || !out || !aligned16(q) || !aligned16(out)) return KVC_EINVAL;
    size_t need = 0;
    kvc_scratch_bytes(&cache->d, n_head_q, &need);
    if (need > decode_noalloc_capacity()) return KVC_ENOSPC;  // more partials than the fixed array holds
    // the partials go to the current device's array: the cache and the output must live there too
    if (!on_current_device(cache->k_q) || !on_current_device(out)) return KVC_EINVAL;
    return launch_decode_noalloc(*cache, layer, pos, q, dtype, n_head_q, out, (cudaStream_t)stream);
}

int decode_attn_batch(const kvc_cache *caches, int32_t n_seq, int32_t layer, const int32_t *pos, const void *q,
                      int32_t dtype, int32_t n_head_q, float *out, void *scratch, size_t scratch_bytes,
                      kvc_stream_t stream) {
    if (!caches || !pos || n_seq < 1 || n_seq > decode_max_batch() || !dtype_ok(dtype)) return KVC_EINVAL;
    const kvc_desc &d = caches[0].d;
    for (int i = 0; i < n_seq; ++i) {
        const kvc_desc &e = caches[i].d;
        if (!cache_ok(&caches[i]) || e.n_layer != d.n_layer || e.n_ctx != d.n_ctx || e.n_head_kv != d.n_head_kv ||
            e.head_dim != d.head_dim || e.type != d.type)
            return KVC_EINVAL;
    }
    if (d.head_dim != 64 && d.head_dim != 128) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_q % d.n_head_kv || n_head_q / d.n_head_kv > 16) return KVC_EINVAL;
    if (layer < 0 || layer >= d.n_layer) return KVC_ERANGE;
    for (int i = 0; i < n_seq; ++i)
        if (pos[i] < 0 || pos[i] >= d.n_ctx) return KVC_ERANGE;
    if (!q || !out || !scratch || !aligned16(q) || !aligned16(out) || !aligned16(scratch)) return KVC_EINVAL;
    size_t need = 0;
    kvc_scratch_bytes(&d, n_head_q, &need);
    if (scratch_bytes / (size_t)n_seq < need) return KVC_ENOSPC;
    return launch_decode_batch(caches, n_seq, layer, pos, q, dtype, n_head_q, out, static_cast<float *>(scratch),
                               need, (cudaStream_t)stream);
}

int kv_state_get(const kvc_cache *cache, int32_t n_tokens, void *dst, size_t dst_bytes, kvc_stream_t stream) {
    if (!cache_ok(cache) || !dst || !aligned16(dst) || n_tokens < 0) return KVC_EINVAL;
    if (n_tokens > cache->d.n_ctx) return KVC_ERANGE;
    if (dst_bytes < kv_state_size(&cache->d, n_tokens)) return KVC_ENOSPC;
    return launch_state_pack(*cache, n_tokens, static_cast<uint8_t *>(dst), (cudaStream_t)stream);
}

int kv_state_set(kvc_cache *cache, const void *src, size_t src_bytes, int32_t *n_tokens_out,
                 kvc_stream_t stream) {
    if (!cache_ok(cache) || !src || !aligned16(src) || !n_tokens_out) return KVC_EINVAL;
    if (src_bytes < STATE_HEADER) return KVC_EFORMAT;
    uint32_t h[8];
    cudaStream_t s = (cudaStream_t)stream;
    if (cudaMemcpyAsync(h, src, sizeof(h), cudaMemcpyDeviceToHost, s) != cudaSuccess) return KVC_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return KVC_ECUDA;
    const kvc_desc &d = cache->d;
    if (h[0] != STATE_MAGIC || h[1] != STATE_VERSION) return KVC_EFORMAT;
    if (h[2] != (uint32_t)d.n_layer || h[3] != (uint32_t)d.n_head_kv || h[4] != (uint32_t)d.head_dim ||
        h[5] != (uint32_t)d.type || h[7] != 0u)
        return KVC_EFORMAT;
    if (h[6] > (uint32_t)d.n_ctx) return KVC_EFORMAT;
    const int32_t n = (int32_t)h[6];
    if (src_bytes != kv_state_size(&d, n)) return KVC_EFORMAT;
    const int rc = launch_state_unpack(*cache, n, static_cast<const uint8_t *>(src), s);
    if (rc == KVC_OK) *n_tokens_out = n;
    return rc;
}

int kv_state_get_heads(const kvc_cache *cache, int32_t head0, int32_t n_head_total, int32_t n_tokens, void *dst,
                       size_t dst_bytes, kvc_stream_t stream) {
    if (!cache_ok(cache) || !dst || !aligned16(dst) || n_tokens < 0) return KVC_EINVAL;
    if (head0 < 0 || n_head_total <= 0 || (int64_t)head0 + cache->d.n_head_kv > n_head_total) return KVC_EINVAL;
    if (n_tokens > cache->d.n_ctx) return KVC_ERANGE;
    kvc_desc whole = cache->d;
    whole.n_head_kv = n_head_total;
    if (dst_bytes < kv_state_size(&whole, n_tokens)) return KVC_ENOSPC;
    return launch_state_pack_heads(*cache, head0, n_head_total, n_tokens, static_cast<uint8_t *>(dst),
                                   (cudaStream_t)stream);
}

int kv_state_set_heads(kvc_cache *cache, int32_t head0, const void *src, size_t src_bytes, int32_t *n_tokens_out,
                       kvc_stream_t stream) {
    if (!cache_ok(cache) || !src || !aligned16(src) || !n_tokens_out || head0 < 0) return KVC_EINVAL;
    if (src_bytes < STATE_HEADER) return KVC_EFORMAT;
    uint32_t h[8];
    cudaStream_t s = (cudaStream_t)stream;
    if (cudaMemcpyAsync(h, src, sizeof(h), cudaMemcpyDeviceToHost, s) != cudaSuccess) return KVC_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return KVC_ECUDA;
    const kvc_desc &d = cache->d;
    if (h[0] != STATE_MAGIC || h[1] != STATE_VERSION) return KVC_EFORMAT;
    if (h[2] != (uint32_t)d.n_layer || h[4] != (uint32_t)d.head_dim || h[5] != (uint32_t)d.type || h[7] != 0u)
        return KVC_EFORMAT;
    if (h[3] == 0u || h[3] > 65536u || (uint64_t)head0 + d.n_head_kv > h[3]) return KVC_EFORMAT;
    if (h[6] > (uint32_t)d.n_ctx) return KVC_EFORMAT;
    const int32_t n = (int32_t)h[6];
    kvc_desc whole = d;
    whole.n_head_kv = (int32_t)h[3];
    if (src_bytes != kv_state_size(&whole, n)) return KVC_EFORMAT;
    const int rc = launch_state_unpack_heads(*cache, head0, (int)h[3], n, static_cast<const uint8_t *>(src), s);
    if (rc == KVC_OK) *n_tokens_out = n;
    return rc;
}

int kv_paged_append(const kvc_cache *pool, const kvc_pages *pages, int32_t layer, const int32_t *row_start,
                    int32_t n_rows, const void *k, const void *v, int64_t ld_k, int64_t ld_v, int32_t dtype,
                    kvc_stream_t stream) {
    if (!pool_ok(pool) || !pages_ok(pool, pages) || !dtype_ok(dtype) || n_rows < 0) return KVC_EINVAL;
    if (!ld_ok(ld_k, pool->d.n_head_kv, pool->d.head_dim, dtype) ||
        !ld_ok(ld_v, pool->d.n_head_kv, pool->d.head_dim, dtype))
        return KVC_EINVAL;
    if (layer < 0 || layer >= pool->d.n_layer) return KVC_ERANGE;
    if (n_rows == 0 || pages->n_seq == 0) return KVC_OK;
    if (!pages->table || !pages->len || !row_start || !k || !v || !aligned16(k) || !aligned16(v)) return KVC_EINVAL;
    return launch_paged_append(*pool, *pages, layer, row_start, n_rows, k, v, ld_k, ld_v, dtype, (cudaStream_t)stream);
}

int kv_paged_read(const kvc_cache *pool, const kvc_pages *pages, int32_t layer, const int32_t *row_start,
                  int32_t n_rows, void *k, void *v, int32_t dtype, kvc_stream_t stream) {
    if (!pool_ok(pool) || !pages_ok(pool, pages) || !dtype_ok(dtype) || n_rows < 0) return KVC_EINVAL;
    if (layer < 0 || layer >= pool->d.n_layer) return KVC_ERANGE;
    if (n_rows == 0 || pages->n_seq == 0) return KVC_OK;
    if (!pages->table || !pages->len || !row_start || !k || !v || !aligned16(k) || !aligned16(v)) return KVC_EINVAL;
    return launch_paged_read(*pool, *pages, layer, row_start, n_rows, k, v, dtype, (cudaStream_t)stream);
}

int kvc_paged_scratch_bytes(const kvc_desc *desc, int32_t n_seq, int32_t n_head_q, size_t *bytes) {
    if (!pool_desc_ok(desc) || !bytes || n_seq < 0 || n_seq > 65535) return KVC_EINVAL;
    if (desc->head_dim != 64 && desc->head_dim != 128) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_q % desc->n_head_kv || n_head_q / desc->n_head_kv > 16) return KVC_EINVAL;
    if (desc->type == KVC_Q4_0 && desc->n_head_kv > 65535) return KVC_EINVAL;   // distances between rows in 32 bits
    *bytes = paged_scratch_bytes(*desc, n_seq, n_head_q);
    return KVC_OK;
}

int decode_attn_paged(const kvc_cache *pool, const kvc_pages *pages, int32_t layer, const void *q, int64_t ld_q,
                      int32_t dtype, int32_t n_head_q, void *out, float *lse, void *scratch, size_t scratch_bytes,
                      kvc_stream_t stream) {
    if (!pool_ok(pool) || !pages_ok(pool, pages) || !dtype_ok(dtype)) return KVC_EINVAL;
    size_t need = 0;
    if (kvc_paged_scratch_bytes(&pool->d, pages->n_seq, n_head_q, &need) != KVC_OK) return KVC_EINVAL;
    if (!ld_ok(ld_q, n_head_q, pool->d.head_dim, dtype)) return KVC_EINVAL;
    if (layer < 0 || layer >= pool->d.n_layer) return KVC_ERANGE;
    if (pages->n_seq == 0) return KVC_OK;
    if (!pages->table || !pages->len || !q || !out || !scratch || !aligned16(q) || !aligned16(out) ||
        !aligned16(scratch))
        return KVC_EINVAL;
    if (scratch_bytes < need) return KVC_ENOSPC;
    return launch_decode_paged(*pool, *pages, layer, q, ld_q, dtype, n_head_q, out, lse, scratch, (cudaStream_t)stream);
}

int kvc_packed_scratch_bytes(int32_t n_rows, int32_t n_seq, int32_t n_head_q, int32_t n_head_kv, int32_t head_dim,
                             size_t *bytes) {
    if (!bytes || n_rows < 0 || n_seq < 0 || n_seq > 65535 || (head_dim != 64 && head_dim != 128)) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_kv <= 0 || n_head_q > 65535 || n_head_q % n_head_kv || n_head_q / n_head_kv > 128)
        return KVC_EINVAL;
    *bytes = packed_scratch_bytes(n_rows, n_seq, n_head_q, n_head_kv, head_dim);
    return KVC_OK;
}

int attn_packed(const void *q, const void *k, const void *v, int64_t ld_q, int64_t ld_k, int64_t ld_v, int32_t dtype,
                const int32_t *q_start, const int32_t *k_start, int32_t n_seq, int32_t n_q, int32_t n_k,
                int32_t n_head_q, int32_t n_head_kv, int32_t head_dim, void *out, float *lse, void *scratch,
                size_t scratch_bytes, kvc_stream_t stream) {
    size_t need = 0;
    if (n_k < 0 || (dtype != KVC_IN_BF16 && dtype != KVC_IN_F16)) return KVC_EINVAL;
    if (kvc_packed_scratch_bytes(n_q, n_seq, n_head_q, n_head_kv, head_dim, &need) != KVC_OK) return KVC_EINVAL;
    if (!ld_ok(ld_q, n_head_q, head_dim, dtype) || !ld_ok(ld_k, n_head_kv, head_dim, dtype) ||
        !ld_ok(ld_v, n_head_kv, head_dim, dtype))
        return KVC_EINVAL;
    if (n_q == 0 || n_seq == 0) return KVC_OK;
    if (!q || !out || !scratch || !q_start || !k_start || !aligned16(q) || !aligned16(out) || !aligned16(scratch))
        return KVC_EINVAL;
    if (n_k > 0 && (!k || !v || !aligned16(k) || !aligned16(v))) return KVC_EINVAL;
    if (scratch_bytes < need) return KVC_ENOSPC;
    const PackedArgs a = {q, k, v, ld_q, ld_k, ld_v, q_start, k_start, n_seq, n_q, n_k, n_head_q, n_head_kv,
                          head_dim, dtype, out, lse};
    return launch_packed(a, scratch, (cudaStream_t)stream);
}

int kv_pages_advance(const kvc_pages *pages, const kvc_free_pages *free_pages, const int32_t *rows, int32_t *row_start,
                     int32_t n_rows, int32_t *positions, int32_t *slots, kvc_stream_t stream) {
    if (!pages || !free_pages || n_rows < 0) return KVC_EINVAL;
    if (pages->n_seq < 0 || pages->n_seq > 65535 || pages->max_pages <= 0 || pages->page_size <= 0 ||
        pages->page_size % 16 != 0 || (int64_t)pages->max_pages * pages->page_size > INT32_MAX)
        return KVC_EINVAL;
    if (free_pages->n_pages <= 0 || (int64_t)free_pages->n_pages * pages->page_size > INT32_MAX) return KVC_EINVAL;
    if (pages->n_seq == 0) return KVC_OK;
    if (!pages->table || !pages->len || !free_pages->ring || !free_pages->state || !rows || !row_start) return KVC_EINVAL;
    const void *all[] = {pages->table, pages->len, free_pages->ring, free_pages->state, rows, row_start, positions, slots};
    for (const void *p : all)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return KVC_EINVAL;
    const AdvanceArgs a = {const_cast<int32_t *>(pages->table), const_cast<int32_t *>(pages->len), pages->n_seq,
                           pages->max_pages, pages->page_size, free_pages->ring, free_pages->state, free_pages->n_pages,
                           rows, row_start, n_rows, positions, slots};
    return launch_pages_advance(a, (cudaStream_t)stream);
}

static bool rope_ok(const kvc_rope *r, int32_t head_dim, float eps) {
    if (!r || r->n_pairs < 0 || r->n_pairs > head_dim / 2) return false;
    if (r->style != KVC_ROPE_HALF && r->style != KVC_ROPE_PAIRS) return false;
    if (r->style == KVC_ROPE_HALF && r->n_pairs % 8 != 0) return false;
    if (r->n_pairs > 0 && (!r->turns || (reinterpret_cast<uintptr_t>(r->turns) & 7u))) return false;
    return eps >= 0.f && eps <= 3.402823466e38f && head_dim > 0 && head_dim % 32 == 0 && head_dim <= 256;
}

// a weight's address has its type's alignment
static bool weight_ok(const void *w, int dtype) {
    return (reinterpret_cast<uintptr_t>(w) & (uintptr_t)(dtype_bytes(dtype) - 1)) == 0;
}

int qk_norm_rope(const kvc_rope *rope, const void *q, const void *k, int64_t ld_q, int64_t ld_k, int32_t dtype,
                 int32_t n_rows, int32_t n_head_q, int32_t n_head_kv, int32_t head_dim, const int32_t *pos,
                 const void *q_weight, const void *k_weight, float eps, void *q_out, void *k_out, int64_t ld_qo,
                 int64_t ld_ko, kvc_stream_t stream) {
    if (!dtype_ok(dtype) || !rope_ok(rope, head_dim, eps) || n_rows < 0) return KVC_EINVAL;
    if (n_head_q <= 0 || n_head_kv < 0 || (int64_t)n_head_q + n_head_kv > 65535) return KVC_EINVAL;
    if (!ld_ok(ld_q, n_head_q, head_dim, dtype) || !ld_ok(ld_qo, n_head_q, head_dim, dtype)) return KVC_EINVAL;
    if (n_head_kv > 0 && (!ld_ok(ld_k, n_head_kv, head_dim, dtype) || !ld_ok(ld_ko, n_head_kv, head_dim, dtype)))
        return KVC_EINVAL;
    if (!weight_ok(q_weight, dtype) || !weight_ok(k_weight, dtype)) return KVC_EINVAL;
    if (n_rows == 0) return KVC_OK;
    if (!q || !q_out || !pos || !aligned16(q) || !aligned16(q_out)) return KVC_EINVAL;
    if (n_head_kv > 0 && (!k || !k_out || !aligned16(k) || !aligned16(k_out))) return KVC_EINVAL;
    const RopeArgs a = {q, k, nullptr, ld_q, ld_k, 0, dtype, n_rows, n_head_q, n_head_kv, head_dim, pos, rope->turns,
                        rope->n_pairs, rope->style, q_weight, k_weight, eps, q_out, k_out, ld_qo, ld_ko};
    return launch_rope(a, (cudaStream_t)stream);
}

int qk_norm_rope_append(const kvc_cache *pool, const kvc_pages *pages, int32_t layer, const int32_t *row_start,
                        int32_t n_rows, const kvc_rope *rope, const void *q, const void *k, const void *v, int64_t ld_q,
                        int64_t ld_k, int64_t ld_v, int32_t dtype, int32_t n_head_q, const void *q_weight,
                        const void *k_weight, float eps, void *q_out, int64_t ld_qo, kvc_stream_t stream) {
    if (!pool_ok(pool) || !pages_ok(pool, pages) || !dtype_ok(dtype) || n_rows < 0) return KVC_EINVAL;
    const int H = pool->d.n_head_kv, D = pool->d.head_dim;
    if (!rope_ok(rope, D, eps)) return KVC_EINVAL;
    if (n_head_q <= 0 || (int64_t)n_head_q + 2 * (int64_t)H > 65535) return KVC_EINVAL;
    if (!ld_ok(ld_q, n_head_q, D, dtype) || !ld_ok(ld_qo, n_head_q, D, dtype) || !ld_ok(ld_k, H, D, dtype) ||
        !ld_ok(ld_v, H, D, dtype))
        return KVC_EINVAL;
    if (!weight_ok(q_weight, dtype) || !weight_ok(k_weight, dtype)) return KVC_EINVAL;
    if (layer < 0 || layer >= pool->d.n_layer) return KVC_ERANGE;
    if (n_rows == 0 || pages->n_seq == 0) return KVC_OK;
    if (!pages->table || !pages->len || !row_start || !q || !k || !v || !q_out) return KVC_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out)) return KVC_EINVAL;
    const RopeArgs a = {q, k, v, ld_q, ld_k, ld_v, dtype, n_rows, n_head_q, H, D, nullptr, rope->turns,
                        rope->n_pairs, rope->style, q_weight, k_weight, eps, q_out, nullptr, ld_qo, 0};
    return launch_rope_append(a, *pool, *pages, layer, row_start, (cudaStream_t)stream);
}

int kv_cache_truncate(const kvc_cache *cache, int32_t n_tokens, kvc_stream_t stream) {
    if (!pool_ok(cache)) return KVC_EINVAL;
    const kvc_desc &d = cache->d;
    if (n_tokens < 0 || n_tokens > d.n_ctx) return KVC_ERANGE;
    if (n_tokens == d.n_ctx) return KVC_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const size_t T = d.n_ctx, n = n_tokens, H = d.n_head_kv, L = d.n_layer;
    // one strided fill per buffer: rows of positions [0, n_ctx), their tail [n_tokens, n_ctx) cleared
    auto clear = [&](void *buf, size_t row_bytes) -> bool {  // row_bytes: one position of one row
        const bool hm = d.layout == KVC_HEAD_MAJOR;
        const size_t per_pos = hm ? row_bytes : row_bytes * H;   // bytes of one position in a row
        const size_t rows = hm ? H * L : L;
        return cudaMemset2DAsync(static_cast<uint8_t *>(buf) + n * per_pos, T * per_pos, 0, (T - n) * per_pos, rows,
                                 s) == cudaSuccess;
    };
    const size_t row_bytes = (size_t)code_bytes(d.type, d.head_dim);
    if (!clear(cache->k_q, row_bytes) || !clear(cache->v_q, row_bytes)) return KVC_ECUDA;
    if (has_scales(d.type)) {
        const size_t scale_bytes = (size_t)(d.head_dim / 32) * 2;
        if (!clear(cache->k_s, scale_bytes) || !clear(cache->v_s, scale_bytes)) return KVC_ECUDA;
    }
    return KVC_OK;
}

const char *kvc_strerror(int status) {
    switch (status) {
        case KVC_OK: return "ok";
        case KVC_EINVAL: return "invalid argument";
        case KVC_ERANGE: return "layer or position outside the cache";
        case KVC_ENOSPC: return "destination or scratch buffer too small";
        case KVC_EFORMAT: return "state stream does not match its header or the cache";
        case KVC_ECUDA: return "CUDA call or launch failed";
        case KVC_EDEVICE: return "a kernel gave up a bounded wait";
        default: return "unknown status";
    }
}

int kvc_device_status(int32_t *status) {
    if (!status) return KVC_EINVAL;
    const int rc = read_and_clear_device_status(status);
    if (rc != KVC_OK) return rc;
    return *status != 0 ? KVC_EDEVICE : KVC_OK;
}

int kvc_test_arm_wait_timeout(int32_t which, uint64_t limit_ns) {
    if (which < KVC_TEST_PREFILL || which > KVC_TEST_PACKED) return KVC_EINVAL;
    arm_test_stall(which, limit_ns);
    return KVC_OK;
}

}  // extern "C"
