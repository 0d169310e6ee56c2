// decode_attn_paged: the launch, and the kernels of f16 and q8_0 pools (decode_paged.cuh).
#include "decode_paged.cuh"

namespace kvc {
namespace {

int slots_of(int ct, int G) { return ctas_per_sm(ct, G <= 8 ? 1 : 2) * sm_count(); }

}  // namespace

size_t paged_scratch_bytes(const kvc_desc &d, int, int n_head_q) {
    const size_t G = n_head_q / d.n_head_kv;
    return (size_t)slots_of(d.type, (int)G) * (2 * G * (d.head_dim + 2) * sizeof(float) + sizeof(int4));
}

int launch_decode_paged(const kvc_cache &c, const kvc_pages &p, int layer, const void *q, int64_t ld_q, int dtype,
                        int n_head_q, void *out, float *lse, void *scratch, cudaStream_t s) {
    const kvc_desc &d = c.d;
    const Geom g = geom_of(d);
    const bool scales = has_scales(d.type);
    Args a;
    a.ks = scales ? static_cast<const uint16_t *>(c.k_s) + layer * g.s_layer : nullptr;
    a.vs = scales ? static_cast<const uint16_t *>(c.v_s) + layer * g.s_layer : nullptr;
    a.s_tok = g.s_tok;
    a.s_head = g.s_head;
    a.q = static_cast<const uint8_t *>(q);
    a.ld_q = ld_q * dtype_bytes(dtype);
    a.out = out;
    a.lse = lse;
    a.H_q = n_head_q;
    a.H_kv = d.n_head_kv;
    a.G = n_head_q / d.n_head_kv;
    a.n_slots = slots_of(d.type, a.G);
    a.desc = static_cast<int4 *>(scratch);
    a.part_o = reinterpret_cast<float *>(a.desc + a.n_slots);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)a.n_slots * 2 * a.G * d.head_dim);
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)d.head_dim);
    a.stall_ns = take_test_stall(KVC_TEST_PAGED);
    const PagedView pg = paged_view(c, p);
    switch (d.type) {
        case KVC_F16: return launch_type<KVC_F16>(c, layer, p.page_size, dtype, pg, a, s);
        case KVC_Q8_0: return launch_type<KVC_Q8_0>(c, layer, p.page_size, dtype, pg, a, s);
        default: return launch_decode_paged_q4(c, layer, p.page_size, dtype, pg, a, s);
    }
}

int read_and_clear_paged_status(int32_t *status) {
    int q4 = 0;
    if (read_and_clear(status) != KVC_OK || read_and_clear_paged_q4_status(&q4) != KVC_OK) return KVC_ECUDA;
    *status |= q4;
    return KVC_OK;
}

}  // namespace kvc
