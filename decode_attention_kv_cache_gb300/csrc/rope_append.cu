// qk_norm_rope_append (rope.cuh).
#include "rope.cuh"

namespace kvc {

int launch_rope_append(const RopeArgs &a, const kvc_cache &c, const kvc_pages &pages, int layer, const int32_t *row_start,
                       cudaStream_t s) {
    const Geom g = geom_of(c.d);
    Args p = {};
    p.a = a;
    p.pg = paged_view(c, pages);
    p.row_start = row_start;
    p.kq = static_cast<uint8_t *>(c.k_q) + code_bytes(c.d.type, layer * g.c_layer);
    p.vq = static_cast<uint8_t *>(c.v_q) + code_bytes(c.d.type, layer * g.c_layer);
    if (has_scales(c.d.type)) {
        p.ks = static_cast<uint16_t *>(c.k_s) + layer * g.s_layer;
        p.vs = static_cast<uint16_t *>(c.v_s) + layer * g.s_layer;
    }
    p.c_tok = g.c_tok;
    p.c_head = g.c_head;
    p.s_tok = g.s_tok;
    p.s_head = g.s_head;
    switch (c.d.type) {
        case KVC_F16: return launch_all<KVC_F16>(p, s);
        case KVC_Q8_0: return launch_all<KVC_Q8_0>(p, s);
        default: return launch_all<KVC_Q4_0>(p, s);
    }
}

}  // namespace kvc
