// decode_attn_paged: the kernels of q4_0 pools (decode_paged.cuh), compiled beside the others.
#include "decode_paged.cuh"

namespace kvc {

int launch_decode_paged_q4(const kvc_cache &c, int layer, int page_size, int dtype, const PagedView &pg,
                           const DecodePagedArgs &a, cudaStream_t s) {
    return launch_type<KVC_Q4_0>(c, layer, page_size, dtype, pg, a, s);
}

int read_and_clear_paged_q4_status(int32_t *status) { return read_and_clear(status); }

}  // namespace kvc
