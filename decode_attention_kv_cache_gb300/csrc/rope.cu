// qk_norm_rope (rope.cuh).
#include "rope.cuh"

namespace kvc {

int launch_rope(const RopeArgs &a, cudaStream_t s) {
    Args p = {};
    p.a = a;
    return launch_all<NO_POOL>(p, s);
}

}  // namespace kvc
