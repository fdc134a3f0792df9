// CUDA-core paged decode kernels with score rules (pa_decode_scored) for head_dim = 128.
#include "pa_decode_cc.cuh"

namespace pa {

cudaError_t launch_decode_cc_d128_scored(int G, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const DecodeParams &p, int B, cudaStream_t stream) {
    switch (G) {
        case 1: return launch_cc_instance<128, 1, true>(kmap, vmap, p, B, stream);
        case 2: return launch_cc_instance<128, 2, true>(kmap, vmap, p, B, stream);
        case 3: return launch_cc_instance<128, 3, true>(kmap, vmap, p, B, stream);
        case 4: return launch_cc_instance<128, 4, true>(kmap, vmap, p, B, stream);
        case 5: return launch_cc_instance<128, 5, true>(kmap, vmap, p, B, stream);
        case 6: return launch_cc_instance<128, 6, true>(kmap, vmap, p, B, stream);
        case 7: return launch_cc_instance<128, 7, true>(kmap, vmap, p, B, stream);
        case 8: return launch_cc_instance<128, 8, true>(kmap, vmap, p, B, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
