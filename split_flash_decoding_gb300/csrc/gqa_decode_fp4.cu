// gqa_decode_fp4.cu -- decode attention over a cache held in 4 bits (attn_decode_fp4).
#include "gqa_decode_codes.cuh"

namespace attn {

cudaError_t launch_gqa_decode_fp4(const Fp8DecodeParams &p, int ctas, cudaStream_t stream) {
    return codes::launch<true>(p, ctas, stream);
}

}  // namespace attn
