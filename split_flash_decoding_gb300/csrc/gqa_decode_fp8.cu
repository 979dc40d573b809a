// gqa_decode_fp8.cu -- decode attention over a cache held in 8 bits (attn_decode_fp8).
#include "gqa_decode_codes.cuh"

namespace attn {

int fp8_decode_ctas(int num_sms) { return codes::kCtasPerSm * num_sms; }

cudaError_t launch_gqa_decode_fp8(const Fp8DecodeParams &p, int ctas, cudaStream_t stream) {
    return codes::launch<false>(p, ctas, stream);
}

}  // namespace attn
