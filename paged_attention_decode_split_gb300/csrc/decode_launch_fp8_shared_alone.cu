// decode_launch_fp8_shared_alone.cu -- the e4m3 decode instantiations for batches
// with shared prefixes that are read without sharing, bf16 outputs: a softmax weight
// enters the product as two f16 numbers, as in the decode that such a call stands for.
// (Against one f16 that is 0 to 3 % slower at head_dim 128, up to 11 % with 16 heads
// per KV head, and at head_dim 256 4 to 14 % with 6 heads, 2 to 22 % with 12.  32
// sequences of up to 3000 tokens, one / two numbers / the decode itself: 30.8 / 31.3 /
// 35.4 us at 128, 38.3 / 41.4 / 34.1 and 37.2 / 45.5 / 50.9 us at 256.)
#include "decode_launch.cuh"

namespace pa {

cudaError_t launch_decode_fp8_shared_alone(int head_dim, int group, const CUtensorMap &tk, const CUtensorMap &tv,
                                           const DecodeParams &p, dim3 grid, cudaStream_t stream) {
    return launch_decode_cfg<false, true, true, 2, false>(head_dim, group, tk, tv, p, grid, stream);
}

}  // namespace pa
