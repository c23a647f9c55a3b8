// decode_launch_fp4.cu -- launches the split-KV decode over the fp4 cache.
#include "decode_launch_fp4.cuh"

namespace pa {

cudaError_t launch_decode_fp4(int head_dim, int group, const DecodeParams &p, dim3 grid, cudaStream_t stream) {
    return launch_decode_fp4_cfg<false>(head_dim, group, p, grid, stream, 146);
}

}  // namespace pa
