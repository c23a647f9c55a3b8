// verify_launch_fp4.cu -- the tensor-core verify over the fp4 cache, in a
// translation unit of its own so it compiles in parallel with the rest.
#include "verify_launch_fp4.cuh"

namespace pa {

cudaError_t launch_verify_fp4(int head_dim, const VerifyParams &p, dim3 grid, cudaStream_t stream) {
    return launch_verify_fp4_cfg<false>(head_dim, p, grid, stream, 140);
}

}  // namespace pa
