// verify_launch_fp4_shared.cu -- the tensor-core kernel as the common part of a
// decode over shared prefixes, fp4 cache, in a translation unit of its own so it
// compiles in parallel with the rest.
#include "verify_launch_fp4.cuh"

namespace pa {

cudaError_t launch_prefix_fp4(int head_dim, const VerifyParams &p, dim3 grid, cudaStream_t stream) {
    return launch_verify_fp4_cfg<true>(head_dim, p, grid, stream, 230);
}

}  // namespace pa
