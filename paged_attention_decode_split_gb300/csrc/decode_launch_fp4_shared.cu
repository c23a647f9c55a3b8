// decode_launch_fp4_shared.cu -- the fp4 decode instantiations for the own parts of
// sequences with a shared prefix, in a translation unit of their own so they
// compile in parallel with the rest.
#include "decode_launch_fp4.cuh"

namespace pa {

cudaError_t launch_decode_fp4_shared(int head_dim, int group, const DecodeParams &p, dim3 grid, cudaStream_t stream) {
    return launch_decode_fp4_cfg<true>(head_dim, group, p, grid, stream, 200);
}

}  // namespace pa
