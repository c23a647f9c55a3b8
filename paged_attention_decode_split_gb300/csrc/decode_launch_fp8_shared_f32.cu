// decode_launch_fp8_shared_f32.cu -- the e4m3 decode instantiations for the own
// parts of sequences with a shared prefix, fp32 outputs.
#include "decode_launch.cuh"

namespace pa {

cudaError_t launch_decode_fp8_shared_f32(int head_dim, int group, const CUtensorMap &tk, const CUtensorMap &tv,
                                 const DecodeParams &p, dim3 grid, cudaStream_t stream) {
    return launch_decode_cfg<false, true, true, 2, true>(head_dim, group, tk, tv, p, grid, stream);
}

}  // namespace pa
