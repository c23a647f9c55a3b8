// decode_launch_fp8_shared.cu -- the e4m3 decode instantiations for the own
// parts of sequences with a shared prefix, in translation units of their own
// (bf16 outputs here, fp32 outputs beside) so they compile in parallel with the rest.
#include "decode_launch.cuh"

namespace pa {

cudaError_t launch_decode_fp8_shared(int head_dim, int group, const CUtensorMap &tk, const CUtensorMap &tv,
                                 const DecodeParams &p, dim3 grid, cudaStream_t stream) {
    if (!p.out_bf16) return launch_decode_fp8_shared_f32(head_dim, group, tk, tv, p, grid, stream);
    if (p.prefix_splits == 0) return launch_decode_fp8_shared_alone(head_dim, group, tk, tv, p, grid, stream);
    return launch_decode_cfg<false, true, true, 1, false>(head_dim, group, tk, tv, p, grid, stream);
}

}  // namespace pa
