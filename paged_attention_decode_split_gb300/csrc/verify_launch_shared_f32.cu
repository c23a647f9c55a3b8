// verify_launch_shared_f32.cu -- the common part of a decode over shared prefixes
// with fp32 outputs: 64-key tiles, a second sum of O, over a bf16 cache three
// numbers per weight and two sums for a score (16 groups of 8 sequences x 4 heads
// behind 1K-8K: 168 us, error 0.8e-6; with one sum 1.1e-6 and 162 us, with two numbers
// 9 us less and 2e-6).
#include "verify_launch.cuh"

namespace pa {

cudaError_t launch_prefix_f32(int head_dim, int rows, const CUtensorMap &tk, const CUtensorMap &tv,
                              const CUtensorMap &tk64, const CUtensorMap &tv64, const VerifyParams &p, dim3 grid,
                              cudaStream_t stream) {
    if (head_dim == 256)
        return launch_verify_tc<256, 2, 3, 0, 2, 64, true, true, 3>(tk, tv, tk64, tv64, p, grid, stream, 236);
    if (head_dim == 128) {
        const int copies = prefix_copies(head_dim, rows);
        return copies == 4   ? launch_verify_tc<128, 2, 2, 0, 1, 64, true, true, 3, 4>(tk, tv, tk64, tv64, p, grid, stream, 284)
               : copies == 2 ? launch_verify_tc<128, 2, 2, 0, 1, 64, true, true, 3, 2>(tk, tv, tk64, tv64, p, grid, stream, 285)
                             : launch_verify_tc<128, 2, 2, 0, 1, 64, true, true, 3>(tk, tv, tk64, tv64, p, grid, stream, 237);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_prefix_fp8_f32(int head_dim, const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tk64,
                                  const CUtensorMap &tv64, const VerifyParams &p, dim3 grid, cudaStream_t stream) {
    if (head_dim == 256)
        return launch_verify_tc<256, 2, 3, 2, 2, 64, true, true, 2>(tk, tv, tk64, tv64, p, grid, stream, 238);
    if (head_dim == 128)
        return launch_verify_tc<128, 4, 4, 4, 2, 64, true, true, 2>(tk, tv, tk64, tv64, p, grid, stream, 239);
    return cudaErrorInvalidValue;
}

}  // namespace pa
