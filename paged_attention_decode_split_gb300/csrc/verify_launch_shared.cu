// verify_launch_shared.cu -- the tensor-core kernel as the common part of a
// decode over shared prefixes, bf16 and e4m3 caches, bf16 outputs, in a
// translation unit of its own so it compiles in parallel with the rest.
#include "verify_launch.cuh"

namespace pa {

// Row copies pay where a CTA's products wait for its softmax: one S/P buffer (16
// groups of 8 sequences x 4 heads behind 1K-8K: 143 -> 136 us, fp32 outputs 185 ->
// 170; at head_dim 256 the products bound a tile, not the softmax).
int prefix_copies(int head_dim, int rows) {
    return head_dim != 128 ? 1 : rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
}

// rows: what the largest group may have, sequences x heads of the group.  The
// layouts are the verify's (verify_launch.cu) with 64-key score tiles at head_dim
// 256, also for several blocks of rows (64 sequences behind 32K: 79 us for the call, 83
// with 128-key tiles, whose one K slot waits for its copy), and but for one block of
// rows at head_dim 128: one S/P buffer, 256 tensor-memory columns and half the rings, so
// that two CTAs share an SM and one's set-up and epilogue pass behind the other's
// tiles (the groups above: 17 us less for the whole call).
cudaError_t launch_prefix(int head_dim, int rows, const CUtensorMap &tk, const CUtensorMap &tv,
                          const CUtensorMap &tk64, const CUtensorMap &tv64, const CUtensorMap &tk128,
                          const VerifyParams &p, dim3 grid, cudaStream_t stream) {
    if (!p.out_bf16) return launch_prefix_f32(head_dim, rows, tk, tv, tk64, tv64, p, grid, stream);
    if (head_dim == 256) return launch_verify_tc<256, 4, 3, 0, 2, 64, true>(tk, tv, tk64, tv64, p, grid, stream, 225);
    if (head_dim == 128) {
        const bool wide = verify_wide_score_tiles(head_dim, rows);
        const int copies = prefix_copies(head_dim, rows);
        return wide          ? launch_verify_tc<128, 3, 6, 0, 2, 128, true>(tk, tv, tk128, tv64, p, grid, stream, 226)
               : copies == 4 ? launch_verify_tc<128, 3, 3, 0, 1, 64, true, false, 2, 4>(tk, tv, tk64, tv64, p, grid, stream, 280)
               : copies == 2 ? launch_verify_tc<128, 3, 3, 0, 1, 64, true, false, 2, 2>(tk, tv, tk64, tv64, p, grid, stream, 283)
                             : launch_verify_tc<128, 3, 3, 0, 1, 64, true>(tk, tv, tk64, tv64, p, grid, stream, 227);
    }
    return cudaErrorInvalidValue;
}

// bf16 outputs: a weight enters the product as one f16, and four warps widen each
// tensor at head_dim 256 (33 sequences of 48 heads behind 16.6K: 8 us less for the
// whole call than with two; with eight it takes 5 more).
cudaError_t launch_prefix_fp8(int head_dim, const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tk64,
                              const CUtensorMap &tv64, const VerifyParams &p, dim3 grid, cudaStream_t stream) {
    if (!p.out_bf16) return launch_prefix_fp8_f32(head_dim, tk, tv, tk64, tv64, p, grid, stream);
    if (head_dim == 256)
        return launch_verify_tc<256, 2, 3, 2, 2, 64, true, false, 1>(tk, tv, tk64, tv64, p, grid, stream, 228);
    if (head_dim == 128)
        return launch_verify_tc<128, 4, 4, 4, 2, 64, true, false, 1>(tk, tv, tk64, tv64, p, grid, stream, 229);
    return cudaErrorInvalidValue;
}

}  // namespace pa
