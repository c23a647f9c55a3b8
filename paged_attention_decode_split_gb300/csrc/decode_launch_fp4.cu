// decode_launch_fp4.cu -- launches the split-KV decode over the fp4 cache.
#include "decode_fp4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

template <int D, int NT, int NW, int SPW, bool RES, bool PACK, bool FAR>
cudaError_t launch_res(int group, const DecodeParams &p, dim3 grid, cudaStream_t stream, int slot) {
    using C = Fp4DecodeCfg<D, NT, NW, SPW>;
    auto kern = pa_decode_fp4_kernel<D, NT, NW, SPW, RES, PACK, FAR>;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), C::SMEM_BYTES, slot);
    if (e != cudaSuccess) return e;
    // programmatic dependent launch, as for the other decode kernels
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int cpp = p.block_size / kChunk;
    const Fp4Params fp{group, cpp, cpp == 1 ? 0xffffffffu : (uint32_t)((1ull << 32) / (unsigned)cpp)};
    return cudaLaunchKernelEx(&cfg, kern, p, fp);
}

// bf16 outputs go without the P residual; fp32 outputs of splits so long that a
// warp's accumulators need the second sum have a kernel of their own; up to 4
// heads carry the residual in the unused columns of the product.  Four kernel
// slots per layout.
template <int D, int NT, int NW, int SPW>
cudaError_t launch_t(int group, const DecodeParams &p, dim3 grid, cudaStream_t stream, int slot) {
    if (p.out_bf16) return launch_res<D, NT, NW, SPW, false, false, false>(group, p, grid, stream, slot);
    if (p.chunks_per_split > 2 * NW * (kFp4FarMin - 1))
        return launch_res<D, NT, NW, SPW, true, false, true>(group, p, grid, stream, slot + 1);
    if constexpr (NT == 1) {
        if (group <= 4) return launch_res<D, NT, NW, SPW, true, true, false>(group, p, grid, stream, slot + 3);
    }
    return launch_res<D, NT, NW, SPW, true, false, false>(group, p, grid, stream, slot + 2);
}

}  // namespace

// One kernel per head_dim and 8-head n-tile count; the group and the window
// are run-time values (they change a handful of instructions per chunk).
// Warps x stages, D = 256: decode_fp4.cuh.  D = 128, up to 8 heads (32 heads on
// 8, 16-token pages; 32 x 1K-32K with bf16 / fp32 output, one 32K sequence):
// 12 x 3 195 / 231 / 15.7 us, 12 x 2 195 / 231 / 15.9, 8 x 4 249 / 275 / 16.2,
// 10 x 4 224 / 264 / 16.9, 16 x 2 187 / 225 / 16.7: the single sequence decides
// against 16.  Up to 16 heads (32 on 2; the sequence: 64 on 4): 8 x 4 69.6 /
// 86.1 / 15.0, 8 x 3 70.1 / 85.2 / 15.1, 10 x 3 77.0 / 92.8 / 16.3, 12 x 3
// 70.4 / 78.1 / 16.0.
cudaError_t launch_decode_fp4(int head_dim, int group, const DecodeParams &p, dim3 grid, cudaStream_t stream) {
    if (head_dim == 256)
        return group <= 8 ? launch_t<256, 1, 8, 2>(group, p, grid, stream, 146)
                          : launch_t<256, 2, 8, 2>(group, p, grid, stream, 150);
    if (head_dim == 128)
        return group <= 8 ? launch_t<128, 1, 12, 3>(group, p, grid, stream, 153)
                          : launch_t<128, 2, 8, 4>(group, p, grid, stream, 157);
    return cudaErrorInvalidValue;
}

}  // namespace pa
