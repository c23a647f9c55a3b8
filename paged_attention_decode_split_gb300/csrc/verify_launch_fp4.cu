// verify_launch_fp4.cu -- the tensor-core verify over the fp4 cache, in a
// translation unit of its own so it compiles in parallel with the rest.
#include "pa_internal.h"

namespace pa {

namespace {

template <int D, int NK, int NV, int NSG, bool RES, bool FAR>
cudaError_t launch_res(const VerifyParams &p, dim3 grid, cudaStream_t stream, int slot) {
    using C = VerifyTcCfg<D, NK, NV, NSG, 2, 64, true>;
    auto kern = pa_verify_tc_kernel<D, NK, NV, NSG, 2, 64, true, RES, FAR>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), C::SMEM_BYTES, slot);
    if (e != cudaSuccess) return e;
    // the warpgroups' register shares draw on the launch's registers: with fewer, setmaxnreg would wait forever
    e = ensure_launch_regs(reinterpret_cast<const void *>(kern), C::REGS_LAUNCH, slot);
    if (e != cudaSuccess) return e;
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
    const CUtensorMap none = {};  // the records are copied without tensor maps
    return cudaLaunchKernelEx(&cfg, kern, none, none, none, none, p);
}

// bf16 outputs go without the P residual; fp32 outputs of long splits need the
// second sum of O (three kernel slots per layout)
template <int D, int NK, int NV, int NSG>
cudaError_t launch_t(const VerifyParams &p, dim3 grid, cudaStream_t stream, int slot) {
    if (p.out_bf16) return launch_res<D, NK, NV, NSG, false, false>(p, grid, stream, slot);
    if (p.chunks_per_split > kVerifyFarTiles * 4)
        return launch_res<D, NK, NV, NSG, true, true>(p, grid, stream, slot + 1);
    return launch_res<D, NK, NV, NSG, true, false>(p, grid, stream, slot + 2);
}

}  // namespace

// The f16 rings of the fp8 form, and as many staging slots (9 KiB per tensor
// and tile at D = 256, 4.5 KiB at D = 128) as fit beside them.
cudaError_t launch_verify_fp4(int head_dim, const VerifyParams &p, dim3 grid, cudaStream_t stream) {
    if (head_dim == 256) return launch_t<256, 2, 3, 3>(p, grid, stream, 140);
    if (head_dim == 128) return launch_t<128, 5, 5, 6>(p, grid, stream, 143);
    return cudaErrorInvalidValue;
}

}  // namespace pa
