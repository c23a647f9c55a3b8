// verify_launch.cuh -- launches one instantiation of the tensor-core verify
// kernel over a bf16 or e4m3 cache; shared by the translation units of the
// verify and of the common part of a decode over shared prefixes.
#pragma once

#include "pa_internal.h"

namespace pa {

template <int D, int NK, int NV, int NSG, int NSB, int TK = 64, bool SH = false, bool FAR = false, int PT = 2,
          int COP = 1>
cudaError_t launch_verify_tc(const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tk64,
                             const CUtensorMap &tv64, const VerifyParams &p, dim3 grid, cudaStream_t stream,
                             int slot) {
    using C = VerifyTcCfg<D, NK, NV, NSG, NSB, TK, false, PT>;
    auto kern = pa_verify_tc_kernel<D, NK, NV, NSG, NSB, TK, false, (PT > 1), FAR, SH, PT, COP>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), C::SMEM_BYTES, slot);
    if (e != cudaSuccess) return e;
    if constexpr (C::RSPLIT) {
        // the warpgroups' register shares draw on the launch's registers: with fewer, setmaxnreg would wait forever
        e = ensure_launch_regs(reinterpret_cast<const void *>(kern), C::REGS_LAUNCH, slot);
        if (e != cudaSuccess) return e;
    }
    // programmatic dependent launch: the set-up overlaps the work before it
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
    return cudaLaunchKernelEx(&cfg, kern, tk, tv, tk64, tv64, p);
}

}  // namespace pa
