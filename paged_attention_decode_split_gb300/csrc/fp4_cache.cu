// fp4_cache.cu -- writing K/V rows into the fp4 cache (reshape_and_cache_fp4)
// and reading them back (gather_cache_fp4).
#include "fp4_cache.cuh"

namespace pa {

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// One CTA per token; a thread quantises one 16-dim block of K or of V.
template <int D>
__global__ void __launch_bounds__(128) pa_reshape_and_cache_fp4_kernel(
    const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, uint8_t *__restrict__ k_cache,
    uint8_t *__restrict__ v_cache, const int64_t *__restrict__ slots, const float *__restrict__ k_scale,
    const float *__restrict__ v_scale, int hkv, int block_size, int64_t num_slots, int32_t *status) {
    pdl_launch_dependents();
    pdl_wait_primary();
    constexpr int NB = D / 16;
    const int64_t s = slots[blockIdx.x];
    if (s < 0) return;  // padding token
    if (s >= num_slots) {
        if (threadIdx.x == 0) set_status(status, PA_DEV_BAD_SLOT);
        return;
    }
    const int64_t page = s / block_size;
    const int pos = (int)(s - page * block_size);
    const uint4 *ks = k_new + (size_t)blockIdx.x * hkv * (D / 8), *vs = v_new + (size_t)blockIdx.x * hkv * (D / 8);
    for (int j = threadIdx.x; j < hkv * NB; j += blockDim.x) {
        const int h = j / NB, blk = j % NB;
        const size_t rec = (((size_t)page * hkv + h) * (block_size / 16) + pos / 16) * fp4::rec_bytes(D);
        fp4::store_block<D, false>(k_cache + rec, pos % 16, blk, ks + 2 * j, k_scale[h]);
        fp4::store_block<D, true>(v_cache + rec, pos % 16, blk, vs + 2 * j, v_scale[h]);
    }
}

// code * S (exact) times g, rounded to binary32 and, for bf16 rows, once more.
template <bool BF>
__device__ __forceinline__ void store_row_block(void *out, size_t elem, const uint32_t (&o)[8], float S, float g) {
    float v[16];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&o[m]));
        v[2 * m] = f.x * S * g;
        v[2 * m + 1] = f.y * S * g;
    }
    if constexpr (BF) {
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + elem);
        p[0] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        p[1] = make_uint4(pack_bf16(v[8], v[9]), pack_bf16(v[10], v[11]), pack_bf16(v[12], v[13]),
                          pack_bf16(v[14], v[15]));
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(out) + elem);
#pragma unroll
        for (int m = 0; m < 4; ++m) p[m] = make_float4(v[4 * m], v[4 * m + 1], v[4 * m + 2], v[4 * m + 3]);
    }
}

template <int D, bool BF>
__global__ void __launch_bounds__(128) pa_gather_cache_fp4_kernel(
    const uint8_t *__restrict__ k_cache, const uint8_t *__restrict__ v_cache, const int64_t *__restrict__ slots,
    const float *__restrict__ k_scale, const float *__restrict__ v_scale, void *__restrict__ k_out,
    void *__restrict__ v_out, int hkv, int block_size, int64_t num_slots, int32_t *status) {
    pdl_launch_dependents();
    pdl_wait_primary();
    constexpr int NB = D / 16;
    const int64_t s = slots[blockIdx.x];
    const bool live = s >= 0 && s < num_slots;
    if (s >= num_slots && threadIdx.x == 0) set_status(status, PA_DEV_BAD_SLOT);
    const int64_t page = live ? s / block_size : 0;
    const int pos = live ? (int)(s - page * block_size) : 0;
    for (int j = threadIdx.x; j < hkv * NB; j += blockDim.x) {
        const int h = j / NB, blk = j % NB;
        const size_t rec = (((size_t)page * hkv + h) * (block_size / 16) + pos / 16) * fp4::rec_bytes(D);
        const size_t elem = ((size_t)blockIdx.x * hkv + h) * D + 16 * blk;
        uint32_t o[8] = {}, sc = 0;
        if (live) fp4::load_block<D, false>(k_cache + rec, pos % 16, blk, o, sc);
        store_row_block<BF>(k_out, elem, o, fp4::e4m3_f32(sc), k_scale[h]);
        if (live) fp4::load_block<D, true>(v_cache + rec, pos % 16, blk, o, sc);
        store_row_block<BF>(v_out, elem, o, fp4::e4m3_f32(sc), v_scale[h]);
    }
}

// The checks both calls share; PA_OK with *nothing set when there is no row.
pa_status check_rows(const void *k_rows, const void *v_rows, const void *k_cache, const void *v_cache,
                     const int64_t *slots, const float *k_scale, const float *v_scale, int32_t num_tokens,
                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_pages, bool *nothing) {
    *nothing = false;
    if (num_tokens < 0 || num_kv_heads < 1 || head_dim < 1 || block_size < 1 || num_pages < 1)
        return PA_ERR_INVALID_ARG;
    if (head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
    if (block_size % 16 != 0 || num_pages > INT32_MAX || num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    *nothing = num_tokens == 0;
    if (*nothing) return PA_OK;
    if (!k_rows || !v_rows || !k_cache || !v_cache || !slots || !k_scale || !v_scale) return PA_ERR_INVALID_ARG;
    if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slots, 8) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

template <typename... KArgs, typename... Args>
pa_status launch_rows(void (*kern)(KArgs...), int num_tokens, void *stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_tokens));
    cfg.blockDim = dim3(128);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_reshape_and_cache_fp4(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                                   const int64_t *slot_mapping, const float *k_scale, const float *v_scale,
                                   int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                   int64_t num_pages, int32_t *device_status, void *stream) {
    bool nothing;
    const pa_status st = check_rows(k_new, v_new, k_cache, v_cache, slot_mapping, k_scale, v_scale, num_tokens,
                                    num_kv_heads, head_dim, block_size, num_pages, &nothing);
    if (st != PA_OK || nothing) return st;
    auto *kern = head_dim == 256 ? pa_reshape_and_cache_fp4_kernel<256> : pa_reshape_and_cache_fp4_kernel<128>;
    return launch_rows(kern, num_tokens, stream, static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new),
                       static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), slot_mapping, k_scale,
                       v_scale, num_kv_heads, block_size, num_pages * block_size, device_status);
}

pa_status pa_gather_cache_fp4(const void *k_cache, const void *v_cache, const int64_t *slot_mapping,
                              const float *k_scale, const float *v_scale, void *k_out, void *v_out, int32_t out_dtype,
                              int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                              int64_t num_pages, int32_t *device_status, void *stream) {
    if (out_dtype != PA_OUT_F32 && out_dtype != PA_OUT_BF16) return PA_ERR_INVALID_ARG;
    bool nothing;
    const pa_status st = check_rows(k_out, v_out, k_cache, v_cache, slot_mapping, k_scale, v_scale, num_tokens,
                                    num_kv_heads, head_dim, block_size, num_pages, &nothing);
    if (st != PA_OK || nothing) return st;
    const bool bf = out_dtype == PA_OUT_BF16;
    auto *kern = head_dim == 256 ? (bf ? pa_gather_cache_fp4_kernel<256, true> : pa_gather_cache_fp4_kernel<256, false>)
                                 : (bf ? pa_gather_cache_fp4_kernel<128, true> : pa_gather_cache_fp4_kernel<128, false>);
    return launch_rows(kern, num_tokens, stream, static_cast<const uint8_t *>(k_cache),
                       static_cast<const uint8_t *>(v_cache), slot_mapping, k_scale, v_scale, k_out, v_out,
                       num_kv_heads, block_size, num_pages * block_size, device_status);
}

}  // extern "C"
