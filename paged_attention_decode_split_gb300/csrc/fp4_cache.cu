// fp4_cache.cu -- writing K/V rows into the fp4 cache (reshape_and_cache_fp4)
// and reading them back (gather_cache_fp4).
#include "fp4_cache.cuh"

namespace pa {

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Both kernels move rows between bf16 (or fp32) and records: a lane holds one
// 16-dim block of a row of K and of V, NB lanes a row, so every value is loaded
// and quantised once with 16-byte accesses; a row's code bytes go through
// shared memory into (or out of) the order of the record, whose 16-byte pieces
// then move with one access each.  16411 tokens of 8 heads x 128 are written in
// 18.5 us (86 MB, 4.6 TB/s) and read back in 17.8 us (4.8 TB/s); one token of 4 x
// 256 takes 1.7 us each way, a launch.  Beside the bytes, the instruction issue
// bounds the write (77 % of the slots, the ALU 70 %: the quantiser and the
// packing of bytes), the load/store path the read (the largest stalls; issue 62
// %): the pieces of a row are 8 and 16 bytes, 32 and 64 bytes apart, the scales
// single bytes.  With a byte per access the two took 23.3 and 21.0 us.
template <int D>
struct RowCfg {
    static constexpr int NB = D / 16;        // lanes per row
    static constexpr int RW = 32 / NB;       // rows per warp
    static constexpr int WARPS = 4;
    static constexpr int ROW_BYTES = D / 2;  // code bytes of a row
};

// Byte offset in a record of piece j of token t's codes: K's 16-byte pieces (j
// = 4 (blk / 8) + c), V's NB-byte pieces (j = r).
__device__ __forceinline__ int k_piece_off(int t, int j) {
    return ((j >> 2) * 2 + (t >> 3)) * 512 + (t & 7) * 64 + (j & 3) * 16;
}
template <int D>
__device__ __forceinline__ int v_piece_off(int t, int j) {
    return fp4::v_code_off<D>(t, 0) + j * (D / 4);
}

struct RowAt {
    bool live;
    int t;       // token of the record
    size_t rec;  // byte offset of the record
};

__device__ __forceinline__ RowAt row_at(int64_t slot, int h, int hkv, int block_size, int64_t num_slots, int rec_bytes) {
    RowAt a{slot >= 0 && slot < num_slots, 0, 0};
    if (a.live) {
        const uint32_t page = (uint32_t)(slot / block_size);
        const int pos = (int)(slot - (int64_t)page * block_size);
        a.t = pos & 15;
        a.rec = (((size_t)page * hkv + h) * (block_size / 16) + (pos >> 4)) * rec_bytes;
    }
    return a;
}

template <int D>
__global__ void __launch_bounds__(128) pa_reshape_and_cache_fp4_kernel(
    const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, uint8_t *__restrict__ k_cache,
    uint8_t *__restrict__ v_cache, const int64_t *__restrict__ slots, const float *__restrict__ k_scale,
    const float *__restrict__ v_scale, int hkv, int64_t rows, int block_size, int64_t num_slots, int32_t *status) {
    using C = RowCfg<D>;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ __align__(16) uint8_t sk[C::WARPS][C::RW][C::ROW_BYTES], sv[C::WARPS][C::RW][C::ROW_BYTES];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rr = lane / C::NB, blk = lane % C::NB;
    const int64_t row = ((int64_t)blockIdx.x * C::WARPS + warp) * C::RW + rr;
    const bool in = row < rows;
    const int64_t row_c = in ? row : 0;
    const int64_t token = row_c / hkv;
    const int h = (int)(row_c - token * hkv);
    const uint4 *ks = k_new + row_c * (D / 8) + 2 * blk, *vs = v_new + row_c * (D / 8) + 2 * blk;
    const int64_t slot = slots[token];
    const uint4 k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
    const float kg = k_scale[h], vg = v_scale[h];
    const RowAt at = row_at(slot, h, hkv, block_size, num_slots, fp4::rec_bytes(D));
    if (in && slot >= num_slots && h == 0 && blk == 0) set_status(status, PA_DEV_BAD_SLOT);
    uint32_t ksc, vsc;
    const uint2 kq = fp4::quantise_block(k0, k1, kg, ksc), vq = fp4::quantise_block(v0, v1, vg, vsc);
    uint8_t *kp = sk[warp][rr] + (blk >> 3) * 64 + 2 * (blk & 7), *vp = sv[warp][rr] + blk;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint16_t *>(kp + 16 * c) = (uint16_t)((c < 2 ? kq.x : kq.y) >> (16 * (c & 1)));
#pragma unroll
    for (int m = 0; m < 8; ++m) vp[m * C::NB] = (uint8_t)fp4::byte_of(vq, m);
    __syncwarp();
    if (!in || !at.live) return;
    uint8_t *kr = k_cache + at.rec, *vr = v_cache + at.rec;
    if constexpr (D == 256) {  // lanes 0-7 of a row: K's pieces, lanes 8-15: V's
        const int j = blk & 7;
        if (blk < 8)
            *reinterpret_cast<uint4 *>(kr + k_piece_off(at.t, j)) = *reinterpret_cast<const uint4 *>(sk[warp][rr] + 16 * j);
        else
            *reinterpret_cast<uint4 *>(vr + v_piece_off<D>(at.t, j)) = *reinterpret_cast<const uint4 *>(sv[warp][rr] + 16 * j);
    } else {
        if (blk < 4)
            *reinterpret_cast<uint4 *>(kr + k_piece_off(at.t, blk)) =
                *reinterpret_cast<const uint4 *>(sk[warp][rr] + 16 * blk);
        *reinterpret_cast<uint2 *>(vr + v_piece_off<D>(at.t, blk)) = *reinterpret_cast<const uint2 *>(sv[warp][rr] + 8 * blk);
    }
    kr[fp4::k_scale_off<D>(at.t, blk)] = (uint8_t)ksc;
    vr[fp4::v_scale_off<D>(at.t, blk)] = (uint8_t)vsc;
}

// Eight code bytes -> 16 values: code * S (exact) times g, rounded to binary32
// and, for bf16 rows, once more.
template <bool BF>
__device__ __forceinline__ void store_row_block(void *out, size_t elem, uint2 codes, float S, float g) {
    float v[16];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t o[4];
        fp4::e2m1x8_f16(k == 0 ? codes.x : codes.y, o);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&o[m]));
            v[8 * k + 2 * m] = f.x * S * g;
            v[8 * k + 2 * m + 1] = f.y * S * g;
        }
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
    void *__restrict__ v_out, int hkv, int64_t rows, int block_size, int64_t num_slots, int32_t *status) {
    using C = RowCfg<D>;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ __align__(16) uint8_t sk[C::WARPS][C::RW][C::ROW_BYTES], sv[C::WARPS][C::RW][C::ROW_BYTES];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rr = lane / C::NB, blk = lane % C::NB;
    const int64_t row = ((int64_t)blockIdx.x * C::WARPS + warp) * C::RW + rr;
    const bool in = row < rows;
    const int64_t row_c = in ? row : 0;
    const int64_t token = row_c / hkv;
    const int h = (int)(row_c - token * hkv);
    const int64_t slot = slots[token];
    const float kg = k_scale[h], vg = v_scale[h];
    const RowAt at = row_at(slot, h, hkv, block_size, num_slots, fp4::rec_bytes(D));
    if (in && slot >= num_slots && h == 0 && blk == 0) set_status(status, PA_DEV_BAD_SLOT);
    uint32_t ksc = 0, vsc = 0;
    if (in && at.live) {
        const uint8_t *kr = k_cache + at.rec, *vr = v_cache + at.rec;
        ksc = kr[fp4::k_scale_off<D>(at.t, blk)];
        vsc = vr[fp4::v_scale_off<D>(at.t, blk)];
        if constexpr (D == 256) {
            const int j = blk & 7;
            if (blk < 8)
                *reinterpret_cast<uint4 *>(sk[warp][rr] + 16 * j) = *reinterpret_cast<const uint4 *>(kr + k_piece_off(at.t, j));
            else
                *reinterpret_cast<uint4 *>(sv[warp][rr] + 16 * j) =
                    *reinterpret_cast<const uint4 *>(vr + v_piece_off<D>(at.t, j));
        } else {
            if (blk < 4)
                *reinterpret_cast<uint4 *>(sk[warp][rr] + 16 * blk) =
                    *reinterpret_cast<const uint4 *>(kr + k_piece_off(at.t, blk));
            *reinterpret_cast<uint2 *>(sv[warp][rr] + 8 * blk) = *reinterpret_cast<const uint2 *>(vr + v_piece_off<D>(at.t, blk));
        }
    }
    __syncwarp();
    if (!in) return;
    uint2 kq = make_uint2(0u, 0u), vq = kq;  // a row that is not there reads as zeros
    if (at.live) {
        const uint8_t *kp = sk[warp][rr] + (blk >> 3) * 64 + 2 * (blk & 7), *vp = sv[warp][rr] + blk;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t w = (uint32_t)*reinterpret_cast<const uint16_t *>(kp + 16 * c) << (16 * (c & 1));
            if (c < 2)
                kq.x |= w;
            else
                kq.y |= w;
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const uint32_t w = (uint32_t)vp[m * C::NB] << (8 * (m & 3));
            if (m < 4)
                vq.x |= w;
            else
                vq.y |= w;
        }
    }
    const size_t elem = (size_t)row * D + 16 * blk;
    store_row_block<BF>(k_out, elem, kq, fp4::e4m3_f32(ksc), kg);
    store_row_block<BF>(v_out, elem, vq, fp4::e4m3_f32(vsc), vg);
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
pa_status launch_rows(void (*kern)(KArgs...), int64_t rows, int head_dim, void *stream, Args... args) {
    const int64_t per_cta = head_dim == 256 ? RowCfg<256>::WARPS * RowCfg<256>::RW : RowCfg<128>::WARPS * RowCfg<128>::RW;
    const int64_t ctas = (rows + per_cta - 1) / per_cta;
    if (ctas > INT32_MAX) return PA_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
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
    const int64_t rows = static_cast<int64_t>(num_tokens) * num_kv_heads;
    return launch_rows(kern, rows, head_dim, stream, static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new),
                       static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), slot_mapping, k_scale,
                       v_scale, num_kv_heads, rows, block_size, num_pages * block_size, device_status);
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
    const int64_t rows = static_cast<int64_t>(num_tokens) * num_kv_heads;
    return launch_rows(kern, rows, head_dim, stream, static_cast<const uint8_t *>(k_cache),
                       static_cast<const uint8_t *>(v_cache), slot_mapping, k_scale, v_scale, k_out, v_out,
                       num_kv_heads, rows, block_size, num_pages * block_size, device_status);
}

}  // extern "C"
