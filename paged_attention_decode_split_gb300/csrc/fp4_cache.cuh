// fp4_cache.cuh -- the 4-bit KV cache: its record layout, its quantiser, and
// the conversions the attention kernels share.
//
// Format.  An element x of KV head h is held as an e2m1 code (1 sign, 2
// exponent bits with bias 1, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) with
// one e4m3 scale S per 16 consecutive dims of its row and one binary32 scale
// g per KV head:  x ~ code * S * g.  4.5 bits per element.  code * S has at
// most six significant bits and lies in [2^-10, 2688] (or is 0), so the
// kernels form it in f16 without rounding and apply g to the sums.
//
// Layout.  The 16 tokens of one (page, KV head) chunk form one record of 9 D
// contiguous bytes: 8 D bytes of codes, then D scales.  A cache tensor is
// [pages, KV heads, block_size / 16, 9 D]: the chunks of a page that one CTA
// reads are contiguous, so a copy needs no tensor map, however small the
// page, and the bytes of a record stand in the order in which a lane of the
// decode's score and P.V products uses them, so every shared-memory read is a
// full-width one at lane * 16 (no ldmatrix, no swizzle).  A byte holds two
// dims of ONE token: a new token is written without reading its neighbours'
// bytes.
//  K code of token t, dims d, d + 1 (d even): with half = t / 8, r = t % 8,
//    d = 16 (8 j + i) + 4 c + 2 b:  (2 j + half) * 512 + (4 r + c) * 16 + 2 i + b
//  K scale of (t, blk = d / 16):    8 D + t * D / 16 + blk
//  V code of token t, dims d, d + 1: with t = 8 half + 2 c + par, u = 2 half +
//    par, d = 16 blk + 2 r:         u * 2 D + (4 r + c) * D / 16 + blk
//  V scale of (t, blk):             8 D + (blk / 4) * 64 + c * 16 + (blk % 4) * 4 + u
// (lane = 4 r + c of the m16n8k16 fragments; low nibble = even dim.)
#pragma once

#include "pa_device.cuh"

namespace pa {

namespace fp4 {

__host__ __device__ constexpr int rec_bytes(int D) { return 9 * D; }

// Byte offset inside a record of the first code byte of 16-dim block `blk` of
// token t; the block's code bytes m = 0..7 (dims 2 m, 2 m + 1) follow at
// k_code_off(...) + (m / 2) * 16 + m % 2 and v_code_off(...) + m * (4 * D / 16).
__device__ __forceinline__ int k_code_off(int t, int blk) {
    return ((blk >> 3) * 2 + (t >> 3)) * 512 + (t & 7) * 64 + 2 * (blk & 7);
}
template <int D>
__device__ __forceinline__ int v_code_off(int t, int blk) {
    const int u = 2 * (t >> 3) + (t & 1), c = (t & 7) >> 1;
    return u * 2 * D + c * (D / 16) + blk;
}
template <int D>
__device__ __forceinline__ int k_scale_off(int t, int blk) {
    return 8 * D + t * (D / 16) + blk;
}
template <int D>
__device__ __forceinline__ int v_scale_off(int t, int blk) {
    const int u = 2 * (t >> 3) + (t & 1), c = (t & 7) >> 1;
    return 8 * D + (blk >> 2) * 64 + c * 16 + (blk & 3) * 4 + u;
}

// Four code bytes (eight codes) -> four f16 pairs, byte order; exact.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

// Two floats -> one code byte (lo in the low nibble): round to nearest even,
// saturating at +-6.
__device__ __forceinline__ uint32_t e2m1x2_rn(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// Four e4m3 codes -> four f16 (two pairs); exact.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// The two scale codes in the low or the high half.
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w) {
    uint32_t r;
    if (HIGH)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ float e4m3_f32(uint32_t code) {
    uint32_t lo, hi;
    e4m3x4_f16(code, lo, hi);
    return __half2float(__ushort_as_half((unsigned short)(lo & 0xffffu)));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
}
// a * (low half of s), a * (high half of s)
__device__ __forceinline__ uint32_t hmul2_lo(uint32_t a, uint32_t s) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a), __low2half2(*reinterpret_cast<const __half2 *>(&s)));
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t hmul2_hi(uint32_t a, uint32_t s) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a), __high2half2(*reinterpret_cast<const __half2 *>(&s)));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The scale code of a block with largest magnitude `amax` (a bf16 bit pattern,
// sign cleared): e4m3(amax / (6 g)), the product and the division in binary32,
// rounding to nearest even and saturating at 448; 0x7F (NaN) for a NaN.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax, float g) {
    const float a = __uint_as_float(amax << 16);
    uint16_t s;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s) : "f"(0.f), "f"(__fdiv_rn(a, __fmul_rn(6.f, g))));
    return amax > 0x7f80u ? 0x7fu : (uint32_t)s & 0xffu;
}

// What an element of the block is multiplied by before it is rounded to e2m1:
// 1 / (S g), product and reciprocal rounded to binary32; 0 (all codes +-0)
// stands for a block without codes (S = 0, or NaN).
__device__ __forceinline__ float code_factor(uint32_t s, float g) {
    const float S = e4m3_f32(s);
    return s == 0x7fu || S == 0.f ? 0.f : __frcp_rn(__fmul_rn(S, g));
}

// Two bf16 (packed) -> one code byte.
__device__ __forceinline__ uint32_t code_byte(uint32_t w, float r) {
    return r == 0.f ? 0u : e2m1x2_rn(__fmul_rn(bf16lo(w), r), __fmul_rn(bf16hi(w), r));
}

// Quantises a 16-dim block (32 bytes of bf16): its eight code bytes (dims 2 m,
// 2 m + 1 in byte m) and its scale code.
__device__ __forceinline__ uint2 quantise_block(const uint4 &a, const uint4 &b, float g, uint32_t &s) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t amax = 0;
#pragma unroll
    for (int m = 0; m < 8; ++m) amax = max(amax, bf16x2_absmax(w[m]));
    s = scale_code(amax, g);
    const float r = code_factor(s, g);
    uint32_t o[2] = {0u, 0u};
#pragma unroll
    for (int m = 0; m < 8; ++m) o[m >> 2] |= code_byte(w[m], r) << (8 * (m & 3));
    return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ uint32_t byte_of(uint2 v, int m) { return ((m < 4 ? v.x : v.y) >> (8 * (m & 3))) & 0xffu; }

// Quantises the 16-dim block `blk` of a new row (32 bytes at src) into token t
// of the record at rec.  V: the V layout, else K's.
template <int D, bool V>
__device__ __forceinline__ void store_block(uint8_t *rec, int t, int blk, const uint4 *src, float g) {
    uint32_t s;
    const uint2 q = quantise_block(src[0], src[1], g, s);
    if constexpr (V) {
        uint8_t *p = rec + v_code_off<D>(t, blk);
#pragma unroll
        for (int m = 0; m < 8; ++m) p[m * (D / 4)] = (uint8_t)byte_of(q, m);
        rec[v_scale_off<D>(t, blk)] = (uint8_t)s;
    } else {
        uint8_t *p = rec + k_code_off(t, blk);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint16_t *>(p + c * 16) = (uint16_t)((c < 2 ? q.x : q.y) >> (16 * (c & 1)));
        rec[k_scale_off<D>(t, blk)] = (uint8_t)s;
    }
}

// D = A B for one m16n8k16 tile of f16 (mm::mma with a zero addend).
__device__ __forceinline__ void mma0_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Untiled bulk copy global -> shared (16-byte aligned addresses, a multiple of
// 16 bytes), completion signalled on `bar` as bytes.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
            "r"(smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

}  // namespace fp4

}  // namespace pa
