// rotary.cu -- rotary positions: the step before a cache write.  rotary turns
// rows of q and k, rotary_and_cache turns them and writes k and v into their
// cache slots (bf16, e4m3 or fp4) in the same pass; rotary_frequencies makes
// the table of angles per position on the host.
//
// Mathematics.  Pair j of a head, (a, b) = elements (j, j + R/2) or (2j, 2j + 1)
// of its first R, becomes
//     (a cos t - b sin t, b cos t + a sin t) * factor,   t = position * w_j;
// the gradient is the same with -t.  The angle is kept as a fraction of a turn
// in 64-bit fixed point: the table holds w_j / 2 pi * 2^64, the product with
// the position wraps modulo whole turns without losing a bit, and the upper 32
// bits, read as a signed number of half turns, go to sincospif.  So a position
// of a million is as exact as one of zero (error of an angle: 2^-25 half turns,
// the conversion to binary32), without 64-bit floating point.
//
// A CTA takes a token: its threads load two 16-byte vectors per item (the two
// halves of eight pairs, or 16 neighbouring elements), four items at once, form
// the R/2 sines and cosines once for all heads while the loads are on their
// way, and store the turned vectors.
//
// Bound by HBM: 16,411 tokens of 24 + 4 heads of 256 (R = 64) with their cache
// write, 538 MB, take 77.8 us = 6.9 TB/s, as fast as a copy; 8192 rows of 32 + 8
// heads of 128 turned back, 168 MB, 29.0 us = 5.8 TB/s (issue slots 52 %; its last
// wave and the stores that are still in L2 at the end).  128 threads of 4 items
// (78.1 / 28.8 us) against 256 of 2 (81 / 30.7), 128 of 2 (78.8 / 27.9, but 11.8
// against 11.5 for 2051 tokens in e4m3), 192 of 2 (84 / 28.7).
// A step of 32 tokens is a launch: 3.8 us.
#include <cmath>

#include "fp4_cache.cuh"

namespace pa {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeItems = 4;       // items of two vectors in flight per thread
constexpr int kRopeMaxDim = 1024;   // head_dim: the table of a token stands in shared memory

enum RopeTo { kRopeRows = 0, kRopeBf16, kRopeFp8, kRopeFp4 };

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;  // rows of a token: [heads, D], q_stride ... elements apart
    __nv_bfloat16 *q_out, *k_out;
    uint8_t *k_cache, *v_cache;
    const int32_t *positions;
    const uint64_t *freqs;
    const int64_t *slots;
    const float *k_scale, *v_scale;
    int32_t *status;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    int64_t num_slots;
    float factor, sign;
    int offset;       // added to every position
    int hq, hkv, D, R, block_size;
    int items;        // q and k (and v) items of a token
    uint32_t item_mul;  // ceil(2^32 / (D / 16)): the division of an item by the items of a head
};

// Eight pairs: (x[i], y[i]) turned by (c[i], s[i]).
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = a;
    a = fmaf(x, c, -b * s);
    b = fmaf(b, c, x * s);
}

__device__ __forceinline__ void widen(const uint4 &w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo(u[i]);
        f[2 * i + 1] = bf16hi(u[i]);
    }
}

__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

template <bool INTER, int TO>
__global__ void __launch_bounds__(kRopeThreads) pa_rotary_kernel(const RopeParams p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ __align__(16) float cosines[kRopeMaxDim / 2], sines[kRopeMaxDim / 2];
    extern __shared__ __align__(16) uint8_t rope_rows[];  // fp4: the token's K and V rows, bf16
    const int64_t token = blockIdx.x;
    const int per_head = p.D / 16, rot = p.R / 16;
    const int heads = TO == kRopeRows ? p.hq + p.hkv : p.hq + 2 * p.hkv;
    const int64_t slot = TO == kRopeRows ? 0 : p.slots[token];
    const int64_t pos = (int64_t)p.positions[token] + p.offset;
    bool live = true;
    if (TO != kRopeRows) {
        live = slot >= 0 && slot < p.num_slots;
        if (slot >= p.num_slots && threadIdx.x == 0) set_status(p.status, PA_DEV_BAD_SLOT);
    }
    bool ready = false;
    for (int first = threadIdx.x; first < p.items || !ready; first += kRopeThreads * kRopeItems) {
        uint4 x[kRopeItems], y[kRopeItems];
        int head[kRopeItems], at[kRopeItems], e0[kRopeItems], e1[kRopeItems];
#pragma unroll
        for (int u = 0; u < kRopeItems; ++u) {
            const int item = first + u * kRopeThreads;
            head[u] = item < p.items ? (int)__umulhi((uint32_t)item, p.item_mul) : heads;
            at[u] = item - head[u] * per_head;
            const bool half = !INTER && at[u] < rot;
            e0[u] = half ? 8 * at[u] : 16 * at[u];
            e1[u] = half ? e0[u] + p.R / 2 : e0[u] + 8;
            const __nv_bfloat16 *row = nullptr;
            if (head[u] < p.hq)
                row = p.q + token * p.q_stride + head[u] * p.D;
            else if (head[u] < p.hq + p.hkv)
                row = p.k + token * p.k_stride + (head[u] - p.hq) * p.D;
            else if (head[u] < heads)
                row = p.v + token * p.v_stride + (head[u] - p.hq - p.hkv) * p.D;
            if (row != nullptr) {
                x[u] = *reinterpret_cast<const uint4 *>(row + e0[u]);
                y[u] = *reinterpret_cast<const uint4 *>(row + e1[u]);
            }
        }
        if (!ready) {  // (every thread comes here once)
            for (int j = threadIdx.x; j < p.R / 2; j += kRopeThreads) {
                const uint64_t turns = (uint64_t)pos * p.freqs[j];
                float s, c;
                sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
                cosines[j] = c * p.factor;
                sines[j] = s * p.factor * p.sign;
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kRopeItems; ++u) {
            if (head[u] >= heads) continue;
            const bool is_v = head[u] >= p.hq + p.hkv, is_q = head[u] < p.hq;
            if (!is_v && at[u] < rot) {
                float a[8], b[8], c[8], s[8];
                widen(x[u], a);
                widen(y[u], b);
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    *reinterpret_cast<float4 *>(c + i) = *reinterpret_cast<const float4 *>(cosines + 8 * at[u] + i);
                    *reinterpret_cast<float4 *>(s + i) = *reinterpret_cast<const float4 *>(sines + 8 * at[u] + i);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (INTER) {
                        if (i < 4)
                            turn(a[2 * i], a[2 * i + 1], c[i], s[i]);
                        else
                            turn(b[2 * i - 8], b[2 * i - 7], c[i], s[i]);
                    } else {
                        turn(a[i], b[i], c[i], s[i]);
                    }
                }
                x[u] = narrow(a);
                y[u] = narrow(b);
            }
            if (is_q || TO == kRopeRows) {
                __nv_bfloat16 *row = is_q ? p.q_out + token * p.q_out_stride + head[u] * p.D
                                          : p.k_out + token * p.k_out_stride + (head[u] - p.hq) * p.D;
                *reinterpret_cast<uint4 *>(row + e0[u]) = x[u];
                *reinterpret_cast<uint4 *>(row + e1[u]) = y[u];
                continue;
            }
            if (!live) continue;
            const int h = is_v ? head[u] - p.hq - p.hkv : head[u] - p.hq;
            const int64_t elem = (slot * p.hkv + h) * p.D;
            if constexpr (TO == kRopeBf16) {
                __nv_bfloat16 *row = reinterpret_cast<__nv_bfloat16 *>(is_v ? p.v_cache : p.k_cache) + elem;
                *reinterpret_cast<uint4 *>(row + e0[u]) = x[u];
                *reinterpret_cast<uint4 *>(row + e1[u]) = y[u];
            } else if constexpr (TO == kRopeFp8) {
                uint8_t *row = (is_v ? p.v_cache : p.k_cache) + elem;
                const float scale = is_v ? p.v_scale[h] : p.k_scale[h];
                *reinterpret_cast<uint2 *>(row + e0[u]) = e4m3x8_div(x[u], scale);
                *reinterpret_cast<uint2 *>(row + e1[u]) = e4m3x8_div(y[u], scale);
            } else if constexpr (TO == kRopeFp4) {
                __nv_bfloat16 *row =
                    reinterpret_cast<__nv_bfloat16 *>(rope_rows) + (size_t)(head[u] - p.hq) * p.D;
                *reinterpret_cast<uint4 *>(row + e0[u]) = x[u];
                *reinterpret_cast<uint4 *>(row + e1[u]) = y[u];
            }
        }
    }
    if constexpr (TO == kRopeFp4) {  // blocks of 16 dims from the staged rows
        __syncthreads();
        if (!live) return;
        const int64_t page = slot / p.block_size;
        const int t = (int)(slot - page * p.block_size), blocks = p.hkv * per_head;
        const int rec_bytes = fp4::rec_bytes(p.D);
        for (int i = threadIdx.x; i < 2 * blocks; i += kRopeThreads) {
            const bool is_v = i >= blocks;
            const int r = is_v ? i - blocks : i, h = r / per_head, blk = r - h * per_head;
            const size_t rec = (((size_t)page * p.hkv + h) * (p.block_size / 16) + t / 16) * rec_bytes;
            const uint4 *src = reinterpret_cast<const uint4 *>(rope_rows) + 2 * (size_t)i;
            if (p.D == 256) {
                if (is_v)
                    fp4::store_block<256, true>(p.v_cache + rec, t % 16, blk, src, p.v_scale[h]);
                else
                    fp4::store_block<256, false>(p.k_cache + rec, t % 16, blk, src, p.k_scale[h]);
            } else {
                if (is_v)
                    fp4::store_block<128, true>(p.v_cache + rec, t % 16, blk, src, p.v_scale[h]);
                else
                    fp4::store_block<128, false>(p.k_cache + rec, t % 16, blk, src, p.k_scale[h]);
            }
        }
    }
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of `width` elements, `stride` apart, of n tokens.
struct Rows {
    const void *at;
    int64_t stride, width;
};

// Whether two sets of rows share no byte (rows of one buffer may lie side by
// side, as q and k of a projection do).
bool disjoint(const Rows &a, const Rows &b, int64_t n) {
    if (!a.at || !b.at || n == 0 || a.width == 0 || b.width == 0) return true;
    const int64_t x = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.at)) / 2;
    const int64_t y = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at)) / 2;
    if (x + (n - 1) * a.stride + a.width <= y || y + (n - 1) * b.stride + b.width <= x) return true;
    if (a.stride != b.stride || a.stride <= 0) return false;
    const int64_t off = ((y - x) % a.stride + a.stride) % a.stride;  // b's row start inside a row of a
    return off >= a.width && off + b.width <= a.stride;
}

// One set of rows that is read and one that is written: the same, or apart.
bool in_place_or_apart(const Rows &in, const Rows &out, int64_t n) {
    return (in.at == out.at && in.width == out.width && (in.stride == out.stride || n == 1)) || disjoint(in, out, n);
}

pa_status check_rope(const RopeParams &p, int64_t n, int flags, bool cache) {
    if (n < 0 || p.hq < 0 || p.hkv < 0 || p.hq + p.hkv < 1 || p.D < 1 || p.R < 1 || p.R > p.D ||
        (flags & ~(PA_ROPE_INTERLEAVED | PA_ROPE_INVERSE)) != 0 || !std::isfinite(p.factor))
        return PA_ERR_INVALID_ARG;
    if (p.D % 16 != 0 || p.D < 32 || p.R % 16 != 0 || p.D > kRopeMaxDim || (p.hq + 2ll * p.hkv) * (p.D / 16) > 65535)
        return PA_ERR_UNSUPPORTED;
    if (n > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (n == 0) return PA_OK;
    if (!p.positions || !p.freqs || (p.hq > 0 && (!p.q || !p.q_out)) || (p.hkv > 0 && !p.k)) return PA_ERR_INVALID_ARG;
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.q_out, 16) ||
        !aligned(p.k_out, 16) || !aligned(p.positions, 4) || !aligned(p.freqs, 8) || p.q_stride % 8 != 0 ||
        p.k_stride % 8 != 0 || p.v_stride % 8 != 0 || p.q_out_stride % 8 != 0 || p.k_out_stride % 8 != 0)
        return PA_ERR_INVALID_ARG;
    const int64_t wq = (int64_t)p.hq * p.D, wk = (int64_t)p.hkv * p.D;
    // rows that are written do not overlap each other; strides of rows that are read may be anything
    if (n > 1 && ((p.hq > 0 && p.q_out_stride < wq) || (p.k_out && p.k_out_stride < wk))) return PA_ERR_INVALID_ARG;
    const Rows q{p.q, p.q_stride, wq}, k{p.k, p.k_stride, wk}, v{p.v, p.v_stride, wk};
    const Rows qo{p.q_out, p.q_out_stride, wq}, ko{p.k_out, p.k_out_stride, wk};
    if (n > 1 && (p.q_stride < 0 || p.k_stride < 0 || p.v_stride < 0)) return PA_ERR_INVALID_ARG;
    if (n > 1)  // (so that offsets of rows stay in 64 bits)
        for (const int64_t stride : {p.q_stride, p.k_stride, p.v_stride, p.q_out_stride, p.k_out_stride})
            if (stride > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (!in_place_or_apart(q, qo, n) || !disjoint(k, qo, n) || !disjoint(v, qo, n)) return PA_ERR_INVALID_ARG;
    if (!cache && (!in_place_or_apart(k, ko, n) || !disjoint(q, ko, n) || !disjoint(qo, ko, n)))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

pa_status launch_rope(RopeParams &p, int64_t n, int flags, int to, void *stream) {
    const bool inter = (flags & PA_ROPE_INTERLEAVED) != 0;
    p.sign = (flags & PA_ROPE_INVERSE) != 0 ? -1.f : 1.f;
    const int per_head = p.D / 16;
    p.items = (p.hq + (to == kRopeRows ? 1 : 2) * p.hkv) * per_head;
    p.item_mul = (uint32_t)(((1ull << 32) + per_head - 1) / per_head);  // (per_head >= 2)
    void (*kern)(RopeParams) = nullptr;
    switch (to) {
        case kRopeRows: kern = inter ? pa_rotary_kernel<true, kRopeRows> : pa_rotary_kernel<false, kRopeRows>; break;
        case kRopeBf16: kern = inter ? pa_rotary_kernel<true, kRopeBf16> : pa_rotary_kernel<false, kRopeBf16>; break;
        case kRopeFp8: kern = inter ? pa_rotary_kernel<true, kRopeFp8> : pa_rotary_kernel<false, kRopeFp8>; break;
        default: kern = inter ? pa_rotary_kernel<true, kRopeFp4> : pa_rotary_kernel<false, kRopeFp4>; break;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = to == kRopeFp4 ? (size_t)4 * p.hkv * p.D : 0;  // K and V rows in bf16
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const RopeParams &>(p)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

RopeParams rope_params(const pa_rotary_desc *d, const void *q, const void *k, const int32_t *positions,
                       const int64_t *freqs, void *q_out) {
    RopeParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.positions = positions;
    p.freqs = reinterpret_cast<const uint64_t *>(freqs);
    p.hq = d->num_q_heads;
    p.hkv = d->num_kv_heads;
    p.D = d->head_dim;
    p.R = d->rotary_dim;
    p.factor = d->factor;
    p.offset = d->position_offset;
    p.q_stride = d->q_stride;
    p.k_stride = d->k_stride;
    p.v_stride = d->v_stride;
    p.q_out_stride = d->q_out_stride;
    p.k_out_stride = d->k_out_stride;
    return p;
}

pa_status rope_cache_call(int to, const void *q, const void *k, const void *v, const int32_t *positions,
                          const int64_t *freqs, void *q_out, void *k_cache, void *v_cache,
                          const int64_t *slot_mapping, const float *k_scale, const float *v_scale,
                          const pa_rotary_desc *d, int32_t block_size, int64_t num_pages, int32_t *status,
                          void *stream) {
    if (!d) return PA_ERR_INVALID_ARG;
    RopeParams p = rope_params(d, q, k, positions, freqs, q_out);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.k_out_stride = 0;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.slots = slot_mapping;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_size = block_size;
    p.status = status;
    if (block_size < 1 || num_pages < 1 || (d->flags & PA_ROPE_INVERSE) != 0 || d->num_kv_heads < 1)
        return PA_ERR_INVALID_ARG;
    if (num_pages > INT32_MAX) return PA_ERR_UNSUPPORTED;
    p.num_slots = num_pages * block_size;
    const pa_status st = check_rope(p, d->num_tokens, d->flags, true);
    if (st != PA_OK) return st;
    if (to == kRopeFp4 && ((d->head_dim != 128 && d->head_dim != 256) || block_size % 16 != 0 ||
                           4ll * d->num_kv_heads * d->head_dim > 40 * 1024))
        return PA_ERR_UNSUPPORTED;
    if (d->num_tokens == 0) return PA_OK;
    if (!v || !k_cache || !v_cache || !slot_mapping || (to != kRopeBf16 && (!k_scale || !v_scale)))
        return PA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_mapping, 8) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4))
        return PA_ERR_INVALID_ARG;
    return launch_rope(p, d->num_tokens, d->flags, to, stream);
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_rotary_frequencies(const pa_rotary_scaling *s, int64_t *freqs, float *factor) {
    if (!s || !freqs || !factor) return PA_ERR_INVALID_ARG;
    const int r = s->rotary_dim;
    if (r < 2 || r % 2 != 0 || !(s->base > 1.0) || !std::isfinite(s->base)) return PA_ERR_INVALID_ARG;
    if (s->kind < PA_ROPE_SCALE_NONE || s->kind > PA_ROPE_SCALE_BANDS) return PA_ERR_INVALID_ARG;
    const bool by_turns = s->kind == PA_ROPE_SCALE_YARN || s->kind == PA_ROPE_SCALE_BANDS;
    if (s->kind != PA_ROPE_SCALE_NONE && !(s->factor >= 1.0 && std::isfinite(s->factor))) return PA_ERR_INVALID_ARG;
    if (by_turns && !(s->original_len > 0 && s->low_turns > 0.0 && s->high_turns > s->low_turns &&
                      std::isfinite(s->high_turns)))
        return PA_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    double base = s->base;
    if (s->kind == PA_ROPE_SCALE_NTK && r > 2) base *= std::pow(s->factor, (double)r / (r - 2));
    double low = 0.0, high = 0.0;  // yarn: the pairs between which the stretch sets in
    if (s->kind == PA_ROPE_SCALE_YARN) {
        const double per = 2.0 * std::log(s->base);
        low = std::floor(r * std::log(s->original_len / (s->high_turns * two_pi)) / per);
        high = std::ceil(r * std::log(s->original_len / (s->low_turns * two_pi)) / per);
        low = std::fmax(low, 0.0);
        high = std::fmin(high, r - 1.0);
    }
    for (int j = 0; j < r / 2; ++j) {
        double w = std::pow(base, -2.0 * j / r);
        double stretched = 0.0;  // share of the pair that is stretched by the factor
        if (s->kind == PA_ROPE_SCALE_LINEAR) {
            stretched = 1.0;
        } else if (s->kind == PA_ROPE_SCALE_YARN) {
            stretched = std::fmin(1.0, std::fmax(0.0, (j - low) / std::fmax(high - low, 0.001)));
        } else if (s->kind == PA_ROPE_SCALE_BANDS) {
            const double turns = s->original_len * w / two_pi;
            stretched = 1.0 - std::fmin(1.0, std::fmax(0.0, (turns - s->low_turns) / (s->high_turns - s->low_turns)));
        }
        if (stretched > 0.0) w = w / s->factor * stretched + w * (1.0 - stretched);
        freqs[j] = (int64_t)std::nearbyint(w / two_pi * 18446744073709551616.0);  // < 2^62: w <= 1
    }
    *factor = s->kind == PA_ROPE_SCALE_YARN ? (float)(0.1 * std::log(s->factor) + 1.0) : 1.0f;
    return PA_OK;
}

pa_status pa_rotary(const void *q, const void *k, const int32_t *positions, const int64_t *freqs, void *q_out,
                    void *k_out, const pa_rotary_desc *d, void *stream) {
    if (!d) return PA_ERR_INVALID_ARG;
    RopeParams p = rope_params(d, q, k, positions, freqs, q_out);
    p.v_stride = 0;
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    const pa_status st = check_rope(p, d->num_tokens, d->flags, false);
    if (st != PA_OK) return st;
    if (d->num_tokens == 0) return PA_OK;
    if (d->num_kv_heads > 0 && !k_out) return PA_ERR_INVALID_ARG;
    return launch_rope(p, d->num_tokens, d->flags, kRopeRows, stream);
}

pa_status pa_rotary_and_cache(const void *q, const void *k, const void *v, const int32_t *positions,
                              const int64_t *freqs, void *q_out, void *k_cache, void *v_cache,
                              const int64_t *slot_mapping, const pa_rotary_desc *d, int32_t block_size,
                              int64_t num_pages, int32_t *device_status, void *stream) {
    return rope_cache_call(kRopeBf16, q, k, v, positions, freqs, q_out, k_cache, v_cache, slot_mapping, nullptr,
                           nullptr, d, block_size, num_pages, device_status, stream);
}

pa_status pa_rotary_and_cache_fp8(const void *q, const void *k, const void *v, const int32_t *positions,
                                  const int64_t *freqs, void *q_out, void *k_cache, void *v_cache,
                                  const int64_t *slot_mapping, const float *k_scale, const float *v_scale,
                                  const pa_rotary_desc *d, int32_t block_size, int64_t num_pages,
                                  int32_t *device_status, void *stream) {
    return rope_cache_call(kRopeFp8, q, k, v, positions, freqs, q_out, k_cache, v_cache, slot_mapping, k_scale,
                           v_scale, d, block_size, num_pages, device_status, stream);
}

pa_status pa_rotary_and_cache_fp4(const void *q, const void *k, const void *v, const int32_t *positions,
                                  const int64_t *freqs, void *q_out, void *k_cache, void *v_cache,
                                  const int64_t *slot_mapping, const float *k_scale, const float *v_scale,
                                  const pa_rotary_desc *d, int32_t block_size, int64_t num_pages,
                                  int32_t *device_status, void *stream) {
    return rope_cache_call(kRopeFp4, q, k, v, positions, freqs, q_out, k_cache, v_cache, slot_mapping, k_scale,
                           v_scale, d, block_size, num_pages, device_status, stream);
}

}  // extern "C"
