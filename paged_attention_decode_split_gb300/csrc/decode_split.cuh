// decode_split.cuh -- what the split-KV attention kernels share: the decode
// launch parameters, the 16-token chunk that is the unit of every split, and
// the partition reduce that merges the splits.
//
// The split method ("Hybrid SSM decode rate on dual Radeon under vLLM", the
// split-KV fix): the context of every (sequence, KV head) is cut into splits
// of whole 16-token chunks, each split is one CTA, so batch 1 with 4 KV heads
// still spreads over every SM; a CTA writes its split's normalised output with
// its max logit and exponential sum, and the splits are merged with
// log-sum-exp weights afterwards.  16 divides 784 = 49 x 16, 832 and 16, so a
// chunk never straddles a page and the 16-token tail of a 784-token page
// (784 = 12 x 64 + 16) is just the 49th chunk of the page ("DCU page832
// attention", Sec.2 and Sec.7).  The decode kernel is decode_mma.cuh.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kChunk = 16;    // tokens per TMA copy and per pipeline stage
// 64 tokens: at 1K tokens, 16 splits of 4 chunks take 5.12 us per hybrid call
// against 5.63 us for 32 of 2 (500 tokens: 5.00 against 5.04 us); from 2K up
// and for the dense shape the plan is the same either way
constexpr int kMinChunksPerSplit = 4;
constexpr int kPageTab = 512;  // block-table entries a CTA stages in shared memory
constexpr float kLazyLog2 = 8.f;  // a head's reference max is raised only when it grows by more than 2^8

struct DecodeParams {
    const __nv_bfloat16 *q;  // [B, Hq, D]
    const int32_t *block_table;
    const int32_t *seq_lens;
    void *out;            // [B, Hq, D], written when num_splits == 1
    float *part_o;        // [B, Hq, S, D]
    float2 *part_ml;      // [B, Hq, S]: (max logit in log2 units, exp sum; -1 = poisoned)
    int32_t *status;
    int64_t num_pages;
    int num_q_heads;
    int max_pages_per_seq;
    int max_seq_len;
    int block_size;
    int chunks_per_split;
    int num_splits;
    float scale_log2;     // scale * log2(e)
    int out_bf16;
    int early_kv;         // stream the context before the new row ahead of the dependency wait
    int window;           // 0: full attention; W > 0: only the last W keys
    const float *k_scale; // fp8 cache: [Hkv] dequantisation scales of K and V
    const float *v_scale;
    // Fused append (decode_append): the new token's rows [B, Hkv, D] bf16, written
    // into the cache slot of token L_b - 1 before the chunk holding it is copied;
    // nullptr for a plain decode.  k_cache / v_cache are the caches' base addresses.
    const __nv_bfloat16 *k_new;
    const __nv_bfloat16 *v_new;
    uint8_t *k_cache;
    uint8_t *v_cache;
    // Decode over shared prefixes (SH kernels): sequence b attends here to the
    // tokens from prefix_lens[b], rounded down to whole chunks, on, cut into
    // suffix_splits splits of its own length; their records stand behind the
    // prefix_splits records of the prefix kernel.  prefix_splits = 0: there is no
    // prefix kernel, and all tokens are read here.
    const int32_t *prefix_lens;   // [B]
    const int32_t *group_starts;  // [num_groups + 1]
    int num_groups;
    int max_members;
    int prefix_splits;
    int suffix_splits;
    int suffix_chunks;  // of a split, where that makes no more than suffix_splits
    int by_length;      // the CTAs take the sequences by the lengths of their parts, long ones first
};

// What a sequence's own part of a shared-prefix decode is: its first chunk, and
// whether its lengths make sense (an idle sequence, L = 0, has nothing).
struct Suffix {
    int first;  // chunk
    int end;    // chunks of the sequence
    int per;    // chunks per split
    bool ok;
};
__device__ __forceinline__ Suffix suffix_of(const DecodeParams &p, int b, int L) {
    const int P = p.prefix_lens[b];
    Suffix s{0, (L + kChunk - 1) / kChunk, 1, L == 0 || (P >= 0 && P <= L)};
    if (L > 0 && s.ok) {
        s.first = p.prefix_splits > 0 ? P / kChunk : 0;
        const int n = s.end - s.first;
        s.per = max(p.suffix_chunks, (n + p.suffix_splits - 1) / p.suffix_splits);
    }
    return s;
}

// The sequence that the CTAs of blockIdx.z work on: the z-th by the length of its
// part, in eighths of the longest one and by number within them.  The CTAs of the
// own parts start on the SMs that the prefix kernel leaves, in waves, and a long
// part that starts last ends last (33 parts of up to 3000 tokens, 12 heads each:
// 64.5 us for the call, 69.5 in order of number; 16 groups of 8 sequences 165, 170).
// By a whole warp, each for itself; a function of its own, so that calls without an
// order do not fetch it.
constexpr int kOrderSeqs = 256;  // that a warp orders: eight a lane
static __device__ __noinline__ int sequence_by_length(const int32_t *seq_lens, const int32_t *prefix_lens,
                                                      int max_seq_len, int z, int n) {
    const int lane = threadIdx.x & 31;
    int own[kOrderSeqs / 32], longest = 0;
#pragma unroll
    for (int u = 0; u < kOrderSeqs / 32; ++u) {
        own[u] = 0;
        const int i = 32 * u + lane;
        if (i < n) {
            const int L = seq_lens[i], P = prefix_lens != nullptr ? prefix_lens[i] : 0;
            own[u] = L < 0 || L > max_seq_len ? 0 : max(0, L - max(0, P));
        }
        longest = max(longest, own[u]);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    const float eighths = 8.f / ((float)longest + 1.f);
    int left = z, seq = z;  // of the class at hand
    bool found = false;
#pragma unroll 1
    for (int k = 0; k < 8 && !found; ++k) {
#pragma unroll
        for (int u = 0; u < kOrderSeqs / 32; ++u) {
            if (32 * u >= n) break;
            const bool mine = 32 * u + lane < n && min(7, (int)((float)(longest - own[u]) * eighths)) == k;
            const uint32_t m = __ballot_sync(0xffffffffu, mine);
            const int c = __popc(m);
            if (!found && left < c) {
                seq = 32 * u + (int)__fns(m, 0, left + 1);
                found = true;
            }
            if (!found) left -= c;
        }
    }
    return seq;
}
__device__ __forceinline__ int sequence_of(const DecodeParams &p, int z) {
    return p.by_length ? sequence_by_length(p.seq_lens, p.prefix_splits > 0 ? p.prefix_lens : nullptr, p.max_seq_len, z,
                                            (int)gridDim.z)
                       : z;
}

// The end of a CTA of the own parts: whoever waits for their kernel must have
// waited for the prefix kernel too.
__device__ __forceinline__ void wait_prefix(bool last_cta) {
    if (last_cta) pdl_wait_primary();
}

// Whether sequence b has a place in a group that makes sense: group_starts
// ascends, b is among the first max_members of its group, and its prefix is that
// of the group's leader.  By one whole warp, for the CTAs
// of a sequence's first split; otherwise (status set) the records that the prefix
// kernel may not write are poisoned, so that b's rows become zeros.
__device__ __forceinline__ bool group_ok(const DecodeParams &p, int b, int L, int hq0, int heads, bool report) {
    const int lane = threadIdx.x & 31;
    int lo = -1, hi = -1;
    bool order = true;
    for (int g = lane; g < p.num_groups; g += 32) {
        const int x = p.group_starts[g], y = p.group_starts[g + 1];
        if (x <= b && b < y) {
            lo = x;
            hi = y;
        }
        order &= x >= 0 && x <= y;
    }
    lo = __reduce_max_sync(0xffffffffu, lo);
    hi = min(__reduce_max_sync(0xffffffffu, hi), (int)gridDim.z);  // (a start past the sequences: their number)
    bool ok = __all_sync(0xffffffffu, order) && lo >= 0 && b - lo < p.max_members;
    const bool written = ok;  // by the prefix kernel
    for (int i0 = lo; ok && L != 0 && i0 < hi; i0 += 32) {
        const int i = i0 + lane, len = i < hi ? p.seq_lens[i] : 0, pre = i < hi ? p.prefix_lens[i] : 0;
        const uint32_t live = __ballot_sync(0xffffffffu, leads_group(len, pre, p.max_seq_len));
        if (live != 0) {
            ok = p.prefix_lens[i0 + __ffs(live) - 1] == p.prefix_lens[b];
            break;
        }
    }
    if (!ok && report && lane == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
    if (!written)
        for (int i = lane; i < heads * p.prefix_splits; i += 32)
            p.part_ml[((size_t)b * p.num_q_heads + hq0 + i / p.prefix_splits) * p.num_splits + i % p.prefix_splits] =
                make_float2(-INFINITY, -1.f);
    return ok;
}

__device__ __forceinline__ void store_out(void *out, size_t idx, float v, int out_bf16) {
    if (out_bf16)
        reinterpret_cast<__nv_bfloat16 *>(out)[idx] = __float2bfloat16_rn(v);
    else
        reinterpret_cast<float *>(out)[idx] = v;
}

// Four consecutive outputs from element idx (a multiple of 4): one 16-byte
// (fp32) or 8-byte (bf16) store.
__device__ __forceinline__ void store_out4(void *out, size_t idx, float4 v, int out_bf16) {
    if (out_bf16)
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(out) + idx) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    else
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + idx) = v;
}

// ---------------------------------------------------------------------------
// Partition reduce: out[row, h, :] = sum_i w_i o_i / sum_i w_i with
// w_i = l_i 2^(m_i - max_j m_j) over the non-empty splits of the row's sequence
// (the "reduce afterwards" step of the split-KV fix).  A poisoned split
// (l = -1: bad page or an abandoned wait) zeroes the row.  Rows are
// (sequence, new row) pairs: q_len = 1 for decode, > 1 for verify.
struct ReduceParams {
    const float *part_o;
    const float2 *part_ml;
    void *out;
    int num_q_heads;
    int num_splits;
    int out_bf16;
};


// Grid (Hq, rows, D / 32), 128 threads: each CTA merges a 32-wide slice of
// one (row, head) output.  Its threads split the splits 16 ways; every thread
// issues the loads of all its splits' statistics and partial outputs at once,
// folds them with a running log-sum-exp, and a single exchange merges the 16
// per-group states.  (32-wide slices measured 0.56 us faster per 32K call than
// 64-wide ones and 0.17 us faster than 16-wide ones: more CTAs, fewer loads
// per thread.)
template <int D>
__global__ void __launch_bounds__(128) pa_split_reduce_kernel(const ReduceParams p) {
    constexpr int QD = 8;   // float4 columns of the 32-wide slice
    constexpr int SG = 16;  // split groups
    constexpr int UNROLL = 4;
    __shared__ float4 red_o[SG][QD];
    __shared__ float2 red_ml[SG];
    pdl_launch_dependents();  // a following attention call may start its set-up
    pdl_wait_primary();       // partials of the split kernel are complete and visible

    const int hq = blockIdx.x, row = blockIdx.y, slice = blockIdx.z;
    // Every split wrote its record (an empty one as m = -inf, l = 0), so all
    // of them are read and the sequence length is not needed here.
    const int S_b = p.num_splits;
    const size_t r = (size_t)row * p.num_q_heads + hq;
    const float2 *ml = p.part_ml + r * p.num_splits;
    const int qd = threadIdx.x % QD, sg = threadIdx.x / QD;
    const float *po = p.part_o + r * p.num_splits * D + slice * 32 + qd * 4;

    float M = -INFINITY, W = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;
    for (int i0 = sg; i0 < S_b; i0 += SG * UNROLL) {
        float2 v[UNROLL];
        float4 o[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {  // all loads first, none behind a branch
            const int i = min(i0 + u * SG, S_b - 1);
            v[u] = ml[i];
            o[u] = *reinterpret_cast<const float4 *>(po + (size_t)i * D);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (i0 + u * SG >= S_b) v[u] = make_float2(-INFINITY, 0.f);  // a repeated load: ignore it
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            bad |= v[u].y < 0.f;
            if (!(v[u].y > 0.f)) continue;  // empty split (or poisoned, flagged above)
            const float Mn = fmaxf(M, v[u].x);
            const float c = fast_exp2(M - Mn), e = fast_exp2(v[u].x - Mn) * v[u].y;
            W = fmaf(W, c, e);
            a.x = fmaf(a.x, c, e * o[u].x); a.y = fmaf(a.y, c, e * o[u].y);
            a.z = fmaf(a.z, c, e * o[u].z); a.w = fmaf(a.w, c, e * o[u].w);
            M = Mn;
        }
    }
    red_o[sg][qd] = a;
    if (qd == 0) red_ml[sg] = make_float2(M, W);
    const bool any_bad = __syncthreads_or(bad) != 0;  // a poisoned split anywhere zeroes the row
    if (sg == 0) {
        float Mt = -INFINITY;
#pragma unroll
        for (int j = 0; j < SG; ++j) Mt = fmaxf(Mt, red_ml[j].x);
        float Wt = 0.f;
        float4 at = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < SG; ++j) {
            const float2 mw = red_ml[j];
            if (!(mw.y > 0.f)) continue;
            const float c = fast_exp2(mw.x - Mt);
            const float4 o = red_o[j][qd];
            Wt = fmaf(mw.y, c, Wt);
            at.x = fmaf(o.x, c, at.x); at.y = fmaf(o.y, c, at.y); at.z = fmaf(o.z, c, at.z); at.w = fmaf(o.w, c, at.w);
        }
        const bool zero = any_bad || !(Wt > 0.f);
        const float inv = zero ? 0.f : 1.f / Wt;
        const size_t base = r * D + slice * 32 + qd * 4;
        // (a poisoned row is zero whatever its other splits hold: not 0 times a NaN)
        store_out(p.out, base + 0, zero ? 0.f : at.x * inv, p.out_bf16);
        store_out(p.out, base + 1, zero ? 0.f : at.y * inv, p.out_bf16);
        store_out(p.out, base + 2, zero ? 0.f : at.z * inv, p.out_bf16);
        store_out(p.out, base + 3, zero ? 0.f : at.w * inv, p.out_bf16);
    }
}

// The same merge for few splits (S <= 8: verify, batched decode).  A warp
// merges PPW (row, head) pairs, a lane owning the 4-dim columns lane,
// lane + 32, ... of each (so a warp's load of one column set is 512
// contiguous bytes, and its stores are 16-byte vectors);
// every load of a warp is issued at once, so the kernel makes one dependent
// round trip and needs no shared-memory exchange.  Its CTAs reserve more than
// half of an SM's shared memory (kReduceSmallSmem, unused), so an SM holds at
// most one of them and none beside a split CTA: they land on SMs as the split
// CTAs leave, one per SM, and the grid is sized to about one CTA per SM.
// Packed several to an SM, small CTAs of this kind queued on that SM's share
// of L2 bandwidth while other SMs idled (the verify workload's 12.6 MB of
// partials: 5.9 us with 4 CTAs on each of 96 SMs).
constexpr int kReduceSmallMaxSplits = 8;
constexpr int kReduceSmallSmem = 120 * 1024;

template <int D, int NSL, int PPW>
__global__ void __launch_bounds__(256, 1) pa_split_reduce_small_kernel(const ReduceParams p, int pairs) {
    static_assert(NSL <= kReduceSmallMaxSplits && NSL * PPW <= 16, "slots held in registers");
    constexpr int E = D / 32;  // dims per lane
    pdl_launch_dependents();   // a following attention call may start its set-up
    pdl_wait_primary();        // partials of the split kernel are complete and visible
    const int pair0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * PPW, lane = threadIdx.x & 31;
    if (pair0 >= pairs) return;
    const int S = p.num_splits;
    float2 v[PPW][NSL];
    float4 o[PPW][NSL][E / 4];
#pragma unroll
    for (int j = 0; j < PPW; ++j) {  // all loads first, none behind a branch
        const int pair = min(pair0 + j, pairs - 1);
        const float2 *ml = p.part_ml + (size_t)pair * S;
        const float *po = p.part_o + (size_t)pair * S * D + 4 * lane;
#pragma unroll
        for (int u = 0; u < NSL; ++u) {
            const int i = min(u, S - 1);
            v[j][u] = ml[i];
#pragma unroll
            for (int e = 0; e < E / 4; ++e) o[j][u][e] = *reinterpret_cast<const float4 *>(po + (size_t)i * D + 128 * e);
        }
    }
#pragma unroll
    for (int j = 0; j < PPW; ++j) {
        if (pair0 + j >= pairs) break;
        float M = -INFINITY, W = 0.f;
        float4 a[E / 4];
#pragma unroll
        for (int e = 0; e < E / 4; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        bool bad = false;
#pragma unroll
        for (int u = 0; u < NSL; ++u) {
            if (u >= S) break;
            bad |= v[j][u].y < 0.f;
            if (!(v[j][u].y > 0.f)) continue;  // empty split (or poisoned, flagged above)
            const float Mn = fmaxf(M, v[j][u].x);
            const float c = fast_exp2(M - Mn), w = fast_exp2(v[j][u].x - Mn) * v[j][u].y;
            W = fmaf(W, c, w);
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
                a[e].x = fmaf(a[e].x, c, w * o[j][u][e].x);
                a[e].y = fmaf(a[e].y, c, w * o[j][u][e].y);
                a[e].z = fmaf(a[e].z, c, w * o[j][u][e].z);
                a[e].w = fmaf(a[e].w, c, w * o[j][u][e].w);
            }
            M = Mn;
        }
        const bool zero = bad || !(W > 0.f);
        const float inv = zero ? 0.f : 1.f / W;
        const size_t base = (size_t)(pair0 + j) * D + 4 * lane;
#pragma unroll
        for (int e = 0; e < E / 4; ++e)
            store_out4(p.out, base + 128 * e,
                       zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(a[e].x * inv, a[e].y * inv, a[e].z * inv, a[e].w * inv),
                       p.out_bf16);
    }
}

// The same merge for many rows of more splits (decode over shared prefixes): a
// warp merges one (row, head) pair.  Its lanes take the statistics of 32 splits at
// a time and form their weights against the common maximum, so that no running
// rescale is needed; the outputs of 8 splits are loaded at once.  Taken from two
// warps per SM on (64 rows of 24 heads, 9 splits of 256 dims, 14 MB: 6.7 us); fewer
// pairs would leave SMs idle, and a CTA per pair and 32 dims has more loads in flight.
template <int D>
__global__ void __launch_bounds__(128) pa_split_reduce_rows_kernel(const ReduceParams p, int pairs) {
    constexpr int E = D / 128;  // float4 columns per lane
    constexpr int U = 8;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int pair = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (pair >= pairs) return;
    const int S = p.num_splits;
    const float2 *ml = p.part_ml + (size_t)pair * S;
    const float *po = p.part_o + (size_t)pair * S * D + 4 * lane;
    float M = -INFINITY;
    bool bad = false;
    for (int i = lane; i < S; i += 32) {
        const float2 v = ml[i];
        bad |= v.y < 0.f;
        if (v.y > 0.f) M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    bad = __any_sync(0xffffffffu, bad);
    float W = 0.f;
    float4 a[E];
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < S; i0 += 32) {
        const float2 v = i0 + lane < S ? ml[i0 + lane] : make_float2(-INFINITY, 0.f);
        const float w = v.y > 0.f ? fast_exp2(v.x - M) * v.y : 0.f;
        const uint32_t full = __ballot_sync(0xffffffffu, v.y > 0.f);  // an empty split's outputs may be anything
        W += w;
        for (int i1 = 0; i1 < min(32, S - i0); i1 += U) {
            float4 o[U][E];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    o[u][e] = *reinterpret_cast<const float4 *>(po + (size_t)min(i0 + i1 + u, S - 1) * D + 128 * e);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float c = __shfl_sync(0xffffffffu, w, i1 + u);
                if ((full >> (i1 + u) & 1) == 0) continue;  // (not by c: a weight of 0 keeps the NaN of what it weighs)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    a[e].x = fmaf(c, o[u][e].x, a[e].x); a[e].y = fmaf(c, o[u][e].y, a[e].y);
                    a[e].z = fmaf(c, o[u][e].z, a[e].z); a[e].w = fmaf(c, o[u][e].w, a[e].w);
                }
            }
        }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) W += __shfl_xor_sync(0xffffffffu, W, k);
    const bool zero = bad || !(W > 0.f);
    const float inv = zero ? 0.f : 1.f / W;
#pragma unroll
    for (int e = 0; e < E; ++e)
        store_out4(p.out, (size_t)pair * D + 4 * lane + 128 * e,
                   zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                        : make_float4(a[e].x * inv, a[e].y * inv, a[e].z * inv, a[e].w * inv),
                   p.out_bf16);
}

}  // namespace pa
