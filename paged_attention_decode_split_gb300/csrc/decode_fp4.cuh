// decode_fp4.cuh -- split-KV paged-attention decode over the fp4 cache
// (fp4_cache.cuh), both products on the tensor cores (mma.sync m16n8k16 in
// f16, fp32 accumulation).
//
// Mathematics: the split-KV decode of decode_mma.cuh -- per (sequence, KV
// head) split of whole 16-token chunks, S^T = K Q^T, online softmax with a
// lazily raised reference max, O^T += V^T P^T, the split's normalised output
// with its max logit and exponential sum for the partition reduce -- with
// K = code * S and V = code * S formed in f16 (exact: six significant bits),
// k_scale[h] joined to the softmax scale and v_scale[h] to the normaliser.
// q enters as f16 scaled by a power of two per head (f16_prescale), P as an
// f16 head plus an f16 residual (22 significant bits): what is rounded to
// fewer than 32 bits is rounded below the sums' own error.
//
// Layout on sm_103a:
//  * A chunk is two records (K, V) of 9 D contiguous bytes.  Every warp owns a
//    ring of SPW stages of one chunk and fills it itself: lane k issues the
//    copies of the warp's k-th chunk up front, lane 0 refills a stage when the
//    warp has read it.  No producer warp and no empty barriers; all of a
//    split's first NW * SPW chunks are in flight at once.
//  * Fragments come from shared memory by 16-byte loads at lane * 16 (the
//    record is laid out for them).  K: a lane's 16 bytes are the codes of one
//    token, dims 16 blk + 4 c .. + 3 of eight blocks; cvt widens a byte to a
//    pair, one multiply applies the block's scale (one scale per token and
//    k16 step).  V: 16 bytes are the codes of one token, dims 16 blk + 2 r, +1
//    of every block; the two tokens of a fragment register are interleaved
//    nibble by nibble (two bit selects per four bytes) before cvt, and one
//    multiply by the tokens' scale pair finishes it (one m16 tile is one scale
//    block).
#pragma once

#include "decode_mma.cuh"
#include "fp4_cache.cuh"

namespace pa {

template <int D, int NT, int NW, int SPW>
struct Fp4DecodeCfg {
    static constexpr int REC = fp4::rec_bytes(D);
    static constexpr int STAGE_BYTES = 2 * REC;  // K record, then V record
    static constexpr int THREADS = NW * 32;
    static constexpr int NB = D / 16;            // scale blocks = k16 steps = m16 tiles of d
    static constexpr int GMAX = 8 * NT;
    static constexpr int HS = D + 4;             // merge row stride in floats (bank spread)
    static constexpr int RING_BYTES = NW * SPW * STAGE_BYTES;
    static constexpr int MERGE_BYTES = NW * GMAX * HS * 4;
    static constexpr int OFF_BAR = RING_BYTES > MERGE_BYTES ? RING_BYTES : MERGE_BYTES;
    static constexpr int OFF_FLAGS = OFF_BAR + NW * SPW * 8;
    static constexpr int OFF_ML = OFF_FLAGS + 16;           // [NW][GMAX] (m, l)
    static constexpr int OFF_W = OFF_ML + NW * GMAX * 8;    // [NW][GMAX] merge weights
    static constexpr int OFF_PT = OFF_W + NW * GMAX * 4;
    static constexpr int SMEM_BYTES = OFF_PT + kPageTab * 4 + 128;  // + slack to align the base
    static_assert(D == 128 || D == 256, "head_dim 128 or 256");
    static_assert(NT == 1 || NT == 2, "up to 16 heads per KV head");
    static_assert(SPW <= 32, "a lane per stage issues the first copies");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
};

// The new token's rows of this CTA's KV head, quantised into their cache slot
// exactly as reshape_and_cache_fp4 would, made visible to the copy engine
// before the chunk that holds them is copied.  Called by the warp that owns
// the chunk.
template <int D>
__device__ __forceinline__ void append_new_row_fp4(const DecodeParams &p, int b, int kvh, int t, int page) {
    const int hkv = gridDim.y, lane = threadIdx.x & 31, pos = t % p.block_size;
    const size_t rec = (((size_t)page * hkv + kvh) * (p.block_size / 16) + pos / 16) * fp4::rec_bytes(D);
    const size_t row = ((size_t)b * hkv + kvh) * D;
    constexpr int NB = D / 16;
    for (int j = lane; j < 2 * NB; j += 32) {
        const int blk = j % NB;
        if (j < NB)
            fp4::store_block<D, false>(p.k_cache + rec, pos % 16, blk,
                                       reinterpret_cast<const uint4 *>(p.k_new + row) + 2 * blk, p.k_scale[kvh]);
        else
            fp4::store_block<D, true>(p.v_cache + rec, pos % 16, blk,
                                      reinterpret_cast<const uint4 *>(p.v_new + row) + 2 * blk, p.v_scale[kvh]);
    }
    asm volatile("fence.proxy.async.global;" ::: "memory");  // generic-proxy writes before the bulk reads
    __syncwarp();
}

template <int D, int NT, int NW, int SPW>
__global__ void __launch_bounds__(NW * 32, 1) pa_decode_fp4_kernel(const DecodeParams p, const int G) {
    using C = Fp4DecodeCfg<D, NT, NW, SPW>;
    constexpr int NB = C::NB, HS = C::HS, GMAX = C::GMAX;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 127) & ~uintptr_t(127));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    volatile int *flags = reinterpret_cast<volatile int *>(smem + C::OFF_FLAGS);  // [0] abort, [1] bad page
    float2 *merge_ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    float *merge_w = reinterpret_cast<float *>(smem + C::OFF_W);
    int32_t *page_tab = reinterpret_cast<int32_t *>(smem + C::OFF_PT);

    const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hq0 = kvh * G, hkv = gridDim.y;

    pdl_launch_dependents();
    if (threadIdx.x < NW * SPW) mbar_init(&full[threadIdx.x], 1);
    if (threadIdx.x == 0) {
        flags[0] = 0;
        flags[1] = 0;
    }
    if (threadIdx.x < NW * SPW) fence_mbar_init();
    // Every global access waits for the work before this call, except that
    // early_kv lets the block table, seq_lens and the chunks wholly before the
    // new row go first.
    if (!p.early_kv) pdl_wait_primary();

    int L = p.seq_lens[b];
    int c_begin = split * p.chunks_per_split;
    if (p.window > 0 && L > p.window && L <= p.max_seq_len) c_begin += (L - p.window) / kChunk;
    const int32_t *bt = p.block_table + (size_t)b * p.max_pages_per_seq;
    const int lp_first = (int)(((int64_t)c_begin * kChunk) / p.block_size);
    const int lp_last = min((int)(((int64_t)(c_begin + p.chunks_per_split) * kChunk - 1) / p.block_size), p.max_pages_per_seq - 1);
    const int n_pt = lp_last - lp_first + 1;
    const bool staged = n_pt <= kPageTab;
    if (staged)
        for (int j = threadIdx.x; j < n_pt; j += C::THREADS) page_tab[j] = bt[lp_first + j];
    if (L < 0 || L > p.max_seq_len) {
        if (threadIdx.x == 0 && split == 0 && kvh == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
        L = 0;
    }
    const int n_chunks = (L + kChunk - 1) / kChunk;
    const int n_my = min(n_chunks - c_begin, p.chunks_per_split);
    if (n_my <= 0) {
        // no key of this sequence in this split: the record says so (m = -inf,
        // l = 0); an unsplit call owns its output rows and zeroes them
        if (p.early_kv) pdl_wait_primary();
        if (p.num_splits == 1) {
            for (int idx = threadIdx.x; idx < G * D; idx += C::THREADS)
                store_out(p.out, ((size_t)b * p.num_q_heads + hq0) * D + idx, 0.f, p.out_bf16);
        } else if (threadIdx.x < G) {
            p.part_ml[((size_t)b * p.num_q_heads + hq0 + threadIdx.x) * p.num_splits + split] =
                make_float2(-INFINITY, 0.f);
        }
        return;
    }
    __syncthreads();  // barrier initialisation and the page table are visible to every thread

    // ---- this warp's chunks: warp, warp + NW, ... of the split ----
    const int n_w = (n_my - warp + NW - 1) / NW;  // (<= 0 for a warp without chunks)
    const uint64_t policy = l2_policy_evict_first();
    uint8_t *ring = smem + warp * SPW * C::STAGE_BYTES;
    uint64_t *bars = full + warp * SPW;
    const int chunks_per_page = p.block_size / kChunk;
    auto page_of = [&](int chunk, int &in_page) {
        const int lp = chunk / chunks_per_page;
        in_page = chunk - lp * chunks_per_page;
        return staged ? page_tab[lp - lp_first] : bt[lp];
    };
    auto issue = [&](int k) {  // the warp's k-th chunk into its stage k % SPW
        int in_page, page = page_of(c_begin + warp + k * NW, in_page);
        if (page < 0 || (int64_t)page >= p.num_pages) {
            flags[1] = 1;  // the outputs of this CTA are zeroed; page 0 is read in its place
            set_status(p.status, PA_DEV_BAD_PAGE);
            page = 0;
        }
        const size_t rec = (((size_t)page * hkv + kvh) * chunks_per_page + in_page) * C::REC;
        uint8_t *st = ring + (k % SPW) * C::STAGE_BYTES;
        uint64_t *bar = &bars[k % SPW];
        mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
        fp4::bulk_load(st, p.k_cache + rec, C::REC, bar, policy);
        fp4::bulk_load(st + C::REC, p.v_cache + rec, C::REC, bar, policy);
    };
    const int i_new = (L - 1) / kChunk - c_begin;  // the split-relative chunk of the new row
    bool first_done = false;                       // this lane's first stage is on its way
    if (p.early_kv) {
        if (lane < min(SPW, n_w) && warp + lane * NW < i_new) {
            issue(lane);
            first_done = true;
        }
        pdl_wait_primary();
    }
    if (p.k_new != nullptr && i_new < n_my && i_new >= 0 && warp == i_new % NW) {
        int in_page;
        const int page = page_of(c_begin + i_new, in_page);
        if (page >= 0 && (int64_t)page < p.num_pages)  // (a bad page is flagged when its chunk is copied)
            append_new_row_fp4<D>(p, b, kvh, L - 1, page);
    }
    if (!first_done && lane < min(SPW, n_w)) issue(lane);

    const int r = lane >> 2, c = lane & 3;
    float m_run[NT][2], l_run[NT][2];
    float oacc[NB][NT][4];
    // Q^T as B fragments, in f16: n-tile nt, k-step ks -> dims 16 ks + 4c (+1)
    // and 16 ks + 4c + 2 (+3) of head 8 nt + r
    uint32_t qf[NT][NB][2];
    float qsc[NT][2];  // multiplier of the raw scores of heads 8 nt + 2c + j (log2 units)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + r;
        const bool live = h < G;
        const __nv_bfloat16 *qrow = p.q + ((size_t)b * p.num_q_heads + hq0 + (live ? h : 0)) * D;
        uint2 w[NB];
        uint32_t amax = 0;
#pragma unroll
        for (int ks = 0; ks < NB; ++ks) {
            w[ks] = live ? *reinterpret_cast<const uint2 *>(qrow + 16 * ks + 4 * c) : make_uint2(0u, 0u);
            amax = max(amax, max(bf16x2_absmax(w[ks].x), bf16x2_absmax(w[ks].y)));
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const float qmul = f16_prescale(amax);
#pragma unroll
        for (int ks = 0; ks < NB; ++ks) {
            qf[nt][ks][0] = bf16x2_to_f16x2_scaled(w[ks].x, qmul);
            qf[nt][ks][1] = bf16x2_to_f16x2_scaled(w[ks].y, qmul);
        }
        const float mine = p.scale_log2 * p.k_scale[kvh] * (1.f / qmul);  // (1 / a power of two: exact)
        qsc[nt][0] = __shfl_sync(0xffffffffu, mine, 8 * c);
        qsc[nt][1] = __shfl_sync(0xffffffffu, mine, 8 * c + 4);
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < NB; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) oacc[mt][nt][i] = 0.f;
    }

    for (int k = 0; k < n_w; ++k) {
        const int s = k % SPW;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars[s], (k / SPW) & 1, &flags[0]))) {
            flags[0] = 1;
            set_status(p.status, PA_DEV_TIMEOUT);
            // giving up: let the copies in flight land before the CTA ends
            for (int kk = k; kk < min(k + SPW, n_w); ++kk)
                for (uint32_t n = 0; n < kWaitPollLimit && !mbar_try_wait(&bars[kk % SPW], (kk / SPW) & 1); ++n) {
                }
            break;
        }
        const uint8_t *kb = ring + s * C::STAGE_BYTES, *vb = kb + C::REC;
        const int t_chunk = (c_begin + warp + k * NW) * kChunk;
        const int nv = min(kChunk, L - t_chunk);  // visible rows [lead, nv)
        const int lead = p.window > 0 ? max(0, L - p.window - t_chunk) : 0;
        const bool partial = nv < kChunk || lead > 0;  // warp-uniform

        // ---- S^T = K Q^T, two accumulators per n-tile (even / odd k-steps) ----
        float sa[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q) sa[nt][u][q] = 0.f;
        uint32_t ksc[2][NB / 4];  // scale bytes of tokens r, r + 8
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t *sp = kb + 8 * D + (r + 8 * h) * NB;
            if constexpr (NB == 16) {
                const uint4 w = *reinterpret_cast<const uint4 *>(sp);
                ksc[h][0] = w.x; ksc[h][1] = w.y; ksc[h][2] = w.z; ksc[h][3] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(sp);
                ksc[h][0] = w.x; ksc[h][1] = w.y;
            }
        }
#pragma unroll
        for (int j = 0; j < NB / 8; ++j) {
            const uint4 k0 = *reinterpret_cast<const uint4 *>(kb + (2 * j) * 512 + lane * 16);
            const uint4 k1 = *reinterpret_cast<const uint4 *>(kb + (2 * j + 1) * 512 + lane * 16);
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // blocks 8 j + 2 q, + 1: one word of each token
                uint32_t a[4], e[4], s0[2], s1[2];
                fp4::e2m1x8_f16(w0[q], a);
                fp4::e2m1x8_f16(w1[q], e);
                const int blk = 8 * j + 2 * q;
                fp4::e4m3x4_f16(ksc[0][blk / 4], s0[0], s0[1]);
                fp4::e4m3x4_f16(ksc[1][blk / 4], s1[0], s1[1]);
                const uint32_t t0 = s0[q & 1], t1 = s1[q & 1];  // scales of blocks blk (low), blk + 1 (high)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mm::mma<true>(sa[nt][0], fp4::hmul2_lo(a[0], t0), fp4::hmul2_lo(e[0], t1), fp4::hmul2_lo(a[1], t0),
                                  fp4::hmul2_lo(e[1], t1), qf[nt][blk][0], qf[nt][blk][1]);
                    mm::mma<true>(sa[nt][1], fp4::hmul2_hi(a[2], t0), fp4::hmul2_hi(e[2], t1), fp4::hmul2_hi(a[3], t0),
                                  fp4::hmul2_hi(e[3], t1), qf[nt][blk + 1][0], qf[nt][blk + 1][1]);
                }
            }
        }

        // ---- online softmax on the fragments (log2 units) ----
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 4; ++q) x[nt][q] = (sa[nt][0][q] + sa[nt][1][q]) * qsc[nt][q & 1];
        if (partial) {
            const bool v0 = r >= lead && r < nv, v1 = r + 8 >= lead && r + 8 < nv;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (!v0) x[nt][0] = x[nt][1] = -INFINITY;
                if (!v1) x[nt][2] = x[nt][3] = -INFINITY;
            }
        }
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 4; ++q) up |= x[nt][q] > m_run[nt][q & 1] + kLazyLog2;
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float cm = fmaxf(x[nt][j], x[nt][j + 2]);
                    cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 4));
                    cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 8));
                    cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 16));
                    if (cm > m_run[nt][j] + kLazyLog2) {
                        const float alpha = fast_exp2(m_run[nt][j] - cm);  // 0 on the first chunk
                        m_run[nt][j] = cm;
                        l_run[nt][j] *= alpha;
#pragma unroll
                        for (int mt = 0; mt < NB; ++mt) {
                            oacc[mt][nt][j] *= alpha;
                            oacc[mt][nt][j + 2] *= alpha;
                        }
                    }
                }
        }
        // P^T fragments: head + residual, each transposed in registers
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float pr[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) pr[q] = fast_exp2(x[nt][q] - m_run[nt][q & 1]);  // 0 for masked rows
            l_run[nt][0] += pr[0] + pr[2];
            l_run[nt][1] += pr[1] + pr[3];
            uint32_t h01, h23, r01, r23;
            split_f16(pr[0], pr[1], h01, r01);
            split_f16(pr[2], pr[3], h23, r23);
            bh[nt][0] = mm::movt(h01);
            bh[nt][1] = mm::movt(h23);
            bl[nt][0] = mm::movt(r01);
            bl[nt][1] = mm::movt(r23);
        }

        // ---- O^T += V^T P^T ----
        uint32_t vw[4][NB / 4];  // codes of tokens 2c, 2c + 1, 8 + 2c, 9 + 2c: byte blk = dims 16 blk + 2r, + 1
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint8_t *vp = vb + u * 2 * D + lane * NB;
            if constexpr (NB == 16) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vp);
                vw[u][0] = w.x; vw[u][1] = w.y; vw[u][2] = w.z; vw[u][3] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(vp);
                vw[u][0] = w.x; vw[u][1] = w.y;
            }
        }
        // rows outside [lead, nv) may hold anything: their scales become 0
        // (the codes themselves are always finite)
        uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
        if (partial) {
            auto in = [&](int t) { return t >= lead && t < nv; };
            mlo = (in(2 * c) ? 0x0000ffffu : 0u) | (in(2 * c + 1) ? 0xffff0000u : 0u);
            mhi = (in(2 * c + 8) ? 0x0000ffffu : 0u) | (in(2 * c + 9) ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int w = 0; w < NB / 4; ++w) {
            const uint4 sc4 = *reinterpret_cast<const uint4 *>(vb + 8 * D + w * 64 + c * 16);
            const uint32_t sc[4] = {sc4.x, sc4.y, sc4.z, sc4.w};
            constexpr uint32_t LO = 0x0f0f0f0fu, HI = 0xf0f0f0f0u;
            uint32_t a0[4], a1[4], a2[4], a3[4];
            fp4::e2m1x8_f16((vw[0][w] & LO) | ((vw[1][w] << 4) & HI), a0);  // dims 16 blk + 2r, tokens 2c, 2c + 1
            fp4::e2m1x8_f16(((vw[0][w] >> 4) & LO) | (vw[1][w] & HI), a1);  // dims 16 blk + 2r + 1
            fp4::e2m1x8_f16((vw[2][w] & LO) | ((vw[3][w] << 4) & HI), a2);  // tokens 8 + 2c, 9 + 2c
            fp4::e2m1x8_f16(((vw[2][w] >> 4) & LO) | (vw[3][w] & HI), a3);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int mt = 4 * w + q;
                uint32_t slo, shi;
                fp4::e4m3x4_f16(sc[q], slo, shi);
                slo &= mlo;
                shi &= mhi;
                const uint32_t f0 = fp4::hmul2(a0[q], slo), f1 = fp4::hmul2(a1[q], slo);
                const uint32_t f2 = fp4::hmul2(a2[q], shi), f3 = fp4::hmul2(a3[q], shi);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mm::mma<true>(oacc[mt][nt], f0, f1, f2, f3, bh[nt][0], bh[nt][1]);
                    mm::mma<true>(oacc[mt][nt], f0, f1, f2, f3, bl[nt][0], bl[nt][1]);
                }
            }
        }
        __syncwarp();  // every lane has read the stage
        if (lane == 0 && k + SPW < n_w) issue(k + SPW);
    }
    // exponential sums: a lane holds tokens r and r + 8; sum over r
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float l = l_run[nt][j];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            l_run[nt][j] = l;
        }

    // ---- CTA merge of the warps' states (log-sum-exp weights) ----
    __syncthreads();  // every chunk is consumed: the stages become the merge area
    const bool poisoned = flags[0] != 0 || flags[1] != 0;
    float *macc = reinterpret_cast<float *>(smem);  // [NW][G][HS], unnormalised sums
#pragma unroll
    for (int mt = 0; mt < NB; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = nt * 8 + 2 * c + j;
                if (h < G)
                    *reinterpret_cast<float2 *>(macc + (warp * G + h) * HS + 16 * mt + 2 * r) =
                        make_float2(oacc[mt][nt][j], oacc[mt][nt][j + 2]);
            }
    if (r == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = nt * 8 + 2 * c + j;
                if (h < G) merge_ml[warp * GMAX + h] = make_float2(m_run[nt][j], l_run[nt][j]);
            }
    }
    __syncthreads();
    if (threadIdx.x < G) {
        const int h = threadIdx.x;
        float M = -INFINITY;
        for (int st = 0; st < NW; ++st) M = fmaxf(M, merge_ml[st * GMAX + h].x);
        float lsum = 0.f;
        for (int st = 0; st < NW; ++st) {
            const float2 ml = merge_ml[st * GMAX + h];
            const float e = ml.y != 0.f ? fast_exp2(ml.x - M) : 0.f;  // 0 for a warp without chunks
            merge_w[st * GMAX + h] = e;
            lsum = fmaf(ml.y, e, lsum);
        }
        const float norm = poisoned || lsum == 0.f ? 0.f : p.v_scale[kvh] / lsum;
        for (int st = 0; st < NW; ++st) merge_w[st * GMAX + h] *= norm;
        // a NaN sum (a NaN in a visible key or in q) goes on as a NaN output with
        // a weight of its own: the reduce takes a sum that is not > 0 for an empty split
        if (p.num_splits > 1)
            p.part_ml[((size_t)b * p.num_q_heads + hq0 + h) * p.num_splits + split] =
                make_float2(M, poisoned ? -1.f : lsum == lsum ? lsum : 1.f);
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < G * D / 4; idx += C::THREADS) {
        const int h = (4 * idx) / D, d = 4 * idx - h * D;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!poisoned) {  // (a bad page's stand-in may hold NaN)
#pragma unroll 4
            for (int st = 0; st < NW; ++st) {
                const float wg = merge_w[st * GMAX + h];
                const float4 v = *reinterpret_cast<const float4 *>(macc + (st * G + h) * HS + d);
                o.x = fmaf(v.x, wg, o.x);
                o.y = fmaf(v.y, wg, o.y);
                o.z = fmaf(v.z, wg, o.z);
                o.w = fmaf(v.w, wg, o.w);
            }
        }
        const size_t row = (size_t)b * p.num_q_heads + hq0 + h;
        if (p.num_splits == 1)
            store_out4(p.out, row * D + d, o, p.out_bf16);
        else
            *reinterpret_cast<float4 *>(p.part_o + (row * p.num_splits + split) * D + d) = o;
    }
}

}  // namespace pa
