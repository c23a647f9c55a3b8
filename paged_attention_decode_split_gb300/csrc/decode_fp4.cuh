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
// fewer than 32 bits is rounded below the sums' own error.  For bf16 outputs
// the residual is left out: a weight is off by half a step of f16, 2^-11 of
// itself, an eighth of the half step that the output is rounded by, and the
// errors of many keys average out.  (Multiplying the V scales to P, which is
// half as many multiplies, rounded a second time and lost small weights to
// f16's end where the scales are small, for 1 % of the time.)  Either way a
// weight is off by 2^-32 of the split's largest at most where it is smaller
// than 2^-21 of it.
//
// Layout on sm_103a:
//  * A chunk is two records (K, V) of 9 D contiguous bytes; a warp works on two
//    chunks (32 tokens) at a time.  Every warp owns a ring of SPW stages of one
//    chunk pair and fills it itself: lanes 2 s and 2 s + 1 issue the copies of K
//    and of V into stage s, up front and again whenever the warp has read it.
//    No producer warp and no empty barriers; the first NW * SPW pairs of a split
//    are in flight at once.  The chunks left after the last whole round of NW
//    pairs are spread over the warps one by one.
//  * Fragments come from shared memory by 16-byte loads at lane * 16 (the
//    record is laid out for them).  K: a lane's 16 bytes are the codes of one
//    token, dims 16 blk + 4 c .. + 3 of eight blocks; cvt widens a byte to a
//    pair, one multiply applies the block's scale (one scale per token and
//    k16 step).  V: 16 bytes are the codes of one token, dims 16 blk + 2 r, +1
//    of every block; the two tokens of a fragment register are interleaved
//    nibble by nibble (two bit selects per four bytes) before cvt, and one
//    multiply by the tokens' scale pair finishes it (one m16 tile is one scale
//    block).
//  * Q^T's fragments stand in shared memory, one 16-byte load per two k-steps,
//    used for both chunks; a pair's scales are widened to f16 once, into shared
//    memory (each is used by four lanes of K, by eight of V).
// What bounds the loop is the chain of dependent instructions with two warps per
// scheduler (8 x 20K-32K tokens: a warp issues every 4.3 clocks, 1.3 of them
// fixed latencies, 0.5 waits for shared memory and copies; 47 % of the issue
// slots and 44 % of the HBM's peak are used).  8 warps of 230 registers measured
// faster all the same than 10 or 12 of 168 (which spill) and than 16 of 128 whose
// pairs share the work on a chunk and exchange P (32 x 1K-32K batch, 24 heads on
// 4, D = 256: 143 us against 163, 150 and 151; 145 us, 4.3 TB/s of records, since
// the V scales meet V).  Outside the loop a CTA spends 5 us on its page table,
// first copies and merge, which bounds the short calls: 32K in one sequence takes
// 16.6 us, 512 tokens with the append 7.5 us, both with the reduce.
#pragma once

#include "decode_mma.cuh"
#include "fp4_cache.cuh"

namespace pa {

// What the fp4 decode needs beyond DecodeParams: the group and the division of
// a chunk index by the chunks of a page (a multiply by floor(2^32 / cpp), one
// correction step).
struct Fp4Params {
    int group;
    int chunks_per_page;
    uint32_t page_mul;
};

template <int D, int NT, int NW, int SPW>
struct Fp4DecodeCfg {
    static constexpr int REC = fp4::rec_bytes(D);
    static constexpr int STAGE_BYTES = 4 * REC;  // K records of a chunk pair, then its V records
    static constexpr int THREADS = NW * 32;
    static constexpr int NB = D / 16;            // scale blocks = k16 steps = m16 tiles of d
    static constexpr int GMAX = 8 * NT;
    static constexpr int HS = D + 4;             // merge row stride in floats (bank spread)
    static constexpr int RING_BYTES = NW * SPW * STAGE_BYTES;
    static constexpr int MERGE_BYTES = NW * GMAX * HS * 4;
    static constexpr int OFF_Q = RING_BYTES > MERGE_BYTES ? RING_BYTES : MERGE_BYTES;  // [NT][NB / 2][32] uint4
    static constexpr int OFF_QSC = OFF_Q + NT * NB / 2 * 512;  // [GMAX] score multipliers
    static constexpr int SC_BYTES = 2 * 2 * 16 * NB * 2;       // per warp: a pair's K, then V scales in f16
    static constexpr int OFF_SC = OFF_QSC + GMAX * 4;
    static constexpr int OFF_BAR = OFF_SC + NW * SC_BYTES;
    static constexpr int OFF_FLAGS = OFF_BAR + (NW * SPW + 1) * 8;  // full[NW * SPW], q_full
    static constexpr int OFF_ML = OFF_FLAGS + 16;           // [NW][GMAX] (m, l)
    static constexpr int OFF_PT = OFF_ML + NW * GMAX * 8;
    static constexpr int SMEM_BYTES = OFF_PT + kPageTab * 4 + 128;  // + slack to align the base
    static_assert(D == 128 || D == 256, "head_dim 128 or 256");
    static_assert(NT == 1 || NT == 2, "up to 16 heads per KV head");
    static_assert(SPW <= 32 && NT <= NW, "a lane per stage issues the first copies; a warp per n-tile lays Q out");
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

// NW warps, SPW stages per warp, RES: the P residual is multiplied too, PACK:
// up to 4 heads, whose heads' and residuals' weights share the 8 columns of one
// product (columns 4-7 repeat Q, and carry the residuals into P.V).
// FAR: the accumulators are moved to a second sum every kFp4FarPairs of a
// warp's pairs (splits that give a warp kFp4FarMin pairs or more, fp32 output).
constexpr int kFp4FarPairs = 8, kFp4FarMin = 12;
// SH: the own part of a decode over shared prefixes (decode_mma.cuh).
template <int D, int NT, int NW, int SPW, bool RES, bool PACK, bool FAR, bool SH = false>
__global__ void __launch_bounds__(NW * 32, 1) pa_decode_fp4_kernel(const DecodeParams p, const Fp4Params fp) {
    using C = Fp4DecodeCfg<D, NT, NW, SPW>;
    constexpr int NB = C::NB, HS = C::HS, GMAX = C::GMAX, REC = C::REC;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 127) & ~uintptr_t(127));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    volatile int *flags = reinterpret_cast<volatile int *>(smem + C::OFF_FLAGS);  // [0] abort, [1] bad page, [2] SH: no place in a group
    float2 *merge_ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    int32_t *page_tab = reinterpret_cast<int32_t *>(smem + C::OFF_PT);
    uint4 *q_frag = reinterpret_cast<uint4 *>(smem + C::OFF_Q);
    float *q_mul = reinterpret_cast<float *>(smem + C::OFF_QSC);

    // The reference max of a head is kept 2^7 below the largest score it was
    // raised for, and raised again when a score passes it by kRaise: P in f16, at
    // most 2^15, holds weights down to 2^-32 of the largest (f16 ends at 2^-25).
    constexpr float kBelow = 7.f, kRaise = kLazyLog2 + kBelow;

    const int split = blockIdx.x, kvh = blockIdx.y;
    int b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = fp.group, hq0 = kvh * G, hkv = gridDim.y;
    [[maybe_unused]] const bool last_cta = split == (int)gridDim.x - 1 && kvh == hkv - 1 && b == (int)gridDim.z - 1;

    pdl_launch_dependents();
    uint64_t *q_full = full + NW * SPW;
    if (threadIdx.x <= NW * SPW) {
        mbar_init(&full[threadIdx.x], threadIdx.x < NW * SPW ? 1 : NT);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        flags[0] = 0;
        flags[1] = 0;
        flags[2] = 0;
    }
    // Every global access waits for the work before this call, except that
    // early_kv lets the block table, seq_lens and the chunks wholly before the
    // new row go first.
    if (SH ? p.prefix_splits == 0 : !p.early_kv) pdl_wait_primary();
    if constexpr (SH) b = sequence_of(p, b);

    // Q^T as B fragments, in f16: n-tile nt, k-step ks -> dims 16 ks + 4c (+1)
    // and 16 ks + 4c + 2 (+3) of head 8 nt + r; warp nt lays its tile out.  Its
    // loads go out first: behind the CTAs' copies they took 3 us to come back.
    const int r = lane >> 2, c = lane & 3;
    uint2 qw[NB];
    float k_scale, v_scale;
    auto load_q = [&]() {
        k_scale = p.k_scale[kvh];
        v_scale = p.v_scale[kvh];
        if (warp < NT) {
            const int h = warp * 8 + (PACK ? r & 3 : r);
            const __nv_bfloat16 *qrow = p.q + ((size_t)b * p.num_q_heads + hq0 + (h < G ? h : 0)) * D;
#pragma unroll
            for (int ks = 0; ks < NB; ++ks) qw[ks] = *reinterpret_cast<const uint2 *>(qrow + 16 * ks + 4 * c);
        }
    };
    if (!p.early_kv) load_q();

    int L = p.seq_lens[b];
    const int record = SH ? p.prefix_splits + split : split;  // of the row's num_splits
    int cps = p.chunks_per_split;
    int c_begin = split * cps;
    [[maybe_unused]] bool own_ok = true;  // SH: the lengths make sense, and a prefix CTA has this sequence
    if constexpr (SH) {
        const bool len_ok = L >= 0 && L <= p.max_seq_len;  // (flagged below)
        const Suffix x = suffix_of(p, b, len_ok ? L : 0);
        own_ok = len_ok && x.ok;
        // (no further than the sequence: the plan's splits may, for all of max_seq_len, reach past 2^31 tokens)
        c_begin = min(x.first + split * x.per, x.end);
        cps = min(x.per, x.end - c_begin);
    }
    if (!SH && p.window > 0) {  // (a branch: without a window the table's loads do not wait for the length)
        if (L > p.window && L <= p.max_seq_len) c_begin += (L - p.window) / kChunk;
    }
    auto page_of_chunk = [&](int chunk, int &in_page) {
        int lp = (int)__umulhi((uint32_t)chunk, fp.page_mul);
        in_page = chunk - lp * fp.chunks_per_page;
        if (in_page >= fp.chunks_per_page) {
            in_page -= fp.chunks_per_page;
            ++lp;
        }
        return lp;
    };
    const int32_t *bt = p.block_table + (size_t)b * p.max_pages_per_seq;
    int unused;
    const int lp_first = page_of_chunk(c_begin, unused);
    const int c_last = SH ? max(c_begin + cps, 1) - 1 : c_begin + cps - 1;  // (SH: an idle sequence has no chunk)
    const int lp_last = min(page_of_chunk(c_last, unused), p.max_pages_per_seq - 1);
    const int n_pt = lp_last - lp_first + 1;
    const bool staged = n_pt <= kPageTab;
    if (staged)
        for (int j = threadIdx.x; j < n_pt; j += C::THREADS) page_tab[j] = bt[lp_first + j];
    if (L < 0 || L > p.max_seq_len) {
        if (threadIdx.x == 0 && split == 0 && kvh == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
        L = 0;
    }
    const int n_chunks = (L + kChunk - 1) / kChunk;
    int n_my = min(n_chunks - c_begin, cps);
    if constexpr (SH) {
        if (!own_ok) {
            n_my = 0;
            if (threadIdx.x == 0 && split == 0 && kvh == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
        }
        if (n_my <= 0 && split == 0 && warp == 0 && !group_ok(p, b, L, hq0, G, kvh == 0)) own_ok = false;
    }
    if (n_my <= 0) {
        // no key of this sequence in this split: the record says so (m = -inf,
        // l = 0); an unsplit call owns its output rows and zeroes them
        if constexpr (SH) wait_prefix(last_cta);
        if (p.early_kv) pdl_wait_primary();
        if (p.num_splits == 1) {
            for (int idx = threadIdx.x; idx < G * D; idx += C::THREADS)
                store_out(p.out, ((size_t)b * p.num_q_heads + hq0) * D + idx, 0.f, p.out_bf16);
        } else if (threadIdx.x < G) {
            p.part_ml[((size_t)b * p.num_q_heads + hq0 + threadIdx.x) * p.num_splits + record] =
                make_float2(-INFINITY, own_ok ? 0.f : -1.f);
        }
        return;
    }
    __syncthreads();  // barrier initialisation and the page table are visible to every thread

    // ---- this warp's chunks: pairs warp, warp + NW, ... of the whole rounds, then its share of the rest ----
    const int rounds = n_my / (2 * NW), rest = n_my - rounds * 2 * NW;
    const int twos = max(0, rest - NW);  // warps that take two chunks of the rest
    const int n_w = rounds + (warp < rest ? 1 : 0);
    auto item = [&](int k, bool &two) {  // the split-relative first chunk of the warp's k-th item
        two = k < rounds || warp < twos;
        return k < rounds ? 2 * (warp + k * NW) : 2 * NW * rounds + warp + min(warp, twos);
    };
    const uint64_t policy = l2_policy_evict_first();
    uint8_t *ring = smem + warp * SPW * C::STAGE_BYTES;
    uint8_t *scales = smem + C::OFF_SC + warp * C::SC_BYTES;  // f16, in the order of the records' scale bytes
    uint64_t *bars = full + warp * SPW;
    // Byte offset of a chunk's record in either cache.
    auto record_of = [&](int chunk, int &in_page) {
        const int lp = page_of_chunk(chunk, in_page);
        int page = staged ? page_tab[lp - lp_first] : bt[lp];
        if (page < 0 || (int64_t)page >= p.num_pages) {
            flags[1] = 1;  // the outputs of this CTA are zeroed; page 0 is read in its place
            set_status(p.status, PA_DEV_BAD_PAGE);
            page = 0;
        }
        return (((size_t)page * hkv + kvh) * fp.chunks_per_page + in_page) * REC;
    };
    // Lane 2 s + tensor issues the copies of one tensor into stage s (two copies
    // by one lane took 0.3 us).  The bytes may land before the other lane's
    // expect_tx: the phase cannot end before that lane's arrival.
    const int tensor = lane & 1;
    uint8_t *my_stage = ring + (lane >> 1) * C::STAGE_BYTES + tensor * 2 * REC;
    uint64_t *my_bar = &bars[lane >> 1];
    const uint8_t *my_cache = tensor == 0 ? p.k_cache : p.v_cache;
    auto issue = [&](int k) {  // the warp's k-th item into the lane's stage
        bool two;
        const int i = item(k, two);
        int in_page;
        const size_t rec = record_of(c_begin + i, in_page);
        if (tensor == 0) mbar_arrive_expect_tx(my_bar, two ? 4 * REC : 2 * REC);
        const bool joined = two && in_page + 1 < fp.chunks_per_page;  // one run of the page
        fp4::bulk_load(my_stage, my_cache + rec, joined ? 2 * REC : REC, my_bar, policy);
        if (two && !joined) {
            const size_t rec2 = record_of(c_begin + i + 1, in_page);
            fp4::bulk_load(my_stage + REC, my_cache + rec2, REC, my_bar, policy);
        }
    };
    const int i_new = (L - 1) / kChunk - c_begin;  // the split-relative chunk of the new row
    // the warp whose items hold the new row's chunk
    const int j_new = i_new - 2 * NW * rounds;
    const int w_new = j_new < 0 ? (i_new >> 1) % NW : j_new < 2 * twos ? j_new >> 1 : j_new - twos;
    // The first copies go out stage by stage, not warp by warp: the copy engine
    // works them off in order, so the first pairs land while the later ones are
    // still on their way (32K call: 19.7 us with all stages of a warp at once).
    const bool my_first = lane < 2 * min(SPW, n_w);  // the lane has a first copy to issue
    bool issued = false;
    if (p.early_kv) {
        bool two;
        const int i = item(lane >> 1, two);
        if (my_first && i + (two ? 1 : 0) < i_new) {
            issue(lane >> 1);
            issued = true;
        }
        pdl_wait_primary();
        load_q();
    } else if (my_first && lane < 2 && (p.k_new == nullptr || n_w > 1 || warp != w_new)) {
        issue(0);
        issued = true;
    }
    if (warp < NT) {
        if (warp * 8 + (PACK ? r & 3 : r) >= G) {  // heads past the group
#pragma unroll
            for (int ks = 0; ks < NB; ++ks) qw[ks] = make_uint2(0u, 0u);
        }
        uint32_t amax = 0;
#pragma unroll
        for (int ks = 0; ks < NB; ++ks) amax = max(amax, max(bf16x2_absmax(qw[ks].x), bf16x2_absmax(qw[ks].y)));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const float mul = f16_prescale(amax);
#pragma unroll
        for (int ks = 0; ks < NB; ks += 2)
            q_frag[(warp * (NB / 2) + ks / 2) * 32 + lane] =
                make_uint4(bf16x2_to_f16x2_scaled(qw[ks].x, mul), bf16x2_to_f16x2_scaled(qw[ks].y, mul),
                           bf16x2_to_f16x2_scaled(qw[ks + 1].x, mul), bf16x2_to_f16x2_scaled(qw[ks + 1].y, mul));
        if (c == 0) q_mul[8 * warp + r] = p.scale_log2 * k_scale * (1.f / mul);  // (1 / a power of two: exact)
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
    }
    if (p.k_new != nullptr && i_new < n_my && i_new >= 0 && warp == w_new) {
        int in_page;
        const int lp = page_of_chunk(c_begin + i_new, in_page);
        const int page = staged ? page_tab[lp - lp_first] : bt[lp];
        if (page >= 0 && (int64_t)page < p.num_pages)  // (a bad page is flagged when its chunk is copied)
            append_new_row_fp4<D>(p, b, kvh, L - 1, page);
    }
    if (my_first && !issued) issue(lane >> 1);

    if constexpr (SH) {
        if (split == 0 && warp == NW - 1 && !group_ok(p, b, L, hq0, G, kvh == 0) && lane == 0) flags[2] = 1;
    }
    // (an mbarrier rather than a CTA barrier: a warp whose copies the copy engine has yet to take holds no other up)
    bool ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0, &flags[0]));
    if (!ok) flags[0] = 1;
    float m_run[NT][2], l_run[NT][2];
    float oacc[NB][NT][4];
    float qsc[NT][2];  // multiplier of the raw scores of heads 8 nt + 2c + j (log2 units)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        qsc[nt][0] = q_mul[8 * nt + 2 * c];
        qsc[nt][1] = q_mul[8 * nt + 2 * c + 1];
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < NB; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) oacc[mt][nt][i] = 0.f;
    }

    // The tensor core cuts each addition to an accumulator off towards zero: the
    // accumulators lose 2.4e-9 of themselves per key.  FAR moves them to a sum in
    // local memory every kFar pairs (256 keys: 6e-7), unless fewer than half as
    // many follow.  A kernel of its own: it costs the other one 0.5 us of 16.5.
    constexpr int kFar = kFp4FarPairs;
    static_assert(!FAR || (RES && !PACK), "a second sum of O: fp32 output");
    [[maybe_unused]] volatile float o_far[FAR ? NB * NT * 4 : 1];  // (volatile: kept out of the registers)
    [[maybe_unused]] volatile float m_far[FAR ? NT * 2 : 1];       // the reference maxima that o_far stands for
    auto far_weight = [&](int nt, int j) { return fast_exp2(m_far[2 * nt + j] - m_run[nt][j]); };

    int s = 0;
    uint32_t phase = 0;
    const int t_rest = (c_begin + 2 * NW * rounds + warp + min(warp, twos)) * kChunk;
    for (int k = 0, t_round = (c_begin + 2 * warp) * kChunk; k < n_w; ++k, t_round += 2 * NW * kChunk) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars[s], phase, &flags[0]));
        if (!ok) {
            flags[0] = 1;
            set_status(p.status, PA_DEV_TIMEOUT);
            // giving up: let the copies in flight land before the CTA ends
            for (int kk = k; kk < min(k + SPW, n_w); ++kk)
                for (uint32_t n = 0; n < kWaitPollLimit && !mbar_try_wait(&bars[kk % SPW], (kk / SPW) & 1); ++n) {
                }
            break;
        }
        const uint8_t *kb = ring + s * C::STAGE_BYTES, *vb = kb + 2 * REC;
        const int t_pair = k < rounds ? t_round : t_rest;
        // visible tokens [lead, nv) of the pair (the second half of a single chunk's stage holds stale bytes)
        const bool two = k < rounds || warp < twos;
        const int nv = min((two ? 2 : 1) * kChunk, L - t_pair);
        const int lead = !SH && p.window > 0 ? max(0, L - p.window - t_pair) : 0;
        const bool partial = nv < 2 * kChunk || lead > 0;  // warp-uniform

        // ---- the pair's scales to f16, once (each is used by 4 lanes of K, by 8 of V) ----
        if (lane < 2 * NB) {
            const int ch = lane / NB, part = (lane % NB) * 16;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint4 w = *reinterpret_cast<const uint4 *>((t == 0 ? kb : vb) + ch * REC + 8 * D + part);
                uint4 lo, hi;
                fp4::e4m3x4_f16(w.x, lo.x, lo.y);
                fp4::e4m3x4_f16(w.y, lo.z, lo.w);
                fp4::e4m3x4_f16(w.z, hi.x, hi.y);
                fp4::e4m3x4_f16(w.w, hi.z, hi.w);
                uint4 *dst = reinterpret_cast<uint4 *>(scales + t * (C::SC_BYTES / 2) + (ch * 16 * NB + part) * 2);
                dst[0] = lo;
                dst[1] = hi;
            }
        }
        __syncwarp();
        const uint8_t *ksc = scales, *vsc = scales + C::SC_BYTES / 2;

        // ---- S^T = K Q^T per chunk, two accumulators per n-tile (even / odd k-steps) ----
        // x: log2 units, [chunk][n-tile][tokens r, r + 8][heads 2c, 2c + 1]
        float x[2][NT][4];
        auto scores = [&](auto chunks) {
            constexpr int NCH = decltype(chunks)::value;
            float sa[NCH][NT][2][4];
#pragma unroll
            for (int j = 0; j < NB / 8; ++j) {
                uint32_t kw[NCH][2][4], ks[NCH][2][4];  // [chunk][token r, r + 8]: codes and scale pairs of blocks 8 j .. + 7
#pragma unroll
                for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t *rec = kb + ch * REC;
                        const uint4 w = *reinterpret_cast<const uint4 *>(rec + (2 * j + h) * 512 + lane * 16);
                        const uint4 sw = *reinterpret_cast<const uint4 *>(ksc + ((ch * 16 + r + 8 * h) * NB + 8 * j) * 2);
                        kw[ch][h][0] = w.x; kw[ch][h][1] = w.y; kw[ch][h][2] = w.z; kw[ch][h][3] = w.w;
                        ks[ch][h][0] = sw.x; ks[ch][h][1] = sw.y; ks[ch][h][2] = sw.z; ks[ch][h][3] = sw.w;
                    }
#pragma unroll
                for (int q = 0; q < 4; ++q) {  // blocks 8 j + 2 q, + 1: one word of each token
                    uint4 qf[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) qf[nt] = q_frag[(nt * (NB / 2) + 4 * j + q) * 32 + lane];
#pragma unroll
                    for (int ch = 0; ch < NCH; ++ch) {
                        uint32_t a[4], e[4];
                        fp4::e2m1x8_f16(kw[ch][0][q], a);
                        fp4::e2m1x8_f16(kw[ch][1][q], e);
                        const uint32_t t0 = ks[ch][0][q], t1 = ks[ch][1][q];  // scales of the even (low) and odd block
                        const uint32_t a0 = fp4::hmul2_lo(a[0], t0), a1 = fp4::hmul2_lo(a[1], t0);
                        const uint32_t a2 = fp4::hmul2_hi(a[2], t0), a3 = fp4::hmul2_hi(a[3], t0);
                        const uint32_t e0 = fp4::hmul2_lo(e[0], t1), e1 = fp4::hmul2_lo(e[1], t1);
                        const uint32_t e2 = fp4::hmul2_hi(e[2], t1), e3 = fp4::hmul2_hi(e[3], t1);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (j == 0 && q == 0) {
                                fp4::mma0_f16(sa[ch][nt][0], a0, e0, a1, e1, qf[nt].x, qf[nt].y);
                                fp4::mma0_f16(sa[ch][nt][1], a2, e2, a3, e3, qf[nt].z, qf[nt].w);
                            } else {
                                mm::mma<true>(sa[ch][nt][0], a0, e0, a1, e1, qf[nt].x, qf[nt].y);
                                mm::mma<true>(sa[ch][nt][1], a2, e2, a3, e3, qf[nt].z, qf[nt].w);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        x[ch][nt][q] = ch < NCH ? (sa[ch < NCH ? ch : 0][nt][0][q] + sa[ch < NCH ? ch : 0][nt][1][q]) * qsc[nt][q & 1]
                                                : -INFINITY;
        };
        if (two)
            scores(std::integral_constant<int, 2>{});
        else
            scores(std::integral_constant<int, 1>{});

        // ---- online softmax on the fragments ----
        if (partial) {
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                const int t0 = 16 * ch + r, t1 = t0 + 8;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (t0 < lead || t0 >= nv) x[ch][nt][0] = x[ch][nt][1] = -INFINITY;
                    if (t1 < lead || t1 >= nv) x[ch][nt][2] = x[ch][nt][3] = -INFINITY;
                }
            }
        }
        float cm[NT][2];  // the lane's largest score per head
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                cm[nt][j] = fmaxf(fmax3(x[0][nt][j], x[0][nt][j + 2], x[1][nt][j]), x[1][nt][j + 2]);
                up |= cm[nt][j] > m_run[nt][j] + kRaise;
            }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float m = cm[nt][j];
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    if (m > m_run[nt][j] + kRaise) {
                        m -= kBelow;
                        const float alpha = fast_exp2(m_run[nt][j] - m);  // 0 on the first pair
                        m_run[nt][j] = m;
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
        uint32_t bh[2][NT][2];
        [[maybe_unused]] uint32_t bl[2][NT][2];
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float pr[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) pr[q] = fast_exp2(x[ch][nt][q] - m_run[nt][q & 1]);  // 0 for masked rows
                l_run[nt][0] += pr[0] + pr[2];
                l_run[nt][1] += pr[1] + pr[3];
                uint32_t h01, h23, r01, r23;
                if constexpr (RES) {
                    split_f16(pr[0], pr[1], h01, r01);
                    split_f16(pr[2], pr[3], h23, r23);
                    if constexpr (PACK) {
                        h01 = c < 2 ? h01 : r01;
                        h23 = c < 2 ? h23 : r23;
                    } else {
                        bl[ch][nt][0] = mm::movt(r01);
                        bl[ch][nt][1] = mm::movt(r23);
                    }
                } else {
                    h01 = pack_f16(pr[0], pr[1]);
                    h23 = pack_f16(pr[2], pr[3]);
                }
                bh[ch][nt][0] = mm::movt(h01);
                bh[ch][nt][1] = mm::movt(h23);
            }

        // ---- O^T += V^T P^T ----
        // Tokens outside [lead, nv) may hold anything: in a partial pair their
        // scales become 0 (the codes themselves are always finite).
        auto pv = [&](auto masked) {
            constexpr bool MASK = decltype(masked)::value;
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                if (MASK && ch == 1 && !two) break;
                const uint8_t *rec = vb + ch * REC;
                uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
                if constexpr (MASK) {
                    auto in = [&](int t) { return 16 * ch + t >= lead && 16 * ch + t < nv; };
                    mlo = (in(2 * c) ? 0x0000ffffu : 0u) | (in(2 * c + 1) ? 0xffff0000u : 0u);
                    mhi = (in(2 * c + 8) ? 0x0000ffffu : 0u) | (in(2 * c + 9) ? 0xffff0000u : 0u);
                }
                uint32_t vw[4][NB / 4];  // codes of tokens 2c, 2c + 1, 8 + 2c, 9 + 2c: byte blk = dims 16 blk + 2r, + 1
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint8_t *vp = rec + u * 2 * D + lane * NB;
                    if constexpr (NB == 16) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(vp);
                        vw[u][0] = w.x; vw[u][1] = w.y; vw[u][2] = w.z; vw[u][3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2 *>(vp);
                        vw[u][0] = w.x; vw[u][1] = w.y;
                    }
                }
#pragma unroll
                for (int w = 0; w < NB / 4; ++w) {
                    const uint4 *sp = reinterpret_cast<const uint4 *>(vsc + ((ch * 16 * NB) + w * 64 + c * 16) * 2);
                    const uint4 sA = sp[0], sB = sp[1];  // per block: scales of tokens 2c, 2c + 1 and 8 + 2c, 9 + 2c
                    uint32_t slo[4] = {sA.x, sA.z, sB.x, sB.z}, shi[4] = {sA.y, sA.w, sB.y, sB.w};
                    if constexpr (MASK) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            slo[q] &= mlo;
                            shi[q] &= mhi;
                        }
                    }
                    constexpr uint32_t LO = 0x0f0f0f0fu, HI = 0xf0f0f0f0u;
                    uint32_t a0[4], a1[4], a2[4], a3[4];
                    fp4::e2m1x8_f16((vw[0][w] & LO) | ((vw[1][w] << 4) & HI), a0);  // dims 16 blk + 2r, tokens 2c, 2c + 1
                    fp4::e2m1x8_f16(((vw[0][w] >> 4) & LO) | (vw[1][w] & HI), a1);  // dims 16 blk + 2r + 1
                    fp4::e2m1x8_f16((vw[2][w] & LO) | ((vw[3][w] << 4) & HI), a2);  // tokens 8 + 2c, 9 + 2c
                    fp4::e2m1x8_f16(((vw[2][w] >> 4) & LO) | (vw[3][w] & HI), a3);
                    // V = code * S (exact); four tiles' heads, then their residuals: no product waits for
                    // the one before it
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        a0[q] = fp4::hmul2(a0[q], slo[q]);
                        a1[q] = fp4::hmul2(a1[q], slo[q]);
                        a2[q] = fp4::hmul2(a2[q], shi[q]);
                        a3[q] = fp4::hmul2(a3[q], shi[q]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            mm::mma<true>(oacc[4 * w + q][nt], a0[q], a1[q], a2[q], a3[q], bh[ch][nt][0], bh[ch][nt][1]);
                        if constexpr (RES && !PACK) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                mm::mma<true>(oacc[4 * w + q][nt], a0[q], a1[q], a2[q], a3[q], bl[ch][nt][0],
                                              bl[ch][nt][1]);
                        }
                    }
                }
            }
        };
        if (partial)
            pv(std::true_type{});
        else
            pv(std::false_type{});
        __syncwarp();  // every lane has read the stage
        if (lane >> 1 == s && k + SPW < n_w) issue(k + SPW);
        if (++s == SPW) {
            s = 0;
            phase ^= 1;
        }
        if constexpr (FAR) {
            if (k % kFar == kFar - 1 && n_w - k > kFp4FarMin - kFar) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float w = k < kFar ? 0.f : far_weight(nt, j);
#pragma unroll
                        for (int mt = 0; mt < NB; ++mt)
#pragma unroll
                            for (int h = 0; h < 4; h += 2) {
                                volatile float &far = o_far[(mt * NT + nt) * 4 + j + h];
                                far = k < kFar ? oacc[mt][nt][j + h] : fmaf(far, w, oacc[mt][nt][j + h]);
                                oacc[mt][nt][j + h] = 0.f;
                            }
                        m_far[2 * nt + j] = m_run[nt][j];
                    }
            }
        }
    }
    if constexpr (FAR) {
        if (n_w >= kFp4FarMin && ok) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float w = far_weight(nt, j);
#pragma unroll
                    for (int mt = 0; mt < NB; ++mt)
#pragma unroll
                        for (int h = 0; h < 4; h += 2)
                            oacc[mt][nt][j + h] = fmaf(o_far[(mt * NT + nt) * 4 + j + h], w, oacc[mt][nt][j + h]);
                }
        }
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

    if constexpr (PACK) {  // head and residual columns of a head: lanes c and c + 2
        static_assert(RES && NT == 1, "packed residuals");
#pragma unroll
        for (int mt = 0; mt < NB; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) oacc[mt][0][i] += __shfl_xor_sync(0xffffffffu, oacc[mt][0][i], 2);
    }

    // ---- CTA merge of the warps' states (log-sum-exp weights) ----
    // Every warp sees all warps' (m, l), scales its own sums by its weight over
    // the total and writes them; the outputs are then plain sums over the warps.
    if (r == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                merge_ml[warp * GMAX + nt * 8 + 2 * c + j] = make_float2(m_run[nt][j], l_run[nt][j]);
    }
    __syncthreads();  // every chunk is consumed: the stages become the merge area
    const bool poisoned = flags[0] != 0 || flags[1] != 0 || (SH && flags[2] != 0);
    const int n_act = min(NW, n_my);  // warps that had a chunk
    float *macc = reinterpret_cast<float *>(smem);  // [NW][G][HS]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = nt * 8 + 2 * c + j;
            float2 ml[NW];
            float M = -INFINITY, lsum = 0.f;
#pragma unroll
            for (int st = 0; st < NW; ++st) ml[st] = merge_ml[st * GMAX + h];
#pragma unroll
            for (int st = 0; st < NW; ++st) M = fmaxf(M, ml[st].x);
#pragma unroll
            for (int st = 0; st < NW; ++st)  // (a warp without chunks has l = 0)
                lsum = fmaf(ml[st].y, ml[st].y != 0.f ? fast_exp2(ml[st].x - M) : 0.f, lsum);
            const float fac = l_run[nt][j] != 0.f && lsum != 0.f ? fast_exp2(m_run[nt][j] - M) * (v_scale / lsum) : 0.f;
            if (h < G && warp < n_act) {
                // a NaN sum (a NaN in a visible key or in q) goes on as a NaN output with a
                // record of its own, max 0 and sum 1: the reduce takes a sum that is not > 0
                // for an empty split, and the max of such a split may be infinite
                if (warp == 0 && r == 0 && p.num_splits > 1)
                    p.part_ml[((size_t)b * p.num_q_heads + hq0 + h) * p.num_splits + record] =
                        poisoned ? make_float2(M, -1.f) : lsum == lsum ? make_float2(M, lsum) : make_float2(0.f, 1.f);
                float *row = macc + (warp * G + h) * HS + 2 * r;
#pragma unroll
                for (int mt = 0; mt < NB; ++mt)
                    *reinterpret_cast<float2 *>(row + 16 * mt) =
                        make_float2(oacc[mt][nt][j] * fac, oacc[mt][nt][j + 2] * fac);
            }
        }
    __syncthreads();
    for (int idx = threadIdx.x; idx < G * D / 4; idx += C::THREADS) {
        const int h = (4 * idx) / D, d = 4 * idx - h * D;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!poisoned) {  // (a bad page's stand-in may hold NaN)
#pragma unroll 4
            for (int st = 0; st < n_act; ++st) {
                const float4 v = *reinterpret_cast<const float4 *>(macc + (st * G + h) * HS + d);
                o.x += v.x;
                o.y += v.y;
                o.z += v.z;
                o.w += v.w;
            }
        }
        const size_t row = (size_t)b * p.num_q_heads + hq0 + h;
        if (p.num_splits == 1)
            store_out4(p.out, row * D + d, o, p.out_bf16);
        else
            *reinterpret_cast<float4 *>(p.part_o + (row * p.num_splits + record) * D + d) = o;
    }
    if constexpr (SH) wait_prefix(last_cta);
}

}  // namespace pa
