// verify_tc.cuh -- multi-row (speculative verify) paged attention on the
// sm_100-family tensor cores: tcgen05 MMAs with accumulators in tensor memory.
//
// What it computes ("Qwen3.8 on MI350P", Lektion 3: verify rows share K/V
// tiles, a causal mask applies per row, partial softmax statistics merge;
// "DCU page832 attention", Sec.5/7 for the paged walk): for the q_len new rows
// of a sequence, row r attends to keys 0 .. L - q_len + r.  All G * q_len query
// rows of one KV head form one M = 128 MMA block (row rho = r * G + g; rows
// past G * q_len are zero padding), so each K/V chunk is read from HBM once
// per CTA and consumed once by the tensor core for all rows.  The context is
// split across CTAs like decode; the same partition reduce merges the splits.
//
// Per 64-token tile i (four 16-token TMA chunks landing side by side):
//   S_i = Q K_i^T     M=128, N=64, K=D: D/16 MMAs with A = Q read from tensor
//                     memory, into one of two tensor-memory S buffers (tile
//                     i+1's scores are formed while the softmax warps work on
//                     tile i)
//   softmax           4 warps, one query row per thread (tensor-memory lane =
//                     row): scale, causal mask, running max and sum, P = 2^(s-m),
//                     written back over S_i in tensor memory
//   O += P_i V_i      M=128, N=D, K=16 per step (4 steps), A = P_i from tensor
//                     memory, carried as a bf16 head plus a bf16 residual (two
//                     MMAs) so it keeps ~16 significant bits
// The running max used for the exponentials is only raised when the row's
// max grows by more than 2^8 (then O and l are rescaled in place, after the
// previous tile's P.V product); otherwise P may exceed 1 by at most 2^8, which
// fp32 and the bf16 pair hold exactly enough, and the final division by l uses
// the same reference max.  Because O is touched only then, the softmax of tile
// i+1 overlaps the P.V product of tile i.
//
// Tensor memory (512 columns x 128 lanes): O fp32 in columns [0, D), NSB = 2
// S/P buffers of 64 columns from D on, and Q as bf16 pairs after them.
// Shared memory holds the K and V tiles in two rings (4 K and 3 V slots of
// 32 KiB for D = 256) and the split's block-table entries; a K slot is
// refilled once S_i is done:
//   K_i [D/64 blocks][64 tokens][128 B], 128-byte swizzle, K-major: one 5-D TMA
//       box of 64 tokens when the tile lies in one page, else 64-dim x 16-token
//       boxes per chunk
//   V_i same layout as K_i, read as the MN-major (N = d) B operand
// Warp roles: 0-3 softmax, 4 MMA issue (and tensor-memory allocation), 5 TMA
// (lane 0 decides, the whole warp issues a tile's boxes).
//
// fp8 e4m3 cache (NSG > 0): the copies land e4m3 tiles as [D/128 blocks][64
// tokens][128 B] with the 128-byte swizzle in a staging ring of NSG slots per
// tensor (so 8 lanes reading one 16-byte column of 8 consecutive tokens hit 8
// different bank groups), and four more warps
// widen them (warps 6-7: K, 8-9: V) into the same swizzled K/V rings as f16
// -- exact, since every e4m3 value is an f16 value -- zeroing rows past the
// tile's last key.  Q and P then enter the products as f16 (kind::f16 with
// f16 A and B), the K scale joins the softmax scale and the V scale the final
// normaliser.  A q row enters scaled by a power of two that brings its
// largest element into [2^14, 2^15), so any finite bf16 q fits f16; the
// inverse power joins the softmax scale.
//
// fp4 cache (F4; fp4_cache.cuh): as over an e4m3 cache, but the staging slots
// hold the tile's four records per tensor, copied by untiled bulk copies (one
// per run of chunks in a page) that a warp per tensor issues (5: K, 6: V), and
// sixteen warps (8-15: K, 16-23: V; half a record each) apply each 16-dim
// block's scale: code * S in f16 (exact).  At the start they fetch and convert
// Q.  The softmax warps take registers from the others (setmaxnreg).  The dims of a row are left in an order that
// makes every ring write a whole 16-byte chunk of what one lane holds: K chunk
// 4 g + c holds dims 4 c .. 4 c + 3 of blocks 2 g and 2 g + 1 (Q is stored in
// the same order, a renaming of registers), V chunk 8 w + r of a row holds dims
// 2 r, 2 r + 1 of blocks 4 w .. 4 w + 3 (so O's columns stand in that order,
// undone by a renaming of registers in the epilogue).  bf16 outputs leave the
// residual of P out; fp32 outputs of long splits keep a second sum (FAR).
// What bounds it: shared memory.  A tile of 64 keys is 64 KiB widened and
// written, 64 KiB (96 with the residual) read by the tensor core and 18 KiB
// copied and read, 1450 (1700) clocks of its 128 bytes per clock and more with
// scales and barriers, at a tile time of 1750 (2250); the products take 1030
// (1540), the issue slots are two thirds full.  2048 rows over 16K (24 heads on
// 4, D = 256): 701 us; 32 x 5 rows over 700-2048 (48 on 4): 38 us.  With 8
// widening warps the prefill took 748 us, with one producer warp for both
// tensors 790, with products issued from a branch of one lane 900.
#pragma once

#include <climits>

#include "decode_split.cuh"
#include "fp4_cache.cuh"

namespace pa {

struct VerifyParams {
    const __nv_bfloat16 *q;  // [B * q_len, Hq, D]
    const int32_t *block_table;
    const int32_t *seq_lens;
    void *out;
    float *part_o;
    float2 *part_ml;
    int32_t *status;
    int64_t num_pages;
    int num_q_heads;
    int q_len;
    int group;  // G
    int max_pages_per_seq;
    int max_seq_len;
    int block_size;
    int chunks_per_split;
    int num_splits;
    float scale_log2;
    int out_bf16;
    int early_kv;  // stream the context before the new rows ahead of the dependency wait
    int num_kv_heads;  // grid y = num_kv_heads x 128-row blocks
    int window;        // 0: full attention; W > 0: each row sees only its last W keys
    const float *k_scale;  // fp8 / fp4 cache: [Hkv] dequantisation scales of K and V
    const float *v_scale;
    const uint8_t *k_cache;  // fp4 cache: the records (copied without a tensor map)
    const uint8_t *v_cache;
    // The common part of a decode over shared prefixes (SH kernels): the rows of
    // a CTA are those of the sequences of group blockIdx.z, one per sequence and
    // head, and see the first prefix_lens tokens, rounded down to whole chunks,
    // through the table of the group's leader (leads_group).
    const int32_t *prefix_lens;   // [num_seqs]
    const int32_t *group_starts;  // [groups + 1]
    int num_seqs;
    int max_members;              // sequences of a group that the grid covers
    int prefix_splits;            // the first records of a row's num_splits
    int prefix_chunks;            // of a split, where that makes no more than prefix_splits
};

// Byte offset of 16-byte column chunk c of row t in a [D/64][rows][128 B]
// tile written with the 128-byte swizzle (chunk index XOR row % 8).
__device__ __forceinline__ uint32_t swz_off(int t, int c, int rows) {
    return (uint32_t)((c >> 3) * rows * 128 + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}

// Eight e4m3 codes (one 32-bit word each of four) -> eight f16 in 16 bytes.
__device__ __forceinline__ uint4 e4m3x8_to_f16x8(uint32_t w0, uint32_t w1) {
    uint4 r;
    asm("{\n\t.reg .b16 a, b, c, d;\n\t"
        "mov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
        "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "r"(w0), "r"(w1));
    return r;
}

// Block-table entries a verify CTA stages in shared memory: with 16-token
// pages a 64-token tile spans 4 pages, and a page lookup per chunk from global
// memory would put a dependent load in front of every copy.
constexpr int kVerifyPageTab = 256;

namespace tc {

__device__ __forceinline__ void tmem_alloc(uint32_t *dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst_smem)),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// D[tmem] (+)= A[smem] * B[smem], bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: A's M = 128 rows are the tensor-memory
// lanes, its K elements packed two per 32-bit column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on the mbarrier when every MMA issued so far by this thread is done.
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// Shared-memory matrix descriptor: start address, leading / stride byte
// offsets, descriptor version 1, layout (0: no swizzle, 2: 128-byte swizzle).
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(layout & 7u) << 61;
    return d;
}
// Instruction descriptor, kind::f16: fp32 accumulator, A and B both bf16
// (ab_f16 = false) or both f16, A K-major, B K-major (b_mn = 0) or MN-major
// (b_mn = 1), shape M x N.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int b_mn, bool ab_f16 = false) {
    return (1u << 4) | (ab_f16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 16 consecutive fp32 columns of this thread's tensor-memory lane.
__device__ __forceinline__ void ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
}
// 16 consecutive fp32 columns, without waiting (tcgen05.wait::ld before use).
__device__ __forceinline__ void ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 32 consecutive 32-bit columns of this thread's tensor-memory lane.
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// N 32-bit columns, without waiting.
template <int N>
__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 32) {
        st32(taddr, r);
    } else {
        static_assert(N % 8 == 0, "whole groups of columns");
#pragma unroll
        for (int c = 0; c < N; c += 8) {
            const uint32_t part[8] = {r[c], r[c + 1], r[c + 2], r[c + 3], r[c + 4], r[c + 5], r[c + 6], r[c + 7]};
            st8(taddr + c, part);
        }
    }
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15]))
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

}  // namespace tc

// NSB: S/P tensor-memory buffers (the Q K^T products run up to NSB tiles ahead
// of P V).  TK: keys per score tile, 64 or 128.  With 128 the score product
// S = Q K^T is M = 128 x N = 128: half as many MMA instructions per key as with
// N = 64, whose instruction rate bounds the tile when the tiles come from L2
// (many row blocks per KV head, chunked prefill), and P V runs over two 64-key
// V tiles per score tile.  At D = 256 two 128-column S/P buffers and O fill
// tensor memory, so Q moves to shared memory as the product's A operand (QSM)
// and the K ring holds one 128-key tile; at D = 128 Q stays in tensor memory.
// PT = 3: a weight enters P V as three bf16 numbers, in 96 columns of its buffer,
// and S is summed in two halves of the dims (8 sequences x 4 heads behind 38,000,
// D = 256: error against float64 2.4e-6 with one sum, 1.4e-6 so, in the same time);
// at D = 256 Q moves to shared memory for their sake too.
template <int D, int NK, int NV, int NSG = 0, int NSB = 2, int TK = 64, bool F4 = false, int PT = 2>
struct VerifyTcCfg {
    static constexpr bool F8 = NSG > 0;                // fp8 or fp4 cache: staging ring of NSG slots per tensor
    static constexpr bool QSM = (D == 256 && TK == 128) || (PT == 3 && (D == 256 || NSB == 1));  // Q in shared memory
    // columns of an S/P buffer (PT = 3: S is summed in two halves of the dims, which halves what the sums lose)
    static constexpr int SPLIT_QK = PT == 3 ? 2 : 1, SW = SPLIT_QK * TK;
    static constexpr int M = 128;                      // MMA rows (query rows, zero padded)
    static constexpr int TT = 64;                      // tokens per V tile (4 TMA chunks)
    static constexpr int CPT = TT / kChunk;            // chunks per V tile
    static constexpr int CPK = TK / kChunk;            // chunks per K (score) tile
    static constexpr int VPK = TK / TT;                // V tiles per score tile
    static constexpr int DB = D / 64;                  // 128-byte column blocks
    static constexpr int TILE_BYTES = TT * D * 2;      // V of one tile (bf16 or f16)
    static constexpr int KTILE_BYTES = TK * D * 2;     // K of one score tile
    static constexpr int KVB = F8 ? 1 : 2;             // bytes per cached element
    static constexpr int CHUNK_BYTES = kChunk * D * KVB;  // one TMA chunk as copied
    static constexpr int STG_BYTES = F4 ? CPT * fp4::rec_bytes(D)  // the tile's records
                                        : TT * D;  // one e4m3 tile, [D/128][64 tokens][128 B] swizzled
    static constexpr int OFF_V = NK * KTILE_BYTES;      // K ring, then V ring
    static constexpr int SROW = D * 4 + 16;             // epilogue: output rows staged in the K/V rings
    static constexpr int RINGS = OFF_V + NV * TILE_BYTES;
    static constexpr int OFF_STG = RINGS > M * SROW ? RINGS : (M * SROW + 1023) / 1024 * 1024;  // K staging, then V staging
    static constexpr int OFF_Q = OFF_STG + 2 * NSG * STG_BYTES;  // QSM: Q as [D/64][M rows][128 B], swizzled
    static constexpr int Q_BYTES = QSM ? M * D * 2 : 0;
    static constexpr int OFF_BAR = OFF_Q + Q_BYTES;
    // k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], s_full[NSB], p_full[NP], o_done[NSB], mma_fin,
    // then (fp8, fp4) kst_full[NSG], kst_empty[NSG], vst_full[NSG], vst_empty[NSG]
    static constexpr bool F8W = F8 && !F4 && PT == 1 && D == 256;  // e4m3, one number per weight: widening bounds it
    static constexpr int CW = F4 ? 8 : F8W ? 4 : 2;    // fp8, fp4: widening warps per tensor
    static constexpr int NP = F8 ? NV : NSB;           // P barriers (fp8, fp4: the V slot's too)
    static constexpr int OFF_TMEM = OFF_BAR + (2 * NK + 2 * NV + 2 * NSB + NP + 1 + 4 * NSG) * 8;
    static constexpr int OFF_FLAGS = OFF_TMEM + 16;
    static constexpr int OFF_PT = OFF_FLAGS + 16;                    // the split's block-table entries
    static constexpr int OFF_NAN = OFF_PT + kVerifyPageTab * 4;      // fp4: NaN V blocks that some rows see
    static constexpr int NAN_WORDS = F4 ? D / 16 * 8 : 0;
    static constexpr int SMEM_BYTES = OFF_NAN + NAN_WORDS * 4 + 1024;
    // tensor-memory columns: O (fp32, D), NSB S/P buffers (TK each), Q (bf16
    // pairs, D / 2; not with QSM).  P of a score tile is written over its S
    // buffer, per 64-key half: a bf16 head in 32 columns, then the residual in 32.
    static constexpr int TMEM_COLS = D + NSB * SW + (QSM ? 0 : D / 2) <= 256 ? 256 : 512;
    static constexpr int CTAS = TMEM_COLS == 256 ? 2 : 1;  // per SM
    static constexpr int O_COL = 0;
    static constexpr int S_COL = D;
    static constexpr int Q_COL = D + NSB * SW;
    static constexpr int Q_TCOLS = QSM ? 0 : D / 2;
    static constexpr int SBUF(int j) { return S_COL + j * SW; }
    static constexpr int QROW = D * 2 + 16;            // fp4: rows of Q in f16, staged in the V ring
    static constexpr int OFF_QPRE = OFF_V + M * QROW;  // and their pre-scales
    static_assert(!F4 || M * (QROW + 4) <= NV * TILE_BYTES, "the staged Q rows fit in the V ring");
    static_assert(M * SROW <= OFF_STG, "the staged output rows fit in the K/V rings");
    static constexpr int W0 = F4 || F8W ? 8 : 6;       // first widening warp
    static constexpr int THREADS = (F8 ? W0 + 2 * CW : 6) * 32;
    // many widening warps: registers of the softmax warpgroup and of the others (setmaxnreg).  Their sum draws on
    // what the block was launched with, which the launch checks.
    static constexpr bool RSPLIT = F4 || F8W;
    static constexpr int REGS_SM = F4 ? 152 : 168, REGS_OTHER = F4 ? 64 : 104;
    static constexpr int REGS_LAUNCH = (128 * REGS_SM + (THREADS - 128) * REGS_OTHER + THREADS - 1) / THREADS;
    static_assert(D == 256 || D == 128, "head_dim 256 or 128");
    static_assert(Q_COL + Q_TCOLS <= TMEM_COLS, "tensor-memory columns");
    static_assert(TK == 64 || (TK == 128 && !F8), "128-key score tiles: bf16 cache only");
    static_assert(!F4 || F8, "an fp4 cache is staged and widened");
    static_assert(PT == 2 || (PT == 1 && F8) || (PT == 3 && !F8 && TK == 64), "numbers per weight");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
};

// NSG > 0: fp8 cache (tm_k / tm_v: e4m3 boxes of 128 codes x 16 tokens,
// tm_k64 / tm_v64: 5-D boxes of a whole 64-token tile, both with the 128-byte
// swizzle).
// tm_k64: 5-D boxes of a whole K tile of TK keys (64, or 128 with TK = 128).
// RES: the residual of P is multiplied too (F4 with bf16 output goes without:
// a weight is then off by half a step of f16, 2^-11 of itself, an eighth of the
// half step that the output is rounded by).
// FAR: O is moved to a second sum every kVerifyFarTiles tiles (splits of more
// tiles with fp32 output).  The tensor core cuts each addition to an accumulator
// off towards zero: O loses 2.4e-9 of itself per key (measured; half a step,
// 2^-24, for each of the eight products of a tile, on a sum that grows), 7e-7 in
// 4 tiles -- what binary32 sums over a thousand keys are off by.
// (8 x 16 rows over 8K, error against float64 and time: 4 tiles 9.4e-7 and 77 us,
// 8 tiles 1.3e-6 and 64, 16 tiles 2.5e-6 and 57, none 51; a 32-bit product and
// softmax in torch is off by 1.7e-6.  Four keeps below that at any length.)
constexpr int kVerifyFarTiles = 4;
// Logits (log2 units) up to which an exponent may be formed as score * scale -
// max in one fused step: the max is that product rounded, off by up to 2^-24 of
// itself, which beyond this would pass through 2^x as a factor of two and more.
constexpr float kExactLogits = 16777216.f;
// SH: the common part of a decode over shared prefixes (VerifyParams): no causal
// mask, a row per sequence and head.
// COP: up to M / COP rows stand in the block COP times, and copy k takes keys k * 64
// / COP .. of every tile, with zeros for its other weights: small groups leave
// most softmax threads without a row, and a tile waits for the few that have one.
// A copy is a split of its own to the merge.
template <int D, int NK, int NV, int NSG, int NSB, int TK = 64, bool F4 = false, bool RES = true,
          bool FAR = false, bool SH = false, int PT = RES ? 2 : 1, int COP = 1>
__global__ void __launch_bounds__(VerifyTcCfg<D, NK, NV, NSG, NSB, TK, F4, PT>::THREADS,
                                  VerifyTcCfg<D, NK, NV, NSG, NSB, TK, F4, PT>::CTAS)
    pa_verify_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_k64, const __grid_constant__ CUtensorMap tm_v64,
                        const VerifyParams p) {
    using C = VerifyTcCfg<D, NK, NV, NSG, NSB, TK, F4, PT>;
    constexpr bool F8 = C::F8, QSM = C::QSM;
    static_assert(RES == (PT > 1) && (RES || (F8 && C::VPK == 1)), "the residual is left out over quantised caches only");
    constexpr int TT = C::TT, CPT = C::CPT, CPK = C::CPK, VPK = C::VPK;
    static_assert(!FAR || (RES && C::VPK == 1), "a second sum of O: fp32 output");
    constexpr int RB = C::M / COP, KPT = TT / COP;  // rows of a copy; keys of a tile per softmax thread
    static_assert(COP == 1 || (SH && VPK == 1 && !F4), "copies of rows: the common part of a shared prefix");
    constexpr float kLazy = 8.f;  // raise the reference max only when it grows by more than 2^8
    // fp4 and, behind shared prefixes, e4m3: the reference is kept 2^7 below the max,
    // so that P in f16, at most 2^15, holds weights down to 2^-32 of the largest (f16
    // ends at 2^-25).
    constexpr float kBelow = F4 || (SH && F8) ? 7.f : 0.f;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    // K and V tiles have their own rings: a K slot is free again as soon as
    // S_i = Q K_i^T is done, long before O += P_i V_i releases the V slot.
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *k_empty = k_full + NK;
    uint64_t *v_full = k_empty + NK;
    uint64_t *v_empty = v_full + NV;
    uint64_t *s_full = v_empty + NV;   // [NSB]: S_i written (buffer i % NSB)
    // [NP] (i % NP): P_i written by the softmax warps and, over an fp8 or fp4
    // cache, V_i widened: one wait for both (NP = NV then, so that V_i, whose
    // slot O += P_{i-NV} V_{i-NV} has freed, never arrives on an open phase of P_{i-NV})
    uint64_t *p_full = s_full + NSB;
    uint64_t *o_done = p_full + C::NP;  // [NSB]: O += P_i V_i finished
    uint64_t *mma_fin = o_done + NSB;
    uint64_t *kst_full = mma_fin + 1;  // fp8, fp4: cached tile landed in a staging slot
    uint64_t *kst_empty = kst_full + NSG;  // fp8: staging slot widened, free again
    uint64_t *vst_full = kst_empty + NSG;
    uint64_t *vst_empty = vst_full + NSG;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    // [0] abort, [1] bad page, [2] nan_bits holds something
    volatile int *flags = reinterpret_cast<volatile int *>(smem + C::OFF_FLAGS);
    int32_t *page_tab = reinterpret_cast<int32_t *>(smem + C::OFF_PT);
    // F4: a V block with a NaN scale whose token only some of the rows see
    // enters the product as zeros (0 * NaN would reach every row) and is noted
    // here; the rows that see the token get their NaN in the epilogue.
    // [scale block][0-3: token - (first row's last key + 1), 4-7: token - k_first]
    uint32_t *nan_bits = reinterpret_cast<uint32_t *>(smem + C::OFF_NAN);

    const int split = blockIdx.x, kvh = blockIdx.y % p.num_kv_heads;
    [[maybe_unused]] int b = blockIdx.z;  // the sequence whose block table is read
    // Row blocks launch last-first: later blocks see more keys (causal), so the
    // longest CTAs go out in the first wave and a partial last wave holds the
    // shortest ones.
    const int n_blocks = gridDim.y / p.num_kv_heads;
    const int row0 = (n_blocks - 1 - (int)(blockIdx.y / p.num_kv_heads)) * C::M;  // first row (rho = r G + g)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row_l = COP > 1 ? (int)threadIdx.x % RB : (int)threadIdx.x;  // softmax threads: row of the block, and its copy
    [[maybe_unused]] const int copy = COP > 1 ? (int)threadIdx.x / RB : 0;
    const int G = p.group;
    size_t row_base = (size_t)blockIdx.z * p.q_len;  // of the call's (sequence, new row) pairs: this CTA's first
    int members = p.q_len;                           // pairs of this CTA's sequence (SH: sequences of its group)
    [[maybe_unused]] int prefix = 0;                 // SH: prefix_lens of the group
    if constexpr (SH) {
        // The kernel behind this one, which works on the sequences' own parts,
        // depends on the work before both, not on this one: it may start now.
        pdl_wait_primary();
        pdl_launch_dependents();
        const int g = blockIdx.z;
        const int lo = min(max(p.group_starts[g], 0), p.num_seqs);
        const int hi = min(max(p.group_starts[g + 1], lo), p.num_seqs);
        row_base = lo;
        members = min(hi - lo, p.max_members);
        // the group's leader has the table and the length of the prefix
        int first = -1;
        for (int i0 = 0; i0 < members && first < 0; i0 += 32) {
            const int i = i0 + (threadIdx.x & 31);
            const int len = i < members ? p.seq_lens[lo + i] : 0, pre = i < members ? p.prefix_lens[lo + i] : 0;
            const uint32_t there = __ballot_sync(0xffffffffu, leads_group(len, pre, p.max_seq_len));
            if (there != 0) first = i0 + __ffs(there) - 1;
        }
        b = lo + max(first, 0);
        if (first >= 0) prefix = max(0, p.prefix_lens[b]);  // (a sequence with a negative one is flagged below)
        if (row0 == 0 && members < hi - lo) {  // more than the host said: rows without a CTA
            if (threadIdx.x == 0 && split == 0 && kvh == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
            for (int rho = members * G + threadIdx.x; rho < (hi - lo) * G; rho += C::THREADS)
                for (int k = 0; k < COP; ++k)
                    p.part_ml[((row_base + rho / G) * p.num_q_heads + kvh * G + rho % G) * p.num_splits + split * COP + k] =
                        make_float2(-INFINITY, -1.f);
        }
        if (row0 >= members * G) return;  // no row in this block
    } else {
        pdl_launch_dependents();
    }
    const int R = min(RB, members * G - row0);  // rows of this block
    // SH: what becomes of row rho: 0 its share of the prefix, 1 nothing (an idle
    // sequence), 2 zeros (its lengths are bad, or not those of the group)
    [[maybe_unused]] auto row_state = [&](int rho) {
        const int s = (int)row_base + rho / G, len = p.seq_lens[s], pre = p.prefix_lens[s];
        if (len == 0) return 1;
        const bool ok = len > 0 && len <= p.max_seq_len && pre == prefix && pre <= len;
        if (!ok && split == 0 && kvh == 0 && rho % G == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
        return ok ? 0 : 2;
    };
    if (threadIdx.x == 0) {
        // a K/V ring slot is filled by the copy engine (one expect-tx arrival),
        // or with an fp8 cache by the CW widening warps of its tensor
        for (int s = 0; s < NK; ++s) {
            mbar_init(&k_full[s], F8 ? C::CW : 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int j = 0; j < NSB; ++j) {
            mbar_init(&s_full[j], 1);
            mbar_init(&o_done[j], 1);
        }
        for (int j = 0; j < C::NP; ++j) mbar_init(&p_full[j], F8 ? 4 + C::CW : 4);
        mbar_init(mma_fin, 1);
        for (int s = 0; s < NSG; ++s) {
            mbar_init(&kst_full[s], 1);
            mbar_init(&kst_empty[s], C::CW);
            mbar_init(&vst_full[s], 1);
            mbar_init(&vst_empty[s], C::CW);
        }
        flags[0] = 0;
        flags[1] = 0;
        flags[2] = 0;
        fence_mbar_init();
    }
    for (int j = threadIdx.x; j < C::NAN_WORDS; j += C::THREADS) nan_bits[j] = 0;
    if (!F4 && warp == 5 && lane == 0) {  // (the fp4 records are copied without tensor maps)
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_k64);
        prefetch_tensormap(&tm_v64);
    }
    // This row's q goes to L2 ahead of the dependency wait: L2 is where global
    // memory is kept coherent, so a row the work before this call is still
    // writing is read in its final state after the wait all the same.
    const int rho_q = row0 + row_l;  // the softmax threads' rows (rows past R are zero padding)
    const __nv_bfloat16 *qrow = p.q + ((row_base + rho_q / G) * p.num_q_heads + kvh * G + rho_q % G) * D;
    if (!SH && !F4 && warp < 4 && (int)threadIdx.x < R) {
#pragma unroll
        for (int o = 0; o < D * 2; o += 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(qrow) + o));
    }
    // fp4: the widening warps, idle until the first records land, fetch and
    // convert Q, 8 rows each, a row's 16-byte pieces by neighbouring lanes.
    // (A row per softmax thread is 1000 instructions that run once, at the pace
    // they come from memory: 4 us until the first product.)
    constexpr int QL = D / 8;              // lanes of a row
    constexpr int QN = F4 ? QL / 4 : 1;    // loads of a lane: 8 rows, 32 / QL at a time
    [[maybe_unused]] uint4 qx[QN];
    [[maybe_unused]] auto fetch_q = [&]() {
        int rl = 8 * (warp - C::W0) + lane / QL;
        const int rho = row0 + rl, qi = rho / G;
        int g = rho - qi * G;
        const __nv_bfloat16 *row =
            p.q + ((row_base + qi) * p.num_q_heads + kvh * G + g) * D + 8 * (lane % QL);
#pragma unroll
        for (int k = 0; k < QN; ++k) {
            qx[k] = rl < R ? *reinterpret_cast<const uint4 *>(row) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int m = 0; m < 32 / QL; ++m) {  // the next row: the next head, or the next query's first
                const bool wrap = ++g == G;
                g = wrap ? 0 : g;
                row += wrap ? (p.num_q_heads - G + 1) * D : D;
            }
            rl += 32 / QL;
        }
    };
    // Every global access waits for the work before this call on the stream,
    // except with early_kv: then the block table, seq_lens and the tiles that
    // end before the new rows are read first (see the producer below).
    if (!p.early_kv) {
        if (!SH) pdl_wait_primary();
        if (F4 && warp >= C::W0) fetch_q();
    }

    int L = SH ? prefix / kChunk * kChunk : p.seq_lens[b];
    const bool bad_len = !SH && (L < 0 || L > p.max_seq_len || L < p.q_len);
    if (bad_len) {
        if (threadIdx.x == 0 && split == 0 && kvh == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
        L = 0;
    }
    const int n_chunks = (L + kChunk - 1) / kChunk;
    // SH: splits of whole 64-token tiles of the group's own prefix, as long as planned or longer
    const int cps = SH ? max(p.prefix_chunks, (n_chunks + 4 * p.prefix_splits - 1) / (4 * p.prefix_splits) * 4)
                       : p.chunks_per_split;
    // with a sliding window the splits start at the chunk of the block's first
    // visible key (its first row's window start)
    const int k_first = !SH && p.window > 0 ? max(0, L - p.q_len + row0 / G - p.window + 1) : 0;
    const int c_begin = k_first / kChunk + split * cps;
    // keys past the block's last row's causal limit are never read
    const int k_last = SH ? L - 1 : L - p.q_len + (row0 + R - 1) / G;
    const int n_my = min((SH ? n_chunks : min(n_chunks, k_last / kChunk + 1)) - c_begin, cps);
    if (SH && n_my <= 0) {  // the row's other splits have its keys, if there are any
        for (int rho = row0 + threadIdx.x; rho < row0 + R; rho += C::THREADS) {
            const float2 empty = make_float2(-INFINITY, row_state(rho) == 2 ? -1.f : 0.f);
            for (int k = 0; k < COP; ++k)
                p.part_ml[((row_base + rho / G) * p.num_q_heads + kvh * G + rho % G) * p.num_splits + split * COP + k] = empty;
        }
        return;
    }
    if (n_my <= 0) {
        // No key of this sequence in this split: an empty record (m = -inf,
        // l = 0) for the reduce, or zero rows when the call is unsplit.
        if (p.early_kv) pdl_wait_primary();
        if (p.num_splits == 1) {
            for (int idx = threadIdx.x; idx < R * D; idx += C::THREADS) {
                const int rho = row0 + idx / D, d = idx % D;
                const size_t row = row_base + rho / G;
                store_out(p.out, (row * p.num_q_heads + kvh * G + rho % G) * D + d, 0.f, p.out_bf16);
            }
        } else {
            for (int rho = row0 + threadIdx.x; rho < row0 + R; rho += C::THREADS) {
                const size_t row = row_base + rho / G;
                p.part_ml[(row * p.num_q_heads + kvh * G + rho % G) * p.num_splits + split] =
                    make_float2(-INFINITY, 0.f);
            }
        }
        return;
    }
    const int n_tiles = (n_my + CPK - 1) / CPK;   // score tiles (K tiles)
    const int n_vtiles = (n_my + CPT - 1) / CPT;  // V tiles (VPK per score tile)
    // tile i starts O anew: what the tiles before it summed goes to the second sum
    // (beside Q K^T's own loss: fewer tiles at D = 256 and for three products a step; a copy adds to its sums in every
    // COP-th step)
    constexpr int kFarTiles = (PT == 3 || (SH && D == 256) ? 3 : kVerifyFarTiles) * COP;
    auto far_at = [&](int i) { return FAR && i > 0 && i % kFarTiles == 0; };

    // The split's block-table entries, staged in shared memory by all threads
    // (visible to the producer after the next __syncthreads); splits spanning
    // more pages read the table from global memory.
    const int32_t *bt = p.block_table + (size_t)b * p.max_pages_per_seq;
    const int lp_first = (c_begin * kChunk) / p.block_size;
    const int n_pt = ((c_begin + n_my) * kChunk - 1) / p.block_size - lp_first + 1;
    const bool staged = n_pt <= kVerifyPageTab;
    if (staged)
        for (int j = threadIdx.x; j < n_pt; j += C::THREADS) page_tab[j] = bt[lp_first + j];

    // TMA copies of one tile of K (CPK chunks) or of V (CPT chunks), issued by
    // the whole producer warp: lane 0 arms the barrier; a tile inside one page
    // is one 5-D box (lane 0), otherwise lane c * NB + b copies column block b
    // of chunk c, so a tile over 16-token pages (16 boxes per tensor for
    // D = 256) costs no more issue time than one box.
    int issued_k = 0, issued_v = 0;
    auto issue_tile = [&](int i, int tensor, uint64_t policy) {
        constexpr int NB = F8 ? D / 128 : C::DB;  // boxes per 16-token chunk (128-byte columns)
        constexpr int BW = F8 ? 128 : 64;         // elements per box row
        const int s = F8 ? i % (NSG > 0 ? NSG : 1) : (tensor == 0 ? i % NK : i % NV);
        uint64_t *bar = F8 ? (tensor == 0 ? &kst_full[s] : &vst_full[s]) : (tensor == 0 ? &k_full[s] : &v_full[s]);
        uint8_t *dst0 = F8 ? smem + C::OFF_STG + (tensor * NSG + s) * C::STG_BYTES
                           : smem + (tensor == 0 ? s * C::KTILE_BYTES : C::OFF_V + s * C::TILE_BYTES);
        const CUtensorMap *m4 = tensor == 0 ? &tm_k : &tm_v;
        const CUtensorMap *m5 = tensor == 0 ? &tm_k64 : &tm_v64;
        const int cpt = tensor == 0 ? CPK : CPT, tt = cpt * kChunk;  // chunks and tokens per tile
        const int nc = min(cpt, n_my - i * cpt);  // chunks in this tile
        if (lane == 0) mbar_arrive_expect_tx(bar, nc * C::CHUNK_BYTES);
        __syncwarp();
        auto page_of = [&](int lp) {
            const int page = staged ? page_tab[lp - lp_first] : bt[lp];
            if (page < 0 || (int64_t)page >= p.num_pages) {
                flags[1] = 1;  // the copy reads zeros (box outside the tensor)
                set_status(p.status, PA_DEV_BAD_PAGE);
            }
            return page;
        };
        const int t00 = (c_begin + i * cpt) * kChunk;
        const int lp0 = t00 / p.block_size, off0 = t00 - lp0 * p.block_size;
        if (nc == cpt && off0 + tt <= p.block_size) {
            // the whole tile lies in one page: one copy lands it as [blocks][tt tokens][128 B]
            if (lane == 0) tma_load_5d(dst0, m5, bar, 0, off0, 0, kvh, page_of(lp0), policy);
        } else if (lane < nc * NB) {
            const int c = lane / NB, db = lane % NB;
            const int t0 = t00 + c * kChunk, lp = t0 / p.block_size;
            tma_load_4d(dst0 + db * tt * 128 + c * kChunk * 128, m4, bar, db * BW, kvh, t0 - lp * p.block_size,
                        page_of(lp), policy);
        }
        __syncwarp();
    };
    static_assert(CPK * (F8 ? D / 128 : C::DB) <= 32, "a lane per box of a tile");
    // fp4: warp 5 copies K, warp 6 V (a copy's issue takes one lane 0.15
    // us: both tensors' would fill one warp's time).  A lane keeps the page and
    // the place in it of its chunk of the next tile.
    [[maybe_unused]] const int f4_tensor = warp == 5 ? 0 : 1, f4_cpp = p.block_size / kChunk;
    [[maybe_unused]] int f4_lp = 0, f4_in = 0, f4_next = 0;
    if (F4 && (warp == 5 || warp == 6)) {
        f4_lp = (c_begin + lane) / f4_cpp;
        f4_in = c_begin + lane - f4_lp * f4_cpp;
    }
    [[maybe_unused]] const int f4_step_lp = CPT / f4_cpp, f4_step_in = CPT % f4_cpp;
    [[maybe_unused]] auto issue_f4 = [&](uint64_t policy) {
        constexpr int REC = fp4::rec_bytes(D);
        const int i = f4_next++, s = i % (NSG > 0 ? NSG : 1);
        const int nc = min(CPT, n_my - i * CPT);
        uint64_t *bar = (f4_tensor == 0 ? kst_full : vst_full) + s;
        if (lane == 0) mbar_arrive_expect_tx(bar, nc * REC);
        // the chunks of a page are contiguous: one copy for a tile inside one page, else one per chunk
        const bool whole = __shfl_sync(0xffffffffu, f4_in, 0) + nc <= f4_cpp;
        if (lane < (whole ? 1 : nc)) {
            int page = staged ? page_tab[f4_lp - lp_first] : bt[f4_lp];
            if (page < 0 || (int64_t)page >= p.num_pages) {
                flags[1] = 1;  // the rows are zeroed; page 0 is read in its place
                set_status(p.status, PA_DEV_BAD_PAGE);
                page = 0;
            }
            const int64_t rec = ((int64_t)page * p.num_kv_heads + kvh) * f4_cpp + f4_in;
            fp4::bulk_load(smem + C::OFF_STG + (f4_tensor * NSG + s) * C::STG_BYTES + lane * REC,
                           (f4_tensor == 0 ? p.k_cache : p.v_cache) + rec * REC, (whole ? nc : 1) * REC, bar, policy);
        }
        f4_lp += f4_step_lp;
        f4_in += f4_step_in;
        if (f4_in >= f4_cpp) {
            f4_in -= f4_cpp;
            ++f4_lp;
        }
        __syncwarp();
    };
    // tiles that end before the new rows (early_kv reads only those before the wait)
    auto before_new_rows = [&](int i, int cpt) {
        return (c_begin + i * cpt + min(cpt, n_my - i * cpt)) * kChunk <= L - p.q_len;
    };
    if (p.early_kv) {
        __syncthreads();  // barrier initialisation and the page table are visible to the producer warp
        if constexpr (F4) {
            if (warp == 5 || warp == 6)
                while (f4_next < min(NSG, n_tiles) && before_new_rows(f4_next, CPT)) issue_f4(l2_policy_evict_first());
        } else if (warp == 5) {
            // first use of each slot: tiles that end before the new rows
            const uint64_t policy = l2_policy_evict_first();
            constexpr int FK = F8 ? NSG : NK, FV = F8 ? NSG : NV;  // slots the copies land in
            while (issued_k < min(FK, n_tiles) && before_new_rows(issued_k, CPK)) issue_tile(issued_k++, 0, policy);
            while (issued_v < min(FV, n_vtiles) && before_new_rows(issued_v, CPT)) issue_tile(issued_v++, 1, policy);
        }
        pdl_wait_primary();
        if (F4 && warp >= C::W0) fetch_q();
    }

    // Q rows: each softmax thread loads its row (D / 8 16-byte words, one
    // round of loads) right after the dependency wait, so the loads are in
    // flight while tensor memory is allocated.
    constexpr int NQ = D / 8;
    [[maybe_unused]] uint4 qv[NQ];
    if (!F4 && warp < 4) {
        const bool qlive = row_l < R;
#pragma unroll
        for (int v = 0; v < NQ; ++v)
            qv[v] = qlive ? *reinterpret_cast<const uint4 *>(qrow + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (warp == 4) {
        tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    // The tensor-memory address reaches the softmax and MMA warps (0-4).  With
    // early_kv the other warps synchronised ahead of the wait (barriers, page
    // table) and go on streaming; without it this is their synchronisation.
    if (p.early_kv) {
        if (warp < 5) named_bar_sync(2, 160);
    } else {
        __syncthreads();
    }
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;  // (read by warps 0-4 only on the early_kv path)
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);  // this warp's tensor-memory lanes

    // Q block -> tensor memory, the A operand of S = Q K^T: row rho in lane
    // rho, dims packed two per column (column c holds elements 2c and 2c + 1);
    // padding rows are zero.  The softmax warps store it while the producer
    // already streams K and V; only the MMA warp waits for it (named barrier
    // 1: warps 0-4).  Over an fp8 cache the products run in f16, and each row
    // enters scaled by q_pre, the power of two that brings its largest element
    // into [2^14, 2^15) (f16_prescale).
    float q_pre = 1.f;
    if (!F4 && warp < 4) {
        if constexpr (F8) {  // the products run in f16: Q too
            uint32_t amax = 0;
#pragma unroll
            for (int v = 0; v < NQ; ++v)
                amax = max(max(amax, max(bf16x2_absmax(qv[v].x), bf16x2_absmax(qv[v].y))),
                           max(bf16x2_absmax(qv[v].z), bf16x2_absmax(qv[v].w)));
            q_pre = f16_prescale(amax);
#pragma unroll
            for (int v = 0; v < NQ; ++v)
                qv[v] = make_uint4(bf16x2_to_f16x2_scaled(qv[v].x, q_pre), bf16x2_to_f16x2_scaled(qv[v].y, q_pre),
                                   bf16x2_to_f16x2_scaled(qv[v].z, q_pre), bf16x2_to_f16x2_scaled(qv[v].w, q_pre));
        }
        if constexpr (QSM) {
            // row rho of the block at [D/64 column blocks][M rows][128 B], 16-byte unit u of a
            // row stored at unit u ^ (row % 8): the K-major operand layout with the 128-byte swizzle
            const int r = threadIdx.x;
#pragma unroll
            for (int v = 0; v < NQ; ++v)
                *reinterpret_cast<uint4 *>(smem + C::OFF_Q + (v / 8) * (C::M * 128) + r * 128 +
                                           (((v % 8) ^ (r % 8)) << 4)) = qv[v];
            tc::fence_async_smem();  // the rows are read by the tensor core
        } else {
#pragma unroll
            for (int c = 0; c < NQ / 8; ++c) {
                uint32_t r[32];
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    r[4 * v] = qv[8 * c + v].x;
                    r[4 * v + 1] = qv[8 * c + v].y;
                    r[4 * v + 2] = qv[8 * c + v].z;
                    r[4 * v + 3] = qv[8 * c + v].w;
                }
                tc::st32(lane_base + C::Q_COL + 32 * c, r);
            }
            tc::wait_st();
        }
        tc::fence_before();
        asm volatile("bar.arrive 1, 160;" ::: "memory");
    } else if (!F4 && warp == 4) {
        asm volatile("bar.sync 1, 160;" ::: "memory");
        tc::fence_after();
    }

    // (a branch for setmaxnreg: what either side may use is known only where the sides are apart)
    if (warp >= 4) {
    if constexpr (C::RSPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    if (F4 && (warp == 5 || warp == 6)) {
        // ---------------- fp4 producers: records of K (warp 5) and V (warp 6) ----------------
        const uint64_t policy = l2_policy_evict_first();
        constexpr int NS = NSG > 0 ? NSG : 1;
        uint64_t *full = f4_tensor == 0 ? kst_full : vst_full, *empty = f4_tensor == 0 ? kst_empty : vst_empty;
        while (f4_next < n_tiles) {
            const int i = f4_next;
            if (i >= NS && !__all_sync(0xffffffffu, mbar_wait(&empty[i % NS], ((i / NS) - 1) & 1, &flags[0]))) {
                if (lane == 0) {
                    flags[0] = 1;
                    set_status(p.status, PA_DEV_TIMEOUT);
                }
                break;
            }
            issue_f4(policy);
        }
        if (lane == 0 && flags[0]) {
            // let the copies in flight land before the CTA ends
            for (int i = max(0, f4_next - NS); i < f4_next; ++i)
                for (uint32_t n = 0; n < kWaitPollLimit && !mbar_try_wait(&full[i % NS], (i / NS) & 1); ++n) {
                }
        }
    } else if (warp == 5) {
        // ---------------- producer: TMA copies of K and V, 4 chunks per tile ----------------
        // Two rings refilled independently: lane 0 probes the next slot of
        // each without blocking and the warp issues the tile; within a ring
        // tiles go in order.  Every decision is lane 0's, so the warp stays
        // converged.
        const uint64_t policy = l2_policy_evict_first();
        uint32_t idle = 0;
        // the slots the copies land in: the K/V rings, or the fp8 staging rings
        constexpr int FK = F8 ? NSG : NK, FV = F8 ? NSG : NV;
        uint64_t *ke = F8 ? kst_empty : k_empty;
        uint64_t *ve = F8 ? vst_empty : v_empty;
        while (issued_k < n_tiles || issued_v < n_vtiles) {
            bool go_k = false, go_v = false;
            if (lane == 0) {
                go_k = issued_k < n_tiles &&
                       (issued_k < FK || mbar_test_wait(&ke[issued_k % FK], ((issued_k / FK) - 1) & 1));
                go_v = issued_v < n_vtiles &&
                       (issued_v < FV || mbar_test_wait(&ve[issued_v % FV], ((issued_v / FV) - 1) & 1));
            }
            go_k = __shfl_sync(0xffffffffu, go_k, 0);
            go_v = __shfl_sync(0xffffffffu, go_v, 0);
            if (go_k) issue_tile(issued_k++, 0, policy);
            if (go_v) issue_tile(issued_v++, 1, policy);
            if (go_k || go_v) {
                idle = 0;
            } else {
                const bool stop = __shfl_sync(0xffffffffu, ++idle > kWaitPollLimit || flags[0] != 0, 0);
                if (stop) {
                    if (lane == 0) flags[0] = 1;
                    break;
                }
            }
        }
        if (lane == 0 && flags[0]) {
            // let the copies in flight land before the CTA ends
            uint64_t *kf = F8 ? kst_full : k_full;
            uint64_t *vf = F8 ? vst_full : v_full;
            for (int i = max(0, issued_k - FK); i < issued_k; ++i)
                for (uint32_t n = 0; n < kWaitPollLimit && !mbar_try_wait(&kf[i % FK], (i / FK) & 1); ++n) {
                }
            for (int i = max(0, issued_v - FV); i < issued_v; ++i)
                for (uint32_t n = 0; n < kWaitPollLimit && !mbar_try_wait(&vf[i % FV], (i / FV) & 1); ++n) {
                }
            set_status(p.status, PA_DEV_TIMEOUT);
        }
    } else if (warp == 4) {
        // ---------------- MMA issue ----------------
        // The warp runs the loop together and one elected lane issues, so that
        // descriptors and addresses stay in uniform registers: issued by a
        // branch of one lane, the 16 products of S_i took 720 clocks and more,
        // not the tensor core's 517.
        {
            if constexpr (F4) {  // (Q stands in tensor memory)
                asm volatile("bar.sync 1, 160;" ::: "memory");
                tc::fence_after();
            }
            constexpr uint32_t kIdQK = tc::idesc_bf16(128, TK, 0, F8);
            constexpr uint32_t kIdPV = tc::idesc_bf16(128, D, 1, F8);
            const bool leader = tc::elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            // descriptors of the first K and V slots; offsets are added in 16-byte units
            // K: 16-element k steps: +32 B inside a 128-byte swizzle row, next 64-dim block further on
            // V: MN-major; 64-dim blocks TT x 128 B apart (LBO), 8-token groups 1 KiB apart (SBO)
            const uint64_t k_desc0 = tc::sdesc(smem_addr(smem), 16, 1024, 2);
            const uint64_t v_desc0 = tc::sdesc(smem_addr(smem + C::OFF_V), TT * 128, 1024, 2);
            [[maybe_unused]] const uint64_t q_desc = tc::sdesc(smem_addr(smem + C::OFF_Q), 16, 1024, 2);
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait(bar, parity, &flags[0]));
            };
            // S_i = Q K_i^T for the first NSB tiles, then per tile O += P_i V_i
            // as soon as the softmax warps have written P_i, and S_{i+NSB},
            // which shares P_i's columns: the tensor core runs this thread's
            // MMAs in issue order, so S_{i+NSB} never overwrites P_i before
            // O += P_i V_i has read it.  (Polling for whichever of the two was
            // ready first left 0.3 us between a product's inputs and its issue:
            // a fixed order can wait without polling.)
            bool ok = true;
            for (int step = 0; step < n_tiles + NSB; ++step) {
                if (step >= NSB) {
                    const int i = step - NSB, j = i % NSB;
                    const int nvt = VPK == 1 ? 1 : min(VPK, n_vtiles - i * VPK);
                    ok = wait(&p_full[i % C::NP], (i / C::NP) & 1);
                    for (int h2 = 0; h2 < nvt && ok; ++h2) {
                        const int vt = i * VPK + h2;
                        if (!F8) ok = wait(&v_full[vt % NV], (vt / NV) & 1);
                        if (!ok) break;
                        tc::fence_after();
                        if (leader) {
                            const uint64_t v_desc = v_desc0 + (uint32_t)(vt % NV) * (C::TILE_BYTES >> 4);
#pragma unroll
                            for (int ks = 0; ks < TT / 16; ++ks) {
#pragma unroll
                                for (int h = 0; h < PT; ++h) {
                                    // P (head, then residual) of this 64-key half: 16 tokens = 8 columns per step
                                    const uint32_t a_tm = tm + C::SBUF(j) + h2 * TT + h * (TT / 2) + ks * 8;
                                    tc::mma_bf16_ta(tm + C::O_COL, a_tm, v_desc + (ks * 16 * 128 >> 4), kIdPV,
                                                    ((i > 0 && !far_at(i)) || h2 > 0 || ks > 0 || h > 0) ? 1u : 0u);
                                }
                            }
                            tc::commit(&v_empty[vt % NV]);
                            if (h2 == nvt - 1) tc::commit(&o_done[j]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                if (step < n_tiles) {
                    const int i = step, s = i % NK, j = i % NSB;
                    ok = wait(&k_full[s], (i / NK) & 1);
                    if (!ok) break;
                    tc::fence_after();
                    if (leader) {
                        const uint64_t k_desc = k_desc0 + (uint32_t)s * (C::KTILE_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t koff = ((kk >> 2) * (TK * 128) + (kk & 3) * 32) >> 4;
                            if constexpr (QSM) {  // Q from shared memory, laid out like K with M rows
                                const uint32_t qoff = ((kk >> 2) * (C::M * 128) + (kk & 3) * 32) >> 4;
                                constexpr int KH = D / 16 / C::SPLIT_QK;
                                tc::mma_bf16(tm + C::SBUF(j) + kk / KH * TK, q_desc + qoff, k_desc + koff, kIdQK,
                                             kk % KH > 0 ? 1u : 0u);
                            } else {
                                tc::mma_bf16_ta(tm + C::SBUF(j), tm + C::Q_COL + kk * 8, k_desc + koff, kIdQK,
                                                kk > 0 ? 1u : 0u);
                            }
                        }
                        tc::commit(&k_empty[s]);
                        tc::commit(&s_full[j]);
                    }
                    __syncwarp();
                }
            }
            if (leader) {
                if (!ok) {
                    flags[0] = 1;
                    set_status(p.status, PA_DEV_TIMEOUT);
                }
                // Whatever happened, let every issued MMA finish before tensor
                // memory is released at the end of the CTA.
                tc::commit(mma_fin);
                for (uint32_t n = 0; n < kWaitPollLimit && !mbar_try_wait(mma_fin, 0); ++n) {
                }
            }
            __syncwarp();
        }
    } else if (warp >= C::W0) {
        if constexpr (F4) {
            // ---------------- fp4: widen staged records into the K (warps 8-15) / V (16-23) ring ----------------
            // A warp takes half a record of the tile: 8 tokens.
            static_assert(C::CW == 2 * C::CPT, "two widening warps per record of a tile");
            constexpr int REC = fp4::rec_bytes(D), NBL = D / 16;
            const int tensor = (warp - C::W0) / C::CW, rc = (warp - C::W0) % C::CW / 2, half = warp & 1;
            const int NR = tensor == 0 ? NK : NV;
            uint64_t *ring_full = tensor == 0 ? k_full : p_full;
            uint64_t *ring_empty = tensor == 0 ? k_empty : v_empty;
            uint64_t *stg_full = tensor == 0 ? kst_full : vst_full;
            uint64_t *stg_empty = tensor == 0 ? kst_empty : vst_empty;
            uint8_t *ring = smem + (tensor == 0 ? 0 : C::OFF_V) + (rc * kChunk + 8 * half) * 128;
            uint8_t *stg = smem + C::OFF_STG + tensor * NSG * C::STG_BYTES + rc * REC;
            const int t_end = min(k_last + 1, (c_begin + n_my) * kChunk);
            // every row sees the tokens [w_last, f_last]
            const int f_last = SH ? L - 1 : L - p.q_len + row0 / G;
            const int w_last = !SH && p.window > 0 ? k_last - p.window + 1 : 0;
            // K: lane = token r of the half, quarter c of every block; r and r ^ 5 in the same quarter-warp, so that
            // its eight 16-byte reads (bit 0) and ring writes (bit 2) fall in eight bank groups
            // V: lane = token pair c, dims 2 r, 2 r + 1 of every block
            const int c = lane & 3, r = tensor == 0 ? (lane >> 3) ^ (lane & 4 ? 5 : 0) : lane >> 2;
            // Q first: as f16 with the row's pre-scale, dims in the order of the widened K tiles (of a 16-byte piece's
            // two halves, dims 4 c .. + 3 of a block, the first goes to an even, the second to the next odd place)
            {
                const int first = 8 * (warp - C::W0) + (QL == 32 ? 0 : lane / QL), piece = lane % QL;
                uint8_t *dst = smem + C::OFF_V + (piece >> 2) * 64 + (piece & 1) * 32 + (piece >> 1 & 1) * 8;
#pragma unroll
                for (int k = 0; k < QN; ++k) {
                    const uint4 x = qx[k];
                    uint32_t amax = max(max(bf16x2_absmax(x.x), bf16x2_absmax(x.y)),
                                        max(bf16x2_absmax(x.z), bf16x2_absmax(x.w)));
#pragma unroll
                    for (int o = QL / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    const float pre = f16_prescale(amax);
                    const int rl = first + k * (32 / QL);
                    uint2 *d = reinterpret_cast<uint2 *>(dst + rl * C::QROW);
                    d[0] = make_uint2(bf16x2_to_f16x2_scaled(x.x, pre), bf16x2_to_f16x2_scaled(x.y, pre));
                    d[2] = make_uint2(bf16x2_to_f16x2_scaled(x.z, pre), bf16x2_to_f16x2_scaled(x.w, pre));
                    if (piece == 0) reinterpret_cast<float *>(smem + C::OFF_QPRE)[rl] = pre;
                }
                asm volatile("bar.arrive 3, 640;" ::: "memory");
                if (tensor == 1) asm volatile("bar.sync 4, 384;" ::: "memory");
            }
            for (int i = 0; i < n_tiles; ++i) {
                // the staged records have landed, and the ring slot's previous tile has been consumed
                bool ok = mbar_wait(&stg_full[i % NSG], (i / NSG) & 1, &flags[0]);
                ok = ok && (i < NR || mbar_wait(&ring_empty[i % NR], ((i / NR) - 1) & 1, &flags[0]));
                if (!__all_sync(0xffffffffu, ok)) {
                    flags[0] = 1;
                    break;
                }
                uint8_t *rec = stg + (i % NSG) * C::STG_BYTES, *ring_rows = ring + (i % NR) * C::TILE_BYTES;
                const int t0 = (c_begin + i * CPT + rc) * kChunk + 8 * half;
                if (tensor == 0) {  // (rows past the tile's end may hold anything: their scores are masked)
                    uint8_t *dst = ring_rows + r * 128;
#pragma unroll
                    for (int j = 0; j < NBL / 8; ++j) {
                        const uint4 kw = *reinterpret_cast<const uint4 *>(rec + (2 * j + half) * 512 + (4 * r + c) * 16);
                        const uint2 sc = *reinterpret_cast<const uint2 *>(rec + 8 * D + (8 * half + r) * NBL + 8 * j);
                        const uint32_t wd[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {  // blocks 8 j + 2 q, + 1
                            uint32_t a[4], s2[2];
                            fp4::e2m1x8_f16(wd[q], a);
                            fp4::e4m3x4_f16(q < 2 ? sc.x : sc.y, s2[0], s2[1]);
                            const uint32_t sv2 = s2[q & 1];
                            const uint4 o = make_uint4(fp4::hmul2_lo(a[0], sv2), fp4::hmul2_lo(a[1], sv2),
                                                       fp4::hmul2_hi(a[2], sv2), fp4::hmul2_hi(a[3], sv2));
                            const int ch = 4 * (4 * j + q) + c;
                            *reinterpret_cast<uint4 *>(dst + (ch >> 3) * (TT * 128) + (((ch & 7) ^ r) << 4)) = o;
                        }
                    }
                } else {
                    // NaN scales of tokens hidden from some rows: noted, and 0 in the staged record
                    if (t0 + 7 > f_last || t0 < w_last) {
                        constexpr int WB = D / 32;  // scale bytes of a lane, both halves'
                        uint8_t *sb = rec + 8 * D + lane * WB;
                        uint32_t found = 0;
#pragma unroll
                        for (int o = 0; o < WB; o += 4)
                            found |= __vcmpeq4(*reinterpret_cast<const uint32_t *>(sb + o) & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        if ((found & (half ? 0xffff0000u : 0x0000ffffu)) != 0) {
#pragma unroll 1
                            for (int o = 0; o < WB; ++o) {
                                const int at = lane * WB + o, blk = (at >> 6) * 4 + ((at >> 2) & 3);
                                const int t = t0 + ((at >> 3) & 6) + (at & 1);
                                if ((at >> 1 & 1) != half || (sb[o] & 0x7f) != 0x7f || t > k_last || t < k_first ||
                                    (t <= f_last && t >= w_last))
                                    continue;
                                const int bit = t > f_last ? t - f_last - 1 : 128 + t - k_first;
                                atomicOr(&nan_bits[blk * 8 + (bit >> 5)], 1u << (bit & 31));
                                flags[2] = 1;
                                sb[o] = 0;
                            }
                            tc::fence_async_smem();  // before the slot's next copy
                        }
                        __syncwarp();
                    }
                    uint32_t wd[2][NBL / 4];  // codes of the lane's tokens 2 c, 2 c + 1
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint8_t *src = rec + (2 * half + u) * 2 * D + lane * NBL;
                        if constexpr (NBL == 16) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(src);
                            wd[u][0] = w.x, wd[u][1] = w.y, wd[u][2] = w.z, wd[u][3] = w.w;
                        } else {
                            const uint2 w = *reinterpret_cast<const uint2 *>(src);
                            wd[u][0] = w.x, wd[u][1] = w.y;
                        }
                    }
                    uint4 sw[NBL / 4];  // scales of blocks 4 w .. 4 w + 3, a word each: tokens 2 c, 2 c + 1 of both halves
#pragma unroll
                    for (int w = 0; w < NBL / 4; ++w)
                        sw[w] = *reinterpret_cast<const uint4 *>(rec + 8 * D + w * 64 + c * 16);
                    // rows outside the block's visible keys may hold anything: their scales become 0
                    if (t0 < k_first || t0 + 8 > t_end) {
                        const int tg = t0 + 2 * c;
                        const uint32_t vm = (tg < t_end && tg >= k_first ? 0x00ff00ffu : 0u) |
                                            (tg + 1 < t_end && tg + 1 >= k_first ? 0xff00ff00u : 0u);
#pragma unroll
                        for (int w = 0; w < NBL / 4; ++w)
                            sw[w] = make_uint4(sw[w].x & vm, sw[w].y & vm, sw[w].z & vm, sw[w].w & vm);
                    }
                    uint8_t *dst = ring_rows + 2 * c * 128;
                    const int p0 = (r ^ (2 * c)) << 4, p1 = (r ^ (2 * c + 1)) << 4;
                    auto store = [&](auto second) {
#pragma unroll
                        for (int w = 0; w < NBL / 4; ++w) {
                            const uint32_t sb[4] = {sw[w].x, sw[w].y, sw[w].z, sw[w].w};
                            uint32_t a[4], s2[4];  // s2: scale pairs of the two tokens
#pragma unroll
                            for (int q = 0; q < 4; ++q) s2[q] = fp4::e4m3x2_f16<decltype(second)::value>(sb[q]);
                            fp4::e2m1x8_f16(wd[0][w], a);
                            *reinterpret_cast<uint4 *>(dst + w * (TT * 128) + p0) =
                                make_uint4(fp4::hmul2_lo(a[0], s2[0]), fp4::hmul2_lo(a[1], s2[1]),
                                           fp4::hmul2_lo(a[2], s2[2]), fp4::hmul2_lo(a[3], s2[3]));
                            fp4::e2m1x8_f16(wd[1][w], a);
                            *reinterpret_cast<uint4 *>(dst + 128 + w * (TT * 128) + p1) =
                                make_uint4(fp4::hmul2_hi(a[0], s2[0]), fp4::hmul2_hi(a[1], s2[1]),
                                           fp4::hmul2_hi(a[2], s2[2]), fp4::hmul2_hi(a[3], s2[3]));
                        }
                    };
                    if (half)
                        store(std::true_type{});
                    else
                        store(std::false_type{});
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&stg_empty[i % NSG]);
                tc::fence_async_smem();  // the tensor core reads the widened tile
                __syncwarp();
                if (lane == 0) mbar_arrive(&ring_full[i % NR]);
            }
        } else if constexpr (F8) {
            // ---------------- fp8: widen staged e4m3 tiles into the K (warps 6, 7) / V (8, 9) ring ----------------
            const int tensor = (warp - C::W0) / C::CW, part = (warp - C::W0) % C::CW;
            constexpr int NR0 = NK, NR1 = NV;
            const int NR = tensor == 0 ? NR0 : NR1;
            uint64_t *ring_full = tensor == 0 ? k_full : p_full;
            uint64_t *ring_empty = tensor == 0 ? k_empty : v_empty;
            uint64_t *stg_full = tensor == 0 ? kst_full : vst_full;
            uint64_t *stg_empty = tensor == 0 ? kst_empty : vst_empty;
            uint8_t *ring = smem + (tensor == 0 ? 0 : C::OFF_V);
            const uint8_t *stg = smem + C::OFF_STG + tensor * NSG * C::STG_BYTES;
            const int t_end = min(L, (c_begin + n_my) * kChunk);
            // A lane widens 16 codes -- 16-byte column j of 128-code block b of
            // token t -- into two 16-byte f16 chunks of the swizzled ring row.
            // The 8 lanes of a shared-memory phase take 8 consecutive tokens of
            // one column (t & 7 = lane & 7), so both the staged reads and the
            // ring writes spread over the 8 bank groups; a lane then walks its
            // column down the tile in steps of 8 tokens (1 KiB in both layouts).
            constexpr int QG = D / 64;  // groups of 4 columns: warp `part` takes every CW-th
            const int t_lo = lane & 7, q_lo = lane >> 3;
            for (int i = 0; i < n_tiles; ++i) {
                // the staged tile has landed, and the ring slot's previous tile has been consumed
                bool ok = __all_sync(0xffffffffu, mbar_wait(&stg_full[i % NSG], (i / NSG) & 1, &flags[0]));
                if (ok && i >= NR)
                    ok = __all_sync(0xffffffffu, mbar_wait(&ring_empty[i % NR], ((i / NR) - 1) & 1, &flags[0]));
                if (!ok) {
                    flags[0] = 1;
                    break;
                }
                const int nvl = min(TT, t_end - (c_begin + i * CPT) * kChunk) - t_lo;  // rows t < nv hold keys
                const uint8_t *stg_tile = stg + (i % NSG) * C::STG_BYTES;
                uint8_t *ring_tile = ring + (i % NR) * C::TILE_BYTES;
                for (int qg = part; qg < QG; qg += C::CW) {
                    const int q = 4 * qg + q_lo, b = q >> 3, j = q & 7, c = (q & 3) * 2;
                    const uint8_t *src = stg_tile + b * (TT * 128) + t_lo * 128 + ((j ^ t_lo) << 4);
                    uint8_t *dst = ring_tile + (q >> 2) * (TT * 128) + t_lo * 128;
                    const int o_lo = (c ^ t_lo) << 4, o_hi = ((c + 1) ^ t_lo) << 4;
#pragma unroll
                    for (int u = 0; u < TT / 8; ++u) {
                        uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                        if (8 * u < nvl) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(src + u * 1024);
                            lo = e4m3x8_to_f16x8(w.x, w.y);
                            hi = e4m3x8_to_f16x8(w.z, w.w);
                        }
                        *reinterpret_cast<uint4 *>(dst + u * 1024 + o_lo) = lo;
                        *reinterpret_cast<uint4 *>(dst + u * 1024 + o_hi) = hi;
                    }
                }
                tc::fence_async_smem();  // the tensor core reads the widened tile
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ring_full[i % NR]);
                    mbar_arrive(&stg_empty[i % NSG]);
                }
            }
        }
    }
    } else {
        // ---------------- softmax: thread = query row = tensor-memory lane ----------------
        if constexpr (C::RSPLIT) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SM));
        if constexpr (F4) {
            // Q, staged by the widening warps (barrier 3), to tensor memory; then the V ring is theirs (barrier 4)
            asm volatile("bar.sync 3, 640;" ::: "memory");
            const uint8_t *qs = smem + C::OFF_V + threadIdx.x * C::QROW;
#pragma unroll 1
            for (int c = 0; c < NQ / 8; ++c) {
                uint32_t r[32];
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(qs + 128 * c + 16 * v);
                    r[4 * v] = w.x, r[4 * v + 1] = w.y, r[4 * v + 2] = w.z, r[4 * v + 3] = w.w;
                }
                tc::st32(lane_base + C::Q_COL + 32 * c, r);
            }
            q_pre = reinterpret_cast<const float *>(smem + C::OFF_QPRE)[threadIdx.x];
            tc::wait_st();
            tc::fence_before();
            asm volatile("bar.arrive 1, 160;" ::: "memory");
            asm volatile("bar.arrive 4, 384;" ::: "memory");
        }
        const int rho = row0 + row_l;  // this thread's row (tensor-memory lane threadIdx.x)
        const bool live = row_l < R;
        const int record = split * COP + copy;  // of the row's num_splits
        // last visible key: the causal limit of the row, and never past this
        // split's last chunk (a tile may reach into the next split's tokens)
        const int t_end = min(L, (c_begin + n_my) * kChunk);
        // (dead rows of a live warp, all zeros, see everything: a mask of their own would send the warp both ways)
        const int lim = !live ? INT_MAX : SH ? t_end - 1 : min(L - p.q_len + rho / G, t_end - 1);
        // a warp without live rows only keeps the phases (its rows of S come from zeros of Q, its rows of O go nowhere)
        const bool idle_warp = F4 && warp * 32 >= R;
        const int lo = !SH && p.window > 0 && live ? L - p.q_len + rho / G - p.window + 1 : 0;  // first key of the row's window
        // fp8: K's scale and the inverse of q's pre-scale (a power of two) join the softmax scale
        const float sl = F8 ? p.scale_log2 * p.k_scale[kvh] * (1.f / q_pre) : p.scale_log2;
        float m_ref = -INFINITY, l_sum = 0.f;
        [[maybe_unused]] float l_low = 0.f;
        // The second sum stands in the warp's own rows of the output, in an order
        // of its own (a lane's float4 j at float4 j * live rows + lane: whole
        // lines per access), and is added to by red while the row's reference max
        // stays.  A kernel of its own: 8 sequences x 16 rows over 8K take 77 us
        // with it and 51 without, 2048 rows over 16K 1344 us (701 with bf16 output);
        // the bytes of the second sum are what it costs (moved by four other warps,
        // or read, added and stored without red: no less).
        [[maybe_unused]] float m_far = -INFINITY;  // the reference max that the second sum stands for
        [[maybe_unused]] const uint32_t my_row =
            live ? (uint32_t)(((row_base + rho / G) * p.num_q_heads + kvh * G + rho % G) * p.num_splits + record) : 0u;
        [[maybe_unused]] const int n_live = min(32, R - (COP > 1 ? warp * 32 % RB : warp * 32));
        [[maybe_unused]] float *far_base = !SH && p.num_splits == 1 ? static_cast<float *>(p.out) : p.part_o;
        [[maybe_unused]] auto far_place = [&](int j) {  // (the whole warp) the lane's float4 j of the second sum
            const int at = j * n_live + min(lane, n_live - 1);
            const uint32_t row = __shfl_sync(0xffffffffu, my_row, at / (D / 4));
            return reinterpret_cast<float4 *>(far_base + (size_t)row * D) + at % (D / 4);
        };
        // O, relative to m_win, joins the second sum.  (Predicated accesses, one loop per kind: branches around every
        // access cost six times the accesses.)
        [[maybe_unused]] auto far_add = [&](float m_win, bool first) {
            const float alpha = m_far == m_win ? 1.f : fast_exp2(m_far - m_win);
            const uint32_t mine = lane < n_live;
            const bool moved = __any_sync(0xffffffffu, mine && m_far != m_win);
            auto add = [&](auto kind) {
                constexpr int KIND = decltype(kind)::value;  // 0: store, 1: red, 2: read, scale, add, store
#pragma unroll 1
                for (int c1 = 0; c1 < D; c1 += 64) {
                    uint32_t r[4][16];
                    [[maybe_unused]] float4 f[KIND == 2 ? 16 : 1];
                    if constexpr (KIND == 2) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) f[j] = __ldcg(far_place(c1 / 4 + j));
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc::ld16_nowait(lane_base + C::O_COL + c1 + 16 * k, r[k]);
                    tc::wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float4 *at = far_place(c1 / 4 + j);
                        float4 v =
                            make_float4(__uint_as_float(r[j / 4][j % 4 * 4]), __uint_as_float(r[j / 4][j % 4 * 4 + 1]),
                                        __uint_as_float(r[j / 4][j % 4 * 4 + 2]), __uint_as_float(r[j / 4][j % 4 * 4 + 3]));
                        if constexpr (KIND == 1) {
                            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                                         "@p red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(at),
                                         "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(mine)
                                         : "memory");
                        } else {
                            if constexpr (KIND == 2)
                                v = make_float4(fmaf(f[j].x, alpha, v.x), fmaf(f[j].y, alpha, v.y),
                                                fmaf(f[j].z, alpha, v.z), fmaf(f[j].w, alpha, v.w));
                            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                                         "@p st.global.cg.v4.f32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(at),
                                         "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(mine)
                                         : "memory");
                        }
                    }
                }
            };
            if (first)
                add(std::integral_constant<int, 0>{});
            else if (!moved)
                add(std::integral_constant<int, 1>{});
            else
                add(std::integral_constant<int, 2>{});
            m_far = m_win;
        };
        bool ok = true;
        // O += P_k V_k of tile k.  S_i being there says that tile i - NSB's
        // product is done (the tensor core ran it first), so a wait for tile
        // i - 1 never tests a phase parity two phases behind the barrier.
        auto wait_pv = [&](int k) {
            return __all_sync(0xffffffffu, mbar_wait(&o_done[k % NSB], (k / NSB) & 1, &flags[0]));
        };
        for (int i = 0; i < n_tiles; ++i) {
            const int j = i % NSB;
            // waits ahead of a warp-collective tensor-memory access end the same way for the whole warp
            if (!__all_sync(0xffffffffu, mbar_wait(&s_full[j], (i / NSB) & 1, &flags[0]))) {
                ok = false;
                break;
            }
            // A 64-key tile keeps its scores in registers from the max to the
            // exponentials (one load); a 128-key tile takes its max over both
            // halves first and loads each half again for P (the one-load form
            // for 128 keys would not fit the registers, and the two-pass form
            // makes the fp8 variants spill).
            if (idle_warp) {
                if (lane == 0) mbar_arrive(&p_full[i % C::NP]);
                continue;
            }
            if constexpr (VPK == 1) {
                tc::fence_after();
                float sv[KPT];
                {
                    uint32_t r[KPT / 16][16];  // the thread's scores: all loads in flight, one wait
#pragma unroll
                    for (int c0 = 0; c0 < KPT / 16; ++c0)
                        tc::ld16_nowait(lane_base + C::SBUF(j) + copy * KPT + 16 * c0, r[c0]);
                    tc::wait_ld();
#pragma unroll
                    for (int c = 0; c < KPT; ++c) sv[c] = __uint_as_float(r[c / 16][c % 16]);
                    if constexpr (C::SPLIT_QK == 2) {
#pragma unroll
                        for (int c0 = 0; c0 < KPT / 16; ++c0)
                            tc::ld16_nowait(lane_base + C::SBUF(j) + TK + copy * KPT + 16 * c0, r[c0]);
                        tc::wait_ld();
#pragma unroll
                        for (int c = 0; c < KPT; ++c) sv[c] += __uint_as_float(r[c / 16][c % 16]);
                    }
                }
                const int t_tile = (c_begin + i * CPT) * kChunk, t0 = t_tile + copy * KPT;
                float mx = -INFINITY;
                // the exponent is 2^(sv * mul - m): raw scores with mul = scale when
                // every key of the tile is visible to this row (no mask, and the
                // max of the scaled scores is the scaled max for scale > 0), else
                // scaled and masked scores with mul = 1
                float mul = 1.f;
                if (sl > 0.f && t0 + KPT - 1 <= lim && t0 >= lo) {
                    float mr[4];  // four chains: one alone is 32 dependent steps
#pragma unroll
                    for (int c = 0; c < 4; ++c) mr[c] = fmax3(sv[c], sv[c + 4], sv[c + 8]);
#pragma unroll
                    for (int c = 12; c + 7 < KPT; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mr[e] = fmax3(mr[e], sv[c + e], sv[c + e + 4]);
                    mr[0] = fmaxf(fmax3(mr[0], sv[KPT - 4], sv[KPT - 3]), sv[KPT - 2]);
                    mx = fmaxf(fmax3(mr[0], mr[1], mr[2]), fmaxf(mr[3], sv[KPT - 1])) * sl;
                    mul = sl;
                    if (SH && fabsf(mx) > kExactLogits) {
#pragma unroll
                        for (int c = 0; c < KPT; ++c) sv[c] *= sl;
                        mul = 1.f;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < KPT; ++c) sv[c] = (t0 + c <= lim && t0 + c >= lo) ? sv[c] * sl : -INFINITY;
#pragma unroll
                    for (int c = 0; c < KPT; c += 2) mx = fmax3(mx, sv[c], sv[c + 1]);
                }
                // lazy rescale: only when the max grows by more than 2^kLazy, and
                // then only after the previous tile's P.V product has finished
                mx -= kBelow;
                const bool raise = mx > m_ref + kLazy;
                const bool need_rescale = raise && m_ref != -INFINITY;
                [[maybe_unused]] const float m_win = m_ref;  // (a window's end: what O stands for)
                if (far_at(i)) {
                    if (need_rescale) {
                        const float alpha = fast_exp2(m_ref - mx);
                        l_sum *= alpha;
                        l_low *= alpha;
                    }
                } else if (__any_sync(0xffffffffu, need_rescale)) {
                    if (!wait_pv(i - 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const float alpha = need_rescale ? fast_exp2(m_ref - mx) : 1.f;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        float ov[16];
                        tc::ld16(lane_base + C::O_COL + c0, ov);
#pragma unroll
                        for (int c = 0; c < 16; ++c) ov[c] *= alpha;
                        tc::st16(lane_base + C::O_COL + c0, ov);
                    }
                    if (need_rescale) {
                        l_sum *= alpha;
                        l_low *= alpha;
                    }
                }
                if (raise) m_ref = mx;
                // The tile may be short or end in a partial chunk: V rows past the
                // end hold stale data (even NaN), and 0 * NaN would reach O through
                // the tensor core, so zero them before the P.V product reads them.
                const int nv = min(TT, t_end - t_tile);
                if (!F8 && nv < TT) {  // (fp8: the widening warp writes those rows as zeros)
                    if (!__all_sync(0xffffffffu, mbar_wait(&v_full[i % NV], (i / NV) & 1, &flags[0]))) {
                        ok = false;
                        break;
                    }
                    uint8_t *vst = smem + C::OFF_V + (i % NV) * C::TILE_BYTES;
                    for (int idx = threadIdx.x; idx < (TT - nv) * C::DB * 8; idx += 128) {
                        const int t = nv + idx / (C::DB * 8), rem = idx % (C::DB * 8);
                        *reinterpret_cast<uint4 *>(vst + (rem >> 3) * (TT * 128) + t * 128 + (rem & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    tc::fence_async_smem();  // zeroed V rows are read by the tensor core
                }
                // P = 2^(s - m) as a bf16 head and a bf16 residual, written over S_i
                // (tokens packed two per column: head in the first 32 columns)
                // with no visible key yet (m = -inf) every p is 0: 2^(x - inf)
                const float m_use = m_ref == -INFINITY ? INFINITY : m_ref;
                float2 ps2 = make_float2(0.f, 0.f);
                uint32_t hw[KPT / 2];
                [[maybe_unused]] uint32_t lw[KPT / 2], xw[PT == 3 ? KPT / 2 : 1];
#pragma unroll
                for (int c = 0; c < KPT / 2; ++c) {
                    const float p0 = fast_exp2(fmaf(sv[2 * c], mul, -m_use));
                    const float p1 = fast_exp2(fmaf(sv[2 * c + 1], mul, -m_use));
                    ps2 = __fadd2_rn(ps2, make_float2(p0, p1));
                    if constexpr (!RES)
                        hw[c] = pack_f16(p0, p1);
                    else if constexpr (PT == 3)
                        split3_bf16(p0, p1, hw[c], lw[c], xw[c]);
                    else if constexpr (F8)
                        split_f16(p0, p1, hw[c], lw[c]);
                    else
                        split_bf16(p0, p1, hw[c], lw[c]);
                }
                if constexpr (FAR) {  // with what the sum's rounding leaves over
                    const float t = ps2.x + ps2.y + l_low, sum = l_sum + t;
                    l_low = t - (sum - l_sum);
                    l_sum = sum;
                } else {
                    l_sum += ps2.x + ps2.y;
                }
                if constexpr (COP > 1) {  // the other copies' keys: no weight
                    const uint32_t none[KPT / 2] = {};
#pragma unroll
                    for (int k = 1; k < COP; ++k)
#pragma unroll
                        for (int h = 0; h < PT; ++h)
                            tc::st_cols(lane_base + C::SBUF(j) + h * (TT / 2) + (copy + k) % COP * (KPT / 2), none);
                }
                tc::st_cols(lane_base + C::SBUF(j) + copy * (KPT / 2), hw);
                if constexpr (RES) tc::st_cols(lane_base + C::SBUF(j) + TT / 2 + copy * (KPT / 2), lw);
                if constexpr (PT == 3) tc::st_cols(lane_base + C::SBUF(j) + TT + copy * (KPT / 2), xw);
                tc::wait_st();
                if constexpr (FAR) {
                    if (far_at(i)) {  // (O is free for P_i V_i once it has been read)
                        if (!wait_pv(i - 1)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after();
                        if (n_live > 0) far_add(m_win, i == kFarTiles);  // (a warp without rows has nothing to move)
                    }
                }
                tc::fence_before();
            } else {
                tc::fence_after();
                const int t0 = (c_begin + i * CPK) * kChunk;        // first key of the score tile
                const int nvt = min(VPK, n_vtiles - i * VPK);       // its 64-key halves with keys of this split
                // The exponent is 2^(sv * mul - m): raw scores with mul = scale when
                // every key of the tile is visible to this row (no mask, and the
                // max of the scaled scores is the scaled max for scale > 0), else
                // scaled and masked scores with mul = 1.
                bool all_visible = sl > 0.f && t0 + TK - 1 <= lim && t0 >= lo;
                float mul = all_visible ? sl : 1.f;
                // 64 scores of half h2 (all loads in flight, one wait), masked and scaled unless all_visible
                float sv[TT];
                auto load_half = [&](int h2) {
                    uint32_t r[TT / 16][16];
#pragma unroll
                    for (int c0 = 0; c0 < TT / 16; ++c0)
                        tc::ld16_nowait(lane_base + C::SBUF(j) + h2 * TT + 16 * c0, r[c0]);
                    tc::wait_ld();
#pragma unroll
                    for (int c = 0; c < TT; ++c) sv[c] = __uint_as_float(r[c / 16][c % 16]);
                    if (!all_visible) {
                        const int th = t0 + h2 * TT;
#pragma unroll
                        for (int c = 0; c < TT; ++c) sv[c] = (th + c <= lim && th + c >= lo) ? sv[c] * sl : -INFINITY;
                    }
                };
                auto half_max = [&]() {
                    float mh;
                    if (all_visible) {
                        mh = sv[0];
#pragma unroll
                        for (int c = 1; c + 1 < TT; c += 2) mh = fmax3(mh, sv[c], sv[c + 1]);
                        mh = fmaxf(mh, sv[TT - 1]) * sl;
                    } else {
                        mh = -INFINITY;
#pragma unroll
                        for (int c = 0; c < TT; c += 2) mh = fmax3(mh, sv[c], sv[c + 1]);
                    }
                    return mh;
                };
                float mx = -INFINITY;
                for (int h2 = 0; h2 < nvt; ++h2) {  // the tile's max, over every half
                    load_half(h2);
                    mx = fmaxf(mx, half_max());
                }
                if (SH && fabsf(mx) > kExactLogits) {
                    all_visible = false;
                    mul = 1.f;
                }
                // lazy rescale: only when the max grows by more than 2^kLazy, and
                // then only after the previous tile's P.V product has finished
                const bool raise = mx > m_ref + kLazy;
                const bool need_rescale = raise && m_ref != -INFINITY;
                if (__any_sync(0xffffffffu, need_rescale)) {
                    if (!wait_pv(i - 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const float alpha = need_rescale ? fast_exp2(m_ref - mx) : 1.f;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        float ov[16];
                        tc::ld16(lane_base + C::O_COL + c0, ov);
#pragma unroll
                        for (int c = 0; c < 16; ++c) ov[c] *= alpha;
                        tc::st16(lane_base + C::O_COL + c0, ov);
                    }
                    if (need_rescale) l_sum *= alpha;
                }
                if (raise) m_ref = mx;
                // A V tile may be short or end in a partial chunk: V rows past the
                // end hold stale data (even NaN), and 0 * NaN would reach O through
                // the tensor core, so zero them before the P.V product reads them.
                bool zero_ok = true;
                for (int h2 = 0; h2 < nvt && !F8; ++h2) {  // (fp8: the widening warp writes those rows as zeros)
                    const int vt = i * VPK + h2;
                    const int nv = min(TT, t_end - (t0 + h2 * TT));
                    if (nv >= TT) continue;
                    if (!__all_sync(0xffffffffu, mbar_wait(&v_full[vt % NV], (vt / NV) & 1, &flags[0]))) {
                        zero_ok = false;
                        break;
                    }
                    uint8_t *vst = smem + C::OFF_V + (vt % NV) * C::TILE_BYTES;
                    for (int idx = threadIdx.x; idx < (TT - nv) * C::DB * 8; idx += 128) {
                        const int t = nv + idx / (C::DB * 8), rem = idx % (C::DB * 8);
                        *reinterpret_cast<uint4 *>(vst + (rem >> 3) * (TT * 128) + t * 128 + (rem & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    tc::fence_async_smem();  // zeroed V rows are read by the tensor core
                }
                if (!zero_ok) {
                    ok = false;
                    break;
                }
                // P = 2^(s - m) per 64-key half as a bf16 head and a bf16 residual,
                // written over that half's S columns (tokens packed two per column:
                // head in the first 32 columns); with no visible key yet (m = -inf)
                // every p is 0: 2^(x - inf)
                const float m_use = m_ref == -INFINITY ? INFINITY : m_ref;
                for (int h2 = 0; h2 < nvt; ++h2) {
                    if (VPK > 1) load_half(h2);  // (one half: its scores are still in sv)
                    float2 ps2 = make_float2(0.f, 0.f);
                    uint32_t hw[TT / 2], lw[TT / 2];
#pragma unroll
                    for (int c = 0; c < TT / 2; ++c) {
                        const float p0 = fast_exp2(fmaf(sv[2 * c], mul, -m_use));
                        const float p1 = fast_exp2(fmaf(sv[2 * c + 1], mul, -m_use));
                        ps2 = __fadd2_rn(ps2, make_float2(p0, p1));
                        if constexpr (F8)
                            split_f16(p0, p1, hw[c], lw[c]);
                        else
                            split_bf16(p0, p1, hw[c], lw[c]);
                    }
                    l_sum += ps2.x + ps2.y;
                    tc::st32(lane_base + C::SBUF(j) + h2 * TT, hw);
                    tc::st32(lane_base + C::SBUF(j) + h2 * TT + TT / 2, lw);
                }
                tc::wait_st();
                tc::fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[i % C::NP]);
        }
        // Epilogue: wait for the last P.V MMA, normalise and write this row.
        if (ok && !wait_pv(n_tiles - 1)) ok = false;
        ok = __all_sync(0xffffffffu, ok);  // the loads below are warp-collective
        if (!ok) flags[0] = 1;
        tc::fence_after();
        const bool poisoned = !ok || flags[1] != 0;
        const float inv = (poisoned || !(l_sum > 0.f)) ? 0.f : (F8 ? p.v_scale[kvh] : 1.f) / l_sum;
        const size_t orow = live ? (row_base + rho / G) * p.num_q_heads + kvh * G + rho % G : 0;
        [[maybe_unused]] auto sees_nan = [&](int blk) {  // the row sees a token of nan_bits in this scale block
            const int f_next = L - p.q_len + row0 / G + 1;
            bool hit = false;
            for (int w = 0; w < 8; ++w) {
                for (uint32_t bits = nan_bits[blk * 8 + w]; bits != 0; bits &= bits - 1) {
                    const int t = (w < 4 ? f_next + w * 32 : k_first + (w - 4) * 32) + __ffs(bits) - 1;
                    hit |= t >= lo && t <= lim;
                }
            }
            return hit;
        };
        const bool direct = !SH && p.num_splits == 1;  // the final output, else this split's record
        if (FAR && !ok) {  // (other lanes' parts of the second sum may be on their way to this row)
            __threadfence();
            __syncwarp();
        }
        if (ok) {
            // Every tile has been consumed by the tensor core, so the K/V rings
            // are free: the row is staged there (rows SROW bytes apart, so the
            // 16-byte stores of 8 consecutive rows fall in 8 different bank
            // groups) and leaves with one bulk copy, instead of a warp's 32
            // rows going out as 32 separate segments per store.
            const bool bf = direct && p.out_bf16;
            uint8_t *srow = smem + threadIdx.x * C::SROW;
            [[maybe_unused]] const float far_w = m_far == m_ref ? 1.f : fast_exp2(m_far - m_ref);
            [[maybe_unused]] const bool some_nan = F4 && flags[2] != 0;
#pragma unroll 1
            for (int c1 = 0; c1 < D; c1 += 64) {
                uint32_t r[4][16];  // 64 columns: four loads in flight, one wait
#pragma unroll
                for (int k = 0; k < 4; ++k) tc::ld16_nowait(lane_base + C::O_COL + c1 + 16 * k, r[k]);
                tc::wait_ld();
                if constexpr (FAR) {
                    if (n_tiles > kFarTiles && n_live > 0) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float4 *at = far_place(c1 / 4 + j);
                            const float4 f = __ldcg(at);
                            const float fv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t &o = r[j / 4][j % 4 * 4 + e];
                                o = __float_as_uint(fmaf(fv[e], far_w, __uint_as_float(o)));
                            }
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c0 = c1 + 16 * k;
                    float ov[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if constexpr (F4) {  // column 8 r' + 2 q + e of a 64-dim group holds dim 16 q + 2 r' + e
                            const int col = (c >> 1) * 8 + 2 * k + (c & 1);
                            const float o = __uint_as_float(r[col >> 4][col & 15]);
                            // (a bad page's stand-in may hold NaN)
                            ov[c] = poisoned ? 0.f : o * inv;
                        } else {
                            ov[c] = __uint_as_float(r[k][c]) * inv;
                        }
                    }
                    if constexpr (F4) {
                        if (some_nan && !poisoned && sees_nan(c0 / 16)) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) ov[c] = NAN;
                        }
                    }
                    if (bf) {
                        uint32_t w[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) w[c] = pack_bf16(ov[2 * c], ov[2 * c + 1]);
                        *reinterpret_cast<uint4 *>(srow + 2 * c0) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4 *>(srow + 2 * c0 + 16) = make_uint4(w[4], w[5], w[6], w[7]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; c += 4)
                            *reinterpret_cast<float4 *>(srow + 4 * (c0 + c)) =
                                make_float4(ov[c], ov[c + 1], ov[c + 2], ov[c + 3]);
                    }
                }
            }
            if constexpr (FAR) {  // the second sum has been read by the whole warp, before any of its rows is written
                asm volatile("fence.proxy.async.global;" ::: "memory");
                __syncwarp();
            }
            if (live) {
                tc::fence_async_smem();  // the staged row is read by the copy engine
                uint8_t *dst = direct ? static_cast<uint8_t *>(p.out) + orow * D * (bf ? 2 : 4)
                                      : reinterpret_cast<uint8_t *>(p.part_o + (orow * p.num_splits + record) * D);
                bulk_store_s2g(dst, srow, bf ? D * 2 : D * 4);
                bulk_commit();
                bulk_wait_read();  // the row has left shared memory before the CTA ends
            }
        } else if (live) {
            // a wait was abandoned (copies may still land in the rings): zero the row with plain stores
#pragma unroll 1
            for (int c = 0; c < D; ++c) {
                if (direct)
                    store_out(p.out, orow * D + c, 0.f, p.out_bf16);
                else
                    p.part_o[(orow * p.num_splits + record) * D + c] = 0.f;
            }
        }
        if (SH && live) {
            const int state = row_state(rho);
            p.part_ml[orow * p.num_splits + record] = poisoned || state == 2 ? make_float2(m_ref, -1.f)
                                                      : state == 1          ? make_float2(-INFINITY, 0.f)
                                                      : l_sum != l_sum      ? make_float2(0.f, 1.f)
                                                                            : make_float2(m_ref, l_sum);
        } else if (live && !direct)
            // (F4: a NaN sum goes on as a NaN row with max 0 and sum 1: the reduce takes a sum that is not > 0 for
            // an empty split, and the max may be infinite)
            p.part_ml[orow * p.num_splits + record] = poisoned                 ? make_float2(m_ref, -1.f)
                                                     : F4 && l_sum != l_sum ? make_float2(0.f, 1.f)
                                                                            : make_float2(m_ref, l_sum);
    }

    tc::fence_before();
    __syncthreads();
    if (warp == 4) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

}  // namespace pa
