// shared_pages.cu -- cache pages that several requests hold: forking a request
// (its full pages get one more holder, its partly filled last page is copied),
// releasing requests (a page returns to the pool with its last holder),
// compacting the pool, and copying pages inside the caches.
//
// share_counts[p] is the number of holders of page p beyond the first, so a
// page of one request has 0 and the calls of block_tables.cu need not know it.
//
// All are integer work, bound by launches and by a few dependent loads.  Counts
// change by atomic adds of whole numbers, whose order does not show; freed pages
// enter the pool in ascending order, whichever request held them last, which
// takes a prefix sum over the pages.  The outputs are buffers of their own, so that
// a replayed call gives the same again.
//
// What bounds them is the chain of launches and of dependent loads.  A release
// and a compaction are one cluster of CTAs (and the rewriting of the tables): the
// pages are spread over the CTAs' shared memories, those of 8 hold 409,600, an entry
// of a block table adds to its page's counter there, and the sums pass through
// distributed shared memory.  Where a cluster would take long to walk the pages and
// the tables, a release goes through kernels that fill the GPU: one copies the
// counts, the next adds to them, a cluster scans.  A fork has nothing to scan; it
// takes two such kernels at any size.  Scans of many pages take 16 CTAs.
// (us per call, requests x pages per request of a pool of so many pages, release
// by one cluster / by three kernels: 64 x 40, 1.2K: 4.9 / 8.0; 256 x 100, 15K: 6.4 /
// 9.0; 256 x 300, 60K: 12 / 9.9.  Compaction by 8 / 16 CTAs: 15K: 11.0 / 10.9; 60K:
// 18.9 / 14.2; 286K: 33.5 / 26.0.  Release by three kernels, 60K: 9.9 / 10.4; 90K: 13.7
// / 10.5; 286K: 28.9 / 21.1.  Fork 4.6 us for 8 requests, 10.0 for 1000 x 600; as one
// cluster it took 6.9 and 12.)
#include <algorithm>

#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kShareThreads = 256;
constexpr int kShareCtas = 304;       // two per SM
constexpr int kScanCtas = 8;          // CTAs of the cluster that scans the pages
constexpr int kScanWide = 16;         // the same, of many pages, where the device has room for it
constexpr int64_t kWideCompact = 16 * 1024, kWideRelease = 64 * 1024;  // from more pages on
constexpr int kScanThreads = 1024;
constexpr int kScanItems = 8;         // pages per thread and step
constexpr int kClusterPages = 50 * 1024;         // counters of a CTA of the cluster (200 KiB)
constexpr int64_t kClusterMost = 64 * 1024;      // pages, and entries of the block table, of a release by one cluster
constexpr int kCopyThreads = 256;
constexpr int kCopyPiece = 16 * 1024; // bytes that a CTA copies at a time: four 16-byte loads per thread
constexpr int kCopyCtas = 152 * 8;

struct ShareParams {
    const int32_t *lens;      // [B]
    const int32_t *count;     // [B] fork: parent; release: non-zero = finished
    int32_t *table;           // [B, width]
    int32_t *free_pages;      // [P]
    const int32_t *num_free;  // [1]
    const int32_t *shares;    // [P]
    int32_t *lens_out;        // [B]
    int32_t *shares_out;      // [P]
    int32_t *num_free_out;    // [1]
    int32_t *src, *dst, *tokens;  // fork: [B]; compact: [M] (no tokens)
    int32_t *free_out, *page_map, *extent;  // compact: [P], [P], [1]
    int32_t *status;
    int64_t num_pages;
    int B, width, block_size, moves;
};

__device__ __forceinline__ int64_t room_of(const ShareParams &p) { return (int64_t)p.width * p.block_size; }

__device__ __forceinline__ int pool_of(const ShareParams &p, bool flag) {
    const int f = p.num_free[0];
    const int F = (int)max((int64_t)0, min((int64_t)f, p.num_pages));
    if (flag && F != f) set_status(p.status, PA_DEV_BAD_PAGE);
    return F;
}

__device__ __forceinline__ bool valid_page(const ShareParams &p, int page) { return page >= 0 && page < p.num_pages; }

// For i = first, first + stride, ... below n: use(i, load(i)), eight loads at a
// time (one by one, every step would wait for its own).
template <typename I, typename Load, typename Use>
__device__ __forceinline__ void for_each(I first, I n, I stride, Load load, Use use) {
    constexpr int U = 8;
    for (I i0 = first; i0 < n; i0 += U * stride) {
        int v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * stride < n) v[u] = load(i0 + u * stride);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * stride < n) use(i0 + u * stride, v[u]);
    }
}

__device__ __forceinline__ void copy_shares(const ShareParams &p) {
    for_each((int64_t)blockIdx.x * blockDim.x + threadIdx.x, p.num_pages, (int64_t)gridDim.x * blockDim.x,
             [&](int64_t i) { return p.shares[i]; }, [&](int64_t i, int v) { p.shares_out[i] = v; });
}

// Sum of v over the CTA (every thread gets it); `tmp`: 32 words.
__device__ __forceinline__ int block_sum(int v, int *tmp) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += tmp[w];
    return s;
}

// Sum of v over the threads before this one, and over all in `total`.
__device__ __forceinline__ int block_before(int v, int *tmp, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, k);
        if (lane >= k) incl += o;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        const int s = tmp[w];
        if (w < warp) before += s;
        total += s;
    }
    return before + incl - v;
}

// ---- fork ---------------------------------------------------------------------

// What request b asks for: a child of `parent` that holds `len` tokens.
struct Child {
    int parent, len;
    bool is, ok;
};
__device__ __forceinline__ Child child_of(const ShareParams &p, int b) {
    Child c{p.count[b], 0, false, false};
    c.is = c.parent >= 0;
    if (!c.is || c.parent >= p.B || c.parent == b) return c;
    c.len = p.lens[c.parent];
    c.ok = p.count[c.parent] < 0 && p.lens[b] == 0 && c.len >= 0 && c.len <= room_of(p);
    return c;
}
__device__ __forceinline__ int wants(const ShareParams &p, const Child &c) {
    return c.ok && c.len % p.block_size != 0 ? 1 : 0;
}

// Each CTA takes `per` requests in a row and sums what those before them want.
__global__ void __launch_bounds__(kShareThreads) pa_fork_tables_kernel(const ShareParams p, int per) {
    pdl_launch_dependents();  // the counting kernel; none behind it starts before that has ended
    pdl_wait_primary();
    __shared__ int tmp[32];
    struct Job {
        int b, parent, full, page;  // page: the new last page, -2: none wanted, -1: refused
    };
    __shared__ Job jobs[kShareThreads];
    const int b0 = blockIdx.x * per, t = threadIdx.x;
    copy_shares(p);
    if (b0 >= p.B) {
        if (blockIdx.x == 0 && t == 0) p.num_free_out[0] = pool_of(p, true);  // no request at all
        return;
    }
    int mine = 0;
    for (int b = t; b < b0; b += kShareThreads) mine += wants(p, child_of(p, b));
    const int before = block_sum(mine, tmp);
    const int F = pool_of(p, blockIdx.x == 0 && t == 0), b = b0 + t;
    const bool in = t < per && b < p.B;
    Child c{-1, 0, false, false};
    if (in) c = child_of(p, b);
    const int want = wants(p, c);
    int total;
    const int upto = before + block_before(want, tmp, total) + want;
    if (t < per) {
        Job j{b, c.parent, c.ok ? c.len / p.block_size : 0, -2};
        if (want) j.page = upto <= F ? p.free_pages[F - upto] : -1;
        const bool served = c.ok && (!want || upto <= F);
        if (!served) j.parent = -1;
        jobs[t] = j;
        if (in) {
            const int len = p.lens[b];
            int bits = 0;
            if (c.is ? !c.ok : (len < 0 || len > room_of(p))) bits |= PA_DEV_BAD_SEQLEN;
            if (c.ok && !served) bits |= PA_DEV_NO_PAGES;
            const bool part = served && want;
            if (part && !valid_page(p, j.page)) bits |= PA_DEV_BAD_PAGE;
            p.lens_out[b] = served ? c.len : max(len, 0);
            p.src[b] = part ? p.table[(int64_t)c.parent * p.width + j.full] : -1;
            p.dst[b] = part ? j.page : -1;
            p.tokens[b] = part ? c.len % p.block_size : 0;
            if (part) p.table[(int64_t)b * p.width + j.full] = j.page;
            if (bits) set_status(p.status, bits);
        }
    }
    __syncthreads();
    for (int i = 0; i < per && b0 + i < p.B; ++i) {
        const Job j = jobs[i];
        if (j.parent < 0) continue;
        const int32_t *from = p.table + (int64_t)j.parent * p.width;
        int32_t *to = p.table + (int64_t)j.b * p.width;
        for (int e = t; e < j.full; e += kShareThreads) to[e] = from[e];
    }
    if (t == 0 && b0 + per >= p.B) p.num_free_out[0] = F - min(F, before + total);
}

// One more holder for every full page of a child.
__global__ void __launch_bounds__(kShareThreads) pa_fork_counts_kernel(const ShareParams p) {
    pdl_wait_primary();  // (no early launch of dependents: a kernel behind may read tables ahead of the stream order)
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const Child c = child_of(p, b);
        if (!c.ok || (c.len % p.block_size != 0 && p.tokens[b] == 0)) continue;  // no child, or refused
        const int full = c.len / p.block_size;
        for (int e = threadIdx.x; e < full; e += kShareThreads) {
            const int page = p.table[(int64_t)c.parent * p.width + e];
            if (valid_page(p, page))
                atomicAdd(p.shares_out + page, 1);
            else
                set_status(p.status, PA_DEV_BAD_PAGE);
        }
    }
}

// ---- release ------------------------------------------------------------------

__device__ __forceinline__ int held_pages(const ShareParams &p, int b) {  // of a finished request
    const int len = p.lens[b];
    if (p.count[b] == 0 || len < 0 || len > room_of(p)) return 0;
    return (int)(((int64_t)len + p.block_size - 1) / p.block_size);
}

__global__ void __launch_bounds__(kShareThreads) pa_release_lens_kernel(const ShareParams p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    copy_shares(p);
    for (int b = blockIdx.x * kShareThreads + threadIdx.x; b < p.B; b += gridDim.x * kShareThreads) {
        const int len = p.lens[b];
        if (len < 0 || len > room_of(p)) set_status(p.status, PA_DEV_BAD_SEQLEN);
        p.lens_out[b] = p.count[b] != 0 ? 0 : max(len, 0);
    }
}

__global__ void __launch_bounds__(kShareThreads) pa_release_counts_kernel(const ShareParams p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const int held = held_pages(p, b);
        for (int e = threadIdx.x; e < held; e += kShareThreads) {
            const int page = p.table[(int64_t)b * p.width + e];
            if (valid_page(p, page))
                atomicSub(p.shares_out + page, 1);
            else
                set_status(p.status, PA_DEV_BAD_PAGE);
        }
    }
}

// ---- a cluster's sums ---------------------------------------------------------

// The kernels that scan are one cluster of CTAS CTAs.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// Every CTA of the cluster gives v (the same in all of its threads) and gets
// all of them in box[0 .. CTAS); a box is used once.  A CTA may leave after
// its last one: what others write into its shared memory is there by then.
template <int CTAS>
__device__ __forceinline__ void cluster_share(int v, int *box) {
    if (threadIdx.x < CTAS) {
        uint32_t there;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_addr(box + blockIdx.x)), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(v) : "memory");
    }
    cluster_sync();
}

// The pages of this CTA: a contiguous share, whole steps of the CTA.
struct Span {
    int64_t lo, hi;
};
template <int CTAS>
__device__ __forceinline__ Span span_of(int64_t pages) {
    const int64_t step = kScanThreads * kScanItems;
    const int64_t per = (pages + step * CTAS - 1) / (step * CTAS) * step;
    const int64_t lo = min(pages, per * blockIdx.x);
    return {lo, min(pages, lo + per)};
}

// The pages of a CTA as counters in its shared memory: page p is counter p -
// rank * per of CTA rank = p / per.
struct Counters {
    uint32_t base;   // shared-memory address in this CTA
    int lo, n, per;  // the CTA's pages [lo, lo + n)
};
template <int CTAS>
__device__ __forceinline__ Counters counters_of(const ShareParams &p, int32_t *smem) {
    const int per = ((int)((p.num_pages + CTAS - 1) / CTAS) + 3) & ~3;
    const int lo = (int)min(p.num_pages, (int64_t)per * blockIdx.x);
    return {smem_addr(smem), lo, (int)min((int64_t)per, p.num_pages - lo), per};
}
__device__ __forceinline__ uint32_t counter_at(const Counters &c, int page) {
    const int rank = page / c.per;
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(c.base + 4u * (uint32_t)(page - rank * c.per)), "r"(rank));
    return there;
}
__device__ __forceinline__ void counter_add(const Counters &c, int page, int v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(counter_at(c, page)), "r"(v) : "memory");
}

// A thread's share of the CTA's pages for a scan: [lo, hi), relative to the CTA's first.
struct Share {
    int lo, hi;
};
__device__ __forceinline__ Share share_of(int n) {
    const int per = (n + kScanThreads - 1) / kScanThreads | 1;  // (odd: a warp's lanes meet 32 banks)
    const int lo = min(n, (int)threadIdx.x * per);
    return {lo, min(n, lo + per)};
}

// Sum of v over the CTAs before this one (and the threads before this one, which
// block_before gave), and over all: `box` is used once.
template <int CTAS>
__device__ __forceinline__ int cluster_before(int total, int *box, int &all) {
    cluster_share<CTAS>(total, box);
    int before = 0;
    all = 0;
    for (int c = 0; c < CTAS; ++c) {
        if (c < (int)blockIdx.x) before += box[c];
        all += box[c];
    }
    return before;
}

template <int CTAS>
__global__ void __launch_bounds__(kScanThreads) pa_release_cluster_kernel(const ShareParams p) {
    pdl_wait_primary();  // (no early launch of dependents, as above)
    extern __shared__ int32_t counts[];
    __shared__ int tmp[32];
    __shared__ int box[CTAS];
    const Counters c = counters_of<CTAS>(p, counts);
    for_each((int)threadIdx.x, c.n, kScanThreads, [&](int i) { return p.shares[c.lo + i]; },
             [&](int i, int v) { counts[i] = v; });
    const int F = pool_of(p, blockIdx.x == 0 && threadIdx.x == 0);
    cluster_sync();
    // a warp per request
    for (int b = blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5); b < p.B; b += CTAS * (kScanThreads / 32)) {
        const int len = p.lens[b], done = p.count[b];
        const bool ok = len >= 0 && len <= room_of(p);
        if ((threadIdx.x & 31) == 0) {
            if (!ok) set_status(p.status, PA_DEV_BAD_SEQLEN);
            p.lens_out[b] = done != 0 ? 0 : max(len, 0);
        }
        const int held = ok && done != 0 ? (int)(((int64_t)len + p.block_size - 1) / p.block_size) : 0;
        for (int e = threadIdx.x & 31; e < held; e += 32) {
            const int page = p.table[(int64_t)b * p.width + e];
            if (valid_page(p, page))
                counter_add(c, page, -1);
            else
                set_status(p.status, PA_DEV_BAD_PAGE);
        }
    }
    cluster_sync();
    const Share s = share_of(c.n);
    int mine = 0;
    for (int i = s.lo; i < s.hi; ++i) mine += counts[i] < 0;
    int total;
    const int in_cta = block_before(mine, tmp, total);
    int all;
    int64_t to = (int64_t)F + cluster_before<CTAS>(total, box, all) + in_cta;
    if (mine > 0) {
        for (int i = s.lo; i < s.hi; ++i) {
            if (counts[i] >= 0) continue;
            // released more often than it was held, or more pages than the pool has
            if (counts[i] < -1 || to >= p.num_pages) set_status(p.status, PA_DEV_BAD_PAGE);
            if (to < p.num_pages) p.free_pages[to] = c.lo + i;
            ++to;
        }
    }
    for (int i = threadIdx.x; i < c.n; i += kScanThreads) p.shares_out[c.lo + i] = max(counts[i], 0);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.num_free_out[0] = (int)min((int64_t)F + all, p.num_pages);
}

// (grid = one cluster)
template <int CTAS>
__global__ void __launch_bounds__(kScanThreads) pa_release_pool_kernel(const ShareParams p) {
    pdl_wait_primary();  // (no early launch of dependents, as above)
    __shared__ int tmp[32];
    __shared__ int box[CTAS];
    const Span s = span_of<CTAS>(p.num_pages);
    const int F = pool_of(p, blockIdx.x == 0 && threadIdx.x == 0);
    cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
    int mine = 0;
    for_each(s.lo + threadIdx.x, s.hi, (int64_t)kScanThreads, [&](int64_t i) { return __ldcg(p.shares_out + i); },
             [&](int64_t, int v) { mine += v < 0; });
    cluster_share<CTAS>(block_sum(mine, tmp), box);
    int64_t at = F, all = F;
    for (int c = 0; c < CTAS; ++c) {
        if (c < (int)blockIdx.x) at += box[c];
        all += box[c];
    }
    for (int64_t i0 = s.lo; i0 < s.hi; i0 += kScanThreads * kScanItems) {
        const int64_t i = i0 + threadIdx.x * kScanItems;
        int n = 0, v[kScanItems];
#pragma unroll
        for (int k = 0; k < kScanItems; ++k) {
            v[k] = i + k < s.hi ? __ldcg(p.shares_out + i + k) : 0;
            n += v[k] < 0;
        }
        int total;
        int64_t to = at + block_before(n, tmp, total);
        at += total;
#pragma unroll
        for (int k = 0; k < kScanItems; ++k) {
            if (v[k] >= 0) continue;
            p.shares_out[i + k] = 0;
            // released more often than it was held, or more pages than the pool has
            if (v[k] < -1 || to >= p.num_pages) set_status(p.status, PA_DEV_BAD_PAGE);
            if (to < p.num_pages) p.free_pages[to] = (int)(i + k);
            ++to;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.num_free_out[0] = (int)min(all, p.num_pages);
}

// ---- compaction ---------------------------------------------------------------
// With n pages in use (not on the free list), those with index >= n move into
// the free pages below n: the highest into the lowest, at most `moves` of them.
// With before(p) = pages in use below p:
//   a page in use is the (n - 1 - before(p))-th from the top,
//   a free page the (p - before(p))-th from the bottom;
// as many free pages lie below n as pages in use lie above, so the k-th of the
// one kind goes with the k-th of the other.  After m moves, before(p) has grown
// by the free pages filled below p and lost the moved ones, which places every
// free page on the new list without a second scan.
// The marks and the ranks stand in the cluster's shared memory; a thread scans a
// stretch of pages of its own.  40,000 pages with 4096 moves: 12 us, half of it the
// barriers of the cluster and the waits for the counters of other CTAs; the copies
// that the call lists take three times as long.
template <int CTAS>
__global__ void __launch_bounds__(kScanThreads) pa_compact_cluster_kernel(const ShareParams p) {
    pdl_launch_dependents();  // (the kernel behind this one rewrites the tables and is the call's last)
    pdl_wait_primary();
    extern __shared__ int32_t used[];
    __shared__ int tmp[32];
    __shared__ int box[3][CTAS];
    __shared__ int top;
    const int P = (int)p.num_pages;
    const Counters c = counters_of<CTAS>(p, used);
    const int F = pool_of(p, blockIdx.x == 0 && threadIdx.x == 0);
    const int tid = blockIdx.x * kScanThreads + threadIdx.x;
    constexpr int stride = CTAS * kScanThreads;
    if (threadIdx.x == 0) top = 0;
    for (int i = threadIdx.x; i < c.n; i += kScanThreads) used[i] = 1;
    cluster_sync();
    for_each(tid, F, stride, [&](int i) { return p.free_pages[i]; }, [&](int, int page) {
        if (valid_page(p, page))
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(counter_at(c, page)), "r"(0) : "memory");
        else
            set_status(p.status, PA_DEV_BAD_PAGE);
    });
    cluster_arrive();
    for_each((int)threadIdx.x, c.n, kScanThreads, [&](int i) { return p.shares[c.lo + i]; }, [&](int i, int v) {
        __stcg(p.page_map + c.lo + i, c.lo + i);
        __stcg(p.shares_out + c.lo + i, v);
    });
    cluster_wait();
    const Share s = share_of(c.n);
    int mine = 0;
    for (int i = s.lo; i < s.hi; ++i) mine += used[i];
    int total;
    const int in_cta = block_before(mine, tmp, total);
    int n;  // (pages are fewer than 2^19 here)
    int bef = cluster_before<CTAS>(total, box[0], n) + in_cta;
    mine = 0;
    for (int i = max(s.lo, n - c.lo); i < s.hi; ++i) mine += used[i];
    int m;
    cluster_before<CTAS>(block_sum(mine, tmp), box[1], m);
    m = min(m, p.moves);
    const int n_free = P - n;
    int highest = 0;
    for (int i = s.lo; i < s.hi; ++i) {
        const int page = c.lo + i, u = used[i];
        const int rank = u ? n - 1 - bef : page - bef;  // from the top, from the bottom
        const bool moves = rank < m && (u ? page >= n : page < n);
        if (moves) __stcg((u ? p.src : p.dst) + rank, page);
        if ((u != 0) != moves) {  // in use from now on
            highest = page + 1;
        } else {
            const int in_use = bef + min(m, page - bef) - max(0, bef - (n - m));
            p.free_out[n_free - 1 - (page - in_use)] = page;
        }
        bef += u;
    }
    for (int64_t i = m + tid; i < p.moves; i += stride) p.src[i] = p.dst[i] = -1;
    for (int i = n_free + tid; i < P; i += stride) p.free_out[i] = -1;
    highest = __reduce_max_sync(0xffffffffu, highest);
    if ((threadIdx.x & 31) == 0) atomicMax(&top, highest);
    __syncthreads();
    cluster_share<CTAS>(top, box[2]);  // (also: every move is listed)
    for (int64_t i = tid; i < m; i += stride) {
        const int from = __ldcg(p.src + i), to = __ldcg(p.dst + i), held = p.shares[from];
        __stcg(p.page_map + from, to);
        __stcg(p.shares_out + to, held);
        __stcg(p.shares_out + from, 0);
    }
    if (tid == 0) {
        int e = 0;
        for (int k = 0; k < CTAS; ++k) e = max(e, box[2][k]);
        p.extent[0] = e;
        p.num_free_out[0] = (int)n_free;
    }
}

// The same for more pages than the cluster's shared memory holds.
template <int CTAS>
__global__ void __launch_bounds__(kScanThreads) pa_compact_pool_kernel(const ShareParams p) {
    pdl_launch_dependents();  // (the kernel behind this one rewrites the tables and is the call's last)
    pdl_wait_primary();
    __shared__ int tmp[32];
    __shared__ int box[3][CTAS];
    __shared__ int top;
    const int64_t P = p.num_pages;
    const Span s = span_of<CTAS>(P);
    const int F = pool_of(p, blockIdx.x == 0 && threadIdx.x == 0);
    const int64_t tid = (int64_t)blockIdx.x * kScanThreads + threadIdx.x, stride = CTAS * kScanThreads;
    if (threadIdx.x == 0) top = 0;
    // page_map holds the marks until the pages are placed: 1 = in use
    for (int64_t i = s.lo + threadIdx.x; i < s.hi; i += kScanThreads) __stcg(p.page_map + i, 1);
    cluster_sync();
    for (int64_t i = tid; i < F; i += stride) {
        const int page = p.free_pages[i];
        if (valid_page(p, page))
            __stcg(p.page_map + page, 0);
        else
            set_status(p.status, PA_DEV_BAD_PAGE);
    }
    cluster_sync();
    int mine = 0;
    auto mark = [&](int64_t i) { return __ldcg(p.page_map + i); };
    for_each(s.lo + threadIdx.x, s.hi, (int64_t)kScanThreads, mark, [&](int64_t, int v) { mine += v; });
    cluster_share<CTAS>(block_sum(mine, tmp), box[0]);
    int64_t before = 0, n = 0;
    for (int c = 0; c < CTAS; ++c) {
        if (c < (int)blockIdx.x) before += box[0][c];
        n += box[0][c];
    }
    mine = 0;
    for_each(max(s.lo, n) + threadIdx.x, s.hi, (int64_t)kScanThreads, mark, [&](int64_t, int v) { mine += v; });
    cluster_share<CTAS>(block_sum(mine, tmp), box[1]);
    int64_t m = 0;
    for (int c = 0; c < CTAS; ++c) m += box[1][c];
    m = min(m, (int64_t)p.moves);
    const int64_t n_free = P - n;
    int highest = 0;
    for (int64_t i0 = s.lo; i0 < s.hi; i0 += kScanThreads * kScanItems) {
        const int64_t i = i0 + threadIdx.x * kScanItems;
        int used[kScanItems], sum = 0;
#pragma unroll
        for (int k = 0; k < kScanItems; ++k) {
            used[k] = i + k < s.hi ? __ldcg(p.page_map + i + k) : 0;
            sum += used[k];
        }
        int total;
        int64_t bef = before + block_before(sum, tmp, total);
        before += total;
#pragma unroll
        for (int k = 0; k < kScanItems; ++k) {
            const int64_t page = i + k;
            if (page >= s.hi) break;
            const int64_t rank = used[k] ? n - 1 - bef : page - bef;  // from the top, from the bottom
            const bool moves = rank < m && (used[k] ? page >= n : page < n);
            if (moves) (used[k] ? p.src : p.dst)[rank] = (int)page;
            if ((used[k] != 0) != moves) {  // in use from now on
                highest = (int)page + 1;
            } else {
                const int64_t in_use = bef + min(m, page - bef) - max((int64_t)0, bef - (n - m));
                p.free_out[n_free - 1 - (page - in_use)] = (int)page;
            }
            __stcg(p.page_map + page, (int)page);
            __stcg(p.shares_out + page, p.shares[page]);
            bef += used[k];
        }
    }
    for (int64_t i = m + tid; i < p.moves; i += stride) p.src[i] = p.dst[i] = -1;
    for (int64_t i = n_free + tid; i < P; i += stride) p.free_out[i] = -1;
    highest = __reduce_max_sync(0xffffffffu, highest);
    if ((threadIdx.x & 31) == 0) atomicMax(&top, highest);
    __syncthreads();
    cluster_share<CTAS>(top, box[2]);  // (also: every move is listed)
    for (int64_t i = tid; i < m; i += stride) {
        const int from = __ldcg(p.src + i), to = __ldcg(p.dst + i);
        __stcg(p.page_map + from, to);
        __stcg(p.shares_out + to, p.shares[from]);
        __stcg(p.shares_out + from, 0);
    }
    if (tid == 0) {
        int e = 0;
        for (int c = 0; c < CTAS; ++c) e = max(e, box[2][c]);
        p.extent[0] = e;
        p.num_free_out[0] = (int)n_free;
    }
}

__global__ void __launch_bounds__(kShareThreads) pa_compact_tables_kernel(const ShareParams p) {
    pdl_wait_primary();  // (no early launch of dependents, as above)
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const int len = p.lens[b];
        if (len < 0 || len > room_of(p)) {
            if (threadIdx.x == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
            continue;
        }
        const int held = (int)(((int64_t)len + p.block_size - 1) / p.block_size);
        int32_t *row = p.table + (int64_t)b * p.width;
        for (int e = threadIdx.x; e < held; e += kShareThreads) {
            const int page = row[e];
            if (valid_page(p, page))
                row[e] = p.page_map[page];
            else
                set_status(p.status, PA_DEV_BAD_PAGE);
        }
    }
}

// ---- copies -------------------------------------------------------------------

struct CopyParams {
    uint8_t *caches[PA_MAX_COPY_CACHES];
    const int32_t *src, *dst, *tokens;
    int32_t *status;
    int64_t num_pages, part_bytes;  // bytes of a page's part (a page is `parts` of them)
    int64_t chunk_bytes;            // bytes of 16 tokens of a part
    int num_caches, num_pairs, parts, pieces;  // pieces of kCopyPiece bytes per part
    int block_size;
};

// The copies of all caches in one launch.  Bound by HBM: 4096 pages of 32 KiB, read
// and written, 268 MB in 39 us = 6.9 TB/s, a plain copy's rate; with 152 x 8 CTAs that
// walk the pieces, every SM has 8 x 4 x 256 16-byte loads in flight.  Loads and
// stores that are not kept in L2: the pages are read much later.
// A CTA copies a piece at a time: unit = ((pair * caches + cache) * parts + part) * pieces + piece.
__global__ void __launch_bounds__(kCopyThreads) pa_copy_cache_pages_kernel(const __grid_constant__ CopyParams p) {
    pdl_wait_primary();  // (no early launch of dependents: the pages are old context to the calls behind)
    const int per_pair = p.num_caches * p.parts * p.pieces;
    const int64_t units = (int64_t)p.num_pairs * per_pair;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int pair = (int)(unit / per_pair);
        int rest = (int)(unit - (int64_t)pair * per_pair);
        const int src = p.src[pair], dst = p.dst[pair];
        if (src < 0 || dst < 0) continue;  // no copy
        if (src >= p.num_pages || dst >= p.num_pages) {
            if (threadIdx.x == 0 && rest == 0) set_status(p.status, PA_DEV_BAD_PAGE);
            continue;
        }
        int64_t bytes = p.part_bytes;
        if (p.tokens != nullptr) {
            const int n = p.tokens[pair];
            if (n < 0 || n > p.block_size) {
                if (threadIdx.x == 0 && rest == 0) set_status(p.status, PA_DEV_BAD_SEQLEN);
                continue;
            }
            bytes = (n + 15) / 16 * p.chunk_bytes;
        }
        const int piece = rest % p.pieces;
        rest /= p.pieces;
        const int part = rest % p.parts, cache = rest / p.parts;
        const int64_t lo = (int64_t)piece * kCopyPiece, here = min((int64_t)kCopyPiece, bytes - lo);
        if (here <= 0 || src == dst) continue;
        const int n = (int)(here / 16);
        const int64_t off = part * p.part_bytes + lo, page = p.part_bytes * p.parts;
        const uint4 *from = reinterpret_cast<const uint4 *>(p.caches[cache] + src * page + off);
        uint4 *to = reinterpret_cast<uint4 *>(p.caches[cache] + dst * page + off);
        constexpr int U = kCopyPiece / 16 / kCopyThreads;
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = threadIdx.x + u * kCopyThreads;
            if (i < n) v[u] = __ldcs(from + i);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = threadIdx.x + u * kCopyThreads;
            if (i < n) __stcs(to + i, v[u]);
        }
    }
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Buffer {
    const void *at;
    int64_t bytes;
    bool written;
    bool needed;
};

// Pointers present and aligned, and no buffer that is written shares bytes with
// another (CTAs read the inputs while others write).
template <int N>
pa_status check_buffers(const Buffer (&buf)[N]) {
    for (const auto &a : buf)
        if (a.needed && a.bytes > 0 && (!a.at || !aligned(a.at, 4))) return PA_ERR_INVALID_ARG;
    for (const auto &a : buf)
        for (const auto &b : buf) {
            const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
            if (&a != &b && a.written && a.at && b.at && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes)
                return PA_ERR_INVALID_ARG;
        }
    return PA_OK;
}

pa_status check_sizes(const ShareParams &p) {
    if (p.B < 0 || p.width < 0 || p.block_size < 1 || p.num_pages < 1 || p.moves < 0) return PA_ERR_INVALID_ARG;
    if (p.num_pages > INT32_MAX || p.B > 65535) return PA_ERR_UNSUPPORTED;
    if ((int64_t)p.width * p.block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;  // lengths are 32-bit
    return PA_OK;
}

template <typename... K, typename... A>
bool launch_on(void (*kern)(K...), int ctas, int threads, bool cluster, size_t smem, void *stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<K>(args)...) == cudaSuccess;
}

// CTAs of 256 threads for the pages and the requests: one per request, or per four pages a thread.
int share_ctas(const ShareParams &p) {
    const int64_t pages = (p.num_pages + 4 * kShareThreads - 1) / (4 * kShareThreads);
    return (int)std::max<int64_t>(1, std::min<int64_t>(kShareCtas, std::max<int64_t>(pages, p.B)));
}

// Whether a release's pages and tables suit one cluster.
bool suits_cluster(const ShareParams &p) {
    return p.num_pages <= kClusterMost && (int64_t)p.B * p.width <= kClusterMost;
}

// Launches a kernel that is one cluster, of kScanCtas CTAs or, for more than
// wide_from pages, of kScanWide; `counters`: it keeps those of its share of the
// pages in every CTA's shared memory.  Clusters of more than 8 CTAs are not
// portable: such a one is taken where the device says that it has room for it.
template <typename Kernel>
pa_status launch_cluster(Kernel few, Kernel many, int64_t wide_from, const ShareParams &p, bool counters, int slot,
                         void *stream) {
    const void *fn = reinterpret_cast<const void *>(many);
    const int most = counters ? kClusterPages * 4 : 0;
    const bool wide = many != nullptr && p.num_pages > wide_from &&
                      (!counters || ensure_smem_limit(fn, most, slot) == cudaSuccess) &&
                      ensure_wide_cluster(fn, kScanWide, kScanThreads, most, slot) == cudaSuccess;
    if (!wide && counters && ensure_smem_limit(reinterpret_cast<const void *>(few), most, slot + 1) != cudaSuccess)
        return PA_ERR_CUDA;
    const int ctas = wide ? kScanWide : kScanCtas;
    const size_t smem = counters ? 4 * ((((size_t)p.num_pages + ctas - 1) / ctas + 3) & ~size_t(3)) : 0;
    return launch_on(wide ? many : few, ctas, kScanThreads, true, smem, stream, p) ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_fork_block_tables(const int32_t *seq_lens, const int32_t *parent, int32_t *block_table,
                               const int32_t *free_pages, const int32_t *num_free, const int32_t *share_counts,
                               int32_t num_seqs, int32_t max_pages_per_seq, int32_t block_size, int64_t num_pages,
                               int32_t *seq_lens_out, int32_t *share_counts_out, int32_t *copy_src, int32_t *copy_dst,
                               int32_t *copy_tokens, int32_t *num_free_out, int32_t *device_status, void *stream) {
    ShareParams p = {};
    p.lens = seq_lens;
    p.count = parent;
    p.table = block_table;
    p.free_pages = const_cast<int32_t *>(free_pages);
    p.num_free = num_free;
    p.shares = share_counts;
    p.lens_out = seq_lens_out;
    p.shares_out = share_counts_out;
    p.num_free_out = num_free_out;
    p.src = copy_src;
    p.dst = copy_dst;
    p.tokens = copy_tokens;
    p.status = device_status;
    p.num_pages = num_pages;
    p.B = num_seqs;
    p.width = max_pages_per_seq;
    p.block_size = block_size;
    pa_status st = check_sizes(p);
    if (st != PA_OK) return st;
    const int64_t rows = 4ll * p.B;
    st = check_buffers<12>({{seq_lens, rows, false, true},
                            {parent, rows, false, true},
                            {block_table, rows * p.width, true, true},
                            {free_pages, 4 * num_pages, false, true},
                            {num_free, 4, false, true},
                            {share_counts, 4 * num_pages, false, true},
                            {seq_lens_out, rows, true, true},
                            {share_counts_out, 4 * num_pages, true, true},
                            {copy_src, rows, true, true},
                            {copy_dst, rows, true, true},
                            {copy_tokens, rows, true, true},
                            {num_free_out, 4, true, true}});
    if (st != PA_OK) return st;
    const int ctas = share_ctas(p);
    // whole CTAs of requests: at least one request, so that the last CTA that has any writes the pool's size
    const int per = std::max(1, (p.B + ctas - 1) / ctas);
    if (!launch_on(pa_fork_tables_kernel, ctas, kShareThreads, false, 0, stream, p, per)) return PA_ERR_CUDA;
    const int count_ctas = std::max(1, std::min(p.B, 4 * kShareCtas));
    return launch_on(pa_fork_counts_kernel, count_ctas, kShareThreads, false, 0, stream, p) ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_release_shared_block_tables(const int32_t *seq_lens, const int32_t *finished, const int32_t *block_table,
                                         int32_t *free_pages, const int32_t *num_free, const int32_t *share_counts,
                                         int32_t num_seqs, int32_t max_pages_per_seq, int32_t block_size,
                                         int64_t num_pages, int32_t *seq_lens_out, int32_t *share_counts_out,
                                         int32_t *num_free_out, int32_t *device_status, void *stream) {
    ShareParams p = {};
    p.lens = seq_lens;
    p.count = finished;
    p.table = const_cast<int32_t *>(block_table);
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.shares = share_counts;
    p.lens_out = seq_lens_out;
    p.shares_out = share_counts_out;
    p.num_free_out = num_free_out;
    p.status = device_status;
    p.num_pages = num_pages;
    p.B = num_seqs;
    p.width = max_pages_per_seq;
    p.block_size = block_size;
    pa_status st = check_sizes(p);
    if (st != PA_OK) return st;
    const int64_t rows = 4ll * p.B;
    st = check_buffers<9>({{seq_lens, rows, false, true},
                           {finished, rows, false, true},
                           {block_table, rows * p.width, false, true},
                           {free_pages, 4 * num_pages, true, true},
                           {num_free, 4, false, true},
                           {share_counts, 4 * num_pages, false, true},
                           {seq_lens_out, rows, true, true},
                           {share_counts_out, 4 * num_pages, true, true},
                           {num_free_out, 4, true, true}});
    if (st != PA_OK) return st;
    if (suits_cluster(p)) return launch_cluster<void (*)(ShareParams)>(pa_release_cluster_kernel<kScanCtas>, nullptr, 0, p, true, 288, stream);
    if (!launch_on(pa_release_lens_kernel, share_ctas(p), kShareThreads, false, 0, stream, p)) return PA_ERR_CUDA;
    const int count_ctas = std::max(1, std::min(p.B, 4 * kShareCtas));
    if (!launch_on(pa_release_counts_kernel, count_ctas, kShareThreads, false, 0, stream, p)) return PA_ERR_CUDA;
    return launch_cluster(pa_release_pool_kernel<kScanCtas>, pa_release_pool_kernel<kScanWide>, kWideRelease, p, false, 290, stream);
}

pa_status pa_compact_block_tables(const int32_t *seq_lens, int32_t *block_table, const int32_t *free_pages,
                                  const int32_t *num_free, const int32_t *share_counts, int32_t num_seqs,
                                  int32_t max_pages_per_seq, int32_t block_size, int64_t num_pages, int32_t max_moves,
                                  int32_t *free_pages_out, int32_t *num_free_out, int32_t *share_counts_out,
                                  int32_t *page_map, int32_t *copy_src, int32_t *copy_dst, int32_t *extent,
                                  int32_t *device_status, void *stream) {
    ShareParams p = {};
    p.lens = seq_lens;
    p.table = block_table;
    p.free_pages = const_cast<int32_t *>(free_pages);
    p.num_free = num_free;
    p.shares = share_counts;
    p.shares_out = share_counts_out;
    p.num_free_out = num_free_out;
    p.src = copy_src;
    p.dst = copy_dst;
    p.free_out = free_pages_out;
    p.page_map = page_map;
    p.extent = extent;
    p.status = device_status;
    p.num_pages = num_pages;
    p.B = num_seqs;
    p.width = max_pages_per_seq;
    p.block_size = block_size;
    p.moves = max_moves;
    pa_status st = check_sizes(p);
    if (st != PA_OK) return st;
    const int64_t rows = 4ll * p.B, moved = 4ll * max_moves;
    st = check_buffers<12>({{seq_lens, rows, false, true},
                            {block_table, rows * p.width, true, true},
                            {free_pages, 4 * num_pages, false, true},
                            {num_free, 4, false, true},
                            {share_counts, 4 * num_pages, false, true},
                            {free_pages_out, 4 * num_pages, true, true},
                            {num_free_out, 4, true, true},
                            {share_counts_out, 4 * num_pages, true, true},
                            {page_map, 4 * num_pages, true, true},
                            {copy_src, moved, true, true},
                            {copy_dst, moved, true, true},
                            {extent, 4, true, true}});
    if (st != PA_OK) return st;
    st = p.num_pages <= (int64_t)kScanCtas * kClusterPages
             ? launch_cluster(pa_compact_cluster_kernel<kScanCtas>, pa_compact_cluster_kernel<kScanWide>, kWideCompact, p, true,
                              292, stream)
             : launch_cluster(pa_compact_pool_kernel<kScanCtas>, pa_compact_pool_kernel<kScanWide>, kWideCompact, p, false, 294,
                              stream);
    if (st != PA_OK) return st;
    const int ctas = std::max(1, std::min(p.B, 4 * kShareCtas));
    return launch_on(pa_compact_tables_kernel, ctas, kShareThreads, false, 0, stream, p) ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_copy_cache_pages(void *const *caches, int32_t num_caches, const int32_t *copy_src,
                              const int32_t *copy_dst, const int32_t *copy_tokens, int32_t num_pairs,
                              int32_t parts_per_page, int64_t chunk_bytes, int32_t block_size, int64_t num_pages,
                              int32_t *device_status, void *stream) {
    if (num_caches < 0 || num_pairs < 0 || parts_per_page < 1 || chunk_bytes < 1 || block_size < 1 || num_pages < 1)
        return PA_ERR_INVALID_ARG;
    if (num_caches > PA_MAX_COPY_CACHES || block_size % 16 != 0 || chunk_bytes % 16 != 0 || num_pages > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    CopyParams p = {};
    p.num_caches = num_caches;
    p.num_pairs = num_pairs;
    p.parts = parts_per_page;
    p.chunk_bytes = chunk_bytes;
    p.block_size = block_size;
    p.num_pages = num_pages;
    if (chunk_bytes > INT32_MAX || chunk_bytes > (1ll << 46) / parts_per_page / (block_size / 16))
        return PA_ERR_UNSUPPORTED;
    p.part_bytes = chunk_bytes * (block_size / 16);
    const int64_t pieces = (p.part_bytes + kCopyPiece - 1) / kCopyPiece;
    if (pieces * parts_per_page * std::max(1, num_caches) > INT32_MAX) return PA_ERR_UNSUPPORTED;
    p.pieces = (int)pieces;
    p.src = copy_src;
    p.dst = copy_dst;
    p.tokens = copy_tokens;
    p.status = device_status;
    if (num_caches == 0 || num_pairs == 0) return PA_OK;
    if (!caches || !copy_src || !copy_dst || !aligned(copy_src, 4) || !aligned(copy_dst, 4) || !aligned(copy_tokens, 4))
        return PA_ERR_INVALID_ARG;
    for (int i = 0; i < num_caches; ++i) {
        if (!caches[i] || !aligned(caches[i], 16)) return PA_ERR_INVALID_ARG;
        p.caches[i] = static_cast<uint8_t *>(caches[i]);
    }
    const int64_t units = (int64_t)num_pairs * num_caches * parts_per_page * pieces;
    return launch_on(pa_copy_cache_pages_kernel, (int)std::min<int64_t>(kCopyCtas, units), kCopyThreads, false, 0, stream, p)
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // extern "C"
