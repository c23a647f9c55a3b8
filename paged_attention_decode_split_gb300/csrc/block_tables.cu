// block_tables.cu -- block tables and slot maps built on the GPU from request
// lengths: extend_block_tables gives every request the pages its new tokens
// need and the slot of each of them, release_block_tables returns the pages of
// finished requests.
//
// Both are prefix sums over the requests -- rows of the packed batch, pages
// wanted -- and gathers through them.  Requests are few next to tokens, so
// every CTA forms the whole prefix for itself (one pass over the requests, a
// block scan) and then writes its share of the slots and of the table entries;
// no CTA waits for another and nothing that one CTA reads is written by
// another (the new lengths and the new pool size go to buffers of their own),
// so a call is one kernel and its results do not depend on any order.
//
// What bounds them is latency: a slot needs its request (a binary search over
// the prefix), then its page (a table entry or a free-list entry), then a
// store.  Up to 512 requests each thread keeps one request and its prefix in
// shared memory, a slot's search reads nothing else, and a thread works on
// four pairs of slots at once, each pair one 16-byte store; beyond that the
// prefix is kept per group of requests and the group is walked.
#include <algorithm>

#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kTabThreads = 512;

struct TableParams {
    const int32_t *lens;      // [B] tokens held
    const int32_t *count;     // [B] extend: new tokens; release: non-zero = finished
    int32_t *table;           // [B, width]
    int32_t *free_pages;      // [P] stack of free pages
    const int32_t *num_free;  // [1]
    int32_t *lens_out;        // [B]
    int64_t *slots;           // [N]
    int32_t *num_free_out;    // [1]
    int32_t *status;
    int64_t num_pages;        // P
    int B, width, block_size, num_tokens;
};

// A request's demand: rows it takes in the packed batch and pages it wants.
struct Demand {
    int64_t rows, pages;
};
__device__ __forceinline__ Demand operator+(Demand a, Demand b) { return {a.rows + b.rows, a.pages + b.pages}; }

__device__ __forceinline__ int pages_of(int64_t tokens, int block_size) {
    return (int)((tokens + block_size - 1) / block_size);
}

// What request b asks for; ok = its lengths make sense.
struct Request {
    int len, n, have, want;
    bool ok;
};

template <bool RELEASE>
__device__ __forceinline__ Request request(const TableParams &p, int b) {
    Request q;
    q.len = p.lens[b];
    q.n = p.count[b];
    const int64_t room = (int64_t)p.width * p.block_size;
    if (RELEASE) {
        q.ok = q.len >= 0 && q.len <= room;
        q.have = q.ok ? pages_of(q.len, p.block_size) : 0;
        q.want = 0;
    } else {
        q.ok = q.len >= 0 && q.n >= 0 && (int64_t)q.len + q.n <= room;
        q.n = max(q.n, 0);
        q.have = q.ok ? pages_of(q.len, p.block_size) : 0;
        q.want = q.ok ? pages_of((int64_t)q.len + q.n, p.block_size) : 0;
    }
    return q;
}

template <bool RELEASE>
__device__ __forceinline__ Demand demand(const TableParams &p, const Request &q) {
    if (RELEASE) return {0, q.n != 0 ? q.have : 0};
    return {q.n, q.want - q.have};
}

// The prefix over the requests, kept per thread: thread t owns requests
// [t * per, (t + 1) * per); first[t] is the demand of all requests before them.
struct Prefix {
    int64_t rows[kTabThreads + 1], pages[kTabThreads + 1];
};

template <bool RELEASE>
__device__ __forceinline__ void build_prefix(const TableParams &p, int per, Prefix &f) {
    __shared__ Demand warp_sum[kTabThreads / 32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    Demand mine{0, 0};
    const int64_t b0 = (int64_t)t * per;
    for (int64_t b = b0; b < min(b0 + per, (int64_t)p.B); ++b) mine = mine + demand<RELEASE>(p, request<RELEASE>(p, (int)b));
    Demand incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t rows = __shfl_up_sync(0xffffffffu, incl.rows, d), pages = __shfl_up_sync(0xffffffffu, incl.pages, d);
        if (lane >= d) incl = incl + Demand{rows, pages};
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    Demand before{0, 0};
    for (int w = 0; w < warp; ++w) before = before + warp_sum[w];
    incl = incl + before;
    if (t == 0) f.rows[0] = f.pages[0] = 0;
    f.rows[t + 1] = incl.rows;
    f.pages[t + 1] = incl.pages;
    __syncthreads();
}

// The last group whose first entry is <= i.
__device__ __forceinline__ int group_of(const int64_t *first, int64_t i) {
    int lo = 0, hi = kTabThreads;  // first[lo] <= i < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int pool_size(const TableParams &p) {
    const int f = p.num_free[0];
    return (int)max((int64_t)0, min((int64_t)f, p.num_pages));
}

// Requests are served in order: one is refused if its lengths make no sense,
// if the packed rows up to its last one do not fit the slot map, or if the
// pages wanted up to it exceed the pool (one that wants none never fails so).
__device__ __forceinline__ bool served(const TableParams &p, const Request &q, Demand upto, int64_t F) {
    return q.ok && upto.rows <= p.num_tokens && (q.want == q.have || upto.pages <= F);
}

// ---- up to kTabThreads requests: one per thread --------------------------------

// A request as the slot and page loops read it.
struct Entry {
    int32_t row_end, page_end;  // prefix sums, its own included (clamped to INT32_MAX)
    int32_t rows, len;          // new tokens; tokens held
    int32_t have, taken;        // pages held; pages taken (0 if refused)
    int32_t served, pad;
};

struct FastPrefix {
    int32_t row_end[kTabThreads], page_end[kTabThreads];
    Entry e[kTabThreads];
    int64_t pages;                       // wanted by all requests
    unsigned long long moved;            // pages taken or returned by the served ones
    Demand warp_sum[kTabThreads / 32];
};

// The first index whose (ascending) entry exceeds i; the entries past the
// requests are INT32_MAX.
__device__ __forceinline__ int upper(const int32_t *end, int32_t i) {
    int b = 0;
#pragma unroll
    for (int step = kTabThreads / 2; step > 0; step >>= 1)
        if (end[b + step - 1] <= i) b += step;
    return b;
}

template <bool RELEASE>
__device__ __forceinline__ int64_t build_fast(const TableParams &p, FastPrefix &f) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int raw_free = p.num_free[0];
    Request q{0, 0, 0, 0, true};
    Demand d{0, 0};
    if (t < p.B) {
        q = request<RELEASE>(p, t);
        d = demand<RELEASE>(p, q);
    }
    Demand incl = d;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int64_t rows = __shfl_up_sync(0xffffffffu, incl.rows, k), pages = __shfl_up_sync(0xffffffffu, incl.pages, k);
        if (lane >= k) incl = incl + Demand{rows, pages};
    }
    if (lane == 31) f.warp_sum[warp] = incl;
    if (t == 0) f.moved = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; ++w)
        if (w < warp) incl = incl + f.warp_sum[w];
    const int64_t F = max((int64_t)0, min((int64_t)raw_free, p.num_pages));
    // extend: pages and rows suffice up to this request; release: the pool has room up to it
    const bool yes = RELEASE ? q.n != 0 && incl.pages <= p.num_pages - F : served(p, q, incl, F);
    const bool live = t < p.B;
    Entry e;
    e.row_end = live ? (int32_t)min(incl.rows, (int64_t)INT32_MAX) : INT32_MAX;
    e.page_end = live ? (int32_t)min(incl.pages, (int64_t)INT32_MAX) : INT32_MAX;
    e.rows = q.n;
    e.len = q.len;
    e.have = q.have;
    e.taken = yes ? (int32_t)d.pages : 0;
    e.served = live && yes;
    e.pad = 0;
    f.row_end[t] = e.row_end;
    f.page_end[t] = e.page_end;
    f.e[t] = e;
    if (t == kTabThreads - 1) f.pages = incl.pages;
    if (blockIdx.x == 0) {
        if (live) {
            p.lens_out[t] = RELEASE ? (yes ? 0 : max(q.len, 0)) : yes ? q.len + q.n : max(q.len, 0);
            if (!q.ok) set_status(p.status, PA_DEV_BAD_SEQLEN);
            else if (RELEASE && q.n != 0 && !yes) set_status(p.status, PA_DEV_BAD_PAGE);
            else if (!RELEASE && incl.rows > p.num_tokens && q.n > 0) set_status(p.status, PA_DEV_BAD_SLOT);
            else if (!RELEASE && !yes && q.n > 0) set_status(p.status, PA_DEV_NO_PAGES);
            if (yes && d.pages > 0) atomicMax(&f.moved, (unsigned long long)incl.pages);
        }
        if (t == 0 && F != raw_free) set_status(p.status, PA_DEV_BAD_PAGE);
    }
    __syncthreads();
    if (blockIdx.x == 0 && t == 0)
        p.num_free_out[0] = (int32_t)(RELEASE ? F + (int64_t)f.moved : F - (int64_t)f.moved);
    return F;
}

__global__ void __launch_bounds__(kTabThreads) pa_extend_block_tables_few_kernel(const TableParams p) {
    // (no early launch of dependents: a kernel behind this one may start a
    // third one early, which must not read the tables before they are written)
    pdl_wait_primary();
    __shared__ FastPrefix f;
    const int64_t F = build_fast<false>(p, f);
    const int64_t tid = (int64_t)blockIdx.x * kTabThreads + threadIdx.x, stride = (int64_t)gridDim.x * kTabThreads;

    // slot of the token at offset `pos` of request b; its page by way of `lp`
    auto page_at = [&](int b, const Entry &e, int lp) {
        return lp < e.have ? p.table[(int64_t)b * p.width + lp]
                           : p.free_pages[F - 1 - ((int64_t)e.page_end - e.taken + (lp - e.have))];
    };
    auto slot_in = [&](int page, int off) {
        return page >= 0 && page < p.num_pages ? (int64_t)page * p.block_size + off : (int64_t)-1;
    };
    auto slot_of = [&](int32_t i) -> int64_t {
        const int b = upper(f.row_end, i);
        if (b >= p.B) return -1;
        const Entry e = f.e[b];
        if (!e.served || i >= e.row_end) return -1;  // (past the last row, upper() ends at the last entry)
        const int pos = e.len + (i - (e.row_end - e.rows)), lp = pos / p.block_size;
        return slot_in(page_at(b, e, lp), pos - lp * p.block_size);
    };
    constexpr int U = 4;
    const int64_t n_pairs = ((int64_t)p.num_tokens + 1) / 2;
    const bool vec = (reinterpret_cast<uintptr_t>(p.slots) & 15u) == 0;
    for (int64_t k0 = tid; k0 < n_pairs; k0 += U * stride) {
        int page[U], off[U], left[U];  // left: tokens of the request from this one on, within its page
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {  // all searches and loads first
            const int64_t k = k0 + u * stride;
            on[u] = false;
            page[u] = -1;
            off[u] = left[u] = 0;
            if (k < n_pairs) {
                const int32_t i = (int32_t)(2 * k);
                const int b = upper(f.row_end, i);
                if (b < p.B) {
                    const Entry e = f.e[b];
                    if (e.served && i < e.row_end) {
                        const int pos = e.len + (i - (e.row_end - e.rows)), lp = pos / p.block_size;
                        off[u] = pos - lp * p.block_size;
                        left[u] = min(e.row_end - i, p.block_size - off[u]);
                        page[u] = page_at(b, e, lp);
                        on[u] = true;
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + u * stride;
            if (k >= n_pairs) break;
            const int64_t s0 = on[u] ? slot_in(page[u], off[u]) : -1;
            const bool second = 2 * k + 1 < p.num_tokens;
            int64_t s1 = -1;
            if (second) s1 = left[u] > 1 ? (s0 < 0 ? -1 : s0 + 1) : slot_of((int32_t)(2 * k + 1));
            if (second && vec) {
                *reinterpret_cast<longlong2 *>(p.slots + 2 * k) = make_longlong2(s0, s1);
            } else {
                p.slots[2 * k] = s0;
                if (second) p.slots[2 * k + 1] = s1;
            }
        }
    }
    // table entry of the k-th page taken from the pool
    const int64_t pages = min(f.pages, F);
#pragma unroll 4
    for (int64_t k = tid; k < pages; k += stride) {
        const int page = p.free_pages[F - 1 - k];
        const int b = upper(f.page_end, (int32_t)k);
        const Entry e = f.e[b];
        if (e.taken == 0) continue;  // refused
        if (page < 0 || page >= p.num_pages) set_status(p.status, PA_DEV_BAD_PAGE);
        p.table[(int64_t)b * p.width + e.have + (k - (e.page_end - e.taken))] = page;
    }
}

__global__ void __launch_bounds__(kTabThreads) pa_release_block_tables_few_kernel(const TableParams p) {
    pdl_wait_primary();  // (no early launch of dependents, as above)
    __shared__ FastPrefix f;
    const int64_t F = build_fast<true>(p, f);
    const int64_t tid = (int64_t)blockIdx.x * kTabThreads + threadIdx.x, stride = (int64_t)gridDim.x * kTabThreads;
    const int64_t pages = min(f.pages, p.num_pages - F);
#pragma unroll 4
    for (int64_t k = tid; k < pages; k += stride) {  // the k-th returned page
        const int b = upper(f.page_end, (int32_t)k);
        const Entry e = f.e[b];
        if (e.taken == 0) continue;  // refused: the pool has no room for all of its pages
        const int page = p.table[(int64_t)b * p.width + (k - (e.page_end - e.taken))];
        if (page < 0 || page >= p.num_pages) set_status(p.status, PA_DEV_BAD_PAGE);
        p.free_pages[F + k] = page;
    }
}

// ---- more requests: the prefix kept per group ----------------------------------

__global__ void __launch_bounds__(kTabThreads) pa_extend_block_tables_kernel(const TableParams p) {
    pdl_wait_primary();  // (no early launch of dependents, as above)
    __shared__ Prefix f;
    const int per = (p.B + kTabThreads - 1) / kTabThreads;
    build_prefix<false>(p, per, f);
    const int64_t F = pool_size(p), rows = f.rows[kTabThreads], pages = f.pages[kTabThreads];
    const int64_t tid = (int64_t)blockIdx.x * kTabThreads + threadIdx.x, stride = (int64_t)gridDim.x * kTabThreads;

    // slot of packed row i
    for (int64_t i = tid; i < p.num_tokens; i += stride) {
        int64_t slot = -1;
        if (i < rows) {
            const int g = group_of(f.rows, i);
            Demand at{f.rows[g], f.pages[g]};
            int64_t b = (int64_t)g * per;
            Request q = request<false>(p, (int)b);
            Demand d = demand<false>(p, q);
            while (i >= at.rows + d.rows) {
                at = at + d;
                q = request<false>(p, (int)++b);
                d = demand<false>(p, q);
            }
            if (served(p, q, at + d, F)) {
                const int pos = q.len + (int)(i - at.rows);  // < width * block_size <= INT32_MAX
                const int lp = pos / p.block_size;
                const int page = lp < q.have ? p.table[b * p.width + lp]
                                             : p.free_pages[F - 1 - (at.pages + (lp - q.have))];
                if (page >= 0 && page < p.num_pages) slot = (int64_t)page * p.block_size + (pos - lp * p.block_size);
            }
        }
        p.slots[i] = slot;
    }
    // table entry of the k-th page taken from the pool
    for (int64_t k = tid; k < min(pages, F); k += stride) {
        const int g = group_of(f.pages, k);
        Demand at{f.rows[g], f.pages[g]};
        int64_t b = (int64_t)g * per;
        Request q = request<false>(p, (int)b);
        Demand d = demand<false>(p, q);
        while (k >= at.pages + d.pages) {
            at = at + d;
            q = request<false>(p, (int)++b);
            d = demand<false>(p, q);
        }
        if (!served(p, q, at + d, F)) continue;
        const int page = p.free_pages[F - 1 - k];
        if (page < 0 || page >= p.num_pages) set_status(p.status, PA_DEV_BAD_PAGE);
        p.table[b * p.width + q.have + (k - at.pages)] = page;
    }
    // lengths and what is left of the pool
    if (blockIdx.x == 0) {
        const int t = threadIdx.x;
        Demand at{f.rows[t], f.pages[t]};
        int64_t taken = 0;
        const int64_t b0 = (int64_t)t * per;
        for (int64_t b = b0; b < min(b0 + per, (int64_t)p.B); ++b) {
            const Request q = request<false>(p, (int)b);
            at = at + demand<false>(p, q);
            const bool yes = served(p, q, at, F);
            p.lens_out[b] = yes ? q.len + q.n : max(q.len, 0);
            if (yes) taken = q.want > q.have ? at.pages : taken;
            if (!q.ok) set_status(p.status, PA_DEV_BAD_SEQLEN);
            else if (at.rows > p.num_tokens && q.n > 0) set_status(p.status, PA_DEV_BAD_SLOT);
            else if (!yes && q.n > 0) set_status(p.status, PA_DEV_NO_PAGES);
        }
        __shared__ unsigned long long most;
        if (t == 0) most = 0;
        __syncthreads();
        if (taken > 0) atomicMax(&most, (unsigned long long)taken);
        __syncthreads();
        if (t == 0) {
            p.num_free_out[0] = (int32_t)(F - (int64_t)most);
            if (F != p.num_free[0]) set_status(p.status, PA_DEV_BAD_PAGE);
        }
    }
}

__global__ void __launch_bounds__(kTabThreads) pa_release_block_tables_kernel(const TableParams p) {
    pdl_wait_primary();  // (no early launch of dependents, as above)
    __shared__ Prefix f;
    const int per = (p.B + kTabThreads - 1) / kTabThreads;
    build_prefix<true>(p, per, f);
    const int64_t F = pool_size(p), pages = f.pages[kTabThreads], room = p.num_pages - F;
    const int64_t tid = (int64_t)blockIdx.x * kTabThreads + threadIdx.x, stride = (int64_t)gridDim.x * kTabThreads;
    // the k-th returned page
    for (int64_t k = tid; k < min(pages, room); k += stride) {
        const int g = group_of(f.pages, k);
        int64_t at = f.pages[g], b = (int64_t)g * per;
        int d = (int)demand<true>(p, request<true>(p, (int)b)).pages;
        while (k >= at + d) {
            at += d;
            d = (int)demand<true>(p, request<true>(p, (int)++b)).pages;
        }
        if (at + d > room) continue;  // refused: the pool has no room for all of its pages
        const int page = p.table[b * p.width + (k - at)];
        if (page < 0 || page >= p.num_pages) set_status(p.status, PA_DEV_BAD_PAGE);
        p.free_pages[F + k] = page;
    }
    if (blockIdx.x == 0) {
        const int t = threadIdx.x;
        int64_t at = f.pages[t], back = 0;
        const int64_t b0 = (int64_t)t * per;
        for (int64_t b = b0; b < min(b0 + per, (int64_t)p.B); ++b) {
            const Request q = request<true>(p, (int)b);
            at += demand<true>(p, q).pages;
            const bool yes = q.n != 0 && at <= room;
            if (yes) back = at;
            p.lens_out[b] = yes ? 0 : max(q.len, 0);
            if (!q.ok) set_status(p.status, PA_DEV_BAD_SEQLEN);
            else if (q.n != 0 && !yes) set_status(p.status, PA_DEV_BAD_PAGE);
        }
        __shared__ unsigned long long most;
        if (t == 0) most = 0;
        __syncthreads();
        if (back > 0) atomicMax(&most, (unsigned long long)back);
        __syncthreads();
        if (t == 0) {
            p.num_free_out[0] = (int32_t)(F + (int64_t)most);
            if (F != p.num_free[0]) set_status(p.status, PA_DEV_BAD_PAGE);
        }
    }
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

pa_status check_tables(const TableParams &p, const void *slots_needed) {
    if (p.B < 0 || p.width < 0 || p.block_size < 1 || p.num_pages < 1 || p.num_tokens < 0) return PA_ERR_INVALID_ARG;
    if (p.num_pages > INT32_MAX || p.B > 65535) return PA_ERR_UNSUPPORTED;
    if ((int64_t)p.width * p.block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;  // lengths are 32-bit
    if (!p.free_pages || !p.num_free || !p.num_free_out || !slots_needed) return PA_ERR_INVALID_ARG;
    if (p.B > 0 && (!p.lens || !p.count || !p.lens_out || (p.width > 0 && !p.table))) return PA_ERR_INVALID_ARG;
    if (!aligned(p.lens, 4) || !aligned(p.count, 4) || !aligned(p.table, 4) || !aligned(p.free_pages, 4) ||
        !aligned(p.num_free, 4) || !aligned(p.lens_out, 4) || !aligned(p.num_free_out, 4) || !aligned(p.slots, 8))
        return PA_ERR_INVALID_ARG;
    // every CTA reads the inputs while one writes these
    if (p.num_free_out == p.num_free || (p.B > 0 && (p.lens_out == p.lens || p.lens_out == p.count)))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

pa_status launch_tables(void (*kern)(TableParams), const TableParams &p, int64_t items, void *stream) {
    cudaLaunchConfig_t cfg = {};
    // about four items per thread, at most two CTAs on each of 152 SMs
    cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(304, (items + 4 * kTabThreads - 1) / (4 * kTabThreads))));
    cfg.blockDim = dim3(kTabThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_extend_block_tables(const int32_t *context_lens, const int32_t *num_new, int32_t *block_table,
                                 const int32_t *free_pages, const int32_t *num_free, int32_t num_seqs,
                                 int32_t max_pages_per_seq, int32_t block_size, int64_t num_pages, int32_t num_tokens,
                                 int32_t *seq_lens, int64_t *slot_mapping, int32_t *num_free_out,
                                 int32_t *device_status, void *stream) {
    const TableParams p{context_lens, num_new, block_table, const_cast<int32_t *>(free_pages), num_free, seq_lens,
                        slot_mapping, num_free_out, device_status, num_pages, num_seqs, max_pages_per_seq, block_size,
                        num_tokens};
    const pa_status st = check_tables(p, num_tokens > 0 ? static_cast<const void *>(slot_mapping) : free_pages);
    if (st != PA_OK) return st;
    return launch_tables(num_seqs <= kTabThreads ? pa_extend_block_tables_few_kernel : pa_extend_block_tables_kernel, p,
                         num_tokens, stream);
}

pa_status pa_release_block_tables(const int32_t *seq_lens, const int32_t *finished, const int32_t *block_table,
                                  int32_t *free_pages, const int32_t *num_free, int32_t num_seqs,
                                  int32_t max_pages_per_seq, int32_t block_size, int64_t num_pages,
                                  int32_t *seq_lens_out, int32_t *num_free_out, int32_t *device_status, void *stream) {
    const TableParams p{seq_lens, finished, const_cast<int32_t *>(block_table), free_pages, num_free, seq_lens_out,
                        nullptr, num_free_out, device_status, num_pages, num_seqs, max_pages_per_seq, block_size, 0};
    const pa_status st = check_tables(p, free_pages);
    if (st != PA_OK) return st;
    return launch_tables(num_seqs <= kTabThreads ? pa_release_block_tables_few_kernel : pa_release_block_tables_kernel,
                         p, (int64_t)num_seqs * max_pages_per_seq, stream);
}

}  // extern "C"
