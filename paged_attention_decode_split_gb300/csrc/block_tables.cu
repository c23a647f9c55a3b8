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
// What bounds them is latency, and for many tokens the index arithmetic: a slot
// needs its request (a binary search over the prefix), then its page (a table
// entry or a free-list entry), then a store.  Up to 512 requests each thread
// keeps one request and its prefix in shared memory, and a thread writes a run
// of consecutive slots from one search, searching again only where a page or a
// request ends: runs of two, which fill the GPU up to 311,000 tokens, and of
// eight beyond that (a step of 32 single tokens: 3.0 us; 1M slots of 509
// requests: 8.1-8.4 us against 9.7 with four slot pairs per search; release and
// admission of 256 requests: 6.4 us in two calls).  CTAs of their own write the table
// entries.  Beyond 512 requests the prefix is kept per group of requests and
// the group is walked: 1M slots of 1000 requests take 18.4 us (8.4 us for 509),
// a step of one token each 7.2 us for 1000 requests and 317 for 65535.
#include <algorithm>

#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kTabThreads = 512;
constexpr int64_t kMost = 304;  // CTAs of 512 threads: two on each of 152 SMs

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
    int slot_ctas;  // extend, up to 512 requests: the CTAs that write slots (the others: table entries)
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

// ---- up to 512 requests: one per thread of CTAs of T = 128, 256 or 512 -----------

// A request as the slot and page loops read it.
struct Entry {
    int32_t row_end, page_end;  // prefix sums, its own included (clamped to INT32_MAX)
    int32_t rows, len;          // new tokens; tokens held
    int32_t have, taken;        // pages held; pages taken (0 if refused)
    int32_t served, pad;
};

// Prefix sums that stop at 2^32 - 1: what passes the rows or the pages there are
// is refused either way.
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
    const uint32_t s = a + b;
    return s < a ? 0xffffffffu : s;
}

template <int T>
struct FastPrefix {
    int32_t row_end[T], page_end[T];
    Entry e[T];
    uint32_t pages;  // wanted by all requests
    uint32_t moved;  // pages taken or returned by the served ones
    uint32_t warp_rows[T / 32], warp_pages[T / 32];
};

// The first index whose (ascending) entry exceeds i; the entries past the
// requests are INT32_MAX.
template <int T>
__device__ __forceinline__ int upper(const int32_t *end, int32_t i) {
    int b = 0;
#pragma unroll
    for (int step = T / 2; step > 0; step >>= 1)
        if (end[b + step - 1] <= i) b += step;
    return b;
}

template <bool RELEASE, int T>
__device__ __forceinline__ int build_fast(const TableParams &p, FastPrefix<T> &f) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int raw_free = p.num_free[0];
    const bool live = t < p.B;
    Request q{0, 0, 0, 0, true};
    if (live) q = request<RELEASE>(p, t);
    const int wants = RELEASE ? (q.n != 0 ? q.have : 0) : q.want - q.have;
    uint32_t rows = RELEASE ? 0u : (uint32_t)q.n, pages = (uint32_t)wants;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const uint32_t r = __shfl_up_sync(0xffffffffu, rows, k), g = __shfl_up_sync(0xffffffffu, pages, k);
        if (lane >= k) {
            rows = add_sat(rows, r);
            pages = add_sat(pages, g);
        }
    }
    if (lane == 31) {
        f.warp_rows[warp] = rows;
        f.warp_pages[warp] = pages;
    }
    if (t == 0) f.moved = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w)
        if (w < warp) {
            rows = add_sat(rows, f.warp_rows[w]);
            pages = add_sat(pages, f.warp_pages[w]);
        }
    const int F = (int)max((int64_t)0, min((int64_t)raw_free, p.num_pages));
    // extend: pages and rows suffice up to this request; release: the pool has room up to it
    const bool fits_rows = rows <= (uint32_t)p.num_tokens;
    const bool yes = RELEASE ? q.n != 0 && pages <= (uint32_t)(p.num_pages - F)
                             : q.ok && fits_rows && (wants == 0 || pages <= (uint32_t)F);
    Entry e;
    e.row_end = live ? (int32_t)min(rows, 0x7fffffffu) : INT32_MAX;
    e.page_end = live ? (int32_t)min(pages, 0x7fffffffu) : INT32_MAX;
    e.rows = q.n;
    e.len = q.len;
    e.have = q.have;
    e.taken = yes ? wants : 0;
    e.served = live && yes;
    e.pad = 0;
    f.row_end[t] = e.row_end;
    f.page_end[t] = e.page_end;
    f.e[t] = e;
    if (t == T - 1) f.pages = pages;
    if (blockIdx.x == 0) {
        if (live) {
            p.lens_out[t] = RELEASE ? (yes ? 0 : max(q.len, 0)) : yes ? q.len + q.n : max(q.len, 0);
            if (!q.ok) set_status(p.status, PA_DEV_BAD_SEQLEN);
            else if (RELEASE && q.n != 0 && !yes) set_status(p.status, PA_DEV_BAD_PAGE);
            else if (!RELEASE && !fits_rows && q.n > 0) set_status(p.status, PA_DEV_BAD_SLOT);
            else if (!RELEASE && !yes && q.n > 0) set_status(p.status, PA_DEV_NO_PAGES);
            if (yes && wants > 0) atomicMax(&f.moved, pages);
        }
        if (t == 0 && F != raw_free) set_status(p.status, PA_DEV_BAD_PAGE);
    }
    __syncthreads();
    if (blockIdx.x == 0 && t == 0) p.num_free_out[0] = RELEASE ? F + (int)f.moved : F - (int)f.moved;
    return F;
}

template <int T, int U>  // U: slots per thread
__global__ void __launch_bounds__(T) pa_extend_block_tables_few_kernel(const TableParams p) {
    // (no early launch of dependents: a kernel behind this one may start a
    // third one early, which must not read the tables before they are written)
    pdl_wait_primary();
    __shared__ FastPrefix<T> f;
    const int F = build_fast<false, T>(p, f);
    const bool slots = (int)blockIdx.x < p.slot_ctas;
    const int64_t tid = (int64_t)(slots ? blockIdx.x : blockIdx.x - p.slot_ctas) * T + threadIdx.x;
    const int64_t stride = (int64_t)(slots ? p.slot_ctas : gridDim.x - p.slot_ctas) * T;

    // the slot of token i, and how many tokens from it on have slots in a row
    // (-1: tokens without one, of a refused request or past the last row)
    auto find = [&](int32_t i, int &run) -> int64_t {
        const int b = upper<T>(f.row_end, i);
        run = INT32_MAX;
        if (b >= p.B) return -1;
        const Entry e = f.e[b];
        if (i >= e.row_end) return -1;  // (past the last row, upper() ends at the last entry)
        run = e.row_end - i;
        if (!e.served) return -1;
        const int pos = e.len + (i - (e.row_end - e.rows)), lp = pos / p.block_size, off = pos - lp * p.block_size;
        run = min(run, p.block_size - off);
        const int page = lp < e.have ? p.table[(int64_t)b * p.width + lp]
                                     : p.free_pages[F - 1 - (e.page_end - e.taken + (lp - e.have))];
        return page >= 0 && page < p.num_pages ? (int64_t)page * p.block_size + off : -1;
    };
    const bool vec = (reinterpret_cast<uintptr_t>(p.slots) & 15u) == 0;
    for (int64_t i0 = U * tid; slots && i0 < p.num_tokens; i0 += U * stride) {
        int64_t slot[U], next = -1;
        int run = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (run == 0 && i0 + u < p.num_tokens) next = find((int32_t)(i0 + u), run);
            slot[u] = next;
            if (next >= 0) ++next;
            --run;
        }
        if (vec && i0 + U <= p.num_tokens) {
#pragma unroll
            for (int u = 0; u < U; u += 2)
                *reinterpret_cast<longlong2 *>(p.slots + i0 + u) = make_longlong2(slot[u], slot[u + 1]);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < p.num_tokens) p.slots[i0 + u] = slot[u];
        }
    }
    // table entry of the k-th page taken from the pool
    const int64_t pages = min(f.pages, (uint32_t)F);
    for (int64_t k = tid; !slots && k < pages; k += stride) {
        const int page = p.free_pages[F - 1 - k];
        const int b = upper<T>(f.page_end, (int32_t)k);
        const Entry e = f.e[b];
        if (e.taken == 0) continue;  // refused
        if (page < 0 || page >= p.num_pages) set_status(p.status, PA_DEV_BAD_PAGE);
        p.table[(int64_t)b * p.width + e.have + (k - (e.page_end - e.taken))] = page;
    }
}

template <int T>
__global__ void __launch_bounds__(T) pa_release_block_tables_few_kernel(const TableParams p) {
    pdl_wait_primary();  // (no early launch of dependents, as above)
    __shared__ FastPrefix<T> f;
    const int F = build_fast<true, T>(p, f);
    const int64_t tid = (int64_t)blockIdx.x * T + threadIdx.x, stride = (int64_t)gridDim.x * T;
    const int64_t pages = min((int64_t)f.pages, p.num_pages - F);
    constexpr int U = 4;
    for (int64_t k0 = tid; k0 < pages; k0 += U * stride) {  // the k-th returned page, four at once
        int page[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = min(k0 + u * stride, pages - 1);
            const int b = upper<T>(f.page_end, (int32_t)k);
            const Entry e = f.e[b];
            on[u] = e.taken > 0 && k0 + u * stride < pages;  // (refused: the pool has no room for all of its pages)
            page[u] = *(on[u] ? p.table + ((int64_t)b * p.width + (k - (e.page_end - e.taken))) : p.num_free);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!on[u]) continue;
            if (page[u] < 0 || page[u] >= p.num_pages) set_status(p.status, PA_DEV_BAD_PAGE);
            p.free_pages[F + k0 + u * stride] = page[u];
        }
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

pa_status check_tables(const TableParams &p, bool release, const void *slots_needed) {
    if (p.B < 0 || p.width < 0 || p.block_size < 1 || p.num_pages < 1 || p.num_tokens < 0) return PA_ERR_INVALID_ARG;
    if (p.num_pages > INT32_MAX || p.B > 65535) return PA_ERR_UNSUPPORTED;
    if ((int64_t)p.width * p.block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;  // lengths are 32-bit
    if (!p.free_pages || !p.num_free || !p.num_free_out || !slots_needed) return PA_ERR_INVALID_ARG;
    if (p.B > 0 && (!p.lens || !p.count || !p.lens_out || (p.width > 0 && !p.table))) return PA_ERR_INVALID_ARG;
    if (!aligned(p.lens, 4) || !aligned(p.count, 4) || !aligned(p.table, 4) || !aligned(p.free_pages, 4) ||
        !aligned(p.num_free, 4) || !aligned(p.lens_out, 4) || !aligned(p.num_free_out, 4) || !aligned(p.slots, 8))
        return PA_ERR_INVALID_ARG;
    // every CTA reads the inputs while others write: no buffer that is written shares bytes with another
    const struct {
        const void *at;
        int64_t bytes;
        bool written;
    } buf[] = {{p.lens, 4ll * p.B, false},
               {p.count, 4ll * p.B, false},
               {p.table, 4ll * p.B * p.width, !release},
               {p.free_pages, 4 * p.num_pages, release},
               {p.num_free, 4, false},
               {p.lens_out, 4ll * p.B, true},
               {p.slots, 8ll * p.num_tokens, true},
               {p.num_free_out, 4, true}};
    for (const auto &a : buf)
        for (const auto &b : buf) {
            const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
            if (&a != &b && a.written && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes)
                return PA_ERR_INVALID_ARG;
        }
    return PA_OK;
}

int64_t ctas_for(int64_t items, int per_thread, int threads) {
    return std::max<int64_t>(1, (items + (int64_t)per_thread * threads - 1) / ((int64_t)per_thread * threads));
}

pa_status launch_tables(void (*kern)(TableParams), const TableParams &p, int64_t ctas, int threads, void *stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
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
    TableParams p{context_lens, num_new, block_table, const_cast<int32_t *>(free_pages), num_free, seq_lens,
                  slot_mapping, num_free_out, device_status, num_pages, num_seqs, max_pages_per_seq, block_size,
                  num_tokens, 0};
    const pa_status st = check_tables(p, false, num_tokens > 0 ? static_cast<const void *>(slot_mapping) : free_pages);
    if (st != PA_OK) return st;
    if (num_seqs > kTabThreads)
        return launch_tables(pa_extend_block_tables_kernel, p, std::min(kMost, ctas_for(num_tokens, 4, kTabThreads)),
                             kTabThreads, stream);
    // as many threads as requests need (the scan of a small batch is shorter), 512 for many tokens
    const bool few = num_tokens <= 2 * kMost * kTabThreads;
    const int T = !few || num_seqs > 256 ? 512 : num_seqs > 128 ? 256 : 128, most = (int)(kMost * (512 / T));
    p.slot_ctas = (int)std::min<int64_t>(most, ctas_for(num_tokens, few ? 2 : 8, T));
    // every page taken holds a new token: at most one per block_size tokens, and one more per request
    const int64_t page_ctas = std::min<int64_t>(most / 2, ctas_for((int64_t)num_tokens / block_size + num_seqs, 1, T));
    auto *kern = !few       ? pa_extend_block_tables_few_kernel<512, 8>
                 : T == 512 ? pa_extend_block_tables_few_kernel<512, 2>
                 : T == 256 ? pa_extend_block_tables_few_kernel<256, 2>
                            : pa_extend_block_tables_few_kernel<128, 2>;
    return launch_tables(kern, p, p.slot_ctas + page_ctas, T, stream);
}

pa_status pa_release_block_tables(const int32_t *seq_lens, const int32_t *finished, const int32_t *block_table,
                                  int32_t *free_pages, const int32_t *num_free, int32_t num_seqs,
                                  int32_t max_pages_per_seq, int32_t block_size, int64_t num_pages,
                                  int32_t *seq_lens_out, int32_t *num_free_out, int32_t *device_status, void *stream) {
    const TableParams p{seq_lens, finished, const_cast<int32_t *>(block_table), free_pages, num_free, seq_lens_out,
                        nullptr, num_free_out, device_status, num_pages, num_seqs, max_pages_per_seq, block_size, 0, 0};
    const pa_status st = check_tables(p, true, free_pages);
    if (st != PA_OK) return st;
    const int64_t items = (int64_t)num_seqs * max_pages_per_seq;
    const int T = num_seqs > 256 ? 512 : num_seqs > 128 ? 256 : 128;
    auto *kern = num_seqs > kTabThreads ? pa_release_block_tables_kernel
                 : T == 512             ? pa_release_block_tables_few_kernel<512>
                 : T == 256             ? pa_release_block_tables_few_kernel<256>
                                        : pa_release_block_tables_few_kernel<128>;
    return launch_tables(kern, p, std::min<int64_t>(kMost * (512 / T), ctas_for(items, 4, T)), T, stream);
}

}  // extern "C"
