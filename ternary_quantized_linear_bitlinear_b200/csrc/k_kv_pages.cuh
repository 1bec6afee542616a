// Page tables of a paged key-value cache, kept on the device, and the copies
// of pages that forks and compaction make.
//
// The bookkeeping (which pages are free, who gets which) is integer work of
// a few thousand entries whose order matters: one CTA does it with prefix
// sums, so that page numbers never depend on the order of atomics.  The page
// copies are bound by memory and run as a launch of their own over the whole
// GPU, a programmatic dependent of the plan.
#pragma once

#include "bl_common.cuh"

namespace bl {

constexpr int KV_THREADS = 1024;
constexpr int KV_MAX_N = 8192;             // entries of a call
constexpr int KV_MAX_SEQS = 1 << 17;
constexpr int KV_COPY_THREADS = 256;

enum : int { KV_OK = 0, KV_NO_PAGES = 1, KV_NO_ROOM = 2, KV_BAD = 3 };

struct KvTables {
    int *tables, *lengths, *refs;
    int num_pages, max_seqs, max_pages, ps_log;
};

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Exclusive prefix sum of one value per thread over the CTA; *total the sum.
// scratch: 33 values of shared memory, reused by the next call.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *total, T *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous call's readers are done
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const T w = lane < nw ? scratch[lane] : 0;
        T s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < nw) scratch[lane] = s - w;
        if (lane == 31) scratch[32] = s;
    }
    __syncthreads();
    *total = scratch[32];
    return scratch[warp] + x - v;
}

// Pages lo .. hi - 1 that are free (or in use), in ascending order: every warp
// takes a contiguous share of whole 32-page groups, counts its pages once,
// and one scan over the warps gives each its first rank.  count() is a CTA-wide
// call and returns the total; give(rank, page) then runs for each page of rank
// < wanted.
struct PagePick {
    const int *refs;
    int lo, hi, begin, end, first;
    bool in_use;

    __device__ __forceinline__ bool is(int i) const { return i < hi && (refs[i] != 0) == in_use; }
    __device__ __forceinline__ int count(const int *r, int lo_, int hi_, bool used, int *scratch) {
        refs = r, lo = lo_, hi = hi_, in_use = used;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int share = (hi > lo ? (hi - lo + KV_THREADS - 1) / KV_THREADS : 0) * 32;
        begin = lo + warp * share;
        end = begin + share < hi ? begin + share : hi;
        int c = 0;
#pragma unroll 4
        for (int i = begin + lane; i < end; i += 32) c += is(i) ? 1 : 0;
        c = __reduce_add_sync(0xffffffffu, c);
        int total;
        first = block_scan(lane == 0 ? c : 0, &total, scratch);
        first = __shfl_sync(0xffffffffu, first, 0);
        return total;
    }
    template <typename F>
    __device__ __forceinline__ void each(int wanted, F give) const {
        const int lane = threadIdx.x & 31;
        int rank = first;
        for (int i0 = begin; i0 < end && rank < wanted; i0 += 32) {
            const bool mine = i0 + lane < end && is(i0 + lane);
            const u32 all = __ballot_sync(0xffffffffu, mine);
            const int r = rank + __popc(all & ((1u << lane) - 1u));
            if (mine && r < wanted) give(r, i0 + lane);
            rank += __popc(all);
        }
    }
};

// Shared memory of the planning kernels: 64 ints of scratch, one bit per
// sequence (twice for a fork), then one int per entry (+ 1).
__host__ __device__ constexpr size_t kv_plan_smem(int max_seqs, int n, int maps) {
    return (64 + (size_t)maps * ((max_seqs + 31) / 32) + n + 1) * 4;
}

struct KvExtendParams {
    KvTables t;
    const int *ids, *counts;
    int n;
    int *status;
    int *active;  // [n] or NULL: the ids when the call succeeds, else -1
};

__global__ void __launch_bounds__(KV_THREADS) k_kv_extend(const __grid_constant__ KvExtendParams p) {
    extern __shared__ int smem[];
    int *scratch = smem;
    int *bad = smem + 48;
    const int words = (p.t.max_seqs + 31) / 32;
    u32 *seen = reinterpret_cast<u32 *>(smem + 64);
    int *first = smem + 64 + words;  // first[i] = pages needed by the entries before i
    const int ps = 1 << p.t.ps_log;
    for (int i = threadIdx.x; i < words; i += KV_THREADS) seen[i] = 0;
    if (threadIdx.x == 0) *bad = 0;
    __syncthreads();
    long long sum = 0;
    for (int i0 = 0; i0 < p.n; i0 += KV_THREADS) {
        const int i = i0 + threadIdx.x;
        int need = 0;
        if (i < p.n && p.ids[i] >= 0) {
            const int s = p.ids[i], c = p.counts[i];
            int fault = 0;
            if (s >= p.t.max_seqs || c < 0) {
                fault = KV_BAD;
            } else {
                const int len = p.t.lengths[s];
                if (len < 0 || (atomicOr(&seen[s >> 5], 1u << (s & 31)) >> (s & 31) & 1u)) fault = KV_BAD;
                else if ((long long)len + c > (long long)p.t.max_pages * ps) fault = KV_NO_ROOM;
                else need = (int)(((long long)len + c + ps - 1) >> p.t.ps_log) - (int)(((long long)len + ps - 1) >> p.t.ps_log);
                if (need > p.t.num_pages) fault = KV_NO_PAGES, need = 0;
            }
            if (fault) atomicMax(bad, fault);
        }
        int total;
        const int before = block_scan(need, &total, scratch);
        // (1024 entries of at most 2^20 pages fit an int; a sum beyond the
        // pool is refused below)
        const long long at = sum + before;
        if (i < p.n) first[i] = (int)(at < 0x7fffffffLL ? at : 0x7fffffffLL);
        sum += total;
    }
    __syncthreads();
    PagePick pick;
    const int free_pages = pick.count(p.t.refs, 0, p.t.num_pages, false, scratch);
    const int status = *bad ? *bad : sum > free_pages ? KV_NO_PAGES : KV_OK;
    if (threadIdx.x == 0) *p.status = status;
    if (p.active != nullptr)
        for (int i = threadIdx.x; i < p.n; i += KV_THREADS) p.active[i] = status == KV_OK ? p.ids[i] : -1;
    if (status != KV_OK) return;
    const int want = (int)sum;
    if (threadIdx.x == 0) first[p.n] = want;
    __syncthreads();
    pick.each(want, [&](int rank, int page) {
        int lo = 0, hi = p.n - 1;  // the last entry with first <= rank
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= rank) lo = mid;
            else hi = mid - 1;
        }
        const int s = p.ids[lo];
        const int have = (p.t.lengths[s] + ps - 1) >> p.t.ps_log;
        p.t.tables[(size_t)s * p.t.max_pages + have + (rank - first[lo])] = page;
        p.t.refs[page] = 1;
    });
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += KV_THREADS)
        if (p.ids[i] >= 0) p.t.lengths[p.ids[i]] += p.counts[i];
}

struct KvFreeParams {
    KvTables t;
    const int *ids;
    int n;
};

// One CTA per entry.  refs counts are sums, so the order of the atomics does
// not show.
__global__ void __launch_bounds__(128) k_kv_free(const __grid_constant__ KvFreeParams p) {
    const int i = blockIdx.x, s = p.ids[i];
    if (s < 0) return;
    if (s >= p.t.max_seqs) {
        if (threadIdx.x == 0) raise_device_error(DEVERR_INDEX);
        return;
    }
    // an id listed twice is freed by its first entry
    int dup = 0;
    for (int j = threadIdx.x; j < i; j += 128) dup |= p.ids[j] == s;
    if (__syncthreads_or(dup)) return;
    const int len = p.t.lengths[s];
    const long long pages = ((long long)len + (1 << p.t.ps_log) - 1) >> p.t.ps_log;
    int *row = p.t.tables + (size_t)s * p.t.max_pages;
    bool fault = len < 0 || pages > p.t.max_pages;
    const int m = len <= 0 ? 0 : (int)(pages < p.t.max_pages ? pages : p.t.max_pages);
    for (int j = threadIdx.x; j < m; j += 128) {
        const int page = row[j];
        if (page >= 0 && page < p.t.num_pages) atomicSub(&p.t.refs[page], 1);
        else fault = true;
        row[j] = -1;
    }
    if (fault) raise_device_error(DEVERR_INDEX);
    __syncthreads();  // every thread has read the length
    if (threadIdx.x == 0) p.t.lengths[s] = 0;
}

struct KvForkParams {
    KvTables t;
    const int *src, *dst;
    int n;
    int *status;
    int *plan;  // [0] 1 when the fork goes ahead, then n pairs (old page, new page), -1: none, then n new pages
};

// Validates, takes a page for every last partial page, and notes the copies.
__global__ void __launch_bounds__(KV_THREADS) k_kv_fork_plan(const __grid_constant__ KvForkParams p) {
    extern __shared__ int smem[];
    int *scratch = smem;
    int *bad = smem + 48;
    const int words = (p.t.max_seqs + 31) / 32;
    u32 *is_src = reinterpret_cast<u32 *>(smem + 64), *is_dst = is_src + words;
    int *first = smem + 64 + 2 * words;
    const int mask = (1 << p.t.ps_log) - 1;
    for (int i = threadIdx.x; i < 2 * words; i += KV_THREADS) is_src[i] = 0;
    if (threadIdx.x == 0) *bad = 0;
    __syncthreads();
    // padding: a negative id on either side
    for (int i = threadIdx.x; i < p.n; i += KV_THREADS) {
        const int a = p.src[i], b = p.dst[i];
        if (a < 0 || b < 0) continue;
        if (a >= p.t.max_seqs || b >= p.t.max_seqs) {
            atomicMax(bad, KV_BAD);
            continue;
        }
        atomicOr(&is_src[a >> 5], 1u << (a & 31));
        const int len = p.t.lengths[a];
        const bool twice = atomicOr(&is_dst[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u;
        if (twice || p.t.lengths[b] != 0 || len < 0 || (long long)len > ((long long)p.t.max_pages << p.t.ps_log))
            atomicMax(bad, KV_BAD);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < words; i += KV_THREADS)
        if (is_src[i] & is_dst[i]) atomicMax(bad, KV_BAD);
    __syncthreads();
    int want = 0;
    for (int i0 = 0; i0 < p.n; i0 += KV_THREADS) {
        const int i = i0 + threadIdx.x;
        int need = 0;
        if (i < p.n && !*bad && p.src[i] >= 0 && p.dst[i] >= 0) need = (p.t.lengths[p.src[i]] & mask) != 0;
        int total;
        const int before = want + block_scan(need, &total, scratch);
        if (i < p.n) {
            first[i] = need ? before : -1;
            p.plan[1 + 2 * i] = -1;
        }
        want += total;
    }
    __syncthreads();
    PagePick pick;
    const int free_pages = pick.count(p.t.refs, 0, p.t.num_pages, false, scratch);
    const int status = *bad ? *bad : want > free_pages ? KV_NO_PAGES : KV_OK;
    if (threadIdx.x == 0) {
        *p.status = status;
        p.plan[0] = status == KV_OK;
    }
    if (status != KV_OK) return;
    // the new pages by rank, behind the pairs; entries pick theirs up below
    int *pages = p.plan + 1 + 2 * p.n;
    pick.each(want, [&](int rank, int page) {
        pages[rank] = page;
        p.t.refs[page] = 1;
    });
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += KV_THREADS) {
        const int a = p.src[i], b = p.dst[i];
        if (a < 0 || b < 0) continue;
        const int len = p.t.lengths[a], full = len >> p.t.ps_log;
        if (first[i] >= 0) {
            const int page = pages[first[i]];
            const int old = p.t.tables[(size_t)a * p.t.max_pages + full];
            p.plan[1 + 2 * i] = old < 0 ? -2 : old;  // (-2: the table names no page; the copy reports it)
            p.plan[2 + 2 * i] = page;
            p.t.tables[(size_t)b * p.t.max_pages + full] = page;
        }
        p.t.lengths[b] = len;
    }
}

// Page copies: pool plane q, page a -> page b, 16 bytes per thread and step.
__device__ __forceinline__ void copy_page(uint8_t *pool, long long plane_bytes, long long page_bytes, int plane,
                                          int from, int to) {
    const uint4 *s = reinterpret_cast<const uint4 *>(pool + plane * plane_bytes + from * page_bytes);
    uint4 *d = reinterpret_cast<uint4 *>(pool + plane * plane_bytes + to * page_bytes);
    const long long m = page_bytes >> 4;
    long long i = threadIdx.x;
    for (; i + 3 * KV_COPY_THREADS < m; i += 4 * KV_COPY_THREADS) {
        const uint4 a = s[i], b = s[i + KV_COPY_THREADS], c = s[i + 2 * KV_COPY_THREADS],
                    e = s[i + 3 * KV_COPY_THREADS];
        d[i] = a;
        d[i + KV_COPY_THREADS] = b;
        d[i + 2 * KV_COPY_THREADS] = c;
        d[i + 3 * KV_COPY_THREADS] = e;
    }
    for (; i < m; i += KV_COPY_THREADS) d[i] = s[i];
}

struct KvCopyParams {
    KvTables t;
    uint8_t *pool;
    long long page_bytes;
    int planes;
    const int *src, *dst;  // fork: the entries
    int n;
    const int *plan;
};

__global__ void __launch_bounds__(KV_COPY_THREADS) k_kv_fork_copy(const __grid_constant__ KvCopyParams p) {
    pdl_wait();
    if (p.plan[0] == 0) return;
    const long long plane_bytes = p.page_bytes * p.t.num_pages;
    // shared pages: one CTA per entry
    for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int a = p.src[i], b = p.dst[i];
        if (a < 0 || b < 0) continue;
        const int full = p.t.lengths[a] >> p.t.ps_log;
        for (int j = threadIdx.x; j < full; j += KV_COPY_THREADS) {
            const int page = p.t.tables[(size_t)a * p.t.max_pages + j];
            p.t.tables[(size_t)b * p.t.max_pages + j] = page;
            if (page >= 0 && page < p.t.num_pages) atomicAdd(&p.t.refs[page], 1);
            else raise_device_error(DEVERR_INDEX);
        }
    }
    const long long items = (long long)p.n * p.planes;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int i = (int)(it / p.planes), plane = (int)(it - (long long)i * p.planes);
        const int from = p.plan[1 + 2 * i];
        if (from == -1) continue;
        if (from < 0 || from >= p.t.num_pages) {
            if (threadIdx.x == 0) raise_device_error(DEVERR_INDEX);
            continue;
        }
        copy_page(p.pool, plane_bytes, p.page_bytes, plane, from, p.plan[2 + 2 * i]);
    }
}

struct KvCompactParams {
    KvTables t;  // lengths unused
    int *plan;   // [0] moves m, [1] n_live, [2 ..] m pairs (from, to), then the new number of every page >= n_live
    int *n_live;
};

__global__ void __launch_bounds__(KV_THREADS) k_kv_compact_plan(const __grid_constant__ KvCompactParams p) {
    __shared__ int scratch[64];
    const int n = p.t.num_pages;
    PagePick holes, movers;
    const int live = holes.count(p.t.refs, 0, n, true, scratch);
    const int m = holes.count(p.t.refs, 0, live, false, scratch);
    movers.count(p.t.refs, live, n, true, scratch);
    int *pair = p.plan + 2, *to = p.plan + 2 + 2 * (size_t)n;
    holes.each(m, [&](int rank, int page) { pair[2 * rank + 1] = page; });
    for (int i = live + threadIdx.x; i < n; i += KV_THREADS) to[i] = i;
    movers.each(m, [&](int rank, int page) { pair[2 * rank] = page; });
    __syncthreads();
    for (int r = threadIdx.x; r < m; r += KV_THREADS) {
        const int a = pair[2 * r], b = pair[2 * r + 1];
        to[a] = b;
        p.t.refs[b] = p.t.refs[a];
        p.t.refs[a] = 0;
    }
    if (threadIdx.x == 0) {
        p.plan[0] = m;
        p.plan[1] = live;
        *p.n_live = live;
    }
}

__global__ void __launch_bounds__(KV_COPY_THREADS) k_kv_compact_copy(const __grid_constant__ KvCopyParams p) {
    pdl_wait();
    const int m = p.plan[0], live = p.plan[1];
    const int *to = p.plan + 2 + 2 * (size_t)p.t.num_pages;
    const long long cells = (long long)p.t.max_seqs * p.t.max_pages;
    for (long long i = (long long)blockIdx.x * KV_COPY_THREADS + threadIdx.x; i < cells;
         i += (long long)gridDim.x * KV_COPY_THREADS) {
        const int e = p.t.tables[i];
        if (e >= live && e < p.t.num_pages) p.t.tables[i] = to[e];
    }
    const long long plane_bytes = p.page_bytes * p.t.num_pages;
    const long long items = (long long)m * p.planes;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int r = (int)(it / p.planes), plane = (int)(it - (long long)r * p.planes);
        copy_page(p.pool, plane_bytes, p.page_bytes, plane, p.plan[2 + 2 * r], p.plan[3 + 2 * r]);
    }
}

}  // namespace bl
