// Causal attention over a ragged batch with a sliding window and sinks, and
// its gradients: what the forward and backward kernels share.
#pragma once

#include "k_rope_append.cuh"

namespace bl {

struct RaggedParams {
    const uint16_t *q, *k, *v, *dout;
    long long q_stride, k_stride, v_stride, do_stride;  // elements
    int Tq, Tk, Hq, Hkv, D, group;
    const int *cu_q, *cu_k;
    int B, max_q, max_k;
    int window, sinks;
    float scale, scale_log2;  // scale, scale * log2(e)
    uint16_t *o;
    float *lse;               // [Hq, Tq]
    const float *delta;       // [Hq, Tq]
    uint16_t *dq, *dk, *dv;
};

// One batch entry: query rows q0 .. q0 + nq - 1, key rows k0 .. k0 + nk - 1;
// query i stands at position i + off.  Queries beyond max_q are left out (no
// CTA computes their lse and delta, so none may read them).
struct Entry {
    int q0, nq, k0, nk, off;
};

__device__ __forceinline__ bool entry_of(const RaggedParams &p, int b, Entry &e) {
    const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
    const int k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
    e = Entry{q0, 0, k0, 0, 0};
    if (q0 < 0 || q1 < q0 || q1 > p.Tq || k0 < 0 || k1 < k0 || k1 > p.Tk) return false;
    e.nq = q1 - q0;
    e.nk = k1 - k0;
    e.off = e.nk - e.nq;
    if (e.nq > p.max_q) e.nq = p.max_q;
    return true;
}

// Reports an entry that a launch cannot compute as described.
__device__ __forceinline__ void check_entry(const RaggedParams &p, int b) {
    Entry e;
    if (!entry_of(p, b, e) || e.nk - e.off > p.max_q || e.nk > p.max_k) raise_device_error(DEVERR_INDEX);
}

// Key tiles of BK keys that queries at positions p0 .. p1 can see: sink tiles
// 0 .. ns - 1, then wt .. wt + nw - 1.
struct KeyTiles {
    int ns, wt, count;
};
template <int BK>
__device__ __forceinline__ KeyTiles key_tiles(const RaggedParams &p, int p0, int p1, int nk) {
    KeyTiles t{0, 0, 0};
    if (p1 > nk - 1) p1 = nk - 1;
    if (p1 < 0) return t;
    if (p0 < 0) p0 = 0;
    const int last = p1 / BK;
    const int lo = p.window > 0 && p0 >= p.window ? p0 - p.window + 1 : 0;
    t.wt = lo / BK;
    const int s = p.sinks < lo ? p.sinks : lo;
    t.ns = (s + BK - 1) / BK;
    if (t.ns > t.wt) t.ns = t.wt;
    t.count = t.ns + last + 1 - t.wt;
    return t;
}

__device__ __forceinline__ void ldsm4(u32 (&r)[4], u32 addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(u32 (&r)[4], u32 addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const u32 (&a)[4], u32 b0, u32 b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Tiles of rows x DP bf16 in shared memory, rows of DP * 2 bytes whose
// 16-byte chunks are permuted by the row (chunk ^ (row & 7)), so that the
// eight rows of an ldmatrix lie in different banks.
template <int DP>
__device__ __forceinline__ u32 tile_at(u32 base, int row, int chunk) {
    return base + (u32)(row * DP * 2) + (u32)((chunk ^ (row & 7)) << 4);
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// B operand for two n-tiles of 8 rows (n = tile rows, k = columns): r[0..1] the first, r[2..3] the second
template <int DP>
__device__ __forceinline__ void b_frag(u32 (&r)[4], u32 base, int row0, int kk) {
    const int lane = threadIdx.x & 31;
    ldsm4(r, tile_at<DP>(base, row0 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
}
// B operand for two n-tiles of 8 columns (n = tile columns, k = rows row0 .. + 15)
template <int DP>
__device__ __forceinline__ void bt_frag(u32 (&r)[4], u32 base, int row0, int chunk) {
    const int lane = threadIdx.x & 31;
    ldsm4t(r, tile_at<DP>(base, row0 + (lane & 15), chunk + (lane >> 4)));
}

__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

}  // namespace bl
