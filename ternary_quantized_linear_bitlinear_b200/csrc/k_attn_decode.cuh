// Attention of one new token per sequence over the paged cache.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j), over the
//   visible keys of the sequence (all, or a window and the first sinks)
//
// Bound by memory: every visible K and V row is read once for all query
// heads of its group (at most eight; a group of more heads is read once per
// eight of them).
//
// Work.  Keys are taken in batches of NB consecutive keys (aligned).  The
// batches of all (sequence, head group) segments form one line, each segment
// preceded by AD_OH empty places for what a segment costs besides its
// batches, and the line is cut into equal pieces, one per warp: lengths that
// live on the device and differ wildly still load every warp alike.  A warp
// walks the segments of its piece with a running maximum and sum; a segment
// inside one piece is finished there.  What spans warps of a CTA is merged in
// shared memory, what spans CTAs leaves float32 partials (maximum, sum,
// unnormalised output; at most two per CTA) in the workspace, joined in order
// by k_attn_join, so the result depends on nothing but the inputs and the
// grid.
//
// Inside a warp (DecodeMma, bfloat16 cache; DecodeFma, float32 cache) the K and
// V rows of a batch pass through the warp's own ring of shared-memory slots,
// half a batch each, filled ahead of the arithmetic, so the bytes in flight
// do not hang on registers.
#pragma once

#include "k_attn_ragged.cuh"
#include "k_kv_pages.cuh"

namespace bl {

constexpr int AD_MAX_B = 65535;
constexpr int AD_G = 8;  // query heads per segment at most
constexpr int AD_JOIN_THREADS = 256;
constexpr int AD_MAX_CTAS = 640;      // of a launch (the workspace is sized for them)

struct DecodeAttnParams {
    const uint8_t *q;
    long long q_stride;  // bytes
    int q_bf16;
    int B, Hq, Hkv, D;
    int group;     // query heads per kv head
    int parts;     // head groups per kv head: ceil(group / AD_G)
    int gsize;     // query heads of a full head group
    KvView kv;
    const int *seq_ids;
    int window, sinks;
    float scale_log2;   // scale * log2(e)
    uint8_t *out;
    float *lse;
    long long *open;    // workspace: [CTAs][4] the segment a CTA begins but does not end: sequence (-1: none), first
                        // query head, query heads, last CTA
    float *part;        // workspace: [2 * CTAs][gsize][DP + 2]
};

// The visible batches of a sequence of `len` tokens: sink batches 0 .. ns - 1,
// then the window's from `wb` on; `lo` the first key of the window.
struct Visible {
    int len, lo, ns, wb, count;
};

template <int NB>
__device__ __forceinline__ Visible visible_of(int len, int window, int sinks) {
    Visible v;
    v.len = len;
    v.lo = window > 0 && len > window ? len - window : 0;
    v.wb = v.lo / NB;
    const int s = sinks < v.lo ? sinks : v.lo;
    v.ns = (s + NB - 1) / NB;
    if (v.ns > v.wb) v.ns = v.wb;
    v.count = len <= 0 ? 0 : v.ns + (len - 1) / NB + 1 - v.wb;
    return v;
}

// Length of batch entry b (0 for padding and for bad indexes).
__device__ __forceinline__ int entry_len(const DecodeAttnParams &p, int b, int *seq) {
    const int s = p.seq_ids != nullptr ? __ldg(p.seq_ids + b) : b;
    *seq = s;
    if (s < 0 || s >= p.kv.max_seqs) return 0;
    const int len = __ldg(p.kv.lengths + s);
    const int most = p.kv.max_pages << p.kv.ps_log;
    if (len < 0 || len > most) raise_device_error(DEVERR_INDEX);
    return len < 0 ? 0 : len < most ? len : most;
}

// The line: segment `seg` of sequence b starts at cum[b] + seg * (count +
// AD_OH); its first batch stands AD_OH places later.
constexpr int AD_OH = 6;

__device__ __forceinline__ float redux_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void put_out(const DecodeAttnParams &p, size_t row, int d, float o) {
    if (p.q_bf16) reinterpret_cast<uint16_t *>(p.out)[row * p.D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
    else reinterpret_cast<float *>(p.out)[row * p.D + d] = o;
}
__device__ __forceinline__ void put_lse(const DecodeAttnParams &p, size_t row, float m, float l) {
    if (p.lse != nullptr) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
}

constexpr unsigned long long AD_TIMEOUT_NS = 2000000000ull;
constexpr int AD_SLOT = 4096;  // bytes of a ring slot: K or V rows of one batch, DP * NB elements

// One warp's share of a segment: batches u0 .. u1 - 1 of sequence b.
struct Segment {
    Visible vis;
    const int *table;
    int b, kvh, h0, gn;  // kv head, first query head, query heads
    int u0, u1;
};

// First key of the 8-key block `grp` of batch u.
template <int NB>
__device__ __forceinline__ int first_key(const Visible &v, int u, int grp) {
    return (u < v.ns ? u : v.wb + (u - v.ns)) * NB + grp * 8;
}
template <int NB>
__device__ __forceinline__ int block_page(const DecodeAttnParams &p, const Segment &s, int u, int grp) {
    const int key = first_key<NB>(s.vis, u, grp);
    return u < s.u1 && key < s.vis.len ? __ldg(s.table + (key >> p.kv.ps_log)) : -1;
}
// Which of a block's 8 keys are visible (none when its page is not there), and
// the row number of the first in k_pages / v_pages.
template <int NB>
__device__ __forceinline__ u32 block_rows(const DecodeAttnParams &p, const Segment &s, int u, int grp, int page,
                                          size_t &row, bool &fault) {
    const int key0 = first_key<NB>(s.vis, u, grp);
    const bool ok = page >= 0 && page < p.kv.num_pages;
    fault |= !ok && key0 < s.vis.len;
    row = 0;
    if (!ok) return 0;
    row = (((size_t)page * p.Hkv + s.kvh) << p.kv.ps_log) + (key0 & ((1 << p.kv.ps_log) - 1));
    if (key0 >= s.vis.lo && key0 + 8 <= s.vis.len) return 0xffu;
    u32 live = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int key = key0 + r;
        live |= (key < s.vis.len && (key >= s.vis.lo || key < p.sinks)) ? 1u << r : 0u;
    }
    return live;
}

// float32 cache: products on the CUDA cores, two per instruction
// (fma.rn.f32x2).  LK lanes share a key, each with a 16-byte chunk of its
// row; the KW = 32 / LK key groups own 8 consecutive keys each, which lie in
// one page (pages are aligned blocks of at least 8 tokens) and are contiguous
// in memory: one bulk copy per group fills its part of a slot.  The dot
// products' partial sums are reduced across a key's lanes by a transposing
// butterfly: log2 steps that halve the number of keys a lane holds, 7
// exchanges for 8 keys instead of 8 log2(LK).  Waits on the copies are
// bounded; a warp that gives up raises the device error word and drains its
// copies.
template <int DP_, int G_, int WARPS_, int OCC_, int SLOTS_>
struct DecodeFma {
    static constexpr int DP = DP_, G = G_, WARPS = WARPS_, OCC = OCC_, SLOTS = SLOTS_;
    static constexpr int E = 4, LK = DP / E, KW = 32 / LK, NB = 8 * KW, ES = 4;
    static constexpr int BARS = WARPS * SLOTS;
    static_assert(NB * DP * ES == AD_SLOT, "ring slot");
    uint8_t *ring;
    u32 ring_u32, bars, done = 0;
    u64 policy;
    bool fault = false;
    float m[G], l[G];
    f32x2 acc[G][E / 2];

    __device__ __forceinline__ static void init(u64 *bar) {
        if (threadIdx.x < BARS) mbar_init(smem_u32(bar + threadIdx.x), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __device__ __forceinline__ DecodeFma(uint8_t *r, u64 *bar)
        : ring(r), ring_u32(smem_u32(r)), bars(smem_u32(bar + (threadIdx.x >> 5) * SLOTS)),
          policy(l2_policy_evict_first()) {}

    // false: a wait gave up (nothing of this warp is in flight any more)
    __device__ __forceinline__ bool segment(const DecodeAttnParams &p, const Segment &sg) {
        const int lane = threadIdx.x & 31, sub = lane & (LK - 1), grp = lane / LK;
        const bool in_d = sub * E < p.D;
        const u32 row_bytes = (u32)p.D * ES;
        // half batch i: K (even) or V (odd) of batch u0 + i / 2 into the next slot; `lives` collects which of the
        // lane's 8 keys are visible, 8 bits per batch from the oldest unconsumed one on
        const int halves = 2 * (sg.u1 - sg.u0);
        int issued = 0, page = block_page<NB>(p, sg, sg.u0, grp);
        size_t row = 0;
        u64 lives = 0;
        auto issue = [&](int consumed) {
            const int u = sg.u0 + (issued >> 1);
            u32 live;
            if ((issued & 1) == 0) {
                live = block_rows<NB>(p, sg, u, grp, page, row, fault);
                lives |= (u64)live << (8 * ((issued - consumed) >> 1));
                page = block_page<NB>(p, sg, u + 1, grp);
            } else {
                live = (u32)(lives >> (8 * ((issued - consumed) >> 1))) & 0xffu;
            }
            const u32 slot = done % SLOTS, bar = bars + slot * 8;
            const u32 groups = __ballot_sync(0xffffffffu, live != 0 && sub == 0);
            if (lane == 0) {
                if (groups) mbar_arrive_expect_tx(bar, (u32)__popc(groups) * 8 * row_bytes);
                else mbar_arrive(bar);
            }
            __syncwarp();
            if (live != 0 && sub == 0)
                bulk_g2s_hint(ring_u32 + slot * AD_SLOT + (u32)grp * 8 * row_bytes,
                              ((issued & 1) ? p.kv.v : p.kv.k) + row * row_bytes, 8 * row_bytes, bar, policy);
            ++issued;
            ++done;
        };
        const u32 first = done;
        while (issued < halves && issued < SLOTS) issue(0);

        // q of the group's heads, scaled into the exponent's base 2
        f32x2 q[G][E / 2];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (g < sg.gn && in_d) {
                const size_t at = (size_t)(sg.h0 + g) * p.D + sub * E;
                const uint8_t *src = p.q + sg.b * p.q_stride;
                if (p.q_bf16) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(src + at * 2);
                    x = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
                } else {
                    x = *reinterpret_cast<const float4 *>(src + at * 4);
                }
            }
            q[g][0] = pack2(x.x * p.scale_log2, x.y * p.scale_log2);
            q[g][1] = pack2(x.z * p.scale_log2, x.w * p.scale_log2);
            m[g] = -INFINITY;
            l[g] = 0.f;
            acc[g][0] = acc[g][1] = 0ull;
        }
        bool stuck = false;
        auto landed = [&](int i) {
            const u32 n = first + i, slot = n % SLOTS;
            stuck = __any_sync(0xffffffffu, !mbar_wait(bars + slot * 8, (n / SLOTS) & 1, AD_TIMEOUT_NS, nullptr));
            return ring + slot * AD_SLOT + (size_t)grp * 8 * row_bytes + sub * 16;
        };
        // row r of a slot; zero for a lane behind the head size or a hidden row
        auto chunk = [&](const uint8_t *rows, int r, bool keep, f32x2 (&x)[2]) {
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
            if (keep) w = *reinterpret_cast<const float4 *>(rows + r * row_bytes);
            x[0] = pack2(w.x, w.y);
            x[1] = pack2(w.z, w.w);
        };
        for (int i = 0; i < halves; i += 2) {
            const u32 now = (u32)lives & 0xffu;
            float s[G][8];
            const uint8_t *rows = landed(i);
            if (stuck) break;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                f32x2 x[2];
                chunk(rows, r, in_d, x);  // (a hidden row's score is dropped below)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float lo, hi;
                    unpack2(fma2(x[1], q[g][1], mul2(x[0], q[g][0])), lo, hi);
                    s[g][r] = lo + hi;
                }
            }
            __syncwarp();  // every lane has read the slot
            if (issued < halves) issue(i);
            // transposing butterfly: after it lane `sub` holds key (sub & 7)'s score
            float sc[G];
            const bool mine = now >> (sub & 7) & 1u;
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) {
                    const bool up = sub & o;
#pragma unroll
                    for (int k = 0; k < o; ++k) {
                        const float keep = up ? s[g][k + o] : s[g][k], give = up ? s[g][k] : s[g][k + o];
                        s[g][k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
                float x = s[g][0];
#pragma unroll
                for (int o = 8; o < LK; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                sc[g] = mine ? x : -INFINITY;
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float mx = redux_max(sc[g]);
                if (mx > m[g]) {  // the same for the whole warp
                    const float c = exp2_fast(m[g] - mx);
                    m[g] = mx;
                    l[g] *= c;
                    const f32x2 c2 = pack2(c, c);
                    acc[g][0] = mul2(acc[g][0], c2);
                    acc[g][1] = mul2(acc[g][1], c2);
                }
                sc[g] = mine ? exp2_fast(sc[g] - m[g]) : 0.f;
                l[g] += sc[g];
            }
            rows = landed(i + 1);
            if (stuck) break;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                f32x2 x[2];
                chunk(rows, r, in_d && (now >> r & 1u), x);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float w = __shfl_sync(0xffffffffu, sc[g], r, LK);
                    const f32x2 w2 = pack2(w, w);
                    acc[g][0] = fma2(x[0], w2, acc[g][0]);
                    acc[g][1] = fma2(x[1], w2, acc[g][1]);
                }
            }
            __syncwarp();
            if (issued < halves) issue(i);
            lives >>= 8;
        }
        if (stuck) {
            // the copies in flight land before the CTA exits
            if (lane == 0) {
                raise_device_error(DEVERR_TIMEOUT_PRODUCER);
                for (u32 n = done > SLOTS ? done - SLOTS : 0; n < done; ++n)
                    mbar_wait(bars + n % SLOTS * 8, (n / SLOTS) & 1, AD_TIMEOUT_NS, nullptr);
            }
            __syncwarp();
            return false;
        }
        // the warp's key groups together
#pragma unroll
        for (int g = 0; g < G; ++g) {
            // lanes 8, 16, 24 on of a key repeat its first 8 lanes' scores
            float lw = sub < 8 ? l[g] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
            l[g] = lw;
        }
        return true;
    }

    // give(g, d, value) for the unnormalised output, once for each g < gn and d < DP over the warp's lanes;
    // stat(g, m, l) on one lane
    template <typename A, typename B>
    __device__ __forceinline__ void emit(int gn, A give, B stat) {
        const int lane = threadIdx.x & 31, sub = lane & (LK - 1), grp = lane / LK;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float x[E];
            unpack2(acc[g][0], x[0], x[1]);
            unpack2(acc[g][1], x[2], x[3]);
#pragma unroll
            for (int i = 0; i < E; ++i) {
#pragma unroll
                for (int o = LK; o < 32; o <<= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
            }
            if (g >= gn) continue;
            if (grp == 0) {
#pragma unroll
                for (int i = 0; i < E; ++i) give(g, sub * E + i, x[i], l[g]);
            }
            if (lane == 0) stat(g, m[g], l[g]);
        }
    }
};

// bfloat16 cache: products on mma.sync (m16n8k16), heads as rows of A.  The
// cache's rows are exact in bfloat16; what is not is split into bfloat16
// terms that stand in the rows of the same product, so that nothing is
// rounded below 32 bits:
//   DEC_BF16  bfloat16 q, up to 8 heads: q is one term (rows 0 - 7); the
//             weights p two (rows 0 - 7 and 8 - 15: 2^-16 relative beside the
//             output's half step of 2^-8)
//   DEC_F32_4 float32 q, up to 4 heads: q and p three terms each (24 bits) in
//             rows g, g + 8 and g + 4
//   DEC_F32_8 float32 q, up to 8 heads: rows g and g + 8, and the third
//             terms in a second product
// Terms of a row g and g + 8 meet in one thread; those of g and g + 4 in two,
// which add them by one exchange and both go on with the sum.  On the CUDA
// cores a batch took 1220 instructions for three heads, 58 % of the issue
// slots at half of the copy bandwidth; here 8 x 65000 keys of 12 / 4 heads
// run at 6.2 TB/s, and the second products of DEC_F32_8 cost a tenth (64 x 1028
// keys of 20 unshared heads 130 instead of 119 us), which is why up to 4 heads
// do without.  Groups of 8 heads of 128, 64 x 6000 keys: 52 us with bfloat16 q,
// 73 us with float32 q (three terms' operands and 64 of output a thread: 208
// bytes of them spill).
// Rows go into the slots by 16-byte cp.async with the chunks permuted by the
// row (tile_at), hidden rows as zeros.
enum { DEC_BF16, DEC_F32_4, DEC_F32_8 };

template <int DP_, int MODE, int WARPS_, int OCC_, int SLOTS_>
struct DecodeMma {
    static constexpr bool PACKED = MODE == DEC_F32_4, THIRD = MODE == DEC_F32_8;
    static constexpr int DP = DP_, G = PACKED ? 4 : 8, WARPS = WARPS_, OCC = OCC_, SLOTS = SLOTS_;
    static constexpr int LK = DP / 8, KW = 32 / LK, NB = 8 * KW;
    static constexpr int BARS = 1;
    static_assert(NB * DP * 2 == AD_SLOT, "ring slot");
    u32 ring;
    bool fault = false;
    float m, l;  // of row lane / 4; l a share of the quad's sum
    float acc[DP / 8][4];

    __device__ __forceinline__ static void init(u64 *) {}
    __device__ __forceinline__ DecodeMma(uint8_t *r, u64 *) : ring(smem_u32(r)) {}

    // bfloat16 pairs of two floats and what they leave
    __device__ __forceinline__ static u32 take(float &a, float &b) {
        const u32 w = pack_bf16(a, b);
        a -= __uint_as_float(w << 16);
        b -= __uint_as_float(w & 0xffff0000u);
        return w;
    }

    __device__ __forceinline__ bool segment(const DecodeAttnParams &p, const Segment &sg) {
        const int lane = threadIdx.x & 31, sub = lane & (LK - 1), grp = lane / LK;
        const bool in_d = sub * 8 < p.D;
        const u32 row_bytes = (u32)p.D * 2;
        const int halves = 2 * (sg.u1 - sg.u0);
        int issued = 0, page = block_page<NB>(p, sg, sg.u0, grp);
        const uint8_t *kp = p.kv.k, *vp = p.kv.v;
        u64 lives = 0;
        // half batch i: K (even) or V (odd) of batch u0 + i / 2
        auto issue = [&](int consumed) {
            if (issued < halves) {
                u32 live;
                if ((issued & 1) == 0) {
                    const int u = sg.u0 + (issued >> 1);
                    size_t row;
                    live = block_rows<NB>(p, sg, u, grp, page, row, fault);
                    lives |= (u64)live << (8 * ((issued - consumed) >> 1));
                    kp = p.kv.k + row * row_bytes + sub * 16;
                    vp = p.kv.v + row * row_bytes + sub * 16;
                    page = block_page<NB>(p, sg, u + 1, grp);
                } else {
                    live = (u32)(lives >> (8 * ((issued - consumed) >> 1))) & 0xffu;
                }
                if (!in_d) live = 0;
                const uint8_t *src = (issued & 1) ? vp : kp;
                const u32 base = ring + (u32)(issued % SLOTS) * AD_SLOT;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const u32 dst = tile_at<DP>(base, grp * 8 + r, sub);
                    const u32 n = (live >> r & 1u) ? 16u : 0u;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                                 "l"(n ? src + r * row_bytes : src), "r"(n)
                                 : "memory");
                }
            }
            cp_commit();  // (an empty group when nothing is left: the waits count groups)
            ++issued;
        };
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) issue(0);

        u32 qa[DP / 16][4], ql[THIRD ? DP / 16 : 1][2];
        const bool low = !PACKED || lane < 16;  // this thread's rows carry the first two terms (else the third)
        {
            const int g = PACKED ? (lane >> 2) & 3 : lane >> 2;
            const uint8_t *src = p.q + sg.b * p.q_stride;
            const size_t at = (size_t)(sg.h0 + g) * p.D + (lane & 3) * 2;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int d = kk * 16 + h * 8;
                    const bool ok = g < sg.gn && d < p.D;
                    if (MODE != DEC_BF16) {
                        float2 x = ok ? *reinterpret_cast<const float2 *>(src + (at + d) * 4) : make_float2(0.f, 0.f);
                        const u32 w1 = take(x.x, x.y), w2 = take(x.x, x.y), w3 = take(x.x, x.y);
                        qa[kk][2 * h] = low ? w1 : w3;
                        qa[kk][2 * h + 1] = low ? w2 : 0u;
                        if (THIRD) ql[kk][h] = w3;
                    } else {
                        qa[kk][2 * h] = ok ? *reinterpret_cast<const u32 *>(src + (at + d) * 2) : 0u;
                        qa[kk][2 * h + 1] = 0u;
                    }
                }
            }
        }
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        const float sl = p.scale_log2;
        for (int i = 0; i < halves; i += 2) {
            const u32 now = (u32)lives & 0xffu;
            const bool full = __all_sync(0xffffffffu, now == 0xffu);
            float s[KW][4], s3[THIRD ? KW : 1][4];  // (the third terms apart: shorter chains of products)
#pragma unroll
            for (int n = 0; n < KW; ++n) {
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
                if (THIRD) s3[n][0] = s3[n][1] = s3[n][2] = s3[n][3] = 0.f;
            }
            cp_wait<SLOTS - 1>();
            __syncwarp();
            const u32 kb = ring + (u32)(i % SLOTS) * AD_SLOT;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
#pragma unroll
                for (int n = 0; n < KW; n += 2) {
                    u32 b[4];
                    b_frag<DP>(b, kb, n * 8, kk);
                    mma_bf16(s[n], qa[kk], b[0], b[1]);
                    mma_bf16(s[n + 1], qa[kk], b[2], b[3]);
                    if (THIRD) {
                        const u32 a[4] = {ql[kk][0], 0u, ql[kk][1], 0u};
                        mma_bf16(s3[n], a, b[0], b[1]);
                        mma_bf16(s3[n + 1], a, b[2], b[3]);
                    }
                }
            }
            __syncwarp();  // every lane has read the slot
            issue(i);
            float mx = -INFINITY;
#pragma unroll
            for (int n = 0; n < KW; ++n) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (MODE != DEC_BF16) s[n][x] += s[n][x + 2];
                    if (THIRD) s[n][x] += s3[n][x];
                    if (PACKED) s[n][x] += __shfl_xor_sync(0xffffffffu, s[n][x], 16);
                    s[n][x] *= sl;
                }
                if (!full) {
                    const u32 live = __shfl_sync(0xffffffffu, now, n * LK) >> ((lane & 3) * 2);
                    if (!(live & 1u)) s[n][0] = -INFINITY;
                    if (!(live & 2u)) s[n][1] = -INFINITY;
                }
                mx = fmaxf(mx, fmaxf(s[n][0], s[n][1]));
            }
            mx = quad_max(mx);
            // the base moves only when a score passes it by 2^8: sums of weights up to 256 are as exact
            if (__any_sync(0xffffffffu, mx > m + 8.f)) {
                const float top = fmaxf(m, mx), c = top == -INFINITY ? 1.f : exp2_fast(m - top);
                m = top;
                l *= c;
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    acc[n][0] *= c, acc[n][1] *= c, acc[n][2] *= c, acc[n][3] *= c;
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int n = 0; n < KW; ++n) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    s[n][x] = exp2_fast(s[n][x] - base);
                    l += s[n][x];
                }
            }
            cp_wait<SLOTS - 1>();
            __syncwarp();
            const u32 vb = ring + (u32)((i + 1) % SLOTS) * AD_SLOT;
#pragma unroll
            for (int kk = 0; kk < KW / 2; ++kk) {
                u32 a[4], al[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = s[2 * kk + h][0], y = s[2 * kk + h][1];
                    const u32 w1 = take(x, y), w2 = take(x, y);
                    if (MODE != DEC_BF16) al[h] = take(x, y);
                    a[2 * h] = low ? w1 : al[h];
                    a[2 * h + 1] = low ? w2 : 0u;
                }
#pragma unroll
                for (int n = 0; n < DP / 16; ++n) {
                    u32 b[4];
                    bt_frag<DP>(b, vb, kk * 16, n * 2);
                    mma_bf16(acc[2 * n], a, b[0], b[1]);
                    mma_bf16(acc[2 * n + 1], a, b[2], b[3]);
                    if (THIRD) {
                        const u32 a2[4] = {al[0], 0u, al[1], 0u};
                        mma_bf16(acc[2 * n], a2, b[0], b[1]);
                        mma_bf16(acc[2 * n + 1], a2, b[2], b[3]);
                    }
                }
            }
            __syncwarp();
            issue(i);
            lives >>= 8;
        }
        cp_wait<0>();
        l = quad_sum(l);
        return true;
    }

    template <typename A, typename B>
    __device__ __forceinline__ void emit(int gn, A give, B stat) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v = acc[n][x] + acc[n][x + 2];
                if (PACKED) v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (g < gn) give(g, n * 8 + (lane & 3) * 2 + x, v, l);
            }
        }
        if (g < gn && (lane & 3) == 0) stat(g, m, l);
    }
};

// Shared memory of a CTA: the warps' rings, then one partial per warp (of the
// segment its piece begins in; the one its piece ends in reuses the ring).
template <typename C>
__host__ __device__ constexpr int ad_smem(int gsize) {
    return C::WARPS * (C::SLOTS * AD_SLOT + gsize * (C::DP + 2) * 4);
}

template <typename C>
__global__ void __launch_bounds__(C::WARPS * 32, C::OCC) k_attn_decode(const __grid_constant__ DecodeAttnParams p) {
    constexpr int WARPS = C::WARPS, DP = C::DP, NB = C::NB, T = WARPS * 32, RING = C::SLOTS * AD_SLOT;
    constexpr int ROW = DP + 2;
    static_assert(C::G * ROW * 4 <= RING, "a partial fits a ring");
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ __align__(8) u64 s_bar[C::BARS];
    __shared__ long long scratch[33], s_before[WARPS];
    __shared__ int s_b[WARPS];
    __shared__ int s_pb[2 * WARPS], s_pseg[2 * WARPS];      // whose partial (sequence, segment), -1: none
    __shared__ long long s_p0[2 * WARPS], s_p1[2 * WARPS];  // line places of that segment's first and last batch
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int segs = p.Hkv * p.parts;              // segments of a sequence
    const long long gw = (long long)gridDim.x * WARPS;
    // partial slot 2 w: of the segment in which warp w's piece begins, 2 w + 1: in which it ends
    auto partial = [&](int e, int g) {
        return (e & 1 ? reinterpret_cast<float *>(s_ring + (size_t)(e >> 1) * RING)
                      : reinterpret_cast<float *>(s_ring + (size_t)WARPS * RING) + (e >> 1) * p.gsize * ROW) +
               g * ROW;
    };
    __shared__ int s_empty;  // some entry of this CTA's share (every gridDim.x-th) sees nothing
    if (threadIdx.x < 2 * WARPS) s_pb[threadIdx.x] = -1;
    if (threadIdx.x == 0) s_empty = 0;
    C::init(s_bar);
    pdl_wait();
    // an entry without a visible key (its sequence is empty, or a bad index says so): zeros, written by the whole CTA
    // (by the thread that met it, 20 heads of 128 took 65 us)
    auto nothing_seen = [&](int b) {
        const int seq = p.seq_ids != nullptr ? __ldg(p.seq_ids + b) : b;
        if (seq < 0) return;  // padding
        if (seq >= p.kv.max_seqs) {
            if (threadIdx.x == 0) raise_device_error(DEVERR_INDEX);
            return;
        }
        const long long row = (long long)p.Hq * p.D * (p.q_bf16 ? 2 : 4);
        uint4 *out = reinterpret_cast<uint4 *>(p.out + b * row);
        for (int i = threadIdx.x; i < (int)(row >> 4); i += T) out[i] = make_uint4(0, 0, 0, 0);
        for (int h = threadIdx.x; h < p.Hq; h += T) put_lse(p, (size_t)b * p.Hq + h, 0.f, 0.f);
    };
    // the sequences in which the pieces of this CTA's warps begin
    auto places = [&](int b) {  // of one segment of sequence b
        int seq, n = 0;
        if (b < p.B) n = visible_of<NB>(entry_len(p, b, &seq), p.window, p.sinks).count;
        return n > 0 ? n + AD_OH : 0;
    };
    const int mine = places(threadIdx.x);  // (a batch of at most T sequences is looked at once)
    long long at = 0;
    if (p.B > T) {
        for (int b0 = 0; b0 < p.B; b0 += T) {
            long long sum;  // (lengths up to 2^31: 64 bits)
            block_scan<long long>(b0 == 0 ? mine : places(b0 + threadIdx.x), &sum, scratch);
            at += sum * segs;
        }
    }
    long long total = at;
    at = 0;
    for (int b0 = 0; b0 < p.B; b0 += T) {
        const int b = b0 + threadIdx.x;
        const int n = b0 == 0 ? mine : places(b);
        long long sum;
        const long long pre = block_scan<long long>(n, &sum, scratch);
        if (p.B <= T) total = sum * segs;
        const long long piece = (total + gw - 1) / gw;
        const long long here = at + pre * segs, next = here + (long long)n * segs;
        if (b < p.B && n == 0 && b % gridDim.x == blockIdx.x) s_empty = 1;
        if (n > 0) {
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const long long begin = ((long long)blockIdx.x * WARPS + w) * piece;
                if (here <= begin && begin < next) {
                    s_b[w] = b;
                    s_before[w] = here;
                }
            }
        }
        at += sum * segs;
    }
    if (threadIdx.x == 0) p.open[blockIdx.x * 4] = -1;
    __syncthreads();
    if (s_empty)
        for (int b = blockIdx.x; b < p.B; b += gridDim.x)
            if (places(b) == 0) nothing_seen(b);
    const long long piece = (total + gw - 1) / gw;
    const long long from = ((long long)blockIdx.x * WARPS + warp) * piece;
    const long long end = from + piece < total ? from + piece : total;
    at = from;
    int b = 0;
    long long before = 0;
    if (at < end) {
        b = s_b[warp];
        before = s_before[warp];
    }

    C core(s_ring + (size_t)warp * RING, s_bar);
    while (at < end && b < p.B) {
        // the segment at `at`
        int seq;
        Segment sg;
        sg.vis = visible_of<NB>(entry_len(p, b, &seq), p.window, p.sinks);
        const int width = sg.vis.count + AD_OH;
        if (sg.vis.count == 0 || at >= before + (long long)width * segs) {
            before += sg.vis.count == 0 ? 0 : (long long)width * segs;
            ++b;
            continue;
        }
        const int seg = (int)((at - before) / width);
        const long long seg_at = before + (long long)seg * width + AD_OH;
        sg.u0 = at > seg_at ? (int)(at - seg_at) : 0;
        sg.u1 = end - seg_at < sg.vis.count ? (int)(end - seg_at) : sg.vis.count;
        at = seg_at + sg.vis.count;
        if (sg.u1 <= sg.u0) continue;  // the piece ends before the segment's first batch
        const int part = seg % p.parts;
        sg.b = b;
        sg.kvh = seg / p.parts;
        sg.h0 = sg.kvh * p.group + part * p.gsize;
        sg.gn = p.group - part * p.gsize < p.gsize ? p.group - part * p.gsize : p.gsize;
        sg.table = p.kv.tables + (size_t)seq * p.kv.max_pages;
        if (!core.segment(p, sg)) break;
        if (sg.u0 == 0 && sg.u1 == sg.vis.count) {
            const size_t row = (size_t)b * p.Hq + sg.h0;
            core.emit(
                sg.gn, [&](int g, int d, float x, float l) { if (d < p.D) put_out(p, row + g, d, l > 0.f ? x / l : 0.f); },
                [&](int g, float m, float l) { put_lse(p, row + g, m, l); });
        } else {
            const int slot = 2 * warp + (seg_at <= from ? 0 : 1);
            __syncwarp();
            if (lane == 0) {
                s_pb[slot] = b;
                s_pseg[slot] = seg;
                s_p0[slot] = seg_at;
                s_p1[slot] = seg_at + sg.vis.count - 1;
            }
            core.emit(
                sg.gn, [&](int g, int d, float x, float) { partial(slot, g)[d] = x; },
                [&](int g, float m, float l) {
                    partial(slot, g)[DP] = m;
                    partial(slot, g)[DP + 1] = l;
                });
        }
    }
    if (core.fault) raise_device_error(DEVERR_INDEX);
    __syncthreads();
    // runs of partials of one segment (neighbours among those present)
    const long long cta_piece = piece * WARPS;
    for (int e = 0; e < 2 * WARPS;) {
        const int pb = s_pb[e], pseg = s_pseg[e];
        if (pb < 0) {
            ++e;
            continue;
        }
        int f = e + 1;  // behind the run
        for (int k = e + 1; k < 2 * WARPS; ++k) {
            if (s_pb[k] < 0) continue;
            if (s_pb[k] != pb || s_pseg[k] != pseg) break;
            f = k + 1;
        }
        const int c0 = (int)(s_p0[e] / cta_piece), c1 = (int)(s_p1[e] / cta_piece);
        const int kvh = pseg / p.parts, part = pseg - kvh * p.parts;
        const int h0 = kvh * p.group + part * p.gsize;
        const int gn = p.group - part * p.gsize < p.gsize ? p.group - part * p.gsize : p.gsize;
        float *out = p.part + ((size_t)blockIdx.x * 2 + (c0 < (int)blockIdx.x ? 0 : 1)) * p.gsize * ROW;
        for (int i = threadIdx.x; i < gn * DP; i += T) {
            const int g = i / DP, d = i - g * DP;
            float mm = -INFINITY;
            for (int k = e; k < f; ++k)
                if (s_pb[k] >= 0) mm = fmaxf(mm, partial(k, g)[DP]);
            float a = 0.f, ll = 0.f;
            for (int k = e; k < f; ++k) {
                if (s_pb[k] < 0) continue;
                const float *row = partial(k, g);
                const float c = row[DP] == -INFINITY ? 0.f : exp2_fast(row[DP] - mm);
                a += c * row[d];
                ll += c * row[DP + 1];
            }
            if (i == 0 && c0 == (int)blockIdx.x && c1 > c0) {
                p.open[blockIdx.x * 4 + 1] = h0;
                p.open[blockIdx.x * 4 + 2] = gn;
                p.open[blockIdx.x * 4 + 3] = c1;
                p.open[blockIdx.x * 4] = pb;
            }
            if (c0 == c1) {
                const size_t row = (size_t)pb * p.Hq + h0 + g;
                if (d < p.D) put_out(p, row, d, ll > 0.f ? a / ll : 0.f);
                if (d == 0) put_lse(p, row, mm, ll);
            } else {
                out[g * ROW + d] = a;
                if (d == 0) {
                    out[g * ROW + DP] = mm;
                    out[g * ROW + DP + 1] = ll;
                }
            }
        }
        e = f;
    }
}

// Joins what spans CTAs: CTA (c, g) the g-th query head of the segment that
// CTA c of the launch before began and left open.
template <int DP>
__global__ void __launch_bounds__(AD_JOIN_THREADS) k_attn_join(const __grid_constant__ DecodeAttnParams p) {
    constexpr int ROW = DP + 2;
    const int c0 = blockIdx.x, g = blockIdx.y, d = threadIdx.x;
    pdl_wait();
    const long long b = p.open[c0 * 4];
    const int h0 = (int)p.open[c0 * 4 + 1], gn = (int)p.open[c0 * 4 + 2], n = (int)p.open[c0 * 4 + 3] - c0 + 1;
    if (b < 0 || g >= gn) return;
    const size_t row = (size_t)b * p.Hq + h0 + g;
    // CTA c0 holds the segment's beginning in its second slot, the others what follows in their first
    auto part_of = [&](int i) {
        return p.part + (((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * p.gsize + g) * ROW;
    };
    __shared__ float s_w[AD_MAX_CTAS], s_red[AD_JOIN_THREADS / 32][2], s_acc[AD_JOIN_THREADS / DP][DP];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float mm = -INFINITY;
    for (int i = threadIdx.x; i < n; i += AD_JOIN_THREADS) {
        s_w[i] = part_of(i)[DP];
        mm = fmaxf(mm, s_w[i]);
    }
    mm = redux_max(mm);
    if (lane == 0) s_red[warp][0] = mm;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < AD_JOIN_THREADS / 32; ++w) mm = fmaxf(mm, s_red[w][0]);
    float ll = 0.f;
    for (int i = threadIdx.x; i < n; i += AD_JOIN_THREADS) {
        const float c = s_w[i] == -INFINITY ? 0.f : exp2_fast(s_w[i] - mm);
        s_w[i] = c;
        ll += c * part_of(i)[DP + 1];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
    if (lane == 0) s_red[warp][1] = ll;
    __syncthreads();
    ll = 0.f;
#pragma unroll
    for (int w = 0; w < AD_JOIN_THREADS / 32; ++w) ll += s_red[w][1];
    // DP threads take a partial each time
    const int dd = threadIdx.x % DP, slice = threadIdx.x / DP;
    float a = 0.f;
#pragma unroll 8
    for (int i = slice; i < n; i += AD_JOIN_THREADS / DP) a += s_w[i] * part_of(i)[dd];
    s_acc[slice][dd] = a;
    __syncthreads();
    if (d < p.D) {
        a = 0.f;
#pragma unroll
        for (int k = 0; k < AD_JOIN_THREADS / DP; ++k) a += s_acc[k][d];
        put_out(p, row, d, ll > 0.f ? a / ll : 0.f);
    }
    if (d == 0) put_lse(p, row, mm, ll);
}

}  // namespace bl
