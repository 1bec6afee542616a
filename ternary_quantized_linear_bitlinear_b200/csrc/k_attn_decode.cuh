// Attention of one new token per sequence over the paged cache.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j), over the
//   visible keys of the sequence (all, or a window and the first sinks)
//
// Bound by memory: every visible K and V row is read once for all query
// heads of its group (4 D bf16 bytes per key and kv head).  At ~23 bytes per
// clock and SM of HBM the products cost 0.5 FMA per byte and query head, so
// float32 FMAs on the CUDA cores (two per instruction, fma.rn.f32x2) keep up
// to eight heads a group, and nothing is rounded below 32 bits.  A group of
// more heads is read once per eight of them.
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
// Layout inside a warp: LK lanes share a key, each with a 16-byte chunk of
// its row, and the KW = 32 / LK key groups own 8 consecutive keys each, all
// in one page (pages are aligned blocks of at least 8 tokens), which are
// contiguous in memory: one bulk copy per group brings a batch's K or V rows
// into the warp's own ring of shared-memory slots, SLOTS half batches deep,
// so that up to 12 KB per warp are in flight whatever the arithmetic does and
// no register holds a row before it is used (with the rows in registers a
// group of three heads had eight warps per SM and read 4.5 TB/s).
// The dot products' partial sums are reduced across a key's lanes by a
// transposing butterfly: log2 steps that halve the number of keys a lane
// holds, 7 exchanges for 8 keys instead of 8 log2(LK).
// Waits on the copies are bounded; a warp that gives up raises the device
// error word and drains its copies.
#pragma once

#include "k_kv_pages.cuh"
#include "k_rope_append.cuh"

namespace bl {

constexpr int AD_MAX_B = 65535;
constexpr int AD_G = 8;  // query heads per segment at most
constexpr int AD_JOIN_THREADS = 128;  // >= the head size
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
    long long *cum;     // workspace: [B + 1] line places before sequence b's segments
    float *part;        // workspace: [2 * CTAs][gsize][DP + 2]
};

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
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
    return len < 0 ? 0 : len < most ? len : most;
}

template <bool BF16, int DP>
struct DecodeShape {
    static constexpr int E = BF16 ? 8 : 4;       // elements of a lane's chunk
    static constexpr int LK = DP / E;            // lanes per key
    static constexpr int KW = 32 / LK;           // key groups of a warp
    static constexpr int NB = 8 * KW;            // keys of a batch
};

// The line: segment `seg` of sequence b starts at cum[b] + seg * (count +
// AD_OH); its first batch stands AD_OH places later.
constexpr int AD_OH = 1;

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

// Shared memory of a CTA: the warps' rings of half batches (DP * NB rows of K
// or V, 4 KiB each), then one partial per warp (of the segment its piece
// begins in; the one its piece ends in reuses the ring).
constexpr int AD_SLOT = 4096;
__host__ __device__ constexpr int ad_smem(int warps, int g, int dp, int slots) {
    return warps * (slots * AD_SLOT + g * (dp + 2) * 4);
}

template <bool BF16, int DP, int G, int WARPS, int OCC, int SLOTS>
__global__ void __launch_bounds__(WARPS * 32, OCC) k_attn_decode(const __grid_constant__ DecodeAttnParams p) {
    using S = DecodeShape<BF16, DP>;
    constexpr int E = S::E, LK = S::LK, KW = S::KW, NB = S::NB, T = WARPS * 32;
    constexpr int ROW = DP + 2, ES = BF16 ? 2 : 4;
    static_assert(NB * DP * ES == AD_SLOT && G * ROW * 4 <= SLOTS * AD_SLOT, "decode attention ring");
    extern __shared__ __align__(128) uint8_t s_ring[];  // [WARPS][SLOTS][AD_SLOT], then [WARPS][G][ROW] floats
    __shared__ __align__(8) u64 s_bar[WARPS * SLOTS];
    __shared__ int scratch[64];
    __shared__ long long s_total, s_before[WARPS];
    __shared__ int s_b[WARPS];
    __shared__ int s_pb[2 * WARPS], s_pseg[2 * WARPS];      // whose partial (sequence, segment), -1: none
    __shared__ long long s_p0[2 * WARPS], s_p1[2 * WARPS];  // line places of that segment's first and last batch
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane & (LK - 1), grp = lane / LK;
    const int segs = p.Hkv * p.parts;              // segments of a sequence
    const long long gw = (long long)gridDim.x * WARPS;
    uint8_t *ring = s_ring + (size_t)warp * SLOTS * AD_SLOT;
    const u32 ring_u32 = smem_u32(ring), bars = smem_u32(s_bar + warp * SLOTS);
    // partial slot 2 w: of the segment in which warp w's piece begins, 2 w + 1: in which it ends
    auto partial = [&](int e, int g) {
        return (e & 1 ? reinterpret_cast<float *>(s_ring + (size_t)(e >> 1) * SLOTS * AD_SLOT)
                      : reinterpret_cast<float *>(s_ring + (size_t)WARPS * SLOTS * AD_SLOT) + (e >> 1) * G * ROW) +
               g * ROW;
    };
    if (threadIdx.x < 2 * WARPS) s_pb[threadIdx.x] = -1;
    if (threadIdx.x < WARPS * SLOTS) mbar_init(smem_u32(s_bar + threadIdx.x), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();

    // places before each sequence (CTA 0 leaves them for the join), and the
    // sequences in which the pieces of this CTA's warps begin
    for (int pass = 0; pass < 2; ++pass) {
        const long long piece = pass == 0 ? 1 : (s_total + gw - 1) / gw;
        long long at = 0;
        for (int b0 = 0; b0 < p.B; b0 += T) {
            const int b = b0 + threadIdx.x;
            int seq, n = 0;
            if (b < p.B) n = visible_of<NB>(entry_len(p, b, &seq), p.window, p.sinks).count;
            if (n > 0) n += AD_OH;
            int sum;
            const int pre = block_scan(n, &sum, scratch);
            if (pass == 1 && b < p.B) {
                const long long here = at + (long long)pre * segs, next = here + (long long)n * segs;
                if (blockIdx.x == 0) p.cum[b] = here;
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
            }
            at += (long long)sum * segs;
        }
        if (threadIdx.x == 0) {
            s_total = at;
            if (pass == 1 && blockIdx.x == 0) p.cum[p.B] = at;
        }
        __syncthreads();
    }
    const long long total = s_total;
    const long long piece = (total + gw - 1) / gw;
    const long long from = ((long long)blockIdx.x * WARPS + warp) * piece;
    const long long end = from + piece < total ? from + piece : total;
    long long at = from;
    int b = 0;
    long long before = 0;
    if (at < end) {
        b = s_b[warp];
        before = s_before[warp];
    }

    bool fault = false, stuck = false;
    u32 done = 0;  // half batches this warp has issued so far (all of them consumed between segments)
    const u64 policy = l2_policy_evict_first();
    while (at < end && !stuck) {
        // the segment at `at`: sequence b, kv head, part; u0 .. u1 its batches of this piece
        int seq;
        const Visible vis = visible_of<NB>(entry_len(p, b, &seq), p.window, p.sinks);
        const int width = vis.count + AD_OH;
        if (vis.count == 0 || at >= before + (long long)width * segs) {
            before += vis.count == 0 ? 0 : (long long)width * segs;
            ++b;
            continue;
        }
        const int seg = (int)((at - before) / width);
        const long long seg_at = before + (long long)seg * width + AD_OH;
        const int u0 = at > seg_at ? (int)(at - seg_at) : 0;
        const int u1 = end - seg_at < vis.count ? (int)(end - seg_at) : vis.count;
        at = seg_at + vis.count;
        if (u1 <= u0) continue;  // the piece ends before the segment's first batch
        const int kvh = seg / p.parts, part = seg - kvh * p.parts;
        const int h0 = kvh * p.group + part * p.gsize;
        const int gn = p.group - part * p.gsize < p.gsize ? p.group - part * p.gsize : p.gsize;
        const int *table = p.kv.tables + (size_t)seq * p.kv.max_pages;
        const bool in_d = sub * E < p.D;
        const u32 row_bytes = (u32)p.D * ES;
        auto key_of = [&](int u) { return (u < vis.ns ? u : vis.wb + (u - vis.ns)) * NB + grp * 8; };
        auto page_of = [&](int u) {
            const int key = key_of(u);
            return u < u1 && key < vis.len ? __ldg(table + (key >> p.kv.ps_log)) : -1;
        };
        // half batch i of the piece: K (even) or V (odd) of batch u0 + i / 2 into the next slot; `lives` collects
        // which of the lane's 8 keys are visible, 8 bits per batch from the oldest unconsumed one on
        const int halves = 2 * (u1 - u0);
        int issued = 0, page = page_of(u0);
        size_t off = 0;
        u64 lives = 0;
        auto issue = [&](int consumed) {
            const int u = u0 + (issued >> 1);
            u32 live = 0;
            if ((issued & 1) == 0) {
                const int key0 = key_of(u);
                const bool ok = page >= 0 && page < p.kv.num_pages;
                fault |= !ok && key0 < vis.len;
                if (ok) {
                    off = (((((size_t)page * p.Hkv + kvh) << p.kv.ps_log) + (key0 & ((1 << p.kv.ps_log) - 1)))) * row_bytes;
                    if (key0 >= vis.lo && key0 + 8 <= vis.len) {
                        live = 0xffu;
                    } else {
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const int key = key0 + r;
                            live |= (key < vis.len && (key >= vis.lo || key < p.sinks)) ? 1u << r : 0u;
                        }
                    }
                }
                lives |= (u64)live << (8 * ((issued - consumed) >> 1));
                page = page_of(u + 1);
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
                              ((issued & 1) ? p.kv.v : p.kv.k) + off, 8 * row_bytes, bar, policy);
            ++issued;
            ++done;
        };
        const u32 first = done;
        while (issued < halves && issued < SLOTS) issue(0);

        // q of the group's heads, scaled into the exponent's base 2
        f32x2 q[G][E / 2];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float x[E];
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = 0.f;
            if (g < gn && in_d) {
                const uint8_t *row = p.q + b * p.q_stride + ((size_t)(h0 + g) * p.D + sub * E) * (p.q_bf16 ? 2 : 4);
                if (p.q_bf16) {
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) {
                        const u32 w = reinterpret_cast<const u32 *>(row)[i];
                        x[2 * i] = __uint_as_float(w << 16);
                        x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < E; i += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(row + 4 * i);
                        x[i] = w.x, x[i + 1] = w.y, x[i + 2] = w.z, x[i + 3] = w.w;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < E / 2; ++i) q[g][i] = pack2(x[2 * i] * p.scale_log2, x[2 * i + 1] * p.scale_log2);
        }
        float m[G], l[G];
        f32x2 acc[G][E / 2];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) acc[g][i] = 0ull;
        }
        // the next half batch's slot, once its copy has landed
        auto landed = [&](int i) {
            const u32 n = first + i, slot = n % SLOTS;
            stuck |= !mbar_wait(bars + slot * 8, (n / SLOTS) & 1, AD_TIMEOUT_NS, nullptr);
            return ring + slot * AD_SLOT + (size_t)grp * 8 * row_bytes + sub * 16;
        };
        // row r of a slot as E floats; zero for a lane behind the head size or a hidden row
        auto chunk = [&](const uint8_t *row, int r, bool keep, f32x2 (&x)[E / 2]) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (keep) w = *reinterpret_cast<const uint4 *>(row + r * row_bytes);
            const u32 a[4] = {w.x, w.y, w.z, w.w};
            if (BF16) {
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                    x[i] = pack2(__uint_as_float(a[i] << 16), __uint_as_float(a[i] & 0xffff0000u));
            } else {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) x[i] = pack2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
            }
        };
        for (int i = 0; i < halves; i += 2) {
            const u32 now = (u32)lives & 0xffu;
            float s[G][8];
            const uint8_t *rows = landed(i);
            if (__any_sync(0xffffffffu, stuck)) {
                stuck = true;
                break;
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                f32x2 x[E / 2];
                chunk(rows, r, in_d, x);  // (a hidden row's score is dropped below)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    f32x2 d = mul2(x[0], q[g][0]);
#pragma unroll
                    for (int k = 1; k < E / 2; ++k) d = fma2(x[k], q[g][k], d);
                    float lo, hi;
                    unpack2(d, lo, hi);
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
#pragma unroll
                    for (int k = 0; k < E / 2; ++k) acc[g][k] = mul2(acc[g][k], c2);
                }
                sc[g] = mine ? exp2_fast(sc[g] - m[g]) : 0.f;
                l[g] += sc[g];
            }
            rows = landed(i + 1);
            if (__any_sync(0xffffffffu, stuck)) {
                stuck = true;
                break;
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                f32x2 x[E / 2];
                chunk(rows, r, in_d && (now >> r & 1u), x);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float w = __shfl_sync(0xffffffffu, sc[g], r, LK);
                    const f32x2 w2 = pack2(w, w);
#pragma unroll
                    for (int k = 0; k < E / 2; ++k) acc[g][k] = fma2(x[k], w2, acc[g][k]);
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
            break;
        }
        // the warp's key groups together, then out or into a partial
        const bool whole = u0 == 0 && u1 == vis.count;
        const int slot = 2 * warp + (seg_at <= from ? 0 : 1);
        if (!whole && lane == 0) {
            s_pb[slot] = b;
            s_pseg[slot] = seg;
            s_p0[slot] = seg_at;
            s_p1[slot] = seg_at + vis.count - 1;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float x[E];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) unpack2(acc[g][i], x[2 * i], x[2 * i + 1]);
            // lanes 8, 16, 24 on of a key repeat its first 8 lanes' scores
            float lw = sub < 8 ? l[g] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
#pragma unroll
            for (int i = 0; i < E; ++i) {
#pragma unroll
                for (int o = LK; o < 32; o <<= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
            }
            if (g >= gn) continue;
            if (whole) {
                const size_t row = (size_t)b * p.Hq + h0 + g;
                const float f = lw > 0.f ? 1.f / lw : 0.f;
                if (grp == 0 && in_d) {
#pragma unroll
                    for (int i = 0; i < E; ++i) put_out(p, row, sub * E + i, x[i] * f);
                }
                if (lane == 0) put_lse(p, row, m[g], lw);
            } else {
                float *d = partial(slot, g);
                if (grp == 0) {
#pragma unroll
                    for (int i = 0; i < E; ++i) d[sub * E + i] = x[i];
                }
                if (lane == 0) {
                    d[DP] = m[g];
                    d[DP + 1] = lw;
                }
            }
        }
    }
    if (fault) raise_device_error(DEVERR_INDEX);
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

// Joins the segments that span CTAs, one CTA per segment; entries without a
// visible key get out = 0, lse = -inf.
template <int DP>
__global__ void __launch_bounds__(AD_JOIN_THREADS) k_attn_join(const __grid_constant__ DecodeAttnParams p, int ctas,
                                                               int warps) {
    constexpr int ROW = DP + 2;
    __shared__ float s_w[AD_MAX_CTAS], s_red[2];
    pdl_wait();
    const int segs = p.Hkv * p.parts;
    const int b = blockIdx.x, seg = blockIdx.y;
    const int seq = p.seq_ids != nullptr ? __ldg(p.seq_ids + b) : b;
    if (seq < 0) return;
    if (seq >= p.kv.max_seqs) {
        if (threadIdx.x == 0 && seg == 0) raise_device_error(DEVERR_INDEX);
        return;
    }
    const int len = p.kv.lengths[seq];
    if (threadIdx.x == 0 && seg == 0 && (len < 0 || len > (long long)p.kv.max_pages << p.kv.ps_log))
        raise_device_error(DEVERR_INDEX);
    const int kvh = seg / p.parts, part = seg - kvh * p.parts;
    const int h0 = kvh * p.group + part * p.gsize;
    const int gn = p.group - part * p.gsize < p.gsize ? p.group - part * p.gsize : p.gsize;
    const long long cum = p.cum[b], width = (p.cum[b + 1] - cum) / segs;
    const long long gw = (long long)ctas * warps;
    const long long cta_piece = (p.cum[p.B] + gw - 1) / gw * warps;
    if (width == 0) {
        for (int i = threadIdx.x; i < gn * p.D; i += AD_JOIN_THREADS) put_out(p, (size_t)b * p.Hq + h0 + i / p.D, i % p.D, 0.f);
        if (threadIdx.x < gn) put_lse(p, (size_t)b * p.Hq + h0 + threadIdx.x, 0.f, 0.f);
        return;
    }
    const long long s0 = cum + seg * width + AD_OH, s1 = cum + (seg + 1) * width - 1;
    const int c0 = (int)(s0 / cta_piece), c1 = (int)(s1 / cta_piece);
    if (c0 == c1) return;  // finished by its CTA
    const int n = c1 - c0 + 1;
    // CTA c0 holds the segment's beginning in its second slot, the others what follows in their first
    auto part_of = [&](int i, int g) {
        return p.part + (((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * p.gsize + g) * ROW;
    };
    for (int g = 0; g < gn; ++g) {
        __syncthreads();
        if (threadIdx.x < 32) {
            float mm = -INFINITY, ll = 0.f;
            for (int i = threadIdx.x; i < n; i += 32) mm = fmaxf(mm, part_of(i, g)[DP]);
            mm = redux_max(mm);
            for (int i = threadIdx.x; i < n; i += 32) {
                const float *row = part_of(i, g);
                const float c = row[DP] == -INFINITY ? 0.f : exp2_fast(row[DP] - mm);
                s_w[i] = c;
                ll += c * row[DP + 1];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
            if (threadIdx.x == 0) {
                s_red[0] = mm;
                s_red[1] = ll;
            }
        }
        __syncthreads();
        const size_t row = (size_t)b * p.Hq + h0 + g;
        const float ll = s_red[1];
        if ((int)threadIdx.x < p.D) {
            float a = 0.f;
#pragma unroll 8
            for (int i = 0; i < n; ++i) a += s_w[i] * part_of(i, g)[threadIdx.x];
            put_out(p, row, threadIdx.x, ll > 0.f ? a / ll : 0.f);
        }
        if (threadIdx.x == 0) put_lse(p, row, s_red[0], ll);
    }
}

}  // namespace bl
