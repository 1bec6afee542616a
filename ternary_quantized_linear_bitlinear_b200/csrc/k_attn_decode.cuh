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
// Work.  Keys are taken in batches of NB consecutive keys (aligned), the
// share of one warp per step.  The batches of all (sequence, head group)
// segments form one line, cut into equal pieces, one per CTA: lengths that
// live on the device and differ wildly still load every SM alike.  A CTA
// walks the segments of its piece; its warps take a segment's batches in
// turn, each with its own running maximum and sum, and merge them in shared
// memory at the segment's end.  A segment inside one piece is finished
// there; one that spans CTAs leaves float32 partials (maximum, sum,
// unnormalised output) in the workspace, joined in order by k_attn_join, so
// the result depends on nothing but the inputs and the grid.
//
// Layout inside a warp: LK lanes share a key, each with a 16-byte chunk of
// its row, and the KW = 32 / LK key groups own 8 consecutive keys each, all
// in one page (pages are aligned blocks of at least 8 tokens), so a lane
// needs one page lookup per batch and keeps 8 rows of K and of V in flight.
// The dot products' partial sums are reduced across a key's lanes by a
// transposing butterfly: log2 steps that halve the number of keys a lane
// holds, 7 exchanges for 8 keys instead of 8 log2(LK).
#pragma once

#include "k_kv_pages.cuh"
#include "k_rope_append.cuh"

namespace bl {

constexpr int AD_MAX_B = 65535;
constexpr int AD_G = 8;  // query heads per segment at most
constexpr int AD_JOIN_THREADS = 128;

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
    long long *cum;     // workspace: [B + 1] batches before sequence b's segments
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

template <bool BF16, int DP, int G, int WARPS, int OCC>
__global__ void __launch_bounds__(WARPS * 32, OCC) k_attn_decode(const __grid_constant__ DecodeAttnParams p) {
    using S = DecodeShape<BF16, DP>;
    constexpr int E = S::E, LK = S::LK, KW = S::KW, NB = S::NB;
    constexpr int T = WARPS * 32;
    extern __shared__ float s_dyn[];
    float *s_acc = s_dyn;                          // [WARPS][G][DP]
    float *s_m = s_dyn + WARPS * G * DP;            // [WARPS][G]
    float *s_l = s_m + WARPS * G;                  // [WARPS][G]
    __shared__ int scratch[64];
    __shared__ long long s_total;
    __shared__ int s_b;
    __shared__ long long s_before;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane & (LK - 1), grp = lane / LK;
    const int segs = p.Hkv * p.parts;              // segments of a sequence
    pdl_wait();

    // batches before each sequence (CTA 0 leaves them for the join), and the
    // sequence in which this CTA's piece begins
    long long total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        // pass 0: the total; pass 1 (the piece is known): where it begins
        const long long share = pass == 0 ? 0 : (s_total + gridDim.x - 1) / gridDim.x;
        const long long piece = share > WARPS ? share : WARPS;
        const long long begin = blockIdx.x * piece;
        long long at = 0;
        for (int b0 = 0; b0 < p.B; b0 += T) {
            const int b = b0 + threadIdx.x;
            int seq, n = 0;
            if (b < p.B) n = visible_of<NB>(entry_len(p, b, &seq), p.window, p.sinks).count;
            int sum;
            // a sequence's batches times its segments may pass 2^31 over the batch: scan batches, then multiply
            const int pre = block_scan(n, &sum, scratch);
            const long long here = at + (long long)pre * segs;
            if (pass == 1 && b < p.B) {
                if (blockIdx.x == 0) p.cum[b] = here;
                if (n > 0 && here <= begin && begin < here + (long long)n * segs) {
                    s_b = b;
                    s_before = here;
                }
            }
            at += (long long)sum * segs;
        }
        total = at;
        if (threadIdx.x == 0) s_total = at;
        __syncthreads();
        if (pass == 1 && blockIdx.x == 0 && threadIdx.x == 0) p.cum[p.B] = at;
    }
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    const long long piece = share > WARPS ? share : WARPS;
    long long at = blockIdx.x * piece;
    const long long end = at + piece < total ? at + piece : total;
    if (at >= end) return;
    int b = s_b;
    long long before = s_before;
    const long long first_at = at;

    bool fault = false;
    while (at < end) {
        // the segment at `at`: sequence b, kv head, part; u0 .. u1 its batches of this piece
        int seq;
        const Visible vis = visible_of<NB>(entry_len(p, b, &seq), p.window, p.sinks);
        if (vis.count == 0 || at >= before + (long long)vis.count * segs) {
            before += (long long)vis.count * segs;
            ++b;
            continue;
        }
        const int seg = (int)((at - before) / vis.count);
        const long long seg_at = before + (long long)seg * vis.count;
        const int u0 = (int)(at - seg_at);
        const int u1 = end - seg_at < vis.count ? (int)(end - seg_at) : vis.count;
        const int kvh = seg / p.parts, part = seg - kvh * p.parts;
        const int h0 = kvh * p.group + part * p.gsize;
        const int gn = p.group - part * p.gsize < p.gsize ? p.group - part * p.gsize : p.gsize;

        // q of the group's heads, scaled into the exponent's base 2
        f32x2 q[G][E / 2];
        const bool in_d = sub * E < p.D;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float x[E];
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = 0.f;
            if (g < gn && in_d) {
                const uint8_t *row = p.q + b * p.q_stride + ((size_t)(h0 + g) * p.D + sub * E) * (p.q_bf16 ? 2 : 4);
                if (p.q_bf16) {
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        x[i] = __uint_as_float((u32) reinterpret_cast<const uint16_t *>(row)[i] << 16);
                } else {
#pragma unroll
                    for (int i = 0; i < E; ++i) x[i] = reinterpret_cast<const float *>(row)[i];
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
        const int *table = p.kv.tables + (size_t)seq * p.kv.max_pages;
        auto batch_of = [&](int u) { return u < vis.ns ? u : vis.wb + (u - vis.ns); };
        auto page_of = [&](int u) {
            const int key = batch_of(u) * NB + grp * 8;
            return key < vis.len ? __ldg(table + (key >> p.kv.ps_log)) : -1;
        };
        int page = u0 + warp < u1 ? page_of(u0 + warp) : -1;
        for (int u = u0 + warp; u < u1; u += WARPS) {
            const int key0 = batch_of(u) * NB + grp * 8;
            const bool ok = page >= 0 && page < p.kv.num_pages;
            fault |= !ok && key0 < vis.len;
            const size_t off =
                ok ? (((((size_t)page * p.Hkv + kvh) << p.kv.ps_log) + (key0 & ((1 << p.kv.ps_log) - 1))) * p.D +
                      (size_t)sub * E) * (BF16 ? 2 : 4)
                   : 0;
            const size_t step = (size_t)p.D * (BF16 ? 2 : 4);
            // which of the 8 keys are visible (rows behind the length are not read: they may hold anything)
            u32 live = 0;
            if (ok) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int key = key0 + r;
                    live |= (key < vis.len && (key >= vis.lo || key < p.sinks)) ? 1u << r : 0u;
                }
            }
            uint4 kr[8], vr[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                kr[r] = make_uint4(0, 0, 0, 0);
                if ((live >> r & 1u) && in_d) kr[r] = ldg_stream_v4(p.kv.k + off + r * step);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                vr[r] = make_uint4(0, 0, 0, 0);
                if ((live >> r & 1u) && in_d) vr[r] = ldg_stream_v4(p.kv.v + off + r * step);
            }
            if (u + WARPS < u1) page = page_of(u + WARPS);
            auto chunk = [&](const uint4 &w, f32x2 (&x)[E / 2]) {
                const u32 a[4] = {w.x, w.y, w.z, w.w};
                if (BF16) {
#pragma unroll
                    for (int i = 0; i < E / 2; ++i)
                        x[i] = pack2(__uint_as_float(a[i] << 16), __uint_as_float(a[i] & 0xffff0000u));
                } else {
#pragma unroll
                    for (int i = 0; i < E / 2; ++i)
                        x[i] = pack2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
                }
            };
            float s[G][8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                f32x2 x[E / 2];
                chunk(kr[r], x);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    f32x2 d = mul2(x[0], q[g][0]);
#pragma unroll
                    for (int i = 1; i < E / 2; ++i) d = fma2(x[i], q[g][i], d);
                    float lo, hi;
                    unpack2(d, lo, hi);
                    s[g][r] = lo + hi;
                }
            }
            // transposing butterfly: after it lane `sub` holds key (sub & 7)'s score
            float sc[G];
            const bool mine = live >> (sub & 7) & 1u;
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) {
                    const bool up = sub & o;
#pragma unroll
                    for (int i = 0; i < o; ++i) {
                        const float keep = up ? s[g][i + o] : s[g][i], give = up ? s[g][i] : s[g][i + o];
                        s[g][i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
                float x = s[g][0];
#pragma unroll
                for (int o = 8; o < LK; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                sc[g] = mine ? x : -INFINITY;
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float mx = sc[g];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (mx > m[g]) {  // the same for the whole warp
                    const float c = exp2_fast(m[g] - mx);
                    m[g] = mx;
                    l[g] *= c;
                    const f32x2 c2 = pack2(c, c);
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) acc[g][i] = mul2(acc[g][i], c2);
                }
                sc[g] = mine ? exp2_fast(sc[g] - m[g]) : 0.f;
                l[g] += sc[g];
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                f32x2 x[E / 2];
                chunk(vr[r], x);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float w = __shfl_sync(0xffffffffu, sc[g], r, LK);
                    const f32x2 w2 = pack2(w, w);
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) acc[g][i] = fma2(x[i], w2, acc[g][i]);
                }
            }
        }
        // the warp's key groups, then the CTA's warps
        __syncthreads();  // the previous segment's readers are done
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
            if (grp == 0) {
                float *d = s_acc + ((size_t)warp * G + g) * DP + sub * E;
#pragma unroll
                for (int i = 0; i < E; ++i) d[i] = x[i];
            }
            if (lane == 0) {
                s_m[warp * G + g] = m[g];
                s_l[warp * G + g] = lw;
            }
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == vis.count;
        float *part_out = p.part + ((size_t)blockIdx.x * 2 + (seg_at <= first_at ? 0 : 1)) * p.gsize * (DP + 2);
        for (int i = threadIdx.x; i < gn * DP; i += T) {
            const int g = i / DP, d = i - g * DP;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, s_m[w * G + g]);
            float a = 0.f, ll = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float c = s_m[w * G + g] == -INFINITY ? 0.f : exp2_fast(s_m[w * G + g] - mm);
                a += c * s_acc[((size_t)w * G + g) * DP + d];
                ll += c * s_l[w * G + g];
            }
            if (whole) {
                if (d < p.D) {
                    const float o = ll > 0.f ? a / ll : 0.f;
                    const size_t at_out = ((size_t)b * p.Hq + h0 + g) * p.D + d;
                    if (p.q_bf16) reinterpret_cast<uint16_t *>(p.out)[at_out] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
                    else reinterpret_cast<float *>(p.out)[at_out] = o;
                }
                if (d == 0 && p.lse != nullptr)
                    p.lse[(size_t)b * p.Hq + h0 + g] = ll > 0.f ? (mm + log2f(ll)) * 0.693147180559945f : -INFINITY;
            } else {
                float *row = part_out + g * (DP + 2);
                row[d] = a;
                if (d == 0) {
                    row[DP] = mm;
                    row[DP + 1] = ll;
                }
            }
        }
        at = seg_at + u1;
    }
    if (fault) raise_device_error(DEVERR_INDEX);
}

// Joins the segments that span CTAs, one CTA per segment; entries without a
// visible key get out = 0, lse = -inf.
template <int DP>
__global__ void __launch_bounds__(AD_JOIN_THREADS) k_attn_join(const __grid_constant__ DecodeAttnParams p, int ctas,
                                                               int warps) {
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
    const long long n = (p.cum[b + 1] - p.cum[b]) / segs;
    const long long total = p.cum[p.B];
    const long long share = (total + ctas - 1) / ctas, piece = share > warps ? share : warps;
    const long long s0 = p.cum[b] + seg * n, s1 = s0 + n;
    const int c0 = (int)(s0 / piece), c1 = n > 0 ? (int)((s1 - 1) / piece) : c0;
    if (n > 0 && c0 == c1) return;  // finished by its CTA
    for (int i = threadIdx.x; i < gn * p.D; i += AD_JOIN_THREADS) {
        const int g = i / p.D, d = i - g * p.D;
        float mm = -INFINITY, a = 0.f, ll = 0.f;
        if (n > 0) {
            for (int c = c0; c <= c1; ++c) {
                const float *row = p.part + (((size_t)c * 2 + (s0 <= c * piece ? 0 : 1)) * p.gsize + g) * (DP + 2);
                const float m2 = row[DP], l2 = row[DP + 1], a2 = row[d];
                const float top = fmaxf(mm, m2);
                if (top == -INFINITY) continue;
                const float x = mm == -INFINITY ? 0.f : exp2_fast(mm - top), y = m2 == -INFINITY ? 0.f : exp2_fast(m2 - top);
                a = a * x + a2 * y;
                ll = ll * x + l2 * y;
                mm = top;
            }
        }
        const float o = ll > 0.f ? a / ll : 0.f;
        const size_t at_out = ((size_t)b * p.Hq + h0 + g) * p.D + d;
        if (p.q_bf16) reinterpret_cast<uint16_t *>(p.out)[at_out] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
        else reinterpret_cast<float *>(p.out)[at_out] = o;
        if (d == 0 && p.lse != nullptr)
            p.lse[(size_t)b * p.Hq + h0 + g] = ll > 0.f ? (mm + log2f(ll)) * 0.693147180559945f : -INFINITY;
    }
}

}  // namespace bl
