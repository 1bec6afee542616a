// Gradients of ragged attention on mma.sync: 64 x 64 tiles, four warps, each
// 16 rows; operands in shared memory.
#pragma once

#include "k_attn_ragged.cuh"

namespace bl {

constexpr int AM_T = 128;
constexpr int AM_B = 64;

template <int DP>
constexpr int am_smem(int tiles) {
    return tiles * AM_B * DP * 2;
}

// S (16 x 64) of a warp: rows of tile A from row0, all 64 rows of tile B.
template <int DP>
__device__ __forceinline__ void warp_gemm_nt(float (&s)[8][4], u32 a_base, int row0, u32 b_base) {
#pragma unroll
    for (int n = 0; n < 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
        u32 a[4];
        a_frag<DP>(a, a_base, row0, kk);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            u32 b[4];
            b_frag<DP>(b, b_base, n * 16, kk);
            mma_bf16(s[2 * n], a, b[0], b[1]);
            mma_bf16(s[2 * n + 1], a, b[2], b[3]);
        }
    }
}

// acc (16 x DP) += X (16 x 64, in registers, rounded to bf16) * tile (64 x DP)
template <int DP>
__device__ __forceinline__ void warp_gemm_nn(float (&acc)[DP / 8][4], const float (&x)[8][4], u32 b_base) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        const u32 a[4] = {pack_bf16(x[2 * kk][0], x[2 * kk][1]), pack_bf16(x[2 * kk][2], x[2 * kk][3]),
                          pack_bf16(x[2 * kk + 1][0], x[2 * kk + 1][1]), pack_bf16(x[2 * kk + 1][2], x[2 * kk + 1][3])};
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
            u32 b[4];
            bt_frag<DP>(b, b_base, kk * 16, n * 2);
            mma_bf16(acc[2 * n], a, b[0], b[1]);
            mma_bf16(acc[2 * n + 1], a, b[2], b[3]);
        }
    }
}

// acc rows to out[(row0 + r) * H * D + d], rows < rows
template <int DP>
__device__ __forceinline__ void store_rows(const float (&acc)[DP / 8][4], uint16_t *out, long long stride, int rows,
                                           int row0, int D, float f0, float f1) {
    const int lane = threadIdx.x & 31, r = row0 + (lane >> 2), c = (lane & 3) * 2;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
        const int d = n * 8 + c;
        if (d >= D) continue;
        if (r < rows) *reinterpret_cast<u32 *>(out + r * stride + d) = pack_bf16(acc[n][0] * f0, acc[n][1] * f0);
        if (r + 8 < rows) *reinterpret_cast<u32 *>(out + (r + 8) * stride + d) = pack_bf16(acc[n][2] * f1, acc[n][3] * f1);
    }
}

// delta[h, t] = sum_d do[t, h, d] * o[t, h, d]; one warp per row.
__global__ void __launch_bounds__(256) k_attn_delta(const __grid_constant__ RaggedParams p, float *delta) {
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= (long long)p.Tq * p.Hq) return;
    const int t = (int)(i / p.Hq), h = (int)(i - (long long)t * p.Hq);
    float sum = 0.f;
    if (lane * 4 < p.D) {
        const uint2 a = *reinterpret_cast<const uint2 *>(p.dout + t * p.do_stride + (size_t)h * p.D + lane * 4);
        const uint2 c = *reinterpret_cast<const uint2 *>(p.o + ((size_t)t * p.Hq + h) * p.D + lane * 4);
        const u32 x[2] = {a.x, a.y}, y[2] = {c.x, c.y};
#pragma unroll
        for (int j = 0; j < 2; ++j)
            sum += __uint_as_float(x[j] << 16) * __uint_as_float(y[j] << 16) +
                   __uint_as_float(x[j] & 0xffff0000u) * __uint_as_float(y[j] & 0xffff0000u);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) delta[(size_t)h * p.Tq + t] = sum;
}

template <int DP>
__global__ void __launch_bounds__(AM_T) k_attn_dq(const __grid_constant__ RaggedParams p) {
    extern __shared__ __align__(128) uint8_t sm[];
    const u32 sq = smem_u32(sm), sdo = sq + am_smem<DP>(1), sk = sdo + am_smem<DP>(1), sv = sk + am_smem<DP>(1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y, b = blockIdx.z;
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) check_entry(p, b);
    Entry e;
    if (!entry_of(p, b, e)) return;
    const int i0 = (gridDim.x - 1 - blockIdx.x) * AM_B;
    if (i0 >= e.nq) return;
    const int rows = e.nq - i0 < AM_B ? e.nq - i0 : AM_B;
    const int kvh = h / p.group;
    load_tile<DP, AM_B, AM_T>(sq, p.q + (e.q0 + i0) * p.q_stride + (size_t)h * p.D, p.q_stride, rows, p.D);
    load_tile<DP, AM_B, AM_T>(sdo, p.dout + (e.q0 + i0) * p.do_stride + (size_t)h * p.D, p.do_stride, rows, p.D);
    const KeyTiles kt = key_tiles<AM_B>(p, i0 + e.off, i0 + rows - 1 + e.off, e.nk);
    const int row = warp * 16 + (lane >> 2);
    float lse[2], delta[2];
    int pos[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const bool ok = row + 8 * r < rows;
        pos[r] = ok ? i0 + row + 8 * r + e.off : -1;
        const size_t at = (size_t)h * p.Tq + e.q0 + i0 + row + 8 * r;
        lse[r] = ok ? p.lse[at] * 1.44269504088896f : 0.f;
        delta[r] = ok ? p.delta[at] : 0.f;
    }
    float dq[DP / 8][4] = {};
    for (int t = 0; t < kt.count; ++t) {
        const int j0 = (t < kt.ns ? t : kt.wt + t - kt.ns) * AM_B;
        const int nk = e.nk - j0 < AM_B ? e.nk - j0 : AM_B;
        load_tile<DP, AM_B, AM_T>(sk, p.k + (e.k0 + j0) * p.k_stride + (size_t)kvh * p.D, p.k_stride, nk, p.D);
        load_tile<DP, AM_B, AM_T>(sv, p.v + (e.k0 + j0) * p.v_stride + (size_t)kvh * p.D, p.v_stride, nk, p.D);
        cp_commit();
        cp_wait<0>();
        __syncthreads();
        float s[8][4], dp[8][4];
        warp_gemm_nt<DP>(s, sq, warp * 16, sk);
        warp_gemm_nt<DP>(dp, sdo, warp * 16, sv);
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = j0 + n * 8 + (lane & 3) * 2 + (x & 1);
                const float pr = key < e.nk && sees(p, pos[x >> 1], key) ? exp2_fast(s[n][x] * p.scale_log2 - lse[x >> 1]) : 0.f;
                s[n][x] = pr * (dp[n][x] - delta[x >> 1]);
            }
        warp_gemm_nn<DP>(dq, s, sk);
        __syncthreads();
    }
    cp_commit();
    cp_wait<0>();
    store_rows<DP>(dq, p.dq + ((size_t)(e.q0 + i0) * p.Hq + h) * p.D, (long long)p.Hq * p.D, rows, warp * 16, p.D, p.scale, p.scale);
}

template <int DP>
__global__ void __launch_bounds__(AM_T) k_attn_dkdv(const __grid_constant__ RaggedParams p) {
    extern __shared__ __align__(128) uint8_t sm[];
    const u32 sk = smem_u32(sm), sv = sk + am_smem<DP>(1), sq = sv + am_smem<DP>(1), sdo = sq + am_smem<DP>(1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.y, b = blockIdx.z;
    Entry e;
    if (!entry_of(p, b, e)) return;
    const int j0 = blockIdx.x * AM_B;
    if (j0 >= e.nk) return;
    const int nk = e.nk - j0 < AM_B ? e.nk - j0 : AM_B;
    load_tile<DP, AM_B, AM_T>(sk, p.k + (e.k0 + j0) * p.k_stride + (size_t)kvh * p.D, p.k_stride, nk, p.D);
    load_tile<DP, AM_B, AM_T>(sv, p.v + (e.k0 + j0) * p.v_stride + (size_t)kvh * p.D, p.v_stride, nk, p.D);
    float dk[DP / 8][4] = {}, dv[DP / 8][4] = {};
    const int key0 = j0 + warp * 16 + (lane >> 2);
    // queries that can see keys j0 .. j0 + nk - 1: positions from j0, to the end for sinks, else within the window
    int i_lo = j0 - e.off, i_hi = e.nq - 1;
    if (i_lo < 0) i_lo = 0;
    if (p.window > 0 && j0 >= p.sinks) {
        const long long last = (long long)j0 + nk - 1 + p.window - 1 - e.off;
        if (last < i_hi) i_hi = (int)last;
    }
    for (int hg = 0; hg < p.group; ++hg) {
        const int h = kvh * p.group + hg;
        for (int i0 = i_lo / AM_B * AM_B; i0 <= i_hi; i0 += AM_B) {
            const int rows = e.nq - i0 < AM_B ? e.nq - i0 : AM_B;
            load_tile<DP, AM_B, AM_T>(sq, p.q + (e.q0 + i0) * p.q_stride + (size_t)h * p.D, p.q_stride, rows, p.D);
            load_tile<DP, AM_B, AM_T>(sdo, p.dout + (e.q0 + i0) * p.do_stride + (size_t)h * p.D, p.do_stride, rows, p.D);
            cp_commit();
            cp_wait<0>();
            __syncthreads();
            float s[8][4], dp[8][4];
            warp_gemm_nt<DP>(s, sk, warp * 16, sq);
            warp_gemm_nt<DP>(dp, sv, warp * 16, sdo);
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = n * 8 + (lane & 3) * 2 + x;
                    const bool ok = i < rows;
                    const size_t at = (size_t)h * p.Tq + e.q0 + i0 + i;
                    const float lse = ok ? p.lse[at] * 1.44269504088896f : 0.f, delta = ok ? p.delta[at] : 0.f;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int key = key0 + 8 * r;
                        const float pr = ok && key < e.nk && sees(p, i0 + i + e.off, key)
                                             ? exp2_fast(s[n][2 * r + x] * p.scale_log2 - lse) : 0.f;
                        s[n][2 * r + x] = pr;
                        dp[n][2 * r + x] = pr * (dp[n][2 * r + x] - delta);
                    }
                }
            warp_gemm_nn<DP>(dv, s, sdo);
            warp_gemm_nn<DP>(dk, dp, sq);
            __syncthreads();
        }
    }
    cp_commit();
    cp_wait<0>();
    const long long stride = (long long)p.Hkv * p.D;
    const size_t at = ((size_t)(e.k0 + j0) * p.Hkv + kvh) * p.D;
    store_rows<DP>(dk, p.dk + at, stride, nk, warp * 16, p.D, p.scale, p.scale);
    store_rows<DP>(dv, p.dv + at, stride, nk, warp * 16, p.D, 1.f, 1.f);
}

}  // namespace bl
