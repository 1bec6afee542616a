// Gradients of ragged causal attention with a sliding window and sinks, on
// tcgen05, without atomics: one kernel forms dQ row tile by row tile, another
// dK and dV key tile by key tile; both rebuild P = exp2(scale log2(e) S -
// lse) from the scores.
//
//   dP = dO V^T,  dS = P o (dP - delta),  dQ = scale dS K
//   dV = P^T dO,  dK = scale dS^T Q
//
// k_attn_dq_tc.  A CTA owns 128 queries of one head (TMEM lanes).  S and dP of
// a key tile come from two products; dS goes back to TMEM as bf16 over S and
// is the A operand of dQ += dS K.  The kernel starts from delta0 = rowsum(dO o
// O) with the O that the forward rounded to bf16, and on the way sums delta =
// rowsum(P o dP), the same quantity without that rounding, which dK uses.
// delta0's error is common to a row, so dQ would be off by it times sum_j P_j
// k_j, which keys with a mean do not average out (K and V of mean 4: a third of
// dQ).  So R += P K is formed as well, P as bf16 beside dS over S, and
//   dQ = scale (sum_j dS_j k_j + (delta0 - delta) R)
// at the end: R's own rounding only weighs on the small difference.
// TMEM is full: at D <= 64 S is double buffered (S(j + 1) is formed while the
// softmax threads work on S(j)); at D > 64 two buffers serve S and dP in turn,
// S(j + 1) taking the place of dP(j), and R(j) runs while the threads form
// dS(j).
//
// k_attn_dkdv_tc.  A CTA owns 128 keys of one kv head (TMEM lanes) and walks
// the query tiles that see them, for every query head that shares them, so dK
// and dV of shared heads are sums in TMEM.  The scores are formed transposed
// (S^T = K Q^T, dP^T = V dO^T): P^T and dS^T then lie with the keys in the
// lanes, as the A operands of dV += P^T dO and dK += dS^T Q need them, and no
// tile is ever transposed through shared memory.  The tensor core works one
// step behind the threads: dV(j), S(j + 1) while they form dS(j), dK(j),
// dP(j + 1) while they form P(j + 1).
// A tile with sinks is seen by every later query of its sequence.  The query
// tiles beyond the window's reach are cut into pieces of their own; the float32
// sums of the sinks' rows go to the workspace and are added in order by
// k_attn_sink_sum.
//
// Bound: eight products of 512 tensor cycles per pair of 128-tiles at D = 128
// against 2 x 1024 cycles of exponentials.
//
// Threads: warp 0 TMA producer, 1 TMEM allocator and MMA issuer, 2 rows'
// statistics and the clearing of rows that belong to nobody, 4 - 11 the
// softmax (two threads per lane, half of the columns each).  Waits are
// bounded as in the forward kernel.
#pragma once

#include "k_attn_fwd_tc.cuh"

namespace bl {

constexpr int AB_THREADS = 384;
constexpr unsigned long long AB_TIMEOUT_NS = 2000000000ull;

// ---------------------------------------------------------------------------
// dQ

template <int DP>
struct DqShape {
    static constexpr int KS = 3, VS = DP == 64 ? 3 : 2;  // stages of K (read for S, and again for dQ and R up to two steps later) and V
    static constexpr int TILE = DP / 64 * TC_BLOCK;
    static constexpr int OFF_DO = TILE, OFF_K = 2 * TILE, OFF_V = OFF_K + KS * TILE, OFF_D = OFF_V + VS * TILE;
    static constexpr int OFF_BAR = OFF_D + 2 * 128 * 4;
    static constexpr int BARS = 1 + 2 * KS + 2 * VS + 11;
    static constexpr bool AHEAD = DP == 64;  // S(j + 1) has a buffer of its own
    static constexpr int SMEM = OFF_BAR + BARS * 8 + 16 + 1024;
};
static_assert(DqShape<128>::SMEM <= 227 * 1024, "dQ shared memory");

template <int DP>
__global__ void __launch_bounds__(AB_THREADS, 1)
    k_attn_dq_tc(const __grid_constant__ RaggedMaps maps, const __grid_constant__ RaggedParams p, float *delta_out) {
    using F = DqShape<DP>;
    constexpr int KS = F::KS, VS = F::VS;
    extern __shared__ uint8_t af_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(af_raw) + 1023) & ~(uintptr_t)1023);
    const u32 sbase = smem_u32(sm), bar0 = sbase + F::OFF_BAR;
    const u32 QF = bar0, KF = bar0 + 8, KE = KF + 8 * KS, VF = KE + 8 * KS, VE = VF + 8 * VS, SF = VE + 8 * VS,
              DPF = SF + 16, PR = DPF + 8, DSR = PR + 16, OUT = DSR + 16, CUT = OUT + 8, FIX = CUT + 8, DRAIN = FIX + 8;
    float *s_delta = reinterpret_cast<float *>(sm + F::OFF_D);  // [2][128]
    u32 *s_tmem = reinterpret_cast<u32 *>(sm + F::OFF_BAR + F::BARS * 8);
    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + F::OFF_BAR + F::BARS * 8 + 4);
    constexpr unsigned long long TO = AB_TIMEOUT_NS;

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc_prefetch(&maps.q);
        tc_prefetch(&maps.k);
        tc_prefetch(&maps.v);
        tc_prefetch(&maps.dout);
    }
    const int h = blockIdx.y, b = blockIdx.z;
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) check_entry(p, b);
    Entry e;
    if (!entry_of(p, b, e)) return;
    const int i0 = (gridDim.x - 1 - blockIdx.x) * 128;
    if (i0 >= e.nq) return;
    const int kvh = h / p.group;
    const int rows = e.nq - i0 < 128 ? e.nq - i0 : 128;
    const int first_pos = i0 + e.off, last_pos = first_pos + rows - 1;
    const KeyTiles all = key_tiles<AF_KEYS>(p, first_pos, last_pos, e.nk);
    const int n = all.count;
    auto tile_of = [&](int u) { return u < all.ns ? u : all.wt + (u - all.ns); };
    // the entry's last tile when it is partial: K and V on a barrier of their own, then cleared behind the last key
    const int cut = e.nk % AF_KEYS;
    const bool cuts = n > 0 && cut != 0 && tile_of(n - 1) == e.nk / AF_KEYS;
    auto k_full = [&](int u) { return cuts && u == n - 1 ? FIX : KF + 8 * (u % KS); };
    auto v_full = [&](int u) { return cuts && u == n - 1 ? FIX : VF + 8 * (u % VS); };
    auto k_phase = [&](int u) { return cuts && u == n - 1 ? 0u : (u32)((u / KS) & 1); };
    auto v_phase = [&](int u) { return cuts && u == n - 1 ? 0u : (u32)((u / VS) & 1); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < F::BARS; ++i) mbar_init(bar0 + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(PR + 8 * i, 8);
            mbar_init(DSR + 8 * i, 8);
        }
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (n > 0) {  // on their way while TMEM is allocated
            mbar_arrive_expect_tx(QF, 2 * F::TILE);
            tc_load_rows<DP>(&maps.q, sbase, h, e.q0 + i0, QF);
            tc_load_rows<DP>(&maps.dout, sbase + F::OFF_DO, h, e.q0 + i0, QF);
        }
    }
    if (warp == 1) tc_alloc(smem_u32(s_tmem), 512);
    tc_before();
    __syncthreads();
    tc_after();
    const u32 tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
    auto s_col = [&](int j) { return tmem + 128u * (j & 1); };
    auto dp_col = [&](int j) { return F::AHEAD ? tmem + 256u : tmem + 128u * (~j & 1); };
    const u32 dq_col = tmem + (F::AHEAD ? 384 : 256), r_col = dq_col + DP;

    if (warp == 0) {
        if (lane == 0 && n > 0) {
            bool ok = true;
            int u = 0, ku = 0;  // tiles of V and of K requested
            for (; u < n; ++u) {
                const int ks = u % KS, vs = u % VS, row = e.k0 + tile_of(u) * AF_KEYS;
                const bool last = cuts && u == n - 1;
                if (u >= KS && !tc_wait(KE + 8 * ks, (u32)((u / KS) & 1) ^ 1, TO, s_abort)) break;
                const u32 kbar = last ? CUT : KF + 8 * ks, vbar = last ? CUT : VF + 8 * vs;
                mbar_arrive_expect_tx(kbar, last ? 2 * F::TILE : F::TILE);
                tc_load_rows<DP>(&maps.k, sbase + F::OFF_K + ks * F::TILE, kvh, row, kbar);
                ku = u + 1;
                if (u >= VS && !tc_wait(VE + 8 * vs, (u32)((u / VS) & 1) ^ 1, TO, s_abort)) break;
                if (!last) mbar_arrive_expect_tx(vbar, F::TILE);
                tc_load_rows<DP>(&maps.v, sbase + F::OFF_V + vs * F::TILE, kvh, row, vbar);
            }
            ok = u == n;
            if (!ok) {
                raise_device_error(DEVERR_TIMEOUT_PRODUCER);
                *s_abort = 1;
            }
            // what was requested lands before the CTA exits
            tc_wait(QF, 0, TO, nullptr);
            // (a last tile of which only K was requested does not complete its barrier: that wait runs its time out,
            // and K has landed by then)
            for (int j = ku - KS > 0 ? ku - KS : 0; j < ku; ++j) {
                if (cuts && j == n - 1) tc_wait(CUT, 0, TO, nullptr);
                else tc_wait(KF + 8 * (j % KS), (u32)((j / KS) & 1), TO, nullptr);
            }
            for (int j = u - VS > 0 ? u - VS : 0; j < u; ++j)
                if (!(cuts && j == n - 1)) tc_wait(VF + 8 * (j % VS), (u32)((j / VS) & 1), TO, nullptr);
        }
    } else if (warp == 1) {
        if (n > 0) {
            constexpr u32 ID_S = tc_idesc(AF_KEYS, false, false), ID_Q = tc_idesc(DP, false, true);
            const bool leader = tc_elect();
            bool ok = TC_WAIT_ALL(QF, 0, TO, s_abort);
            const u64 q_desc = tc_desc_k(sbase), do_desc = tc_desc_k(sbase + F::OFF_DO), k_desc = tc_desc_k(sbase + F::OFF_K),
                      v_desc = tc_desc_k(sbase + F::OFF_V), kt_desc = tc_desc_mn(sbase + F::OFF_K);
            auto k_ready = [&](int u) { ok = ok && TC_WAIT_ALL(k_full(u), k_phase(u), TO, s_abort); };
            auto v_ready = [&](int u) { ok = ok && TC_WAIT_ALL(v_full(u), v_phase(u), TO, s_abort); };
            auto form_s = [&](int u, int ks) {
                tc_after();
                if (leader) {
                    tc_gemm_nt<DP>(s_col(u), q_desc, k_desc + (u64)(ks * F::TILE >> 4), ID_S);
                    tc_commit(SF + 8 * (u & 1));
                }
                __syncwarp();
            };
            auto form_dp = [&](int u) {
                tc_after();
                if (leader) {
                    tc_gemm_nt<DP>(dp_col(u), do_desc, v_desc + (u64)(u % VS * F::TILE >> 4), ID_S);
                    tc_commit(DPF);
                    tc_commit(VE + 8 * (u % VS));
                }
                __syncwarp();
            };
            k_ready(0);
            if (ok) form_s(0, 0);
            v_ready(0);
            if (ok) form_dp(0);
            if (F::AHEAD && n > 1) k_ready(1);
            if (F::AHEAD && ok && n > 1) form_s(1, 1);
            int ks = 0;  // u % KS
            for (int u = 0; u < n && ok; ++u) {
                const u64 k = kt_desc + (u64)(ks * F::TILE >> 4);
                const int ks1 = ks == KS - 1 ? 0 : ks + 1, ks2 = ks == 0 ? 2 : ks - 1;  // (u + 1) % KS, (u + 2) % KS
                // columns 0 - 63 of dS are at the buffer's start, 64 - 127 at its column 64; the first half of each is
                // ready first (part 0: steps 0, 1, 4, 5)
                auto add = [&](int part) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = (i & 1) + (i >> 1) * 4 + 2 * part;
                        tc_mma_ts(dq_col, s_col(u) + (kk / 4) * 64 + (kk % 4) * 8, k + (u64)(kk * 2048 >> 4), ID_Q,
                                  u != 0 || part != 0 || i != 0);
                    }
                };
                // (the next V, and at D > 64 the next K, have landed long before the weights of this tile are ready; the
                // K after the next is only asked for when the last step's dQ is done)
                if (u + 1 < n) v_ready(u + 1);
                if (!F::AHEAD && u + 1 < n) k_ready(u + 1);
                ok = ok && TC_WAIT_ALL(PR + 8 * (u & 1), (u32)((u >> 1) & 1), TO, s_abort);
                if (!ok) break;
                tc_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc_mma_ts(r_col, s_col(u) + (kk / 4) * 64 + 32 + (kk % 4) * 8, k + (u64)(kk * 2048 >> 4), ID_Q,
                                  u != 0 || kk != 0);
                }
                __syncwarp();
                ok = TC_WAIT_ALL(DSR, (u32)(u & 1), TO, s_abort);
                if (!ok) break;
                tc_after();
                if (leader) add(0);
                __syncwarp();
                ok = TC_WAIT_ALL(DSR + 8, (u32)(u & 1), TO, s_abort);
                if (!ok) break;
                tc_after();
                // first what the threads wait for next: dP, or where it takes dP's place S (every thread has read dP)
                if (u + 1 < n) {
                    if (F::AHEAD) form_dp(u + 1);
                    else form_s(u + 1, ks1);
                }
                if (leader) {
                    add(1);
                    tc_commit(KE + 8 * ks);
                }
                __syncwarp();
                // (dP takes the place of P and dS, which the products before it have read)
                if (!F::AHEAD && u + 1 < n) form_dp(u + 1);
                if (F::AHEAD && u + 2 < n) {
                    k_ready(u + 2);
                    if (ok) form_s(u + 2, ks2);
                }
                ks = ks == KS - 1 ? 0 : ks + 1;
            }
            if (!ok && lane == 0) {
                raise_device_error(DEVERR_TIMEOUT_MMA);
                *s_abort = 1;
            }
            if (leader) {
                if (ok) tc_commit(OUT);
                tc_commit(DRAIN);
            }
            __syncwarp();
            tc_wait(DRAIN, 0, TO, nullptr);
        }
    } else if (warp == 2) {
        if (cuts) {
            if (__all_sync(0xffffffffu, tc_wait(CUT, 0, TO, s_abort))) {
                tc_zero_rows<DP>(sm + F::OFF_K + (n - 1) % KS * F::TILE, cut);
                tc_zero_rows<DP>(sm + F::OFF_V + (n - 1) % VS * F::TILE, cut);
                if (lane == 0) mbar_arrive(FIX);
            } else if (lane == 0) {
                raise_device_error(DEVERR_TIMEOUT_EXPAND);
                *s_abort = 1;
            }
        }
    } else if (warp >= 4) {
        const int c = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;  // columns 64 c .. 64 c + 63 of row r
        const int row = i0 + r, pos = r < rows ? row + e.off : -1;
        const u32 lane_at = (u32)((warp & 3) * 32) << 16;
        const float sl = p.scale_log2;
        const size_t stat = (size_t)h * p.Tq + e.q0 + row;
        // delta: each warp takes 16 rows, 16 lanes a row (one row per thread instead, its loads a row apart, took 12 000
        // of the kernel's 58 000 cycles)
        {
            const int w8 = warp - 4, sub = lane & 15;
            uint4 x[8], y[8];
            const bool in_d = sub * 8 < p.D;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // (a row or column that is not there reads the tile's first element instead: no branch between loads)
                const int rr = w8 * 16 + 2 * k + (lane >> 4);
                const size_t t = (size_t)(e.q0 + i0 + (rr < rows ? rr : 0));
                const int d = in_d ? sub * 8 : 0;
                x[k] = *reinterpret_cast<const uint4 *>(p.dout + t * p.do_stride + (size_t)h * p.D + d);
                y[k] = *reinterpret_cast<const uint4 *>(p.o + (t * p.Hq + h) * p.D + d);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const u32 a[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, c4[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
                float part = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part += __uint_as_float(a[i] << 16) * __uint_as_float(c4[i] << 16) +
                            __uint_as_float(a[i] & 0xffff0000u) * __uint_as_float(c4[i] & 0xffff0000u);
                if (!in_d) part = 0.f;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
                if (sub == 0) s_delta[w8 * 16 + 2 * k + (lane >> 4)] = part;
            }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float delta0 = s_delta[r];
        // (a row that sees nothing has lse = -inf and only hidden keys)
        const float lse = r < rows ? p.lse[stat] * 1.44269504088896f : 0.f;
        const f32x2 sl2 = pack2(sl, sl), nlse2 = pack2(-lse, -lse);
        f32x2 sum2 = 0ull;
        bool ok = true;
        for (int u = 0; u < n; ++u) {
            ok = __all_sync(0xffffffffu, tc_wait(SF + 8 * (u & 1), (u32)((u >> 1) & 1), TO, s_abort));
            if (!ok) break;
            tc_after();
            u32 w[64];
            tc_ld32(w, s_col(u) + lane_at + 64 * c);
            tc_ld32(w + 32, s_col(u) + lane_at + 64 * c + 32);
            tc_wait_ld();
            const int j0 = tile_of(u) * AF_KEYS;
            const bool whole = j0 + AF_KEYS - 1 <= first_pos && j0 + AF_KEYS <= e.nk && rows == 128 &&
                               (p.window == 0 || last_pos - j0 < p.window || j0 + AF_KEYS <= p.sinks);
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(w[j]), __uint_as_float(w[j + 1])), sl2, nlse2), x, y);
                w[j] = __float_as_uint(exp2_fast(x));
                w[j + 1] = __float_as_uint(exp2_fast(y));
            }
            if (!whole) {
                const int at = j0 + 64 * c;
                const int lo = p.window > 0 && pos >= p.window ? pos - p.window + 1 - at : 0;
                const int hi = (pos < e.nk - 1 ? pos : e.nk - 1) - at;
                const int sk = p.sinks - at;
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    if (j > hi || (j < lo && j >= sk)) w[j] = 0u;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                u32 pk[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    pk[j] = pack_bf16(__uint_as_float(w[32 * q + 2 * j]), __uint_as_float(w[32 * q + 2 * j + 1]));
                tc_st16(s_col(u) + lane_at + 64 * c + 32 + 16 * q, pk);
            }
            tc_hand_over(PR + 8 * (u & 1));
            ok = __all_sync(0xffffffffu, tc_wait(DPF, (u32)(u & 1), TO, s_abort));
            if (!ok) break;
            tc_after();
            const f32x2 nd2 = pack2(-delta0, -delta0);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                u32 g[32], pk[16];
                tc_ld32(g, dp_col(u) + lane_at + 64 * c + 32 * q);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const f32x2 pp = pack2(__uint_as_float(w[32 * q + 2 * j]), __uint_as_float(w[32 * q + 2 * j + 1]));
                    const f32x2 dd = pack2(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1]));
                    sum2 = fma2(pp, dd, sum2);
                    float x, y;
                    unpack2(mul2(pp, add2(dd, nd2)), x, y);
                    pk[j] = pack_bf16(x, y);
                }
                tc_st16(s_col(u) + lane_at + 64 * c + 16 * q, pk);
                tc_hand_over(DSR + 8 * q);
            }
        }
        // delta, over both halves of the columns (the barriers are met whatever the waits said)
        asm volatile("bar.sync 1, 256;" ::: "memory");
        float sum, sum_hi;
        unpack2(sum2, sum, sum_hi);
        s_delta[c * 128 + r] = sum + sum_hi;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float delta = s_delta[r] + s_delta[128 + r];
        if (ok && n > 0) ok = __all_sync(0xffffffffu, tc_wait(OUT, 0, TO, s_abort));
        if (!ok) {
            if (lane == 0) {
                raise_device_error(DEVERR_TIMEOUT_EPILOGUE);
                *s_abort = 1;
            }
        } else {
            tc_after();
            if (c == 0 && r < rows) delta_out[stat] = delta;
            // (the Q tile is not read any more)
            const int first = 32 * (warp & 3);
            tc_store_rows<DP / 2>(dq_col + lane_at + DP / 2 * c, n == 0, p.scale, sm + (warp - 4) * 32 * DP,
                                  p.dq + ((size_t)(e.q0 + i0 + first) * p.Hq + h) * p.D + DP / 2 * c,
                                  (long long)p.Hq * p.D, rows - first, p.D - DP / 2 * c, DP, delta0 - delta);
        }
    }
    tc_before();
    __syncthreads();
    if (warp == 1) {
        tc_after();
        tc_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// dK, dV

template <int DP>
struct DkvShape {
    static constexpr int ST = DP == 64 ? 4 : 2;
    static constexpr int TILE = DP / 64 * TC_BLOCK;
    static constexpr int OFF_V = TILE, OFF_Q = 2 * TILE, OFF_DO = OFF_Q + ST * TILE, OFF_L = OFF_DO + ST * TILE;
    static constexpr int OFF_BAR = OFF_L + ST * 2 * 128 * 4;
    static constexpr int BARS = 1 + 3 * ST + 8;
    static constexpr int SMEM = OFF_BAR + BARS * 8 + 16 + 1024;
};
static_assert(DkvShape<128>::SMEM <= 227 * 1024, "dK, dV shared memory");

// How a launch is cut: `tiles` key tiles of every entry, the first
// `sink_tiles` of them with `pieces` more CTAs each for the queries beyond the
// window's reach, `chunk` query tiles (of every head) per piece; `rows` keys
// are sinks.  An entry with at most `chunk` query tiles for a sink tile has no
// pieces for it.
//
// chunk: at least as many query tiles as an ordinary key tile has, and one
// more, so that the first piece holds all that the keys behind the sinks in the
// last sink tile are seen by; and not fewer than the sink tiles, which bounds
// the workspace (below).  When the sinks fill more than half of the key tiles
// nothing is cut: those tiles are then CTAs enough.
struct DkvCut {
    int tiles, sink_tiles, pieces, chunk, rows;
};

inline DkvCut dkv_cut(int64_t max_q, int64_t max_k, int64_t window, int64_t sinks) {
    DkvCut c{(int)((max_k + 127) / 128), 0, 0, 1, 0};
    if (window > 0 && sinks > 0) {
        const int64_t qt = (max_q + 127) / 128, rows = sinks < max_k ? sinks : max_k, st = (rows + 127) / 128;
        int64_t chunk = (window + 127) / 128 + 2;
        if (chunk < 4) chunk = 4;
        if (chunk < st) chunk = st;
        if (qt > chunk && 2 * st <= c.tiles) {
            c.sink_tiles = (int)st;
            c.chunk = (int)chunk;
            c.pieces = (int)((qt + chunk - 1) / chunk - 1);
            c.rows = (int)rows;
        }
    }
    return c;
}

// float32 sums of a piece (0: the first) of an entry whose queries begin at row
// q0, for one kv head: [dk, dv][rows][D].  An entry with k > 1 pieces has more
// than 128 chunk (k - 1) queries, so from one entry to the next q0 / (64 chunk)
// grows by at least 2 (k - 1) >= k: the places of different entries are apart,
// and Tq / (64 chunk) of them are enough.  rows <= 128 chunk: at most 2 Tq rows
// for each kv head.
__host__ __device__ inline size_t sink_places(const DkvCut &c, int64_t Tq) {
    return c.rows > 0 ? (size_t)(Tq / (64 * (int64_t)c.chunk)) : 0;
}
__host__ __device__ inline size_t sink_sums(const DkvCut &c, int Hkv, int D, size_t place, int kvh) {
    return (place * Hkv + kvh) * 2 * c.rows * D;
}
__device__ __forceinline__ size_t piece_sums(const DkvCut &c, const RaggedParams &p, const Entry &e, int kvh, int piece) {
    return sink_sums(c, p.Hkv, p.D, (size_t)(e.q0 / (64ll * c.chunk) + piece), kvh);
}

template <int DP>
__global__ void __launch_bounds__(AB_THREADS, 1)
    k_attn_dkdv_tc(const __grid_constant__ RaggedMaps maps, const __grid_constant__ RaggedParams p,
                   const __grid_constant__ DkvCut cutting, float *sums) {
    using F = DkvShape<DP>;
    constexpr int ST = F::ST;
    extern __shared__ uint8_t af_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(af_raw) + 1023) & ~(uintptr_t)1023);
    const u32 sbase = smem_u32(sm), bar0 = sbase + F::OFF_BAR;
    const u32 KVF = bar0, QF = bar0 + 8, QE = QF + 8 * ST, LF = QE + 8 * ST, SF = LF + 8 * ST, DPF = SF + 8, PR = DPF + 8,
              DSR = PR + 16, OUT = DSR + 16, DRAIN = OUT + 8;
    float *s_stat = reinterpret_cast<float *>(sm + F::OFF_L);  // [stage][-lse, -delta][128]
    u32 *s_tmem = reinterpret_cast<u32 *>(sm + F::OFF_BAR + F::BARS * 8);
    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + F::OFF_BAR + F::BARS * 8 + 4);
    constexpr unsigned long long TO = AB_TIMEOUT_NS;

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc_prefetch(&maps.q);
        tc_prefetch(&maps.k);
        tc_prefetch(&maps.v);
        tc_prefetch(&maps.dout);
    }
    const int kvh = blockIdx.y, b = blockIdx.z;
    Entry e;
    if (!entry_of(p, b, e)) return;
    if (e.nk > p.max_k) e.nk = p.max_k;  // further keys' gradients are left as they were
    // the sink tiles' pieces come first, then the key tiles
    const int extra = cutting.sink_tiles * cutting.pieces;
    const bool far = (int)blockIdx.x < extra;
    const int t = far ? (int)blockIdx.x / cutting.pieces : (int)blockIdx.x - extra;
    const int piece = far ? (int)blockIdx.x % cutting.pieces + 1 : 0;
    const int j0 = t * 128;
    if (j0 >= e.nk) return;
    const int keys = e.nk - j0 < 128 ? e.nk - j0 : 128;
    // query tiles that see the tile: from its first key's query on, to the window's reach of its last key
    int q_lo = j0 - e.off, q_hi = e.nq - 1;
    if (q_lo < 0) q_lo = 0;
    int t_lo = q_lo / 128, t_hi = q_hi >= q_lo ? q_hi / 128 : t_lo - 1;  // tiles t_lo .. t_hi
    const bool sink = j0 < p.sinks && p.window > 0;
    const bool to_sums = t < cutting.sink_tiles && t_hi - t_lo + 1 > cutting.chunk;
    if (t < cutting.sink_tiles) {
        // the main CTA keeps the first `chunk` tiles, piece i the i-th `chunk` after them
        t_lo += piece * cutting.chunk;
        if (t_hi > t_lo + cutting.chunk - 1) t_hi = t_lo + cutting.chunk - 1;
    } else if (p.window > 0 && !sink) {
        const long long last = (long long)j0 + keys - 1 + p.window - 1 - e.off;
        if (last < q_hi) t_hi = last < q_lo ? t_lo - 1 : (int)(last / 128);
    }
    const int qt = t_hi - t_lo + 1 > 0 ? t_hi - t_lo + 1 : 0, n = qt * p.group;
    if (far && n == 0) return;  // (its sums are not read)
    // the walk: query tiles t_lo .. t_hi of the group's first head, then of the next
    struct Walk {
        int head, tile;
    };
    auto advance = [&](Walk &w) {
        if (++w.tile > t_hi) {
            w.tile = t_lo;
            ++w.head;
        }
    };
    const Walk start{kvh * p.group, t_lo};

    if (threadIdx.x == 0) {
        for (int i = 0; i < F::BARS; ++i) mbar_init(bar0 + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(PR + 8 * i, 8);
            mbar_init(DSR + 8 * i, 8);
        }
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (n > 0) {  // on their way while TMEM is allocated
            mbar_arrive_expect_tx(KVF, 2 * F::TILE);
            tc_load_rows<DP>(&maps.k, sbase, kvh, e.k0 + j0, KVF);
            tc_load_rows<DP>(&maps.v, sbase + F::OFF_V, kvh, e.k0 + j0, KVF);
        }
    }
    if (warp == 1) tc_alloc(smem_u32(s_tmem), 512);
    tc_before();
    __syncthreads();
    tc_after();
    const u32 tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
    const u32 s_col = tmem, dp_col = tmem + 128, dv_col = tmem + 256, dk_col = tmem + 384;

    if (warp == 0) {
        if (lane == 0 && n > 0) {
            bool ok = true;
            int u = 0;
            Walk at = start;
            for (; u < n; ++u, advance(at)) {
                const int s = u % ST, row = e.q0 + at.tile * 128, h = at.head;
                if (u >= ST && !tc_wait(QE + 8 * s, (u32)((u / ST) & 1) ^ 1, TO, s_abort)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(QF + 8 * s, 2 * F::TILE);
                tc_load_rows<DP>(&maps.q, sbase + F::OFF_Q + s * F::TILE, h, row, QF + 8 * s);
                tc_load_rows<DP>(&maps.dout, sbase + F::OFF_DO + s * F::TILE, h, row, QF + 8 * s);
            }
            if (!ok) {
                raise_device_error(DEVERR_TIMEOUT_PRODUCER);
                *s_abort = 1;
            }
            tc_wait(KVF, 0, TO, nullptr);
            for (int j = u - ST > 0 ? u - ST : 0; j < u; ++j) tc_wait(QF + 8 * (j % ST), (u32)((j / ST) & 1), TO, nullptr);
        }
    } else if (warp == 1) {
        if (n > 0) {
            constexpr u32 ID_S = tc_idesc(128, false, false), ID_O = tc_idesc(DP, false, true);
            const bool leader = tc_elect();
            bool ok = TC_WAIT_ALL(KVF, 0, TO, s_abort);
            const u64 k_desc = tc_desc_k(sbase), v_desc = tc_desc_k(sbase + F::OFF_V), q_desc = tc_desc_k(sbase + F::OFF_Q),
                      do_desc = tc_desc_k(sbase + F::OFF_DO), qt_desc = tc_desc_mn(sbase + F::OFF_Q),
                      dot_desc = tc_desc_mn(sbase + F::OFF_DO);
            auto stage = [&](int u) { return (u64)(u % ST * F::TILE >> 4); };
            // columns 0 - 63 of P, dS are at the region's start, 64 - 127 at its column 64; the first half of each is
            // ready first (part 0: steps 0, 1, 4, 5)
            auto add = [&](u32 d, u32 a, u64 bt, int part, bool more) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kk = (i & 1) + (i >> 1) * 4 + 2 * part;
                    tc_mma_ts(d, a + (kk / 4) * 64 + (kk % 4) * 8, bt + (u64)(kk * 2048 >> 4), ID_O,
                              more || part != 0 || i != 0);
                }
            };
            auto add_when = [&](u32 bar, int u, u32 d, u32 a, u64 bt) {
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    ok = ok && TC_WAIT_ALL(bar + 8 * part, (u32)(u & 1), TO, s_abort);
                    if (!ok) return;
                    tc_after();
                    if (leader) add(d, a, bt, part, u != 0);
                    __syncwarp();
                }
            };
            auto q_ready = [&](int u) {
                const u32 ph = (u32)((u / ST) & 1);
                ok = ok && TC_WAIT_ALL(QF + 8 * (u % ST), ph, TO, s_abort) && TC_WAIT_ALL(LF + 8 * (u % ST), ph, TO, s_abort);
                tc_after();
            };
            q_ready(0);
            if (ok && leader) {
                tc_gemm_nt<DP>(s_col, k_desc, q_desc + stage(0), ID_S);
                tc_commit(SF);
                tc_gemm_nt<DP>(dp_col, v_desc, do_desc + stage(0), ID_S);
                tc_commit(DPF);
            }
            __syncwarp();
            for (int u = 0; u < n && ok; ++u) {
                // with more than two stages the next query tile has landed long before this one's weights are ready
                if (ST > 2 && u + 1 < n) q_ready(u + 1);
                add_when(PR, u, dv_col, s_col, dot_desc + stage(u));
                if (!ok) break;
                if (u + 1 < n) {
                    if (ST == 2) q_ready(u + 1);
                    if (!ok) break;
                    if (leader) {
                        tc_gemm_nt<DP>(s_col, k_desc, q_desc + stage(u + 1), ID_S);
                        tc_commit(SF);
                    }
                    __syncwarp();
                }
                add_when(DSR, u, dk_col, dp_col, qt_desc + stage(u));
                if (!ok) break;
                if (leader) {
                    tc_commit(QE + 8 * (u % ST));
                    if (u + 1 < n) {
                        tc_gemm_nt<DP>(dp_col, v_desc, do_desc + stage(u + 1), ID_S);
                        tc_commit(DPF);
                    }
                }
                __syncwarp();
            }
            if (!ok && lane == 0) {
                raise_device_error(DEVERR_TIMEOUT_MMA);
                *s_abort = 1;
            }
            if (leader) {
                if (ok) tc_commit(OUT);
                tc_commit(DRAIN);
            }
            __syncwarp();
            tc_wait(DRAIN, 0, TO, nullptr);
        }
    } else if (warp == 2) {
        // lse and delta of a query tile; rows behind the last query are cleared and get weights of zero
        bool ok = true;
        Walk at = start;
        for (int u = 0; u < n; ++u, advance(at)) {
            const int s = u % ST, i0 = at.tile * 128;
            const int rows = e.nq - i0 < 128 ? e.nq - i0 : 128;
            float lse[4], delta[4];
            const size_t stat = (size_t)at.head * p.Tq + e.q0 + i0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = lane + 32 * k;
                lse[k] = r < rows ? p.lse[stat + r] : -INFINITY;
                delta[k] = r < rows ? p.delta[stat + r] : 0.f;
            }
            ok = __all_sync(0xffffffffu, tc_wait(QF + 8 * s, (u32)((u / ST) & 1), TO, s_abort));
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // negated, to be added; a query that sees nothing has lse = -inf: its weights are exp2(S - inf) = 0 too
                s_stat[(s * 2) * 128 + lane + 32 * k] = lse[k] == -INFINITY ? -INFINITY : lse[k] * -1.44269504088896f;
                s_stat[(s * 2 + 1) * 128 + lane + 32 * k] = -delta[k];
            }
            if (rows < 128) {
                tc_zero_rows<DP>(sm + F::OFF_Q + s * F::TILE, rows);
                tc_zero_rows<DP>(sm + F::OFF_DO + s * F::TILE, rows);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(LF + 8 * s);
        }
        if (!ok && lane == 0) {
            raise_device_error(DEVERR_TIMEOUT_EXPAND);
            *s_abort = 1;
        }
    } else if (warp >= 4) {
        const int c = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;  // columns (queries) 64 c .. + 63 of key r
        const int key = j0 + r;
        const u32 lane_at = (u32)((warp & 3) * 32) << 16;
        const f32x2 sl2 = pack2(p.scale_log2, p.scale_log2);
        bool ok = true;
        Walk walk = start;
        for (int u = 0; u < n; ++u, advance(walk)) {
            const int s = u % ST, i0 = walk.tile * 128;
            ok = __all_sync(0xffffffffu, tc_wait(LF + 8 * s, (u32)((u / ST) & 1), TO, s_abort) &&
                                             tc_wait(SF, (u32)(u & 1), TO, s_abort));
            if (!ok) break;
            tc_after();
            u32 w[64];
            tc_ld32(w, s_col + lane_at + 64 * c);
            tc_ld32(w + 32, s_col + lane_at + 64 * c + 32);
            const float4 *nlse = reinterpret_cast<const float4 *>(s_stat + (s * 2) * 128 + 64 * c);
            const float4 *ndel = reinterpret_cast<const float4 *>(s_stat + (s * 2 + 1) * 128 + 64 * c);
            tc_wait_ld();
            const int first = i0 + e.off;  // position of column 0
            const bool whole = j0 + 127 <= first && (p.window == 0 || first + 127 - j0 < p.window || j0 + 128 <= p.sinks);
            const int lo = key - first - 64 * c;                                         // first query
            const int hi = p.window > 0 && key >= p.sinks ? lo + p.window : 0x7fffffff;  // behind the last one
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                u32 *v = w + 32 * q;
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 x = nlse[8 * q + j / 4];
                    float a, b2;
                    unpack2(fma2(pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), sl2, pack2(x.x, x.y)), a, b2);
                    v[j] = __float_as_uint(exp2_fast(a));
                    v[j + 1] = __float_as_uint(exp2_fast(b2));
                    unpack2(fma2(pack2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), sl2, pack2(x.z, x.w)), a, b2);
                    v[j + 2] = __float_as_uint(exp2_fast(a));
                    v[j + 3] = __float_as_uint(exp2_fast(b2));
                }
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * q + j < lo || 32 * q + j >= hi) v[j] = 0u;
                }
                u32 pk[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) pk[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                tc_st16(s_col + lane_at + 64 * c + 16 * q, pk);
                tc_hand_over(PR + 8 * q);
            }
            ok = __all_sync(0xffffffffu, tc_wait(DPF, (u32)(u & 1), TO, s_abort));
            if (!ok) break;
            tc_after();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                u32 g[32], pk[16];
                tc_ld32(g, dp_col + lane_at + 64 * c + 32 * q);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float4 x = ndel[8 * q + j / 2];
                    const u32 *v = w + 32 * q + 2 * j;
                    float a, b2;
                    unpack2(mul2(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                                 add2(pack2(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1])), pack2(x.x, x.y))), a, b2);
                    pk[j] = pack_bf16(a, b2);
                    unpack2(mul2(pack2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                                 add2(pack2(__uint_as_float(g[2 * j + 2]), __uint_as_float(g[2 * j + 3])), pack2(x.z, x.w))), a, b2);
                    pk[j + 1] = pack_bf16(a, b2);
                }
                tc_st16(dp_col + lane_at + 64 * c + 16 * q, pk);
                tc_hand_over(DSR + 8 * q);
            }
        }
        if (ok && n > 0) ok = __all_sync(0xffffffffu, tc_wait(OUT, 0, TO, s_abort));
        if (!ok) {
            if (lane == 0) {
                raise_device_error(DEVERR_TIMEOUT_EPILOGUE);
                *s_abort = 1;
            }
        } else {
            tc_after();
            // the first four warps write dV, the others dK
            const float f = c == 0 ? 1.f : p.scale;
            const u32 col = (c == 0 ? dv_col : dk_col) + lane_at;
            if (!far) {
                // (the query stages are not read any more; what has further pieces is written again by k_attn_sink_sum)
                const int at = 32 * (warp & 3);
                tc_store_rows<DP>(col, n == 0, f, sm + F::OFF_Q + (warp - 4) * 32 * DP * 2,
                                  (c == 0 ? p.dv : p.dk) + ((size_t)(e.k0 + j0 + at) * p.Hkv + kvh) * p.D,
                                  (long long)p.Hkv * p.D, keys - at, p.D);
            }
            if (to_sums && j0 + 32 * (warp & 3) < cutting.rows) {
                float *acc = sums + piece_sums(cutting, p, e, kvh, piece) + ((size_t)(c == 0 ? cutting.rows : 0) + key) * p.D;
#pragma unroll 1
                for (int k = 0; k < DP / 32; ++k) {
                    u32 o[32];
                    tc_ld32(o, col + 32 * k);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        if (r >= keys || key >= cutting.rows || 32 * k + j >= p.D) continue;
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(o[j + i]) * f;
                        store8(reinterpret_cast<uint8_t *>(acc + 32 * k + j), x, false);
                    }
                }
            }
        }
    }
    tc_before();
    __syncthreads();
    if (warp == 1) {
        tc_after();
        tc_dealloc(tmem, 512);
    }
}

// Sink tiles: the pieces' float32 sums, in order, to dk and dv.  AB_SUM_CTAS
// CTAs per (sink tile, kv head, entry): latency decides, so a thread adds up
// one or two places.
constexpr int AB_SUM_CTAS = 8;

__global__ void __launch_bounds__(256) k_attn_sink_sum(const __grid_constant__ RaggedParams p,
                                                       const __grid_constant__ DkvCut cutting, const float *sums) {
    const int t = blockIdx.x / AB_SUM_CTAS, kvh = blockIdx.y, b = blockIdx.z;
    Entry e;
    if (!entry_of(p, b, e)) return;
    if (e.nk > p.max_k) e.nk = p.max_k;
    const int j0 = t * 128;
    if (j0 >= e.nk) return;
    const int end = e.nk < cutting.rows ? e.nk : cutting.rows, keys = end - j0 < 128 ? end - j0 : 128;
    const int q_lo = j0 - e.off > 0 ? j0 - e.off : 0;
    const int t_lo = q_lo / 128, t_hi = e.nq - 1 >= q_lo ? (e.nq - 1) / 128 : t_lo - 1;
    const int tiles = t_hi - t_lo + 1;
    if (tiles <= cutting.chunk) return;  // (the first piece was all)
    const int pieces = (tiles + cutting.chunk - 1) / cutting.chunk;
    const float *base = sums + piece_sums(cutting, p, e, kvh, 0);
    const size_t step = sink_sums(cutting, p.Hkv, p.D, 1, 0);
    for (int i = (blockIdx.x % AB_SUM_CTAS * 256 + threadIdx.x) * 8; i < 2 * keys * p.D; i += AB_SUM_CTAS * 256 * 8) {
        const int which = i / (keys * p.D), at = i - which * keys * p.D;  // 0: dk, 1: dv
        const int r = at / p.D, d = at - r * p.D;
        float x[8] = {};
#pragma unroll 4
        for (int k = 0; k < pieces; ++k) {
            float y[8];
            load8<false>(reinterpret_cast<const uint8_t *>(base + k * step + ((size_t)which * cutting.rows + j0 + r) * p.D + d), y);
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] += y[c];
        }
        uint16_t *out = (which == 0 ? p.dk : p.dv) + ((size_t)(e.k0 + j0 + r) * p.Hkv + kvh) * p.D + d;
        store8(reinterpret_cast<uint8_t *>(out), x, true);
    }
}

}  // namespace bl
