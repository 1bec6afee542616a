// Ragged causal attention with a sliding window and sinks, forward, on
// tcgen05.
//
//   S = Q K^T, P = exp2(scale log2(e) (S - m)), O = P V / rowsum(P), one pass
//   over the visible key tiles with the running maximum m
//
// A CTA owns 256 consecutive queries of one head as two halves of 128 rows
// (TMEM lanes) that share the K and V tiles of 128 keys.  S of a half (128
// float32 columns of TMEM) is read by its softmax warpgroup, one thread per
// row; P goes back to TMEM as bf16 over the same columns and is the A operand
// of O += P V, whose accumulator stays in TMEM.  While one half is in its
// softmax the tensor core works for the other.  A half takes part only in
// tiles that some of its rows see; a tile that all of them see whole is not
// masked.  m moves (and O is rescaled) only when a row's maximum grows by more
// than 2^8, which sums in float32 absorb.
//
// Bound by the exponentials: a 128 x 128 tile is 1024 cycles of the special
// function unit beside 1024 cycles of tensor work at D = 128 (768 at 64).
//
// Warps: 0 TMA producer, 1 TMEM allocator and MMA issuer, 2 clears the rows
// behind the last key of a partial V tile, 4 - 7 and 8 - 11 the softmax of
// the halves.  Every wait is bounded (a wait that gives up raises the device
// error word and the CTA's abort flag; copies and MMAs in flight are awaited,
// bounded too, before TMEM is freed).
#pragma once

#include "k_attn_ragged.cuh"
#include "tc05.cuh"

namespace bl {

constexpr int AF_THREADS = 384;
constexpr int AF_ROWS = 256;
constexpr int AF_KEYS = 128;
// registers a thread: 168 at launch (the first warpgroup gives its share up,
// the softmax warpgroups take it); what is taken, (64 + 2 x 208) x 128, is
// checked against the kernel's own count before it is first launched
constexpr int AF_REGS_LOW = 64, AF_REGS_HIGH = 208;

template <int DP>
struct FwdShape {
    static constexpr int STAGES = DP == 64 ? 4 : 2;
    static constexpr int TILE = DP / 64 * TC_BLOCK;  // 128 rows
    static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + STAGES * TILE, OFF_BAR = OFF_V + STAGES * TILE;
    static constexpr int BARS = 2 + 4 * STAGES + 11;
    static constexpr int SMEM = OFF_BAR + BARS * 8 + 16 + 1024;
};

struct RaggedMaps {
    CUtensorMap q, k, v, dout;
};

// Which of a CTA's tiles (numbered as the CTA walks them) a half takes part in:
// the first ns and lo .. hi.
struct HalfTiles {
    int ns, lo, hi;
    __device__ __forceinline__ bool has(int u) const { return u < ns || (u >= lo && u <= hi); }
    __device__ __forceinline__ bool any() const { return hi >= 0; }
};
__device__ __forceinline__ HalfTiles half_tiles(const RaggedParams &p, const KeyTiles &all, int p0, int p1, int nk) {
    const KeyTiles t = key_tiles<AF_KEYS>(p, p0, p1, nk);
    if (t.count == 0) return HalfTiles{0, 0, -1};
    const int by = all.ns - all.wt;  // number of tile t among the CTA's: t + by from all.wt on
    // (a half that starts above the CTA's first window tile may count sink tiles of its own among those)
    const int ns = t.ns <= all.ns ? t.ns : t.ns >= all.wt ? t.ns + by : all.ns;
    return HalfTiles{ns, t.wt + by, t.wt + t.count - t.ns - 1 + by};
}

template <int DP>
__global__ void __launch_bounds__(AF_THREADS, 1)
    k_attn_fwd_tc(const __grid_constant__ RaggedMaps maps, const __grid_constant__ RaggedParams p) {
    using F = FwdShape<DP>;
    constexpr int ST = F::STAGES;
    extern __shared__ uint8_t af_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(af_raw) + 1023) & ~(uintptr_t)1023);
    const u32 sbase = smem_u32(sm), bar0 = sbase + F::OFF_BAR;
    const u32 QF = bar0, KF = bar0 + 16, KE = KF + 8 * ST, VF = KE + 8 * ST, VE = VF + 8 * ST, SF = VE + 8 * ST,
              PF = SF + 16, OF = PF + 32, CUT = OF + 16, FIX = CUT + 8, DRAIN = FIX + 8;
    u32 *s_tmem = reinterpret_cast<u32 *>(sm + F::OFF_BAR + F::BARS * 8);
    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + F::OFF_BAR + F::BARS * 8 + 4);
    constexpr unsigned long long TO = 2000000000ull;

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc_prefetch(&maps.q);
        tc_prefetch(&maps.k);
        tc_prefetch(&maps.v);
    }
    const int h = blockIdx.y, b = blockIdx.z;
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) check_entry(p, b);
    Entry e;
    if (!entry_of(p, b, e)) return;
    const int i0 = (gridDim.x - 1 - blockIdx.x) * AF_ROWS;  // the longest rows first
    if (i0 >= e.nq) return;
    const int kvh = h / p.group;
    const int rows0 = e.nq - i0 < 128 ? e.nq - i0 : 128;
    const int rows1 = e.nq - i0 <= 128 ? 0 : e.nq - i0 - 128 < 128 ? e.nq - i0 - 128 : 128;
    const int pos0 = i0 + e.off;
    const KeyTiles all = key_tiles<AF_KEYS>(p, pos0, pos0 + rows0 + rows1 - 1, e.nk);
    const HalfTiles ht0 = half_tiles(p, all, pos0, pos0 + rows0 - 1, e.nk);
    const HalfTiles ht1 = rows1 > 0 ? half_tiles(p, all, pos0 + 128, pos0 + 128 + rows1 - 1, e.nk) : HalfTiles{0, 0, -1};
    const int count = all.count;
    auto tile_of = [&](int u) { return u < all.ns ? u : all.wt + (u - all.ns); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < F::BARS; ++i) mbar_init(bar0 + 8 * i, 1);
        for (int i = 0; i < 4; ++i) mbar_init(PF + 8 * i, 4);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        // Q is on its way while TMEM is allocated
        for (int half = 0; half < 2; ++half) {
            if (!(half ? ht1 : ht0).any()) continue;
            mbar_arrive_expect_tx(QF + 8 * half, F::TILE);
            tc_load_rows<DP>(&maps.q, sbase + half * F::TILE, h, e.q0 + i0 + 128 * half, QF + 8 * half);
        }
    }
    if (warp == 1) tc_alloc(smem_u32(s_tmem), 512);
    tc_before();
    __syncthreads();
    tc_after();
    const u32 tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
    // TMEM columns: S / P of the halves at 0 and 128, O at 256 and 256 + DP
    auto s_col = [&](int half) { return tmem + 128u * half; };
    auto o_col = [&](int half) { return tmem + 256u + (u32)DP * half; };
    // the entry's last tile when it is partial (cut rows; then it can only be the last of this CTA): its V has a
    // barrier of its own, and another one that says its rows behind the last key are clear
    const int cut = e.nk % AF_KEYS;
    const int cut_tile = cut ? e.nk / AF_KEYS : -1;
    const bool cuts = count > 0 && tile_of(count - 1) == cut_tile;
    auto v_full = [&](int u) { return cuts && u == count - 1 ? CUT : VF + 8 * (u % ST); };
    auto v_phase = [&](int u) { return cuts && u == count - 1 ? 0u : (u32)((u / ST) & 1); };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(AF_REGS_LOW));
        if (warp == 0) {
            if (lane == 0) {
                bool failed = false;
                int u = 0, ks = 0;  // tiles of V and of K requested
                for (; u < count; ++u) {
                    const int s = u % ST, row = e.k0 + tile_of(u) * AF_KEYS;
                    const u32 ph = (u32)((u / ST) & 1) ^ 1;
                    // (K is wanted a step before V, and its stage is free that much earlier)
                    if (u >= ST && !tc_wait(KE + 8 * s, ph, TO, s_abort)) {
                        failed = true;
                        break;
                    }
                    mbar_arrive_expect_tx(KF + 8 * s, F::TILE);
                    tc_load_rows<DP>(&maps.k, sbase + F::OFF_K + s * F::TILE, kvh, row, KF + 8 * s);
                    ks = u + 1;
                    if (u >= ST && !tc_wait(VE + 8 * s, ph, TO, s_abort)) {
                        failed = true;
                        break;
                    }
                    mbar_arrive_expect_tx(v_full(u), F::TILE);
                    tc_load_rows<DP>(&maps.v, sbase + F::OFF_V + s * F::TILE, kvh, row, v_full(u));
                }
                if (failed) {
                    raise_device_error(DEVERR_TIMEOUT_PRODUCER);
                    *s_abort = 1;
                }
                // what was requested lands before the CTA exits
                for (int half = 0; half < 2; ++half)
                    if ((half ? ht1 : ht0).any()) tc_wait(QF + 8 * half, 0, TO, nullptr);
                for (int j = ks - ST > 0 ? ks - ST : 0; j < ks; ++j)
                    tc_wait(KF + 8 * (j % ST), (u32)((j / ST) & 1), TO, nullptr);
                for (int j = u - ST > 0 ? u - ST : 0; j < u; ++j) tc_wait(v_full(j), v_phase(j), TO, nullptr);
            }
        } else if (warp == 1) {
            if (count > 0) {
                constexpr u32 ID_QK = tc_idesc(AF_KEYS, false, false), ID_PV = tc_idesc(DP, false, true);
                const bool leader = tc_elect();
                const u64 q_desc = tc_desc_k(sbase), k_desc = tc_desc_k(sbase + F::OFF_K), v_desc = tc_desc_mn(sbase + F::OFF_V);
                bool ok = true;
                int n0 = 0, n1 = 0;  // tiles of a half whose P was consumed
                for (int half = 0; half < 2; ++half)
                    if ((half ? ht1 : ht0).any()) ok = ok && TC_WAIT_ALL(QF + 8 * half, 0, TO, s_abort);
                auto qk = [&](int half, int s) {
                    if (leader) {
                        tc_gemm_nt<DP>(s_col(half), q_desc + (u64)(half * F::TILE >> 4), k_desc + (u64)(s * F::TILE >> 4), ID_QK);
                        tc_commit(SF + 8 * half);
                    }
                    __syncwarp();
                };
                auto pv = [&](int half, int &n, int s, bool last) {
                    const u64 v = v_desc + (u64)(s * F::TILE >> 4);
                    // the weights of the first 64 keys are ready before the others
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        ok = ok && TC_WAIT_ALL(PF + 8 * (2 * half + part), (u32)(n & 1), TO, s_abort);
                        if (!ok) return;
                        tc_after();
                        if (leader) {
#pragma unroll
                            for (int kk = 4 * part; kk < 4 * part + 4; ++kk)
                                tc_mma_ts(o_col(half), s_col(half) + 8 * kk, v + (u64)(kk * 2048 >> 4), ID_PV, n != 0 || kk != 0);
                        }
                        __syncwarp();
                    }
                    ++n;
                    if (last && leader) tc_commit(OF + 8 * half);
                };
                ok = ok && TC_WAIT_ALL(KF, 0, TO, s_abort);
                if (ok) {
                    tc_after();
                    if (ht0.has(0)) qk(0, 0);
                    if (ht1.has(0)) qk(1, 0);
                    if (leader) tc_commit(KE);
                }
                for (int u = 0; u < count && ok; ++u) {
                    const int s = u % ST, s1 = (u + 1) % ST;
                    const bool more = u + 1 < count;
                    ok = TC_WAIT_ALL(cuts && !more ? FIX : VF + 8 * s, v_phase(u), TO, s_abort);
                    if (more) ok = ok && TC_WAIT_ALL(KF + 8 * s1, (u32)(((u + 1) / ST) & 1), TO, s_abort);
                    if (!ok) break;
                    if (ht0.has(u)) pv(0, n0, s, u == ht0.hi);
                    if (ok && more && ht0.has(u + 1)) qk(0, s1);
                    if (ok && ht1.has(u)) pv(1, n1, s, u == ht1.hi);
                    if (ok && more && ht1.has(u + 1)) qk(1, s1);
                    if (!ok) break;
                    if (leader) {
                        tc_commit(VE + 8 * s);
                        if (more) tc_commit(KE + 8 * s1);
                    }
                    __syncwarp();
                }
                if (!ok && lane == 0) {
                    raise_device_error(DEVERR_TIMEOUT_MMA);
                    *s_abort = 1;
                }
                // everything issued completes before TMEM is freed
                if (leader) tc_commit(DRAIN);
                __syncwarp();
                tc_wait(DRAIN, 0, TO, nullptr);
            }
        } else if (warp == 2) {
            if (cuts) {
                if (__all_sync(0xffffffffu, tc_wait(CUT, 0, TO, s_abort))) {
                    tc_zero_rows<DP>(sm + F::OFF_V + (count - 1) % ST * F::TILE, cut);
                    if (lane == 0) mbar_arrive(FIX);
                } else if (lane == 0) {
                    raise_device_error(DEVERR_TIMEOUT_EXPAND);
                    *s_abort = 1;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(AF_REGS_HIGH));
        const int half = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
        const int row = i0 + 128 * half + r, rows = half ? rows1 : rows0;
        const int pos = row + e.off;
        const u32 lane_at = (u32)((warp & 3) * 32) << 16;
        const HalfTiles mine = half ? ht1 : ht0;
        const int first_pos = pos0 + 128 * half, last_pos = first_pos + rows - 1;
        const float sl = p.scale_log2;
        float m = -INFINITY, l = 0.f;
        int n = 0;
        bool ok = true;
        for (int u = 0; u < count; ++u) {
            const int t = tile_of(u);
            if (!mine.has(u)) continue;
            ok = __all_sync(0xffffffffu, tc_wait(SF + 8 * half, (u32)(n & 1), TO, s_abort));
            if (!ok) break;
            tc_after();
            u32 w[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc_ld32(w + 32 * c, s_col(half) + lane_at + 32 * c);
            tc_wait_ld();
            const int j0 = t * AF_KEYS;
            // keys that some row of the half must not see: behind its position or the last key, or before its window
            const bool cut_hi = j0 + AF_KEYS - 1 > first_pos || j0 + AF_KEYS > e.nk;
            const bool cut_lo = p.window > 0 && last_pos - j0 >= p.window && j0 + AF_KEYS > p.sinks;
            if (cut_hi) {
                const int hi = (pos < e.nk - 1 ? pos : e.nk - 1) - j0;
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (j > hi) w[j] = 0xff800000u;
            }
            if (cut_lo) {
                const int lo = pos - p.window + 1 - j0, sk = p.sinks - j0;
                if (sk <= 0) {
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j < lo) w[j] = 0xff800000u;
                } else {
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j < lo && j >= sk) w[j] = 0xff800000u;
                }
            }
            float mq[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) mq[j] = __uint_as_float(w[j]);
#pragma unroll
            for (int j = 8; j < 128; ++j) mq[j & 7] = fmaxf(mq[j & 7], __uint_as_float(w[j]));
            const float mx = fmaxf(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])), fmaxf(fmaxf(mq[4], mq[5]), fmaxf(mq[6], mq[7])));
            // (rows behind the last query have no vote: they are another entry's, whose bits must not decide this one's)
            if (__any_sync(0xffffffffu, r < rows && ((mx - m) * sl > 8.f || m == -INFINITY))) {
                const float top = fmaxf(m, mx), c = m == -INFINITY ? 0.f : exp2_fast((m - top) * sl);
                m = top;
                l *= c;
                if (n > 0) {
#pragma unroll
                    for (int k = 0; k < DP / 32; ++k) {
                        u32 o[32];
                        tc_ld32(o, o_col(half) + lane_at + 32 * k);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * c);
                        tc_st32(o_col(half) + lane_at + 32 * k, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : m * sl;
            const f32x2 sl2 = pack2(sl, sl), nb2 = pack2(-base, -base);
            f32x2 sum[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                u32 pk[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float x, y;
                    unpack2(fma2(pack2(__uint_as_float(w[32 * c + 2 * j]), __uint_as_float(w[32 * c + 2 * j + 1])), sl2, nb2), x, y);
                    x = exp2_fast(x);
                    y = exp2_fast(y);
                    sum[j & 1] = add2(sum[j & 1], pack2(x, y));
                    pk[j] = pack_bf16(x, y);
                }
                tc_st16(s_col(half) + lane_at + 16 * c, pk);
                if (c & 1) {
                    tc_hand_over(PF + 8 * (2 * half + (c >> 1)));
                }
            }
            float x0, x1, x2, x3;
            unpack2(sum[0], x0, x1);
            unpack2(sum[1], x2, x3);
            l += (x0 + x1) + (x2 + x3);
            ++n;
        }
        if (ok && n > 0) ok = __all_sync(0xffffffffu, tc_wait(OF + 8 * half, 0, TO, s_abort));
        if (!ok) {
            if (lane == 0) {
                raise_device_error(DEVERR_TIMEOUT_EPILOGUE);
                *s_abort = 1;
            }
        } else if (rows > 0) {
            tc_after();
            const float f = l > 0.f ? 1.f / l : 0.f;
            // (the half's Q tile is not read any more)
            const int first = 32 * (warp & 3);
            tc_store_rows<DP>(o_col(half) + lane_at, n == 0, f, sm + half * F::TILE + first * DP * 2,
                              p.o + ((size_t)(e.q0 + i0 + 128 * half + first) * p.Hq + h) * p.D, (long long)p.Hq * p.D,
                              rows - first, p.D);
            if (r < rows)
                p.lse[(size_t)h * p.Tq + e.q0 + row] = l > 0.f ? m * p.scale + logf(l) : -INFINITY;
        }
    }
    tc_before();
    __syncthreads();
    if (warp == 1) {
        tc_after();
        tc_dealloc(tmem, 512);
    }
}

}  // namespace bl
