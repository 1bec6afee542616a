// tcgen05 and TMA pieces the attention kernels share (sm_100a): descriptors
// of 128-byte-swizzled bf16 tiles, MMA issue, TMEM loads and stores.
//
// A tile of R rows x 64 bf16 columns is R rows of 128 bytes in shared memory,
// 16-byte chunks permuted by the row (SWIZZLE_128B), 1024-byte aligned; wider
// matrices are several such blocks.  Read along its columns it is a K-major
// operand, read along its rows (rows = the contracted index) an MN-major one.
#pragma once

#include <cuda.h>

#include "bl_common.cuh"

namespace bl {

constexpr int TC_BLOCK = 128 * 128;  // bytes of 128 rows x 64 bf16 columns

// Descriptors; an operand `bytes` further on is the descriptor + (bytes >> 4).
// K-major: 8-row groups 1024 bytes apart; a step of 16 columns is +32 bytes.
__device__ __forceinline__ u64 tc_desc_k(u32 saddr) {
    return (u64)((saddr >> 4) & 0x3FFFu) | (u64)1u << 16 | (u64)(1024u >> 4) << 32 | (u64)1u << 46 | (u64)2u << 61;
}
// MN-major: 64-column blocks TC_BLOCK bytes apart, 8-row groups (of the
// contracted index) 1024 bytes apart; a step of 16 rows is +2048 bytes.
__device__ __forceinline__ u64 tc_desc_mn(u32 saddr) {
    return (u64)((saddr >> 4) & 0x3FFFu) | (u64)(TC_BLOCK >> 4) << 16 | (u64)(1024u >> 4) << 32 | (u64)1u << 46 |
           (u64)2u << 61;
}
// One lane of a converged warp.  The MMA warps stay converged and issue under
// this predicate, with operands the compiler can see to be uniform: from a
// branch on the lane number it moved every descriptor into uniform registers
// anew, 130 cycles per instruction of 64 cycles of work.
__device__ __forceinline__ bool tc_elect() {
    u32 e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// A converged warp's wait: true for all lanes or for none.
#define TC_WAIT_ALL(...) (__all_sync(0xffffffffu, tc_wait(__VA_ARGS__)) != 0)

// Bounded wait as mbar_wait, without its suspend-time hint: a phase of the
// attention kernels lasts a few hundred cycles, and a thread that was put to
// sleep comes back too late for the next one.
__device__ __forceinline__ bool tc_try(u32 bar, u32 parity) {
    u32 ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool tc_wait(u32 bar, u32 parity, unsigned long long timeout_ns, const volatile int *abort_flag) {
    if (tc_try(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (int it = 1;; ++it) {
        if (tc_try(bar, parity)) return true;
        if ((it & 63) == 0) {
            if (abort_flag != nullptr && *abort_flag) return false;
            if (globaltimer() - t0 > timeout_ns) return false;
        }
    }
}

// D float32, A and B bf16, M = 128; transposed operands are MN-major.
__host__ __device__ constexpr u32 tc_idesc(int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((u32)(n >> 3) << 17) |
           ((u32)(128 >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_ss(u32 d, u64 a, u64 b, u32 idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((u32)add)
        : "memory");
}
// A in TMEM (bf16 pairs, 8 columns per 16 of the contracted index).
__device__ __forceinline__ void tc_mma_ts(u32 d, u32 a, u64 b, u32 idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((u32)add)
        : "memory");
}
__device__ __forceinline__ void tc_commit(u32 bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_alloc(u32 slot, u32 cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(u32 tmem, u32 cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (+)= A B^T, both K-major, 128 rows each, DP columns.
template <int DP>
__device__ __forceinline__ void tc_gemm_nt(u32 d, u64 a, u64 b, u32 idesc) {
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
        const u64 at = (u64)(((kk / 4) * TC_BLOCK + (kk % 4) * 32) >> 4);
        tc_mma_ss(d, a + at, b + at, idesc, kk != 0);
    }
}

// What the warp stored to TMEM is handed over: one arrival per warp (an arrival
// per thread costs the barrier a few cycles each).
__device__ __forceinline__ void tc_hand_over(u32 bar) {
    tc_wait_st();
    tc_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// 32 columns of this thread's TMEM lane (call tc_wait_ld before using them).
__device__ __forceinline__ void tc_ld32(u32 *r, u32 addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_st32(u32 addr, const u32 *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_st16(u32 addr, const u32 *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tc_prefetch(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// 128 rows x DP columns of one head of a [T, H, D] tensor (map: D, H, T) into
// DP / 64 blocks; rows and columns beyond the tensor are zero.
template <int DP>
__device__ __forceinline__ void tc_load_rows(const CUtensorMap *map, u32 dst, int head, int row, u32 bar) {
#pragma unroll
    for (int c = 0; c < DP; c += 64)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                dst + (u32)(c / 64) * TC_BLOCK),
            "l"(map), "r"(c), "r"(head), "r"(row), "r"(bar)
            : "memory");
}

// A warp's 32 TMEM lanes x COLS columns (from column address `col`, lanes
// included), plus g times those `beside` columns further on (0: none), times f,
// as bf16 to rows of global memory: through the warp's own
// 32 x COLS x 2 bytes of shared memory (16-byte chunks permuted by the row), so
// that a row is written by neighbouring lanes.  Lane i's row goes to
// out + i * stride, columns below `cols`, if i < rows.  empty: zeros instead.
template <int COLS>
__device__ __forceinline__ void tc_store_rows(u32 col, bool empty, float f, uint8_t *stage, uint16_t *out, long long stride,
                                              int rows, int cols, int beside = 0, float g = 0.f) {
    constexpr int CH = COLS / 8, SWZ = CH < 8 ? CH - 1 : 7;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < COLS / 32; ++k) {
        u32 o[32];
        if (empty) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
        } else {
            tc_ld32(o, col + 32 * k);
            tc_wait_ld();
            if (beside != 0) {
                u32 x[32];
                tc_ld32(x, col + beside + 32 * k);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(fmaf(g, __uint_as_float(x[j]), __uint_as_float(o[j])));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 w;
            w.x = pack_bf16(__uint_as_float(o[8 * j]) * f, __uint_as_float(o[8 * j + 1]) * f);
            w.y = pack_bf16(__uint_as_float(o[8 * j + 2]) * f, __uint_as_float(o[8 * j + 3]) * f);
            w.z = pack_bf16(__uint_as_float(o[8 * j + 4]) * f, __uint_as_float(o[8 * j + 5]) * f);
            w.w = pack_bf16(__uint_as_float(o[8 * j + 6]) * f, __uint_as_float(o[8 * j + 7]) * f);
            *reinterpret_cast<uint4 *>(stage + lane * (COLS * 2) + (((4 * k + j) ^ (lane & SWZ)) << 4)) = w;
        }
    }
    __syncwarp();
    const int c = lane % CH;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int r = i * (32 / CH) + lane / CH;
        if (r < rows && c * 8 < cols)
            *reinterpret_cast<uint4 *>(out + r * stride + c * 8) =
                *reinterpret_cast<const uint4 *>(stage + r * (COLS * 2) + ((c ^ (r & SWZ)) << 4));
    }
}

// Rows from .. 127 of a tile to zero (one warp).  A tile's rows beyond its
// sequence belong to others or to nobody: their values must not meet a zero
// weight in a product, which would make NaN of an infinity.
template <int DP>
__device__ __forceinline__ void tc_zero_rows(uint8_t *tile, int from) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
        for (int i = from * 8 + lane; i < 128 * 8; i += 32)
            reinterpret_cast<uint4 *>(tile + c * TC_BLOCK)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

}  // namespace bl
