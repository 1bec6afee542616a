// Rotary positions on q and k, rounding to the output types, and the new
// K / V rows into the pages of a cache, in one launch.
//
//   (y_i, y_{i + D/2}) = (x_i c - x_{i + D/2} s, x_{i + D/2} c + x_i s)
//
// A thread owns eight rotation pairs of one head of one token: elements
// i .. i + 7 and i + D/2 .. i + D/2 + 7 (16 values in, 16 out, all accesses
// 16 bytes), so the rotation needs no exchange and an output may be its
// input.  Bound by memory: every input is read once and every output written
// once; the rope rows (D floats per token, shared by its heads) come from L1.
#pragma once

#include "bl_common.cuh"

namespace bl {

constexpr int RA_THREADS = 128;

// The cache as the attention kernels see it (bl_kv_cache with narrow sizes).
struct KvView {
    uint8_t *k;
    uint8_t *v;
    const int *tables;
    const int *lengths;
    int num_pages, max_seqs, max_pages, ps_log;
};

struct RopeParams {
    const uint8_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;  // bytes
    long long units;                         // T * units_per_token
    int units_per_token;                     // (Hq + 2 Hkv) * D / 16 (absent inputs left out)
    int T, Hq, Hkv, D;
    const float *rope;
    int rope_len;
    float sign;  // of the sine: -1 rotates back
    const int *cu;
    int B;
    const int *seq_ids;
    const int *lengths;
    int max_seqs;
    int has_cache;
    KvView kv;
    uint8_t *q_out, *k_out, *v_out;
};

// 8 consecutive elements as floats.
template <bool BF16>
__device__ __forceinline__ void load8(const uint8_t *p, float (&x)[8]) {
    if (BF16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const u32 w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

// 8 consecutive elements, rounded once (to nearest, ties to even).
__device__ __forceinline__ void store8(uint8_t *p, const float (&x)[8], bool bf16) {
    if (bf16) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

template <bool SRC_BF16>
__global__ void __launch_bounds__(RA_THREADS) k_rope_append(const __grid_constant__ RopeParams p, int out_bf16,
                                                            int cache_bf16) {
    const long long u = (long long)blockIdx.x * RA_THREADS + threadIdx.x;
    if (u >= p.units) return;
    const int t = (int)(u / p.units_per_token);
    const int r = (int)(u - (long long)t * p.units_per_token);
    const int per = p.D >> 4;  // units of a head
    int head = r / per;
    const int i0 = (r - head * per) * 8;
    // which of q, k, v (an absent input has no units)
    const int hq = p.q != nullptr ? p.Hq : 0;
    const int hk = p.k != nullptr ? p.Hkv : 0;
    int which = 0;
    if (head >= hq) {
        head -= hq;
        which = 1;
        if (head >= hk) {
            head -= hk;
            which = 2;
        }
    }
    // batch entry of token t: the last b with cu[b] <= t
    int b = t, first = t, count = 1;
    if (p.cu != nullptr) {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(p.cu + mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        first = __ldg(p.cu + b);
        const int end = __ldg(p.cu + b + 1);
        if (t < first || t >= end) return;  // rows behind the last entry
        count = end - first;
    }
    const int seq = p.seq_ids != nullptr ? __ldg(p.seq_ids + b) : b;
    if (seq < 0) return;  // padding
    long long pos = t - first;
    if (p.lengths != nullptr) {
        if (seq >= p.max_seqs) {
            raise_device_error(DEVERR_INDEX);
            return;
        }
        pos += (long long)__ldg(p.lengths + seq) - count;
    }
    if (pos < 0 || (p.rope != nullptr && pos >= p.rope_len)) {
        raise_device_error(DEVERR_INDEX);
        return;
    }
    const int half = p.D >> 1;
    constexpr int ES = SRC_BF16 ? 2 : 4;
    const uint8_t *src = which == 0   ? p.q + t * p.q_stride
                         : which == 1 ? p.k + t * p.k_stride
                                      : p.v + t * p.v_stride;
    src += ((size_t)head * p.D + i0) * ES;
    float a[8], c[8];
    load8<SRC_BF16>(src, a);
    load8<SRC_BF16>(src + (size_t)half * ES, c);
    if (which < 2 && p.rope != nullptr) {
        const uint8_t *row = reinterpret_cast<const uint8_t *>(p.rope + (size_t)pos * p.D + i0);
        float cs[8], sn[8];
        load8<false>(row, cs);
        load8<false>(row + (size_t)half * 4, sn);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = sn[i] * p.sign, lo = a[i], hi = c[i];
            a[i] = lo * cs[i] - hi * s;
            c[i] = hi * cs[i] + lo * s;
        }
    }
    uint8_t *out = which == 0 ? p.q_out : which == 1 ? p.k_out : p.v_out;
    if (out != nullptr) {
        const int es = out_bf16 ? 2 : 4;
        const int H = which == 0 ? p.Hq : p.Hkv;
        out += (((size_t)t * H + head) * p.D + i0) * es;
        store8(out, a, out_bf16);
        store8(out + (size_t)half * es, c, out_bf16);
    }
    if (which > 0 && p.has_cache) {
        const long long col = pos >> p.kv.ps_log;
        const int page = col < p.kv.max_pages ? __ldg(p.kv.tables + (size_t)seq * p.kv.max_pages + col) : -1;
        if (page < 0 || page >= p.kv.num_pages) {
            raise_device_error(DEVERR_INDEX);
            return;
        }
        const int es = cache_bf16 ? 2 : 4;
        const int slot = (int)(pos & ((1 << p.kv.ps_log) - 1));
        uint8_t *d = (which == 1 ? p.kv.k : p.kv.v) +
                     ((((((size_t)page * p.Hkv + head) << p.kv.ps_log) + slot) * p.D + i0) * es);
        store8(d, a, cache_bf16);
        store8(d + (size_t)half * es, c, cache_bf16);
    }
}

}  // namespace bl
