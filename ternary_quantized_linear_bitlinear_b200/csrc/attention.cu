// libbitlinear.so: the attention entry points declared in
// include/bitlinear_attn.h (rotary append, single-token attention over a
// paged cache, the cache's page tables, ragged causal attention with its
// gradients).  As in bitlinear.cu the host side only validates, chooses a
// launch and enqueues it on the caller's stream.
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>
#include <mutex>

#include "bitlinear_attn.h"
#include "bl_common.cuh"
#include "k_attn_bwd_tc.cuh"
#include "k_attn_decode.cuh"
#include "k_attn_fwd_tc.cuh"
#include "k_kv_pages.cuh"
#include "k_rope_append.cuh"

using namespace bl;

namespace bl {
// Reads and clears this translation unit's device error word.
bool attn_take_device_error(u32 *out) {
    u32 v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(v)) != cudaSuccess) return false;
    if (v != 0 && cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero)) != cudaSuccess) return false;
    *out = v;
    return true;
}
}  // namespace bl

namespace {

constexpr int MAX_DEVICES = 64;
constexpr int64_t I32_MAX = 0x7fffffffLL;
constexpr float LOG2E = 1.44269504088896f;

struct AttnDevice {
    bool init = false, ok = false;
    int sms = 0;
};
AttnDevice g_attn_dev[MAX_DEVICES];
std::mutex g_attn_mu;

template <typename K>
bool big_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

// Whether a kernel's registers at launch cover what its warpgroups ask for
// later (a request beyond them would wait for ever).
template <typename K>
bool covers_split(K kernel) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kernel) == cudaSuccess &&
           a.numRegs * AF_THREADS >= 128 * (AF_REGS_LOW + 2 * AF_REGS_HIGH);
}

bl_status attn_device(AttnDevice **out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return BL_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_attn_mu);
    AttnDevice &d = g_attn_dev[dev];
    if (!d.init) {
        int major = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return BL_ERR_CUDA;
        d.ok = major == 10;
        if (d.ok) {
            const int plan = (int)kv_plan_smem(KV_MAX_SEQS, KV_MAX_N, 2);
            if (!covers_split(k_attn_fwd_tc<64>) || !covers_split(k_attn_fwd_tc<128>)) return BL_ERR_CUDA;
            if (!big_smem(k_kv_extend, plan) || !big_smem(k_kv_fork_plan, plan) ||
                !big_smem(k_attn_fwd_tc<64>, FwdShape<64>::SMEM) || !big_smem(k_attn_fwd_tc<128>, FwdShape<128>::SMEM) ||
                !big_smem(k_attn_dq_tc<64>, DqShape<64>::SMEM) || !big_smem(k_attn_dq_tc<128>, DqShape<128>::SMEM) ||
                !big_smem(k_attn_dkdv_tc<64>, DkvShape<64>::SMEM) || !big_smem(k_attn_dkdv_tc<128>, DkvShape<128>::SMEM))
                return BL_ERR_CUDA;
        }
        d.init = true;
    }
    if (!d.ok) return BL_ERR_DEVICE;
    *out = &d;
    return BL_OK;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
inline bool good_dtype(bl_dtype t) { return t == BL_F32 || t == BL_BF16; }
inline int esize(bl_dtype t) { return t == BL_BF16 ? 2 : 4; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

bl_status check_heads(int64_t Hq, int64_t Hkv, int64_t D) {
    if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq > 65535) return BL_ERR_SHAPE;
    if (D < 16 || D > 128 || D % 16 != 0) return BL_ERR_SHAPE;
    return BL_OK;
}

// A strided tensor of rows of `width` elements.
bl_status check_rows(const void *p, int64_t stride, int64_t width, int es) {
    if (stride < width || stride > I32_MAX) return BL_ERR_SHAPE;
    if (!aligned16(p) || (stride * es) % 16 != 0) return BL_ERR_ALIGN;
    return BL_OK;
}

int log2_of(int64_t x) {
    int n = 0;
    while ((1LL << n) < x) ++n;
    return n;
}

bl_status check_tables(int64_t num_pages, int64_t page_size, int64_t max_seqs, int64_t max_pages) {
    if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return BL_ERR_SHAPE;
    if (num_pages < 1 || num_pages > (1 << 20) || max_seqs < 1 || max_seqs > KV_MAX_SEQS || max_pages < 1 ||
        max_pages > I32_MAX / page_size)
        return BL_ERR_SHAPE;
    return BL_OK;
}

bl_status kv_view(const bl_kv_cache *c, KvView *v) {
    if (!c->k_pages || !c->v_pages || !c->tables || !c->lengths) return BL_ERR_NULL;
    if (!good_dtype(c->dtype)) return BL_ERR_DTYPE;
    bl_status rc = check_tables(c->num_pages, c->page_size, c->max_seqs, c->max_pages);
    if (rc) return rc;
    if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned4(c->tables) || !aligned4(c->lengths))
        return BL_ERR_ALIGN;
    *v = KvView{reinterpret_cast<uint8_t *>(c->k_pages), reinterpret_cast<uint8_t *>(c->v_pages), c->tables, c->lengths,
                (int)c->num_pages, (int)c->max_seqs, (int)c->max_pages, log2_of(c->page_size)};
    return BL_OK;
}

// A launch that may start while the kernel before it ends (it waits for it
// with griddepcontrol.wait before it reads anything).
template <typename... A>
bl_status launch_after(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? BL_OK : BL_ERR_CUDA;
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(ptr);
    });
    return fn;
}

// Map of rows of heads [T, H, D] bf16 (row stride in elements): boxes of 128
// rows x 64 columns of one head, 128-byte swizzle, zeros outside.
bool head_map(CUtensorMap *m, const void *base, int64_t T, int64_t H, int64_t D, int64_t stride) {
    EncodeTiled enc = encode_tiled();
    if (enc == nullptr) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, 128}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dim, str, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------------------
// single-token attention

// Query heads of a segment, and head groups per kv head.
inline void head_groups(int64_t group, int *parts, int *gsize) {
    *parts = (int)((group + AD_G - 1) / AD_G);
    *gsize = (int)((group + *parts - 1) / *parts);
}

template <typename C>
bl_status launch_decode(DecodeAttnParams &P, const AttnDevice &d, int64_t batches_at_most, cudaStream_t st) {
    int ctas = d.sms * C::OCC;
    if (ctas > AD_MAX_CTAS) ctas = AD_MAX_CTAS;
    // no more warps than batches
    const int64_t need = (batches_at_most + C::WARPS - 1) / C::WARPS;
    if (need < ctas) ctas = (int)(need < 1 ? 1 : need);
    static std::atomic<u64> ready{0};  // devices this kernel's shared memory is set up on
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BL_ERR_CUDA;
    if (!(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
        if (!big_smem(k_attn_decode<C>, ad_smem<C>(C::G))) return BL_ERR_CUDA;
        ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    k_attn_decode<C><<<ctas, C::WARPS * 32, ad_smem<C>(P.gsize), st>>>(P);
    if (cudaGetLastError() != cudaSuccess) return BL_ERR_CUDA;
    if (ctas == 1) return BL_OK;  // nothing spans CTAs
    return launch_after(k_attn_join<C::DP>, dim3((unsigned)ctas - 1, (unsigned)P.gsize), AD_JOIN_THREADS, 0, st, P);
}

template <int DP>
bl_status decode_by_type(DecodeAttnParams &P, const AttnDevice &d, bool bf16_cache, int64_t batches, cudaStream_t st) {
    if (bf16_cache) {
        // 12 warps an SM (168 registers a thread); three slots a warp where a partial of up to 8 heads takes the
        // room of a fourth
        if (P.q_bf16)
            return P.gsize <= 4 ? launch_decode<DecodeMma<DP, DEC_BF16, 4, 3, 4>>(P, d, batches, st)
                                : launch_decode<DecodeMma<DP, DEC_BF16, 4, 3, 3>>(P, d, batches, st);
        return P.gsize <= 4 ? launch_decode<DecodeMma<DP, DEC_F32_4, 4, 3, 4>>(P, d, batches, st)
                            : launch_decode<DecodeMma<DP, DEC_F32_8, 4, 3, 3>>(P, d, batches, st);
    }
    // float32 cache: a head group's registers decide how many warps an SM holds (16 up to 3 heads, 8 above).  64 x 1028
    // keys of 20 unshared heads of 128: 236 us for one head, 244 us in the kernel for 3, 324 us in that for 8;
    // 64 x 3000 of 12 / 4 heads 150 us (5.2 TB/s) against 199 us.  8 heads: 3.9 TB/s, bound by the products.
    if (P.gsize == 1) return launch_decode<DecodeFma<DP, 1, 8, 2, 3>>(P, d, batches, st);
    if (P.gsize <= 3) return launch_decode<DecodeFma<DP, 3, 8, 2, 3>>(P, d, batches, st);
    return launch_decode<DecodeFma<DP, 8, 8, 1, 4>>(P, d, batches, st);
}

}  // namespace

extern "C" {

bl_status bl_rope_append(const void *q, const void *k, const void *v, bl_dtype xdt, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                         const float *rope, int64_t rope_len, int inverse, const int32_t *cu_seqlens, int64_t B,
                         const int32_t *seq_ids, const int32_t *lengths, int64_t max_seqs, const bl_kv_cache *cache,
                         void *q_out, void *k_out, void *v_out, bl_dtype odt, bl_stream_t stream) {
    if (!q && !k) return BL_ERR_NULL;
    if ((q == nullptr) != (q_out == nullptr)) return BL_ERR_NULL;
    if ((k == nullptr) != (v == nullptr)) return BL_ERR_NULL;
    if (!k && (k_out || v_out || cache)) return BL_ERR_NULL;
    if (k && !k_out && !v_out && !cache) return BL_ERR_NULL;
    if (!good_dtype(xdt) || !good_dtype(odt)) return BL_ERR_DTYPE;
    bl_status rc = check_heads(Hq, Hkv, D);
    if (rc) return rc;
    if (T < 1 || T > I32_MAX || B < 1 || B > I32_MAX - 1 || (!cu_seqlens && T != B)) return BL_ERR_SHAPE;
    if (rope && (rope_len < 1 || rope_len > I32_MAX)) return BL_ERR_SHAPE;
    if (cache && lengths) return BL_ERR_SHAPE;
    if (lengths && (max_seqs < 1 || max_seqs > KV_MAX_SEQS)) return BL_ERR_SHAPE;
    const int es = esize(xdt);
    if (q && (rc = check_rows(q, q_stride, Hq * D, es))) return rc;
    if (k && ((rc = check_rows(k, k_stride, Hkv * D, es)) || (rc = check_rows(v, v_stride, Hkv * D, es)))) return rc;
    if (!aligned16(q_out) || !aligned16(k_out) || !aligned16(v_out) || !aligned16(rope) || !aligned4(cu_seqlens) ||
        !aligned4(seq_ids) || !aligned4(lengths))
        return BL_ERR_ALIGN;
    RopeParams P;
    memset(&P, 0, sizeof(P));
    if (cache && (rc = kv_view(cache, &P.kv))) return rc;
    P.q = reinterpret_cast<const uint8_t *>(q);
    P.k = reinterpret_cast<const uint8_t *>(k);
    P.v = reinterpret_cast<const uint8_t *>(v);
    P.q_stride = q_stride * es;
    P.k_stride = k_stride * es;
    P.v_stride = v_stride * es;
    P.units_per_token = (int)(((q ? Hq : 0) + (k ? 2 * Hkv : 0)) * (D / 16));
    P.units = T * P.units_per_token;
    P.T = (int)T;
    P.Hq = (int)Hq;
    P.Hkv = (int)Hkv;
    P.D = (int)D;
    P.rope = rope;
    P.rope_len = (int)rope_len;
    P.sign = inverse ? -1.f : 1.f;
    P.cu = cu_seqlens;
    P.B = (int)B;
    P.seq_ids = seq_ids;
    P.lengths = cache ? cache->lengths : lengths;
    P.max_seqs = (int)(cache ? cache->max_seqs : max_seqs);
    P.has_cache = cache != nullptr;
    P.q_out = reinterpret_cast<uint8_t *>(q_out);
    P.k_out = reinterpret_cast<uint8_t *>(k_out);
    P.v_out = reinterpret_cast<uint8_t *>(v_out);
    const int64_t blocks = (P.units + RA_THREADS - 1) / RA_THREADS;
    if (blocks > I32_MAX) return BL_ERR_SHAPE;
    AttnDevice *d;
    if ((rc = attn_device(&d))) return rc;
    const int ob = odt == BL_BF16, cb = cache && cache->dtype == BL_BF16;
    if (xdt == BL_BF16) k_rope_append<true><<<(unsigned)blocks, RA_THREADS, 0, (cudaStream_t)stream>>>(P, ob, cb);
    else k_rope_append<false><<<(unsigned)blocks, RA_THREADS, 0, (cudaStream_t)stream>>>(P, ob, cb);
    return cudaGetLastError() == cudaSuccess ? BL_OK : BL_ERR_CUDA;
}

size_t bl_attn_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
    if (B < 1 || B > AD_MAX_B || check_heads(Hq, Hkv, D) != BL_OK) return 0;
    int parts, gsize;
    head_groups(Hq / Hkv, &parts, &gsize);
    return align256((size_t)AD_MAX_CTAS * 32) + (size_t)2 * AD_MAX_CTAS * gsize * ((D <= 64 ? 64 : 128) + 2) * 4;
}

bl_status bl_attn_decode(const void *q, bl_dtype xdt, int64_t q_stride, int64_t B, int64_t Hq, int64_t Hkv,
                         int64_t D, const bl_kv_cache *cache, const int32_t *seq_ids, int64_t window,
                         int64_t sinks, float scale, void *workspace, size_t workspace_bytes, void *out,
                         float *lse, bl_stream_t stream) {
    if (!q || !cache || !out) return BL_ERR_NULL;
    if (!good_dtype(xdt)) return BL_ERR_DTYPE;
    bl_status rc = check_heads(Hq, Hkv, D);
    if (rc) return rc;
    if (B < 1 || B > AD_MAX_B || window < 0 || sinks < 0) return BL_ERR_SHAPE;
    if (!(scale > 0.f && scale < 1e30f)) return BL_ERR_SHAPE;
    if ((rc = check_rows(q, q_stride, Hq * D, esize(xdt)))) return rc;
    if (!aligned16(out) || !aligned4(lse) || !aligned4(seq_ids)) return BL_ERR_ALIGN;
    DecodeAttnParams P;
    memset(&P, 0, sizeof(P));
    if ((rc = kv_view(cache, &P.kv))) return rc;
    if (!seq_ids && B > cache->max_seqs) return BL_ERR_SHAPE;
    if (!workspace || workspace_bytes < bl_attn_decode_workspace_bytes(B, Hq, Hkv, D)) return BL_ERR_WORKSPACE;
    if (!aligned16(workspace)) return BL_ERR_ALIGN;
    P.q = reinterpret_cast<const uint8_t *>(q);
    P.q_stride = q_stride * esize(xdt);
    P.q_bf16 = xdt == BL_BF16;
    P.B = (int)B;
    P.Hq = (int)Hq;
    P.Hkv = (int)Hkv;
    P.D = (int)D;
    P.group = (int)(Hq / Hkv);
    head_groups(P.group, &P.parts, &P.gsize);
    P.seq_ids = seq_ids;
    const int64_t most = cache->max_pages * cache->page_size;
    P.window = (int)(window > most ? most : window);
    P.sinks = (int)(sinks > most ? most : sinks);
    P.scale_log2 = scale * LOG2E;
    P.out = reinterpret_cast<uint8_t *>(out);
    P.lse = lse;
    P.open = reinterpret_cast<long long *>(workspace);
    P.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(workspace) + align256((size_t)AD_MAX_CTAS * 32));
    AttnDevice *d;
    if ((rc = attn_device(&d))) return rc;
    // the line of batches at most, for small calls (8 keys per batch is the least)
    const int64_t seen = window > 0 && P.window + (int64_t)P.sinks < most ? P.window + P.sinks + 64 : most;
    const int64_t batches = B * Hkv * P.parts * (seen / 8 + 1);
    cudaStream_t st = (cudaStream_t)stream;
    const bool bf16 = cache->dtype == BL_BF16;
    return D <= 64 ? decode_by_type<64>(P, *d, bf16, batches, st) : decode_by_type<128>(P, *d, bf16, batches, st);
}

// ---------------------------------------------------------------------------
// page tables

bl_status bl_kv_extend(int32_t *tables, int32_t *lengths, int32_t *refs, int64_t num_pages, int64_t page_size,
                       int64_t max_seqs, int64_t max_pages, const int32_t *seq_ids, const int32_t *counts,
                       int64_t n, int32_t *status, int32_t *active, bl_stream_t stream) {
    if (!tables || !lengths || !refs || !seq_ids || !counts || !status) return BL_ERR_NULL;
    bl_status rc = check_tables(num_pages, page_size, max_seqs, max_pages);
    if (rc) return rc;
    if (n < 1 || n > KV_MAX_N) return BL_ERR_SHAPE;
    if (!aligned4(tables) || !aligned4(lengths) || !aligned4(refs) || !aligned4(seq_ids) || !aligned4(counts) ||
        !aligned4(status) || !aligned4(active))
        return BL_ERR_ALIGN;
    AttnDevice *d;
    if ((rc = attn_device(&d))) return rc;
    const KvExtendParams P{{tables, lengths, refs, (int)num_pages, (int)max_seqs, (int)max_pages, log2_of(page_size)},
                           seq_ids, counts, (int)n, status, active};
    k_kv_extend<<<1, KV_THREADS, kv_plan_smem((int)max_seqs, (int)n, 1), (cudaStream_t)stream>>>(P);
    return cudaGetLastError() == cudaSuccess ? BL_OK : BL_ERR_CUDA;
}

bl_status bl_kv_free(int32_t *tables, int32_t *lengths, int32_t *refs, int64_t num_pages, int64_t page_size,
                     int64_t max_seqs, int64_t max_pages, const int32_t *seq_ids, int64_t n, bl_stream_t stream) {
    if (!tables || !lengths || !refs || !seq_ids) return BL_ERR_NULL;
    bl_status rc = check_tables(num_pages, page_size, max_seqs, max_pages);
    if (rc) return rc;
    if (n < 1 || n > KV_MAX_N) return BL_ERR_SHAPE;
    if (!aligned4(tables) || !aligned4(lengths) || !aligned4(refs) || !aligned4(seq_ids)) return BL_ERR_ALIGN;
    AttnDevice *d;
    if ((rc = attn_device(&d))) return rc;
    const KvFreeParams P{{tables, lengths, refs, (int)num_pages, (int)max_seqs, (int)max_pages, log2_of(page_size)},
                         seq_ids, (int)n};
    k_kv_free<<<(unsigned)n, 128, 0, (cudaStream_t)stream>>>(P);
    return cudaGetLastError() == cudaSuccess ? BL_OK : BL_ERR_CUDA;
}

size_t bl_kv_fork_workspace_bytes(int64_t n) {
    return n < 1 || n > KV_MAX_N ? 0 : align256((size_t)(1 + 3 * n) * 4);
}

bl_status bl_kv_fork(void *pool, int64_t planes, int64_t page_bytes, int32_t *tables, int32_t *lengths,
                     int32_t *refs, int64_t num_pages, int64_t page_size, int64_t max_seqs, int64_t max_pages,
                     const int32_t *src, const int32_t *dst, int64_t n, void *workspace, size_t workspace_bytes,
                     int32_t *status, bl_stream_t stream) {
    if (!pool || !tables || !lengths || !refs || !src || !dst || !status) return BL_ERR_NULL;
    bl_status rc = check_tables(num_pages, page_size, max_seqs, max_pages);
    if (rc) return rc;
    if (n < 1 || n > KV_MAX_N || planes < 1 || planes > 65536 || page_bytes < 16 || page_bytes > I32_MAX)
        return BL_ERR_SHAPE;
    if (!aligned16(pool) || page_bytes % 16 != 0 || !aligned4(tables) || !aligned4(lengths) || !aligned4(refs) ||
        !aligned4(src) || !aligned4(dst) || !aligned4(status))
        return BL_ERR_ALIGN;
    if (!workspace || workspace_bytes < bl_kv_fork_workspace_bytes(n)) return BL_ERR_WORKSPACE;
    if (!aligned16(workspace)) return BL_ERR_ALIGN;
    AttnDevice *d;
    if ((rc = attn_device(&d))) return rc;
    const KvTables t{tables, lengths, refs, (int)num_pages, (int)max_seqs, (int)max_pages, log2_of(page_size)};
    int *plan = reinterpret_cast<int *>(workspace);
    const KvForkParams P{t, src, dst, (int)n, status, plan};
    k_kv_fork_plan<<<1, KV_THREADS, kv_plan_smem((int)max_seqs, (int)n, 2), (cudaStream_t)stream>>>(P);
    if (cudaGetLastError() != cudaSuccess) return BL_ERR_CUDA;
    const KvCopyParams C{t, reinterpret_cast<uint8_t *>(pool), page_bytes, (int)planes, src, dst, (int)n, plan};
    const int64_t items = n * planes, most = (int64_t)d->sms * 8;
    return launch_after(k_kv_fork_copy, dim3((unsigned)(items < most ? items : most)), KV_COPY_THREADS, 0,
                        (cudaStream_t)stream, C);
}

size_t bl_kv_compact_workspace_bytes(int64_t num_pages) {
    return num_pages < 1 || num_pages > (1 << 20) ? 0 : align256((size_t)(2 + 3 * num_pages) * 4);
}

bl_status bl_kv_compact(void *pool, int64_t planes, int64_t page_bytes, int32_t *tables, int32_t *refs,
                        int64_t num_pages, int64_t max_seqs, int64_t max_pages, void *workspace,
                        size_t workspace_bytes, int32_t *n_live, bl_stream_t stream) {
    if (!pool || !tables || !refs || !n_live) return BL_ERR_NULL;
    bl_status rc = check_tables(num_pages, 8, max_seqs, max_pages);
    if (rc) return rc;
    if (planes < 1 || planes > 65536 || page_bytes < 16 || page_bytes > I32_MAX) return BL_ERR_SHAPE;
    if (!aligned16(pool) || page_bytes % 16 != 0 || !aligned4(tables) || !aligned4(refs) || !aligned4(n_live))
        return BL_ERR_ALIGN;
    if (!workspace || workspace_bytes < bl_kv_compact_workspace_bytes(num_pages)) return BL_ERR_WORKSPACE;
    if (!aligned16(workspace)) return BL_ERR_ALIGN;
    AttnDevice *d;
    if ((rc = attn_device(&d))) return rc;
    const KvTables t{tables, nullptr, refs, (int)num_pages, (int)max_seqs, (int)max_pages, 3};
    int *plan = reinterpret_cast<int *>(workspace);
    const KvCompactParams P{t, plan, n_live};
    k_kv_compact_plan<<<1, KV_THREADS, 0, (cudaStream_t)stream>>>(P);
    if (cudaGetLastError() != cudaSuccess) return BL_ERR_CUDA;
    const KvCopyParams C{t, reinterpret_cast<uint8_t *>(pool), page_bytes, (int)planes, nullptr, nullptr, 0, plan};
    const int64_t items = num_pages * planes, most = (int64_t)d->sms * 8;
    return launch_after(k_kv_compact_copy, dim3((unsigned)(items < most ? items : most)), KV_COPY_THREADS, 0,
                        (cudaStream_t)stream, C);
}

// ---------------------------------------------------------------------------
// ragged attention

// A window or sinks beyond every length mean no window, or every key.
static int norm_window(int64_t w) { return (int)(w > (1 << 25) ? 0 : w); }
static int norm_sinks(int64_t s) { return (int)(s > (1 << 25) ? (1 << 25) : s); }

static bl_status ragged_params(RaggedParams *P, const void *q, const void *k, const void *v, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv,
                               int64_t D, const int32_t *cu_q, const int32_t *cu_k, int64_t B, int64_t max_q,
                               int64_t max_k, int64_t window, int64_t sinks, float scale) {
    if (!q || !k || !v || !cu_q || !cu_k) return BL_ERR_NULL;
    bl_status rc = check_heads(Hq, Hkv, D);
    if (rc) return rc;
    if (Tq < 1 || Tk < 1 || B < 1 || B > 65535 || Tq * Hq > I32_MAX || Tk * Hkv > I32_MAX || Tq > I32_MAX || Tk > I32_MAX)
        return BL_ERR_SHAPE;
    if (max_q < 1 || max_k < 1 || max_q >= (1 << 24) || max_k >= (1 << 24) || window < 0 || sinks < 0) return BL_ERR_SHAPE;
    if (!(scale > 0.f && scale < 1e30f)) return BL_ERR_SHAPE;
    if ((rc = check_rows(q, q_stride, Hq * D, 2)) || (rc = check_rows(k, k_stride, Hkv * D, 2)) ||
        (rc = check_rows(v, v_stride, Hkv * D, 2)))
        return rc;
    if (!aligned4(cu_q) || !aligned4(cu_k)) return BL_ERR_ALIGN;
    memset(P, 0, sizeof(*P));
    P->q = reinterpret_cast<const uint16_t *>(q);
    P->k = reinterpret_cast<const uint16_t *>(k);
    P->v = reinterpret_cast<const uint16_t *>(v);
    P->q_stride = q_stride;
    P->k_stride = k_stride;
    P->v_stride = v_stride;
    P->Tq = (int)Tq;
    P->Tk = (int)Tk;
    P->Hq = (int)Hq;
    P->Hkv = (int)Hkv;
    P->D = (int)D;
    P->group = (int)(Hq / Hkv);
    P->cu_q = cu_q;
    P->cu_k = cu_k;
    P->B = (int)B;
    P->max_q = (int)max_q;
    P->max_k = (int)max_k;
    P->window = norm_window(window);
    P->sinks = norm_sinks(sinks);
    P->scale = scale;
    P->scale_log2 = scale * LOG2E;
    return BL_OK;
}

bl_status bl_attn_forward(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                          int64_t v_stride, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                          const int32_t *cu_q, const int32_t *cu_k, int64_t B, int64_t max_q, int64_t max_k,
                          int64_t window, int64_t sinks, float scale, void *o, float *lse, bl_stream_t stream) {
    RaggedParams P;
    bl_status rc = ragged_params(&P, q, k, v, q_stride, k_stride, v_stride, Tq, Tk, Hq, Hkv, D, cu_q, cu_k, B, max_q,
                                 max_k, window, sinks, scale);
    if (rc) return rc;
    if (!o || !lse) return BL_ERR_NULL;
    if (!aligned16(o) || !aligned4(lse)) return BL_ERR_ALIGN;
    P.o = reinterpret_cast<uint16_t *>(o);
    P.lse = lse;
    AttnDevice *d;
    if ((rc = attn_device(&d))) return rc;
    RaggedMaps maps;
    memset(&maps, 0, sizeof(maps));
    if (!head_map(&maps.q, q, Tq, Hq, D, q_stride) || !head_map(&maps.k, k, Tk, Hkv, D, k_stride) ||
        !head_map(&maps.v, v, Tk, Hkv, D, v_stride))
        return BL_ERR_CUDA;
    const dim3 grid((unsigned)((P.max_q + AF_ROWS - 1) / AF_ROWS), (unsigned)Hq, (unsigned)B);
    if (D <= 64) k_attn_fwd_tc<64><<<grid, AF_THREADS, FwdShape<64>::SMEM, (cudaStream_t)stream>>>(maps, P);
    else k_attn_fwd_tc<128><<<grid, AF_THREADS, FwdShape<128>::SMEM, (cudaStream_t)stream>>>(maps, P);
    return cudaGetLastError() == cudaSuccess ? BL_OK : BL_ERR_CUDA;
}

size_t bl_attn_backward_workspace_bytes(int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D, int64_t B,
                                        int64_t max_q, int64_t max_k, int64_t window, int64_t sinks) {
    if (Tq < 1 || Tk < 1 || B < 1 || max_q < 1 || max_k < 1 || window < 0 || sinks < 0 || check_heads(Hq, Hkv, D) != BL_OK)
        return 0;
    if (max_q >= (1 << 24) || max_k >= (1 << 24) || B > 65535) return 0;
    const DkvCut cut = dkv_cut(max_q, max_k, norm_window(window), norm_sinks(sinks));
    return align256((size_t)Tq * Hq * 4) + sink_sums(cut, (int)Hkv, (int)D, sink_places(cut, Tq), 0) * 4;
}

bl_status bl_attn_backward(const void *do_, const void *q, const void *k, const void *v, const void *o,
                           const float *lse, int64_t do_stride, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                           const int32_t *cu_q, const int32_t *cu_k, int64_t B, int64_t max_q, int64_t max_k,
                           int64_t window, int64_t sinks, float scale, void *workspace, size_t workspace_bytes,
                           void *dq, void *dk, void *dv, bl_stream_t stream) {
    RaggedParams P;
    bl_status rc = ragged_params(&P, q, k, v, q_stride, k_stride, v_stride, Tq, Tk, Hq, Hkv, D, cu_q, cu_k, B, max_q,
                                 max_k, window, sinks, scale);
    if (rc) return rc;
    if (!do_ || !o || !lse || !dq || !dk || !dv) return BL_ERR_NULL;
    if ((rc = check_rows(do_, do_stride, Hq * D, 2))) return rc;
    if (!aligned16(o) || !aligned4(lse) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv)) return BL_ERR_ALIGN;
    if (!workspace || workspace_bytes < bl_attn_backward_workspace_bytes(Tq, Tk, Hq, Hkv, D, B, max_q, max_k, window, sinks))
        return BL_ERR_WORKSPACE;
    if (!aligned16(workspace)) return BL_ERR_ALIGN;
    P.dout = reinterpret_cast<const uint16_t *>(do_);
    P.do_stride = do_stride;
    P.o = reinterpret_cast<uint16_t *>(const_cast<void *>(o));
    P.lse = const_cast<float *>(lse);
    P.dq = reinterpret_cast<uint16_t *>(dq);
    P.dk = reinterpret_cast<uint16_t *>(dk);
    P.dv = reinterpret_cast<uint16_t *>(dv);
    float *delta = reinterpret_cast<float *>(workspace);
    P.delta = delta;
    AttnDevice *d;
    if ((rc = attn_device(&d))) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    RaggedMaps maps;
    memset(&maps, 0, sizeof(maps));
    if (!head_map(&maps.q, q, Tq, Hq, D, q_stride) || !head_map(&maps.k, k, Tk, Hkv, D, k_stride) ||
        !head_map(&maps.v, v, Tk, Hkv, D, v_stride) || !head_map(&maps.dout, do_, Tq, Hq, D, do_stride))
        return BL_ERR_CUDA;
    const DkvCut cut = dkv_cut(P.max_q, P.max_k, P.window, P.sinks);
    float *sums = delta + align256((size_t)Tq * Hq * 4) / 4;
    const dim3 gq((unsigned)((P.max_q + 127) / 128), (unsigned)Hq, (unsigned)B);
    const dim3 gk((unsigned)(cut.tiles + cut.sink_tiles * cut.pieces), (unsigned)Hkv, (unsigned)B);
    // dQ first: it leaves delta for dK
    if (D <= 64) {
        k_attn_dq_tc<64><<<gq, AB_THREADS, DqShape<64>::SMEM, st>>>(maps, P, delta);
        k_attn_dkdv_tc<64><<<gk, AB_THREADS, DkvShape<64>::SMEM, st>>>(maps, P, cut, sums);
    } else {
        k_attn_dq_tc<128><<<gq, AB_THREADS, DqShape<128>::SMEM, st>>>(maps, P, delta);
        k_attn_dkdv_tc<128><<<gk, AB_THREADS, DkvShape<128>::SMEM, st>>>(maps, P, cut, sums);
    }
    if (cut.sink_tiles > 0)
        k_attn_sink_sum<<<dim3((unsigned)(cut.sink_tiles * AB_SUM_CTAS), (unsigned)Hkv, (unsigned)B), 256, 0, st>>>(P, cut, sums);
    return cudaGetLastError() == cudaSuccess ? BL_OK : BL_ERR_CUDA;
}

}  // extern "C"
