// internal.h -- parameter blocks and launchers shared between the host API
// (sa_api.cu) and the kernel files.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "sa.h"

namespace sa {

// Launches `kernel` with programmatic stream serialization, so that its
// launch overlaps the tail of the previous kernel in the stream (the kernel
// itself calls pdl_wait before touching anything that kernel wrote).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t s, Args &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Lets `kernel` be launched with up to `most` bytes of dynamic shared memory.  The
// limit belongs to the function on the device, not to a launch or a host thread:
// a kernel whose launches differ in size always gets its largest, or one thread's
// smaller limit would have another's launch refused.
template <typename... KArgs>
cudaError_t allow_smem(void (*kernel)(KArgs...), size_t most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

// Limits of the shapes that the host checks let through.
constexpr int kMaxLatent = 512, kMaxRow = 1024;  // d_latent, d_latent + d_rope
constexpr int kMaxIndexHeads = 128, kMaxIndexDim = 256;

// Everything a kernel needs to know about the paged caches and the queries.
struct PathParams {
    // paging
    const int32_t *page_table;
    const int32_t *seq_len;
    int32_t batch, max_pages, num_pages;
    // indexer keys
    const void *k_index;
    const float *k_index_scale;
    int32_t d_index;
    int32_t index_dtype;  // sa_dtype: SA_E4M3, SA_BF16 (unscaled) or SA_F32
    // latent cache
    const void *kv;
    const void *kv_rope;
    const float *kv_scale;
    int32_t d_latent, d_rope;
    int32_t kv_dtype;  // sa_dtype
    int32_t kv_scale_tokens, kv_scale_dims;  // scale tile (resolved, > 0; 4 bits: 1 x group)
    // queries
    int32_t n_q;
    const int32_t *q_seq, *q_pos;
    int32_t max_visible;
    const void *q_index;
    const float *q_index_scale;
    const float *w;
    int32_t h_index;
    const void *q;
    int32_t q_dtype;  // sa_dtype
    int32_t heads;
    float sm_scale;
    int32_t q_group;  // queries in runs of this many of one sequence (4: chunked prefill)
    // status word (first 2 ints of the workspace)
    int32_t *status;
};

// Visible length of query t after validating its sequence and position
// against the cache; returns 0 (and reports) for an invalid query.
__device__ __forceinline__ int32_t visible_len(const PathParams &p, int32_t t);

// Count one kernel launch (see sa_kernel_launches).
void count_launch();

// SM count of the current device (cached).
int num_sms();

// 2-D TMA tensor map over a row-major [outer, inner] array (elements of
// dtype_bytes = 1 (u8), 2 (bf16) or 4 (f32)), box [box_outer, box_inner].
bool encode_tmap_2d(CUtensorMap *map, int dtype_bytes, const void *base, uint64_t inner,
                    uint64_t outer, uint64_t row_stride_bytes, uint32_t box_inner,
                    uint32_t box_outer, bool swizzle128);

// ---- launchers (each returns the launch error, if any) --------------------
// Visible length per query and the inclusive prefix of ceil(V / tile); also
// zeroes `zero_words` 32-bit words at `zero` (histograms and counters) and,
// with `clear_status`, the status word before anything can report into it.
cudaError_t launch_plan(const PathParams &p, int32_t *vis, int32_t *tile_end, int32_t tile,
                        uint32_t *zero, size_t zero_words, bool clear_status, cudaStream_t s,
                        int32_t group = 1);

cudaError_t launch_indexer_simt(const PathParams &p, float *scores, int64_t ld, cudaStream_t s);

// Tensor-core FP8 indexer (e4m3 keys, 64 heads x 128 dims); needs the plan.
// indexer_query_group(p): how many consecutive queries share each key tile
// (4 for flagged chunked prefill with e4m3 keys, else 1); the plan's tile
// prefix must run over groups of that size.
bool indexer_mma_supported(const PathParams &p);
int32_t indexer_query_group(const PathParams &p);
cudaError_t launch_indexer_mma(const PathParams &p, const int32_t *vis, const int32_t *tile_end,
                               float *scores, int64_t ld, uint32_t *hist, cudaStream_t s);

// Row-wise exact top-K.  Row t has valid_len[t] entries, or q_pos[t] + 1 when
// valid_len is null (rows then validated as queries of `p`).
cudaError_t launch_topk_rowwise(const float *scores, int64_t ld, const int32_t *valid_len,
                                int32_t max_valid, const PathParams *p, int32_t n_q,
                                int32_t top_k, int32_t *idx, int32_t *status, cudaStream_t s);

// Histogram-guided exact top-K for rows scored by the tensor-core indexer
// (which filled `hist`, [n_q, kHistBins]).  Scratch: sel [n_q, top_k],
// counts [n_q, kTopkCountsPerQuery] (zeroed), cand [n_q, cap], chunk_info.
constexpr int32_t kTopkCandCap = 8192;
constexpr int32_t kTopkCountsPerQuery = 2;
// Rows longer than this many positions per chunk split into chunks; chunk_info
// [n_q, topk_chunk_slots(ld)] (int4) holds each chunk's list slots.
constexpr int32_t kTopkChunk = 8192;
inline int64_t topk_chunk_slots(int64_t ld) { return (ld + kTopkChunk - 1) / kTopkChunk; }
// With `rows` non-null it also writes the physical cache rows of the
// selection for the tensor-core attention (compact_rows layout, tile 64,
// leading dimension ld_rows) and their count n_valid [n_q].
cudaError_t launch_topk_hist(const float *scores, int64_t ld, const int32_t *vis,
                             const uint32_t *hist, int32_t n_q, int32_t max_valid, int32_t top_k,
                             int32_t *sel, int32_t *counts, uint64_t *cand, int32_t cap,
                             int4 *chunk_info, int32_t *idx, const PathParams &p, int32_t *rows,
                             int32_t ld_rows, int32_t *n_valid, cudaStream_t s);

cudaError_t launch_attn_simt(const PathParams &p, const int32_t *idx, int32_t top_k, void *out,
                             int32_t out_dtype, float *lse, cudaStream_t s);

// Tensor-core sparse attention (bf16 query, 128 heads, 512 + 64 dims, K <= 2048):
// one CTA per 64 heads of a query and key split, over the physical rows of its
// selection: `rows` [n_q, sfa_rows_ld(K)] and n_valid [n_q] from the top-K
// kernel, or, where rows is null, compacted from idx [n_q, K] by each CTA
// itself.  With `splits` > 1 the partial outputs go to o_part [n_q, splits, 128,
// 512] / lse_part [n_q, splits, 128] and a second kernel merges them.
bool sfa_mma_supported(const PathParams &p, int32_t top_k);
int32_t sfa_splits(int32_t n_q, int32_t top_k);
int32_t sfa_rows_ld(int32_t top_k);
cudaError_t launch_sfa_mma(const PathParams &p, const int32_t *idx, int32_t top_k, int32_t splits,
                           const int32_t *rows, const int32_t *n_valid, void *out,
                           int32_t out_dtype, float *lse, float *o_part, float *lse_part,
                           cudaStream_t s);

// Accumulated attention weights (weights.cu).  Each query's selection is compacted
// into physical rows (n_q * weights_lists of them: one per query or per CTA) and kept
// positions (n_valid of them), `starts` notes where each range of positions begins
// in them, w [n_q, weights_ld] takes one weight per kept entry, and the sum kernel
// adds those to the sequences' rows.  Leading dimension of rows, kept and w:
// weights_ld(K); of starts: weights_starts_ld(n_q, batch, max_visible).
int32_t weights_splits(int32_t n_q, int32_t top_k, int32_t kv_dtype);
int32_t weights_lists(int32_t n_q, int32_t top_k, int32_t kv_dtype);
bool weights_rows_first(int32_t n_q, int32_t top_k, int32_t kv_dtype);
int32_t weights_ld(int32_t top_k);
int32_t weights_starts_ld(int32_t n_q, int32_t batch, int32_t max_visible);
cudaError_t launch_accumulate_weights(const PathParams &p, const int32_t *idx, int32_t top_k,
                                      const float *lse, const float *acc_in, float decay,
                                      float *acc_out, int64_t ld_acc, int32_t *rows,
                                      int32_t *kept, int32_t *n_valid, int32_t *starts, float *w,
                                      cudaStream_t s);

// Context-parallel decode steps (cp.cu).
int32_t cp_merge_max_candidates();
int32_t cp_combine_max_parts();
cudaError_t launch_cand_emit(const float *scores, int64_t ld, const int32_t *idx, int32_t n_q,
                             int32_t top_k, const int32_t *offset, float *cand_score,
                             int32_t *cand_pos, cudaStream_t s);
cudaError_t launch_cp_merge(const float *cand_score, const int32_t *cand_pos, int32_t n_ranks,
                            int32_t n_q, int32_t top_k, const int32_t *pos_lo,
                            const int32_t *pos_hi, int32_t *idx_global, int32_t *idx_local,
                            cudaStream_t s);
cudaError_t launch_cp_combine(const float *o_part, const float *lse_part, int32_t n_parts,
                              int64_t rows, int32_t d, void *out, int32_t out_dtype, float *lse,
                              cudaStream_t s);

}  // namespace sa

// ---- inline device definitions -------------------------------------------
#ifdef __CUDACC__
#include "common.cuh"
namespace sa {
__device__ __forceinline__ int32_t visible_len(const PathParams &p, int32_t t) {
    int32_t b = __ldg(p.q_seq + t);
    int32_t pos = __ldg(p.q_pos + t);
    if (b < 0 || b >= p.batch || pos < 0 || pos >= __ldg(p.seq_len + b) ||
        pos >= p.max_visible) {
        report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_POSITION);
        return 0;
    }
    return pos + 1;
}

// Scale of latent dim d of physical row `row` of the e4m3 cache: one fp32 per
// tile of kv_scale_tokens tokens x kv_scale_dims dims of a 64-token page,
// laid out [num_pages, 64 / kv_scale_tokens, d_latent / kv_scale_dims].
__device__ __forceinline__ float kv_scale_at(const PathParams &p, int64_t row, int32_t d) {
    const int64_t page = row >> 6;
    const int32_t tok = static_cast<int32_t>(row & 63);
    const int32_t tiles_t = 64 / p.kv_scale_tokens, tiles_d = p.d_latent / p.kv_scale_dims;
    return __ldg(p.kv_scale + (page * tiles_t + tok / p.kv_scale_tokens) * tiles_d +
                 d / p.kv_scale_dims);
}

// Latent dim or rope dim dd of physical row `row`, as fp32, of a cache of dtype kKv.
template <int kKv>
__device__ __forceinline__ float kv_value_of(const PathParams &p, int64_t row, int dd) {
    const int D = p.d_latent + p.d_rope;
    if constexpr (kKv == SA_F32) return static_cast<const float *>(p.kv)[row * D + dd];
    if constexpr (kKv == SA_BF16)
        return bf16_bits_to_float(static_cast<const uint16_t *>(p.kv)[row * D + dd]);
    if (dd >= p.d_latent)
        return bf16_bits_to_float(
            static_cast<const uint16_t *>(p.kv_rope)[row * p.d_rope + (dd - p.d_latent)]);
    if constexpr (kKv == SA_E4M3) {
        const uint8_t c = static_cast<const uint8_t *>(p.kv)[row * p.d_latent + dd];
        return e4m3x2_to_float2(c).x * kv_scale_at(p, row, dd);
    }
    const uint32_t two = static_cast<const uint8_t *>(p.kv)[(row * p.d_latent + dd) >> 1];
    const uint32_t sb = reinterpret_cast<const uint8_t *>(
        p.kv_scale)[(row * p.d_latent + dd) / fp4_group(kKv)];
    return e2m1x2_to_float2((dd & 1) ? two >> 4 : two & 15u).x * fp4_scale_value(kKv, sb);
}

// f(dtype) with the cache's dtype as a constant: a loop over kv_value_of inside it
// does not look at the dtype for every value (the CUDA-core attention of 8 queries,
// 16 heads and 1000 bf16 rows: 1886 us with a look for each, 1599 without).
template <typename F>
__device__ __forceinline__ void with_kv_dtype(const PathParams &p, F f) {
    switch (p.kv_dtype) {
    case SA_F32: return f(std::integral_constant<int, SA_F32>());
    case SA_BF16: return f(std::integral_constant<int, SA_BF16>());
    case SA_E4M3: return f(std::integral_constant<int, SA_E4M3>());
    case SA_MXFP4: return f(std::integral_constant<int, SA_MXFP4>());
    default: return f(std::integral_constant<int, SA_NVFP4>());
    }
}

// Physical cache rows of query t's selected positions sel[0, K): list order,
// -1 entries dropped, out-of-range positions and bad page ids skipped and
// reported; then padded with the first row up to a multiple of `tile`.
// Writes rows[0, padded) and *n_valid.  Called by every thread of a CTA
// (blockDim.x a multiple of 32); `scratch` is shared memory of 33 ints.
__device__ __forceinline__ void compact_rows(const PathParams &p, int32_t t, const int32_t *sel,
                                             int32_t K, int32_t tile, int32_t *rows,
                                             int32_t *n_valid, int32_t *scratch) {
    const int nwarps = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t V = visible_len(p, t);
    const int32_t seq = __ldg(p.q_seq + t);
    int32_t base = 0;
    for (int32_t r0 = 0; r0 < K; r0 += blockDim.x) {
        const int32_t k = r0 + threadIdx.x;
        const int32_t s = k < K ? sel[k] : -1;
        int32_t v = -1;
        if (s >= V) {
            report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_INDEX);
        } else if (s >= 0) {
            const int64_t row = phys_row(p.page_table, p.max_pages, p.num_pages, seq, s);
            if (row < 0) report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_PAGE);
            else v = static_cast<int32_t>(row);
        }
        const unsigned bal = __ballot_sync(0xffffffffu, v >= 0);
        if (lane == 0) scratch[w] = __popc(bal);
        __syncthreads();
        int32_t off = base, tot = 0;
        for (int i = 0; i < nwarps; ++i) {
            if (i < w) off += scratch[i];
            tot += scratch[i];
        }
        const int32_t pos = off + __popc(bal & ((1u << lane) - 1u));
        if (v >= 0) {
            rows[pos] = v;
            if (pos == 0) scratch[32] = v;
        }
        __syncthreads();
        base += tot;
    }
    const int32_t padded = (base + tile - 1) / tile * tile;
    if (base > 0)
        for (int32_t c = base + threadIdx.x; c < padded; c += blockDim.x) rows[c] = scratch[32];
    if (threadIdx.x == 0) *n_valid = base;
}

// compact_rows with more loads in flight: a thread takes kEntries entries of a
// step, blockDim.x apart, and one scan over the warps' counts places them (2048
// entries by 512 threads, four each: 9 instead of 11 us with cold caches).  With
// `kept` it also writes the positions behind rows[0, *n_valid).  `scratch`:
// kCompactScratch ints; kEntries times the warps of the CTA are at most 128.
// `first`: this thread's entries of the first step, from load_entries before.
constexpr int kCompactScratch = 128 + 2;
template <int kEntries>
__device__ __forceinline__ void load_entries(const int32_t *sel, int32_t K, int64_t r0,
                                             int32_t (&s)[kEntries]) {
#pragma unroll
    for (int j = 0; j < kEntries; ++j) {
        const int64_t k = r0 + j * blockDim.x + threadIdx.x;
        s[j] = k < K ? sel[k] : -1;
    }
}
template <int kEntries>
__device__ __forceinline__ void compact_selection(const PathParams &p, int32_t t,
                                                  const int32_t *sel, int32_t K, int32_t tile,
                                                  int32_t *rows, int32_t *n_valid,
                                                  int32_t *scratch, int32_t (&first)[kEntries],
                                                  int32_t *kept = nullptr) {
    const int nwarps = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t seq = __ldg(p.q_seq + t);
    const bool seq_ok = seq >= 0 && seq < p.batch;
    int32_t V = -1;  // known after the first loads are on their way
    int32_t base = 0;
    for (int64_t r0 = 0; r0 < K; r0 += kEntries * blockDim.x) {
        int32_t (&s)[kEntries] = first, v[kEntries];
        if (r0 > 0) load_entries(sel, K, r0, s);
#pragma unroll
        for (int j = 0; j < kEntries; ++j) {
            v[j] = -1;
            if (s[j] >= 0 && seq_ok)
                v[j] = static_cast<int32_t>(
                    phys_row(p.page_table, p.max_pages, p.num_pages, seq, s[j]));
        }
        if (V < 0) V = visible_len(p, t);
        unsigned bal[kEntries];
#pragma unroll
        for (int j = 0; j < kEntries; ++j) {
            if (s[j] >= V) {
                report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_INDEX);
                v[j] = -1;
            } else if (s[j] >= 0 && v[j] < 0) {
                report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_PAGE);
            }
            bal[j] = __ballot_sync(0xffffffffu, v[j] >= 0);
            if (lane == 0) scratch[j * nwarps + w] = __popc(bal[j]);
        }
        __syncthreads();
        if (w == 0) {  // exclusive scan of the counts, four per lane
            const int counts = kEntries * nwarps;
            int32_t c[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = 4 * lane + i < counts ? scratch[4 * lane + i] : 0;
                sum += c[i];
            }
            int32_t inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            int32_t at = inc - sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * lane + i < counts) scratch[4 * lane + i] = at;
                at += c[i];
            }
            if (lane == 31) scratch[128] = inc;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEntries; ++j) {
            if (v[j] >= 0) {
                const int32_t pos =
                    base + scratch[j * nwarps + w] + __popc(bal[j] & ((1u << lane) - 1u));
                rows[pos] = v[j];
                if (kept != nullptr) kept[pos] = s[j];
                if (pos == 0) scratch[129] = v[j];
            }
        }
        base += scratch[128];
        __syncthreads();
    }
    const int32_t padded = (base + tile - 1) / tile * tile;
    if (base > 0)
        for (int32_t c = base + threadIdx.x; c < padded; c += blockDim.x) rows[c] = scratch[129];
    if (threadIdx.x == 0) *n_valid = base;
}
}  // namespace sa
#endif
