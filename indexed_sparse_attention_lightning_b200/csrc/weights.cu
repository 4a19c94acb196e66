// weights.cu -- attention weight received by cache positions, summed over the
// heads and queries of a step and added to per-sequence running sums.
//
// For query t and its selected rows s (the attention's own selection and lse):
//     w[t,s] = sum_h exp(sm_scale * q[t,h,:] . kv[s,:] - lse[t,h])
//     acc_out[b,s] = decay * acc_in[b,s] + sum_{t of b} w[t,s]
// Three kernels: rows (each query's selection as physical rows and positions),
// weights (one fp32 w per selected entry) and sum.  Sums over queries are taken
// in the order of t without atomics between CTAs, so results are reproducible:
// in the sum kernel each warp owns a range of one sequence's positions, keeps
// its sums in shared memory and walks the queries in order.
#include "common.cuh"
#include "internal.h"

namespace sa {
namespace {

constexpr int kTile = 64;  // selected entries per tile: rows are padded to it

// ------------------------------------------------------------------- rows ---
constexpr int kRowsThreads = 512;
__global__ void __launch_bounds__(kRowsThreads)
weights_rows_kernel(const PathParams p, const int32_t *__restrict__ idx, int32_t K, int32_t ld,
                    int32_t *rows, int32_t *kept, int32_t *n_valid, int32_t *ascending) {
    pdl_wait();
    pdl_trigger();
    __shared__ int32_t scratch[33];
    __shared__ int32_t n_s;
    const int t = blockIdx.x;
    int32_t *pos = kept + (int64_t)t * ld;
    compact_rows(p, t, idx + (int64_t)t * K, K, kTile, rows + (int64_t)t * ld, &n_s, scratch, pos);
    __syncthreads();
    const int32_t n = n_s;
    int32_t falls = 0;
    for (int32_t i = threadIdx.x; i + 1 < n; i += kRowsThreads) falls |= pos[i] > pos[i + 1];
    falls = __syncthreads_or(falls);
    if (threadIdx.x == 0) {
        n_valid[t] = n;
        ascending[t] = !falls;
    }
}

// ---------------------------------------------------- weights, any shape ---
// One CTA per 32 selected rows of a query: the rows are staged once, the heads
// pass by eight at a time (one warp each, one row per lane).
constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 32;
constexpr int kSimtHeads = kSimtThreads / 32;

__device__ __forceinline__ float load_q(const PathParams &p, int64_t i) {
    if (p.q_dtype == SA_BF16) return bf16_bits_to_float(static_cast<const uint16_t *>(p.q)[i]);
    return static_cast<const float *>(p.q)[i];
}

__global__ void __launch_bounds__(kSimtThreads)
weights_simt_kernel(const PathParams p, const float *__restrict__ lse, int32_t ld,
                    const int32_t *__restrict__ rows, const int32_t *__restrict__ n_valid,
                    float *__restrict__ w) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ float smem[];
    const int D = p.d_latent + p.d_rope, ldr = D + 1;
    float *rows_s = smem;                     // [kSimtRows][D + 1]
    float *q_s = rows_s + kSimtRows * ldr;    // [kSimtHeads][D]
    float *sum_s = q_s + kSimtHeads * D;      // [kSimtHeads][kSimtRows]
    const int t = blockIdx.y, tid = threadIdx.x, lane = tid & 31, hw = tid >> 5;
    const int32_t k0 = blockIdx.x * kSimtRows, n = n_valid[t];
    if (k0 >= n) return;
    for (int e = tid; e < kSimtRows * D; e += kSimtThreads) {
        const int r = e / D, dd = e - r * D;
        rows_s[r * ldr + dd] =
            k0 + r < n ? kv_value(p, rows[(int64_t)t * ld + k0 + r], dd) : 0.0f;
    }
    float sum = 0.0f;
    for (int h0 = 0; h0 < p.heads; h0 += kSimtHeads) {
        const int hn = min(kSimtHeads, p.heads - h0);
        __syncthreads();
        for (int i = tid; i < hn * D; i += kSimtThreads)
            q_s[i] = load_q(p, ((int64_t)t * p.heads + h0) * D + i);
        __syncthreads();
        if (hw < hn) {
            float dot = 0.0f;
            for (int dd = 0; dd < D; ++dd) dot = fmaf(q_s[hw * D + dd], rows_s[lane * ldr + dd], dot);
            const float l = lse[(int64_t)t * p.heads + h0 + hw];
            if (l != -INFINITY) sum += expf(p.sm_scale * dot - l);
        }
    }
    sum_s[hw * kSimtRows + lane] = sum;
    __syncthreads();
    if (hw == 0 && k0 + lane < n) {
        for (int i = 1; i < kSimtHeads; ++i) sum += sum_s[i * kSimtRows + lane];
        w[(int64_t)t * ld + k0 + lane] = sum;
    }
}

// -------------------------------------------------------------------- sum ---
constexpr int kSumWarps = 8;
constexpr int kSumRange = 512;  // positions per warp

// First entry of pos[0, n) (ascending) that is >= v.
__device__ __forceinline__ int32_t lower_bound(const int32_t *pos, int32_t n, int32_t v) {
    int32_t lo = 0, hi = n;
    while (lo < hi) {
        const int32_t mid = (lo + hi) >> 1;
        if (pos[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(32 * kSumWarps)
weights_sum_kernel(const PathParams p, int32_t chunks, int32_t limit, int32_t ld,
                   const int32_t *__restrict__ kept, const int32_t *__restrict__ n_valid,
                   const int32_t *__restrict__ ascending, const float *__restrict__ w,
                   const float *acc_in, float decay, float *acc_out, int64_t ld_acc) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sums[kSumWarps][kSumRange];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t b = (int32_t)(blockIdx.x / chunks), c = (int32_t)(blockIdx.x % chunks);
    int32_t len = p.seq_len[b];
    if (len > limit) {
        if (c == 0 && threadIdx.x == 0)
            report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_POSITION);
        len = limit;
    }
    const int64_t p0 = ((int64_t)c * kSumWarps + warp) * kSumRange;
    if (p0 >= len) return;
    const int32_t lo = (int32_t)p0, hi = (int32_t)min((int64_t)len, p0 + kSumRange);
    float *s = sums[warp];
    for (int i = lane; i < kSumRange; i += 32) s[i] = 0.0f;
    __syncwarp();
    for (int32_t t0 = 0; t0 < p.n_q; t0 += 32) {
        // lane l looks query t0 + l up: its entries [k0, k1) may fall in the range
        const int32_t t = t0 + lane;
        int32_t k0 = 0, k1 = 0;
        if (t < p.n_q && p.q_seq[t] == b) {
            k1 = n_valid[t];
            if (ascending[t]) {
                const int32_t *pos = kept + (int64_t)t * ld;
                const int32_t n = k1;
                k0 = lower_bound(pos, n, lo);
                k1 = k0 + lower_bound(pos + k0, n - k0, hi);
            }
        }
        uint32_t todo = __ballot_sync(0xffffffffu, k1 > k0);
        while (todo != 0) {
            const int u = __ffs(todo) - 1;
            todo &= todo - 1;
            const int32_t e0 = __shfl_sync(0xffffffffu, k0, u);
            const int32_t e1 = __shfl_sync(0xffffffffu, k1, u);
            const int64_t row = (int64_t)(t0 + u) * ld;
            for (int32_t k = e0 + lane; k < e1; k += 32) {
                const int32_t at = kept[row + k];
                // an entry that occurs twice in a query adds the same weight
                // twice: the order of the two does not matter
                if (at >= lo && at < hi) atomicAdd(&s[at - lo], w[row + k]);
            }
            __syncwarp();
        }
    }
    const int64_t base = (int64_t)b * ld_acc;
    for (int32_t i = lo + lane; i < hi; i += 32) {
        const float old = acc_in != nullptr ? decay * acc_in[base + i] : 0.0f;
        acc_out[base + i] = old + s[i - lo];
    }
}

}  // namespace

int32_t weights_ld(int32_t top_k) { return (int32_t)round_up(top_k > 0 ? top_k : 1, kTile); }

cudaError_t launch_accumulate_weights(const PathParams &p, const int32_t *idx, int32_t top_k,
                                      const float *lse, const float *acc_in, float decay,
                                      float *acc_out, int64_t ld_acc, int32_t *rows,
                                      int32_t *kept, int32_t *n_valid, int32_t *ascending,
                                      float *w, cudaStream_t s) {
    const int32_t ld = weights_ld(top_k);
    cudaError_t e;
    if (p.n_q > 0) {
        count_launch();
        e = launch_pdl(weights_rows_kernel, dim3((unsigned)p.n_q), dim3(kRowsThreads), 0, s, p, idx,
                       top_k, ld, rows, kept, n_valid, ascending);
        if (e != cudaSuccess) return e;
        const int D = p.d_latent + p.d_rope;
        const size_t smem = sizeof(float) * ((size_t)kSimtRows * (D + 1) + (size_t)kSimtHeads * D +
                                             kSimtHeads * kSimtRows);
        e = cudaFuncSetAttribute(weights_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem);
        if (e != cudaSuccess) return e;
        count_launch();
        e = launch_pdl(weights_simt_kernel, dim3((unsigned)(ld / kSimtRows), (unsigned)p.n_q),
                       dim3(kSimtThreads), smem, s, p, lse, ld, (const int32_t *)rows,
                       (const int32_t *)n_valid, w);
        if (e != cudaSuccess) return e;
    }
    const int64_t limit = std::min(ld_acc, (int64_t)p.max_pages * 64);
    const int64_t chunks = ceil_div(limit, kSumWarps * kSumRange);
    count_launch();
    return launch_pdl(weights_sum_kernel, dim3((unsigned)(chunks * p.batch)), dim3(32 * kSumWarps),
                      0, s, p, (int32_t)chunks, (int32_t)limit, ld, (const int32_t *)kept,
                      (const int32_t *)n_valid, (const int32_t *)ascending, (const float *)w,
                      acc_in, decay, acc_out, ld_acc);
}

}  // namespace sa
