// evict.cu -- shrinking a paged cache to a budget of tokens per sequence by
// the attention weight that its positions accumulated.
//
// Of a sequence of n > budget tokens the first F, the last R and, between
// them, the budget - F - R positions with the largest acc stay (ties to the
// lower position).  Two kernels:
//   select  finds the threshold of the middle part exactly by a radix select on
//           order-preserving keys and lists the kept positions in ascending
//           order with their physical rows;
//   move    copies each kept token's index key, latent row and scales byte for
//           byte to its place in the destination pages.
// Both are bound by memory: select reads acc, move reads and writes the kept
// rows.
#include "evict.h"

#include <algorithm>

#include "internal.h"

namespace sa {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMaxFields = 5;

struct EvictArgs {
    const int32_t *src_table, *src_len;
    const int32_t *dst_table;
    int32_t *dst_len;
    int32_t batch, src_max_pages, src_pages, dst_max_pages, dst_pages;
    const float *acc;
    int64_t ld_acc;
    int32_t budget, first, last;
    float *acc_out;
    int64_t ld_out;
    int32_t *src_pos;  // may be null
    int32_t *src_row;  // [batch, budget]
    int32_t *kept;     // [batch]
    int32_t *status;
};

// One pool's rows: `units` pieces of `unit` bytes (16, 8, 4, 2 or 1).
struct EvictField {
    const uint8_t *src;
    uint8_t *dst;
    int32_t unit, units;
};

struct EvictFields {
    EvictField f[kMaxFields];
    int32_t n;
};

// Larger is kept first; every NaN is the largest.
__device__ __forceinline__ uint32_t keep_key(float a) {
    return a != a ? 0xFFFFFFFFu : order_key(a);
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
    __shared__ int32_t hist[256];
    __shared__ int32_t scratch[2 * kSelectWarps];
    __shared__ int32_t pick[2];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t n = a.src_len[b];
    const float *acc = a.acc + (int64_t)b * a.ld_acc;
    const int32_t *st = a.src_table + (int64_t)b * a.src_max_pages;
    const int32_t *dt = a.dst_table + (int64_t)b * a.dst_max_pages;
    const int64_t out0 = (int64_t)b * a.budget;

    const bool fits = n >= 0 && n <= (int64_t)a.src_max_pages * 64 && n <= a.ld_acc;
    int32_t bad = 0;
    if (fits) {
        const int32_t kept = min(n, a.budget);
        for (int32_t i = tid; i < (n + 63) / 64; i += kSelectThreads)
            bad |= st[i] < 0 || st[i] >= a.src_pages;
        for (int32_t i = tid; i < (kept + 63) / 64; i += kSelectThreads)
            bad |= dt[i] < 0 || dt[i] >= a.dst_pages;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0 && !fits) report(a.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_POSITION);
    if (tid == 0 && bad) report(a.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_PAGE);
    const int32_t len = fits && !bad ? n : 0;
    const int32_t kept = min(len, a.budget);

    // the middle part [lo, hi) keeps its `want` largest keys: all above the
    // threshold and the first `ties` equal to it
    int32_t lo = 0, hi = 0, want = 0;
    if (len > a.budget) {
        lo = a.first;
        hi = len - a.last;
        want = a.budget - a.first - a.last;
    }
    uint32_t threshold = 0xFFFFFFFFu;
    int32_t ties = 0;
    if (want > 0) {
        uint32_t prefix = 0, mask = 0;
        int32_t left = want;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (int32_t i = lo + tid; i < hi; i += kSelectThreads) {
                const uint32_t k = keep_key(acc[i]);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int32_t above = 0, d = 255;
                while (d > 0 && above + hist[d] < left) above += hist[d--];
                pick[0] = d;
                pick[1] = above;
            }
            __syncthreads();
            prefix |= (uint32_t)pick[0] << shift;
            mask |= 255u << shift;
            left -= pick[1];
            __syncthreads();
        }
        threshold = prefix;
        ties = left;
    }

    int32_t at = 0, tied = 0;  // kept and tied entries before this step
    for (int32_t i0 = 0; i0 < len; i0 += kSelectThreads) {
        const int32_t i = i0 + tid;
        bool keep = i < len, tie = false;
        if (keep && i >= lo && i < hi) {
            const uint32_t k = want > 0 ? keep_key(acc[i]) : 0u;
            keep = want > 0 && k > threshold;
            tie = want > 0 && k == threshold;
        }
        const uint32_t tie_bits = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) scratch[warp] = __popc(tie_bits);
        __syncthreads();
        int32_t before = tied, all_ties = 0;
        for (int w = 0; w < kSelectWarps; ++w) {
            if (w < warp) before += scratch[w];
            all_ties += scratch[w];
        }
        if (tie) keep = before + __popc(tie_bits & ((1u << lane) - 1u)) < ties;
        const uint32_t keep_bits = __ballot_sync(0xffffffffu, keep);
        if (lane == 0) scratch[kSelectWarps + warp] = __popc(keep_bits);
        __syncthreads();
        int32_t slot = at, all_keep = 0;
        for (int w = 0; w < kSelectWarps; ++w) {
            if (w < warp) slot += scratch[kSelectWarps + w];
            all_keep += scratch[kSelectWarps + w];
        }
        slot += __popc(keep_bits & ((1u << lane) - 1u));
        if (keep) {
            a.src_row[out0 + slot] = st[i >> 6] * 64 + (i & 63);
            if (a.src_pos != nullptr) a.src_pos[out0 + slot] = i;
            if (a.acc_out != nullptr) a.acc_out[(int64_t)b * a.ld_out + slot] = acc[i];
        }
        at += all_keep;
        tied += all_ties;
        __syncthreads();
    }
    if (a.src_pos != nullptr)
        for (int32_t i = kept + tid; i < a.budget; i += kSelectThreads) a.src_pos[out0 + i] = -1;
    if (a.acc_out != nullptr)
        for (int64_t i = kept + tid; i < a.ld_out; i += kSelectThreads)
            a.acc_out[(int64_t)b * a.ld_out + i] = 0.0f;
    if (tid == 0) {
        a.kept[b] = kept;
        a.dst_len[b] = kept;
    }
}

template <typename T>
__device__ __forceinline__ void move_row(const EvictField &f, int64_t from, int64_t to, int lane) {
    const T *src = reinterpret_cast<const T *>(f.src) + from * f.units;
    T *dst = reinterpret_cast<T *>(f.dst) + to * f.units;
    for (int i = lane; i < f.units; i += 32) dst[i] = src[i];
}

// One warp per kept token (grid-stride).
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const EvictArgs a, const EvictFields fields) {
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.batch * a.budget;
    const int64_t warps = (int64_t)gridDim.x * (kMoveThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); r < rows;
         r += warps) {
        const int32_t b = (int32_t)(r / a.budget), i = (int32_t)(r % a.budget);
        if (i >= a.kept[b]) continue;
        const int64_t from = a.src_row[r];
        const int64_t to =
            (int64_t)a.dst_table[(int64_t)b * a.dst_max_pages + (i >> 6)] * 64 + (i & 63);
        for (int k = 0; k < fields.n; ++k) {
            const EvictField &f = fields.f[k];
            if (f.unit == 16) move_row<uint4>(f, from, to, lane);
            else if (f.unit == 4) move_row<uint32_t>(f, from, to, lane);
            else if (f.unit == 2) move_row<uint16_t>(f, from, to, lane);
            else move_row<uint8_t>(f, from, to, lane);
        }
    }
}

void add_field(EvictFields &fs, const void *src, const void *dst, int64_t row_bytes) {
    if (row_bytes <= 0) return;
    const int32_t unit = row_bytes % 16 == 0 ? 16 : row_bytes % 4 == 0 ? 4 : row_bytes % 2 ? 1 : 2;
    fs.f[fs.n++] = EvictField{static_cast<const uint8_t *>(src),
                              static_cast<uint8_t *>(const_cast<void *>(dst)), unit,
                              (int32_t)(row_bytes / unit)};
}

int64_t elem_bytes(int32_t dtype) {
    return dtype == SA_F32 ? 4 : dtype == SA_BF16 ? 2 : 1;
}

EvictFields make_fields(const sa_cache *s, const sa_cache *d) {
    EvictFields fs{};
    add_field(fs, s->k_index, d->k_index, s->d_index * elem_bytes(s->index_dtype));
    if (s->index_dtype == SA_E4M3) add_field(fs, s->k_index_scale, d->k_index_scale, 4);
    if (s->index_dtype == SA_MXFP8)
        add_field(fs, s->k_index_scale, d->k_index_scale, s->d_index / 32);
    if (s->kv_dtype == SA_F32 || s->kv_dtype == SA_BF16) {
        add_field(fs, s->kv, d->kv, (s->d_latent + s->d_rope) * elem_bytes(s->kv_dtype));
        return fs;
    }
    add_field(fs, s->kv, d->kv, is_fp4(s->kv_dtype) ? s->d_latent / 2 : s->d_latent);
    add_field(fs, s->kv_rope, d->kv_rope, s->d_rope * 2);
    add_field(fs, s->kv_scale, d->kv_scale,
              is_fp4(s->kv_dtype) ? s->d_latent / fp4_group(s->kv_dtype)
                                  : 4 * (s->d_latent / s->kv_scale_dims));
    return fs;
}

}  // namespace

cudaError_t launch_evict(const sa_cache *src, const float *acc, int64_t ld_acc, int32_t budget,
                         int32_t keep_first, int32_t keep_last, const sa_cache *dst,
                         float *acc_out, int64_t ld_out, int32_t *src_pos, void *workspace,
                         cudaStream_t s) {
    char *base = static_cast<char *>(workspace);
    EvictArgs a{};
    a.src_table = src->page_table;
    a.src_len = src->seq_len;
    a.dst_table = dst->page_table;
    // the destination's lengths and pools are caller-owned writable memory
    a.dst_len = const_cast<int32_t *>(dst->seq_len);
    a.batch = src->batch;
    a.src_max_pages = src->max_pages;
    a.src_pages = src->num_pages;
    a.dst_max_pages = dst->max_pages;
    a.dst_pages = dst->num_pages;
    a.acc = acc;
    a.ld_acc = ld_acc;
    a.budget = budget;
    a.first = keep_first;
    a.last = keep_last;
    a.acc_out = acc_out;
    a.ld_out = ld_out;
    a.src_pos = src_pos;
    a.src_row = reinterpret_cast<int32_t *>(base + kStatusBytes);
    a.kept = reinterpret_cast<int32_t *>(base + evict_kept_offset(src->batch, budget));
    a.status = reinterpret_cast<int32_t *>(base);
    count_launch();
    evict_select_kernel<<<src->batch, kSelectThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)src->batch * budget;
    const int64_t grid = std::min<int64_t>((rows + 7) / 8, (int64_t)num_sms() * 32);
    count_launch();
    evict_move_kernel<<<(unsigned)grid, kMoveThreads, 0, s>>>(a, make_fields(src, dst));
    return cudaGetLastError();
}

}  // namespace sa
