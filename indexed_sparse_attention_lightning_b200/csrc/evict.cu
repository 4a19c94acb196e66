// evict.cu -- shrinking a paged cache to a budget of tokens per sequence by
// the attention weight that its positions accumulated.
//
// Of a sequence of n > budget tokens the first F, the last R and, between
// them, the budget - F - R positions with the largest acc stay (ties to the
// lower position).  Two kernels:
//   select  one CTA, or a cluster of up to sixteen, per sequence: its positions'
//           acc in shared memory where they fit, the threshold of the middle
//           part by an exact radix select on order-preserving keys (four 8-bit
//           digits; the CTAs' histograms are added through distributed shared
//           memory), then the kept positions in ascending order with their
//           physical rows;
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
constexpr int kSelectBins = 256;
constexpr int kSelectCopies = 8;  // of a histogram, so that equal digits collide less
constexpr int kSelectStep = 128;  // positions of a warp at a time: four per lane
// Keys of a CTA kept in shared memory: 48K of them; longer sequences are read
// again in every pass.
constexpr int64_t kSelectCached = 48 * 1024;
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
    int32_t *fault;    // [batch]: SA_DETAIL_* of a skipped sequence, or 0
    int32_t *status;   // written by the move kernel, from `fault`
};

// One pool's rows: `units` pieces of `unit` bytes (16, 4, 2 or 1).
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

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// A word of shared memory of the cluster's CTA `rank`, at this CTA's address `p`.
__device__ __forceinline__ int32_t peer_word(const int32_t *p, int rank) {
    uint32_t at;
    int32_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// The sum of such a word over CTAs [0, n) of the cluster of `ctas`, eight loads
// in flight.
__device__ __forceinline__ int32_t peer_sum(const int32_t *p, int n, int ctas) {
    int32_t sum = 0;
    for (int r0 = 0; r0 < n; r0 += 8) {
        int32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = peer_word(p, min(r0 + i, ctas - 1));
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += r0 + i < n ? v[i] : 0;
    }
    return sum;
}

// A warp's positions [w0, w1) of a sequence, four consecutive ones per lane and
// step.  keys() gives those of the middle part [lo, hi), and 0, which is no
// value's key, for the others.
template <bool kCached>
struct WarpKeys {
    const float *acc;
    uint32_t *cache;  // the warp's keys
    int32_t w0, w1, lo, hi, lane;

    __device__ __forceinline__ uint4 fresh(int32_t i0) const {
        uint32_t k[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int32_t i = i0 + 4 * lane + e;
            k[e] = i >= lo && i < min(hi, w1) ? keep_key(acc[i]) : 0u;
        }
        return make_uint4(k[0], k[1], k[2], k[3]);
    }
    __device__ __forceinline__ void fill() const {
        if constexpr (kCached) {
#pragma unroll 4
            for (int32_t i0 = w0; i0 < w1; i0 += kSelectStep)
                reinterpret_cast<uint4 *>(cache + (i0 - w0))[lane] = fresh(i0);
        }
    }
    __device__ __forceinline__ uint4 keys(int32_t i0) const {
        if constexpr (kCached) return reinterpret_cast<const uint4 *>(cache + (i0 - w0))[lane];
        else return fresh(i0);
    }
    // f(key) for every position of the middle part
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 4
        for (int32_t i0 = w0; i0 < w1; i0 += kSelectStep) {
            const uint4 k = keys(i0);
            f(k.x);
            f(k.y);
            f(k.z);
            f(k.w);
        }
    }
};

// ctas: CTAs of a sequence's cluster.  cache_per: keys of a warp in the dynamic
// shared memory.
template <bool kCached>
__global__ void __launch_bounds__(kSelectThreads, 1)
evict_select_kernel(const EvictArgs a, int32_t ctas, int32_t cache_per) {
    pdl_trigger();
    extern __shared__ uint4 cache[];
    __shared__ int32_t copies[kSelectCopies][kSelectBins];
    __shared__ int32_t hist[4][kSelectBins];
    __shared__ int32_t scan[kSelectWarps];
    __shared__ int32_t gt_s[kSelectWarps], eq_s[kSelectWarps];
    __shared__ int32_t totals[2];  // this CTA's entries above the threshold, and on it
    __shared__ int32_t pick[2];
    const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t n = a.src_len[b];
    const float *acc = a.acc + (int64_t)b * a.ld_acc;
    const int32_t *st = a.src_table + (int64_t)b * a.src_max_pages;
    const int32_t *dt = a.dst_table + (int64_t)b * a.dst_max_pages;
    const int64_t out0 = (int64_t)b * a.budget;
    for (int i = tid; i < kSelectCopies * kSelectBins; i += kSelectThreads) (&copies[0][0])[i] = 0;

    // every CTA checks the whole sequence, so that all take the same way
    const bool fits = n >= 0 && n <= (int64_t)a.src_max_pages * 64 && n <= a.ld_acc;
    int32_t bad = 0;
    if (fits) {
        const int32_t kept = min(n, a.budget);
        for (int32_t i = tid; i < (n + 63) / 64; i += kSelectThreads)
            bad |= st[i] < 0 || st[i] >= a.src_pages;
        for (int32_t i = tid; i < (kept + 63) / 64; i += kSelectThreads)
            bad |= dt[i] < 0 || dt[i] >= a.dst_pages;
    }
    // the middle part [lo, hi) keeps its `want` largest keys: all above the
    // threshold and the first `ties` on it
    const bool shrink = fits && n > a.budget;
    const int32_t lo = shrink ? a.first : 0, hi = shrink ? n - a.last : 0;
    const int32_t want = shrink ? a.budget - a.first - a.last : 0;
    // this warp's positions: whole steps of the sequence
    const int32_t span = fits ? n : 0;
    const int64_t per = round_up(ceil_div(span, ctas * kSelectWarps), kSelectStep);
    const int64_t begin = (rank * kSelectWarps + warp) * per;
    const WarpKeys<kCached> mine{
        acc, reinterpret_cast<uint32_t *>(cache) + (int64_t)warp * cache_per,
        (int32_t)min(begin, (int64_t)span), (int32_t)min(begin + per, (int64_t)span), lo, hi, lane};
    if (want > 0) mine.fill();
    bad = __syncthreads_or(bad);
    if (tid == 0 && rank == 0)
        a.fault[b] = !fits ? SA_DETAIL_BAD_POSITION : bad ? SA_DETAIL_BAD_PAGE : SA_DETAIL_NONE;
    const int32_t kept = bad ? 0 : min(span, a.budget);

    uint32_t threshold = 0xFFFFFFFFu;
    int32_t ties = 0;
    if (want > 0 && !bad) {
        const uint32_t zero_key = keep_key(0.0f);
        uint32_t prefix = 0, mask = 0;
        int32_t left = want;
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            int32_t *h = copies[lane & (kSelectCopies - 1)];
            // positions that never received weight share one key: they are
            // counted in registers, not by colliding atomics
            int32_t zeros = 0;
            mine.each([&](uint32_t k) {
                if (k == zero_key) ++zeros;
                else if (k != 0u && (k & mask) == prefix) atomicAdd(&h[(k >> shift) & 255u], 1);
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) zeros += __shfl_xor_sync(0xffffffffu, zeros, o);
            if (lane == 0 && (zero_key & mask) == prefix && zeros > 0)
                atomicAdd(&h[(zero_key >> shift) & 255u], zeros);
            __syncthreads();
            if (tid < kSelectBins) {
                int32_t sum = 0;
#pragma unroll
                for (int c = 0; c < kSelectCopies; ++c) {
                    sum += copies[c][tid];
                    copies[c][tid] = 0;
                }
                hist[pass][tid] = sum;
            }
            if (ctas > 1) cluster_sync();
            else __syncthreads();
            // the sequence's histogram, one bin a thread from the top, and the bin
            // in which the `left`-th largest key lies
            int32_t count = 0, inc = 0;
            if (tid < kSelectBins) {
                const int32_t *d = &hist[pass][kSelectBins - 1 - tid];
                count = ctas == 1 ? *d : peer_sum(d, ctas, ctas);
                inc = count;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int32_t up = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += up;
                }
                if (lane == 31) scan[warp] = inc;
            }
            __syncthreads();
            if (tid < kSelectBins) {
                int32_t above = inc - count;
                for (int w = 0; w < warp; ++w) above += scan[w];
                if (above < left && left <= above + count) {
                    pick[0] = kSelectBins - 1 - tid;
                    pick[1] = above;
                }
            }
            __syncthreads();
            prefix |= (uint32_t)pick[0] << shift;
            mask |= 255u << shift;
            left -= pick[1];
            __syncthreads();  // scan and pick are written again
        }
        threshold = prefix;
        ties = left;
    }

    // entries of each warp that stay for certain, and those on the threshold
    const int32_t w0 = mine.w0, w1 = bad ? mine.w0 : mine.w1;
    int32_t gt = 0, eq = 0;
    if (want > 0 && !bad) {
        mine.each([&](uint32_t k) {
            gt += k > threshold;
            eq += k == threshold;
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            gt += __shfl_xor_sync(0xffffffffu, gt, o);
            eq += __shfl_xor_sync(0xffffffffu, eq, o);
        }
    }
    if (lane == 0) {
        // and the first and last tokens
        gt_s[warp] = gt + (w1 - w0) - max(0, min(w1, hi) - max(w0, lo));
        eq_s[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {  // exclusive sums over the CTA's warps
        const int32_t g = gt_s[lane], e = eq_s[lane];
        int32_t gi = g, ei = e;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t gu = __shfl_up_sync(0xffffffffu, gi, o);
            const int32_t eu = __shfl_up_sync(0xffffffffu, ei, o);
            if (lane >= o) {
                gi += gu;
                ei += eu;
            }
        }
        gt_s[lane] = gi - g;
        eq_s[lane] = ei - e;
        if (lane == 31) {
            totals[0] = gi;
            totals[1] = ei;
        }
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    int32_t gt_before = gt_s[warp], eq_before = eq_s[warp];
    gt_before += peer_sum(&totals[0], rank, ctas);
    eq_before += peer_sum(&totals[1], rank, ctas);
    if (ctas > 1) cluster_arrive();  // this CTA has read the others' shared memory

    // ascending emission: a warp's entries start behind all earlier ones that stay
    int32_t on = eq_before;                    // entries on the threshold so far
    int32_t slot = gt_before + min(on, ties);  // kept entries so far
    const uint32_t below = (1u << lane) - 1u;
    constexpr int kSteps = 4;  // whose pages and sums are loaded together
    for (int32_t g0 = w0; g0 < w1; g0 += kSteps * kSelectStep) {
        int32_t page[kSteps];
        float sum[kSteps][4];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int32_t i = g0 + u * kSelectStep + 4 * lane;
            page[u] = i < w1 ? __ldg(st + (i >> 6)) : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[u][e] = a.acc_out != nullptr && i + e < w1 ? __ldg(acc + i + e) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int32_t i0 = g0 + u * kSelectStep;
            if (i0 >= w1) break;
            const uint4 k4 = want > 0 ? mine.keys(i0) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
            int32_t rank_on = on;  // entries on the threshold before this lane's
            bool tie[4], keep[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                tie[e] = k[e] != 0u && k[e] == threshold && want > 0;
                const uint32_t bits = __ballot_sync(0xffffffffu, tie[e]);
                rank_on += __popc(bits & below);
                on += __popc(bits);
            }
            int32_t at = slot;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int32_t i = i0 + 4 * lane + e;
                keep[e] = k[e] > threshold || (tie[e] && rank_on < ties) ||
                          (i < w1 && (i < lo || i >= hi));
                rank_on += tie[e];
                const uint32_t bits = __ballot_sync(0xffffffffu, keep[e]);
                at += __popc(bits & below);
                slot += __popc(bits);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!keep[e]) continue;
                const int32_t i = i0 + 4 * lane + e;
                a.src_row[out0 + at] = page[u] * 64 + (i & 63);
                if (a.src_pos != nullptr) a.src_pos[out0 + at] = i;
                if (a.acc_out != nullptr) a.acc_out[(int64_t)b * a.ld_out + at] = sum[u][e];
                ++at;
            }
        }
    }
    const int32_t first = rank * kSelectThreads + tid;
    if (a.src_pos != nullptr)
        for (int64_t i = (int64_t)kept + first; i < a.budget; i += ctas * kSelectThreads)
            a.src_pos[out0 + i] = -1;
    if (a.acc_out != nullptr)
        for (int64_t i = (int64_t)kept + first; i < a.ld_out; i += ctas * kSelectThreads)
            a.acc_out[(int64_t)b * a.ld_out + i] = 0.0f;
    if (first == 0) {
        a.kept[b] = kept;
        a.dst_len[b] = kept;
    }
    __syncwarp();
    if (ctas > 1) cluster_wait();  // no CTA leaves while another reads its shared memory
}

// blockIdx.y: the sequence.  One warp moves `rows` consecutive kept tokens at a
// time.  The 16-byte pieces of all their rows in all pools are dealt to the
// lanes, at most kMovePieces each, and all loads are in flight before the first
// store; the next tokens' places are looked up meanwhile.
//
// Many warps with few pieces each, in one wave: 64 sequences to 4096 bf16 tokens
// (682 MB read and written) take 128 us with 3 pieces and 4 CTAs per SM, 5.3
// TB/s; 145 with 8 and 2, 146 with 5 and 4, 150 with 3 and 6, and 142 with 3 and
// as many waves as it takes.  Longer rows (over 96 pieces: fp32) take 10 pieces.
template <int kMovePieces, int kMoveCtas>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas)
evict_move_kernel(const EvictArgs a, const EvictFields fields, int32_t pieces, int32_t rows) {
    const int lane = threadIdx.x & 31;
    // this lane's pieces: token of the group (none: 32), and where the piece lies
    // in a pool's first row
    int32_t token[kMovePieces], row_bytes[kMovePieces];
    const uint8_t *src[kMovePieces];
    uint8_t *dst[kMovePieces];
#pragma unroll
    for (int j = 0; j < kMovePieces; ++j) {
        const int32_t q = lane + 32 * j;
        int32_t piece = q % pieces;
        token[j] = 32;
        row_bytes[j] = 0;
        src[j] = nullptr;
        dst[j] = nullptr;
#pragma unroll
        for (int k = 0; k < kMaxFields; ++k) {
            if (k >= fields.n || fields.f[k].unit != 16) continue;
            if (piece >= 0 && piece < fields.f[k].units && q / pieces < rows) {
                token[j] = q / pieces;
                row_bytes[j] = 16 * fields.f[k].units;
                src[j] = fields.f[k].src + 16 * piece;
                dst[j] = fields.f[k].dst + 16 * piece;
            }
            piece -= fields.f[k].units;
        }
    }
    pdl_wait();
    const int32_t b = blockIdx.y, kept = a.kept[b];
    // the status word: the first skipped sequence's fault
    if (blockIdx.x == 0 && b == 0 && threadIdx.x < 32) {
        int32_t first = a.batch;
        for (int32_t i = lane; i < a.batch && first == a.batch; i += 32)
            if (a.fault[i] != SA_DETAIL_NONE) first = i;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        if (lane == 0) {
            a.status[0] = first < a.batch ? SA_ERR_DEVICE_FAULT : SA_OK;
            a.status[1] = first < a.batch ? a.fault[first] : SA_DETAIL_NONE;
        }
    }
    const int32_t *row_of = a.src_row + (int64_t)b * a.budget;
    const int32_t *table = a.dst_table + (int64_t)b * a.dst_max_pages;
    // kept places are below 2^31, those that a step leads to may be above
    const uint32_t end = kept, step = gridDim.x * (kMoveThreads / 32) * rows;
    // lane r looks token r of a group up
    auto places = [&](uint32_t i0, int32_t &from, int32_t &to) {
        const uint32_t i = i0 + lane;
        from = to = 0;
        if (lane >= rows || i >= end) return;
        from = row_of[i];
        to = table[i >> 6] * 64 + (i & 63);
    };
    int32_t from, to;
    uint32_t i0 = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * rows;
    places(i0, from, to);
    for (; i0 < end; i0 += step) {
        const int32_t n = min((uint32_t)rows, end - i0);
        uint4 x[kMovePieces];
#pragma unroll
        for (int j = 0; j < kMovePieces; ++j) {
            const int64_t r = __shfl_sync(0xffffffffu, from, token[j] & 31);
            if (token[j] < n)
                x[j] = __ldcs(reinterpret_cast<const uint4 *>(src[j] + r * row_bytes[j]));
        }
        int32_t from1, to1;
        places(i0 + step, from1, to1);
#pragma unroll
        for (int j = 0; j < kMovePieces; ++j) {
            const int64_t r = __shfl_sync(0xffffffffu, to, token[j] & 31);
            if (token[j] < n) __stcs(reinterpret_cast<uint4 *>(dst[j] + r * row_bytes[j]), x[j]);
        }
        // rows that are not whole 16-byte pieces: a few small units each
#pragma unroll
        for (int k = 0; k < kMaxFields; ++k) {
            if (k >= fields.n || fields.f[k].unit == 16) continue;
            const EvictField &f = fields.f[k];
            for (int32_t u0 = 0; u0 < n * f.units; u0 += 32) {
                const int32_t u = u0 + lane, r = u / f.units, c = u % f.units;
                const int64_t s = (int64_t)__shfl_sync(0xffffffffu, from, r & 31) * f.units + c;
                const int64_t d = (int64_t)__shfl_sync(0xffffffffu, to, r & 31) * f.units + c;
                if (r >= n) continue;
                if (f.unit == 4)
                    reinterpret_cast<uint32_t *>(f.dst)[d] =
                        reinterpret_cast<const uint32_t *>(f.src)[s];
                else if (f.unit == 2)
                    reinterpret_cast<uint16_t *>(f.dst)[d] =
                        reinterpret_cast<const uint16_t *>(f.src)[s];
                else
                    f.dst[d] = f.src[s];
            }
        }
        from = from1;
        to = to1;
    }
}

// The unit divides the row and both pools' addresses (the fp32 scales of an e4m3
// latent may start at any float).
void add_field(EvictFields &fs, const void *src, const void *dst, int64_t row_bytes) {
    if (row_bytes <= 0) return;
    const uintptr_t all = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) |
                          static_cast<uintptr_t>(row_bytes);
    const int32_t unit = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
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

template <int kMovePieces, int kMoveCtas>
cudaError_t launch_move(const EvictArgs &a, const EvictFields &fields, int32_t pieces,
                        cudaStream_t s) {
    const int32_t rows = std::min(32, std::max(1, 32 * kMovePieces / pieces));
    const int64_t groups = ceil_div(ceil_div(a.budget, rows), kMoveThreads / 32);
    const int64_t share = std::max(1, num_sms() * kMoveCtas / a.batch);
    const dim3 grid((unsigned)std::min(groups, share), (unsigned)a.batch);
    count_launch();
    return launch_pdl(evict_move_kernel<kMovePieces, kMoveCtas>, grid, dim3(kMoveThreads), 0, s, a,
                      fields, pieces, rows);
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
    a.fault = a.kept + src->batch;
    a.status = reinterpret_cast<int32_t *>(base);
    // CTAs per sequence: while they fill no more than the GPU, and each has at
    // least 4096 positions (64 sequences of 32K: 159 us with two, 171 with one; 2 of
    // 256K: 54 us with sixteen, 64 with eight)
    const int64_t most = std::min(ld_acc, (int64_t)src->max_pages * 64);
    int32_t ctas = 1;
    while (ctas < 16 && 2 * ctas * src->batch <= num_sms() && 2 * ctas * 4096 <= most) ctas *= 2;
    const int64_t per = round_up(ceil_div(most, ctas * kSelectWarps), kSelectStep);
    const int32_t cache_per = per * kSelectWarps <= kSelectCached ? (int32_t)per : 0;
    const size_t smem = sizeof(uint32_t) * kSelectWarps * (size_t)cache_per;
    const auto select = cache_per > 0 ? evict_select_kernel<true> : evict_select_kernel<false>;
    cudaError_t e =
        cache_per > 0 ? allow_smem(select, sizeof(uint32_t) * kSelectCached) : cudaSuccess;
    if (e == cudaSuccess && ctas > 8)
        e = cudaFuncSetAttribute(select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(src->batch * ctas));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launch();
    e = cudaLaunchKernelEx(&cfg, select, a, ctas, cache_per);
    if (e != cudaSuccess) return e;
    const EvictFields fields = make_fields(src, dst);
    int32_t pieces = 0;
    for (int k = 0; k < fields.n; ++k)
        if (fields.f[k].unit == 16) pieces += fields.f[k].units;
    pieces = std::max(pieces, 1);
    return pieces <= 96 ? launch_move<3, 4>(a, fields, pieces, s)
                        : launch_move<10, 2>(a, fields, pieces, s);
}

}  // namespace sa
