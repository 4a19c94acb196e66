// weights.cu -- attention weight received by cache positions, summed over the
// heads and queries of a step and added to per-sequence running sums.
//
// For query t and its selected rows s (the attention's own selection and lse):
//     w[t,s] = sum_h exp(sm_scale * q[t,h,:] . kv[s,:] - lse[t,h])
//     acc_out[b,s] = decay * acc_in[b,s] + sum_{t of b} w[t,s]
// For the attention's production shape two kernels: weights (each query's
// selection as physical rows and positions, then one fp32 w per selected entry, on
// the tensor cores) and sum; a rows kernel in front makes rows and positions for
// very long selections (weights_rows_first) and for the CUDA-core weights kernel
// of other shapes.  Sums over queries are taken in the order of t without
// atomics between CTAs, so results are reproducible: in the sum kernel each warp
// owns a range of one sequence's positions, keeps its sums in shared memory and
// walks the queries in order.
#include "common.cuh"
#include "internal.h"
#include "sfa_gather.cuh"
#include "sm100.cuh"

namespace sa {
namespace {
using namespace sfa;

// The sum kernel's shape: positions per CTA, warps, and queries that a warp looks
// up at a time.
template <int R, int W, int G>
struct SumShape {
    static constexpr int kRange = R, kWarps = W, kGroup = G;
};
// Few queries a sequence (a decode step has one): many small CTAs, one wave of
// them for 64 sequences of 32K.  Many (a prompt's last queries): more warps share
// the queries of a smaller range.
using SumFew = SumShape<1024, 2, 32>;
using SumMany = SumShape<256, 32, 8>;
static_assert(SumFew::kRange == 1 << 10 && SumMany::kRange == 1 << 8, "range_log2 below");
bool sum_many(int32_t n_q, int32_t batch) { return n_q > 16 * (int64_t)batch; }

// ------------------------------------------------------------------- rows ---
// What the sum kernel needs to find a query's entries, from its n kept positions
// (by `count` threads of one CTA): starts[c] = first kept entry at or past position
// c * range (the last column: all of them).  starts[0], which would be 0, is the
// caller's 0, or -1 where the kept positions do not ascend strictly.
__device__ __forceinline__ void write_starts(const int32_t *pos, int32_t n, int32_t *starts,
                                             int32_t ld_starts, int32_t range_log2, int32_t thread,
                                             int32_t count) {
    for (int32_t i = thread; i <= n; i += count) {
        const int32_t at = i < n ? pos[i] : -1, before = i > 0 ? pos[i - 1] : -1;
        if (i > 0 && i < n && before >= at) {
            starts[0] = -1;
            continue;
        }
        const int32_t c0 = i > 0 ? (before >> range_log2) + 1 : 1;
        const int32_t c1 = i < n ? at >> range_log2 : ld_starts - 1;
        for (int32_t c = c0; c <= c1; ++c) starts[c] = i;
    }
}

constexpr int kRowsThreads = 512;
__global__ void __launch_bounds__(kRowsThreads)
weights_rows_kernel(const PathParams p, const int32_t *__restrict__ idx, int32_t K, int32_t ld,
                    int32_t ld_starts, int32_t range_log2, int32_t *rows, int32_t *kept,
                    int32_t *n_valid, int32_t *starts) {
    pdl_wait();
    pdl_trigger();
    __shared__ int32_t scratch[kCompactScratch];
    __shared__ int32_t n_s;
    const int t = blockIdx.x;
    int32_t *pos = kept + (int64_t)t * ld, *st = starts + (int64_t)t * ld_starts;
    const int32_t *sel = idx + (int64_t)t * K;
    int32_t entries[4];
    load_entries(sel, K, 0, entries);
    if (threadIdx.x == 0) st[0] = 0;
    compact_selection(p, t, sel, K, kTile, rows + (int64_t)t * ld, &n_s, scratch, entries, pos);
    __syncthreads();
    write_starts(pos, n_s, st, ld_starts, range_log2, threadIdx.x, kRowsThreads);
    if (threadIdx.x == 0) n_valid[t] = n_s;
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
    with_kv_dtype(p, [&](auto kv) {
        for (int e = tid; e < kSimtRows * D; e += kSimtThreads) {
            const int r = e / D, dd = e - r * D;
            rows_s[r * ldr + dd] =
                k0 + r < n ? kv_value_of<kv.value>(p, rows[(int64_t)t * ld + k0 + r], dd) : 0.0f;
        }
    });
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

cudaError_t launch_weights_simt(const PathParams &p, const float *lse, int32_t ld,
                                const int32_t *rows, const int32_t *n_valid, float *w,
                                cudaStream_t s) {
    const auto bytes = [](size_t D) {
        return sizeof(float) * (kSimtRows * (D + 1) + kSimtHeads * D + kSimtHeads * kSimtRows);
    };
    const size_t smem = bytes(p.d_latent + p.d_rope);
    const cudaError_t e = allow_smem(weights_simt_kernel, bytes(kMaxRow));
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_pdl(weights_simt_kernel, dim3((unsigned)(ld / kSimtRows), (unsigned)p.n_q),
                      dim3(kSimtThreads), smem, s, p, lse, ld, rows, n_valid, w);
}

// ---------------------------------------- weights on the tensor cores ---
// 128 heads x 512 + 64 dims.  One CTA takes all heads of one query and a split
// of its tiles: S = Q K^T with M = 128 heads, N = 64 keys, K = 576, Q in TMEM
// (288 columns), two S buffers behind it.  There is no P V, so a row is gathered
// once per query, and a stage is free again as soon as its S is done.
//   all         turn the query's selection into rows, each CTA for itself while Q
//               is on its way (64 queries 51.6 us, with a kernel in front 53.7; 256
//               queries, two CTAs after one another, 128 and 126.5), unless the rows
//               kernel has (see weights_rows_first);
//   warp 0      lane 0 loads Q by TMA (its halves into ring stages 1 and 2), then
//               the warp issues the MMAs;
//   warps 1-7   gather the rows (sfa_gather.cuh; with warp 12 for a 4-bit latent);
//               those of the query's first CTA then note where each range of
//               positions starts, for the sum kernel;
//   warps 8-11  move Q into TMEM (warp 8 + j: heads 32j .. 32j + 31, one per
//               lane), then read S with 16-lane loads, so that a thread holds
//               four heads of sixteen keys: exp2 of the logits minus the heads'
//               lse, summed over the thread's heads, over the eight lanes of the
//               same keys by halving exchanges (14 shuffles; one head per lane
//               would take 62) and over the four warps through shared memory,
//               all in a fixed order.
// All waits are bounded; a timeout is reported in the workspace status word.
// An e4m3 latent value is code x fp32 scale, 24 significant bits: rounded to one
// bf16 its logits, and with them the fp32 weights, would be off by 2^-9 of
// every product.  Such a row goes into the stage as two: row k the value's
// nearest bf16, row k + 32 the nearest bf16 of what that left (2^-18 is left
// then), and the epilogue adds the two columns; a tile holds 32 keys.  The
// bf16 and 4-bit rows are exact in bf16: 64 keys.
template <int kKv>
constexpr int kKeysOf = kKv == SA_E4M3 ? 32 : kTile;

constexpr int kHeads = 128;
constexpr int kEpiWarp0 = 8;
constexpr uint32_t kWTmemCols = 512;
constexpr uint32_t kWColS = 288;

struct WeightsSmem {
    uint8_t kv[kStages][kStageBytes];
    float part[2][4][kTile];  // per tile parity: each warp's sums over its 32 heads
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t s_full[2], s_empty[2], q_full, q_ready, done;
    uint32_t tmem_base;
    int abort;
    int32_t n_valid, scratch[kCompactScratch];
};
static_assert(sizeof(WeightsSmem) + 1024 <= 232448, "shared memory budget of one CTA");

// Sums v[i] over the eight lanes that differ in bits 2-4: each gives half of
// its sums away and keeps the other, three times.  Afterwards v[0 .. N/8) hold
// the totals of entries N/8 * sum_block(lane) and those behind.
template <int N>
__device__ __forceinline__ void octet_sums(float (&v)[N], int lane) {
#pragma unroll
    for (int half = N / 2, bit = 4; bit < 32; half >>= 1, bit <<= 1) {
        const bool up = (lane & bit) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = up ? v[i] : v[i + half];
            const float keep = up ? v[i + half] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
        }
    }
}
__device__ __forceinline__ int sum_block(int lane) {
    return (lane & 4) | ((lane >> 2) & 2) | ((lane >> 4) & 1);
}

// Row producers of an e4m3 latent: tiles of 32 keys as 64 rows (see kKeysOf).
// As in produce_rows, a tile's codes and scales are in registers before its
// stage is free.
__device__ __forceinline__ void produce_e4m3_pairs(const PathParams &p, const int32_t *tile_rows,
                                                   int T, int pw, WeightsSmem &sm,
                                                   volatile int *abort_flag, int32_t *status) {
    constexpr int kKeys = kKeysOf<SA_E4M3>;
    constexpr int kSlots = (kKeys + kProducerWarps - 1) / kProducerWarps;
    const int lane = lane_id();
    const uint8_t *kv = static_cast<const uint8_t *>(p.kv);
    const uint8_t *rope = static_cast<const uint8_t *>(p.kv_rope);
    uint4 code[kSlots], rp[kSlots];
    float sc[kSlots];
    auto load = [&](int32_t rows, uint4 *c, uint4 *r4, float *s) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int k = pw + kProducerWarps * i;
            if (k < kKeys) {
                const int32_t r = __shfl_sync(0xffffffffu, rows, k);
                c[i] = __ldg(reinterpret_cast<const uint4 *>(kv + (int64_t)r * kDl) + lane);
                s[i] = kv_scale_at(p, r, 16 * lane);
                if (lane < 8)
                    r4[i] = __ldg(reinterpret_cast<const uint4 *>(rope + (int64_t)r * (kDr * 2)) +
                                  lane);
            }
        }
    };
    auto rows_of = [&](int n) { return n < T ? tile_rows[n * kKeys + lane] : 0; };
    int32_t rows1 = rows_of(1);
    if (T > 0) load(rows_of(0), code, rp, sc);
    for (int n = 0; n < T; ++n) {
        const int st = n % kStages;
        uint4 next_code[kSlots], next_rp[kSlots];
        float next_sc[kSlots];
        const int32_t rows2 = rows_of(n + 2);
        if (n + 1 < T) load(rows1, next_code, next_rp, next_sc);
        if (!warp_wait(&sm.kv_empty[st], ((n / kStages) & 1) ^ 1, abort_flag, status)) break;
        if (n == 1 && !warp_wait(&sm.q_ready, 0, abort_flag, status)) break;
        uint8_t *stage = sm.kv[st];
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int k = pw + kProducerWarps * i;
            if (k < kKeys) {
                const uint32_t xw[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
                uint32_t near[8], left[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f =
                        e4m3x2_to_float2(static_cast<uint16_t>(xw[j >> 1] >> (16 * (j & 1))));
                    const float x = f.x * sc[i], y = f.y * sc[i];
                    const __nv_bfloat162 a = __floats2bfloat162_rn(x, y);
                    const __nv_bfloat162 b = __floats2bfloat162_rn(
                        x - __low2float(a), y - __high2float(a));
                    near[j] = *reinterpret_cast<const uint32_t *>(&a);
                    left[j] = *reinterpret_cast<const uint32_t *>(&b);
                }
                const int sw = k & 7, b = lane >> 2, c0 = 2 * (lane & 3);
                uint8_t *dk = stage + (k >> 3) * kGroupBytes + (k & 7) * 128;
                uint8_t *dl = dk + (kKeys / 8) * kGroupBytes;
                const uint32_t o0 = b * 1024 + ((c0 ^ sw) << 4);
                const uint32_t o1 = b * 1024 + (((c0 + 1) ^ sw) << 4);
                *reinterpret_cast<uint4 *>(dk + o0) = make_uint4(near[0], near[1], near[2], near[3]);
                *reinterpret_cast<uint4 *>(dk + o1) = make_uint4(near[4], near[5], near[6], near[7]);
                *reinterpret_cast<uint4 *>(dl + o0) = make_uint4(left[0], left[1], left[2], left[3]);
                *reinterpret_cast<uint4 *>(dl + o1) = make_uint4(left[4], left[5], left[6], left[7]);
                if (lane < 8) {
                    const uint32_t o = (kBlocks - 1) * 1024 + ((lane ^ sw) << 4);
                    *reinterpret_cast<uint4 *>(dk + o) = rp[i];
                    *reinterpret_cast<uint4 *>(dl + o) = make_uint4(0, 0, 0, 0);
                }
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(&sm.kv_full[st]);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            code[i] = next_code[i];
            rp[i] = next_rp[i];
            sc[i] = next_sc[i];
        }
        rows1 = rows2;
    }
}

template <int kKv>
constexpr int kProducers = is_fp4(kKv) ? kFp4Warps : kProducerWarps;
template <int kKv>
constexpr int kCtaThreads = 32 * (5 + kProducers<kKv>);

// Entries of a selection that a thread looks up in one step of a CTA.
constexpr int kEntries = 6;

// rows_ready: the rows kernel has made rows (one list per query), kept, n_valid and
// starts; otherwise each CTA makes its own list, and the query's first the others.
template <int kKv>  // sa_dtype of the latent cache
__global__ void __launch_bounds__(kCtaThreads<kKv>, 1)
weights_mma_kernel(const __grid_constant__ CUtensorMap tm_q, const PathParams p,
                   const int32_t *__restrict__ idx, int32_t K, int32_t splits, bool rows_ready,
                   const float *__restrict__ lse, int32_t ld, int32_t ld_starts,
                   int32_t range_log2, int32_t *rows_of, int32_t *kept, int32_t *n_valid_of,
                   int32_t *starts_of, float *__restrict__ w) {
    extern __shared__ uint8_t smem_raw[];
    WeightsSmem &sm = *reinterpret_cast<WeightsSmem *>(align1024(smem_raw));
    const int t = blockIdx.x / splits, split = blockIdx.x % splits;
    const int warp = warp_id(), lane = lane_id();
    const int32_t *sel = idx + (int64_t)t * K;
    int32_t *rows = rows_of + (int64_t)(rows_ready ? t : blockIdx.x) * ld;
    int32_t *pos = kept + (int64_t)t * ld, *starts = starts_of + (int64_t)t * ld_starts;
    int32_t entries[kEntries];
    pdl_wait();
    if (!rows_ready) load_entries(sel, K, 0, entries);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.kv_full[s], 32 * kProducers<kKv>);
            mbar_init(&sm.kv_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.s_full[b], 1);
            mbar_init(&sm.s_empty[b], 4);  // the four epilogue warps
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_ready, 4);
        mbar_init(&sm.done, 1);
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(&sm.tmem_base, kWTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // after the TMEM allocation: a waiting successor holds none
    if (warp == 0 && lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full, kBlocks * kHeads * 128);
        for (int half = 0; half < 2; ++half)
            for (int b = 0; b < kBlocks; ++b)
                tma_load_2d(sm.kv[1 + half] + b * (64 * 128), &tm_q, 64 * b,
                            t * kHeads + 64 * half, &sm.q_full);
    }
    if (rows_ready) {
        if (threadIdx.x == 0) sm.n_valid = n_valid_of[t];
    } else {
        if (threadIdx.x == 0 && split == 0) starts[0] = 0;
        compact_selection(p, t, sel, K, kTile, rows, &sm.n_valid, sm.scratch, entries,
                          split == 0 ? pos : nullptr);
    }
    __syncthreads();
    const uint32_t tmem = sm.tmem_base;
    volatile int *abort_flag = &sm.abort;
    int32_t *status = p.status;
    const int32_t n_valid = sm.n_valid;
    int32_t j0, j1;
    constexpr int kKeys = kKeysOf<kKv>;
    split_range<kKeys>(n_valid, split, splits, j0, j1);
    const int T = j1 - j0;

    if (warp >= kEpiWarp0 && warp < kEpiWarp0 + 4) {
        const int j = warp & 3;  // TMEM subpartition of this warp
        const int h = 32 * j + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * j) << 16;
        bool ok = true;
        if (T > 0) {
            ok = warp_wait(&sm.q_full, 0, abort_flag, status);
            if (ok) {
                const int hr = h & 63;  // row within its half
#pragma unroll 1
                for (int b = 0; b < kBlocks; ++b) {
                    const uint8_t *qr = sm.kv[1 + (h >> 6)] + b * (64 * 128) + hr * 128;
                    uint32_t v[32];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint4 x = *reinterpret_cast<const uint4 *>(qr + ((c ^ (hr & 7)) << 4));
                        if (is_fp4(kKv)) x = b < kBlocks - 1 ? fp4_order(x) : fp4_rope(x);
                        v[4 * c] = x.x;
                        v[4 * c + 1] = x.y;
                        v[4 * c + 2] = x.z;
                        v[4 * c + 3] = x.w;
                    }
                    tmem_st32_u(tmem + lanes + 32 * b, v);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_ready);  // also frees ring stages 1 and 2
        }
        const float sl2 = p.sm_scale * kLog2e * (is_fp4(kKv) ? kFp4Up : 1.0f);
        // this thread's heads in S: 32j + lane / 4 + 8i; one with nothing selected
        // (lse = -inf) adds nothing
        float minus[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float l =
                T > 0 ? __ldg(lse + (int64_t)t * kHeads + 32 * j + (lane >> 2) + 8 * i) : 0.f;
            minus[i] = l == -INFINITY ? -INFINITY : -l * kLog2e;
        }
        float *wt = w + (int64_t)t * ld + (int64_t)j0 * kKeys;
        const int block = sum_block(lane), q2 = 2 * (lane & 3);
        // After a failed wait the loop keeps going without waiting or touching
        // TMEM, so that the warps still meet at the named barrier.
        for (int n = 0; n < T; ++n) {
            const int sb = n & 1;
            if (ok) ok = warp_wait(&sm.s_full[sb], (n >> 1) & 1, abort_flag, status);
            // v[2r + e]: key 8r + 2 (lane % 4) + e, over this thread's four heads
            constexpr int kSums = kKeys / 4;
            float v[kSums];
            if (ok) {
                tc_fence_after();
                uint32_t a[32], b[32];
                tmem_ld_16x256b_x8(tmem + lanes + kWColS + kTile * sb, a);
                tmem_ld_16x256b_x8(tmem + lanes + (16u << 16) + kWColS + kTile * sb, b);
                tmem_wait_ld_keep(a);
                tmem_wait_ld_keep(b);
#pragma unroll
                for (int i = 0; i < kSums; ++i) {
                    float z[4];  // column i of the four heads
#pragma unroll
                    for (int h4 = 0; h4 < 4; ++h4) {
                        const uint32_t *s = h4 < 2 ? a : b;
                        const int at = 4 * (i >> 1) + (i & 1) + 2 * (h4 & 1);
                        z[h4] = __uint_as_float(s[at]);
                        if constexpr (kKeys == 32) z[h4] += __uint_as_float(s[at + 16]);
                    }
                    v[i] = (ex2(fmaf(z[0], sl2, minus[0])) + ex2(fmaf(z[1], sl2, minus[1]))) +
                           (ex2(fmaf(z[2], sl2, minus[2])) + ex2(fmaf(z[3], sl2, minus[3])));
                }
            } else {
#pragma unroll
                for (int i = 0; i < kSums; ++i) v[i] = 0.f;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_empty[sb]);
            octet_sums(v, lane);
            float *part = sm.part[sb][j];
            if constexpr (kKeys == 32) {
                part[8 * (block >> 1) + q2 + (block & 1)] = v[0];
            } else {
                *reinterpret_cast<float2 *>(part + 8 * block + q2) = make_float2(v[0], v[1]);
            }
            // one barrier a tile: the other parity's sums are read before it
            named_barrier(1, 128);
            const int k = 32 * j + lane;  // the first warps finish one key per lane
            if (k < kKeys && (j0 + n) * kKeys + k < n_valid) {
                const float(*ps)[kTile] = sm.part[sb];
                wt[n * kKeys + k] = (ps[0][k] + ps[1][k]) + (ps[2][k] + ps[3][k]);
            }
        }
    } else if (warp >= 1) {
        const int32_t *tile_rows = rows + (int64_t)j0 * kKeys;
        if constexpr (kKv == SA_E4M3)
            produce_e4m3_pairs(p, tile_rows, T, warp - 1, sm, abort_flag, status);
        else
            produce_rows<kKv>(p, tile_rows, T, producer_index(warp), sm.kv, sm.kv_full,
                              sm.kv_empty, &sm.q_ready, 1, abort_flag, status);
        if (split == 0 && !rows_ready) {
            const int32_t thread = 32 * producer_index(warp) + lane;
            write_starts(pos, n_valid, starts, ld_starts, range_log2, thread,
                         32 * kProducers<kKv>);
            if (thread == 0) n_valid_of[t] = n_valid;
        }
    } else if (T > 0) {
        // the whole warp waits and computes descriptors, one lane issues
        constexpr uint32_t id_s = instr_desc(kHeads, kTile, 1 /*bf16*/, 0, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        bool ok = warp_wait(&sm.q_ready, 0, abort_flag, status);
        for (int n = 0; ok && n < T; ++n) {
            const int st = n % kStages, sb = n & 1;
            ok = warp_wait(&sm.s_empty[sb], ((n >> 1) & 1) ^ 1, abort_flag, status) &&
                 warp_wait(&sm.kv_full[st], (n / kStages) & 1, abort_flag, status);
            if (!ok) break;
            if constexpr (kKv == SA_BF16) fence_proxy_async_smem();  // cp.async rows
            tc_fence_after();
            const uint32_t d = tm + kWColS + kTile * sb;
            const uint32_t stage = smem_u32(sm.kv[st]);
            if (elect_one()) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const uint64_t bd = desc_kmajor_sw128_sbo(stage + b * 1024, kGroupBytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ts(d, tm + 32 * b + 8 * k, bd + 2 * k, id_s, (b | k) != 0);
                }
                mma_commit(&sm.s_full[sb]);
                if (n + kStages < T) mma_commit(&sm.kv_empty[st]);
            }
            __syncwarp();
        }
        // every MMA issued above has completed before TMEM is released, after a
        // timeout too
        if (elect_one()) mma_commit(&sm.done);
        __syncwarp();
        int never = 0;
        warp_wait(&sm.done, 0, &never, status);
    }
    // with no tiles nobody waited for Q: its copy must land before the CTA ends
    if (warp == 0 && lane == 0 && T == 0) mbar_wait(&sm.q_full, 0, abort_flag, status);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kWTmemCols);
    }
}

// The attention's tensor-core shape; other shapes take the CUDA-core kernel.
bool weights_mma_supported(const PathParams &p) {
    const bool kv_ok = p.kv_dtype == SA_BF16 ||
                       ((p.kv_dtype == SA_E4M3 || is_fp4(p.kv_dtype)) && p.kv_rope != nullptr);
    return kv_ok && p.q_dtype == SA_BF16 && p.heads == kHeads && p.d_latent == kDl &&
           p.d_rope == kDr;
}

cudaError_t launch_weights_mma(const PathParams &p, const int32_t *idx, int32_t top_k,
                               const float *lse, int32_t ld, int32_t ld_starts,
                               int32_t range_log2, int32_t *rows, int32_t *kept, int32_t *n_valid,
                               int32_t *starts, float *w, cudaStream_t s) {
    CUtensorMap tq;
    if (!encode_tmap_2d(&tq, 2, p.q, kD, (uint64_t)p.n_q * kHeads, kD * 2, 64, 64, true))
        return cudaErrorInvalidValue;
    const size_t smem = sizeof(WeightsSmem) + 1024;
    const auto kernel = p.kv_dtype == SA_BF16    ? weights_mma_kernel<SA_BF16>
                        : p.kv_dtype == SA_E4M3  ? weights_mma_kernel<SA_E4M3>
                        : p.kv_dtype == SA_MXFP4 ? weights_mma_kernel<SA_MXFP4>
                                                 : weights_mma_kernel<SA_NVFP4>;
    const cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    const int32_t splits = weights_splits(p.n_q, top_k, p.kv_dtype);
    const int threads = is_fp4(p.kv_dtype) ? kCtaThreads<SA_MXFP4> : kCtaThreads<SA_BF16>;
    count_launch();
    return launch_pdl(kernel, dim3((unsigned)((int64_t)p.n_q * splits)), dim3(threads), smem,
                      s, tq, p, idx, top_k, splits, weights_rows_first(p.n_q, top_k, p.kv_dtype),
                      lse, ld, ld_starts, range_log2, rows, kept, n_valid, starts, w);
}

// -------------------------------------------------------------------- sum ---
// One CTA per range of a sequence's positions.  Warp w walks query groups w,
// w + kWarps, ...: its lanes look the queries' entries in the range up, then
// the entries are added to the warp's own sums in shared memory, one query
// after another (four queries' loads in flight).  The warps' sums are added in
// the order of w at the end.
constexpr int kSumQueries = 4;  // queries whose entries are loaded together
constexpr int kSumEntries = 2;  // of each, 32 entries this many times; the rest follow one by one

template <typename Shape>
__global__ void __launch_bounds__(32 * Shape::kWarps)
weights_sum_kernel(const PathParams p, int32_t chunks, int32_t limit, int32_t ld,
                   int32_t ld_starts, const int32_t *__restrict__ kept,
                   const int32_t *__restrict__ n_valid, const int32_t *__restrict__ starts,
                   const float *__restrict__ w, const float *acc_in, float decay, float *acc_out,
                   int64_t ld_acc) {
    pdl_wait();
    pdl_trigger();
    constexpr int kSumRange = Shape::kRange, kSumWarps = Shape::kWarps;
    constexpr int kSumThreads = 32 * kSumWarps;
    __shared__ float sums[kSumWarps][kSumRange];
    __shared__ int32_t used[kSumWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t b = (int32_t)(blockIdx.x / chunks), c = (int32_t)(blockIdx.x % chunks);
    int32_t len = p.seq_len[b];
    if (len > limit) {
        if (c == 0 && tid == 0) report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_POSITION);
        len = limit;
    }
    const int32_t lo = c * kSumRange;
    if (lo >= len) return;
    const int32_t hi = min(len, lo + kSumRange);
    const int64_t base = (int64_t)b * ld_acc;
    constexpr int kPer = (kSumRange + kSumThreads - 1) / kSumThreads;
    float old[kPer];  // on its way while the entries are added
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int32_t at = lo + i * kSumThreads + tid;
        old[i] = acc_in != nullptr && at < hi ? acc_in[base + at] : 0.0f;
    }
    float *s = sums[warp];
    bool cleared = false;
    for (int32_t t0 = Shape::kGroup * warp; t0 < p.n_q; t0 += Shape::kGroup * kSumWarps) {
        const int32_t t = lane < Shape::kGroup ? t0 + lane : p.n_q;
        int32_t k0 = 0, k1 = 0;
        bool plain = true;
        if (t < p.n_q && p.q_seq[t] == b) {
            // a query sees fewer positions than the sequence has when others follow
            const int32_t *st = starts + (int64_t)t * ld_starts;
            k0 = st[min(c, ld_starts - 1)];
            k1 = st[min(c + 1, ld_starts - 1)];
            if (st[0] < 0) {  // in no order, or with repeats: look at all of them
                plain = false;
                k0 = 0;
                k1 = n_valid[t];
            }
        }
        uint32_t todo = __ballot_sync(0xffffffffu, k1 > k0);
        const uint32_t distinct = __ballot_sync(0xffffffffu, plain);
        if (todo != 0 && !cleared) {
            for (int i = lane; i < kSumRange; i += 32) s[i] = 0.0f;
            __syncwarp();
            cleared = true;
        }
        while (todo != 0) {
            int32_t at[kSumQueries][kSumEntries], from[kSumQueries], to[kSumQueries];
            float x[kSumQueries][kSumEntries];
            int64_t row[kSumQueries];
            bool once[kSumQueries];  // the query's positions are distinct
#pragma unroll
            for (int j = 0; j < kSumQueries; ++j) {
                const int u = todo != 0 ? __ffs(todo) - 1 : 0;
                once[j] = (distinct >> u) & 1u;
                from[j] = __shfl_sync(0xffffffffu, k0, u);
                to[j] = todo != 0 ? __shfl_sync(0xffffffffu, k1, u) : from[j];
                row[j] = (int64_t)(t0 + u) * ld;
                todo &= todo - 1;
#pragma unroll
                for (int e = 0; e < kSumEntries; ++e) {
                    const int32_t k = from[j] + 32 * e + lane;
                    at[j][e] = k < to[j] ? kept[row[j] + k] - lo : -1;
                    x[j][e] = k < to[j] ? w[row[j] + k] : 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < kSumQueries; ++j) {
                // entries that repeat a position add the same weight each: their
                // order does not matter
                auto add = [&](int32_t a, float y) {
                    if (a < 0 || a >= kSumRange) return;
                    if (once[j]) s[a] += y;
                    else atomicAdd(&s[a], y);
                };
#pragma unroll
                for (int e = 0; e < kSumEntries; ++e) add(at[j][e], x[j][e]);
                for (int32_t k = from[j] + 32 * kSumEntries + lane; k < to[j]; k += 32)
                    add(kept[row[j] + k] - lo, w[row[j] + k]);
                __syncwarp();
            }
        }
    }
    if (lane == 0) used[warp] = cleared;
    __syncthreads();
    float total[kPer] = {};
#pragma unroll 8
    for (int v = 0; v < kSumWarps; ++v) {
        if (!used[v]) continue;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = i * kSumThreads + tid;
            if (at < kSumRange) total[i] += sums[v][at];
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int32_t at = lo + i * kSumThreads + tid;
        if (at < hi)
            acc_out[base + at] = (acc_in != nullptr ? decay * old[i] : 0.0f) + total[i];
    }
}

template <typename Shape>
cudaError_t launch_weights_sum(const PathParams &p, int32_t ld, int32_t ld_starts,
                               const int32_t *kept, const int32_t *n_valid,
                               const int32_t *starts, const float *w, const float *acc_in,
                               float decay, float *acc_out, int64_t ld_acc, cudaStream_t s) {
    const int64_t limit = std::min(ld_acc, (int64_t)p.max_pages * 64);
    const int64_t chunks = ceil_div(limit, Shape::kRange);
    count_launch();
    return launch_pdl(weights_sum_kernel<Shape>, dim3((unsigned)(chunks * p.batch)),
                      dim3(32 * Shape::kWarps), 0, s, p, (int32_t)chunks, (int32_t)limit, ld,
                      ld_starts, kept, n_valid, starts, w, acc_in, decay, acc_out, ld_acc);
}

}  // namespace

// one CTA per SM: split a query's tiles while there are SMs without one
int32_t weights_splits(int32_t n_q, int32_t top_k, int32_t kv_dtype) {
    if (n_q <= 0 || top_k <= 0) return 1;
    const int32_t tiles =
        (int32_t)ceil_div(top_k, kv_dtype == SA_E4M3 ? kKeysOf<SA_E4M3> : kTile);
    return std::max(1, std::min(tiles, num_sms() / n_q));
}

// Whether the rows kernel runs in front of the tensor-core one: for selections that
// take a CTA more than four steps, if several CTAs share a query: each would make and
// store the whole list for its few tiles.  Two queries over e4m3, 5000 entries: 50 us
// with the kernel in front and 44 without; one query over bf16, 9400 entries: 46 and
// 53, 300000 entries: 638 and 1140, with 3.6 and 180 MB of workspace.
bool weights_rows_first(int32_t n_q, int32_t top_k, int32_t kv_dtype) {
    return top_k > 4 * kEntries * kCtaThreads<SA_BF16> &&
           weights_splits(n_q, top_k, kv_dtype) > 1;
}

int32_t weights_lists(int32_t n_q, int32_t top_k, int32_t kv_dtype) {
    if (weights_rows_first(n_q, top_k, kv_dtype)) return 1;
    return weights_splits(n_q, top_k, kv_dtype);
}

int32_t weights_ld(int32_t top_k) { return (int32_t)round_up(top_k > 0 ? top_k : 1, kTile); }

int32_t weights_starts_ld(int32_t n_q, int32_t batch, int32_t max_visible) {
    const int32_t range = sum_many(n_q, batch) ? SumMany::kRange : SumFew::kRange;
    return (int32_t)ceil_div(max_visible > 0 ? max_visible : 1, range) + 1;
}

cudaError_t launch_accumulate_weights(const PathParams &p, const int32_t *idx, int32_t top_k,
                                      const float *lse, const float *acc_in, float decay,
                                      float *acc_out, int64_t ld_acc, int32_t *rows,
                                      int32_t *kept, int32_t *n_valid, int32_t *starts, float *w,
                                      cudaStream_t s) {
    const bool many = sum_many(p.n_q, p.batch);
    const int32_t ld = weights_ld(top_k);
    const int32_t ld_starts = weights_starts_ld(p.n_q, p.batch, p.max_visible);
    cudaError_t e;
    const int32_t range_log2 = many ? 8 : 10;
    const bool mma = weights_mma_supported(p);
    if (p.n_q > 0 && (!mma || weights_rows_first(p.n_q, top_k, p.kv_dtype))) {
        count_launch();
        e = launch_pdl(weights_rows_kernel, dim3((unsigned)p.n_q), dim3(kRowsThreads), 0, s, p, idx,
                       top_k, ld, ld_starts, range_log2, rows, kept, n_valid, starts);
        if (e != cudaSuccess) return e;
    }
    if (p.n_q > 0) {
        e = mma ? launch_weights_mma(p, idx, top_k, lse, ld, ld_starts, range_log2, rows, kept,
                                     n_valid, starts, w, s)
                : launch_weights_simt(p, lse, ld, rows, n_valid, w, s);
        if (e != cudaSuccess) return e;
    }
    return many ? launch_weights_sum<SumMany>(p, ld, ld_starts, kept, n_valid, starts, w, acc_in,
                                              decay, acc_out, ld_acc, s)
                : launch_weights_sum<SumFew>(p, ld, ld_starts, kept, n_valid, starts, w, acc_in,
                                             decay, acc_out, ld_acc, s);
}

}  // namespace sa
