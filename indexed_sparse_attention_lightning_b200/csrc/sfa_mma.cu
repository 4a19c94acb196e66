// sfa_mma.cu -- sparse MLA attention on the 5th-generation tensor cores.
//
// For query t and its selected latent rows s ("Optimizing Next-Gen LLM
// Inference" §3.3: attention only on the selected positions, reading the cache
// by index; "Inference Acceleration for New Large Model Architectures" §3.2:
// aggregated, vectorised sparse reads; "Engineering Practices for Optimizing
// Ultra-Large Sparse Attention Model Inference" §3.1: index construction, block
// loading with asynchronous prefetch, local attention on matrix units):
//     z_s = sm_scale * q[t,h,:] . kv[s,:]   (576-d: 512 latent + 64 rope)
//     out[t,h,:] = sum_s softmax(z)_s kv[s, 0:512],   lse = log sum_s exp(z_s)
//
// B200 mapping.  All 128 absorbed-query heads share the selected rows, so both
// contractions are dense per key tile.  One CTA owns 64 heads of one query
// (two CTAs per query) and walks 64-key tiles of its selected rows:
//     S  = Q K^T   M = 64 heads, N = 64 keys, K = 576   (A = Q from TMEM)
//     O += P V     M = 64 heads, N = 2 x 256 dims, K = 64 keys
// An M = 64 accumulator fills lanes 0-15 of each 32-lane TMEM subpartition; a
// second one may sit on lanes 16-31.  So Q (288 columns of bf16 pairs) and two
// S buffers live on the lower half-lanes and O (64 x 512 fp32, all 512
// columns) on the upper half-lanes: head m's S row is lane 32(m/16) + m%16,
// its O row that lane + 16, i.e. the same warp.  Each tile's 64 full 1152-byte
// rows are copied once into a 128-byte-swizzled stage that is the K-major B
// operand of S and, read MN-major, the B operand of P V.  The stage's rope
// block (the last 64 dims of every row, 8 KB) is read by S only, so once S is
// done the softmax writes that tile's P (64 heads x 64 keys bf16, also 8 KB)
// over it: every stage carries its own P, and the softmax of the next tile
// never waits for P V of this one to release a shared P buffer.
//
// Roles (384 threads, 416 for a 4-bit latent; one CTA per SM):
//   warp 0     lane 0 loads Q by TMA (into the third ring stage; this copy
//              starts before the wait on the top-K kernel); then one lane
//              issues the MMAs, S of tile n + 1 before P V of tile n, and
//              commits them to mbarriers;
//   warps 1-7  copy the selected rows (16-byte cp.async, the swizzle applied
//              in the addresses) into a 3-stage ring freed by each tile's P V;
//              random 1152-byte rows reach shared memory fastest this way (an
//              e4m3 or 4-bit latent is loaded, decoded to bf16 and stored, the
//              4-bit one with the help of warp 12);
//   warps 8-11 move Q into TMEM, then run the online softmax.  Warp 8 + j
//              owns heads 16j .. 16j + 15 and reads their S rows with 16-lane
//              loads: thread i holds heads 16j + i/4 and 16j + i/4 + 8, keys
//              8r + 2(i%4) and 8r + 2(i%4) + 1 of each 8-key group r, so a row
//              maximum takes two shuffles and P goes to shared memory in
//              bf16 pairs.  O is rescaled in TMEM (16-lane accesses with the
//              same thread-to-head mapping, leaving Q and S alone) only when a
//              head's running maximum grows by more than 2^8; finally they
//              write O / l, with the help of warps 4-7 (write_output).
// The fused decode gets the selection's physical rows from the top-K kernel;
// otherwise every CTA turns its query's positions into rows itself, in shared
// memory, while Q is on its way (a kernel in front of this one took 9 us).  All
// waits are bounded; a timeout is reported in the workspace status word.
#include "common.cuh"
#include "internal.h"
#include "sfa_gather.cuh"
#include "sm100.cuh"

namespace sa {
namespace {
using namespace sfa;

constexpr int kHeadsCta = 64;
constexpr int kSoftmaxWarp0 = 8;  // warps 8-11, one per TMEM subpartition
constexpr int kMaxK = 2048;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColQ = 0;    // lower half-lanes: Q, 288 columns
constexpr uint32_t kColS = 288;  // lower half-lanes: two S buffers of 64 columns
constexpr uint32_t kLaneO = 16;  // O: upper half-lanes, columns [0, 512)
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;
// After S, block 8 of a stage (the rope) holds P: head h's 64 keys at
// (h/8)*kGroupBytes + 8*1024 + (h%8)*128 (+ swizzle), the K-major A operand of
// P V with 8-head groups kGroupBytes apart.
constexpr uint32_t kPOffset = (kBlocks - 1) * 1024;  // the rope block
// The output's way through shared memory: 128 columns of 16 rows per warp, fp32
// or bf16, each row with eight columns of space behind it.
constexpr int kOutCols = 128, kOutBytes = 16 * (kOutCols + 8) * 4;
static_assert(8 * kOutBytes <= (int)kStageBytes, "the eight warps' rows fit in a stage");
constexpr int kOutBarrier = 1;  // the eight warps that write the output

struct SfaSmem {
    // ring stage: 8 groups of 8 rows; a group holds the 9 column blocks of its
    // rows, each 8 x 128 bytes with the 128-byte swizzle (see kGroupBytes)
    uint8_t kv[kStages][kStageBytes];
    uint64_t kv_full[kStages], kv_empty[kStages];
    // kv_empty: one phase per P V of its stage, which frees the stage (and lets a
    // rescale of the next tile at O); o_final: once, after the last P V, for the
    // final read of O
    uint64_t s_full[2], p_full[kStages], o_final, q_full, q_ready;
    uint32_t tmem_base;
    int abort;
    float inv[kHeadsCta];  // 1 / l (4 bits: times kFp4Up)
    int32_t n_valid, scratch[kCompactScratch];
    int32_t rows[kMaxK];  // the selection's physical rows, whole tiles
};

static_assert(sizeof(SfaSmem) + 1024 <= 232448, "shared memory budget of one CTA");
static_assert(kColS + 2 * kTile <= kTmemCols && kBlocks * 32 == (int)kColS, "TMEM columns");

// Maximum over the four lanes of a row.
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

struct SfaArgs {
    PathParams p;
    const int32_t *rows;     // [n_q, ld_rows] physical rows, padded to whole tiles, or null
    const int32_t *n_valid;  // [n_q] with rows
    int32_t ld_rows;
    const int32_t *idx;      // [n_q, top_k] selected positions, without rows
    int32_t top_k;
    int32_t splits;
    void *out;               // [n_q, 128, 512] (splits == 1)
    int32_t out_dtype;
    float *lse;              // [n_q, 128] or null (splits == 1)
    float *o_part;           // [n_q, splits, 128, 512] (splits > 1)
    float *lse_part;         // [n_q, splits, 128]      (splits > 1)
};

template <int kKv>
constexpr int kProducers = is_fp4(kKv) ? kFp4Warps : kProducerWarps;
template <int kKv>
constexpr int kCtaThreads = 32 * (5 + kProducers<kKv>);

// Columns [256 half, 256 half + 256) of O / l of heads 16j .. 16j + 15 (warp 8 +
// j, and 4 + j for the second half; both see TMEM lanes 32j and up), 128 columns
// at a time through shared memory (stage 0: every MMA is done, and a CTA without
// tiles has only Q's copy in flight, into stage 2), so that a store of the warp
// writes whole lines of two rows.  It takes 4000 cycles for bf16 and 6900 for
// fp32, the first pass twice the second; one warp per 16 heads, storing 16 bytes
// of 16 rows at a time, took 6000 and 10500.
template <int kKv>
__device__ __forceinline__ void write_output(SfaSmem &sm, const SfaArgs &a, int t, int split,
                                             int hh, int j, int half, bool any, uint32_t tmem_o) {
    const int lane = lane_id(), q4 = lane & 3;
    const float inv_a = sm.inv[16 * j + (lane >> 2)], inv_b = sm.inv[16 * j + (lane >> 2) + 8];
    const bool part = a.splits > 1, wide = part || a.out_dtype == SA_F32;
    const int bytes = wide ? 4 : 2;
    const int stride = kOutCols * bytes + 8 * bytes;  // no two lanes of a store in one bank
    uint8_t *buf = sm.kv[0] + (4 * half + j) * kOutBytes;
    const int64_t row0 =
        (part ? (int64_t)t * a.splits + split : t) * 128 + kHeadsCta * hh + 16 * j;
    uint8_t *dst =
        (part ? reinterpret_cast<uint8_t *>(a.o_part) : static_cast<uint8_t *>(a.out)) +
        row0 * (kDl * bytes);
#pragma unroll 1
    for (int c = 256 * half; c < 256 * half + 256; c += kOutCols) {
        uint32_t v[2][32] = {};
        if (any) {
#pragma unroll
            for (int h = 0; h < 2; ++h) tmem_ld_16x256b_x8(tmem_o + c + 64 * h, v[h]);
            tmem_wait_ld_keep(v[0]);
            tmem_wait_ld_keep(v[1]);
        }
        // columns 8i + 2 q4 and the next one of two heads
        uint8_t *ra = buf + (lane >> 2) * stride + 2 * q4 * bytes, *rb = ra + 8 * stride;
        if (wide) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t *x = v[i >> 3] + 4 * (i & 7);
                *reinterpret_cast<float2 *>(ra + 32 * i) = make_float2(
                    __uint_as_float(x[0]) * inv_a, __uint_as_float(x[1]) * inv_a);
                *reinterpret_cast<float2 *>(rb + 32 * i) = make_float2(
                    __uint_as_float(x[2]) * inv_b, __uint_as_float(x[3]) * inv_b);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t *x = v[i >> 3] + 4 * (i & 7);
                *reinterpret_cast<__nv_bfloat162 *>(ra + 16 * i) = __floats2bfloat162_rn(
                    __uint_as_float(x[0]) * inv_a, __uint_as_float(x[1]) * inv_a);
                *reinterpret_cast<__nv_bfloat162 *>(rb + 16 * i) = __floats2bfloat162_rn(
                    __uint_as_float(x[2]) * inv_b, __uint_as_float(x[3]) * inv_b);
            }
        }
        __syncwarp();
        // eight columns per lane, two rows at a time; of a 4-bit latent in the order
        // of the stages
        const uint8_t *from = buf + (lane >> 4) * stride + 8 * bytes * (lane & 15);
        uint8_t *to = dst + ((lane >> 4) * kDl + c + 8 * (lane & 15)) * bytes;
        if (wide) {
            const int turn = (lane >> 2) & 1;  // so that eight lanes' pieces meet all banks once
#pragma unroll
            for (int r = 0; r < 16; r += 8) {
                uint4 x[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 *f =
                        reinterpret_cast<const uint4 *>(from + (r + 2 * i) * stride);
                    const uint4 y0 = f[turn], y1 = f[1 - turn];
                    const uint4 lo = turn ? y1 : y0, hi = turn ? y0 : y1;
                    x[i][0] = is_fp4(kKv) ? make_uint4(lo.x, lo.z, hi.x, hi.z) : lo;
                    x[i][1] = is_fp4(kKv) ? make_uint4(lo.y, lo.w, hi.y, hi.w) : hi;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 *d = reinterpret_cast<uint4 *>(to + (r + 2 * i) * (kDl * 4));
                    if (part) {  // in the workspace: aligned to 32 bytes
                        store_32_bytes(d, x[i][0], x[i][1]);
                    } else {
                        d[0] = x[i][0];
                        d[1] = x[i][1];
                    }
                }
            }
        } else {
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = *reinterpret_cast<const uint4 *>(from + 2 * i * stride);
                if (is_fp4(kKv)) x[i] = fp4_natural(x[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4 *>(to + 2 * i * (kDl * 2)) = x[i];
        }
        __syncwarp();
    }
}

template <int kKv>  // sa_dtype of the latent cache
__global__ void __launch_bounds__(kCtaThreads<kKv>, 1)
sfa_mma_kernel(const __grid_constant__ CUtensorMap tm_q, const SfaArgs a) {
    extern __shared__ uint8_t smem_raw[];
    SfaSmem &sm = *reinterpret_cast<SfaSmem *>(align1024(smem_raw));
    const PathParams &p = a.p;
    const int hh = blockIdx.x & 1;  // which 64 heads
    const int unit = blockIdx.x >> 1;
    const int t = unit / a.splits, split = unit % a.splits;
    const int warp = warp_id(), lane = lane_id();
    // the selection's entries, 384 threads or more: one step
    const int32_t *sel = a.idx + (int64_t)t * a.top_k;
    int32_t entries[6];
    if (a.rows == nullptr) {
        pdl_wait();
        load_entries(sel, a.top_k, 0, entries);
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.kv_full[s], 32 * kProducers<kKv>);
            mbar_init(&sm.kv_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) mbar_init(&sm.s_full[b], 1);
        for (int s = 0; s < kStages; ++s) mbar_init(&sm.p_full[s], 4);  // the four softmax warps
        mbar_init(&sm.o_final, 1);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_ready, 4);
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(&sm.tmem_base, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // after the TMEM allocation: a waiting successor holds none
    // Q is an input, not the previous kernel's output: its copy (into ring
    // stage 2) starts before the wait on that kernel
    if (warp == 0 && lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full, kBlocks * kHeadsCta * 128);
        for (int b = 0; b < kBlocks; ++b)
            tma_load_2d(sm.kv[2] + b * (kHeadsCta * 128), &tm_q, 64 * b, t * 128 + kHeadsCta * hh,
                        &sm.q_full);
    }
    const int32_t *rows = sm.rows;
    if (a.rows != nullptr) {
        pdl_wait();  // they come from the kernel before
        rows = a.rows + (int64_t)t * a.ld_rows;
        if (threadIdx.x == 0) sm.n_valid = a.n_valid[t];
    } else {
        compact_selection(p, t, sel, a.top_k, kTile, sm.rows, &sm.n_valid, sm.scratch, entries);
    }
    __syncthreads();
    const uint32_t tmem = sm.tmem_base;
    volatile int *abort_flag = &sm.abort;
    int32_t *status = p.status;
    const int32_t n_valid = sm.n_valid;
    int32_t j0, j1;
    split_range(n_valid, split, a.splits, j0, j1);
    const int T = j1 - j0;

    if (warp >= kSoftmaxWarp0 && warp < kSoftmaxWarp0 + 4) {
        const int j = warp & 3;  // TMEM subpartition of this warp
        const int q4 = lane & 3;
        const int ha = 16 * j + (lane >> 2), hb = ha + 8;  // the two heads of this thread
        const uint32_t lane_lo = static_cast<uint32_t>(32 * j) << 16;
        const uint32_t lane_hi = static_cast<uint32_t>(32 * j + kLaneO) << 16;
        bool ok = true;
        // ----------------------------------------------- Q into TMEM ---
        // Q (128-byte-swizzled, in ring stage 2) -> lanes 32j .. 32j + 15;
        // the 32-lane stores also put a copy on O's columns of lanes 16-31,
        // which the first P V overwrites.
        if (T > 0) {
            ok = warp_wait(&sm.q_full, 0, abort_flag, status);
            if (ok) {
                const int h = 16 * j + (lane & 15);
#pragma unroll 1
                for (int b = 0; b < kBlocks; ++b) {
                    const uint8_t *qr = sm.kv[2] + b * (kHeadsCta * 128) + h * 128;
                    uint32_t v[32];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint4 x = *reinterpret_cast<const uint4 *>(qr + ((c ^ (h & 7)) << 4));
                        if (is_fp4(kKv)) x = b < kBlocks - 1 ? fp4_order(x) : fp4_rope(x);
                        v[4 * c] = x.x;
                        v[4 * c + 1] = x.y;
                        v[4 * c + 2] = x.z;
                        v[4 * c + 3] = x.w;
                    }
                    tmem_st32_u(tmem + lane_lo + kColQ + 32 * b, v);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_ready);  // also frees ring stage 2
        }

        // ----------------------------------------------- online softmax ---
        // The loop never leaves early: after a failed wait (a timeout raised
        // the abort flag) it keeps going without waiting or touching TMEM.
        const float sl2 = p.sm_scale * kLog2e * (is_fp4(kKv) ? kFp4Up : 1.0f);
        // this lane's row of the P matrices it addresses
        const uint32_t p_row = lane & 7, p_key = lane >> 3;
        const uint32_t p_at = 2 * j * kGroupBytes + p_row * 128;
        float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
        for (int n = 0; n < T; ++n) {
            const int sb = n & 1;
            if (ok) ok = warp_wait(&sm.s_full[sb], (n >> 1) & 1, abort_flag, status);
            uint32_t v[32];
            if (ok) {
                tc_fence_after();
                tmem_ld_16x256b_x8(tmem + lane_lo + kColS + kTile * sb, v);
                tmem_wait_ld();
            }
            const int kvalid = ok ? n_valid - (j0 + n) * kTile : 0;
            float xa[16], xb[16];
            float ta, tb;
            if constexpr (is_fp4(kKv)) {
                // The row maximum is taken of the raw sums (their minimum under a
                // negative scale); scale and maximum are applied together below.
                const float none = sl2 < 0.f ? INFINITY : -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    xa[i] = __uint_as_float(v[4 * (i >> 1) + (i & 1)]);
                    xb[i] = __uint_as_float(v[4 * (i >> 1) + 2 + (i & 1)]);
                }
                if (kvalid < kTile) {  // the last tile: mask the padding
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const bool valid = 8 * (i >> 1) + 2 * q4 + (i & 1) < kvalid;
                        xa[i] = valid ? xa[i] : none;
                        xb[i] = valid ? xb[i] : none;
                    }
                }
                ta = xa[0];
                tb = xb[0];
                if (sl2 < 0.f) {
#pragma unroll
                    for (int i = 1; i < 16; ++i) {
                        ta = fminf(ta, xa[i]);
                        tb = fminf(tb, xb[i]);
                    }
                    ta = -quad_max(-ta) * sl2;
                    tb = -quad_max(-tb) * sl2;
                } else {
#pragma unroll
                    for (int i = 1; i < 16; ++i) {
                        ta = fmaxf(ta, xa[i]);
                        tb = fmaxf(tb, xb[i]);
                    }
                    ta = quad_max(ta) * sl2;
                    tb = quad_max(tb) * sl2;
                }
            } else {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        xa[2 * r + e] = __uint_as_float(v[4 * r + e]) * sl2;
                        xb[2 * r + e] = __uint_as_float(v[4 * r + 2 + e]) * sl2;
                    }
                }
                if (kvalid < kTile) {  // the last tile: mask the padding
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const bool valid = 8 * r + 2 * q4 + e < kvalid;
                            xa[2 * r + e] = valid ? xa[2 * r + e] : -INFINITY;
                            xb[2 * r + e] = valid ? xb[2 * r + e] : -INFINITY;
                        }
                    }
                }
                ta = xa[0];
                tb = xb[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) {
                    ta = fmaxf(ta, xa[i]);
                    tb = fmaxf(tb, xb[i]);
                }
                ta = quad_max(ta);
                tb = quad_max(tb);
            }
            // lazy rescaling: a running maximum moves only on a large jump
            const bool grow_a = ta > m_a + kRescaleLog2, grow_b = tb > m_b + kRescaleLog2;
            const float mn_a = grow_a ? ta : m_a, mn_b = grow_b ? tb : m_b;
            const float f_a = (grow_a && n > 0) ? exp2f(m_a - mn_a) : 1.f;
            const float f_b = (grow_b && n > 0) ? exp2f(m_b - mn_b) : 1.f;
            uint32_t pa[8], pb[8];
            float la = 0.f, lb = 0.f;
            if constexpr (is_fp4(kKv)) {
                float2 sum_a = make_float2(0.f, 0.f), sum_b = sum_a;
                const float2 scale = make_float2(sl2, sl2);
                const float2 off_a = make_float2(-mn_a, -mn_a), off_b = make_float2(-mn_b, -mn_b);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    float2 ya = fma2(make_float2(xa[2 * r], xa[2 * r + 1]), scale, off_a);
                    float2 yb = fma2(make_float2(xb[2 * r], xb[2 * r + 1]), scale, off_b);
                    if (kvalid < kTile) {  // a scale of 0 would leave the padding at 0
                        const int k = 8 * r + 2 * q4;
                        if (k >= kvalid) ya.x = yb.x = -INFINITY;
                        if (k + 1 >= kvalid) ya.y = yb.y = -INFINITY;
                    }
                    ya = make_float2(ex2(ya.x), ex2(ya.y));
                    yb = make_float2(ex2(yb.x), ex2(yb.y));
                    sum_a = add2(sum_a, ya);
                    sum_b = add2(sum_b, yb);
                    const __nv_bfloat162 x = __floats2bfloat162_rn(ya.x, ya.y);
                    const __nv_bfloat162 y = __floats2bfloat162_rn(yb.x, yb.y);
                    pa[r] = *reinterpret_cast<const uint32_t *>(&x);
                    pb[r] = *reinterpret_cast<const uint32_t *>(&y);
                }
                la = sum_a.x + sum_a.y;
                lb = sum_b.x + sum_b.y;
            } else {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float a0 = ex2(xa[2 * r] - mn_a), a1 = ex2(xa[2 * r + 1] - mn_a);
                    const float b0 = ex2(xb[2 * r] - mn_b), b1 = ex2(xb[2 * r + 1] - mn_b);
                    la += a0 + a1;
                    lb += b0 + b1;
                    __nv_bfloat162 x = __floats2bfloat162_rn(a0, a1);
                    __nv_bfloat162 y = __floats2bfloat162_rn(b0, b1);
                    pa[r] = *reinterpret_cast<uint32_t *>(&x);
                    pb[r] = *reinterpret_cast<uint32_t *>(&y);
                }
            }
            // O belongs to P V of the previous tile until it is done: only a
            // rescale has to wait for it (P goes to this tile's own stage)
            const bool rescale = __any_sync(0xffffffffu, (grow_a || grow_b) && n > 0);
            if (rescale && ok)
                ok = warp_wait(&sm.kv_empty[(n - 1) % kStages], ((n - 1) / kStages) & 1,
                               abort_flag, status);
            if (ok && rescale) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t w[32];
                    tmem_ld_16x256b_x8(tmem + lane_hi + 64 * c, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        w[4 * r] = __float_as_uint(__uint_as_float(w[4 * r]) * f_a);
                        w[4 * r + 1] = __float_as_uint(__uint_as_float(w[4 * r + 1]) * f_a);
                        w[4 * r + 2] = __float_as_uint(__uint_as_float(w[4 * r + 2]) * f_b);
                        w[4 * r + 3] = __float_as_uint(__uint_as_float(w[4 * r + 3]) * f_b);
                    }
                    tmem_st_16x256b_x8(tmem + lane_hi + 64 * c, w);
                }
                tmem_wait_st();
            }
            l_a = l_a * f_a + la;
            l_b = l_b * f_b + lb;
            m_a = mn_a;
            m_b = mn_b;
            // P's heads 16j + 8h .. + 7, keys 8r .. 8r + 7 are an 8 x 8 matrix as
            // the lanes hold it: four matrices per store, in the rope block of
            // this tile's stage (S has read it: s_full)
            const uint32_t pbase = smem_u32(sm.kv[n % kStages]) + kPOffset + p_at;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t(&ph)[8] = h == 0 ? pa : pb;
#pragma unroll
                for (int r = 0; r < 8; r += 4)
                    store_matrix_x4(pbase + h * kGroupBytes + (((r + p_key) ^ p_row) << 4), ph[r],
                                    ph[r + 1], ph[r + 2], ph[r + 3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[n % kStages]);
        }
        if (ok && T > 0) ok = warp_wait(&sm.o_final, 0, abort_flag, status);
        tc_fence_after();
        // full row sums: the four threads of a head each hold a quarter
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
        constexpr float kUp = is_fp4(kKv) ? kFp4Up : 1.f;
        const float inv_a = (ok && l_a > 0.f) ? 1.f / l_a * kUp : 0.f;
        const float inv_b = (ok && l_b > 0.f) ? 1.f / l_b * kUp : 0.f;
        // the helpers write the second half of the columns
        if (q4 == 0) {
            sm.inv[ha] = inv_a;
            sm.inv[hb] = inv_b;
        }
        named_barrier(kOutBarrier, 256);
        write_output<kKv>(sm, a, t, split, hh, j, 0, ok && T > 0, tmem + lane_hi);
        if (q4 == 0) {
            const float lse_a = (ok && l_a > 0.f) ? (m_a + log2f(l_a)) * kLn2 : -INFINITY;
            const float lse_b = (ok && l_b > 0.f) ? (m_b + log2f(l_b)) * kLn2 : -INFINITY;
            const int64_t row_a = (int64_t)t * 128 + kHeadsCta * hh + ha;
            const int64_t row_b = row_a + 8;
            if (a.splits == 1) {
                if (a.lse != nullptr) {
                    a.lse[row_a] = lse_a;
                    a.lse[row_b] = lse_b;
                }
            } else {
                const int64_t base = ((int64_t)t * a.splits + split) * 128 + kHeadsCta * hh;
                a.lse_part[base + ha] = lse_a;
                a.lse_part[base + hb] = lse_b;
            }
        }
    } else if (warp >= 1) {
        // ---------------------------------------------- row producers ---
        // ring stage 2 holds Q until the softmax warps have moved it to TMEM
        produce_rows<kKv>(p, rows + j0 * kTile, T, producer_index(warp), sm.kv, sm.kv_full,
                          sm.kv_empty, &sm.q_ready, 2, abort_flag, status);
        if (warp >= 4 && warp < 8) {  // their rows done, they help with the output
            const bool done = T > 0 && warp_wait(&sm.o_final, 0, abort_flag, status);
            tc_fence_after();
            named_barrier(kOutBarrier, 256);
            write_output<kKv>(sm, a, t, split, hh, warp - 4, 1, done,
                              tmem + (static_cast<uint32_t>(32 * (warp - 4) + kLaneO) << 16));
        }
    } else if (T > 0) {
        // ------------------------------------------------- MMA issuer ---
        // One elected lane waits and issues: with the whole warp waiting and meeting
        // again around each branch, in a sub-partition that two producers and a
        // softmax warp keep busy, the steps between the MMAs took 500 of 2700 cycles a
        // tile (512 queries: 375 us over MXFP4 and 363 over bf16, so 395 and 384).
        // S of the next tile goes out before P V of this one, so that the tensor
        // pipe works while the softmax does; the two then alternate.
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        constexpr uint32_t id_s = instr_desc(64, kTile, 1 /*bf16*/, 0, 0);
        constexpr uint32_t id_pv = instr_desc(64, 256, 1 /*bf16*/, 0, 1);
        if (elect_one()) {
            bool ok = mbar_wait(&sm.q_ready, 0, abort_flag, status);
            for (int n = 0; ok && n <= T; ++n) {
                if (n < T) {  // S(n): its S buffer is free since P V (n - 2) was issued
                    const int st = n % kStages;
                    ok = mbar_wait(&sm.kv_full[st], (n / kStages) & 1, abort_flag, status);
                    if (!ok) break;
                    if constexpr (kKv == SA_BF16) fence_proxy_async_smem();  // cp.async rows
                    tc_fence_after();
                    const uint32_t d = tm + kColS + kTile * (n & 1);
                    const uint32_t stage = smem_u32(sm.kv[st]);
#pragma unroll  // 36 MMAs straight-line: measured faster than a loop over the blocks
                    for (int b = 0; b < kBlocks; ++b) {
                        const uint64_t bd = desc_kmajor_sw128_sbo(stage + b * 1024, kGroupBytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 16 dims (32 bytes) per instruction
                            mma_bf16_ts(d, tm + kColQ + 32 * b + 8 * k, bd + 2 * k, id_s,
                                        (b | k) != 0);
                    }
                    mma_commit(&sm.s_full[n & 1]);
                }
                if (n > 0) {  // P V (n - 1)
                    const int np = n - 1, st = np % kStages;
                    const uint32_t stage = smem_u32(sm.kv[st]);
                    const uint64_t ad = desc_kmajor_sw128_sbo(stage + kPOffset, kGroupBytes);
                    ok = mbar_wait(&sm.p_full[st], (np / kStages) & 1, abort_flag, status);
                    if (!ok) break;
                    tc_fence_after();  // P's writers have fenced for the tensor core
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 16 keys (two groups) per instruction
                            mma_bf16(tm + (kLaneO << 16) + 256 * half, ad + 2 * k,
                                     desc_mnmajor_sw128(stage + 4 * half * 1024 +
                                                            2 * k * kGroupBytes,
                                                        1024, kGroupBytes),
                                     id_pv, (np > 0 || k > 0) ? 1u : 0u);
                    }
                    mma_commit(&sm.kv_empty[st]);
                }
            }
        }
        __syncwarp();
        // o_final: every MMA issued above (all P V of the tiles) has completed;
        // after a timeout too, so that TMEM is never released under an MMA
        if (elect_one()) mma_commit(&sm.o_final);
        __syncwarp();
        int never = 0;
        warp_wait(&sm.o_final, 0, &never, status);
    }
    // with no tiles nobody waited for Q: its copy must land before the CTA ends
    if (warp == 0 && lane == 0 && T == 0) mbar_wait(&sm.q_full, 0, abort_flag, status);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// out = sum_s w_s o_s with w_s = exp(lse_s - lse), lse = log sum_s exp(lse_s).
// One CTA per (query, head): the split weights are computed once in shared
// memory, then each thread merges four output dims over all splits with the
// partial loads unrolled.
constexpr int kMaxSplits = 128;
__global__ void __launch_bounds__(128)
sfa_combine_kernel(const float *__restrict__ o_part, const float *__restrict__ lse_part,
                   int32_t splits, void *out, int32_t out_dtype, float *lse) {
    pdl_wait();
    pdl_trigger();
    __shared__ float w_s[kMaxSplits];
    const int64_t row = blockIdx.x;  // t * 128 + head
    const int64_t t = row >> 7, head = row & 127;
    const float4 *src = reinterpret_cast<const float4 *>(o_part + (t * splits * 128 + head) * kDl) +
                        threadIdx.x;
    const int64_t stride = 128 * kDl / 4;  // one split, in float4
    // sixteen splits' rows in flight, the first ones while the weights are computed
    constexpr int kAhead = 16;
    float4 v[kAhead];
    auto load = [&](int s0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (s0 + i < splits) v[i] = src[(s0 + i) * stride];
    };
    load(0);
    if (threadIdx.x < splits) w_s[threadIdx.x] = lse_part[(t * splits + threadIdx.x) * 128 + head];
    __syncthreads();
    if (threadIdx.x < 32) {
        float m = -INFINITY;
        for (int s = threadIdx.x; s < splits; s += 32) m = fmaxf(m, w_s[s]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float sum = 0.f;
        for (int s = threadIdx.x; s < splits; s += 32) {
            const float ls = w_s[s];
            const float w = (m == -INFINITY || ls == -INFINITY) ? 0.f : __expf(ls - m);
            w_s[s] = w;
            sum += w;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        for (int s = threadIdx.x; s < splits; s += 32) w_s[s] *= inv;
        if (lse != nullptr && threadIdx.x == 0) lse[row] = sum > 0.f ? m + logf(sum) : -INFINITY;
    }
    __syncthreads();
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < splits; s0 += kAhead) {
        if (s0 > 0) load(s0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s0 + i >= splits) break;
            const float w = w_s[s0 + i];
            acc[0] += w * v[i].x;
            acc[1] += w * v[i].y;
            acc[2] += w * v[i].z;
            acc[3] += w * v[i].w;
        }
    }
    if (out_dtype == SA_BF16) {
        __nv_bfloat162 a = __floats2bfloat162_rn(acc[0], acc[1]);
        __nv_bfloat162 b = __floats2bfloat162_rn(acc[2], acc[3]);
        uint2 w = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
        reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + row * kDl)[threadIdx.x] = w;
    } else {
        reinterpret_cast<float4 *>(static_cast<float *>(out) + row * kDl)[threadIdx.x] =
            make_float4(acc[0], acc[1], acc[2], acc[3]);
    }
}

}  // namespace

bool sfa_mma_supported(const PathParams &p, int32_t top_k) {
    const bool kv_ok = p.kv_dtype == SA_BF16 ||
                       ((p.kv_dtype == SA_E4M3 || is_fp4(p.kv_dtype)) && p.kv_rope != nullptr &&
                        p.kv_scale != nullptr);
    return kv_ok && p.q_dtype == SA_BF16 && p.heads == 128 &&
           p.d_latent == kDl && p.d_rope == kDr && top_k <= kMaxK &&
           (int64_t)p.num_pages * 64 < (int64_t(1) << 31);
}

int32_t sfa_splits(int32_t n_q, int32_t top_k) {
    const int32_t ctas = std::max(1, num_sms());
    const int32_t max_tiles = (top_k + kTile - 1) / kTile;
    if (n_q <= 0) return 1;
    return std::max(1, std::min({max_tiles, ctas / (2 * n_q), kMaxSplits}));
}

int32_t sfa_rows_ld(int32_t top_k) { return (int32_t)round_up(top_k > 0 ? top_k : 1, kTile); }

cudaError_t launch_sfa_mma(const PathParams &p, const int32_t *idx, int32_t top_k, int32_t splits,
                           const int32_t *rows, const int32_t *n_valid, void *out,
                           int32_t out_dtype, float *lse, float *o_part, float *lse_part,
                           cudaStream_t s) {
    if (p.n_q == 0) return cudaSuccess;
    cudaError_t e;
    CUtensorMap tq;
    if (!encode_tmap_2d(&tq, 2, p.q, kD, (uint64_t)p.n_q * 128, kD * 2, 64, kHeadsCta, true))
        return cudaErrorInvalidValue;
    SfaArgs a{p,     rows, n_valid,   sfa_rows_ld(top_k), idx,    top_k,
              splits, out,  out_dtype, lse,                o_part, lse_part};
    const size_t smem = sizeof(SfaSmem) + 1024;
    const auto kernel = p.kv_dtype == SA_BF16    ? sfa_mma_kernel<SA_BF16>
                        : p.kv_dtype == SA_E4M3  ? sfa_mma_kernel<SA_E4M3>
                        : p.kv_dtype == SA_MXFP4 ? sfa_mma_kernel<SA_MXFP4>
                                                 : sfa_mma_kernel<SA_NVFP4>;
    e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    const int threads = is_fp4(p.kv_dtype) ? kCtaThreads<SA_MXFP4> : kCtaThreads<SA_BF16>;
    const int64_t grid = 2 * (int64_t)p.n_q * splits;
    count_launch();
    e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, s, tq, a);
    if (e != cudaSuccess || splits == 1) return e;
    count_launch();
    return launch_pdl(sfa_combine_kernel, dim3(static_cast<unsigned>(p.n_q * 128)), dim3(128), 0,
                      s, (const float *)o_part, (const float *)lse_part, splits, out, out_dtype,
                      lse);
}

}  // namespace sa
