// prep.cu -- input preparation before the indexer: FP8 quantisation of the
// indexer query and the append of new tokens to the paged caches
// ("Optimizing Next-Gen LLM Inference", §3.2 and the §4 table; "Inference
// Acceleration for New Large Model Architectures", §3.3 and §4.1-4.2).
//
// Dynamic FP8 quantisation, per group of values, in fp32:
//     amax = max |x|,  scale = amax / 448 (1 for an all-zero group),
//     code = e4m3(x / scale), round to nearest even, saturated to +-448,
// so the largest magnitude of a group lands on e4m3's largest finite value.
// The division is IEEE round-to-nearest (__fdiv_rn): the codes depend on it.
//
// A 4-bit latent takes, per group of 32 (MXFP4) or 16 values (NVFP4), a scale
// byte that puts the largest magnitude near e2m1's 6: 2^(floor(log2 amax) - 2),
// or e4m3(amax / 6); code = e2m1(x / scale), nearest even, saturated to +-6.  e2m1
// has neither infinity nor NaN, so a group that holds one takes the scale byte that
// is NaN: the whole group reads back as NaN.
//
// The kernels are memory-bound: one warp per quantised row of the query
// (d_index values), per token of a 4-bit cache and per row read back, one CTA
// per other appended token.
#include <cfloat>

#include "common.cuh"
#include "internal.h"
#include "prep.h"

namespace sa {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr int kAppendThreads = 128;
constexpr int kMaxGroups = 32;  // latent groups per token: d_latent <= 512, group >= 16

__device__ __forceinline__ float fp8_scale(float amax) {
    return amax > 0.0f ? __fdiv_rn(amax, kE4m3Max) : 1.0f;
}

__device__ __forceinline__ uint8_t to_e4m3(float x, float scale) {
    return static_cast<uint8_t>(
        __nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ float load_value(const void *base, int64_t i, bool bf16) {
    return bf16 ? bf16_bits_to_float(static_cast<const uint16_t *>(base)[i])
                : static_cast<const float *>(base)[i];
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// ---------------------------------------------------------------------------
// Query quantisation.  Rows of d = 32 * C values: lane l holds values
// [l*C, l*C + C) (one 8- or 16-byte load for bf16, one or two 16-byte loads
// for fp32) and stores its C codes with one 4- or 8-byte store.
// ---------------------------------------------------------------------------
template <int C, bool BF16>
__global__ void __launch_bounds__(256) quantize_rows_vec_kernel(const void *__restrict__ in,
                                                                int64_t n_rows,
                                                                uint8_t *__restrict__ codes,
                                                                float *__restrict__ scales) {
    static_assert(C == 4 || C == 8, "4 or 8 values per lane");
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < n_rows;
         r += warps) {
        const int64_t base = r * (32 * C) + (int64_t)lane * C;
        float v[C];
        if constexpr (BF16) {
            const uint16_t *src = static_cast<const uint16_t *>(in) + base;
            uint32_t w[C / 2];
            if constexpr (C == 4) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(src));
                w[0] = u.x, w[1] = u.y;
            } else {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src));
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
            }
#pragma unroll
            for (int j = 0; j < C / 2; j++) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        } else {
            const float *src = static_cast<const float *>(in) + base;
#pragma unroll
            for (int j = 0; j < C; j += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(src + j));
                v[j] = f.x, v[j + 1] = f.y, v[j + 2] = f.z, v[j + 3] = f.w;
            }
        }
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < C; j++) amax = fmaxf(amax, fabsf(v[j]));
        const float scale = fp8_scale(warp_max(amax));
        uint32_t packed[C / 4];
#pragma unroll
        for (int j = 0; j < C / 4; j++) {
            packed[j] = 0;
#pragma unroll
            for (int b = 0; b < 4; b++)
                packed[j] |= static_cast<uint32_t>(to_e4m3(v[4 * j + b], scale)) << (8 * b);
        }
        if constexpr (C == 4) {
            *reinterpret_cast<uint32_t *>(codes + base) = packed[0];
        } else {
            *reinterpret_cast<uint2 *>(codes + base) = make_uint2(packed[0], packed[1]);
        }
        if (lane == 0) scales[r] = scale;
    }
}

// Any row length: lanes stride over the row (coalesced), two passes.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const void *__restrict__ in,
                                                            int32_t bf16, int64_t n_rows,
                                                            int32_t d,
                                                            uint8_t *__restrict__ codes,
                                                            float *__restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < n_rows;
         r += warps) {
        const int64_t base = r * d;
        float amax = 0.0f;
        for (int32_t i = lane; i < d; i += 32)
            amax = fmaxf(amax, fabsf(load_value(in, base + i, bf16 != 0)));
        const float scale = fp8_scale(warp_max(amax));
        for (int32_t i = lane; i < d; i += 32)
            codes[base + i] = to_e4m3(load_value(in, base + i, bf16 != 0), scale);
        if (lane == 0) scales[r] = scale;
    }
}

// ---------------------------------------------------------------------------
// Append.  One CTA per new token (grid-stride); group maxima go through
// shared-memory atomics on the bit patterns of |x| (non-negative floats order
// like their bits).
// ---------------------------------------------------------------------------

// n values starting at element s0 of src -> codes at dst[0..n) and one scale
// per group of g values at scl[0..n/g).  Every thread of the CTA calls it.
__device__ void quantize_groups(const void *src, int64_t s0, bool bf16, int32_t n, int32_t g,
                                uint8_t *dst, float *scl, int32_t *gmax) {
    const int32_t groups = n / g;
    for (int32_t i = threadIdx.x; i < groups; i += blockDim.x) gmax[i] = 0;
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += blockDim.x)
        atomicMax(&gmax[i / g], __float_as_int(fabsf(load_value(src, s0 + i, bf16))));
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += blockDim.x)
        dst[i] = to_e4m3(load_value(src, s0 + i, bf16), fp8_scale(__int_as_float(gmax[i / g])));
    for (int32_t i = threadIdx.x; i < groups; i += blockDim.x)
        scl[i] = fp8_scale(__int_as_float(gmax[i]));
    __syncthreads();  // gmax is reused by the next call
}

// The scale bytes that are NaN.
constexpr uint32_t kE8m0Nan = 255u, kE4m3Nan = 0x7Fu;

// amax of a group (NaN if one of its values is) -> its scale byte of a 4-bit latent.
__device__ __forceinline__ uint32_t fp4_scale_byte(int32_t dtype, float amax) {
    if (!(amax <= FLT_MAX)) return dtype == SA_MXFP4 ? kE8m0Nan : kE4m3Nan;
    if (dtype == SA_MXFP4) {
        if (!(amax > 0.0f)) return 127u;
        // floor(log2 amax): the exponent field of a normal number; of a subnormal
        // one the scale is clamped to 2^-127 either way
        const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 255u) - 2;
        return static_cast<uint32_t>(max(e, 0));
    }
    const float s = amax > 0.0f ? fminf(__fdiv_rn(amax, 6.0f), kE4m3Max) : 1.0f;
    return static_cast<uint32_t>(__nv_cvt_float_to_fp8(s, __NV_SATFINITE, __NV_E4M3));
}

// Sixteen values -> eight bytes of codes of a 4-bit latent.  An E8M0 scale is a
// power of two, and a product with its reciprocal the same as the quotient.  An
// e4m3 scale s is divided by (IEEE) when the values are fp32.  A bf16 value x
// has 8 significant bits and a border m s between two codes at most 7 (m: 3, s:
// 4), so x / s either is m or differs from it by 2^-8 of it or more: the product
// with fp32's 1 / s, within 2^-23 of x / s and rounded to 16 bits, is m in the
// one case and on x / s's side of it in the other, and the code is the
// quotient's (a division per value: 40001 rows appended in 35 us).  A scale
// that rounded to 0, or is NaN, gives zeros.
template <int kKv, bool kBf16>
__device__ __forceinline__ uint2 to_fp4x16(const float (&x)[16], uint32_t scale_byte) {
    float q[16];
    if constexpr (kKv == SA_MXFP4) {
        if (scale_byte == kE8m0Nan) return make_uint2(0u, 0u);
        // 2^(127 - byte): byte <= 252, so neither end leaves the normal range
        const float inv = __uint_as_float((254u - scale_byte) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = x[i] * inv;
    } else {
        const float scale = fp4_scale_value(SA_NVFP4, scale_byte);
        if constexpr (kBf16) {
            if (!(scale > 0.0f)) return make_uint2(0u, 0u);
            const float inv = __fdiv_rn(1.0f, scale);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                q[i] = __uint_as_float((__float_as_uint(x[i] * inv) + 0x80u) & 0xFFFFFF00u);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) q[i] = scale > 0.0f ? __fdiv_rn(x[i], scale) : 0.0f;
        }
    }
    return make_uint2(float_to_e2m1x8(q), float_to_e2m1x8(q + 8));
}

__device__ __forceinline__ uint16_t to_bf16_bits(const void *src, int64_t i, bool bf16) {
    if (bf16) return static_cast<const uint16_t *>(src)[i];
    return __bfloat16_as_ushort(__float2bfloat16_rn(static_cast<const float *>(src)[i]));
}

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
    __shared__ int32_t gmax[kMaxGroups];
    const bool bf16 = p.in_bf16 != 0;
    for (int32_t t = blockIdx.x; t < p.n_new; t += gridDim.x) {
        const int32_t seq = __ldg(p.seq + t), pos = __ldg(p.pos + t);
        if (seq < 0 || seq >= p.batch || pos < 0 || (pos >> 6) >= p.max_pages) {
            if (threadIdx.x == 0) report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_POSITION);
            continue;  // uniform over the CTA
        }
        const int64_t row = phys_row(p.page_table, p.max_pages, p.num_pages, seq, pos);
        if (row < 0) {
            if (threadIdx.x == 0) report(p.status, SA_ERR_DEVICE_FAULT, SA_DETAIL_BAD_PAGE);
            continue;
        }
        if (p.k_new != nullptr) {
            const int64_t s0 = (int64_t)t * p.d_index;
            if (p.index_dtype == SA_E4M3) {
                quantize_groups(p.k_new, s0, bf16, p.d_index, p.d_index,
                                static_cast<uint8_t *>(p.k_index) + row * p.d_index,
                                p.k_index_scale + row, gmax);
            } else if (p.index_dtype == SA_BF16) {
                uint16_t *dst = static_cast<uint16_t *>(p.k_index) + row * p.d_index;
                for (int32_t i = threadIdx.x; i < p.d_index; i += blockDim.x)
                    dst[i] = to_bf16_bits(p.k_new, s0 + i, bf16);
            } else {
                float *dst = static_cast<float *>(p.k_index) + row * p.d_index;
                for (int32_t i = threadIdx.x; i < p.d_index; i += blockDim.x)
                    dst[i] = load_value(p.k_new, s0 + i, bf16);
            }
        }
        if (p.kv_new != nullptr) {
            const int32_t D = p.d_latent + p.d_rope;
            const int64_t s0 = (int64_t)t * D;
            if (p.kv_dtype == SA_E4M3) {
                const int32_t groups = p.d_latent / p.kv_scale_dims;
                quantize_groups(p.kv_new, s0, bf16, p.d_latent, p.kv_scale_dims,
                                static_cast<uint8_t *>(p.kv) + row * p.d_latent,
                                p.kv_scale + row * groups, gmax);
                uint16_t *rope = static_cast<uint16_t *>(p.kv_rope) + row * p.d_rope;
                for (int32_t i = threadIdx.x; i < p.d_rope; i += blockDim.x)
                    rope[i] = to_bf16_bits(p.kv_new, s0 + p.d_latent + i, bf16);
            } else if (p.kv_dtype == SA_BF16) {
                uint16_t *dst = static_cast<uint16_t *>(p.kv) + row * D;
                for (int32_t i = threadIdx.x; i < D; i += blockDim.x)
                    dst[i] = to_bf16_bits(p.kv_new, s0 + i, bf16);
            } else {
                float *dst = static_cast<float *>(p.kv) + row * D;
                for (int32_t i = threadIdx.x; i < D; i += blockDim.x)
                    dst[i] = load_value(p.kv_new, s0 + i, bf16);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Append to a 4-bit latent cache, and rows back out of any latent pool: one
// warp per token, a lane takes 16 dims at a time (32 or 64 bytes of the row, 8
// of the codes), so that every access is whole 16- or 8-byte pieces and a
// warp's are contiguous.  40001 rows written and read back: 19.2 us of traffic.
// ---------------------------------------------------------------------------
constexpr int kWarpThreads = 256;
constexpr int kWarpTokens = kWarpThreads / 32;

// N values to element i of dst, rounded to nearest even for bf16.
template <int N>
__device__ __forceinline__ void store_values(void *dst, int64_t i, bool bf16,
                                             const float (&x)[N]) {
    if (bf16) {
        uint4 *d = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + i);
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 b =
                    __floats2bfloat162_rn(x[8 * j + 2 * k], x[8 * j + 2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t *>(&b);
            }
            d[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(dst) + i);
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
            d[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    }
}

// Physical row of a token, or -1 and why it has none.
__device__ __forceinline__ int64_t token_row(const int32_t *page_table, int32_t batch,
                                             int32_t max_pages, int32_t num_pages, int32_t seq,
                                             int32_t pos, int32_t &detail) {
    detail = SA_DETAIL_BAD_POSITION;
    if (seq < 0 || seq >= batch || pos < 0 || (pos >> 6) >= max_pages) return -1;
    const int64_t row = phys_row(page_table, max_pages, num_pages, seq, pos);
    detail = row < 0 ? SA_DETAIL_BAD_PAGE : SA_DETAIL_NONE;
    return row;
}

// Calls of at most this many tokens need no cleared status word: their first CTA
// looks every token up once more and writes the word, error or not (a clearing
// memset in front costs a call of 64 tokens about 2 us on either side).
constexpr int32_t kStatusTokens = 2048;

// Called by every thread of the first CTA of such a launch.
__device__ void write_status(const int32_t *page_table, int32_t batch, int32_t max_pages,
                             int32_t num_pages, int32_t n, const int32_t *seq, const int32_t *pos,
                             int32_t *status) {
    __shared__ int32_t first_s[kWarpTokens];
    int32_t first = INT32_MAX;  // (token << 2 | detail) of the first one that has no row
    for (int32_t i = threadIdx.x; i < n; i += kWarpThreads) {
        int32_t detail;
        (void)token_row(page_table, batch, max_pages, num_pages, __ldg(seq + i), __ldg(pos + i),
                        detail);
        if (detail != SA_DETAIL_NONE) first = min(first, i << 2 | detail);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
    if ((threadIdx.x & 31) == 0) first_s[threadIdx.x >> 5] = first;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarpTokens; ++w) first = min(first, first_s[w]);
        status[0] = first == INT32_MAX ? SA_OK : SA_ERR_DEVICE_FAULT;
        status[1] = first == INT32_MAX ? SA_DETAIL_NONE : first & 3;
    }
}

// A warp takes `block` consecutive tokens: its lanes look their rows up at once,
// then kTokens of them at a time have their loads in flight together.
constexpr int kMaxBlock = 32;

// 16-byte pieces of N values, as they are stored.
template <int N, bool kBf16>
struct RawValues {
    uint4 w[kBf16 ? N / 8 : N / 4];

    __device__ __forceinline__ void load(const void *src, int64_t i) {
        const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(src) +
                                                         i * (kBf16 ? 2 : 4));
#pragma unroll
        for (int j = 0; j < (kBf16 ? N / 8 : N / 4); ++j) w[j] = __ldcs(s + j);
    }
    __device__ __forceinline__ void values(float (&x)[N]) const {
        const uint32_t *u = reinterpret_cast<const uint32_t *>(w);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            x[2 * j] = __uint_as_float(kBf16 ? u[j] << 16 : u[2 * j]);
            x[2 * j + 1] = __uint_as_float(kBf16 ? u[j] & 0xffff0000u : u[2 * j + 1]);
        }
    }
};

template <int kKv, bool kBf16>
__global__ void __launch_bounds__(kWarpThreads)
append_fp4_kernel(const AppendParams p, int32_t block) {
    constexpr int kTokens = kBf16 ? 3 : 2;
    const int lane = threadIdx.x & 31;
    const int32_t D = p.d_latent + p.d_rope, chunks = p.d_latent / 16;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarpTokens + (threadIdx.x >> 5)) * block;
    const int32_t count = (int32_t)min((int64_t)block, p.n_new - t0);
    if (p.set_status && blockIdx.x == 0)
        write_status(p.page_table, p.batch, p.max_pages, p.num_pages, p.n_new, p.seq, p.pos,
                     p.status);
    if (count <= 0) return;
    int32_t my_seq = 0, my_pos = 0;
    if (lane < count) {
        my_seq = __ldg(p.seq + t0 + lane);
        my_pos = __ldg(p.pos + t0 + lane);
    }
    int64_t my_row = -1;
    for (int32_t u0 = 0; u0 < count; u0 += kTokens) {
        RawValues<16, kBf16> raw[kTokens];
        RawValues<8, kBf16> raw_rope[kTokens];
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            const int64_t s0 = (t0 + u0 + u) * D;
            if (u0 + u >= count) break;
            if (lane < chunks) raw[u].load(p.kv_new, s0 + 16 * lane);
            if (8 * lane < p.d_rope) raw_rope[u].load(p.kv_new, s0 + p.d_latent + 8 * lane);
        }
        if (u0 == 0 && lane < count) {  // while the first rows are on their way
            int32_t detail;
            my_row = token_row(p.page_table, p.batch, p.max_pages, p.num_pages, my_seq, my_pos,
                               detail);
            if (my_row < 0 && !p.set_status) report(p.status, SA_ERR_DEVICE_FAULT, detail);
        }
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            const int64_t row = __shfl_sync(0xffffffffu, my_row, (u0 + u) & 31);
            if (u0 + u >= count || row < 0) continue;
            if (lane < chunks) {  // an even number of lanes, at most 32: d_latent <= 512
                uint2 *codes = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.kv) +
                                                         row * (p.d_latent / 2));
                uint8_t *scales =
                    reinterpret_cast<uint8_t *>(p.kv_scale) + row * (p.d_latent / fp4_group(kKv));
                float x[16], amax = 0.0f;
                raw[u].values(x);
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = max_keep_nan(amax, fabsf(x[i]));
                if (kKv == SA_MXFP4) {
                    const uint32_t lanes = 0xffffffffu >> (32 - chunks);
                    amax = max_keep_nan(amax, __shfl_xor_sync(lanes, amax, 1));
                }
                const uint32_t byte = fp4_scale_byte(kKv, amax);
                codes[lane] = to_fp4x16<kKv, kBf16>(x, byte);
                if (kKv == SA_NVFP4) scales[lane] = static_cast<uint8_t>(byte);
                else if ((lane & 1) == 0) scales[lane >> 1] = static_cast<uint8_t>(byte);
            }
            uint16_t *rope = static_cast<uint16_t *>(p.kv_rope) + row * p.d_rope;
            for (int32_t c = lane; 8 * c < p.d_rope; c += 32) {
                float x[8];
                if (c != lane)
                    raw_rope[u].load(p.kv_new, (t0 + u0 + u) * D + p.d_latent + 8 * c);
                raw_rope[u].values(x);
                store_values(rope, 8 * c, true, x);
            }
        }
    }
}

// Sixteen dims (piece c) of a row's latent -- of the whole row where latent and
// rope lie in one (bf16, fp32) -- as they are stored, and their values.
template <int kKv>
struct LatentPiece {
    uint4 w[kKv == SA_F32 ? 4 : kKv == SA_BF16 ? 2 : 1];
    float scale;

    __device__ __forceinline__ void load(const PathParams &p, int64_t row, int c) {
        const uint8_t *kv = static_cast<const uint8_t *>(p.kv);
        const int32_t dl = p.d_latent, D = dl + p.d_rope;
        if constexpr (kKv == SA_F32 || kKv == SA_BF16) {
            constexpr int kBytes = kKv == SA_F32 ? 4 : 2;
            const uint4 *s = reinterpret_cast<const uint4 *>(kv + (row * D + 16 * c) * kBytes);
#pragma unroll
            for (int j = 0; j < kBytes; ++j) w[j] = __ldg(s + j);
        } else if constexpr (kKv == SA_E4M3) {
            w[0] = __ldg(reinterpret_cast<const uint4 *>(kv + row * dl) + c);
            scale = kv_scale_at(p, row, 16 * c);
        } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(kv + row * (dl / 2)) + c);
            w[0] = make_uint4(u.x, u.y, 0u, 0u);
            scale = fp4_scale_value(
                kKv, __ldg(reinterpret_cast<const uint8_t *>(p.kv_scale) +
                           row * (dl / fp4_group(kKv)) + 16 * c / fp4_group(kKv)));
        }
    }

    __device__ __forceinline__ void values(float (&x)[16]) const {
        const uint32_t *u = reinterpret_cast<const uint32_t *>(w);
        if constexpr (is_fp4(kKv)) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                e2m1x8_to_float(u[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[8 * j + i] = v[i] * scale;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (kKv == SA_F32) {
                    x[2 * j] = __uint_as_float(u[2 * j]);
                    x[2 * j + 1] = __uint_as_float(u[2 * j + 1]);
                } else if constexpr (kKv == SA_BF16) {
                    x[2 * j] = __uint_as_float(u[j] << 16);
                    x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
                } else {
                    const float2 f =
                        e4m3x2_to_float2(static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1))));
                    x[2 * j] = f.x * scale;
                    x[2 * j + 1] = f.y * scale;
                }
            }
        }
    }
};

// Blocks of tokens as in append_fp4_kernel.  kWide: rows are whole 16-dim
// pieces; otherwise a lane takes single values.
template <int kKv, bool kWide>
__global__ void __launch_bounds__(kWarpThreads)
read_kernel(const PathParams p, int32_t n, const int32_t *__restrict__ seq_of,
            const int32_t *__restrict__ pos_of, void *out, bool out_bf16, int32_t block,
            bool set_status) {
    constexpr int kTokens = kKv == SA_F32 ? 2 : 4;
    const int lane = threadIdx.x & 31;
    const int32_t dl = p.d_latent, dr = p.d_rope, D = dl + dr;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarpTokens + (threadIdx.x >> 5)) * block;
    const int32_t count = (int32_t)min((int64_t)block, n - t0);
    if (set_status && blockIdx.x == 0)
        write_status(p.page_table, p.batch, p.max_pages, p.num_pages, n, seq_of, pos_of, p.status);
    if (count <= 0) return;
    int64_t my_row = -1;
    if (lane < count) {
        int32_t detail;
        my_row = token_row(p.page_table, p.batch, p.max_pages, p.num_pages,
                           __ldg(seq_of + t0 + lane), __ldg(pos_of + t0 + lane), detail);
        if (my_row < 0 && !set_status) report(p.status, SA_ERR_DEVICE_FAULT, detail);
    }
    if constexpr (!kWide) {
        for (int32_t u = 0; u < count; ++u) {
            const int64_t row = __shfl_sync(0xffffffffu, my_row, u);
            for (int32_t i = lane; i < D; i += 32) {
                const float v = row >= 0 ? kv_value_of<kKv>(p, row, i) : 0.0f;
                const int64_t o = (t0 + u) * D + i;
                if (out_bf16) static_cast<__nv_bfloat16 *>(out)[o] = __float2bfloat16_rn(v);
                else static_cast<float *>(out)[o] = v;
            }
        }
    } else {
        constexpr bool kOne = kKv == SA_BF16 || kKv == SA_F32;
        const int32_t pieces = (kOne ? D : dl) / 16, rope_pieces = kOne ? 0 : dr / 8;
        for (int32_t u0 = 0; u0 < count; u0 += kTokens) {
            int64_t row[kTokens];
#pragma unroll
            for (int u = 0; u < kTokens; ++u)
                row[u] = __shfl_sync(0xffffffffu, my_row, (u0 + u) & 31);
            for (int32_t c = lane; c < pieces || c < rope_pieces; c += 32) {
                LatentPiece<kKv> piece[kTokens];
                uint4 rope[kTokens];
#pragma unroll
                for (int u = 0; u < kTokens; ++u) {
                    if (u0 + u >= count || row[u] < 0) continue;
                    if (c < pieces) piece[u].load(p, row[u], c);
                    if (c < rope_pieces)
                        rope[u] = __ldg(reinterpret_cast<const uint4 *>(
                                            static_cast<const uint16_t *>(p.kv_rope) +
                                            row[u] * dr) +
                                        c);
                }
#pragma unroll
                for (int u = 0; u < kTokens; ++u) {
                    if (u0 + u >= count) break;
                    const int64_t o = (t0 + u0 + u) * D;
                    if (c < pieces) {
                        float x[16] = {};
                        if (row[u] >= 0) piece[u].values(x);
                        store_values(out, o + 16 * c, out_bf16, x);
                    }
                    if (c < rope_pieces) {
                        const uint32_t w[4] = {rope[u].x, rope[u].y, rope[u].z, rope[u].w};
                        float x[8] = {};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (row[u] < 0) break;
                            x[2 * j] = __uint_as_float(w[j] << 16);
                            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                        }
                        store_values(out, o + dl + 8 * c, out_bf16, x);
                    }
                }
            }
        }
    }
}

// Tokens per warp: one while the GPU has a warp for each (24 warps an SM; a decode
// step: the latency of one row), then as many as keep one wave, up to 32.
int32_t token_block(int64_t n) {
    return (int32_t)std::min<int64_t>(kMaxBlock, ceil_div(n, (int64_t)num_sms() * 24));
}
dim3 token_grid(int64_t n, int32_t block) {
    return dim3((unsigned)ceil_div(n, (int64_t)kWarpTokens * block));
}

template <int kKv>
cudaError_t launch_read_kv(const PathParams &p, int32_t n, const int32_t *seq, const int32_t *pos,
                           void *out, bool out_bf16, cudaStream_t s) {
    const bool one = kKv == SA_BF16 || kKv == SA_F32;
    const bool wide = one ? (p.d_latent + p.d_rope) % 16 == 0
                          : p.d_latent % 16 == 0 && p.d_rope % 8 == 0;
    const int32_t block = token_block(n);
    const auto kernel = wide ? read_kernel<kKv, true> : read_kernel<kKv, false>;
    count_launch();
    kernel<<<token_grid(n, block), kWarpThreads, 0, s>>>(p, n, seq, pos, out, out_bf16, block,
                                                      read_sets_status(n));
    return cudaGetLastError();
}

}  // namespace

bool read_sets_status(int32_t n) { return n > 0 && n <= kStatusTokens; }

cudaError_t launch_read(const PathParams &p, int32_t n, const int32_t *seq, const int32_t *pos,
                        void *out, int32_t out_dtype, cudaStream_t s) {
    if (n <= 0) return cudaSuccess;
    const bool bf16 = out_dtype == SA_BF16;
    switch (p.kv_dtype) {
    case SA_BF16: return launch_read_kv<SA_BF16>(p, n, seq, pos, out, bf16, s);
    case SA_F32: return launch_read_kv<SA_F32>(p, n, seq, pos, out, bf16, s);
    case SA_E4M3: return launch_read_kv<SA_E4M3>(p, n, seq, pos, out, bf16, s);
    case SA_MXFP4: return launch_read_kv<SA_MXFP4>(p, n, seq, pos, out, bf16, s);
    default: return launch_read_kv<SA_NVFP4>(p, n, seq, pos, out, bf16, s);
    }
}

cudaError_t launch_quantize_rows(const void *in, sa_dtype in_dtype, int64_t n_rows, int32_t d,
                                 uint8_t *codes, float *scales, cudaStream_t s) {
    if (n_rows <= 0) return cudaSuccess;
    constexpr int kThreads = 256, kWarps = kThreads / 32;
    const int64_t want = (n_rows + kWarps - 1) / kWarps;
    const int grid = (int)std::min<int64_t>(want, (int64_t)num_sms() * 16);
    const bool bf16 = in_dtype == SA_BF16;
    count_launch();
    if (d == 128) {
        if (bf16)
            quantize_rows_vec_kernel<4, true><<<grid, kThreads, 0, s>>>(in, n_rows, codes, scales);
        else
            quantize_rows_vec_kernel<4, false><<<grid, kThreads, 0, s>>>(in, n_rows, codes, scales);
    } else if (d == 256) {
        if (bf16)
            quantize_rows_vec_kernel<8, true><<<grid, kThreads, 0, s>>>(in, n_rows, codes, scales);
        else
            quantize_rows_vec_kernel<8, false><<<grid, kThreads, 0, s>>>(in, n_rows, codes, scales);
    } else {
        quantize_rows_kernel<<<grid, kThreads, 0, s>>>(in, bf16 ? 1 : 0, n_rows, d, codes, scales);
    }
    return cudaGetLastError();
}

template <int kKv>
static void launch_append_fp4(const AppendParams &p, cudaStream_t s) {
    const int32_t block = token_block(p.n_new);
    const auto kernel = p.in_bf16 ? append_fp4_kernel<kKv, true> : append_fp4_kernel<kKv, false>;
    count_launch();
    kernel<<<token_grid(p.n_new, block), kWarpThreads, 0, s>>>(p, block);
}

bool append_sets_status(int32_t kv_dtype, int32_t n_new, const void *k_new, const void *kv_new) {
    // with index keys a second kernel reports too
    return is_fp4(kv_dtype) && kv_new != nullptr && k_new == nullptr && n_new > 0 &&
           n_new <= kStatusTokens;
}

cudaError_t launch_append(const AppendParams &params, cudaStream_t s) {
    if (params.n_new <= 0) return cudaSuccess;
    AppendParams p = params;
    p.set_status = append_sets_status(p.kv_dtype, p.n_new, p.k_new, p.kv_new);
    if (is_fp4(p.kv_dtype) && p.kv_new != nullptr) {
        if (p.kv_dtype == SA_MXFP4) launch_append_fp4<SA_MXFP4>(p, s);
        else launch_append_fp4<SA_NVFP4>(p, s);
        p.kv_new = nullptr;
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || p.k_new == nullptr) return e;
    }
    const int grid = std::min(p.n_new, num_sms() * 16);
    count_launch();
    append_kernel<<<grid, kAppendThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sa
