// Rotary positions on the new tokens' queries and keys, fused with the cache
// write ("PagedAttention por dentro", section "La tabla de páginas (block
// table)": the new token's K/V go into the slot of its block), into pools of
// float32 or bfloat16 rows, or of E4M3 codes with one scale per block of 16
// tokens and KV head.
//
// Rotation.  A head's first rotary_dim elements are pairs (x0, x1), either
// element i with element i + rotary_dim / 2 or neighbours 2i and 2i + 1, turned
// by the angle p * theta_i of position p:
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin   (times the attention factor).
// Angles.  At far positions p * theta_i in 32 bits has lost the angle (p = 10^6:
// an error of 0.06 rad), so theta_i comes as a 64-bit fixed-point fraction of a
// full turn: the 64-bit product p * turns_i wraps at whole turns by itself and
// its upper half is the angle to 2^-32 of a turn at any position.
//
// Block scales.  A block's scale is the smallest power of two 2^e, e in
// [-32, 31], that holds its largest magnitude: amax <= 448 * 2^e.  E4M3 is a
// floating-point code, so a power of two loses no precision against amax / 448,
// the division of an element by it is exact, and a block whose scale grows when
// a row is appended has its earlier rows re-encoded without error (apart from
// codes that become subnormal).
#include <cuda_runtime.h>
#include <math.h>

#include <cmath>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kWindow = 32;          // entries of slot_mapping among which a block's tokens lie
constexpr int kMinExp = -32, kMaxExp = 31;

struct RopeArgs {
    const void *query, *key, *value;
    void *query_out;
    void *key_cache, *value_cache;
    float *k_scales, *v_scales;
    const int32_t *positions;
    const uint64_t *turns;
    const int64_t *slot_mapping;
    int32_t *status;
    int64_t q_stride, k_stride, v_stride, q_out_stride;   // elements between tokens
    float factor;
    int num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim;
    int interleaved;
    int num_blocks;
    int tokens_per_cta;              // of the row CTAs
    int row_ctas;                    // CTAs that turn rows; the rest take blocks
    int tile_tokens;                 // tokens of a block CTA
};

// cos and sin of position p's angle for one pair, times the attention factor
__device__ __forceinline__ float2 turn_of(int32_t p, uint64_t turns, float factor) {
    const uint64_t at = (uint64_t)(int64_t)p * turns;          // modulo one turn
    const float x = (float)(int32_t)(at >> 32) * 0x1p-31f;     // half turns, in [-1, 1]
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * factor, s * factor);
}

// N consecutive elements as floats; a vector access when `whole`
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, bool whole, int n, float (&x)[4]) {
        if (whole) {
            const float4 v = *reinterpret_cast<const float4 *>(p);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = i < n ? p[i] : 0.f;
        }
    }
    static __device__ __forceinline__ void store(float *p, bool whole, int n, const float (&x)[4]) {
        if (whole) {
            *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) p[i] = x[i];
        }
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool whole, int n, float (&x)[8]) {
        if (whole) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = i < n ? __bfloat162float(p[i]) : 0.f;
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, bool whole, int n, const float (&x)[8]) {
        if (whole) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                       pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = __float2bfloat16_rn(x[i]);
        }
    }
};

// A row is cut into units that touch nothing of one another, so that rows may
// be turned in place: `pair` units (N pairs of halves, or N / 2 neighbouring
// pairs) and units of up to N elements behind rotary_dim.  Accesses are vectors
// where the pieces begin on 16 bytes, else single elements.
template <typename T>
__device__ __forceinline__ void turn_unit(const T *src, T *dst, int unit, int pair_units, int dim, int rot,
                                          bool interleaved, const float2 *table) {
    constexpr int N = Vec<T>::N;
    if (unit >= pair_units) {
        const int at = rot + (unit - pair_units) * N;
        const int n = min(N, dim - at);
        const bool whole = n == N && at % N == 0;
        float x[N];
        Vec<T>::load(src + at, whole, n, x);
        Vec<T>::store(dst + at, whole, n, x);
    } else if (interleaved) {
        const int at = unit * N;
        const int n = min(N, rot - at);
        float x[N];
        Vec<T>::load(src + at, n == N, n, x);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 cs = i < n ? table[(at + i) >> 1] : make_float2(1.f, 0.f);
            const float x0 = x[i], x1 = x[i + 1];
            x[i] = x0 * cs.x - x1 * cs.y;
            x[i + 1] = x1 * cs.x + x0 * cs.y;
        }
        Vec<T>::store(dst + at, n == N, n, x);
    } else {
        const int half = rot / 2, at = unit * N;
        const int n = min(N, half - at);
        const bool whole = half % N == 0;
        float x[N], y[N];
        Vec<T>::load(src + at, whole, n, x);
        Vec<T>::load(src + half + at, whole, n, y);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 cs = i < n ? table[at + i] : make_float2(1.f, 0.f);
            const float x0 = x[i], x1 = y[i];
            x[i] = x0 * cs.x - x1 * cs.y;
            y[i] = x1 * cs.x + x0 * cs.y;
        }
        Vec<T>::store(dst + at, whole, n, x);
        Vec<T>::store(dst + half + at, whole, n, y);
    }
}

// Rows: queries to query_out and, with float pools, keys and values to their slots.
template <typename T>
__device__ __forceinline__ void turn_rows(const RopeArgs &a, float2 *table, bool pools) {
    constexpr int N = Vec<T>::N;
    const int D = a.head_dim, rot = a.rotary_dim, half = rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_cta;
    const int nt = (int)min((int64_t)a.tokens_per_cta, a.num_tokens - t0);
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int t = i / half;
        table[i] = turn_of(a.positions[t0 + t], a.turns[i - t * half], a.factor);
    }
    __syncthreads();
    const int pair_units = a.interleaved ? (rot + N - 1) / N : (half + N - 1) / N;
    const int units = pair_units + (D - rot + N - 1) / N;
    const int copy_units = D / N;
    const int q_items = a.num_q_heads * units;
    const int k_items = pools ? a.num_kv_heads * units : 0;
    const int v_items = pools ? a.num_kv_heads * copy_units : 0;
    const int per_token = q_items + k_items + v_items;
    for (int i = threadIdx.x; i < nt * per_token; i += kRopeThreads) {
        const int t = i / per_token;
        int item = i - t * per_token;
        const int64_t tok = t0 + t;
        if (item < q_items) {
            const int h = item / units;
            turn_unit<T>(static_cast<const T *>(a.query) + tok * a.q_stride + (int64_t)h * D,
                         static_cast<T *>(a.query_out) + tok * a.q_out_stride + (int64_t)h * D, item - h * units,
                         pair_units, D, rot, a.interleaved, table + t * half);
            continue;
        }
        item -= q_items;
        const int64_t slot = a.slot_mapping[tok];
        if (slot < 0) continue;
        if (slot >= (int64_t)a.num_blocks * kBlockSize) {
            if (item == 0) report(a.status, PA_DEV_BAD_SLOT);
            continue;
        }
        const int64_t blk = slot / kBlockSize, off = slot - blk * kBlockSize;
        if (item < k_items) {
            const int h = item / units;
            turn_unit<T>(static_cast<const T *>(a.key) + tok * a.k_stride + (int64_t)h * D,
                         static_cast<T *>(a.key_cache) + ((blk * a.num_kv_heads + h) * kBlockSize + off) * D,
                         item - h * units, pair_units, D, rot, a.interleaved, table + t * half);
        } else {
            item -= k_items;
            const int h = item / copy_units, at = (item - h * copy_units) * N;
            const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.value) + tok * a.v_stride +
                                                             (int64_t)h * D + at);
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.value_cache) +
                                       ((blk * a.num_kv_heads + h) * kBlockSize + off) * D + at) = v;
        }
    }
}

// The smallest e in [kMinExp, kMaxExp] with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int k = (int)(u >> 23) - 127;              // amax = m * 2^k, m in [1, 2)
    const int e = (u & 0x7fffffu) <= 0x600000u ? k - 8 : k - 7;
    return max(kMinExp, min(kMaxExp, e));
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Blocks: a CTA takes the blocks whose first token of this call lies among its
// tile_tokens entries; a warp takes one (block, KV head) of K or of V at a time,
// stages its turned rows in shared memory, finds the scale and encodes.
// Shared memory: cos and sin of tile_tokens + 31 tokens, then per warp 16 rows
// of head_dim floats.
template <typename T>
__device__ __forceinline__ void encode_blocks(const RopeArgs &a, float2 *table) {
    constexpr int N = Vec<T>::N;
    const int D = a.head_dim, rot = a.rotary_dim, half = rot / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)(blockIdx.x - a.row_ctas) * a.tile_tokens;
    const int nt = (int)min((int64_t)a.tile_tokens, a.num_tokens - t0);
    const int reach = (int)min((int64_t)nt + kWindow - 1, a.num_tokens - t0);
    float *rows = reinterpret_cast<float *>(table + (a.tile_tokens + kWindow - 1) * half) + warp * kBlockSize * D;
    const int64_t limit = (int64_t)a.num_blocks * kBlockSize;
    const int pair_units = a.interleaved ? (rot + N - 1) / N : (half + N - 1) / N;
    const int units = pair_units + (D - rot + N - 1) / N;

    // the leaders (a block's first token: none of the kWindow - 1 entries before
    // has the same block) and how many tokens of the reach belong to them
    __shared__ int s_lead[kWindow], s_count, s_last;
    if (threadIdx.x == 0) s_count = s_last = 0;
    __syncthreads();
    for (int i = warp; i < nt; i += kRopeWarps) {
        const int64_t tok = t0 + i;
        const int64_t slot = a.slot_mapping[tok];
        if (slot >= limit && lane == 0) report(a.status, PA_DEV_BAD_SLOT);
        if (slot < 0 || slot >= limit) continue;
        const int64_t blk = slot / kBlockSize, prev = tok - 1 - lane, far = prev - (kWindow - 1), next = tok + lane;
        const int64_t sp = lane < kWindow - 1 && prev >= 0 ? a.slot_mapping[prev] : -1;
        const int64_t sf = lane < kWindow - 1 && far >= 0 ? a.slot_mapping[far] : -1;
        const int64_t sn = next < a.num_tokens ? a.slot_mapping[next] : -1;
        const unsigned mine = __ballot_sync(0xffffffffu, sn >= 0 && sn / kBlockSize == blk);
        // the block's tokens spread over more than kWindow entries: this one is
        // out of its leader's reach, or would lead a second time
        if (__any_sync(0xffffffffu, sf >= 0 && sf / kBlockSize == blk)) {
            if (lane == 0) report(a.status, PA_DEV_BAD_SLOT);
            continue;
        }
        if (__any_sync(0xffffffffu, sp >= 0 && sp / kBlockSize == blk)) continue;
        if (lane == 0) {
            s_lead[atomicAdd(&s_count, 1)] = i;
            atomicMax(&s_last, i + 31 - __clz((int)mine));
        }
    }
    __syncthreads();
    const int leads = s_count;
    if (leads == 0) return;
    for (int i = threadIdx.x; i < (min(s_last, reach - 1) + 1) * half; i += kRopeThreads) {
        const int t = i / half;
        table[i] = turn_of(a.positions[t0 + t], a.turns[i - t * half], a.factor);
    }
    __syncthreads();

    for (int item = warp; item < leads * a.num_kv_heads * 2; item += kRopeWarps) {
        const int which = item & 1, h = (item >> 1) % a.num_kv_heads, lead = s_lead[(item >> 1) / a.num_kv_heads];
        const int64_t tok = t0 + lead;
        const int64_t blk = a.slot_mapping[tok] / kBlockSize;
        const int64_t mine_slot = tok + lane < a.num_tokens ? a.slot_mapping[tok + lane] : -1;
        const bool is_mine = mine_slot >= 0 && mine_slot / kBlockSize == blk;
        const unsigned members = __ballot_sync(0xffffffffu, is_mine);
        const int off = is_mine ? (int)(mine_slot % kBlockSize) : kBlockSize;
        const int low = __reduce_min_sync(0xffffffffu, off);
        const unsigned put = __reduce_or_sync(0xffffffffu, is_mine ? 1u << off : 0u);   // offsets written
        uint8_t *tile = static_cast<uint8_t *>(which ? a.value_cache : a.key_cache) +
                        (blk * a.num_kv_heads + h) * kBlockSize * (int64_t)D;
        float *scale_at = (which ? a.v_scales : a.k_scales) + blk * a.num_kv_heads + h;
        const float old = low > 0 ? *scale_at : 0.f;
        // turned rows; a slot that is listed twice keeps the later token
        for (unsigned m = members; m != 0; m &= m - 1) {
            const int j = __ffs((int)m) - 1;
            float *row = rows + __shfl_sync(0xffffffffu, off, j) * D;
            const T *src = static_cast<const T *>(which ? a.value : a.key) +
                           (tok + j) * (which ? a.v_stride : a.k_stride) + (int64_t)h * D;
            if (which) {
                for (int at = lane * N; at < D; at += 32 * N) {
                    float x[N];
                    Vec<T>::load(src + at, true, N, x);
#pragma unroll
                    for (int i = 0; i < N; ++i) row[at + i] = x[i];
                }
            } else {
                const float2 *cs = table + (lead + j) * half;
                for (int u = lane; u < units; u += 32) {
                    float x[N], y[N];
                    if (u >= pair_units) {
                        const int at = rot + (u - pair_units) * N, n = min(N, D - at);
                        Vec<T>::load(src + at, n == N && at % N == 0, n, x);
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if (i < n) row[at + i] = x[i];
                    } else if (a.interleaved) {
                        const int at = u * N, n = min(N, rot - at);
                        Vec<T>::load(src + at, n == N, n, x);
#pragma unroll
                        for (int i = 0; i < N; i += 2)
                            if (i < n) {
                                const float2 c = cs[(at + i) >> 1];
                                row[at + i] = x[i] * c.x - x[i + 1] * c.y;
                                row[at + i + 1] = x[i + 1] * c.x + x[i] * c.y;
                            }
                    } else {
                        const int at = u * N, n = min(N, half - at);
                        const bool whole = half % N == 0;
                        Vec<T>::load(src + at, whole, n, x);
                        Vec<T>::load(src + half + at, whole, n, y);
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if (i < n) {
                                const float2 c = cs[at + i];
                                row[at + i] = x[i] * c.x - y[i] * c.y;
                                row[half + at + i] = y[i] * c.x + x[i] * c.y;
                            }
                    }
                }
            }
            __syncwarp();
        }
        float amax = 0.f;                            // fmaxf passes over NaN
        for (unsigned m = put; m != 0; m &= m - 1) {
            const float *row = rows + (__ffs((int)m) - 1) * D;
            for (int c = lane * 4; c < D; c += 128) {
                const float4 x = *reinterpret_cast<const float4 *>(row + c);
                amax = fmaxf(fmaxf(fmaxf(amax, fabsf(x.x)), fmaxf(fabsf(x.y), fabsf(x.z))), fabsf(x.w));
            }
        }
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        if (amax > 448.f * pow2i(kMaxExp) && lane == 0) report(a.status, PA_DEV_RANGE);
        const float scale = fmaxf(pow2i(scale_exponent(amax)), old);
        // dividing by a power of two is multiplying by its inverse; a scale that
        // someone else chose is divided by
        const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
        const float inv = 1.f / scale;
        if (low > 0 && scale != old) {
            const float f = old / scale;
            for (int r = 0; r < low; ++r)
                for (int c = lane * 4; c < D; c += 128) {
                    uint32_t *p = reinterpret_cast<uint32_t *>(tile + r * D + c);
                    uint32_t lo, hi;
                    e4m3x4_to_f16x2x2(*p, lo, hi);
                    *p = f32x2_to_e4m3x2(f16lo(lo) * f, f16hi(lo) * f) |
                         (f32x2_to_e4m3x2(f16lo(hi) * f, f16hi(hi) * f) << 16);
                }
        }
        for (unsigned m = put; m != 0; m &= m - 1) {
            const int r = __ffs((int)m) - 1;
            for (int c = lane * 4; c < D; c += 128) {
                float4 x = *reinterpret_cast<const float4 *>(rows + r * D + c);
                if (pow2)
                    x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
                else
                    x = make_float4(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale), __fdiv_rn(x.z, scale),
                                    __fdiv_rn(x.w, scale));
                *reinterpret_cast<uint32_t *>(tile + r * D + c) =
                    f32x2_to_e4m3x2(x.x, x.y) | (f32x2_to_e4m3x2(x.z, x.w) << 16);
            }
        }
        if (lane == 0) *scale_at = scale;
        __syncwarp();                                // the rows are read
    }
}

template <typename T, bool kBlocks>
__global__ void __launch_bounds__(kRopeThreads) pa_rope_write_kernel(const RopeArgs a) {
    extern __shared__ __align__(16) float2 s_table[];
    grid_dependency_wait();
    grid_dependents_launch();
    if constexpr (kBlocks) {
        if ((int)blockIdx.x >= a.row_ctas) {
            encode_blocks<T>(a, s_table);
            return;
        }
    }
    turn_rows<T>(a, s_table, !kBlocks);
}

// Frequencies for rotary positions; see the header.
double ramp_index(double turns, double dim, double base, double context) {
    return dim * log(context / (turns * 2.0 * M_PI)) / (2.0 * log(base));
}

template <typename T>
pa_status launch_rope(RopeArgs &a, bool blocks, cudaStream_t stream) {
    const int half = a.rotary_dim / 2;
    // enough CTAs to fill the GPU, and tokens together where there are many
    // (their cos and sin are computed side by side)
    int tpc = 1;
    while (tpc < 16 && a.num_tokens / (2 * tpc) >= 4 * 152) tpc *= 2;
    a.tokens_per_cta = tpc;
    const int64_t rows = a.num_q_heads > 0 || !blocks ? ((int64_t)a.num_tokens + tpc - 1) / tpc : 0;
    int64_t grid = rows;
    size_t smem = (size_t)tpc * half * sizeof(float2);
    if (blocks) {
        a.tile_tokens = tpc;
        grid += ((int64_t)a.num_tokens + a.tile_tokens - 1) / a.tile_tokens;
        smem = std::max(smem, (size_t)(a.tile_tokens + kWindow - 1) * half * sizeof(float2) +
                                  (size_t)kRopeWarps * kBlockSize * a.head_dim * sizeof(float));
    }
    if (grid >= ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;
    a.row_ctas = (int)rows;
    auto kernel = blocks ? pa_rope_write_kernel<T, true> : pa_rope_write_kernel<T, false>;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return cuda_failure(e, "cudaFuncSetAttribute(rope)");
    }
    cudaError_t e = launch_chained(kernel, dim3((unsigned)grid), dim3(kRopeThreads), smem, stream, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_rope_write_kernel launch");
    count_launches(1);
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_rotary_turns(uint64_t *turns, float *attention_factor, int rotary_dim, double base,
                                     pa_rotary_scaling scaling, double factor, double original_context,
                                     double beta_fast, double beta_slow) {
    if (!turns || !attention_factor || rotary_dim < 0 || rotary_dim % 2 != 0 || !(base > 1.0) || !(factor > 0.0) ||
        !std::isfinite(base) || !std::isfinite(factor))
        return PA_ERR_INVALID_ARG;
    if (scaling != PA_ROTARY_NONE && scaling != PA_ROTARY_LINEAR && scaling != PA_ROTARY_NTK &&
        scaling != PA_ROTARY_BY_PARTS)
        return PA_ERR_INVALID_ARG;
    if (scaling == PA_ROTARY_BY_PARTS && (!(original_context >= 1.0) || !std::isfinite(original_context) ||
                                          !(beta_fast > 0.0) || !(beta_slow > 0.0) || !std::isfinite(beta_fast) ||
                                          !std::isfinite(beta_slow)))
        return PA_ERR_INVALID_ARG;
    const double d = rotary_dim;
    if (scaling == PA_ROTARY_NTK && rotary_dim > 2) base *= pow(factor, d / (d - 2.0));
    double lo = 0, hi = 1;
    if (scaling == PA_ROTARY_BY_PARTS) {
        lo = std::max(floor(ramp_index(beta_fast, d, base, original_context)), 0.0);
        hi = std::min(ceil(ramp_index(beta_slow, d, base, original_context)), d - 1.0);
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double theta = pow(base, -2.0 * i / d);
        if (scaling == PA_ROTARY_LINEAR) theta /= factor;
        if (scaling == PA_ROTARY_BY_PARTS) {
            const double r = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
            theta = theta * (1.0 - r) + theta / factor * r;
        }
        const double t = theta / (2.0 * M_PI);       // turns per position
        const double frac = t - floor(t);
        turns[i] = frac >= 1.0 ? 0 : (uint64_t)ldexp(frac, 64);
    }
    *attention_factor = scaling == PA_ROTARY_BY_PARTS && factor > 1.0 ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return PA_OK;
}

extern "C" pa_status pa_rope_cache_write(void *query_out, const void *query, const void *key, const void *value,
                                         const int32_t *positions, const uint64_t *turns, float attention_factor,
                                         int rotary_dim, int interleaved, void *key_cache, void *value_cache,
                                         float *k_scales, float *v_scales, const int64_t *slot_mapping,
                                         int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                         int64_t query_out_stride, int64_t query_stride, int64_t key_stride,
                                         int64_t value_stride, int block_size, int num_blocks, pa_dtype dtype,
                                         pa_dtype cache_dtype, int32_t *device_status, void *stream) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || head_dim <= 0 || rotary_dim < 0 ||
        rotary_dim > head_dim || rotary_dim % 2 != 0 || block_size != kBlockSize || num_blocks <= 0 ||
        !std::isfinite(attention_factor))
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16) return PA_ERR_INVALID_ARG;
    if (cache_dtype != dtype && cache_dtype != PA_DTYPE_FP8_E4M3) return PA_ERR_INVALID_ARG;
    const bool blocks = cache_dtype == PA_DTYPE_FP8_E4M3;
    const int esize = dtype == PA_DTYPE_F32 ? 4 : 2;
    if (head_dim > 256 || (head_dim * esize) % 16 != 0 || (blocks && head_dim % 16 != 0)) return PA_ERR_UNSUPPORTED;
    const int64_t q_row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    if (num_tokens == 0) return PA_OK;
    if (num_q_heads > 0 && (!query || !query_out || query_stride < q_row || query_out_stride < q_row ||
                            !aligned16(query) || !aligned16(query_out) || (query_stride * esize) % 16 != 0 ||
                            (query_out_stride * esize) % 16 != 0))
        return PA_ERR_INVALID_ARG;
    if (!key || !value || !key_cache || !value_cache || !slot_mapping || key_stride < kv_row ||
        value_stride < kv_row || !aligned16(key) || !aligned16(value) || !aligned16(key_cache) ||
        !aligned16(value_cache) || (key_stride * esize) % 16 != 0 || (value_stride * esize) % 16 != 0 ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PA_ERR_INVALID_ARG;
    if (rotary_dim > 0 && (!positions || !turns || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
                           (reinterpret_cast<uintptr_t>(turns) & 7u)))
        return PA_ERR_INVALID_ARG;
    if (blocks && (!k_scales || !v_scales || (reinterpret_cast<uintptr_t>(k_scales) & 3u) ||
                   (reinterpret_cast<uintptr_t>(v_scales) & 3u)))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && query == query_out && query_stride != query_out_stride) return PA_ERR_INVALID_ARG;
    // items of one CTA are counted in 32 bits
    if ((q_row + 2 * kv_row) * 16 >= ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;
    RopeArgs a = {};
    a.query = query;
    a.key = key;
    a.value = value;
    a.query_out = query_out;
    a.key_cache = key_cache;
    a.value_cache = value_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.positions = positions;
    a.turns = turns;
    a.slot_mapping = slot_mapping;
    a.status = device_status;
    a.q_stride = query_stride;
    a.k_stride = key_stride;
    a.v_stride = value_stride;
    a.q_out_stride = query_out_stride;
    a.factor = attention_factor;
    a.num_tokens = num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved != 0;
    a.num_blocks = num_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PA_DTYPE_F32 ? launch_rope<float>(a, blocks, st) : launch_rope<__nv_bfloat16>(a, blocks, st);
}
