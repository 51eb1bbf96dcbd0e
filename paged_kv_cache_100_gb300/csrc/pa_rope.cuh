// Rotary positions on rows, shared by the kernels that write the cache
// (pa_rope.cu: float pools and E4M3 codes with a scale per block; pa_fp4_cache.cu:
// 4-bit codes).  The mathematics of the angles is in pa_rope.cu.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
// Error of a turned element in 32 bits, per |x0| + |x1|: the angle is held to
// 2^-24 of half a turn (pi 2^-24), sincospi to 2 units of 2^-23, and three
// roundings of 2^-24: below 2^-20.8; a multiplication by the inverse of a scale
// that is no power of two adds 2^-23.
constexpr float kTurnError = 7.2e-7f;            // 2^-20.4

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
    double factor;
    int num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim;
    int interleaved;
    int num_blocks;
    int table_row;                   // entries of a token in a table of cos and sin: rotary_dim / 2, rounded up to 4
    int whole;                       // every unit of a row is a whole vector
    int unit_tiles;                  // encode_units' rows: bf16, neighbouring pairs or rotary_dim a multiple of 8
    int tile_ctas, tile_tokens;      // CTAs that encode blocks, and the entries each looks at
    int tile_splits;                 // CTAs that share the KV heads of the same entries
    int far_ctas, far_parts;         // CTAs that look for far tokens of a block, and those of the same own entries
    int row_tokens, row_splits;      // tokens of a row CTA; CTAs that share a token's rows
};

// cos and sin of position p's angle for one pair, times the attention factor
__device__ __forceinline__ float2 turn_of(int32_t p, uint64_t turns, float factor) {
    const uint64_t at = (uint64_t)(int64_t)p * turns;          // modulo one turn
    const float x = (float)(int32_t)(at >> 32) * 0x1p-31f;     // half turns, in [-1, 1]
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * factor, s * factor);
}

// The same rotation in 64 bits: y0, or y1 when `second`.
__device__ __noinline__ double exact_turn(float x0, float x1, bool second, int32_t p, uint64_t turns, double factor) {
    double s, c;
    sincospi((double)(int64_t)((uint64_t)(int64_t)p * turns) * 0x1p-63, &s, &c);
    return (second ? fma((double)x1, c, (double)x0 * s) : fma((double)x0, c, -(double)x1 * s)) * factor;
}

// 16 bytes of a row as floats
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void widen(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 narrow(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void widen(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
    }
    static __device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};
template <typename T>
__device__ __forceinline__ float to_float(T x) {
    if constexpr (sizeof(T) == 4) return x;
    else return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else return __float2bfloat16_rn(x);
}

// A row whose pieces are whole vectors is cut into units that touch nothing of one
// another, so that rows may be turned in place: with neighbouring pairs N elements
// each, the last of the turned ones perhaps in part; with halves N pairs each, then
// N elements each behind rotary_dim.
template <typename T>
__device__ __forceinline__ int pair_units(const RopeArgs &a) {
    constexpr int N = Vec<T>::N;
    return a.interleaved ? (a.rotary_dim + N - 1) / N : a.rotary_dim / 2 / N;
}
template <typename T>
__device__ __forceinline__ int row_units(const RopeArgs &a) {
    return a.interleaved ? a.head_dim / Vec<T>::N : pair_units<T>(a) + (a.head_dim - a.rotary_dim) / Vec<T>::N;
}

// N elements of a row from element `at` on, a multiple of N, and in `o` the other
// element of each one's pair (where there is one).
template <typename T>
__device__ __forceinline__ void load_pairs(const T *row, int at, int rot, bool interleaved, float (&x)[Vec<T>::N],
                                           float (&o)[Vec<T>::N]) {
    constexpr int N = Vec<T>::N;
    const int half = rot / 2;
    Vec<T>::widen(*reinterpret_cast<const uint4 *>(row + at), x);
    if (interleaved || at >= rot) {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = x[i ^ 1];
    } else if (half % N == 0) {
        Vec<T>::widen(*reinterpret_cast<const uint4 *>(row + (at < half ? at + half : at - half)), o);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int d = at + i;
            o[i] = d < rot ? to_float(row[d < half ? d + half : d - half]) : 0.f;
        }
    }
}
// Element d < rot turned: x itself, o the other one of its pair.
__device__ __forceinline__ float turned(float x, float o, int d, int half, bool interleaved, const float2 *table) {
    const bool second = interleaved ? d & 1 : d >= half;
    const float2 cs = table[interleaved ? d >> 1 : (second ? d - half : d)];
    return second ? x * cs.x + o * cs.y : x * cs.x - o * cs.y;
}

// Where row `row` of token `tok` is read and written: queries, then keys, then
// values (float pools).  False when the token has no slot.
template <typename T>
__device__ __forceinline__ bool row_at(const RopeArgs &a, int64_t tok, int row, const T **src, T **dst) {
    const int D = a.head_dim;
    if (row < a.num_q_heads) {
        *src = static_cast<const T *>(a.query) + tok * a.q_stride + (int64_t)row * D;
        *dst = static_cast<T *>(a.query_out) + tok * a.q_out_stride + (int64_t)row * D;
        return true;
    }
    row -= a.num_q_heads;
    const bool v = row >= a.num_kv_heads;
    if (v) row -= a.num_kv_heads;
    const int64_t slot = a.slot_mapping[tok];
    if (slot < 0) return false;
    if (slot >= (int64_t)a.num_blocks * kBlockSize) {
        if (row == 0) report(a.status, PA_DEV_BAD_SLOT);
        return false;
    }
    const int64_t blk = slot / kBlockSize, off = slot - blk * kBlockSize;
    *src = static_cast<const T *>(v ? a.value : a.key) + tok * (v ? a.v_stride : a.k_stride) + (int64_t)row * D;
    *dst = static_cast<T *>(v ? a.value_cache : a.key_cache) + ((blk * a.num_kv_heads + row) * kBlockSize + off) * D;
    return true;
}

// Rows whose units are whole vectors.  A thread keeps one unit of the row and
// the cos and sin of its pairs in registers while it goes through a token's
// rows, two at a time; the loads of both are issued before either is turned.
// Tokens of few rows are turned side by side.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void turn_whole_rows(const RopeArgs &a, int64_t t0, int nt, int split, int rows,
                                                const float2 *table) {
    constexpr int N = Vec<T>::N, P = kInterleaved ? N / 2 : N;
    const int half = a.rotary_dim / 2, pairs = pair_units<T>(a), units = row_units<T>(a);
    const int per_pass = kRopeThreads / units;
    const int unit = threadIdx.x % units, place = threadIdx.x / units;
    const int abreast = max(1, per_pass / rows);         // tokens of a pass
    const int t_first = abreast > 1 ? place / rows : 0, first = place - t_first * rows;
    if (place >= per_pass || t_first >= abreast) return;
    const bool pair = unit < pairs;
    const int at = kInterleaved || pair ? unit * N : a.rotary_dim + (unit - pairs) * N;
    const int some = kInterleaved ? half - unit * P : P;     // pairs of the unit that are turned, if below P
    const int step = per_pass * a.row_splits;
    for (int t = t_first; t < nt; t += abreast) {
        float2 cs[P];
        if (pair) {
            const float4 *c = reinterpret_cast<const float4 *>(table + t * a.table_row + unit * P);
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 v = c[i / 2];
                cs[i] = make_float2(v.x, v.y);
                cs[i + 1] = make_float2(v.z, v.w);
            }
        }
        for (int r = first + split * per_pass; r < rows; r += 2 * step) {
            const T *src[2];
            T *dst[2];
            bool on[2];
            uint4 x[2], y[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                on[u] = r + u * step < rows && row_at<T>(a, t0 + t, r + u * step, &src[u], &dst[u]);
                if (on[u]) {
                    x[u] = *reinterpret_cast<const uint4 *>(src[u] + at);
                    if (!kInterleaved && pair) y[u] = *reinterpret_cast<const uint4 *>(src[u] + at + half);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (!on[u]) continue;
                // values are not turned
                if (pair && r + u * step < a.num_q_heads + a.num_kv_heads) {
                    float p[N], q[N];
                    Vec<T>::widen(x[u], p);
                    if constexpr (kInterleaved) {
#pragma unroll
                        for (int i = 0; i < N; i += 2) {
                            q[i] = i / 2 < some ? p[i] * cs[i / 2].x - p[i + 1] * cs[i / 2].y : p[i];
                            q[i + 1] = i / 2 < some ? p[i + 1] * cs[i / 2].x + p[i] * cs[i / 2].y : p[i + 1];
                        }
                        x[u] = Vec<T>::narrow(q);
                    } else {
                        float s[N], o[N];
                        Vec<T>::widen(y[u], q);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            s[i] = p[i] * cs[i].x - q[i] * cs[i].y;
                            o[i] = q[i] * cs[i].x + p[i] * cs[i].y;
                        }
                        x[u] = Vec<T>::narrow(s);
                        y[u] = Vec<T>::narrow(o);
                    }
                }
                *reinterpret_cast<uint4 *>(dst[u] + at) = x[u];
                if (!kInterleaved && pair) *reinterpret_cast<uint4 *>(dst[u] + at + half) = y[u];
            }
        }
    }
}

__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// The same for CTAs that turn several tokens into float pools: a thread's loads go
// kAhead - 1 rows ahead into places of its own in shared memory (nothing is shared,
// so nothing waits but the thread for its own copies), as registers do not hold
// that many.  27832 tokens of 8 f32 heads of 128 44.5 us against 57.7, 8192 tokens
// of 80 bf16 heads 56.6 / 60.3, of 80 f32 heads 106.2 / 104.8; one token a CTA 0.3
// us slower; beside CTAs that encode blocks, which wait longer then, 67.2 / 65.7; 4
// or 6 rows ahead 44.3 and 47.4 us.
constexpr int kAhead = 3;
template <typename T, bool kInterleaved>
__device__ __forceinline__ void turn_many_rows(const RopeArgs &a, int64_t t0, int nt, int split, int rows,
                                               const float2 *table, uint4 *places) {
    constexpr int N = Vec<T>::N, P = kInterleaved ? N / 2 : N;
    const int half = a.rotary_dim / 2, pairs = pair_units<T>(a), units = row_units<T>(a);
    const int per_pass = kRopeThreads / units;
    const int unit = threadIdx.x % units, place = threadIdx.x / units;
    const int abreast = max(1, per_pass / rows);         // tokens of a pass
    const int t_first = abreast > 1 ? place / rows : 0, first = place - t_first * rows;
    if (place >= per_pass || t_first >= abreast) return;
    const bool pair = unit < pairs;
    const int at = kInterleaved || pair ? unit * N : a.rotary_dim + (unit - pairs) * N;
    const int some = kInterleaved ? half - unit * P : P;     // pairs of the unit that are turned, if below P
    const int step = per_pass * a.row_splits, r0 = first + split * per_pass;
    if (r0 >= rows) return;
    uint4 *mine = places + threadIdx.x;                  // [kAhead][2][kRopeThreads]
    int pt = t_first, pr = r0, pslot = 0;
    auto prefetch = [&]() {
        const T *src;
        T *dst;
        if (pt < nt && row_at<T>(a, t0 + pt, pr, &src, &dst)) {
            copy_async16(mine + pslot * 2 * kRopeThreads, src + at);
            if (!kInterleaved && pair) copy_async16(mine + (pslot * 2 + 1) * kRopeThreads, src + at + half);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        pslot = pslot + 1 == kAhead ? 0 : pslot + 1;
        pr += step;
        if (pr >= rows) pr = r0, pt += abreast;
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) prefetch();
    int slot = 0;
    for (int t = t_first; t < nt; t += abreast) {
        float2 cs[P];
        if (pair) {
            const float4 *c = reinterpret_cast<const float4 *>(table + t * a.table_row + unit * P);
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 v = c[i / 2];
                cs[i] = make_float2(v.x, v.y);
                cs[i + 1] = make_float2(v.z, v.w);
            }
        }
        for (int r = r0; r < rows; r += step) {
            prefetch();
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            const uint4 *from = mine + slot * 2 * kRopeThreads;
            slot = slot + 1 == kAhead ? 0 : slot + 1;
            const T *src;
            T *dst;
            if (!row_at<T>(a, t0 + t, r, &src, &dst)) continue;
            uint4 x = from[0];
            if (pair && r < a.num_q_heads + a.num_kv_heads) {
                float p[N], q[N];
                Vec<T>::widen(x, p);
                if constexpr (kInterleaved) {
#pragma unroll
                    for (int i = 0; i < N; i += 2) {
                        q[i] = i / 2 < some ? p[i] * cs[i / 2].x - p[i + 1] * cs[i / 2].y : p[i];
                        q[i + 1] = i / 2 < some ? p[i + 1] * cs[i / 2].x + p[i] * cs[i / 2].y : p[i + 1];
                    }
                    x = Vec<T>::narrow(q);
                } else {
                    float s[N], o[N];
                    Vec<T>::widen(from[kRopeThreads], q);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        s[i] = p[i] * cs[i].x - q[i] * cs[i].y;
                        o[i] = q[i] * cs[i].x + p[i] * cs[i].y;
                    }
                    x = Vec<T>::narrow(s);
                    *reinterpret_cast<uint4 *>(dst + at + half) = Vec<T>::narrow(o);
                }
            } else if (!kInterleaved && pair) {
                *reinterpret_cast<uint4 *>(dst + at + half) = from[kRopeThreads];
            }
            *reinterpret_cast<uint4 *>(dst + at) = x;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rows of halves that are no whole vectors: a thread has one vector of a row, and
// reads the other elements of its pairs where they are.  All of a row is read in one pass, so that a barrier
// before the stores is enough to turn rows in place.
template <typename T>
__device__ __forceinline__ void turn_any_rows(const RopeArgs &a, int64_t t0, int nt, int split, int rows,
                                              const float2 *table) {
    constexpr int N = Vec<T>::N;
    const int rot = a.rotary_dim, half = rot / 2, chunks = a.head_dim / N;
    const int per_pass = kRopeThreads / chunks;
    const int at = threadIdx.x % chunks * N, place = threadIdx.x / chunks;
    const int abreast = max(1, per_pass / rows);
    const int t_first = abreast > 1 ? place / rows : 0, first = place - t_first * rows;
    const bool mine = place < per_pass && t_first < abreast;
    const int turned_rows = a.num_q_heads + a.num_kv_heads;
    const bool meet = a.query == a.query_out;
    for (int tb = 0; tb < nt; tb += abreast) {
        for (int rb = split * per_pass; rb < rows; rb += per_pass * a.row_splits) {
            const int t = tb + t_first, r = rb + first;
            const T *src;
            T *dst;
            float x[N], o[N];
            const bool on = mine && t < nt && r < rows && row_at<T>(a, t0 + t, r, &src, &dst);
            if (on) {
                load_pairs<T>(src, at, r < turned_rows ? rot : 0, false, x, o);
                if (r < turned_rows && at < rot) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (at + i < rot) o[i] = turned(x[i], o[i], at + i, half, false, table + t * a.table_row);
                        else o[i] = x[i];
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) o[i] = x[i];
                }
            }
            if (meet) __syncthreads();
            if (on) *reinterpret_cast<uint4 *>(dst + at) = Vec<T>::narrow(o);
        }
    }
}

// The rows of a CTA's tokens: queries to query_out and, with float pools, keys
// and values to their slots.
template <typename T>
__device__ __forceinline__ void turn_rows(const RopeArgs &a, int cta, float2 *table, bool pools) {
    const int half = a.rotary_dim / 2;
    const int group = cta / a.row_splits, split = cta - group * a.row_splits;
    const int64_t t0 = (int64_t)group * a.row_tokens;
    const int nt = (int)min((int64_t)a.row_tokens, a.num_tokens - t0);
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int t = i / half;
        table[t * a.table_row + i - t * half] = turn_of(a.positions[t0 + t], a.turns[i - t * half], (float)a.factor);
    }
    __syncthreads();
    const int rows = a.num_q_heads + (pools ? 2 * a.num_kv_heads : 0);
    if (pools && a.whole && a.row_tokens >= 2) {
        uint4 *places = reinterpret_cast<uint4 *>(table + a.row_tokens * a.table_row);
        if (a.interleaved) turn_many_rows<T, true>(a, t0, nt, split, rows, table, places);
        else turn_many_rows<T, false>(a, t0, nt, split, rows, table, places);
        return;
    }
    if (a.whole) {
        if (a.interleaved) turn_whole_rows<T, true>(a, t0, nt, split, rows, table);
        else turn_whole_rows<T, false>(a, t0, nt, split, rows, table);
        return;
    }
    turn_any_rows<T>(a, t0, nt, split, rows, table);
}

// The pair of element d of a row: false when d is not turned.
__device__ __forceinline__ bool pair_of(const RopeArgs &a, int d, int *first, int *second, int *pair) {
    const int half = a.rotary_dim / 2;
    if (d >= a.rotary_dim) return false;
    *pair = a.interleaved ? d >> 1 : (d < half ? d : d - half);
    *first = a.interleaved ? d & ~1 : *pair;
    *second = a.interleaved ? d | 1 : *pair + half;
    return true;
}

// Whether rows of w bytes, n of them s bytes apart from p, touch rows of v bytes
// t apart from q (a slice of one buffer's rows does not touch the slice beside it;
// with unlike strides the whole ranges count).
bool rows_touch(const void *p, int64_t s, int64_t w, const void *q, int64_t t, int64_t v, int64_t n) {
    const intptr_t x = reinterpret_cast<intptr_t>(p), y = reinterpret_cast<intptr_t>(q);
    if (w == 0 || v == 0 || x >= y + (n - 1) * t + v || y >= x + (n - 1) * s + w) return false;
    if (n == 1 || s != t) return true;
    const int64_t r = ((y - x) % s + s) % s;         // the other row begins r behind one of ours
    return r < w || r + v > s;
}

// How rows are shared out: table layout, tokens of a CTA and CTAs of a token; returns
// the CTAs that turn `rows` rows of every token.
template <typename T>
int64_t plan_rows(RopeArgs &a, int rows) {
    constexpr int N = 16 / (int)sizeof(T);
    const int D = a.head_dim, rot = a.rotary_dim, half = rot / 2;
    a.table_row = (half + 3) & ~3;
    a.whole = a.interleaved || half % N == 0;
    // tokens share a CTA where there are enough for four CTAs per SM, more than
    // eight where a token has few rows (64 query heads of 128: 61 us with 4 or 8
    // tokens a CTA, 64.5 with 16); where there are fewer than SMs, CTAs share a
    // token's rows
    const int64_t n = a.num_tokens, sms = device_sms();
    const int units = a.whole && !a.interleaved ? (half + D - rot) / N : D / N;
    const int most = std::max(8, std::min(32, 4096 / std::max(1, rows * units)));
    a.row_tokens = 1;
    while (2 * a.row_tokens <= most && n / (2 * a.row_tokens) >= 4 * sms) a.row_tokens *= 2;
    const int passes = (rows + kRopeThreads / units - 1) / (kRopeThreads / units);
    a.row_splits = (int)std::max<int64_t>(1, std::min<int64_t>(passes, 2 * sms / n));
    return rows > 0 ? (n + a.row_tokens - 1) / a.row_tokens * a.row_splits : 0;
}

}  // namespace
}  // namespace pa
