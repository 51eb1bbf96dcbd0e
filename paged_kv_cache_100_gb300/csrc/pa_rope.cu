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
// full turn, the nearest one: the 64-bit product p * turns_i wraps at whole turns by
// itself and its upper half is the angle to 2^-32 of a turn at any position.
//
// Block scales.  A block's scale is the smallest power of two 2^e, e in
// [-32, 31], that holds its largest magnitude: amax <= 448 * 2^e.  E4M3 is a
// floating-point code, so a power of two loses no precision against amax / 448,
// the division of an element by it is exact, and a block whose scale grows when
// a row is appended has its earlier rows re-encoded without error (apart from
// codes that become subnormal).
// A key's code is that of its exact rotation rounded to f32: an element whose
// 32-bit value lies so near a border of two codes that its error could cross it
// (about one in 7000) is computed again in 64 bits, and so is the largest
// magnitude when it lies next to a scale's border.
//
// The kernel moves bytes: a launch has CTAs that turn rows (queries; keys and
// values too for float pools) and, first, a few that look for far tokens of a block and
// CTAs that encode blocks.
// 8192 tokens of 64 query and 8 KV heads of 128 into E4M3 pools: 63 us for 319 MB,
// 5.1 TB/s or 0.75 of a copy.  The query rows alone take 48 us and the blocks alone
// 36, mostly the arithmetic of two passes (the maximum, then the codes), of which
// the rows' traffic hides half; the two kinds of CTA mixed from the start instead
// of blocks first took 65 to 74 us.  A step of 256 tokens of that shape takes 8.4
// us, of 64 tokens into bf16 pools 2.9: latency.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rope.cuh"

namespace pa {
namespace {

constexpr int kWindow = 32;          // entries of slot_mapping among which a block's tokens lie
constexpr int kMostTokens = 1 << 26; // of a call into block-scaled pools (find_far's CTAs are counted in 32 bits)
constexpr int kFarOwn = 1024;        // entries whose blocks a CTA of find_far looks for,
constexpr int kFarPart = 16384;      // and entries among which it does
constexpr int kFarSlots = 2048;      // places of its table: a power of two, never more than half full
static_assert(kFarPart % kFarOwn == 0, "a CTA's own entries are looked at by one CTA");
constexpr int kMaxTile = 64;         // entries of slot_mapping whose blocks a CTA encodes
constexpr int kMostTables = 100 * 1024;   // dynamic shared memory of a CTA at most
constexpr int kMinExp = -32, kMaxExp = 31;

// Code of y / scale, y in 64 bits: of the f32 quotient, as everywhere.
__device__ __forceinline__ uint32_t exact_code(double y, float scale) {
    return f32x2_to_e4m3x2((float)(y / (double)scale), 0.f) & 0xffu;
}

// The smallest e in [kMinExp, kMaxExp] with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int k = (int)(u >> 23) - 127;              // amax = m * 2^k, m in [1, 2)
    const int e = (u & 0x7fffffu) <= 0x600000u ? k - 8 : k - 7;
    return max(kMinExp, min(kMaxExp, e));
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The block of one KV head that a warp encodes, K or V.
struct Tile {
    int64_t tok;                     // first token
    int h, value;                    // KV head; 1: values
    int lead;                        // tok's place in the CTA's table of cos and sin
    int low, n;                      // lowest offset written; rows written
    const uint16_t *list;            // their (entry - tok) | offset << 8
    uint8_t *codes;
    float *scale;
};
template <typename T>
__device__ __forceinline__ const T *tile_row(const RopeArgs &a, const Tile &w, int j) {
    return static_cast<const T *>(w.value ? a.value : a.key) + (w.tok + j) * (w.value ? a.v_stride : a.k_stride) +
           (int64_t)w.h * a.head_dim;
}

// Element d of the row of entry `tok + j` in 64 bits.
template <typename T>
__device__ __forceinline__ double exact_element(const RopeArgs &a, const Tile &w, int j, int d) {
    const T *row = tile_row<T>(a, w, j);
    int first, second, pair;
    if (!pair_of(a, d, &first, &second, &pair)) return (double)to_float(row[d]);
    return exact_turn(to_float(row[first]), to_float(row[second]), d == second, a.positions[w.tok + j], a.turns[pair], a.factor);
}

// Scale exponent of a tile of turned keys whose 32-bit maximum lies next to a
// border: the elements near the maximum again in 64 bits.  A whole warp.
template <typename T>
__device__ __noinline__ int exact_exponent(const RopeArgs &a, const Tile &w, float amax, const float2 *table) {
    double top = 0.0;
    for (int k = 0; k < w.n; ++k) {
        const int j = w.list[k] & 0xff;
        const T *row = tile_row<T>(a, w, j);
        for (int d = threadIdx.x & 31; d < a.head_dim; d += 32) {
            int first, second, pair;
            float x = to_float(row[d]);
            if (pair_of(a, d, &first, &second, &pair)) {
                const float2 cs = table[(w.lead + j) * a.table_row + pair];
                const float x0 = to_float(row[first]), x1 = to_float(row[second]);
                x = d == second ? x1 * cs.x + x0 * cs.y : x0 * cs.x - x1 * cs.y;
            }
            if (fabsf(x) >= amax * (1.f - 0x1p-17f)) top = fmax(top, fabs(exact_element<T>(a, w, j, d)));
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
    int e = scale_exponent(amax * (1.f - 0x1p-18f));
    return top <= 448.0 * (double)pow2i(e) ? e : min(e + 1, kMaxExp);
}

// The tile's scale from the largest magnitudes of the rows written, of turned
// elements (to 2^-18 of it) and of others (exact): at least the old one where
// earlier rows stay, which are then re-encoded if it grew.
template <typename T>
__device__ __forceinline__ float tile_scale(const RopeArgs &a, const Tile &w, float turned_max, float other_max, float old,
                                            const float2 *table) {
    const int lane = threadIdx.x & 31, D = a.head_dim;
    turned_max = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(turned_max)));
    other_max = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(other_max)));
    const float amax = fmaxf(turned_max, other_max);
    if (amax > 448.f * pow2i(kMaxExp) && lane == 0) report(a.status, PA_DEV_RANGE);
    int e = scale_exponent(amax);
    if (scale_exponent(fmaxf(turned_max * (1.f - 0x1p-18f), other_max)) !=
        scale_exponent(fmaxf(turned_max * (1.f + 0x1p-18f), other_max)))
        e = exact_exponent<T>(a, w, amax, table);
    const float scale = fmaxf(pow2i(e), old);
    if (w.low > 0 && scale != old) {
        const float f = old / scale;
        for (int i = lane * 4; i < w.low * D; i += 128) {
            uint32_t *p = reinterpret_cast<uint32_t *>(w.codes + i);
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(*p, lo, hi);
            *p = f32x2_to_e4m3x2(f16lo(lo) * f, f16hi(lo) * f) | (f32x2_to_e4m3x2(f16lo(hi) * f, f16hi(hi) * f) << 16);
        }
    }
    if (lane == 0) *w.scale = scale;
    return scale;
}
__device__ __forceinline__ bool is_pow2(float x) { return (__float_as_uint(x) & 0x7fffffu) == 0; }

// Encodes a tile of bf16 rows that are cut into whole units of 8 elements (neighbouring
// pairs, or rotary_dim a multiple of 8): a lane keeps its unit u and goes through the rows, 32 / units of
// them abreast.  A unit of the turned part is 4 u .. and their partners half + 4 u ..
// (kMode 1, halves) or 8 u .. (kMode 2, neighbours); others are 8 u .. (kMode 0: all).
// The rows are turned once for the maximum and, read again from L1, once more for
// the codes.  kDim: head_dim, all of which is turned (or none, kMode 0), or 0 where
// that is not known beforehand.
template <int kMode, int kDim>
__device__ __forceinline__ void encode_units(const RopeArgs &a, const Tile &w, float old, const float2 *table) {
    const int D = kDim > 0 ? kDim : a.head_dim, units = D / 8, abreast = 32 / units;
    const int lane = threadIdx.x & 31, side = lane / units, u = lane - side * units;
    const int half = kDim > 0 ? kDim / 2 : a.rotary_dim / 2;
    const bool turned = kMode != 0 && (kDim > 0 || 8 * u < a.rotary_dim);
    // pairs of the unit that are turned: all or none but at the end of neighbouring ones
    const int some = !turned ? 0 : kMode == 2 && kDim == 0 ? min(half - 4 * u, 4) : 4;
    const int d0 = kMode == 1 && turned ? 4 * u : 8 * u, d1 = kMode == 1 && turned ? half + 4 * u : 8 * u + 4;
    const int n = side < abreast ? w.n : 0;
    auto row_of = [&](int i) { return abreast * i + side; };
    auto load = [&](int i) {
        uint4 r = make_uint4(0u, 0u, 0u, 0u);
        if (row_of(i) < n) {
            const __nv_bfloat16 *row = tile_row<__nv_bfloat16>(a, w, w.list[row_of(i)] & 0xff);
            if constexpr (kMode == 1) {
                const uint2 x = *reinterpret_cast<const uint2 *>(row + d0);
                const uint2 y = *reinterpret_cast<const uint2 *>(row + d1);
                r = make_uint4(x.x, x.y, y.x, y.y);
            } else {
                r = *reinterpret_cast<const uint4 *>(row + d0);
            }
        }
        return r;
    };
    // the lane's pairs of row i: x0[k], x1[k] and their cos and sin
    auto pairs = [&](int i, const uint4 &raw, float (&x0)[4], float (&x1)[4], float4 (&cs)[2]) {
        const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (kMode == 1) {
                x0[k] = k & 1 ? bf16hi(r[k >> 1]) : bf16lo(r[k >> 1]);
                x1[k] = k & 1 ? bf16hi(r[2 + (k >> 1)]) : bf16lo(r[2 + (k >> 1)]);
            } else {
                x0[k] = bf16lo(r[k]);
                x1[k] = bf16hi(r[k]);
            }
        }
        if (turned) {
            const int j = row_of(i) < n ? w.list[row_of(i)] & 0xff : 0;
            const float4 *c = reinterpret_cast<const float4 *>(table + (w.lead + j) * a.table_row + 4 * u);
            cs[0] = c[0];
            cs[1] = c[1];
        }
    };
    // (what is not turned passes unchanged: 1 x0 - 0 x1 would not where x1 is infinite)
    auto turn = [&](float &x0, float &x1, const float4 (&cs)[2], int k) {
        const float c = k & 1 ? cs[k >> 1].z : cs[k >> 1].x, s = k & 1 ? cs[k >> 1].w : cs[k >> 1].y;
        const float y = x0 * c - x1 * s;
        x1 = k < some ? x1 * c + x0 * s : x1;
        x0 = k < some ? y : x0;
    };
    float amax = 0.f, other = 0.f;                   // of turned pairs and others; fmaxf passes over NaN
#pragma unroll 1
    for (int b = 0; abreast * b < w.n; b += 4) {
        uint4 raw[4];                                // four rows of the lane on their way
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = load(b + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (abreast * (b + i) >= w.n) break;
            float x0[4], x1[4];
            float4 cs[2];
            pairs(b + i, raw[i], x0, x1, cs);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (kMode != 0) turn(x0[k], x1[k], cs, k);
                const float top = fmaxf(fabsf(x0[k]), fabsf(x1[k]));
                if (k < some) amax = fmaxf(amax, top);
                else other = fmaxf(other, top);
            }
        }
    }
    const float scale = tile_scale<__nv_bfloat16>(a, w, amax, other, old, table);
    const float inv = 1.f / scale;
    const bool exact = is_pow2(scale);
    uint4 ahead = load(0);
#pragma unroll 1
    for (int i = 0; abreast * i < w.n; ++i) {
        const uint4 raw = ahead;
        ahead = load(i + 1);
        float x0[4], x1[4];
        float4 cs[2];
        pairs(i, raw, x0, x1, cs);
        uint32_t out[2];                             // codes of x0 and of x1 (mode 1), else in order
        if (!exact) {                                // a scale that someone else chose is divided by
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k >= some) x0[k] = __fdiv_rn(x0[k], scale), x1[k] = __fdiv_rn(x1[k], scale);
        }
        if constexpr (kMode == 0) {
            const float m = exact ? inv : 1.f;
            out[0] = f32x2_to_e4m3x2(x0[0] * m, x1[0] * m) | (f32x2_to_e4m3x2(x0[1] * m, x1[1] * m) << 16);
            out[1] = f32x2_to_e4m3x2(x0[2] * m, x1[2] * m) | (f32x2_to_e4m3x2(x0[3] * m, x1[3] * m) << 16);
        } else {
            // the codes of the value less and more its error: where they differ the
            // pair's codes come from 64 bits
            float y0[4], y1[4], err[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float m = exact || k < some ? inv : 1.f;
                err[k] = k < some ? (fabsf(x0[k]) + fabsf(x1[k])) * (kTurnError * (float)a.factor * inv) : 0.f;
                y0[k] = x0[k];
                y1[k] = x1[k];
                turn(y0[k], y1[k], cs, k);
                y0[k] *= m;
                y1[k] *= m;
            }
            uint32_t lo[2], hi[2];
            auto code4 = [&](float p, float q, float r, float t) {
                return f32x2_to_e4m3x2(p, q) | (f32x2_to_e4m3x2(r, t) << 16);
            };
            if constexpr (kMode == 1) {
                lo[0] = code4(y0[0] - err[0], y0[1] - err[1], y0[2] - err[2], y0[3] - err[3]);
                hi[0] = code4(y0[0] + err[0], y0[1] + err[1], y0[2] + err[2], y0[3] + err[3]);
                lo[1] = code4(y1[0] - err[0], y1[1] - err[1], y1[2] - err[2], y1[3] - err[3]);
                hi[1] = code4(y1[0] + err[0], y1[1] + err[1], y1[2] + err[2], y1[3] + err[3]);
            } else {
                lo[0] = code4(y0[0] - err[0], y1[0] - err[0], y0[1] - err[1], y1[1] - err[1]);
                hi[0] = code4(y0[0] + err[0], y1[0] + err[0], y0[1] + err[1], y1[1] + err[1]);
                lo[1] = code4(y0[2] - err[2], y1[2] - err[2], y0[3] - err[3], y1[3] - err[3]);
                hi[1] = code4(y0[2] + err[2], y1[2] + err[2], y0[3] + err[3], y1[3] + err[3]);
            }
            out[0] = lo[0];
            out[1] = lo[1];
            if (((lo[0] ^ hi[0]) | (lo[1] ^ hi[1])) != 0 && row_of(i) < n) {
                const int j = w.list[row_of(i)] & 0xff;
#pragma unroll 1
                for (int b = 0; b < 8; ++b) {
                    if ((((lo[b >> 2] ^ hi[b >> 2]) >> (8 * (b & 3))) & 0xffu) == 0) continue;
                    const int d = (b < 4 ? d0 : d1) + (b & 3);
                    const uint32_t c = exact_code(exact_element<__nv_bfloat16>(a, w, j, d), scale);
                    const uint32_t mask = 0xffu << (8 * (b & 3));
                    if (b < 4) out[0] = (out[0] & ~mask) | (c << (8 * (b & 3)));
                    else out[1] = (out[1] & ~mask) | (c << (8 * (b & 3)));
                }
            }
        }
        if (row_of(i) < n) {
            uint8_t *row = w.codes + (w.list[row_of(i)] >> 8) * D;
            if constexpr (kMode == 1) {
                *reinterpret_cast<uint32_t *>(row + d0) = out[0];
                *reinterpret_cast<uint32_t *>(row + d1) = out[1];
            } else {
                *reinterpret_cast<uint2 *>(row + d0) = make_uint2(out[0], out[1]);
            }
        }
    }
}
template <int kMode>
__device__ __noinline__ void encode_units_any(const RopeArgs &a, const Tile &w, float old, const float2 *table) {
    encode_units<kMode, 0>(a, w, old, table);
}

// Encodes a tile of any shape: a lane keeps its place in the rows and goes through
// them, once for the maximum and once for the codes.
template <typename T>
__device__ __noinline__ void encode_any(const RopeArgs &a, const Tile &w, float old, const float2 *table) {
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x & 31, D = a.head_dim, rot = w.value ? 0 : a.rotary_dim, half = rot / 2;
    const int chunks = D / N, abreast = max(1, 32 / chunks), sub = chunks < 32 ? lane / chunks : 0;
    const int first = sub < abreast ? sub : w.n;     // row
    const int at0 = (lane - sub * chunks) * N;
    float turned_max = 0.f, other_max = 0.f;         // fmaxf passes over NaN
    for (int at = at0; at < D; at += 32 * N) {
#pragma unroll 1
        for (int k = first; k < w.n; k += abreast) {
            const int j = w.list[k] & 0xff;
            const float2 *cs = table + (w.lead + j) * a.table_row;
            float x[N], o[N];
            load_pairs<T>(tile_row<T>(a, w, j), at, rot, a.interleaved, x, o);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (at + i < rot) turned_max = fmaxf(turned_max, fabsf(turned(x[i], o[i], at + i, half, a.interleaved, cs)));
                else other_max = fmaxf(other_max, fabsf(x[i]));
            }
        }
    }
    const float scale = tile_scale<T>(a, w, turned_max, other_max, old, table);
    const float inv = 1.f / scale;
    const bool exact = is_pow2(scale);
    const float unit = kTurnError * (float)a.factor * inv;
    for (int at = at0; at < D; at += 32 * N) {
#pragma unroll 1
        for (int k = first; k < w.n; k += abreast) {
            const int j = w.list[k] & 0xff;
            const float2 *cs = table + (w.lead + j) * a.table_row;
            float x[N], o[N];
            load_pairs<T>(tile_row<T>(a, w, j), at, rot, a.interleaved, x, o);
            uint32_t lo[N / 4], hi[N / 4];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int d = at + i;
                // the codes of the value less and more its error; where they differ the code
                // comes from 64 bits
                if (d < rot) {
                    const float err = (fabsf(x[i]) + fabsf(o[i])) * unit;
                    const float y = turned(x[i], o[i], d, half, a.interleaved, cs) * inv;
                    x[i] = y - err;
                    o[i] = y + err;
                } else {
                    x[i] = o[i] = exact ? x[i] * inv : __fdiv_rn(x[i], scale);
                }
            }
#pragma unroll
            for (int b = 0; b < N / 4; ++b) {
                lo[b] = f32x2_to_e4m3x2(x[4 * b], x[4 * b + 1]) | (f32x2_to_e4m3x2(x[4 * b + 2], x[4 * b + 3]) << 16);
                hi[b] = f32x2_to_e4m3x2(o[4 * b], o[4 * b + 1]) | (f32x2_to_e4m3x2(o[4 * b + 2], o[4 * b + 3]) << 16);
            }
#pragma unroll
            for (int b = 0; b < N / 4; ++b) {
                if (lo[b] == hi[b]) continue;
                const uint32_t differ = lo[b] ^ hi[b];
#pragma unroll 1
                for (int i = 0; i < 4; ++i)
                    if ((differ >> (8 * i)) & 0xffu)
                        lo[b] = (lo[b] & ~(0xffu << (8 * i))) |
                                (exact_code(exact_element<T>(a, w, j, at + 4 * b + i), scale) << (8 * i));
            }
            uint8_t *out = w.codes + (w.list[k] >> 8) * D + at;
            if constexpr (N == 8) *reinterpret_cast<uint2 *>(out) = make_uint2(lo[0], lo[1]);
            else *reinterpret_cast<uint32_t *>(out) = lo[0];
        }
    }
}

// Blocks: a CTA takes the blocks whose first token of this call lies among its
// tile_tokens entries; a warp takes one (block, KV head) of K or of V at a time.
// Shared memory: cos and sin of tile_tokens + 31 tokens.
template <typename T>
__device__ __forceinline__ void encode_blocks(const RopeArgs &a, int cta, float2 *table) {
    const int half = a.rotary_dim / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = cta % a.tile_splits;
    const int64_t t0 = (int64_t)(cta / a.tile_splits) * a.tile_tokens;
    const int nt = (int)min((int64_t)a.tile_tokens, a.num_tokens - t0);
    const int64_t limit = (int64_t)a.num_blocks * kBlockSize;

    // the leaders (a block's first token: none of the kWindow - 1 entries before
    // has the same block), and their blocks' rows
    __shared__ int s_low[kMaxTile], s_n[kMaxTile], s_count, s_last;
    __shared__ uint8_t s_lead[kMaxTile];                 // in order: CTAs that share a tile agree on it
    __shared__ int64_t s_blk[kMaxTile];
    __shared__ uint16_t s_list[kMaxTile][kBlockSize];
    if (threadIdx.x == 0) s_last = 0;
    if (threadIdx.x < kMaxTile) s_n[threadIdx.x] = 0;
    // this thread's first position and frequency, on their way while the leaders
    // are found
    const int t_first = half > 0 ? threadIdx.x / half : 0;
    const bool first_in = half > 0 && t0 + t_first < a.num_tokens && t_first < nt + kWindow - 1;
    const int32_t pos_first = first_in ? a.positions[t0 + t_first] : 0;
    const uint64_t turns_first = first_in ? a.turns[threadIdx.x - t_first * half] : 0;
    __syncthreads();
    for (int i = warp; i < nt; i += kRopeWarps) {
        const int64_t tok = t0 + i;
        const int64_t prev = tok - 1 - lane, far = prev - (kWindow - 1), next = tok + lane;
        const int64_t sp = lane < kWindow - 1 && prev >= 0 ? a.slot_mapping[prev] : -1;
        const int64_t sf = lane < kWindow - 1 && far >= 0 ? a.slot_mapping[far] : -1;
        const int64_t sn = next < a.num_tokens ? a.slot_mapping[next] : -1;
        const int64_t slot = __shfl_sync(kAll, sn, 0);
        if (slot >= limit && lane == 0) report(a.status, PA_DEV_BAD_SLOT);
        if (slot < 0 || slot >= limit) continue;
        const int64_t blk = slot / kBlockSize;
        // the block's tokens spread over more than kWindow entries: this one is
        // out of its leader's reach, or would lead a second time
        if (__any_sync(kAll, sf >= 0 && sf / kBlockSize == blk)) {
            if (lane == 0) report(a.status, PA_DEV_BAD_SLOT);
            continue;
        }
        if (__any_sync(kAll, sp >= 0 && sp / kBlockSize == blk)) continue;
        // rows: of two tokens with one slot the later one
        const bool mine = sn >= 0 && sn / kBlockSize == blk;
        const int off = mine ? (int)(sn % kBlockSize) : kBlockSize + lane;
        const unsigned same = __match_any_sync(kAll, off);
        const bool kept = mine && lane == 31 - __clz((int)same);
        const unsigned rows = __ballot_sync(kAll, kept);
        const int low = __reduce_min_sync(kAll, off);
        if (lane == 0) {
            atomicMax(&s_last, i + 31 - __clz((int)rows));
            s_low[i] = low;
            s_n[i] = __popc(rows);
            s_blk[i] = blk;
        }
        if (kept) s_list[i][__popc(rows & ((1u << lane) - 1u))] = (uint16_t)(lane | (off << 8));
    }
    __syncthreads();
    if (warp == 0) {
        static_assert(kMaxTile == 64, "two entries per lane");
        const unsigned lo = __ballot_sync(kAll, s_n[lane] > 0), hi = __ballot_sync(kAll, s_n[lane + 32] > 0);
        const unsigned below = (1u << lane) - 1u;
        if ((lo >> lane) & 1u) s_lead[__popc(lo & below)] = (uint8_t)lane;
        if ((hi >> lane) & 1u) s_lead[__popc(lo) + __popc(hi & below)] = (uint8_t)(lane + 32);
        if (lane == 0) s_count = __popc(lo) + __popc(hi);
    }
    __syncthreads();
    const int leads = s_count;
    if (leads == 0) return;
    const int pairs = (s_last + 1) * half;
    if ((int)threadIdx.x < pairs)
        table[t_first * a.table_row + threadIdx.x - t_first * half] = turn_of(pos_first, turns_first, (float)a.factor);
    for (int i = threadIdx.x + kRopeThreads; i < pairs; i += kRopeThreads) {
        const int t = i / half;
        table[t * a.table_row + i - t * half] = turn_of(a.positions[t0 + t], a.turns[i - t * half], (float)a.factor);
    }
    __syncthreads();

    const int per_lead = 2 * a.num_kv_heads;
    for (int item = warp + split * kRopeWarps; item < leads * per_lead; item += kRopeWarps * a.tile_splits) {
        const int rank = item / per_lead, rest = item - rank * per_lead, at = s_lead[rank];
        Tile w;
        w.value = rest >= a.num_kv_heads;
        w.h = w.value ? rest - a.num_kv_heads : rest;
        w.lead = at;
        w.tok = t0 + w.lead;
        w.low = s_low[at];
        w.n = s_n[at];
        w.list = s_list[at];
        const int64_t place = s_blk[at] * a.num_kv_heads + w.h;
        w.codes = static_cast<uint8_t *>(w.value ? a.value_cache : a.key_cache) + place * kBlockSize * a.head_dim;
        w.scale = (w.value ? a.v_scales : a.k_scales) + place;
        const float old = w.low > 0 ? *w.scale : 0.f;
        if constexpr (sizeof(T) == 2) {
            const int mode = w.value || half == 0 ? 0 : a.interleaved ? 2 : 1;
            if (a.head_dim == 128 && (mode == 0 || a.rotary_dim == 128)) {
                if (mode == 0) encode_units<0, 128>(a, w, old, table);
                else if (mode == 1) encode_units<1, 128>(a, w, old, table);
                else encode_units<2, 128>(a, w, old, table);
                continue;
            }
            if (a.unit_tiles || w.value) {
                if (mode == 0) encode_units_any<0>(a, w, old, table);
                else if (mode == 1) encode_units_any<1>(a, w, old, table);
                else encode_units_any<2>(a, w, old, table);
                continue;
            }
        }
        encode_any<T>(a, w, old, table);
    }
}

// Tokens of one block must lie within kWindow entries.  Those a little farther apart are
// seen (and dropped) where blocks are led; two groups farther apart are encoded by
// CTAs that know nothing of one another, so these CTAs look for them and flag the call.
// A CTA puts its own entries' blocks into a table in shared memory and looks up the
// entries of its part of the list behind them.  Quadratic, but of 8 bytes an entry and
// 1024 at a time: 40192 tokens of one head of 64 34.5 us, 33.2 without; 8192 tokens of 80
// heads of 128 62.3 / 62.2.  (Looking in the CTAs that encode, so that one group could be
// chosen and the others dropped, took 61 and 63.3 us.)
__device__ __forceinline__ void find_far(const RopeArgs &a, int cta, uint32_t *keys) {
    uint32_t *first = keys + kFarSlots;                  // an entry of the block at the same place
    const int owner = cta / a.far_parts, part = cta - owner * a.far_parts;
    const int64_t own = (int64_t)owner * kFarOwn, limit = (int64_t)a.num_blocks * kBlockSize;
    const int64_t lo = max(own, (int64_t)part * kFarPart), hi = min((int64_t)a.num_tokens, (int64_t)(part + 1) * kFarPart);
    if (lo >= hi) return;
    for (int i = threadIdx.x; i < kFarSlots; i += kRopeThreads) keys[i] = 0;
    __syncthreads();
    auto place_of = [](uint32_t blk) { return (blk * 2654435761u) >> 21; };
    static_assert(kFarSlots == 1 << 11, "place_of");
    for (int i = threadIdx.x; i < kFarOwn && own + i < a.num_tokens; i += kRopeThreads) {
        const int64_t slot = a.slot_mapping[own + i];
        if (slot < 0 || slot >= limit) continue;
        const uint32_t blk = (uint32_t)(slot / kBlockSize);
        for (uint32_t h = place_of(blk);; h = (h + 1) % kFarSlots) {
            const uint32_t old = atomicCAS(&keys[h], 0u, blk + 1);
            if (old == 0) first[h] = (uint32_t)(own + i);
            if (old == 0 || old == blk + 1) break;
        }
    }
    __syncthreads();
    bool far = false;
    for (int64_t e = lo + threadIdx.x; e < hi; e += 8 * kRopeThreads) {
        int64_t slot[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) slot[u] = e + u * kRopeThreads < hi ? a.slot_mapping[e + u * kRopeThreads] : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (slot[u] < 0 || slot[u] >= limit) continue;
            const uint32_t blk = (uint32_t)(slot[u] / kBlockSize);
            for (uint32_t h = place_of(blk); keys[h] != 0; h = (h + 1) % kFarSlots)
                if (keys[h] == blk + 1) {
                    const int64_t d = e + u * kRopeThreads - first[h];
                    far |= d >= kWindow || d <= -kWindow;
                    break;
                }
        }
    }
    if (far) report(a.status, PA_DEV_BAD_SLOT);
}

template <typename T, bool kBlocks>
__global__ void __launch_bounds__(kRopeThreads, 4) pa_rope_write_kernel(const RopeArgs a) {
    extern __shared__ __align__(16) float2 s_table[];
    grid_dependency_wait();
    grid_dependents_launch();
    if constexpr (kBlocks) {
        if ((int)blockIdx.x < a.far_ctas) {
            find_far(a, blockIdx.x, reinterpret_cast<uint32_t *>(s_table));
            return;
        }
        if ((int)blockIdx.x < a.far_ctas + a.tile_ctas) {
            encode_blocks<T>(a, blockIdx.x - a.far_ctas, s_table);
            return;
        }
    }
    turn_rows<T>(a, blockIdx.x - a.far_ctas - a.tile_ctas, s_table, !kBlocks);
}

// Numbers of about 106 bits, hi + lo with lo at most half a unit of hi's last place (T. J.
// Dekker, "A floating-point technique for extending the available precision", 1971).  A
// frequency has to hold 64 bits of a turn, as positions up to 2^31 multiply its
// error: in 53 bits the angle of position 2^31 would be off by 2^-25 of a turn.  Products are
// written with fma, so that a compiler has none to contract and every machine agrees.
struct Wide {
    double hi, lo;
};
Wide sum_of(double a, double b) {
    const double s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
Wide plus(Wide a, Wide b) {
    const Wide s = sum_of(a.hi, b.hi);
    return sum_of(s.hi, s.lo + (a.lo + b.lo));
}
Wide times(Wide a, Wide b) {
    const double p = a.hi * b.hi;
    return sum_of(p, std::fma(a.lo, b.hi, std::fma(a.hi, b.lo, std::fma(a.hi, b.hi, -p))));
}
Wide times(Wide a, double b) { return times(a, Wide{b, 0.0}); }
Wide over(Wide a, double b) {
    const double q = a.hi / b;
    return sum_of(q, (std::fma(-q, b, a.hi) + a.lo) / b);
}
// e^x, |x| below 700: 2^k e^r, e^r by its series at r / 512.
Wide exp_of(Wide x) {
    const double k = std::nearbyint(x.hi * 1.4426950408889634);
    Wide r = plus(x, times(Wide{0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56}, -k));      // ln 2
    r = {r.hi / 512.0, r.lo / 512.0};
    Wide e = {1.0, 0.0};
    for (int n = 9; n >= 1; --n) e = plus(Wide{1.0, 0.0}, over(times(r, e), n));         // |r|^10 / 10! is below 2^-126
    for (int n = 0; n < 9; ++n) e = times(e, e);
    return {std::ldexp(e.hi, (int)k), std::ldexp(e.lo, (int)k)};
}
// ln x: a step of Newton's method on e^y from y in 53 bits leaves about a third of the square of its error.
Wide log_of(double x) {
    const double y = std::log(x);
    const Wide f = plus(times(exp_of(Wide{-y, 0.0}), x), Wide{-1.0, 0.0});               // x e^-y - 1
    return plus(Wide{y, 0.0}, plus(f, times(times(f, f), -0.5)));
}
// The fraction of t, at least 0 and below 2^20, in units of 2^-64, to the nearest one modulo 1.
uint64_t fraction_of(Wide t) {
    const double f = t.hi - std::floor(t.hi), top = std::floor(f * 0x1p32);
    const double rest = (f * 0x1p32 - top) * 0x1p32;                                     // exact
    return ((uint64_t)top << 32) + (uint64_t)std::llround(rest + t.lo * 0x1p64);
}

double ramp_index(double turns, double dim, double base, double context) {
    return dim * log(context / (turns * 2.0 * M_PI)) / (2.0 * log(base));
}

template <typename T>
pa_status launch_rope(RopeArgs &a, bool blocks, cudaStream_t stream) {
    const int rows = a.num_q_heads + (blocks ? 0 : 2 * a.num_kv_heads);
    int64_t grid = plan_rows<T>(a, rows);
    a.unit_tiles = blocks && sizeof(T) == 2 && (a.interleaved || a.rotary_dim % 8 == 0);
    const int64_t n = a.num_tokens, sms = device_sms();
    // blocks: 16 tokens a CTA where there are enough, more where the KV heads are too
    // few to give each warp two tiles (and the table leaves room for two CTAs: 14554
    // tokens of one head of 256 47 us, 57 with 16 tokens a CTA)
    const int tile_most = std::min(kMaxTile, std::max(16, 16 * kRopeWarps / a.num_kv_heads));
    a.tile_tokens = 1;
    while (a.tile_tokens < tile_most && n / (2 * a.tile_tokens) >= 2 * sms &&
           (a.tile_tokens < 8 || (2 * a.tile_tokens + kWindow - 1) * a.table_row * (int)sizeof(float2) <= kMostTables))
        a.tile_tokens *= 2;
    size_t smem = (size_t)a.row_tokens * a.table_row * sizeof(float2);
    if (!blocks && a.whole && a.row_tokens >= 2) smem += (size_t)kAhead * 2 * kRopeThreads * sizeof(uint4);
    a.tile_ctas = a.far_ctas = 0;
    if (blocks) {
        if (n > kWindow) {
            a.far_parts = (int)((n + kFarPart - 1) / kFarPart);
            a.far_ctas = (int)((n + kFarOwn - 1) / kFarOwn * a.far_parts);
            grid += a.far_ctas;
            smem = std::max(smem, (size_t)2 * kFarSlots * sizeof(uint32_t));
        }
        const int items = 2 * a.num_kv_heads;
        // CTAs share a block's tiles where there are fewer than SMs, and where one would
        // have more than two a warp: it would end the grid alone (3696 tokens of 32 KV
        // heads of 128 50 us, 79 by one CTA, 58 with one tile a warp; of 64 52 / 85 / 53)
        a.tile_splits = (int)std::max<int64_t>(1, std::min<int64_t>((items + kRopeWarps - 1) / kRopeWarps,
                                                                    std::max<int64_t>(4 * sms / n, items / 16)));
        a.tile_ctas = (int)((n + a.tile_tokens - 1) / a.tile_tokens * a.tile_splits);
        grid += a.tile_ctas;
        smem = std::max(smem, (size_t)(a.tile_tokens + kWindow - 1) * a.table_row * sizeof(float2));
    }
    if (grid >= ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;
    auto kernel = blocks ? pa_rope_write_kernel<T, true> : pa_rope_write_kernel<T, false>;
    if (smem > 44 * 1024) {                          // with the static arrays above the default limit of 48 KiB
        cudaError_t e = allow_smem(kernel, kMostTables);
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

extern "C" pa_status pa_rotary_turns(uint64_t *turns, double *attention_factor, int rotary_dim, double base,
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
    Wide log_base = log_of(base);
    if (scaling == PA_ROTARY_NTK && rotary_dim > 2) log_base = plus(log_base, over(times(log_of(factor), d), d - 2.0));
    double lo = 0, hi = 1;
    if (scaling == PA_ROTARY_BY_PARTS) {
        lo = std::max(floor(ramp_index(beta_fast, d, base, original_context)), 0.0);
        hi = std::min(ceil(ramp_index(beta_slow, d, base, original_context)), d - 1.0);
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const Wide power = over(times(log_base, -2.0 * i), d);
        if (!(fabs(power.hi) < 700.0)) return PA_ERR_INVALID_ARG;
        Wide theta = exp_of(power);
        if (scaling == PA_ROTARY_LINEAR) theta = over(theta, factor);
        if (scaling == PA_ROTARY_BY_PARTS) {
            Wide r = hi - lo < 0.001 ? Wide{i > lo ? 1.0 : 0.0, 0.0} : over(Wide{i - lo, 0.0}, hi - lo);
            if (!(r.hi > 0.0)) r = Wide{0.0, 0.0};
            if (!(r.hi < 1.0)) r = Wide{1.0, 0.0};
            theta = plus(times(theta, plus(Wide{1.0, 0.0}, Wide{-r.hi, -r.lo})), times(over(theta, factor), r));
        }
        const Wide t = times(theta, Wide{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57});     // turns per position
        if (!(t.hi < 0x1p20)) return PA_ERR_INVALID_ARG;
        turns[i] = fraction_of(t);
    }
    *attention_factor = scaling == PA_ROTARY_BY_PARTS && factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0;
    return PA_OK;
}

extern "C" pa_status pa_rope_cache_write(void *query_out, const void *query, const void *key, const void *value,
                                         const int32_t *positions, const uint64_t *turns, double attention_factor,
                                         int rotary_dim, int interleaved, void *key_cache, void *value_cache,
                                         float *k_scales, float *v_scales, const int64_t *slot_mapping,
                                         int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                         int64_t query_out_stride, int64_t query_stride, int64_t key_stride,
                                         int64_t value_stride, int block_size, int num_blocks, pa_dtype dtype,
                                         pa_dtype cache_dtype, int32_t *device_status, void *stream) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || head_dim <= 0 || rotary_dim < 0 ||
        rotary_dim > head_dim || rotary_dim % 2 != 0 || block_size != kBlockSize || num_blocks <= 0 ||
        !(attention_factor >= 0x1p-20 && attention_factor <= 0x1p20))
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16) return PA_ERR_INVALID_ARG;
    if (cache_dtype != dtype && cache_dtype != PA_DTYPE_FP8_E4M3) return PA_ERR_INVALID_ARG;
    const bool blocks = cache_dtype == PA_DTYPE_FP8_E4M3;
    const int esize = dtype == PA_DTYPE_F32 ? 4 : 2;
    if (head_dim > 256 || (head_dim * esize) % 16 != 0 || (blocks && head_dim % 16 != 0)) return PA_ERR_UNSUPPORTED;
    if (blocks && num_tokens > kMostTokens) return PA_ERR_UNSUPPORTED;
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
    if (num_q_heads > 0) {
        // rows are read and written by many CTAs: query_out is query itself or apart from the inputs
        const int64_t n = num_tokens, qs = query_stride * esize, os = query_out_stride * esize, w = q_row * esize;
        const bool same = query == query_out && (query_stride == query_out_stride || n == 1);
        if ((!same && rows_touch(query_out, os, w, query, qs, w, n)) ||
            rows_touch(query_out, os, w, key, key_stride * esize, kv_row * esize, n) ||
            rows_touch(query_out, os, w, value, value_stride * esize, kv_row * esize, n))
            return PA_ERR_INVALID_ARG;
    }
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
