// Quantising a paged cache to 4 bits as it is written, with rotary positions on the
// new tokens' queries and keys, and reading it back ("PagedAttention por dentro",
// section "La tabla de páginas (block table)"; "KV cache: la memoria de trabajo que
// sostiene la inferencia LLM", section "Trucos para que el cuaderno sea más fino").
// The format is in pa_fp4.cuh, the mathematics of the angles in pa_rope.cu.
//
// Write.  Sixteen elements of a row are the unit: their scale depends on nothing
// else, so a token's row is written without a look at the rest of its block.  Two lanes
// take two units of a row (a thread one, where rows are not made of pairs of them):
// they turn the elements, find the scales and the codes, and store 8 bytes of codes and
// one of scale a unit.  Other CTAs of the launch turn the queries' rows.  8192 tokens of
// 64 query and 8 KV heads of 128, 311 MB in bf16, 59 us (5.3 TB/s, 0.78 of a copy): the query rows take 48
// alone and the keys and values 24, mostly arithmetic (440 instructions for the 16 elements of each
// of 32 lanes), which the rows' traffic hides but for some 11.  In f32, 613 MB, 99 us (0.92), as neighbours or
// half of the elements turned 117, not turned 108.  64 tokens of 32 KV heads 6 us.
//   A key's codes and scale are those of its exact rotation: where a 32-bit value
// lies so near a border of two codes that its error could cross it (or the largest
// magnitude so near one of two scales) it is computed again in 64 bits, and so is a whole unit whose
// pairs could leave f32's range on the way (8192 tokens of 8 KV heads of nothing but infinities: 1.5 ms).
//
// Read.  Blocks of the contexts become blocks of bf16 or f32 rows, a warp a tile.  It is
// bound by memory, four fifths of it the rows that are written: 65536 tokens of 8 KV heads
// of 128 to bf16, 312 MB, 51 us (6.1 TB/s, 0.91 of a copy); 777 tokens to f32 3.9 us.  Up to 8
// tiles a CTA: 4, 16 and 32 of them 52, 53 and 58 us; four units ahead of a lane's eight 53; tiles
// brought and taken by bulk copies through shared memory 51 and 4.5, and the kernels before and
// after such a one waited for its share of the L1 (write and read of 8192 tokens 79 us, 67 so).
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_fp4.cuh"
#include "pa_rope.cuh"

namespace pa {
namespace {

constexpr int kMostEncodeTokens = 16;            // tokens of a CTA that encodes

// Entry of pair `p` in a token's row of the table of cos and sin: 16 bytes of room
// behind every 16 pairs, so that lanes that read the pairs of neighbouring units meet
// in no bank.
__host__ __device__ constexpr int skewed(int p) { return p + (p >> 4) * 2; }

// 1 / x to 2^-22 of it (x a normal number).
__device__ __forceinline__ float inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Element d of a row of token `tok` in 64 bits.
template <typename T>
__device__ __forceinline__ double exact_of(const RopeArgs &a, const T *row, int64_t tok, int d) {
    int first, second, pair;
    if (!pair_of(a, d, &first, &second, &pair)) return (double)to_float(row[d]);
    // At position 0 nothing turns, and bf16 elements often are borders: one such token takes 8 us without sines, 13 to 21 with.
    if (a.positions[tok] == 0 && isfinite(to_float(row[first])) && isfinite(to_float(row[second])))
        return (double)to_float(row[d]) * a.factor;
    return exact_turn(to_float(row[first]), to_float(row[second]), d == second, a.positions[tok], a.turns[pair], a.factor);
}

// The larger of two magnitudes; NaN where one is.
__device__ __forceinline__ double larger(double a, double b) { return isnan(a) ? a : isnan(b) ? b : fmax(a, b); }

// The largest magnitude in 64 bits (NaN where one of them is) of those elements from d0 on that
// `which` has, which the unit's others do not reach.  (An element takes more than a microsecond: 64-bit units are few.  With all
// 16 of a unit 8192 tokens of 8 KV heads took 43 us, as one CTA had such a unit; with these 24.)
template <typename T>
__device__ __noinline__ double exact_top(const RopeArgs &a, const T *row, int64_t tok, int d0, uint32_t which) {
    double top = 0.0;
    for (; which != 0; which &= which - 1) top = larger(top, fabs(exact_of<T>(a, row, tok, d0 + __ffs((int)which) - 1)));
    return top;
}

// Error of elements turned in 32 bits from pairs of |x0| + |x1| up to `most`: infinite where one of them
// may leave f32's range on the way, so that the whole unit is found in 64 bits, which no f32 pair leaves.
// (At least the smallest normal number: products below it round by up to 2^-150, to zero too.)
__device__ __forceinline__ float turn_error(const RopeArgs &a, float most) {
    const float f = (float)a.factor, e = most * f >= 0x1p127f ? INFINITY : most * (kTurnError * f);
    return most > 0.f ? fmaxf(e, 0x1p-126f) : e;
}

// Whether the scale of a unit of largest magnitude amax, off by e, is asked for in 64 bits: the border
// that the 32-bit value was compared with lies within e, or the range's end, or another border may (the
// nearest lies amax / 32 away, below the first scale of a binade).
__device__ __forceinline__ bool scale_unsure(float amax, float border, float e) {
    return e > 0.f && (fabsf(amax - border) <= e || fabsf(amax - kFp4Top) <= e || amax <= 64.f * e);
}

// Midway between the magnitudes of codes c and c + 1, c at most 6.
__device__ __forceinline__ float code_border(uint32_t c) {
    return c < 4 ? 0.25f + 0.5f * (float)c : c == 4 ? 2.5f : c == 5 ? 3.5f : 5.f;
}

// Eight codes of -6 and of 6: `below` and `above` where nothing is known.
constexpr uint32_t kAllLow = 0xffffffffu, kAllHigh = 0x77777777u;

// Eight codes, of which `below` and `above` differ in some, from element d on of a row: those in 64 bits.
template <typename T, bool kTurned>
__device__ __noinline__ uint32_t exact_codes(const RopeArgs &a, const T *row, int64_t tok, int d, uint32_t below, uint32_t above,
                                             float scale) {
    uint32_t out = below;
    for (int i = 0; i < 8; ++i) {
        const uint32_t p = (below >> (4 * i)) & 15u, q = (above >> (4 * i)) & 15u;
        if (p == q) continue;
        uint32_t c = 0;                                  // a zero of either sign
        if (((p | q) & 7u) != 0) {
            const uint32_t most = max(p & 7u, q & 7u);
            const double x = kTurned ? exact_of<T>(a, row, tok, d + i) : (double)to_float(row[d + i]);
            c = ((p ^ q) & 8u) != 0 ? 0u : min(p & 7u, q & 7u);
            for (; c < most; ++c) {
                const double border = (double)(code_border(c) * scale);          // exact: 3 bits times 4
                if (!(fabs(x) > border || (fabs(x) == border && (c & 1u) != 0))) break;
            }
            c |= x < 0.0 ? 8u : 0u;
        }
        out = (out & ~(15u << (4 * i))) | (c << (4 * i));
    }
    return out;
}

// Encodes a unit, elements y of token tok's row from element d0 on.  most: the largest
// |x0| + |x1| of the pairs that were turned into them (0: none were).
template <typename T, bool kTurned>
__device__ __forceinline__ void encode16(const RopeArgs &a, const T *row, int64_t tok, int d0, const float (&y)[16], float most,
                                         uint8_t *codes, uint8_t *scale_at) {
    constexpr bool kSnapped = !kTurned && sizeof(T) == 2;
    uint32_t top = 0;                                    // as bits: magnitudes compare like integers, NaN above all
#pragma unroll
    for (int k = 0; k < 16; ++k) top = max(top, __float_as_uint(y[k]) & 0x7fffffffu);
    const float amax = __uint_as_float(top), e = kTurned ? turn_error(a, most) : 0.f;     // error of an element
    const bool wild = kTurned && e == INFINITY;
    bool nan = top > 0x7f800000u, beyond = amax > kFp4Top;
    float border = 0.f;
    uint32_t byte = fp4_scale_of(amax, amax, &border);
    if (kTurned && (wild || (!nan && scale_unsure(amax, border, e)))) {
        uint32_t which = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) which |= wild || fabsf(y[k]) >= amax - 2.f * e ? 1u << k : 0u;
        const double exact = exact_top<T>(a, row, tok, d0, which);
        nan = isnan(exact);
        beyond = exact > (double)kFp4Top;
        byte = fp4_scale_of<double>((float)exact, exact, &border);
    }
    if (!nan && beyond) report(a.status, PA_DEV_RANGE);
    if (nan) {
        *reinterpret_cast<uint2 *>(codes) = make_uint2(0u, 0u);
        *scale_at = (uint8_t)kFp4NanScale;
        return;
    }
    const float scale = fp4_scale_value(byte), inv = byte != 0 ? 1.f / scale : 0.f;
    // of a quotient, which is at most 6.4 near a border (larger ones saturate)
    const float eq = e * inv + 0x1p-20f;
    uint32_t out[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (kSnapped) {
                // A bf16 element divided by a scale of 4 bits is a border of two codes or at least
                // 2^-9 of it away; the product with the inverse is off by 2^-23, which rounding to
                // 16 bits takes back.
                lo[i] = __uint_as_float((__float_as_uint(y[8 * p + i] * inv) + 0x80u) & 0xffffff00u);
            } else {
                lo[i] = fmaf(y[8 * p + i], inv, -eq);
                hi[i] = fmaf(y[8 * p + i], inv, eq);
            }
        }
        out[p] = f32x8_to_e2m1x8(lo);
        if constexpr (!kSnapped) {
            // The codes of the value less and more its error: where they differ (in more than the
            // sign of a zero) the code comes from 64 bits.
            uint32_t above = f32x8_to_e2m1x8(hi);
            if (wild) out[p] = kAllLow, above = kAllHigh;
            if (out[p] != above) out[p] = exact_codes<T, kTurned>(a, row, tok, d0 + 8 * p, out[p], above, scale);
        }
    }
    *reinterpret_cast<uint2 *>(codes) = make_uint2(out[0], out[1]);
    *scale_at = (uint8_t)byte;
}

// How a key's elements are turned: not at all, as halves or as neighbours, where two
// lanes take two units of a row at a time, or in any way, where a thread takes one.
// (kPartHalves: some units are not turned; 8192 tokens of 64 query and 8 KV heads wholly turned took
// 68.6 us with its choices, 66.9 without.)
enum { kPlain = 0, kHalves = 1, kNeighbours = 2, kAny = 3, kPartHalves = 4 };

// Where a row of new keys or values lies.
template <typename T>
__device__ __forceinline__ const T *new_row(const RopeArgs &a, bool value, int64_t tok, int h) {
    return static_cast<const T *>(value ? a.value : a.key) + tok * (value ? a.v_stride : a.k_stride) + (int64_t)h * a.head_dim;
}

// Two lanes' part of two units, A and B, of a row that is read in whole vectors: the
// even lane has the first eight elements of each and finds A's scale, the odd one the
// others and B's.  With halves the units lie rotary_dim / 2 apart, else (and behind
// rotary_dim) they follow one another.  (Half the registers of a thread with both units: 64 leave
// the query rows' CTAs of the same kernel 32 warps on an SM.  They do not hold everything: by -Xptxas -v the turned
// kinds keep 172 to 188 bytes a thread in local memory in bf16, 100 to 116 in f32, rows that are not turned 92 and 36;
// 80 registers and no such bytes took 69 us for the 8192 tokens.)
template <typename T, int kMode>
struct Pair {
    static constexpr int N = Vec<T>::N, V = 8 / N;
    static constexpr bool kTurned = kMode != kPlain, kSnapped = !kTurned && sizeof(T) == 2;
    uint4 raw[2][V];
    // d: this lane's first element of A and of B
    __device__ __forceinline__ void load(const T *row, int d0, int d1) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) raw[u][v] = reinterpret_cast<const uint4 *>(row + (u ? d1 : d0))[v];
    }
    // tile: where the row's block goes; nullptr: nothing is written.  cs: the token's row of the table.  kValue: the
    // rows are values.  Whole warps.
    template <bool kValue>
    __device__ __forceinline__ void encode(const RopeArgs &a, int64_t tok, int h, const int (&d)[2], const float2 *cs, uint8_t *tile,
                                           int off) const {
        const bool odd = (threadIdx.x & 1) != 0, on = tile != nullptr;
        float y[2][8];
        uint32_t most[2] = {0, 0}, top[2] = {0, 0};      // the largest |x0| + |x1| of a pair, |y|: as bits, which compare like integers
        bool turns[2] = {kTurned, kTurned};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float w[N];
                Vec<T>::widen(raw[u][v], w);
#pragma unroll
                for (int i = 0; i < N; ++i) y[u][v * N + i] = w[i];
            }
        if constexpr (kMode == kHalves || kMode == kPartHalves) {
            // (elements past rotary_dim and a value's lane that goes along lie past the table)
            const bool r = kMode == kHalves || (on && d[0] < a.rotary_dim / 2);
            const float4 *c = reinterpret_cast<const float4 *>(cs + skewed(r && on ? d[0] : 0));
            turns[0] = turns[1] = r;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float4 w = c[i / 2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float p = y[0][i + k], q = y[1][i + k], cosine = k ? w.z : w.x, sine = k ? w.w : w.y;
                    most[0] = max(most[0], __float_as_uint(fabsf(p) + fabsf(q)));
                    y[0][i + k] = r ? p * cosine - q * sine : p;
                    y[1][i + k] = r ? q * cosine + p * sine : q;
                }
            }
            most[1] = most[0];
        } else if constexpr (kMode == kNeighbours) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int at = d[u] / 2, some = a.rotary_dim / 2 - at;       // of the four pairs, those that are turned
                const float4 *c = reinterpret_cast<const float4 *>(cs + skewed(some > 0 ? at : 0));
                turns[u] = some > 0;
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float4 w = c[i / 2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float p = y[u][2 * (i + k)], q = y[u][2 * (i + k) + 1], cosine = k ? w.z : w.x, sine = k ? w.w : w.y;
                        most[u] = max(most[u], __float_as_uint(fabsf(p) + fabsf(q)));
                        y[u][2 * (i + k)] = i + k < some ? p * cosine - q * sine : p;
                        y[u][2 * (i + k) + 1] = i + k < some ? q * cosine + p * sine : q;
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if constexpr (kSnapped) {
                // on the bf16 pairs as they came
                uint32_t m = 0;
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (uint32_t w : {raw[u][v].x, raw[u][v].y, raw[u][v].z, raw[u][v].w}) m = __vmaxu2(m, w & 0x7fff7fffu);
                top[u] = max(m << 16, m & 0xffff0000u);
            } else {
                if constexpr (kTurned) {
                    float m = 0.f;                       // passes over NaN: most then is one, or infinite
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[u][i]));
                    top[u] = __float_as_uint(m);
                }
                if (!kTurned || !(__uint_as_float(most[u]) * (float)a.factor < INFINITY)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) top[u] = max(top[u], __float_as_uint(y[u][i]) & 0x7fffffffu);
                }
            }
        }
        // each lane gets the whole of its own unit
        const uint32_t mine = max(odd ? top[1] : top[0], __shfl_xor_sync(kAll, odd ? top[0] : top[1], 1));
        float e = 0.f;                                   // error of an element of the lane's own unit
        if constexpr (kTurned) {
            const uint32_t m0 = turns[0] ? most[0] : 0u, m1 = turns[1] ? most[1] : 0u;
            e = turn_error(a, __uint_as_float(max(odd ? m1 : m0, __shfl_xor_sync(kAll, odd ? m0 : m1, 1))));
        }
        const float amax = __uint_as_float(mine);
        const bool nan = mine > 0x7f800000u, wild = kTurned && e == INFINITY;
        float border = 0.f;
        uint32_t byte = nan ? kFp4NanScale : fp4_scale_of(amax, amax, &border);
        bool beyond = !nan && amax > kFp4Top;
        if constexpr (kTurned) {
            const bool unsure = on && (wild || (!nan && scale_unsure(amax, border, e)));
            if (__any_sync(kAll, unsure)) {
                // both lanes' elements that may be the largest, in 64 bits: all of them where 32 say nothing
                const float floor = !unsure ? INFINITY : wild ? -INFINITY : amax - 2.f * e;
                const float other_floor = __shfl_xor_sync(kAll, floor, 1);
                uint32_t which[2] = {0, 0};
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) which[u] |= fabsf(y[u][i]) < (odd == (u == 1) ? floor : other_floor) ? 0u : 1u << i;
                const T *row = new_row<T>(a, false, tok, h);
                const double a0 = exact_top<T>(a, row, tok, d[0], which[0]), a1 = exact_top<T>(a, row, tok, d[1], which[1]);
                __syncwarp();
                const double exact = larger(odd ? a1 : a0, __shfl_xor_sync(kAll, odd ? a0 : a1, 1));
                if (unsure) {
                    byte = isnan(exact) ? kFp4NanScale : fp4_scale_of<double>((float)exact, exact, &border);
                    beyond = exact > (double)kFp4Top;
                }
            }
        }
        if (beyond && on) report(a.status, PA_DEV_RANGE);
        const float scale = fp4_scale_value(byte), inv = byte != 0 ? inverse(scale) : 0.f;
        const float other_inv = __shfl_xor_sync(kAll, inv, 1);
        float other_e = 0.f, other_scale = 0.f;
        if constexpr (kTurned) other_e = __shfl_xor_sync(kAll, e, 1);
        if constexpr (!kSnapped) other_scale = __shfl_xor_sync(kAll, scale, 1);
        if (!on) return;                                 // (no lane waits for this one from here on)
        const int D = a.head_dim;
        uint8_t *codes = tile + off * (D / 2);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const bool own = odd == (u == 1);
            const float f = own ? inv : other_inv;
            float lo[8];
            uint32_t out;
            if constexpr (kSnapped) {
                // A bf16 element divided by a scale of 4 bits is a border of two codes or at least 2^-9 of it
                // away; the product with the inverse is off by 2^-22, which rounding to multiples of 2^-16
                // (the last place of numbers from 128 to 256) takes back.
#pragma unroll
                for (int i = 0; i < 8; ++i) lo[i] = fmaf(y[u][i], f, 192.f) - 192.f;
                out = f32x8_to_e2m1x8(lo);
            } else {
                // The codes of the value less and more its error: where they differ (in more than the sign of a
                // zero) the code comes from 64 bits.  A quotient is at most 6.4 near a border (larger ones saturate).
                // bf16 elements that are not turned are rounded as above instead: they often are borders.
                const bool snap = sizeof(T) == 2 && kMode != kHalves && !turns[u];
                const float of_y = own ? e : other_e, eq = snap ? 0.f : of_y * f + 0x1p-18f, round = snap ? 192.f : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[u][i] = sizeof(T) == 2 && kMode != kHalves ? fmaf(y[u][i], f, round) - round : y[u][i] * f;
                    lo[i] = y[u][i] - eq;
                }
                out = f32x8_to_e2m1x8(lo);
#pragma unroll
                for (int i = 0; i < 8; ++i) lo[i] = y[u][i] + eq;
                uint32_t above = f32x8_to_e2m1x8(lo);
                if (kTurned && of_y == INFINITY) out = kAllLow, above = kAllHigh;
                if (out != above)
                    out = exact_codes<T, kTurned>(a, new_row<T>(a, kValue, tok, h), tok, d[u], out, above, own ? scale : other_scale);
            }
            *reinterpret_cast<uint32_t *>(codes + d[u] / 2) = isnan(f) ? 0u : out;
            if (own) tile[fp4_scales_at(D) + off * (D / 16) + d[u] / 16] = (uint8_t)byte;
        }
    }
};

// The unit from element d0 on of a row, turned in any way.
template <typename T, bool kTurned>
__device__ __noinline__ void encode_any(const RopeArgs &a, const T *row, int64_t tok, int d0, const float2 *cs, uint8_t *codes,
                                        uint8_t *scale) {
    constexpr int N = Vec<T>::N;
    const int rot = a.rotary_dim, half = rot / 2;
    float y[16], most = 0.f;
#pragma unroll
    for (int v = 0; v < 16 / N; ++v) {
        float x[N], o[N];
        if constexpr (kTurned) load_pairs<T>(row, d0 + v * N, rot, a.interleaved, x, o);
        else Vec<T>::widen(reinterpret_cast<const uint4 *>(row + d0)[v], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int d = d0 + v * N + i;
            y[v * N + i] = x[i];
            if constexpr (kTurned) {
                if (d < rot) {
                    const bool second = a.interleaved ? d & 1 : d >= half;
                    const float2 w = cs[skewed(a.interleaved ? d >> 1 : (second ? d - half : d))];
                    y[v * N + i] = second ? x[i] * w.x + o[i] * w.y : x[i] * w.x - o[i] * w.y;
                    most = fmaxf(most, fabsf(x[i]) + fabsf(o[i]));
                }
            }
        }
    }
    encode16<T, kTurned>(a, row, tok, d0, y, most, codes + d0 / 2, scale + d0 / 16);
}

// The keys' and values' units of a CTA's tokens.  A thread keeps its 16 elements' place in
// the rows, a unit (kAny) or a lane's part of two, and goes through the rows.
template <typename T, int kMode>
__device__ __forceinline__ void encode_tokens(const RopeArgs &a, int cta, float2 *table) {
    const int half = a.rotary_dim / 2, D = a.head_dim, per_row = D / 16, rows = 2 * a.num_kv_heads;
    const int per_pass = kRopeThreads / per_row;
    const int group = cta / a.tile_splits, split = cta - group * a.tile_splits;
    const int64_t t0 = (int64_t)group * a.tile_tokens, limit = (int64_t)a.num_blocks * kBlockSize;
    const int nt = (int)min((int64_t)a.tile_tokens, a.num_tokens - t0);
    const int table_row = skewed(a.table_row);
    const int item = threadIdx.x % per_row, place = threadIdx.x / per_row, first = place + split * per_pass;
    // row of the token, and the token: `rows` rows a token, per_pass * tile_splits rows on with every step
    int t = first / rows, row = first - t * rows;
    const int step = per_pass * a.tile_splits, step_t = step / rows, step_row = step - step_t * rows;
    auto next = [&]() {
        t += step_t;
        row += step_row;
        if (row >= rows) row -= rows, ++t;
    };
    // the tile and the row in it where the token goes (nullptr: it is not written)
    auto tile_of = [&](int *off) -> uint8_t * {
        if (place >= per_pass || t >= nt) return nullptr;
        const int64_t slot = a.slot_mapping[t0 + t];
        if (slot >= limit && row == 0 && item == 0) report(a.status, PA_DEV_BAD_SLOT);
        if (slot < 0 || slot >= limit) return nullptr;
        const bool value = row >= a.num_kv_heads;
        *off = (int)slot & (kBlockSize - 1);
        return static_cast<uint8_t *>(value ? a.value_cache : a.key_cache) +
               ((slot / kBlockSize) * a.num_kv_heads + (value ? row - a.num_kv_heads : row)) * fp4_tile_bytes(D);
    };
    auto make_table = [&]() {
        for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
            const int at = i / half, k = i - at * half;
            table[at * table_row + skewed(k)] = turn_of(a.positions[t0 + at], a.turns[k], (float)a.factor);
        }
        __syncthreads();
    };
    if constexpr (kMode == kAny) {
        make_table();
        for (; place < per_pass && t < nt; next()) {
            int off;
            uint8_t *tile = tile_of(&off);
            if (tile == nullptr) continue;
            const bool value = row >= a.num_kv_heads;
            const T *src = new_row<T>(a, value, t0 + t, value ? row - a.num_kv_heads : row);
            uint8_t *codes = tile + off * (D / 2), *scales = tile + fp4_scales_at(D) + off * per_row;
            if (value || 16 * item >= a.rotary_dim) encode_any<T, false>(a, src, t0 + t, 16 * item, nullptr, codes, scales);
            else encode_any<T, true>(a, src, t0 + t, 16 * item, table + t * table_row, codes, scales);
        }
    } else {
        // The first row's elements are on their way while the table is made.  Warps stay whole: lanes
        // without a row, or whose token has no slot, go along.
        Pair<T, kMode> x;
        uint8_t *tile;
        int off = 0, d[2], h, at;
        bool value;
        auto take = [&]() {
            at = min(t, nt - 1);
            value = row >= a.num_kv_heads;
            h = value ? row - a.num_kv_heads : row;
            const bool apart = !value && (kMode == kHalves || (kMode == kPartHalves && 32 * (item >> 1) < a.rotary_dim));
            d[0] = (apart ? 16 : 32) * (item >> 1) + 8 * (item & 1);
            d[1] = d[0] + (apart ? half : 16);
            tile = tile_of(&off);
            x.load(new_row<T>(a, value, t0 + at, h), d[0], d[1]);
        };
        take();
        if constexpr (kMode != kPlain) make_table();
        for (;;) {
            const bool any_key = __any_sync(kAll, tile != nullptr && !value), any_value = __any_sync(kAll, tile != nullptr && value);
            if (any_value)
                reinterpret_cast<const Pair<T, kPlain> &>(x).template encode<true>(a, t0 + at, h, d, nullptr, value ? tile : nullptr, off);
            __syncwarp();
            if (any_key) x.template encode<false>(a, t0 + at, h, d, table + at * table_row, value ? nullptr : tile, off);
            __syncwarp();
            next();
            if (!__any_sync(kAll, place < per_pass && t < nt)) break;
            take();
        }
    }
}

// The query rows of a CTA's tokens where halves are no whole vectors: a lane keeps up to
// kPairs pairs, those of its number and every 32nd behind it, and goes through the rows; it
// alone touches their elements, so that rows may be turned in place.  (8192 tokens of 64 heads of
// 128 of which 94 elements turn: 119 us, by vectors whose partners are read one by one 171.)
template <typename T, int kPairs>
__device__ __forceinline__ void turn_pair_rows(const RopeArgs &a, int cta, float2 *table) {
    constexpr int kRows = 16 / kPairs;                   // of a warp on their way
    const int half = a.rotary_dim / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = cta / a.row_splits, split = cta - group * a.row_splits;
    const int64_t t0 = (int64_t)group * a.row_tokens;
    const int nt = (int)min((int64_t)a.row_tokens, a.num_tokens - t0);
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int t = i / half;
        table[t * a.table_row + i - t * half] = turn_of(a.positions[t0 + t], a.turns[i - t * half], (float)a.factor);
    }
    __syncthreads();
    const int step = kRopeWarps * a.row_splits;
    // behind rotary_dim: elements up to a whole vector, then vectors
    constexpr int N = Vec<T>::N;
    const int edge = (a.rotary_dim + N - 1) / N * N, odd = edge - a.rotary_dim, vectors = (a.head_dim - edge) / N;
    const bool copies = a.query != a.query_out;
    for (int t = 0; t < nt; ++t) {
        const T *from = static_cast<const T *>(a.query) + (t0 + t) * a.q_stride;
        T *to = static_cast<T *>(a.query_out) + (t0 + t) * a.q_out_stride;
        float2 cs[kPairs];
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            if (lane + 32 * i < half) cs[i] = table[t * a.table_row + lane + 32 * i];
        for (int r = warp + split * kRopeWarps; r < a.num_q_heads; r += kRows * step) {
            T x[kRows][kPairs], y[kRows][kPairs], z[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u)
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const int p = lane + 32 * i;
                    if (p >= half || r + u * step >= a.num_q_heads) continue;
                    const T *row = from + (int64_t)(r + u * step) * a.head_dim;
                    x[u][i] = row[p];
                    y[u][i] = row[p + half];
                }
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                if (copies && lane < odd && r + u * step < a.num_q_heads)
                    z[u] = from[(int64_t)(r + u * step) * a.head_dim + a.rotary_dim + lane];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                if (r + u * step >= a.num_q_heads) break;
                T *out = to + (int64_t)(r + u * step) * a.head_dim;
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const int p = lane + 32 * i;
                    if (p >= half) break;
                    const float x0 = to_float(x[u][i]), x1 = to_float(y[u][i]);
                    out[p] = from_float<T>(x0 * cs[i].x - x1 * cs[i].y);
                    out[p + half] = from_float<T>(x1 * cs[i].x + x0 * cs[i].y);
                }
                if (copies && lane < odd) out[a.rotary_dim + lane] = z[u];
            }
        }
        if (copies)
            for (int i = threadIdx.x + split * kRopeThreads; i < a.num_q_heads * vectors; i += kRopeThreads * a.row_splits) {
                const int r = i / vectors, d = edge + (i - r * vectors) * N;
                *reinterpret_cast<uint4 *>(to + (int64_t)r * a.head_dim + d) =
                    *reinterpret_cast<const uint4 *>(from + (int64_t)r * a.head_dim + d);
            }
    }
}

template <typename T, int kMode>
__global__ void __launch_bounds__(kRopeThreads, kMode == kAny ? 3 : 4) pa_rope_write_fp4_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ __align__(16) float2 s_table[];
    grid_dependency_wait();
    grid_dependents_launch();
    // the two kinds spread evenly over the grid
    const int before = (int)((uint64_t)blockIdx.x * a.tile_ctas / gridDim.x);
    if ((int)((uint64_t)(blockIdx.x + 1) * a.tile_ctas / gridDim.x) > before) encode_tokens<T, kMode>(a, before, s_table);
    else if (a.whole) turn_rows<T>(a, blockIdx.x - before, s_table, false);
    else if (a.rotary_dim <= 128) turn_pair_rows<T, 2>(a, blockIdx.x - before, s_table);
    else turn_pair_rows<T, 4>(a, blockIdx.x - before, s_table);
}

template <typename T>
pa_status launch_write(RopeArgs &a, cudaStream_t stream) {
    const int64_t n = a.num_tokens, sms = device_sms();
    const int64_t row_ctas = plan_rows<T>(a, a.num_q_heads);
    const int half = a.rotary_dim / 2;
    a.tile_tokens = 1;
    while (a.tile_tokens < kMostEncodeTokens && n / (2 * a.tile_tokens) >= 4 * sms) a.tile_tokens *= 2;
    // units in pairs where rows are whole pairs of them and halves are whole units
    const bool pairs = a.head_dim % 32 == 0 && (half == 0 || a.interleaved || a.rotary_dim % 32 == 0);
    const int per_pass = kRopeThreads / (a.head_dim / 16);
    const int64_t passes = ((int64_t)a.tile_tokens * 2 * a.num_kv_heads + per_pass - 1) / per_pass;
    a.tile_splits = (int)std::max<int64_t>(1, std::min<int64_t>(passes, 4 * sms * a.tile_tokens / n));
    const int64_t tiles = (n + a.tile_tokens - 1) / a.tile_tokens * a.tile_splits, grid = tiles + row_ctas;
    if (grid >= ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;
    a.tile_ctas = (int)tiles;
    const size_t smem = std::max((size_t)a.tile_tokens * skewed(a.table_row), (size_t)a.row_tokens * a.table_row) * sizeof(float2);
    const auto kernel = !pairs          ? pa_rope_write_fp4_kernel<T, kAny>
                        : half == 0     ? pa_rope_write_fp4_kernel<T, kPlain>
                        : a.interleaved ? pa_rope_write_fp4_kernel<T, kNeighbours>
                        : a.rotary_dim < a.head_dim ? pa_rope_write_fp4_kernel<T, kPartHalves>
                                                    : pa_rope_write_fp4_kernel<T, kHalves>;
    // (16 tokens' tables of 144 entries or 32 rows' of 128, 8 bytes each: below the default limit of 48 KiB)
    cudaError_t e = launch_chained(kernel, dim3((unsigned)grid), dim3(kRopeThreads), smem, stream, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_rope_write_fp4_kernel launch");
    count_launches(1);
    return PA_OK;
}

// ---------------------------------------------------------------------------
// Reading back
// ---------------------------------------------------------------------------
constexpr int kReadWarps = 4;
constexpr int kMostTiles = 8;                    // of a CTA
constexpr int kReadAhead = 8;                    // units of a lane on their way

struct ReadArgs {
    void *key_out, *value_out;       // [num_seqs * width][num_kv_heads][16][head_dim]
    const uint8_t *key_cache, *value_cache;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;      // nullptr, or chunks whose rows each have their window
    int32_t *tables_out;             // nullptr, or [num_seqs][width]: where each block went
    uint32_t *ticket;                // nullptr, or a word to be zeroed
    int32_t *lens_out;               // with query_start: the lengths, -1 where a sequence's rows leave the query's
    int32_t *status;
    int num_seqs, num_kv_heads, head_dim;
    int max_blocks, num_blocks, width, window;
    int num_rows;                    // of the query
    int tiles, groups;               // tiles of a CTA; CTAs of a sequence
};

// f16 pair times f16 pair, exact, as two floats
__device__ __forceinline__ float2 product_of(uint32_t codes, uint32_t scale) {
    const uint32_t v = mul_f16x2(codes, scale);
    return make_float2(f16lo(v), f16hi(v));
}

// A CTA widens up to kMostTiles tiles of a sequence: of its table's entries in order, of
// an entry the keys' by KV head, then the values'.  Each warp takes every kReadWarps-th
// one.  A lane's unit is 16 bytes of rows; codes, scales and rows of a tile follow one
// another in the same order, so that its number is its place in each.
// kHalfValues: values become f16, which is what prefill's second product takes.
template <typename T, bool kHalfValues>
__global__ void __launch_bounds__(32 * kReadWarps) pa_read_fp4_kernel(const ReadArgs a) {
    constexpr int kUnit = 16 / (int)sizeof(T);           // elements
    grid_dependency_wait();
    grid_dependents_launch();
    const int D = a.head_dim, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / a.groups, group = blockIdx.x - b * a.groups, per_block = 2 * a.num_kv_heads;
    int64_t i0 = (int64_t)group * a.tiles, i1 = min(i0 + a.tiles, (int64_t)a.width * per_block);
    const int j0 = (int)(i0 / per_block);                // the CTA's first entry; lane k holds entry j0 + k
    int len = a.context_lens[b];
    const bool mine = (int64_t)(j0 + lane) * per_block < i1;
    int phys = mine ? a.block_tables[(int64_t)b * a.max_blocks + j0 + lane] : 0;
    if (len < 0 || len > a.width * kBlockSize) {
        if (threadIdx.x == 0 && group == 0) report(a.status, PA_DEV_BAD_CONTEXT_LEN);
        len = len < 0 ? 0 : a.width * kBlockSize;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.ticket != nullptr) *a.ticket = 0;
    if (warp == 0 && mine && a.tables_out != nullptr) a.tables_out[b * a.width + j0 + lane] = b * a.width + j0 + lane;
    int64_t chunk = 1;
    if (a.query_start != nullptr) {
        const int64_t from = a.query_start[b], end = a.query_start[b + 1];
        const bool outside = from < 0 || end < from || end > a.num_rows;
        chunk = end - from;
        if (threadIdx.x == 0 && group == 0) a.lens_out[b] = outside ? -1 : a.context_lens[b];
        if (outside || chunk == 0) return;               // no row attends to the context
    }
    // a chunk's first row is the one that looks farthest back
    const int64_t start = a.window > 0 ? max(len - chunk + 1 - a.window, (int64_t)0) : 0;
    const int first = (int)(start / kBlockSize), last = (len + kBlockSize - 1) / kBlockSize;     // entries that are read
    i0 = max(i0, (int64_t)first * per_block);
    i1 = min(i1, (int64_t)last * per_block);
    if (i0 >= i1) return;
    if (mine && j0 + lane >= first && j0 + lane < last && (unsigned)phys >= (unsigned)a.num_blocks) {
        if (warp == 0) report(a.status, PA_DEV_BAD_BLOCK_ID);
        phys = 0;
    }
    const int skip = (int)(i0 - (int64_t)j0 * per_block), all = skip + (int)(i1 - i0);     // tiles of the first entry that are not read
    for (int i = skip + warp; i < all; i += kReadWarps) {
        const int entry = i / per_block, tile = i - entry * per_block, j = j0 + entry;
        const int at = __shfl_sync(kAll, phys, entry);
        const bool value = tile >= a.num_kv_heads;
        const int h = value ? tile - a.num_kv_heads : tile;
        const uint8_t *codes = (value ? a.value_cache : a.key_cache) + ((int64_t)at * a.num_kv_heads + h) * fp4_tile_bytes(D);
        const uint8_t *scales = codes + fp4_scales_at(D);
        uint4 *rows = reinterpret_cast<uint4 *>(static_cast<T *>(value ? a.value_out : a.key_out) +
                                                ((int64_t)(b * a.width + j) * a.num_kv_heads + h) * kBlockSize * D);
        const int held = min(len - j * kBlockSize, kBlockSize) * (D / kUnit);    // units of rows of the context
        // (a tile is 32 units or a multiple of it)
        for (int u0 = lane; u0 < kBlockSize * D / kUnit; u0 += 32 * kReadAhead) {
            uint32_t c[kReadAhead], s[kReadAhead];
#pragma unroll
            for (int k = 0; k < kReadAhead; ++k) {
                const int u = u0 + 32 * k;
                if (u >= kBlockSize * D / kUnit) break;
                if constexpr (kUnit == 8) c[k] = reinterpret_cast<const uint32_t *>(codes)[u];
                else c[k] = reinterpret_cast<const uint16_t *>(codes)[u];
                s[k] = scales[u / (16 / kUnit)];
            }
#pragma unroll
            for (int k = 0; k < kReadAhead; ++k) {
                const int u = u0 + 32 * k;
                if (u >= kBlockSize * D / kUnit) break;
                uint32_t x[4];
                e2m1x8_to_f16x2x4(c[k], x);
                const uint32_t sc = fp4_scale_pair<0>(s[k]);
                float2 v[kUnit / 2];
#pragma unroll
                for (int i = 0; i < kUnit / 2; ++i) v[i] = product_of(x[i], sc);
                uint4 w;
                if (kHalfValues && value)
                    w = make_uint4(mul_f16x2(x[0], sc), mul_f16x2(x[1], sc), mul_f16x2(x[2], sc), mul_f16x2(x[3], sc));
                else if constexpr (kUnit == 4)
                    w = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
                else
                    w = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                                   pack_bf16x2(v[3].x, v[3].y));
                rows[u] = u < held ? w : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
}

template <typename T, bool kHalfValues = false>
pa_status launch_read(ReadArgs &a, cudaStream_t stream) {
    // a CTA has as many tiles as leave sixteen CTAs an SM, one a warp at least
    const int64_t per_seq = (int64_t)a.width * 2 * a.num_kv_heads;
    a.tiles = (int)std::max<int64_t>(kReadWarps, std::min<int64_t>(kMostTiles, a.num_seqs * per_seq / (16LL * device_sms())));
    const int64_t groups = (per_seq + a.tiles - 1) / a.tiles, grid = a.num_seqs * groups;
    if (grid >= ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;
    a.groups = (int)groups;
    const auto kernel = pa_read_fp4_kernel<T, kHalfValues>;
    cudaError_t e = launch_chained(kernel, dim3((unsigned)grid), dim3(32 * kReadWarps), 0, stream, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_read_fp4_kernel launch");
    count_launches(1);
    return PA_OK;
}

// Whether n bytes from p on meet m bytes from q on.
bool ranges_meet(const void *p, size_t n, const void *q, size_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && x < y + m && y < x + n;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sizes of head_dim that a pool's rows may have.
bool pool_head_dim(int head_dim) { return head_dim > 0 && head_dim <= 256 && head_dim % 16 == 0; }

// What prefill keeps in its workspace.  By tiles: the tensor-core kernel's own, tables,
// lengths, then the staged blocks.  By rows: chunks of a few rows and their lengths, then
// decode's.
struct Stage {
    bool by_rows;
    int chunks;
    size_t tables, lens, keys, values, bytes;
};

// Chunks of a few rows are rows of a decode, each of which (up to eight together, where a group has
// few heads) reads its context again, from L2: a tile of 256 rows takes a step of 128 positions
// 1.75 us however few rows it has, on one SM.
// The estimates that are compared: 12 us, a wave's steps and the staging at 5.5 TB/s, and a twentieth
// (tiles take up to a fifth more than that); decode's own, its waves' starts and 3 us.  Of 975 shapes measured
// both ways (1 to 256 chunks of 1 to 256 rows on 256 to 65536 tokens, groups of 8, 4 and 1: profiles/
// prefill_fp4_ways.csv) it takes the faster one or is within 12% of it (us, rows against tiles): one chunk on 8192
// tokens, 64 query and 8 KV heads, of 2 rows 16 : 150, of 64 123 : 160, of 256 408 : 160; 32 and 8 heads, of 16
// 24 : 150, of 64 65 : 160; 64 chunks on 2048 of 4 rows, 64 and 8 heads 126 : 259, 32 and 8 68 : 258, 8 and 8
// 40 : 258; 16 chunks of 16 on 256 30 : 19.
constexpr int kMostRows = 4096;
Stage stage_of(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int width, int num_rows, int max_query_len,
               int window) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    Stage s = {};
    if (num_rows <= kMostRows) {
        const int group = num_q_heads / num_kv_heads;
        const int64_t items = std::min(((int64_t)max_query_len * group + 255) / 256 * num_seqs,
                                       (int64_t)num_rows * group / 256 + num_seqs) * num_kv_heads;
        const int64_t seen = window > 0 ? std::min<int64_t>(width, ((int64_t)window + max_query_len) / kBlockSize + 2) : width;
        const double waves = (double)((items + device_sms() - 1) / device_sms());
        const double staged = (double)num_seqs * seen * num_kv_heads * 2 * (fp4_tile_bytes(head_dim) + 32.0 * head_dim) / 5.5e6;
        // a sequence's last chunk may be short
        const int each = decode_fp4_chunk_rows(num_q_heads, num_kv_heads);
        s.chunks = (int)std::min<int64_t>(num_rows, (int64_t)num_rows / each + num_seqs);
        size_t partials;
        const double rows = 3.0 + decode_fp4_chunks_time(s.chunks, num_q_heads, num_kv_heads, head_dim, width, window, &partials);
        if (rows < 1.05 * (12.0 + staged + waves * (double)((seen + 7) / 8) * 1.75)) {
            s.by_rows = true;
            s.lens = up((size_t)s.chunks * sizeof(int4));
            s.keys = s.lens + up((size_t)s.chunks * sizeof(int32_t));
            s.bytes = s.keys + partials;
            return s;
        }
    }
    const size_t pool = up((size_t)num_seqs * width * num_kv_heads * kBlockSize * head_dim * 2);
    s.tables = up(pa_prefill_workspace_bytes());
    s.lens = s.tables + up((size_t)num_seqs * width * sizeof(int32_t));
    s.keys = s.lens + up((size_t)num_seqs * sizeof(int32_t));
    s.values = s.keys + pool;
    s.bytes = s.values + pool;
    return s;
}

// The chunks, of `each` rows at most, that the sequences' rows are cut into, and how many positions
// the last row of each attends to; entries of no chunk have -1.  One CTA.
constexpr int kRowsThreads = 512;
__global__ void __launch_bounds__(kRowsThreads)
    pa_rows_fp4_kernel(const int32_t *query_start, const int32_t *context_lens, int4 *chunks, int32_t *chunk_lens, int num_chunks,
                       int each, int num_seqs, int num_rows, int max_query_len, int most, int32_t *status) {
    __shared__ int s_sum[kRowsThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int done = 0;                                        // chunks of the sequences before
    for (int b0 = 0; b0 < num_seqs; b0 += kRowsThreads) {
        const int b = b0 + threadIdx.x;
        int from = 0, rows = 0, len = 0, taken = 0;
        if (b < num_seqs) {
            from = query_start[b];
            len = context_lens[b];
            const int end = query_start[b + 1];
            if (from < 0 || end < from || end > num_rows || end - from > len || len > most) {
                report(status, PA_DEV_BAD_CONTEXT_LEN);
            } else {
                rows = end - from;
                if (rows > max_query_len) report(status, PA_DEV_BAD_QUERY_LEN);
                taken = min(rows, max_query_len);
            }
        }
        const int n = (taken + each - 1) / each;
        int before = n;                                  // this sequence's and those of the warp before it
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int x = __shfl_up_sync(kAll, before, k);
            before += lane >= k ? x : 0;
        }
        if (lane == 31) s_sum[warp] = before;
        __syncthreads();
        int all = 0, ahead = 0;
#pragma unroll
        for (int w = 0; w < kRowsThreads / 32; ++w) {
            ahead += w < warp ? s_sum[w] : 0;
            all += s_sum[w];
        }
        const int at = done + ahead + before - n;
        // chunk c of the sequence that has its first one at `to`
        auto put = [&](int c, int to, int seq, int first_row, int of_all, int seen) {
            const int first = c * each, here = min(each, of_all - first);
            // (more chunks than entries: rows that several sequences claim)
            if (to + c >= num_chunks) {
                report(status, PA_DEV_BAD_CONTEXT_LEN);
                return;
            }
            chunks[to + c] = make_int4(seq, first_row + first, here, 0);
            chunk_lens[to + c] = seen + first + here;
        };
        // a few chunks by the sequence's own thread, the others by its warp (64 sequences by the warp alone 6 us
        // longer, one of 64 chunks by its thread alone 2)
        constexpr int kOwn = 8;
        for (int c = 0; c < min(n, kOwn); ++c) put(c, at, b, from, taken, len - rows);
        for (unsigned left = __ballot_sync(kAll, n > kOwn); left != 0; left &= left - 1) {
            const int s = __ffs((int)left) - 1, count = __shfl_sync(kAll, n, s), to = __shfl_sync(kAll, at, s);
            const int s_from = __shfl_sync(kAll, from, s), s_taken = __shfl_sync(kAll, taken, s), seen = __shfl_sync(kAll, len - rows, s);
            for (int c = kOwn + lane; c < count; c += 32) put(c, to, b - lane + s, s_from, s_taken, seen);
        }
        done = min(done + all, num_chunks);
        __syncthreads();
    }
    for (int c = done + threadIdx.x; c < num_chunks; c += kRowsThreads) {
        chunks[c] = make_int4(-1, 0, 0, 0);
        chunk_lens[c] = 0;
    }
}

// Blocks of a sequence that are read: max_context_len's, or the table's where it is 0.
int width_of(int max_blocks_per_seq, int max_context_len) {
    if (max_context_len == 0) return max_blocks_per_seq;
    return std::min(max_blocks_per_seq, (int)(((int64_t)max_context_len + kBlockSize - 1) / kBlockSize));
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_rope_cache_write_fp4(void *query_out, const void *query, const void *key, const void *value,
                                             const int32_t *positions, const uint64_t *turns, double attention_factor,
                                             int rotary_dim, int interleaved, void *key_cache, void *value_cache,
                                             const int64_t *slot_mapping, int num_tokens, int num_q_heads,
                                             int num_kv_heads, int head_dim, int64_t query_out_stride,
                                             int64_t query_stride, int64_t key_stride, int64_t value_stride,
                                             int block_size, int num_blocks, pa_dtype dtype, int32_t *device_status,
                                             void *stream) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || head_dim <= 0 || rotary_dim < 0 ||
        rotary_dim > head_dim || rotary_dim % 2 != 0 || block_size != kBlockSize || num_blocks <= 0 ||
        !(attention_factor >= 0x1p-20 && attention_factor <= 0x1p20) || (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16))
        return PA_ERR_INVALID_ARG;
    if (!pool_head_dim(head_dim)) return PA_ERR_UNSUPPORTED;
    const int esize = dtype == PA_DTYPE_F32 ? 4 : 2;
    const int64_t q_row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    if (num_tokens == 0) return PA_OK;
    if (num_q_heads > 0 && (!query || !query_out || query_stride < q_row || query_out_stride < q_row ||
                            !aligned16(query) || !aligned16(query_out) || (query_stride * esize) % 16 != 0 ||
                            (query_out_stride * esize) % 16 != 0))
        return PA_ERR_INVALID_ARG;
    if (!key || !value || !key_cache || !value_cache || !slot_mapping || key_stride < kv_row || value_stride < kv_row ||
        !aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (key_stride * esize) % 16 != 0 || (value_stride * esize) % 16 != 0 ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PA_ERR_INVALID_ARG;
    if (rotary_dim > 0 && (!positions || !turns || !aligned4(positions) || (reinterpret_cast<uintptr_t>(turns) & 7u)))
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
    if ((q_row + 2 * kv_row) * kMostEncodeTokens >= ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;
    RopeArgs a = {};
    a.query = query;
    a.key = key;
    a.value = value;
    a.query_out = query_out;
    a.key_cache = key_cache;
    a.value_cache = value_cache;
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
    return dtype == PA_DTYPE_F32 ? launch_write<float>(a, st) : launch_write<__nv_bfloat16>(a, st);
}

extern "C" pa_status pa_cache_read_fp4(void *key_out, void *value_out, const void *key_cache, const void *value_cache,
                                       const int32_t *block_tables, const int32_t *context_lens, int num_seqs,
                                       int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                                       int num_blocks, int max_context_len, int window, pa_dtype dtype,
                                       int32_t *device_status, void *stream) {
    if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size != kBlockSize || max_blocks_per_seq < 0 ||
        max_blocks_per_seq > 0x7fffffff / kBlockSize || num_blocks <= 0 || max_context_len < 0 || window < 0 ||
        (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16))
        return PA_ERR_INVALID_ARG;
    if (!pool_head_dim(head_dim)) return PA_ERR_UNSUPPORTED;
    const int width = width_of(max_blocks_per_seq, max_context_len);
    if (num_seqs == 0 || width == 0) return PA_OK;
    if (!key_out || !value_out || !key_cache || !value_cache || !block_tables || !context_lens || !aligned16(key_out) ||
        !aligned16(value_out) || !aligned16(key_cache) || !aligned16(value_cache) || !aligned4(block_tables) ||
        !aligned4(context_lens))
        return PA_ERR_INVALID_ARG;
    // units of a block and blocks of a call are counted in 32 bits
    if ((int64_t)num_kv_heads * 4 * head_dim >= ((int64_t)1 << 30) || (int64_t)num_seqs * width >= ((int64_t)1 << 31))
        return PA_ERR_UNSUPPORTED;
    const size_t in = (size_t)num_blocks * num_kv_heads * fp4_tile_bytes(head_dim);
    const size_t out = (size_t)num_seqs * width * num_kv_heads * kBlockSize * head_dim * (dtype == PA_DTYPE_F32 ? 4 : 2);
    for (const void *o : {key_out, value_out})
        if (ranges_meet(o, out, key_cache, in) || ranges_meet(o, out, value_cache, in) ||
            ranges_meet(o, out, block_tables, (size_t)num_seqs * max_blocks_per_seq * sizeof(int32_t)) ||
            ranges_meet(o, out, context_lens, (size_t)num_seqs * sizeof(int32_t)))
            return PA_ERR_INVALID_ARG;
    if (ranges_meet(key_out, out, value_out, out)) return PA_ERR_INVALID_ARG;
    ReadArgs a = {};
    a.key_out = key_out;
    a.value_out = value_out;
    a.key_cache = static_cast<const uint8_t *>(key_cache);
    a.value_cache = static_cast<const uint8_t *>(value_cache);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.width = width;
    a.window = window;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PA_DTYPE_F32 ? launch_read<float>(a, st) : launch_read<__nv_bfloat16>(a, st);
}

extern "C" size_t pa_prefill_fp4_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                                 int max_blocks_per_seq, int num_query_tokens, int max_query_len,
                                                 int max_context_len, int window) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || head_dim != 128 ||
        max_blocks_per_seq < 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize || num_query_tokens < 0 || max_query_len < 0 ||
        max_context_len < 0 || window < 0)
        return (size_t)-1;
    return stage_of(num_seqs, num_q_heads, num_kv_heads, head_dim, width_of(max_blocks_per_seq, max_context_len),
                    num_query_tokens, max_query_len, window).bytes;
}

extern "C" pa_status pa_prefill_fp4(void *out, const void *query, const void *key_cache, const void *value_cache,
                                    const int32_t *block_tables, const int32_t *context_lens,
                                    const int32_t *query_start, int num_seqs, int num_q_heads, int num_kv_heads,
                                    int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                                    int num_query_tokens, int max_query_len, int max_context_len, float scale, int window,
                                    void *workspace, size_t workspace_bytes, int32_t *device_status, void *stream) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || head_dim <= 0 ||
        block_size != kBlockSize || max_blocks_per_seq < 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize ||
        num_blocks <= 0 || num_query_tokens < 0 || max_query_len < 0 || max_context_len < 0 || window < 0 ||
        !(scale == scale))
        return PA_ERR_INVALID_ARG;
    const int group = num_q_heads / num_kv_heads;
    if (head_dim != 128 || (group != 1 && group != 2 && group != 4 && group != 8 && group != 16)) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_query_tokens == 0 || max_query_len == 0) return PA_OK;
    const int width = width_of(max_blocks_per_seq, max_context_len);
    if (!out || !query || !key_cache || !value_cache || !context_lens || !query_start || !block_tables || width == 0 ||
        !aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(query_start))
        return PA_ERR_INVALID_ARG;
    const int64_t staged = (int64_t)num_seqs * width;
    if ((int64_t)num_kv_heads * 4 * head_dim >= ((int64_t)1 << 30) || staged * num_kv_heads * kBlockSize >= ((int64_t)1 << 31))
        return PA_ERR_UNSUPPORTED;
    const Stage s = stage_of(num_seqs, num_q_heads, num_kv_heads, head_dim, width, num_query_tokens, max_query_len, window);
    if (workspace == nullptr || workspace_bytes < s.bytes || !aligned16(workspace)) return PA_ERR_WORKSPACE;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    if (s.by_rows) {
        int4 *chunks = reinterpret_cast<int4 *>(w);
        int32_t *chunk_lens = reinterpret_cast<int32_t *>(w + s.lens);
        const cudaError_t e = launch_chained(pa_rows_fp4_kernel, dim3(1), dim3(kRowsThreads), 0, static_cast<cudaStream_t>(stream),
                                             query_start, context_lens, chunks, chunk_lens, s.chunks,
                                             decode_fp4_chunk_rows(num_q_heads, num_kv_heads), num_seqs, num_query_tokens,
                                             max_query_len, width * kBlockSize, device_status);
        if (e != cudaSuccess) return cuda_failure(e, "pa_rows_fp4_kernel launch");
        count_launches(1);
        return decode_fp4_chunks(out, query, key_cache, value_cache, block_tables, chunk_lens, chunks, s.chunks,
                                 num_query_tokens, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, width, num_blocks,
                                 scale, window, w + s.keys, s.bytes - s.keys, device_status, stream);
    }
    ReadArgs a = {};
    a.key_out = w + s.keys;
    a.value_out = w + s.values;
    a.key_cache = static_cast<const uint8_t *>(key_cache);
    a.value_cache = static_cast<const uint8_t *>(value_cache);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.tables_out = reinterpret_cast<int32_t *>(w + s.tables);
    a.lens_out = reinterpret_cast<int32_t *>(w + s.lens);
    a.ticket = reinterpret_cast<uint32_t *>(w);
    a.num_rows = num_query_tokens;
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.width = width;
    a.window = window;
    const pa_status rc = launch_read<__nv_bfloat16, true>(a, static_cast<cudaStream_t>(stream));
    if (rc != PA_OK) return rc;
    return prefill_f16_values(out, query, a.key_out, a.value_out, a.tables_out, a.lens_out, query_start, num_seqs, num_q_heads,
                              num_kv_heads, head_dim, width, (int)staged, num_query_tokens, max_query_len, scale, window, w,
                              s.tables, device_status, stream);
}
