// Chunked (paged) prefill attention over E4M3 pools with one scale per block of
// 16 tokens and KV head, on 5th-generation tensor cores ("PagedAttention por
// dentro", section "Chunked prefill integrado con paged KV"; "KV cache: la
// memoria de trabajo que sostiene la inferencia LLM", section "Trucos para que
// el cuaderno sea más fino").  The mathematics of the scales is in
// pa_block8.cuh: a block's key scale multiplies its 16 columns of scores, the
// logarithm of its value scale is added to them, and the sum of its weights is
// divided by the value scale.
//
// One CTA computes two 128-row tiles (A, then B) of (token, query head of the
// group) rows of one sequence and KV head over 128-position K/V tiles.
//   Q K^T runs on the codes as they are (kind::f8f6f4).  A bf16 query has 8
//   significant bits and E4M3 has 4, so a query row is the sum of two rows of
//   codes times a power of two, q = 2^e (q1 + q2) with q1 the nearest code and
//   q2 the rest, exact but for elements below 2^-9 of the row's largest, which
//   are off by at most 2^-17 of it; S = Q1 K^T + Q2 K^T at the 8-bit rate costs
//   what one 16-bit product would, and K is not touched.
//   P V runs on f16: the weights need 11 bits (bf16's 8 would be too coarse for
//   the output), so V's codes are widened to f16 (exact) in shared memory.
//   warp 0       TMA producer: both Q tiles, then the K and V codes of each step;
//   warp 1       MMA issuer, ping-pong between the tiles:
//                  S_A(0) S_B(0) | PV_A(j) S_A(j+1) PV_B(j) S_B(j+1) | ...
//                S and O += P V accumulate in tensor memory, P is read from
//                tensor memory, written there over its own S;
//   warps 2..9   softmax of tile A, warps 10..17 of tile B: two threads per row,
//                64 of the 128 columns of S and O each, one pass over S per step
//                against an integer reference that rises only when a chunk's
//                weights would leave f16's range; they also split their Q tile;
//   warps 18, 19 widen each V tile, zeroing positions outside the item's range,
//                and stage the scales of the step after.
// With fewer items than SMs each is cut along its context into parts, whose
// (reference, sum, output) a second kernel merges: a chunk of a few tokens over a
// long context would otherwise keep one SM per KV head busy (16 tokens on 8192
// with 8 KV heads: 123 us whole, 28 us in 16 parts).
// 16 chunks of 512 tokens on contexts of up to 8192 with 64 query heads on 8: 940 us,
// 1133 TFLOP/s (0.66 of the sustained 16-bit rate).  A step of 128 positions takes
// about 3400 cycles, of which the tensor pipe is busy for 2048 (Q K^T 8-bit, both
// halves of the query, 1024; P V 1024); the rest is the exchange between softmax and
// MMA that two tiles in turn do not hide, and some 20000 cycles at an item's ends
// (split of the query, first step, output).  K and V widened to f16 for a 16-bit
// Q K^T took 1308 us.
// Persistent CTAs take items from a ticket counter; barrier phases are counted
// across items, so an item's loads start under the end of the one before.
// Every wait is bounded (about a second); one that gives up sets PA_DEV_TIMEOUT,
// the CTA drains its tensor-core work and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "pa_block8.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;               // rows per Q tile (M of every MMA)
constexpr int kQT = 2;                   // Q tiles per CTA
constexpr int kKv = 128;                 // positions per step (8 blocks)
constexpr int kD = 128;                  // head_dim
constexpr int kHalf = 16384;             // one 64-column swizzled region of a tile
constexpr int kTile = 2 * kHalf;         // 128 rows x 256 bytes
constexpr int kCols = 64;                // S / O columns per softmax thread (two per row)
constexpr int kGroup = 2 * kRows;        // softmax threads per Q tile
constexpr int kWidenWarp0 = 2 + kQT * kGroup / 32;
constexpr int kWidenThreads = 64;
constexpr int kThreads = kWidenWarp0 * 32 + kWidenThreads;   // 640: one warp more would cost 16 registers a thread
constexpr int kCodeTile = kKv * kD;      // codes of a K or V tile
constexpr int kKStages = 3;              // K code tiles
constexpr int kCodeStages = 2;           // V code tiles
constexpr int kVStages = 2;              // f16 V tiles
constexpr int kScaleSlots = 4;
constexpr int kPartSteps = 3;            // steps of a part at least

constexpr float kChunkSumMax = 32768.f;  // largest weight sum of a 32-column chunk kept as computed: f16 holds its weights
constexpr size_t kWorkspaceBytes = 256;  // the ticket counter (rounded up)

// shared memory map (offsets from the 1024-byte aligned dynamic base)
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kQT * kTile;
constexpr int kOffV = kOffK + kKStages * kCodeTile;
constexpr int kOffCode = kOffV + kVStages * kTile;
constexpr int kOffScale = kOffCode + kCodeStages * kCodeTile;    // float4 [kScaleSlots][8]
constexpr int kOffQScale = kOffScale + kScaleSlots * 8 * 16;     // float [kQT][128]
constexpr int kOffRed = kOffQScale + kQT * kRows * 4;        // float [kQT][2 parities][2][128]
constexpr int kPermMax = 64;
constexpr int kOffPerm = kOffRed + kQT * 2 * 2 * kRows * 4;      // int [kPermMax]
constexpr int kOffBar = kOffPerm + kPermMax * 4;

constexpr int kQFull = 0, kQFree = 1, kDrain = 2, kQSplit = 3, kKFull = kQSplit + kQT, kKEmpty = kKFull + kKStages,
              kCodeFull = kKEmpty + kKStages, kCodeEmpty = kCodeFull + kCodeStages, kVConv = kCodeEmpty + kCodeStages,
              kVEmpty = kVConv + kVStages, kSFull = kVEmpty + kVStages, kPFull = kSFull + kQT, kPvDone = kPFull + kQT,
              kOFree = kPvDone + kQT, kItemFull = kOFree + kQT, kItemEmpty = kItemFull + 2,
              kScaleFull = kItemEmpty + 2, kEnd = kScaleFull + kScaleSlots, kNumBars = kEnd + 1;
constexpr int kOffMisc = kOffBar + kNumBars * 8;                 // TMEM slot, failure flag, item order, item queue [2], NaN marks [4], items taken [4]
constexpr int kSmemBytes = kOffMisc + 64;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

constexpr uint32_t kTmemCols = 512;      // S_A, S_B, O_A, O_B
__device__ __forceinline__ uint32_t col_s(int x) { return (uint32_t)(x * kKv); }
__device__ __forceinline__ uint32_t col_o(int x) { return (uint32_t)(kQT * kKv + x * kD); }

__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// D[tmem] (+)= A[smem] * B[smem], both E4M3; issued by one thread.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: E4M3 operands (format 0), K-major, f32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

struct PrefillArgs {
    void *out;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;
    const float *k_scales;
    const float *v_scales;
    const uint8_t *value_cache;
    int32_t *status;
    int num_seqs, num_q_heads, num_kv_heads, group;
    int max_blocks, num_blocks;
    int num_query_tokens, max_query_len;
    int window;
    float scale_log2;
    int n_mt;                            // pair tiles per (sequence, KV head)
    int num_items;
    unsigned int *work_counter;          // nullptr: one item per CTA
    int splits;                          // parts an item is cut into at most
    float *part_o;                       // [(token * Hq + head) * splits + part][128]
    float2 *part_ml;                     // (reference, sum)
};

// A phase that is complete passes at once; the failure flag (another shared
// memory round trip) is looked at only before a wait that may last.
__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, volatile int *fail, int32_t *status) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*fail) return false;
    if (mbar_wait_bounded(bar, parity)) return true;
    *fail = 1;
    report(status, PA_DEV_TIMEOUT);
    return false;
}

// A bounded wait whose outcome is the same for every lane of the warp (the
// tensor-memory instructions after it are warp-wide).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *fail, int32_t *status) {
    return __all_sync(0xffffffffu, wait_or_fail(bar, parity, fail, status));
}

// pairs of floats for f32x2 arithmetic
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^(a - b) for references a <= b that are integers or -inf: exact, 0 when a is
// -inf or far below b.
__device__ __forceinline__ float pow2_diff(float a, float b) {
    if (a == b) return 1.f;
    if (!(a > -INFINITY) || !(b - a < 256.f)) return 0.f;
    return ldexpf(1.f, (int)(a - b));
}

// A block's scales as the softmax uses them: x = key scale * softmax scale *
// log2(e), y = log2 of the value scale, z = 1 / value scale.
//
// The general form of a 32-column chunk's weights (S at taddr, first column at
// position kc, its two blocks' scales e[0], e[1], the row's query scale qs), for chunks that some row sees
// only in part and for those whose weights would grow past the reference's
// range: a row whose largest attended exponent is more than 2^10 above its
// reference (or has none) raises it to the next integer at or above.  The
// weights replace S as 16 f16 pairs.  Returns (weights divided by the value
// scales, summed; reference).  Out of line, so that the common path is short and
// keeps its registers; called by all lanes of a warp.
__device__ __noinline__ float2 chunk_weights_general(uint32_t taddr, const float4 *e, float qs, float ref, int kc, int qpos,
                                                     int wlo) {
    const int lo = wlo - kc, hi = qpos - kc;         // attended columns
    if (__all_sync(0xffffffffu, hi < 0 || lo > 31)) {
        // past the diagonal (or before the window) for all of the warp's rows
        uint32_t zero[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) zero[i] = 0u;
        tmem_st16(taddr, zero);
        return make_float2(0.f, ref);
    }
    uint32_t v[32];
    tmem_ld32(taddr, v);
    tmem_wait_ld();
    float rmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float x = i >= lo && i <= hi ? fmaf(__uint_as_float(v[i]), e[i >> 4].x * qs, e[i >> 4].y) : -INFINITY;
        v[i] = __float_as_uint(x);
        rmax = fmaxf(rmax, x);
    }
    if (rmax > ref + 10.f) ref = ceilf(rmax);
    // before a row has seen anything its weights are 0: any finite reference does
    const float r = ref == -INFINITY ? 0.f : ref;
    uint32_t pp[16];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float p0 = ex2_fast(__uint_as_float(v[i]) - r), p1 = ex2_fast(__uint_as_float(v[i + 1]) - r);
        sum[i >> 4] += p0 + p1;
        pp[i >> 1] = pack_f16x2(p0, p1);
    }
    tmem_st16(taddr, pp);
    return make_float2(fmaf(sum[0], e[0].z, sum[1] * e[1].z), ref);
}

// Scales the f16 weights of this thread's two 32-column chunks by f0 and f1.
__device__ __noinline__ void scale_chunk_weights(uint32_t taddr, float f0, float f1) {
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
        const float f = c == 0 ? f0 : f1;
        uint32_t w[32];
        tmem_ld32(taddr + c, w);
        tmem_wait_ld();
        uint32_t q[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = pack_f16x2(f16lo(w[i]) * f, f16hi(w[i]) * f);
        tmem_st16(taddr + c, q);
    }
    tmem_wait_st();
}

// x + 0 * w per half: NaN once w was (w finite otherwise).
__device__ __forceinline__ void note_nan(uint32_t &x, uint32_t w) {
    asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(x) : "r"(w), "r"(0u));
}

// Zeroes the NaNs among a widening thread's f16 values of a V tile; true if there
// were any (rows outside the item's range are zero already).
template <int kRowStep>
__device__ __noinline__ bool clear_nan(uint8_t *dst, int at0, int at1) {
    uint32_t seen[2] = {0u, 0u};
#pragma unroll 4
    for (int i = 0; i < kKv / kRowStep; ++i) {
        const uint4 x = *reinterpret_cast<const uint4 *>(dst + i * kRowStep * 128 + at0);
        const uint4 y = *reinterpret_cast<const uint4 *>(dst + i * kRowStep * 128 + at1);
        note_nan(seen[0], x.x), note_nan(seen[1], x.y), note_nan(seen[0], x.z), note_nan(seen[1], x.w);
        note_nan(seen[0], y.x), note_nan(seen[1], y.y), note_nan(seen[0], y.z), note_nan(seen[1], y.w);
    }
    if (((seen[0] | seen[1]) & 0x7fff7fffu) == 0u) return false;
#pragma unroll 1
    for (int i = 0; i < 2 * kKv / kRowStep; ++i) {
        uint32_t *p = reinterpret_cast<uint32_t *>(dst + (i >> 1) * kRowStep * 128 + (i & 1 ? at1 : at0));
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            uint32_t w = p[k];
            if ((w & 0x7fffu) > 0x7c00u) w &= 0xffff0000u;
            if ((w & 0x7fff0000u) > 0x7c000000u) w &= 0xffffu;
            p[k] = w;
        }
    }
    return true;
}

// Steps that every row of an item attends to whole begin in [lo, hi].  In the other
// ones NaN codes of V are 0 in the widened tile.
struct Whole {
    int lo, hi;
    __device__ __forceinline__ bool has(int k0) const { return k0 >= lo && k0 <= hi; }
};

// NaN codes among the 64 columns that a thread holds of O (V's columns from
// `column` on), at those positions of `steps` steps from block blk_lo on, in steps
// that some row attends to only in part, that its row, at position qpos, attends
// to: these elements of O become NaN.  (The NaNs of the other steps went through
// the product.)  A whole warp, whose lanes read 8 positions' codes at a time; the
// steps with a part of the diagonal or of the window's start are few whatever the
// context's length.  16 chunks of 512 tokens on contexts of up to 8192, NaN codes in
// every chunk: 1.08 ms, 0.95 without.  (Each thread reading all positions of its row for
// itself took 239 ms, and other warps wait a second at most.)
__device__ __noinline__ void poison_output(const PrefillArgs &a, uint32_t o_base, int b, int kvh, int column, int blk_lo,
                                           int steps, int kv_hi, Whole whole, int qpos) {
    const int32_t *table = a.block_tables + (int64_t)b * a.max_blocks;
    const int lane = threadIdx.x & 31;
    const int first = a.window > 0 ? qpos + 1 - a.window : 0;
    uint64_t mask = 0;
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
        const int k0 = blk_lo * kBlockSize + j * kKv;
        if (whole.has(k0)) continue;
#pragma unroll 1
        for (int p0 = k0; p0 < min(k0 + kKv, kv_hi); p0 += 8) {
            const int p = p0 + (lane >> 2);
            uint32_t nans = 0;                       // one bit for each of 16 codes
            if (p < kv_hi) {
                const int phys = table[p / kBlockSize];
                const int64_t tile = (int64_t)((unsigned)phys < (unsigned)a.num_blocks ? phys : 0) * a.num_kv_heads + kvh;
                const uint4 w = *reinterpret_cast<const uint4 *>(
                    a.value_cache + (tile * kBlockSize + p % kBlockSize) * kD + column + (lane & 3) * 16);
                const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // the top bit of each byte that is 0x7f without its sign; then side by side
                    const uint32_t top = ((words[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    nans |= (((top >> 7) * 0x01020408u) >> 24) << (4 * k);
                }
            }
            uint32_t hits = __ballot_sync(0xffffffffu, nans != 0);
            while (hits != 0) {
                const int src = __ffs(hits) - 1, at = p0 + (src >> 2);
                hits &= hits - 1;
                const uint32_t bits = __shfl_sync(0xffffffffu, nans, src);
                if (at >= first && at <= qpos) mask |= (uint64_t)bits << (16 * (src & 3));
            }
        }
    }
    __syncwarp();
#pragma unroll 1
    for (int c = 0; c < kCols; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_base + c, o);
        tmem_wait_ld();
        const uint32_t m = (uint32_t)(mask >> c);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = (m >> i) & 1u ? 0x7fc00000u : o[i];
        tmem_st32(o_base + c, o);
    }
    tmem_wait_st();
}

// Scales this thread's 64 columns of O by alpha.
__device__ __noinline__ void scale_output(uint32_t taddr, float alpha) {
    const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
    for (int c = 0; c < kCols; c += 32) {
        uint32_t o[32];
        tmem_ld32(taddr + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float r0, r1;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), a2), r0, r1);
            o[i] = __float_as_uint(r0);
            o[i + 1] = __float_as_uint(r1);
        }
        tmem_st32(taddr + c, o);
    }
    tmem_wait_st();
}

// Splits rows [first, 128), every `step`-th, of a Q tile (bf16, two 128-byte pieces
// per row) in place into q1 and q2 (E4M3, one piece each), and leaves the rows'
// scales 2^e.  Eight neighbouring lanes share a row: lane c owns elements 16 c ..
// 16 c + 15, two chunks of the bf16 row and one of each row of codes.
__device__ __forceinline__ void split_query(uint8_t *tile, float *scales, int first, int step, int c) {
#pragma unroll 1
    for (int r = first; r < kRows; r += step) {
        const int sw = r & 7;
        uint8_t *row = tile + r * 128;
        const uint8_t *src = row + (c >> 2) * kHalf;
        const uint4 w0 = *reinterpret_cast<const uint4 *>(src + (((2 * (c & 3)) ^ sw) << 4));
        const uint4 w1 = *reinterpret_cast<const uint4 *>(src + (((2 * (c & 3) + 1) ^ sw) << 4));
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        uint32_t amax = 0;                           // as bits: magnitudes compare like integers
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // 2^e with amax < 2^(e + 8): every code is below 256; an infinite or NaN
        // element makes the row NaN
        const int e = max((int)(amax >> 23) - 127 - 7, -100);
        const float up = __uint_as_float((uint32_t)(127 - e) << 23);      // 2^-e
        const bool bad = amax >= 0x7f800000u;
        uint32_t c1[4], c2[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the scaled pair is exact in f16 (down to 2^-24), its first codes'
            // difference too
            const uint32_t x = pack_f16x2(bf16lo(w[i]) * up, bf16hi(w[i]) * up);
            const uint32_t p1 = f16x2_to_e4m3x2(x);
            const uint32_t p2 = f16x2_to_e4m3x2(sub_f16x2(x, e4m3x2_to_f16x2(p1)));
            if (i & 1) {
                c1[i >> 1] |= p1 << 16;
                c2[i >> 1] |= p2 << 16;
            } else {
                c1[i >> 1] = p1;
                c2[i >> 1] = p2;
            }
        }
        if (bad) c1[0] = c1[1] = c1[2] = c1[3] = 0x7f7f7f7fu;
        __syncwarp();                                // the rows have been read
        *reinterpret_cast<uint4 *>(row + ((c ^ sw) << 4)) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
        *reinterpret_cast<uint4 *>(row + kHalf + ((c ^ sw) << 4)) = make_uint4(c2[0], c2[1], c2[2], c2[3]);
        if (c == 0) scales[r] = 1.f / up;
    }
}

// Four lanes with four rows' chunks q of 16 bytes each, a[4 q ..]: afterwards lane
// p holds chunk p of the four rows, a[4 i ..] that of row i.
__device__ __forceinline__ void quad_transpose(uint32_t (&a)[16], int lane) {
#pragma unroll
    for (int s = 1; s <= 2; s <<= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q & s) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t send = up ? a[4 * q + k] : a[4 * (q + s) + k];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, send, s);
                if (up) a[4 * q + k] = got;
                else a[4 * (q + s) + k] = got;
            }
        }
    }
}

// The two warps of a softmax group that hold the same 32 rows meet here.
__device__ __forceinline__ void pair_sync(int x, int quarter) {
    asm volatile("bar.sync %0, 64;" ::"r"(5 + 4 * x + quarter) : "memory");
}
// The same, with the OR of `v` over their threads.
__device__ __forceinline__ bool pair_any(int x, int quarter, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(5 + 4 * x + quarter)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void group_sync(int x) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + x), "n"(kGroup) : "memory");
}

// AND of `v` over the threads of softmax group x.
__device__ __forceinline__ bool group_all(int x, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(3 + x), "n"(kGroup)
        : "memory");
    return r != 0;
}

// Two 128-row Q tiles of one sequence and KV head against a range of positions.
struct Item {
    int b, kvh;
    int q0, T, C;       // first query row of the chunk, its tokens, context before it
    int t0;             // first token of tile A
    int kv_lo, kv_hi, blk_lo, blk_hi, n_tiles;
    int part, parts;
    bool has_b;
};

// The positions, blocks and steps of the 256-row tile that begins at token t0 of
// d's chunk (d.C, d.T), and the parts they are cut into.
__device__ __forceinline__ void tile_range(const PrefillArgs &a, Item &d) {
    const int tok_per_tile = kRows / a.group;
    d.kv_hi = d.C + min(d.T, d.t0 + kQT * tok_per_tile);
    d.kv_lo = a.window > 0 ? max(0, d.C + d.t0 + 1 - a.window) : 0;
    d.blk_lo = d.kv_lo / kBlockSize;
    d.blk_hi = (d.kv_hi + kBlockSize - 1) / kBlockSize;
    d.n_tiles = (d.blk_hi - d.blk_lo + 7) / 8;
    d.parts = max(1, min(a.splits, d.n_tiles / kPartSteps));
}

// The steps that all of the item's rows, from position C + t0 to kv_hi - 1, attend to whole.
__device__ __forceinline__ Whole whole_steps(const PrefillArgs &a, const Item &d) {
    return Whole{a.window > 0 ? d.kv_hi - a.window : 0, d.C + d.t0 + 1 - kKv};
}

template <bool kCut>
__device__ __forceinline__ bool describe_item(const PrefillArgs &a, int item, bool by_length, bool say, const int *perm,
                                              Item &d) {
    const int tok_per_tile = kRows / a.group;
    const int lmax = a.max_blocks * kBlockSize;
    d.part = kCut ? item % a.splits : 0;
    if constexpr (kCut) item /= a.splits;
    // by_length: every group's longest tile, then every group's next one, ...;
    // else the tiles of a (sequence, KV head) together, longest first
    const int groups = a.num_seqs * a.num_kv_heads;
    const int x = by_length ? item / groups : item % a.n_mt;
    const int rest = by_length ? item - x * groups : item / a.n_mt;
    d.kvh = rest % a.num_kv_heads;
    d.b = rest / a.num_kv_heads;
    if (perm != nullptr) d.b = perm[d.b];
    d.q0 = a.query_start[d.b];
    const int end = a.query_start[d.b + 1];
    const int L = a.context_lens[d.b];
    const bool first = say && x == 0 && d.kvh == 0 && d.part == 0;
    if (d.q0 < 0 || end < d.q0 || end > a.num_query_tokens || end - d.q0 > L || L > lmax) {
        if (first) report(a.status, PA_DEV_BAD_CONTEXT_LEN);
        return false;
    }
    d.T = end - d.q0;
    if (first && d.T > a.max_query_len) report(a.status, PA_DEV_BAD_QUERY_LEN);
    d.t0 = (a.n_mt - 1 - x) * kQT * tok_per_tile;
    if (d.t0 >= d.T) return false;
    d.C = L - d.T;
    tile_range(a, d);
    if constexpr (kCut) {
        if (d.part >= d.parts) return false;
        const int lo = d.part * d.n_tiles / d.parts, hi = (d.part + 1) * d.n_tiles / d.parts;
        d.blk_hi = min(d.blk_hi, d.blk_lo + 8 * hi);
        d.blk_lo += 8 * lo;
        d.n_tiles = hi - lo;
    }
    d.has_b = d.t0 + tok_per_tile < d.T;
    return true;
}

// kCut: items are cut along the context and leave partial outputs.
template <bool kCut>
__global__ void __launch_bounds__(kThreads, 1)
    pa_prefill_block8_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                             const __grid_constant__ CUtensorMap vmap, const PrefillArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int tok_per_tile = kRows / a.group;

    extern __shared__ __align__(1024) uint8_t base[];
    if (smem_u32(base) & 1023u) {
        if (threadIdx.x == 0) report(a.status, PA_DEV_SMEM_ALIGN);
        return;
    }
    uint8_t *sQ = base + kOffQ, *sK = base + kOffK, *sV = base + kOffV, *sCode = base + kOffCode;
    float4 *s_scale = reinterpret_cast<float4 *>(base + kOffScale);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(base + kOffMisc);
    volatile int *fail = reinterpret_cast<volatile int *>(base + kOffMisc + 4);
    volatile int *s_order = reinterpret_cast<volatile int *>(base + kOffMisc + 8);
    volatile int *s_item = reinterpret_cast<volatile int *>(base + kOffMisc + 16);   // [2]
    volatile int *s_nan = reinterpret_cast<volatile int *>(base + kOffMisc + 32);    // [4]
    volatile int *s_taken = reinterpret_cast<volatile int *>(base + kOffMisc + 48);  // [4]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            int n = 1;
            if ((i >= kCodeEmpty && i < kCodeEmpty + kCodeStages) || (i >= kVConv && i < kVConv + kVStages))
                n = kWidenThreads;
            if ((i >= kQSplit && i < kQSplit + kQT) || (i >= kPFull && i < kPFull + kQT) || (i >= kOFree && i < kOFree + kQT)) n = kGroup;
            if (i >= kItemEmpty && i < kItemEmpty + 2) n = 1 + kQT * kGroup + kWidenThreads;
            mbar_init(&bars[i], n);
        }
        *fail = 0;
        for (int i = 0; i < 4; ++i) s_nan[i] = 0, s_taken[i] = -1;
        fence_mbar_init();
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    // Item order, where CTAs take items in turn: longest first across all groups
    // when the chunks bring more tokens than the contexts held before (causal tiles
    // from short to long); else a group's tiles together, their K/V shared in L2.
    if (warp == 2 && a.work_counter != nullptr) {
        long long cached = 0, fresh = 0;
        for (int i = lane; i < a.num_seqs; i += 32) {
            const int T = a.query_start[i + 1] - a.query_start[i];
            const int L = a.context_lens[i];
            fresh += T > 0 ? T : 0;
            cached += L - T > 0 ? L - T : 0;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            cached += __shfl_xor_sync(0xffffffffu, cached, o);
            fresh += __shfl_xor_sync(0xffffffffu, fresh, o);
        }
        if (lane == 0) *s_order = cached < fresh ? 1 : 0;
        if (a.num_seqs <= kPermMax) {
            // sequences longest context first (ties by index), so that the call ends
            // on short ones
            static_assert(kPermMax == 64, "two sequences per lane");
            int *perm = reinterpret_cast<int *>(base + kOffPerm);
            const int l0 = lane < a.num_seqs ? a.context_lens[lane] : INT_MIN;
            const int l1 = lane + 32 < a.num_seqs ? a.context_lens[lane + 32] : INT_MIN;
            int r0 = 0, r1 = 0;
            for (int j = 0; j < a.num_seqs; ++j) {
                const int lj = __shfl_sync(0xffffffffu, j < 32 ? l0 : l1, j & 31);
                r0 += (lj > l0) | ((lj == l0) & (j < lane));
                r1 += (lj > l1) | ((lj == l1) & (j < lane + 32));
            }
            if (lane < a.num_seqs) perm[r0] = lane;
            if (lane + 32 < a.num_seqs) perm[r1] = lane + 32;
        }
    }
    if (warp == 1) tmem_alloc(tslot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const bool by_length = a.work_counter != nullptr && *s_order != 0;
    const int *perm = a.work_counter != nullptr && a.num_seqs <= kPermMax ? reinterpret_cast<const int *>(base + kOffPerm) : nullptr;

    // the next item of a consumer role, -1 at the end (or after a wait gave up)
    auto next_item = [&](int it) -> int {
        const int slot = it & 1;
        const int item = wait_or_fail(&bars[kItemFull + slot], (it >> 1) & 1, fail, a.status) ? s_item[slot] : -1;
        mbar_arrive(&bars[kItemEmpty + slot]);
        return item;
    };

    if (warp == 0) {
        // ---------------- TMA producer (and item fetch) ----------------
        if (lane == 0) {
            int q_issued = -1;
            uint32_t gstep = 0, k_issued = 0, v_issued = 0;
            bool ok = true, taken = false;
            for (int it = 0;; ++it) {
                int item = -1;
                Item d;
                while (ok) {
                    int t = a.num_items;
                    if (a.work_counter != nullptr) t = (int)atomicAdd(a.work_counter, 1u);
                    else if (it == 0 && !taken) t = blockIdx.x;
                    taken = true;
                    if (t >= a.num_items) break;
                    if (describe_item<kCut>(a, t, by_length, true, perm, d)) {
                        item = t;
                        break;
                    }
                }
                const int slot = it & 1;
                if (item >= 0) s_taken[it & 3] = item;
                if (it >= 2 && !wait_or_fail(&bars[kItemEmpty + slot], ((it >> 1) - 1) & 1, fail, a.status)) item = -1;
                s_item[slot] = item;
                mbar_arrive(&bars[kItemFull + slot]);
                if (item < 0) break;
                // Q once the last QK^T of the item before has run
                if (it >= 1 && !wait_or_fail(&bars[kQFree], (it - 1) & 1, fail, a.status)) {
                    ok = false;
                    continue;
                }
                const int nq = d.has_b ? kQT : 1;
                mbar_arrive_expect_tx(&bars[kQFull], nq * kTile);
                for (int x = 0; x < nq; ++x) {
                    const int row0 = d.q0 + d.t0 + x * tok_per_tile;
                    tma_load_4d(sQ + x * kTile, &qmap, 0, 0, d.kvh, row0, &bars[kQFull]);
                    tma_load_4d(sQ + x * kTile + kHalf, &qmap, 64, 0, d.kvh, row0, &bars[kQFull]);
                }
                q_issued = it;
                const int32_t *trow = a.block_tables + (int64_t)d.b * a.max_blocks;
                for (int j = 0; ok && j < d.n_tiles; ++j) {
                    int rows[8];
                    const int blk0 = d.blk_lo + 8 * j, nb = min(8, d.blk_hi - blk0);
                    for (int i = 0; i < nb; ++i) {
                        int phys = trow[blk0 + i];
                        if ((unsigned)phys >= (unsigned)a.num_blocks) {
                            report(a.status, PA_DEV_BAD_BLOCK_ID);
                            phys = 0;
                        }
                        rows[i] = (phys * a.num_kv_heads + d.kvh) * kBlockSize;
                    }
                    const uint32_t gs = gstep + j;
                    if (gs >= kKStages &&
                        !wait_or_fail(&bars[kKEmpty + gs % kKStages], (gs / kKStages - 1) & 1, fail, a.status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bars[kKFull + gs % kKStages], nb * kBlockSize * kD);
                    for (int i = 0; i < nb; ++i)
                        tma_load_2d(sK + (gs % kKStages) * kCodeTile + i * kBlockSize * kD, &kmap, 0, rows[i],
                                    &bars[kKFull + gs % kKStages]);
                    k_issued = gs + 1;
                    if (gs >= kCodeStages &&
                        !wait_or_fail(&bars[kCodeEmpty + gs % kCodeStages], (gs / kCodeStages - 1) & 1, fail, a.status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bars[kCodeFull + gs % kCodeStages], nb * kBlockSize * kD);
                    for (int i = 0; i < nb; ++i)
                        tma_load_2d(sCode + (gs % kCodeStages) * kCodeTile + i * kBlockSize * kD, &vmap, 0, rows[i],
                                    &bars[kCodeFull + gs % kCodeStages]);
                    v_issued = gs + 1;
                }
                gstep += d.n_tiles;
            }
            // no copy of ours may still be landing when the CTA leaves
            if (q_issued >= 0) (void)mbar_wait_bounded(&bars[kQFull], q_issued & 1);
            for (uint32_t j = k_issued > kKStages ? k_issued - kKStages : 0; j < k_issued; ++j)
                (void)mbar_wait_bounded(&bars[kKFull + j % kKStages], (j / kKStages) & 1);
            for (uint32_t j = v_issued > kCodeStages ? v_issued - kCodeStages : 0; j < v_issued; ++j)
                (void)mbar_wait_bounded(&bars[kCodeFull + j % kCodeStages], (j / kCodeStages) & 1);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        // The whole warp runs the loop and one elected lane issues: descriptors then
        // stay in uniform registers.  Issued from a one-lane branch, a batch of eight
        // products took about 600 cycles and the issuing lane bounded the step.
        constexpr uint32_t idS = idesc_e4m3_f32(kRows, kKv);
        constexpr uint32_t idPV = idesc_f16_f32(kRows, kD, true);
        const uint64_t q_desc = sw128_desc(smem_u32(sQ), 16, 1024), k_desc = sw128_desc(smem_u32(sK), 16, 1024),
                       v_desc = sw128_desc(smem_u32(sV), kHalf, 1024);
        uint32_t gstep = 0;
        uint32_t pcount[kQT] = {0, 0}, b_items = 0;
        bool ok = true;
        // S_x = Q_x K^T: q1, then q2, in steps of 32 codes (descriptors count 16 bytes)
        auto issue_s = [&](int x, uint32_t gs) {
            tc_fence_after();
            const uint64_t qd = q_desc + (uint64_t)(x * (kTile / 16)), kd = k_desc + (uint64_t)((gs % kKStages) * (kCodeTile / 16));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma_f8(tmem + col_s(x), qd + (uint64_t)((k >> 2) * (kHalf / 16) + (k & 3) * 2), kd + (uint64_t)((k & 3) * 2),
                            idS, k > 0 ? 1u : 0u);
                umma_commit(&bars[kSFull + x]);
            }
            __syncwarp();
        };
        // O_x += P_x V: P of tokens [16 k, 16 k + 16) is f16 pairs from column
        // 32 (k / 2) + 8 (k % 2) of the S buffer
        auto issue_pv = [&](int x, uint32_t gs, int j, int it) -> bool {
            if (!warp_wait(&bars[kPFull + x], pcount[x] & 1, fail, a.status)) return false;
            ++pcount[x];
            // the first P.V of an item overwrites O: the item before must have read it out
            if (j == 0 && it >= 1 && !warp_wait(&bars[kOFree + x], (it - 1) & 1, fail, a.status)) return false;
            tc_fence_after();
            const uint64_t vd = v_desc + (uint64_t)((gs % kVStages) * (kTile / 16));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma_bf16_tmem_a(tmem + col_o(x), tmem + col_s(x) + 32 * (k >> 1) + 8 * (k & 1),
                                     vd + (uint64_t)(k * (2048 / 16)), idPV, (j > 0 || k > 0) ? 1u : 0u);
                umma_commit(&bars[kPvDone + x]);
            }
            __syncwarp();
            return true;
        };
        auto commit = [&](int bar) {
            if (elect_one()) umma_commit(&bars[bar]);
            __syncwarp();
        };
        for (int it = 0; ok; ++it) {
            const int slot = it & 1;
            const int item = warp_wait(&bars[kItemFull + slot], (it >> 1) & 1, fail, a.status) ? s_item[slot] : -1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kItemEmpty + slot]);
            if (item < 0) break;
            Item d;
            describe_item<kCut>(a, item, by_length, false, perm, d);
            const int n = d.n_tiles;
            if (!warp_wait(&bars[kQSplit], it & 1, fail, a.status) ||
                !warp_wait(&bars[kKFull + gstep % kKStages], (gstep / kKStages) & 1, fail, a.status))
                break;
            issue_s(0, gstep);
            if (d.has_b) {
                if (!warp_wait(&bars[kQSplit + 1], b_items++ & 1, fail, a.status)) break;
                issue_s(1, gstep);
            }
            commit(kKEmpty + gstep % kKStages);
            if (n == 1) commit(kQFree);
            for (int j = 0; j < n; ++j) {
                const uint32_t gs = gstep + j, gk = gs + 1;
                const bool more = j + 1 < n;
                // what is usually there already first: these waits run beside the
                // products in flight, the one for P does not
                if (!warp_wait(&bars[kVConv + gs % kVStages], (gs / kVStages) & 1, fail, a.status) ||
                    (more && !warp_wait(&bars[kKFull + gk % kKStages], (gk / kKStages) & 1, fail, a.status)) ||
                    !issue_pv(0, gs, j, it)) {
                    ok = false;
                    break;
                }
                if (more) issue_s(0, gk);
                if (d.has_b && !issue_pv(1, gs, j, it)) {
                    ok = false;
                    break;
                }
                commit(kVEmpty + gs % kVStages);
                if (more) {
                    if (d.has_b) issue_s(1, gk);
                    commit(kKEmpty + gk % kKStages);
                    if (j + 2 == n) commit(kQFree);
                }
            }
            // Group 1 keeps no other phase of an item without a tile B in step, and waits for
            // this one by parity: it completes for item `it` only when the group has left
            // item it - 1, or two short items could pass while the group is still at the end
            // of a longer one, and its wait would then match a phase that is still running.
            // (Group 0 is waited for before the item's first P V.)
            if (it >= 1 && !warp_wait(&bars[kOFree + 1], (it - 1) & 1, fail, a.status)) ok = false;
            commit(kDrain);                          // every MMA of the item has completed once it flips
            gstep += n;
        }
        // after a wait that gave up products may still be running: the CTA's memory is
        // theirs until they are done
        commit(kEnd);
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[kEnd], 0)) && lane == 0) report(a.status, PA_DEV_TIMEOUT);
    } else if (warp >= kWidenWarp0) {
        // ---------------- widening ----------------
        // 16 codes of a row become two 16-byte chunks of f16 in one of the tile's
        // 64-column halves; threads of the two halves write their chunks in opposite
        // order, so that eight threads of a row never meet in a bank.  Eight rows are
        // loaded before the first is written: the loop is bound by latency.
        const int ct = threadIdx.x - kWidenWarp0 * 32;
        const int c16 = ct & 7, half = c16 >> 2, c = 2 * (c16 & 3);
        constexpr int kRowStep = kWidenThreads / 8, kBatch = 8;
        static_assert(kKv % (kRowStep * kBatch) == 0 && kRowStep % 8 == 0, "whole batches, one swizzle phase per thread");
        // A NaN code reaches every row of the tile, as 0 * NaN those that do not attend
        // to it.  In tiles that some row attends to in part it becomes 0 here, and the
        // item is marked (four marks: this loop runs at most two items ahead of the
        // softmax), so that its rows get their NaNs at the end.  (Looking for NaNs in
        // the loop above, in every tile or in a second copy of it, cost 9 and 7 %.)
        uint32_t gstep = 0;
        bool ok = true;
        for (int it = 0;; ++it) {
            const int item = next_item(it);
            if (item < 0) break;
            Item d;
            describe_item<kCut>(a, item, by_length, false, perm, d);
            // The scales of a step's blocks, one thread per block of the first warp.  The
            // table entry is read two steps ahead and the scales one step, so that no
            // step waits for the chain of loads; the slot written last held the scales of
            // four steps back, whose softmax came before P.V of two steps back, which
            // this loop has waited for.
            const int32_t *trow = a.block_tables + (int64_t)d.b * a.max_blocks;
            float ks = 0.f, vs = 1.f;
            int phys = -1;
            auto table_at = [&](int j) {
                const int blk = d.blk_lo + 8 * j + ct;
                phys = ct < 8 && blk < d.blk_hi ? trow[blk] : -1;
            };
            auto fetch_scales = [&](int j) {
                ks = 0.f;
                vs = 1.f;
                if (ct < 8 && d.blk_lo + 8 * j + ct < d.blk_hi) {
                    const int64_t at = (int64_t)((unsigned)phys < (unsigned)a.num_blocks ? phys : 0) * a.num_kv_heads + d.kvh;
                    ks = a.k_scales[at];
                    vs = a.v_scales[at];
                }
            };
            auto stage_scales = [&](uint32_t gs) {
                if (ct >= 32) return;
                if (ct < 8) {
                    const float sv = value_scale(vs, a.status);
                    s_scale[(gs % kScaleSlots) * 8 + ct] = make_float4(ks * a.scale_log2, log2_scale(sv), 1.f / sv, 0.f);
                }
                __syncwarp();
                if (ct == 0) mbar_arrive(&bars[kScaleFull + gs % kScaleSlots]);
            };
            table_at(0);
            fetch_scales(0);
            table_at(1);
            if (ok) stage_scales(gstep);
            fetch_scales(1);
            table_at(2);
            for (int j = 0; ok && j < d.n_tiles; ++j) {
                const uint32_t gs = gstep + j;
                if (!wait_or_fail(&bars[kCodeFull + gs % kCodeStages], (gs / kCodeStages) & 1, fail, a.status) ||
                    (gs >= kVStages &&
                     !wait_or_fail(&bars[kVEmpty + gs % kVStages], (gs / kVStages - 1) & 1u, fail, a.status))) {
                    ok = false;
                    break;
                }
                const uint4 *src = reinterpret_cast<const uint4 *>(sCode + (gs % kCodeStages) * kCodeTile) + ct;
                uint8_t *dst = sV + (gs % kVStages) * kTile + half * kHalf + (ct >> 3) * 128;
                const int sw = (ct >> 3) & 7, at0 = ((c + half) ^ sw) << 4, at1 = ((c + 1 - half) ^ sw) << 4;
#pragma unroll
                for (int b = 0; b < kKv / kRowStep; b += kBatch) {
                    uint4 w[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) w[i] = src[(b + i) * kWidenThreads];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        uint4 x, y;
                        e4m3x4_to_f16x2x2(w[i].x, x.x, x.y);
                        e4m3x4_to_f16x2x2(w[i].y, x.z, x.w);
                        e4m3x4_to_f16x2x2(w[i].z, y.x, y.y);
                        e4m3x4_to_f16x2x2(w[i].w, y.z, y.w);
                        *reinterpret_cast<uint4 *>(dst + (b + i) * kRowStep * 128 + at0) = half ? y : x;
                        *reinterpret_cast<uint4 *>(dst + (b + i) * kRowStep * 128 + at1) = half ? x : y;
                    }
                }
                mbar_arrive(&bars[kCodeEmpty + gs % kCodeStages]);
                // positions outside the item's range may hold anything, NaN among it
                const int k0 = (d.blk_lo + 8 * j) * kBlockSize;
                if (k0 < d.kv_lo || k0 + kKv > d.kv_hi) {
                    for (int r = ct >> 3; r < kKv; r += kRowStep)
                        if (k0 + r < d.kv_lo || k0 + r >= d.kv_hi) {
                            uint8_t *row = dst + (r - (ct >> 3)) * 128;
                            *reinterpret_cast<uint4 *>(row + at0) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(row + at1) = make_uint4(0, 0, 0, 0);
                        }
                }
                if (!whole_steps(a, d).has(k0) && clear_nan<kRowStep>(dst, at0, at1)) s_nan[it & 3] = it + 1;
                fence_proxy_async_smem();
                mbar_arrive(&bars[kVConv + gs % kVStages]);
                if (j + 1 < d.n_tiles) {
                    stage_scales(gs + 1);
                    fetch_scales(j + 2);
                    table_at(j + 3);
                }
            }
            gstep += d.n_tiles;
        }
    } else {
        // ---------------- softmax groups ----------------
        const int x = (warp - 2) / (kGroup / 32);
        const int gw = (warp - 2) % (kGroup / 32);
        const int quarter = warp & 3;
        const int part = gw >> 2;                     // columns [64 part, + 64)
        const int r = quarter * 32 + lane;            // tile row = TMEM lane
        const int tr = r / a.group;
        const uint32_t lane_off = ((uint32_t)(quarter * 32) << 16) + part * kCols;
        const uint32_t s_base = tmem + col_s(x) + lane_off;
        const uint32_t o_base = tmem + col_o(x) + lane_off;
        float *red = reinterpret_cast<float *>(base + kOffRed) + x * 2 * 2 * kRows;
        uint32_t sc = 0;      // S / P / P.V phases of this group (global)
        uint32_t ex = 0;      // exchanges through `red` (their slot alternates)
        uint32_t gstep = 0;
        bool ok = true;
        for (int it = 0;; ++it) {
            const int slot = it & 1;
            const bool got_item = warp_wait(&bars[kItemFull + slot], (it >> 1) & 1, fail, a.status);
            const int item = got_item ? s_item[slot] : -1;
            mbar_arrive(&bars[kItemEmpty + slot]);
            // all threads of the group decide alike, so that they reach its named barriers equally often
            if (!group_all(x, item >= 0 && ok && !*fail)) break;
            Item d;
            describe_item<kCut>(a, item, by_length, false, perm, d);
            if (x == 0 || d.has_b) {
                const int tx0 = d.t0 + x * tok_per_tile;
                const int ntok = min(tok_per_tile, d.T - tx0);
                const bool real = tr < ntok;
                // this row attends to positions [wlo, qpos]; a 32-column chunk needs no
                // mask when it lies inside every row's range of the tile
                const int qpos = d.C + tx0 + min(tr, ntok - 1);
                const int qpos_lo = d.C + tx0, qpos_hi = d.C + tx0 + ntok - 1;
                const int wlo = a.window > 0 ? max(0, qpos + 1 - a.window) : 0;
                // The row's reference (log2 units): an integer, or -inf before the row
                // has seen a position; O and l are relative to it.
                float m_used = -INFINITY, l = 0.f;
                // the group splits its Q tile
                float *q_scale = reinterpret_cast<float *>(base + kOffQScale) + x * kRows;
                ok = warp_wait(&bars[kQFull], it & 1, fail, a.status) && ok;
                if (ok) {
                    const int t = threadIdx.x - 64 - x * kGroup;
                    split_query(sQ + x * kTile, q_scale, t >> 3, kGroup / 8, t & 7);
                    fence_proxy_async_smem();
                    mbar_arrive(&bars[kQSplit + x]);
                }
                group_sync(x);
                const float qs = q_scale[r];
                for (int j = 0; j < d.n_tiles; ++j) {
                    const uint32_t gs = gstep + j;
                    const bool got = ok && warp_wait(&bars[kSFull + x], sc & 1, fail, a.status) &&
                                     warp_wait(&bars[kScaleFull + gs % kScaleSlots], (gs / kScaleSlots) & 1, fail, a.status);
                    const int k0 = (d.blk_lo + 8 * j) * kBlockSize + part * kCols;
                    const float4 *scales = s_scale + (gs % kScaleSlots) * 8 + part * (kCols / kBlockSize);
                    // One pass over S: a chunk's weights 2^(s ck + lv - ref) replace it in
                    // f16, unless they sum to more than 2^15 or some row sees only part
                    // of the chunk: those take the general form, where the reference may
                    // rise.  Each chunk keeps the reference it was written with.
                    float mref = m_used;
                    float cref0 = m_used, cref1 = m_used, csum0 = 0.f, csum1 = 0.f;
                    if (got) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < kCols; c += 32) {
                            const int kc = k0 + c;
                            const float4 *e = scales + (c >> 4);
                            bool general = kc + 31 > qpos_lo || (a.window > 0 && kc < qpos_hi + 1 - a.window);
                            float psum;
                            if (!general) {
                                uint32_t v[32], pp[16];
                                tmem_ld32(s_base + c, v);
                                const float4 e0 = e[0], e1 = e[1];
                                tmem_wait_ld();
                                float sum[2];
#pragma unroll
                                for (int blk = 0; blk < 2; ++blk) {
                                    const float ck = (blk ? e1.x : e0.x) * qs, off = (blk ? e1.y : e0.y) - mref;
                                    const uint64_t k2 = f2_pack(ck, ck), nm2 = f2_pack(off, off);
                                    uint64_t ps2 = f2_pack(0.f, 0.f);
#pragma unroll
                                    for (int i = 16 * blk; i < 16 * blk + 16; i += 2) {
                                        float x0, x1;
                                        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), k2, nm2), x0, x1);
                                        const float p0 = ex2_fast(x0), p1 = ex2_fast(x1);
                                        ps2 = f2_add(ps2, f2_pack(p0, p1));
                                        pp[i >> 1] = pack_f16x2(p0, p1);
                                    }
                                    float lo, hi;
                                    f2_unpack(ps2, lo, hi);
                                    sum[blk] = lo + hi;
                                }
                                psum = fmaf(sum[0], e0.z, sum[1] * e1.z);
                                general = __any_sync(0xffffffffu, !(sum[0] + sum[1] <= kChunkSumMax));
                                if (!general) tmem_st16(s_base + c, pp);
                            }
                            if (general) {           // the whole warp; S is still in place
                                const float2 r2 = chunk_weights_general(s_base + c, e, qs, mref, kc, qpos, wlo);
                                psum = r2.x;
                                mref = r2.y;
                            }
                            if (c == 0) {
                                cref0 = mref;
                                csum0 = psum;
                            } else {
                                cref1 = mref;
                                csum1 = psum;
                            }
                        }
                        tmem_wait_st();
                    }
                    const uint32_t my_sc = sc++;
                    float psum = csum0 + csum1;
                    // A reference that rose anywhere in the 32 rows (rare after the first
                    // steps): the two threads of each row agree on the larger one.
                    if (pair_any(x, quarter, mref != m_used)) {
                        const int rp = ex & 1;
                        ++ex;
                        red[(rp * 2 + part) * kRows + r] = mref;
                        pair_sync(x, quarter);
                        const float rref = fmaxf(mref, red[(rp * 2 + (part ^ 1)) * kRows + r]);
                        if (got) {
                            // chunks written against a smaller reference are scaled by
                            // the exact power of two between them
                            const float f0 = pow2_diff(cref0, rref), f1 = pow2_diff(cref1, rref);
                            if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) scale_chunk_weights(s_base, f0, f1);
                            psum = csum0 * f0 + csum1 * f1;
                            // O and l follow, once every P.V of this tile issued so far
                            // has landed
                            const float alpha = rref > m_used ? pow2_diff(m_used, rref) : 1.f;
                            if (j >= 1) {
                                if (!warp_wait(&bars[kPvDone + x], (my_sc - 1) & 1, fail, a.status)) ok = false;
                                tc_fence_after();
                                if (ok) scale_output(o_base, alpha);
                            }
                            l *= alpha;
                            m_used = rref > m_used ? rref : m_used;
                        }
                    }
                    if (!got || !ok) {
                        ok = false;
                        continue;
                    }
                    l += psum;
                    tc_fence_before();
                    mbar_arrive(&bars[kPFull + x]);
                }
                // the row sum is the two parts' sums
                const int sx = ex & 1;
                ++ex;
                red[(sx * 2 + part) * kRows + r] = l;
                pair_sync(x, quarter);
                const float l_row = l + red[(sx * 2 + (part ^ 1)) * kRows + r];
                const bool drained = warp_wait(&bars[kDrain], it & 1, fail, a.status);
                if (drained && s_nan[it & 3] == it + 1) {
                    tc_fence_after();
                    poison_output(a, o_base, d.b, d.kvh, part * kCols, d.blk_lo, d.n_tiles, d.kv_hi, whole_steps(a, d), qpos);
                }
                if (kCut && __all_sync(0xffffffffu, ok) && drained && d.parts > 1) {
                    tc_fence_after();
                    const int64_t prow = ((int64_t)(d.q0 + tx0 + tr) * a.num_q_heads + d.kvh * a.group + (r % a.group)) *
                                             a.splits + d.part;
                    float4 *po = reinterpret_cast<float4 *>(a.part_o + prow * kD + part * kCols);
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(o_base + c, o);
                        tmem_wait_ld();
                        if (real) {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                po[c / 4 + q] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                                            __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
                        }
                    }
                    if (real && part == 0) a.part_ml[prow] = make_float2(m_used, l_row);
                } else if (__all_sync(0xffffffffu, ok) && drained) {
                    tc_fence_after();
                    const float inv = l_row == 0.f ? 0.f : 1.f / l_row;
                    // four lanes exchange their rows' chunks, so that they write 64
                    // bytes of one row together: a lane's own row would be written in
                    // half sectors, 32 rows at a time
                    const int64_t out_row =
                        real ? (int64_t)(d.q0 + tx0 + tr) * a.num_q_heads + d.kvh * a.group + (r % a.group) : -1;
                    int64_t row[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) row[i] = __shfl_sync(0xffffffffu, out_row, (lane & ~3) + i);
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + part * kCols + 8 * (lane & 3);
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 32) {
                        uint32_t o[32], w[16];
                        tmem_ld32(o_base + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            w[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
                        quad_transpose(w, lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (row[i] >= 0)
                                *reinterpret_cast<uint4 *>(out + row[i] * kD + c) =
                                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    }
                }
                if (!drained) ok = false;
            } else {
                // tile B has no rows in this item: keep the drain phase in step
                if (!warp_wait(&bars[kDrain], it & 1, fail, a.status)) ok = false;
            }
            tc_fence_before();
            mbar_arrive(&bars[kOFree + x]);          // O has been read out
            gstep += d.n_tiles;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    // After a wait that gave up, the parts that this CTA was at (it has four items at most in
    // hand) become NaN: what an earlier call left in the workspace must not pass for an output.
    if (kCut && *fail) {
        for (int k = 0; k < 4; ++k) {
            Item d;
            if (s_taken[k] < 0 || !describe_item<kCut>(a, s_taken[k], by_length, false, perm, d)) continue;
            const int rows = min(kQT * tok_per_tile, d.T - d.t0) * a.group;
            for (int i = threadIdx.x; i < rows; i += kThreads) {
                const int64_t row = (int64_t)(d.q0 + d.t0 + i / a.group) * a.num_q_heads + d.kvh * a.group + i % a.group;
                a.part_ml[row * a.splits + d.part] = make_float2(-INFINITY, __int_as_float(0x7fffffff));
            }
        }
    }
}

// Merges the parts of the rows whose tile was cut, one warp a row.
__global__ void __launch_bounds__(128) pa_merge_prefill8_kernel(const PrefillArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)a.num_query_tokens * a.num_q_heads) return;
    const int token = (int)(row / a.num_q_heads);
    // The sequence that the token belongs to, among those that were computed: entries of
    // query_start that fall or leave the rows say nothing about the others, so all are
    // looked at (a cut call has no more sequences than the GPU has SMs).
    Item d;
    int end = 0, L = 0, found = -1;
    for (int b = lane; b - lane < a.num_seqs && found < 0; b += 32) {
        bool mine = false;
        if (b < a.num_seqs) {
            d.q0 = a.query_start[b];
            end = a.query_start[b + 1];
            L = a.context_lens[b];
            mine = d.q0 >= 0 && token >= d.q0 && token < end && end <= a.num_query_tokens && end - d.q0 <= L &&
                   L <= a.max_blocks * kBlockSize;
        }
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (who != 0) found = __ffs(who) - 1;
    }
    if (found < 0) return;
    d.q0 = __shfl_sync(0xffffffffu, d.q0, found);
    end = __shfl_sync(0xffffffffu, end, found);
    L = __shfl_sync(0xffffffffu, L, found);
    if (token - d.q0 >= a.n_mt * (kQT * kRows / a.group)) return;
    d.T = end - d.q0;
    d.C = L - d.T;
    const int tokens = kQT * kRows / a.group;
    d.t0 = (token - d.q0) / tokens * tokens;
    tile_range(a, d);
    if (d.parts <= 1) return;
    const float2 *ml = a.part_ml + row * a.splits;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + row * a.splits * kD);
    float M = -INFINITY;
    for (int p = 0; p < d.parts; ++p) M = fmaxf(M, ml[p].x);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < d.parts; p0 += 8) {
        float4 v[8];
        float2 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = p0 + i < d.parts;
            v[i] = in ? po[(int64_t)(p0 + i) * 32 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
            x[i] = in ? ml[p0 + i] : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = pow2_diff(x[i].x, M);
            sum = fmaf(f, x[i].y, sum);
            acc.x = fmaf(f, v[i].x, acc.x);
            acc.y = fmaf(f, v[i].y, acc.y);
            acc.z = fmaf(f, v[i].z, acc.z);
            acc.w = fmaf(f, v[i].w, acc.w);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row * kD + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// The query as [rows][KV head][head of the group][head_dim]: a box of 128 / group
// rows x group heads x 64 elements is one half of a 128-row tile.
bool encode_query_map(CUtensorMap *map, const void *query, int rows, int num_q_heads, int num_kv_heads) {
    static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (enc == nullptr) return false;
    bind_context();
    const int group = num_q_heads / num_kv_heads;
    cuuint64_t dims[4] = {kD, (cuuint64_t)group, (cuuint64_t)num_kv_heads, (cuuint64_t)rows};
    cuuint64_t strides[3] = {kD * 2, (cuuint64_t)group * kD * 2, (cuuint64_t)num_q_heads * kD * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)group, 1, (cuuint32_t)(kRows / group)};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(query), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pa

using namespace pa;

namespace {

bool group_ok(int group) { return group == 1 || group == 2 || group == 4 || group == 8 || group == 16; }

// Items of a call, and the parts they are cut into at most.  With no more items than
// SMs it is the number with the least estimated time on full-length contexts, in
// steps: an item costs some five beside its own (its CTA's start and end), the merge
// kernel three and the partial outputs their traffic (a step is about 1.7 us).  10
// chunks of up to 9 tokens on up to 5712 with 8 heads, 80 items: 64 us in 3 parts, 83
// whole.  More items than SMs are left whole: they differ in length, and tickets even
// that out (272 items of 2 chunks of up to 526 tokens: 157 us, 183 in 2 parts; 228 of
// two of up to 1817: 91 / 118).
struct Cut {
    int64_t tiles, items;
    int splits;
};
Cut cut_of(int num_seqs, int num_q_heads, int num_kv_heads, int max_blocks, int window, int num_query_tokens,
           int max_query_len) {
    Cut c;
    const int group = num_q_heads / num_kv_heads;
    c.tiles = ((int64_t)max_query_len * group + kQT * kRows - 1) / (kQT * kRows);
    c.items = c.tiles * num_kv_heads * num_seqs;
    c.splits = 1;
    int64_t blocks = max_blocks;
    if (window > 0) blocks = std::min<int64_t>(blocks, ((int64_t)window + kQT * kRows / group) / kBlockSize + 2);
    const int64_t steps = (blocks + 7) / 8, n = device_sms();
    if (c.items == 0 || c.items > n) return c;
    const double row_steps = 2. * (kD * sizeof(float) + sizeof(float2)) * num_query_tokens * num_q_heads / 6.0e6 / 1.7;
    double best = 1e300;
    for (int64_t k = 1; k == 1 || (k <= 64 && k <= steps / kPartSteps); ++k) {
        const double cost = (double)((c.items * k + n - 1) / n * (5 + (steps + k - 1) / k)) + (k > 1 ? 3. + k * row_steps : 0.);
        if (cost < best) best = cost, c.splits = (int)k;
    }
    return c;
}
size_t part_rows_bytes(int64_t rows) { return (size_t)rows * kD * sizeof(float); }

}  // namespace

extern "C" size_t pa_prefill_block_fp8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                                       int max_blocks_per_seq, int num_query_tokens,
                                                       int max_query_len, int window) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || head_dim != kD ||
        !group_ok(num_q_heads / num_kv_heads) || max_blocks_per_seq < 0 ||
        max_blocks_per_seq > 0x7fffffff / kBlockSize || num_query_tokens < 0 || max_query_len < 0 || window < 0)
        return (size_t)-1;
    const Cut c = cut_of(num_seqs, num_q_heads, num_kv_heads, max_blocks_per_seq, window, num_query_tokens, max_query_len);
    if (c.splits <= 1) return kWorkspaceBytes;
    const int64_t rows = (int64_t)num_query_tokens * num_q_heads * c.splits;
    return kWorkspaceBytes + part_rows_bytes(rows) + (size_t)rows * sizeof(float2);
}

extern "C" pa_status pa_prefill_block_fp8(void *out, const void *query, const void *key_cache, const void *value_cache,
                                          const float *k_scales, const float *v_scales, const int32_t *block_tables,
                                          const int32_t *context_lens, const int32_t *query_start, int num_seqs,
                                          int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                          int max_blocks_per_seq, int num_blocks, int num_query_tokens,
                                          int max_query_len, float scale, int window, void *workspace,
                                          size_t workspace_bytes, int32_t *device_status, void *stream) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        block_size != kBlockSize || max_blocks_per_seq < 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize ||
        num_blocks <= 0 || num_query_tokens < 0 || max_query_len < 0 || window < 0 || !(scale == scale))
        return PA_ERR_INVALID_ARG;
    const int group = num_q_heads / num_kv_heads;
    if (head_dim != kD || !group_ok(group)) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_query_tokens == 0 || max_query_len == 0) return PA_OK;
    if (!out || !query || !key_cache || !value_cache || !k_scales || !v_scales || !context_lens || !query_start ||
        (!block_tables && max_blocks_per_seq > 0))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales) |
          reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(query_start)) & 3u))
        return PA_ERR_INVALID_ARG;
    const size_t need = pa_prefill_block_fp8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                             max_blocks_per_seq, num_query_tokens, max_query_len, window);
    if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)) return PA_ERR_WORKSPACE;
    const int64_t rows = (int64_t)num_blocks * num_kv_heads * kBlockSize;
    const Cut cut = cut_of(num_seqs, num_q_heads, num_kv_heads, max_blocks_per_seq, window, num_query_tokens, max_query_len);
    const int64_t items = cut.items * cut.splits;
    if (rows >= ((int64_t)1 << 31) || items >= ((int64_t)1 << 31) - kThreads) return PA_ERR_UNSUPPORTED;
    CUtensorMap qmap, kmap, vmap;
    if (!encode_query_map(&qmap, query, num_query_tokens, num_q_heads, num_kv_heads) ||
        !encode_block8_map(&kmap, key_cache, rows, true) || !encode_block8_map(&vmap, value_cache, rows, false))
        return cuda_failure(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
    PrefillArgs a = {};
    a.out = out;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.value_cache = static_cast<const uint8_t *>(value_cache);
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = group;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.num_query_tokens = num_query_tokens;
    a.max_query_len = max_query_len;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.n_mt = (int)cut.tiles;
    a.num_items = (int)items;
    a.splits = cut.splits;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t grid = std::min<int64_t>(items, device_sms());
    cudaError_t e;
    if (cut.splits > 1) {
        a.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kWorkspaceBytes);
        a.part_ml = reinterpret_cast<float2 *>(reinterpret_cast<uint8_t *>(a.part_o) +
                                               part_rows_bytes((int64_t)num_query_tokens * num_q_heads * cut.splits));
    }
    if (items > grid) {
        a.work_counter = static_cast<unsigned int *>(workspace);
        e = cudaMemsetAsync(workspace, 0, sizeof(unsigned int), st);
        if (e != cudaSuccess) return cuda_failure(e, "cudaMemsetAsync(prefill ticket)");
    }
    auto kernel = cut.splits > 1 ? pa_prefill_block8_kernel<true> : pa_prefill_block8_kernel<false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return cuda_failure(e, "cudaFuncSetAttribute(block-scaled prefill)");
    e = launch_chained(kernel, dim3((unsigned)grid), dim3(kThreads), (size_t)kSmemBytes, st, qmap,
                       kmap, vmap, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_prefill_block8_kernel launch");
    count_launches(1);
    if (cut.splits == 1) return PA_OK;
    const int64_t merge = ((int64_t)num_query_tokens * num_q_heads + 3) / 4;
    e = launch_chained(pa_merge_prefill8_kernel, dim3((unsigned)merge), dim3(128), 0, st, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_merge_prefill8_kernel launch");
    count_launches(1);
    return PA_OK;
}
