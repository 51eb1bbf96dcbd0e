// Paged decode attention over pools held in 4 bits ("KV cache: la memoria de trabajo
// que sostiene la inferencia LLM", section "Trucos para que el cuaderno sea más fino":
// quantising the cache), one query token per sequence.  The format is in pa_fp4.cuh.
//
// One CTA handles one (sequence, KV head, partition).  Each warp owns every NW-th
// pair of blocks of the partition and streams it through its own ring of slots: a
// block's K and V tiles are 9 head_dim bytes each, whole in the pool, so a bulk copy
// brings one.
// The group's query heads are the N columns of mma.sync m16n8k16 tiles in transposed
// form, S^T[16 tokens x 8 heads] = K Q^T and O^T[head_dim x 8 heads] += V^T P^T, so
// one pass over K/V serves the group; a group of more than 8 heads is split over
// CTAs that follow one another and find the tiles in L2.  Codes times scales are
// exact in f16.
//
// Few sequences: a context goes to a CTA of 8 or 16 warps, or is cut into parts so that
// the GPU is full.  Up to eight parts form a thread-block cluster that merges through
// distributed shared memory; more leave partials in the workspace for a second kernel.
// Many ragged ones, long for their number: CTAs take the longest first.
//
// A prefill of short chunks runs here too: where a group has few heads the columns are those of up
// to eight rows that follow one another, each of which ends a position later.
//
// 64 contexts of up to 2048 tokens with 32 KV heads, 315 MB, 62 us (5.1 TB/s, 0.75 of a
// copy); 256 of up to 4096 with 64 query heads on 8, 701 MB, 132 us (0.79); eight of 32768, 1.21
// GB, 200 us (0.89).  Bound by instructions before memory: a pair of blocks takes a warp
// 588, of which 128 conversions and 128 products with scales run at half the issue rate (ALU
// pipe 0.57 busy, issue slots 0.65).  Four warps with rings of two pairs each were the best
// shape: 2 and 8 warps 61, 132, 203 and 74, 154, 226 us, rings of three pairs 62, 132, 199, three
// and five CTAs an SM 66, 140, 208 and 62, 132, 202.  One block at a time took 77, 166 and 232 us,
// masks in every block's path 72, 150 and 210, sequences in the table's order 65, 140 and 196.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>

#include <algorithm>
#include <climits>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kHeads = 8;                        // query heads of a CTA at most
// a head's reference maximum moves only when a score exceeds it by more than
// 2^8: the weights stay in [0, 256], which f16 holds
constexpr float kLazyLog2 = 8.f;

struct Fp4Args {
    void *out;
    const void *query;
    const uint8_t *key_cache, *value_cache;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;  // sequence b's row is query_start[b]; nullptr: row b
    const int4 *chunks;          // nullptr, or chunks of rows in place of sequences: table's row (-1: none), first row, rows
    float *part_o;               // [((b * axis + kvh * splits + split) * cols + col) * max_parts + part][head_dim]
    float2 *part_ml;             // (reference, sum)
    int32_t *status;
    int num_seqs, num_rows, num_q_heads, num_kv_heads;
    int heads;                   // query heads of a CTA
    int cols;                    // its columns: those of up to eight heads, or heads of several rows (a power of two each)
    int splits;                  // CTAs of a (sequence, KV head, partition)
    int max_blocks, num_blocks;
    int part_blocks, max_parts;
    int window;
    int reach;                   // positions that a row attends to at most
    int ordered;                 // CTAs take sequences longest first
    float scale_log2;
};

struct Span {
    int L, start, blk0, nblk, nparts;
};

// Blocks of a context of `len` tokens that its last `rows` tokens attend to: [*first, *blocks),
// the first position attended in *start; *L the length, clamped.
__device__ __forceinline__ void range_of(const Fp4Args &a, int len, int rows, bool say, int *L, int *start, int *first,
                                         int *blocks) {
    const int lmax = a.max_blocks * kBlockSize;
    if (len < 0 || len > lmax) {
        if (say) report(a.status, PA_DEV_BAD_CONTEXT_LEN);
        len = len < 0 ? 0 : lmax;
    }
    *L = len;
    *start = max(len - (rows - 1) - a.reach, 0);
    *first = *start / kBlockSize;
    *blocks = (len + kBlockSize - 1) / kBlockSize;
}

// Part `part` of `parts` of a context, cut evenly.
__device__ __forceinline__ void even_span(const Fp4Args &a, int len, int rows, int part, int parts, bool say, Span &w) {
    int first, blocks;
    range_of(a, len, rows, say, &w.L, &w.start, &first, &blocks);
    const int n = max(blocks - first, 0);
    w.blk0 = first + (int)((int64_t)part * n / parts);
    w.nblk = first + (int)((int64_t)(part + 1) * n / parts) - w.blk0;
    w.nparts = 1;
}

// Partition `part` of a context of `len` tokens; false when it lies past the end.
__device__ __forceinline__ bool span_of(const Fp4Args &a, int len, int rows, int part, bool say, Span &w) {
    int first, blocks;
    range_of(a, len, rows, say, &w.L, &w.start, &first, &blocks);
    w.nparts = blocks <= first ? 1 : (blocks - first + a.part_blocks - 1) / a.part_blocks;
    if (part >= w.nparts) return false;
    w.blk0 = first + part * a.part_blocks;
    w.nblk = max(min(w.blk0 + a.part_blocks, blocks) - w.blk0, 0);
    return true;
}

// The row of query and output that is sequence b's, or -1: it brings none, or more
// than the one that a decode step has.
__device__ __forceinline__ int row_of(const Fp4Args &a, int b, bool say) {
    if (a.query_start == nullptr) return b;
    const int at = a.query_start[b], end = a.query_start[b + 1];
    if (end == at) return -1;
    const bool outside = at < 0 || end < at || end > a.num_rows;
    if (!outside && end == at + 1) return at;
    if (say) report(a.status, outside ? PA_DEV_BAD_CONTEXT_LEN : PA_DEV_BAD_QUERY_LEN);
    return -1;
}

// The sequence of rank `rank` by length, longest first, in kClasses classes of length (within one,
// in order).  A warp's work; every warp of the grid that asks agrees.
// A lane holds the lengths of eight sequences.  (With room for 1024: 320 sequences of 8 KV heads of up to 4096
// tokens 156 us against 163 in the table's order, 384 177 / 179, 512 245 / 242; 256 of 32 KV heads of up to 2048 245
// against 229 with room for 256.)
constexpr int kOrdered = 256;                    // sequences at most
constexpr int kClasses = 8;
__device__ __forceinline__ int ranked(const Fp4Args &a, int rank) {
    const int lane = threadIdx.x & 31, chunks = (a.num_seqs + 31) / 32;
    int len[kOrdered / 32], most = 0;
#pragma unroll
    for (int c = 0; c < kOrdered / 32; ++c) {
        const int i = 32 * c + lane;
        len[c] = i < a.num_seqs ? max(a.context_lens[i], 0) : -1;
        if (a.window > 0) len[c] = min(len[c], a.window);
        most = max(most, len[c]);
    }
    most = __reduce_max_sync(kFull, most);
    const float unit = (float)kClasses / ((float)most + 1.f);
#pragma unroll
    for (int c = 0; c < kOrdered / 32; ++c) len[c] = len[c] < 0 ? -1 : min((int)((float)len[c] * unit), kClasses - 1);
    for (int k = kClasses - 1; k >= 0; --k) {
#pragma unroll
        for (int c = 0; c < kOrdered / 32; ++c) {
            if (c >= chunks) break;
            const unsigned here = __ballot_sync(kFull, len[c] == k);
            const int n = __popc(here);
            if (rank < n) {
                const bool mine = ((here >> lane) & 1u) != 0 && __popc(here & ((1u << lane) - 1u)) == rank;
                return 32 * c + __ffs((int)__ballot_sync(kFull, mine)) - 1;
            }
            rank -= n;
        }
    }
    return 0;                                    // (every rank below num_seqs is found)
}

__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
// kWords (1, 2 or 4) words from a place aligned to them
template <int kWords>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t *w) {
    if constexpr (kWords == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    else if constexpr (kWords == 2) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr));
}

// The low half of every byte of a, the high half of every byte of b.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xe4;" : "=r"(d) : "r"(a), "r"(b), "r"(0x0f0f0f0fu));      // a & c | b & ~c
    return d;
}

// mma_f16_16816 that a compiler may move
__device__ __forceinline__ void mma_pure(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A tile, whole and contiguous in its pool, into shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// Column `col`'s (row, head) in query and output, as a number of heads: the heads of the
// CTA's first row, then of those behind it.
template <bool kChunks>
__device__ __forceinline__ int64_t at_of(const Fp4Args &a, int row, int first_head, int col) {
    const int r = kChunks ? col / a.heads : 0;
    return (int64_t)(row + r) * a.num_q_heads + first_head + col - r * a.heads;
}

// One warp's attention state over its blocks: 8 query heads (columns; those past
// the group have a zero query and are not stored).  Lane (g, t) = (lane / 4, lane %
// 4) holds scores of tile rows g and g + 8 for heads 2t and 2t + 1.
//  * S^T: the contraction may visit the head dimension in any order as long as K and
//    Q agree, so lane t of a row reads a quarter of it (of each 128 elements) in
//    consecutive pieces of 16 bytes, 32 codes under two scales.
//  * O^T: the A operand needs two tokens of one element in a register.  Lane g reads
//    the 16 codes under scale g of four tokens; codes of two tokens are paired
//    within bytes (the even elements, then the odd ones), so that widening gives the pair.
//  * Tile row r stands for token r, but rows 4, 5 and 6, 7 (and 12 to 15) are
//    swapped: the four tokens that lanes t = 0 to 3 read together are then two even
//    and two odd ones, which meet in each bank twice instead of four times.
// kChunks: the columns are those of several rows.
template <int D, bool kChunks>
struct Warp4 {
    static constexpr int kRow = D / 2;           // bytes of a row's codes
    static constexpr int kScales = D / 16;       // of a row
    static constexpr int kKWords = D / 32;       // words of a row's codes that a lane reads for K
    static constexpr int kLoad = D == 64 ? 2 : 4;        // words of one load for K

    uint32_t qb[D / 16][2];
    float o[D / 16][4];
    float m0, m1, l0, l1;
    float qs0, qs1;              // powers of two of heads 2t and 2t + 1: what their scores are multiplied by
    int lane, g, t;
    uint32_t kcode, kscale, vcode[2], vscale[2];

    // First element of this lane's K word w, and of its V word v.
    __device__ __forceinline__ int k_at(int w) const { return D == 64 ? 16 * t + 8 * w : 128 * (w / 4) + 32 * t + 8 * (w % 4); }
    __device__ __forceinline__ int v_at(int v) const { return D == 64 ? 8 * g : 128 * (v / 2) + 16 * g + 8 * (v % 2); }

    __device__ __forceinline__ void load(const Fp4Args &a, int row, int rows, int first_head, int lane_, uint4 (&w)[kKWords]) {
        lane = lane_;
        g = lane >> 2;
        t = lane & 3;
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.query) + at_of<kChunks>(a, row, first_head, g) * D;
#pragma unroll
        for (int c = 0; c < kKWords; ++c)
            w[c] = g < a.heads * rows ? *reinterpret_cast<const uint4 *>(q + k_at(c)) : make_uint4(0u, 0u, 0u, 0u);
    }

    __device__ __forceinline__ void init(const Fp4Args &a, const uint4 (&w)[kKWords]) {
        const int token = g < 4 ? g : g ^ 1, pair = t < 2 ? 2 * t : 2 * t + 1;
        kcode = (uint32_t)(token * kRow + k_at(0) / 2);
        kscale = (uint32_t)(fp4_scales_at(D) + token * kScales + k_at(0) / 16);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            vcode[i] = (uint32_t)((pair ^ i) * kRow + v_at(0) / 2);
            vscale[i] = (uint32_t)(fp4_scales_at(D) + (pair ^ i) * kScales + v_at(0) / 16);
        }
        uint32_t amax = 0;                               // as bits: magnitudes compare like integers
#pragma unroll
        for (int c = 0; c < kKWords; ++c)
#pragma unroll
            for (uint32_t x : {w[c].x, w[c].y, w[c].z, w[c].w})
                amax = max(amax, max((x << 16) & 0x7fffffffu, x & 0x7fff0000u));
        amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = max(amax, __shfl_xor_sync(kFull, amax, 2));
        // A row is brought up or down by a power of two so that its largest magnitude lies in
        // [2^14, 2^15): f16 then holds every element exactly but those below 2^-29 of it,
        // which are off by at most 2^-39 of it.
        const int up = min(14 + 127 - (int)(amax >> 23), 126);
        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
        const int down = (127 - up) << 23;               // 2^-up, of row g
        qs0 = __int_as_float(__shfl_sync(kFull, down, 8 * t)) * a.scale_log2;
        qs1 = __int_as_float(__shfl_sync(kFull, down, 8 * t + 4)) * a.scale_log2;
#pragma unroll
        for (int c = 0; c < kKWords; ++c) {
            qb[2 * c][0] = pack_f16x2(bf16lo(w[c].x) * f, bf16hi(w[c].x) * f);
            qb[2 * c][1] = pack_f16x2(bf16lo(w[c].y) * f, bf16hi(w[c].y) * f);
            qb[2 * c + 1][0] = pack_f16x2(bf16lo(w[c].z) * f, bf16hi(w[c].z) * f);
            qb[2 * c + 1][1] = pack_f16x2(bf16lo(w[c].w) * f, bf16hi(w[c].w) * f);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        // (of several rows one may attend to nothing of the first blocks: the least number lets its
        // weights there, of scores of -infinity, be zero)
        m0 = m1 = kChunks ? -FLT_MAX : -INFINITY;
        l0 = l1 = 0.f;
    }

    // S^T of two tiles in this lane's fragment, times the scales of the query's heads and the
    // softmax.  The tiles' products alternate, each tile's in two sums: a product waits for the fourth one before.
    __device__ __forceinline__ void scores(uint32_t ktile, uint32_t stride, float (&s)[2][4]) const {
        float part[2][2][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) part[i >> 3][(i >> 2) & 1][i & 3] = 0.f;
#pragma unroll
        for (int c = 0; c < kKWords / kLoad; ++c) {
            uint32_t r[2][2][kLoad], sc[2][2][2];        // [tile][row g, g + 8]
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lds_words<kLoad>(ktile + u * stride + kcode + 64 * c + 8 * i * kRow, r[u][i]);
                    const uint32_t at = ktile + u * stride + kscale + 8 * c + 8 * i * kScales;
                    const uint32_t w = D == 64 ? lds8(at) : lds16(at);
                    sc[u][i][0] = fp4_scale_pair<0>(w);
                    sc[u][i][1] = fp4_scale_pair<1>(w);
                }
#pragma unroll
            for (int w = 0; w < kLoad; ++w) {
                const int k = 2 * (c * kLoad + w);
                uint32_t x[2][4], y[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    e2m1x8_to_f16x2x4(r[u][0][w], x[u]);
                    e2m1x8_to_f16x2x4(r[u][1][w], y[u]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[u][i] = mul_f16x2(x[u][i], sc[u][0][w / 2]);
                        y[u][i] = mul_f16x2(y[u][i], sc[u][1][w / 2]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t f[4] = {x[u][2 * e], y[u][2 * e], x[u][2 * e + 1], y[u][2 * e + 1]};
                        mma_pure(part[u][e], f, qb[k + e][0], qb[k + e][1]);
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][i] = (part[u][0][i] + part[u][1][i]) * (i & 1 ? qs1 : qs0);
    }

    // O^T += V^T P^T of a tile.
    __device__ __forceinline__ void values(uint32_t vtile, uint32_t b0, uint32_t b1) {
#pragma unroll
        for (int c = 0; c < (D + 127) / 128; ++c) {
            constexpr int kWords = D == 64 ? 1 : 2;
            uint32_t w[4][kWords];                       // of tokens 2t, 2t + 1, 2t + 8, 2t + 9 (in swapped order)
            uint32_t sc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lds_words<kWords>(vtile + vcode[i & 1] + 64 * c + (i & 2) * 4 * kRow, w[i]);
                sc[i] = lds8(vtile + vscale[i & 1] + 8 * c + (i & 2) * 4 * kScales);
            }
            const uint32_t sa = __byte_perm(sc[0], sc[1], 0x4101) >> 1, sb = __byte_perm(sc[2], sc[3], 0x4101) >> 1;
#pragma unroll
            for (int v = 0; v < kWords; ++v) {
                uint32_t ea[4], oa[4], eb[4], ob[4];
                e2m1x8_to_f16x2x4(low_halves(w[0][v], w[1][v] << 4), ea);
                e2m1x8_to_f16x2x4(low_halves(w[0][v] >> 4, w[1][v]), oa);
                e2m1x8_to_f16x2x4(low_halves(w[2][v], w[3][v] << 4), eb);
                e2m1x8_to_f16x2x4(low_halves(w[2][v] >> 4, w[3][v]), ob);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t x[4] = {mul_f16x2(ea[k], sa), mul_f16x2(oa[k], sa), mul_f16x2(eb[k], sb), mul_f16x2(ob[k], sb)};
                    mma_pure(o[4 * (c * kWords + v) + k], x, b0, b1);
                }
            }
        }
    }

    // Two blocks side by side in shared memory (K, V, K, V), of whose 32 rows the first `limit` are there
    // (16: what the second block's place holds does not matter), and the last query row of `rows` attends to
    // `reach` ones before the one numbered `end`, each earlier one to a place less.  (At least one of them attends to one.)
    __device__ __forceinline__ void blocks(const Fp4Args &a, uint32_t tiles, int end, int limit, int rows) {
        constexpr uint32_t kTile = fp4_tile_bytes(D);
        float s[2][4];
        scores(tiles, 2 * kTile, s);
        if (end > a.reach || min(limit, end - rows + 1) < 2 * kBlockSize) {
            // rows that are not attended may hold any scale, NaN among them, and would reach the sum as 0 * NaN
            const int nlo = end - rows + 1 - a.reach, nvalid = min(limit, end);
            if (lane < nlo || lane >= nvalid) {
                const uint32_t at = tiles + (2 * (lane / kBlockSize) + 1) * kTile + fp4_scales_at(D) + lane % kBlockSize * kScales;
#pragma unroll
                for (int i = 0; i < kScales; i += 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + i), "r"(0u) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            const int token = g < 4 ? g : g ^ 1;
            // the rows behind those of columns 2t and 2t + 1
            const int cut0 = kChunks ? max(rows - 1 - 2 * t / a.heads, 0) : 0, cut1 = kChunks ? max(rows - 1 - (2 * t + 1) / a.heads, 0) : 0;
            auto outside = [&](int r, int cut) { return r >= min(limit, end - cut) || r < end - cut - a.reach; };
#pragma unroll
            for (int i = 0; i < 4; ++i) {                // row token + 8 i
                float *x = &s[i >> 1][2 * (i & 1)];
                x[0] = outside(token + 8 * i, cut0) ? -INFINITY : x[0];
                x[1] = outside(token + 8 * i, cut1) ? -INFINITY : x[1];
            }
        }
        // every lane looks at its own scores; the column's maximum is only found where one rises
        float mx0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
        float mx1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
        if (__any_sync(kFull, mx0 > m0 + kLazyLog2 || mx1 > m1 + kLazyLog2)) {
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, k));
                mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, k));
            }
            const bool need0 = mx0 > m0 + kLazyLog2, need1 = mx1 > m1 + kLazyLog2;
            const float a0 = need0 ? exp2f(m0 - mx0) : 1.f;      // 0 while m0 is -inf
            const float a1 = need1 ? exp2f(m1 - mx1) : 1.f;
            m0 = need0 ? mx0 : m0;
            m1 = need1 ? mx1 : m1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                o[i][0] *= a0;
                o[i][1] *= a1;
                o[i][2] *= a0;
                o[i][3] *= a1;
            }
        }
        uint32_t p[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float w0 = ex2_fast(s[u][0] - m0), w1 = ex2_fast(s[u][1] - m1);
            const float w2 = ex2_fast(s[u][2] - m0), w3 = ex2_fast(s[u][3] - m1);
            l0 += w0 + w2;
            l1 += w1 + w3;
            // the weights enter the second product as f16, rounded once: 11 bits
            // move an output by at most 2^-11 of the largest value it weighs, where
            // bf16's 8 bits would be as coarse as the output's own rounding
            p[u][0] = movmatrix_trans(pack_f16x2(w0, w1));
            p[u][1] = movmatrix_trans(pack_f16x2(w2, w3));
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) values(tiles + (2 * u + 1) * kTile, p[u][0], p[u][1]);
    }

    // The state as acc[heads][D], m[heads], l[heads].
    __device__ __forceinline__ void finish(int heads, float *acc, float *m, float *l) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) {
            l0 += __shfl_xor_sync(kFull, l0, k);
            l1 += __shfl_xor_sync(kFull, l1, k);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = 2 * t + e;
            if (h >= heads) continue;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                *reinterpret_cast<float2 *>(acc + h * D + v_at(i / 4) + 2 * (i & 3)) = make_float2(o[i][e], o[i][2 + e]);
            if (g == 0) {
                m[h] = e ? m1 : m0;
                l[h] = e ? l1 : l0;
            }
        }
    }
};

template <int D, int NW, int STAGES>
struct Shape {
    static constexpr int kStage = 4 * fp4_tile_bytes(D);         // K, V, K, V of two blocks
    static constexpr int kRing = NW * STAGES * kStage;
    static_assert(STAGES * kStage >= kHeads * D * 4, "a warp's state is merged over its ring");
    static_assert(kRing % 16 == 0 && kStage % 16 == 0, "bulk copies");
    static size_t smem(int part_blocks) {
        return kRing + (size_t)((part_blocks + 1) & ~1) * sizeof(int) + NW * STAGES * 8 + 2 * NW * kHeads * sizeof(float);
    }
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float of another CTA of the cluster, at the same shared-memory offset as ours.
__device__ __forceinline__ float remote_f32(const float *mine, uint32_t rank) {
    uint32_t addr;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// kParts > 1: the grid's clusters of kParts CTAs each work on one (sequence, KV head).
// kChunks: on chunks of rows (an instance of its own: looking at them cost a single context 1.5 us of
// 5.4, 256 of them 2 of 132).
template <int D, int NW, int STAGES, int kParts, bool kChunks>
__global__ void __launch_bounds__(NW * 32, D == 256 ? 1 : 16 / NW) pa_decode_fp4_kernel(const Fp4Args a) {
    using S = Shape<D, NW, STAGES>;
    constexpr uint32_t kTile = fp4_tile_bytes(D);
    grid_dependency_wait();
    grid_dependents_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // CTAs go partition by partition, so that the shorter last partitions (and
    // the empty ones of short sequences) end the grid
    const int axis = a.num_kv_heads * a.splits;
    int idx = blockIdx.x, part;
    if constexpr (kParts > 1) {
        part = (int)cluster_rank();
        idx /= kParts;
    } else {
        part = idx / (a.num_seqs * axis);
        idx -= part * a.num_seqs * axis;
    }
    int b = idx / axis;
    idx -= b * axis;
    if (kParts == 1 && a.ordered) b = ranked(a, b);
    const int kvh = idx / a.splits;
    const int first_head = kvh * a.heads * a.splits + (idx - kvh * a.splits) * a.heads;
    // What depends on the CTA's place alone is loaded together, so that a CTA waits one
    // memory round trip before its first tile is requested: the length, the table
    // entries of the warp's first blocks (a window moves the partition with the length;
    // then the table follows it) and the query.  All of it is the warp's own business:
    // no barrier before the merge.
    const int len = a.context_lens[b];
    int4 chunk = make_int4(b, 0, 1, 0);
    if constexpr (kChunks) {
        chunk = a.chunks[b];
        if (chunk.x < 0) return;                         // (a cluster's CTAs all leave)
    }
    const int rows = kChunks ? chunk.z : 1;
    const int32_t *row_table = a.block_tables + (int64_t)chunk.x * a.max_blocks;
    const bool early = kParts == 1 && a.window == 0;     // the partition does not move with the length
    const int in_part = 2 * (warp + NW * (lane >> 1)) + (lane & 1), ahead = part * a.part_blocks + in_part;
    int first_phys = early && in_part < a.part_blocks && ahead < a.max_blocks ? row_table[ahead] : -1;
    const bool say = threadIdx.x == 0 && part == 0 && idx == 0;
    const int row = kChunks ? chunk.y : row_of(a, b, say);
    if (row < 0) return;                                 // (a cluster's CTAs all leave)
    Warp4<D, kChunks> state;
    uint4 query[Warp4<D, kChunks>::kKWords];
    state.load(a, row, rows, first_head, lane, query);
    Span w;
    if constexpr (kParts > 1) even_span(a, len, rows, part, kParts, say, w);
    else if (!span_of(a, len, rows, part, say, w)) return;

    extern __shared__ __align__(128) uint8_t ring[];
    int *entries = reinterpret_cast<int *>(ring + S::kRing);     // physical blocks of the partition
    uint64_t *bars = reinterpret_cast<uint64_t *>(entries + ((a.part_blocks + 1) & ~1));
    float *s_m = reinterpret_cast<float *>(bars + NW * STAGES);
    float *s_l = s_m + NW * kHeads;
    __shared__ int s_fail[NW];
    const int pairs = (w.nblk + 1) / 2, count = pairs > warp ? (pairs - warp + NW - 1) / NW : 0;
    uint64_t *my_bars = bars + warp * STAGES;
    uint8_t *my_ring = ring + warp * STAGES * S::kStage;
    if (lane == 0) {
        s_fail[warp] = 0;
#pragma unroll
        for (int s = 0; s < STAGES; ++s) mbar_init(&my_bars[s], 1);
        fence_mbar_init();
    }
    auto entry_of = [&](int phys) {
        if ((unsigned)phys >= (unsigned)a.num_blocks) {
            report(a.status, PA_DEV_BAD_BLOCK_ID);
            phys = 0;
        }
        return phys;
    };
    // the warp's blocks in its own order: block k is half of its pair k / 2
    auto place_of = [&](int k) { return 2 * (warp + NW * (k >> 1)) + (k & 1); };
    const int32_t *table = row_table + w.blk0;
    if (!early) first_phys = place_of(lane) < w.nblk ? table[place_of(lane)] : -1;
    const int first_at = place_of(lane) < w.nblk ? entry_of(first_phys) : 0;

    const uint64_t policy = l2_policy_evict_first();     // tiles are read once: they leave L2 first
    // lanes 0 to 3 each bring a tile of pair `it`, whose blocks are phys (of the lane's)
    const uint8_t *pool = lane & 1 ? a.value_cache : a.key_cache;
    auto issue = [&](int it, int phys) {
        const int s = it % STAGES, here = min(2, w.nblk - place_of(2 * it));
        if (lane == 0) mbar_arrive_expect_tx(&my_bars[s], 2 * kTile * here);
        __syncwarp();
        if (lane < 2 * here)
            bulk_load(my_ring + s * S::kStage + lane * kTile, pool + ((int64_t)phys * a.num_kv_heads + kvh) * kTile, kTile,
                      &my_bars[s], policy);
    };
#pragma unroll
    for (int it = 0; it < STAGES; ++it) {
        const int at = __shfl_sync(kFull, first_at, 2 * it + (lane >> 1 & 1));
        if (it < count) issue(it, at);
    }
    state.init(a, query);                                // under the tiles' latency
    for (int k = lane; place_of(k) < w.nblk; k += 32) entries[place_of(k)] = k == lane ? first_at : entry_of(table[place_of(k)]);
    __syncwarp();
    bool ok = true;
    int it = 0;
    for (; it < count; ++it) {
        const int s = it % STAGES;
        if (!__all_sync(kFull, mbar_wait_bounded(&my_bars[s], (it / STAGES) & 1))) {
            ok = false;
            break;
        }
        const int place = place_of(2 * it), tok = (w.blk0 + place) * kBlockSize;
        state.blocks(a, smem_u32(my_ring + s * S::kStage), w.L - tok, kBlockSize * min(2, w.nblk - place), rows);
        __syncwarp();
        if (it + STAGES < count) {
            if (lane < 4) fence_proxy_async_smem();
            issue(it + STAGES, entries[min(place_of(2 * (it + STAGES) + (lane >> 1 & 1)), w.nblk - 1)]);
        }
    }
    if (!ok) {
        // copies in flight get a bounded chance to land before the memory is given up
        for (int k = it; k < count && k < it + STAGES; ++k)
            (void)mbar_wait_bounded(&my_bars[k % STAGES], (k / STAGES) & 1);
        if (lane == 0) {
            report(a.status, PA_DEV_TIMEOUT);
            s_fail[warp] = 1;
        }
    }
    // the ring is idle: the warps' states are merged over it
    float *acc = reinterpret_cast<float *>(my_ring);
    const int cols = a.heads * rows;
    state.finish(cols, acc, s_m + warp * kHeads, s_l + warp * kHeads);
    __syncthreads();
    bool failed = false;
#pragma unroll
    for (int k = 0; k < NW; ++k) failed |= s_fail[k] != 0;
    auto merged = [&](int i, float &M, float &sum) {     // element i of the CTA's state
        const int h = i / D;
        float O = 0.f;
        M = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) M = fmaxf(M, s_m[k * kHeads + h]);
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const float mk = s_m[k * kHeads + h];
            const float f = mk == -INFINITY ? 0.f : exp2f(mk - M);
            sum = fmaf(f, s_l[k * kHeads + h], sum);
            O = fmaf(f, reinterpret_cast<const float *>(ring + k * STAGES * S::kStage)[i], O);
        }
        // after a wait that gave up the row is NaN, through its partial sums too: what an earlier
        // call left in the workspace must not pass for an output
        if (failed) sum = __int_as_float(0x7fffffff);
        return O;
    };
    // the CTA's first column, among the partials and in the output
    const int64_t col0 = kChunks ? ((int64_t)b * axis + idx) * a.cols : (int64_t)b * a.num_q_heads + first_head;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)row * a.num_q_heads + first_head) * D;
    auto put = [&](int i, float x) {                     // element i of the CTA's columns
        const int skipped = kChunks ? i / D / a.heads * (a.num_q_heads - a.heads) * D : 0;
        out[i + skipped] = __float2bfloat16_rn(x);
    };
    if constexpr (kParts > 1) {
        // The parts' states side by side in the cluster's shared memory: each CTA
        // merges its share of the elements.  A part that gave up keeps its place at
        // the barriers; its sum makes the row NaN.
        constexpr int kEach = kHeads * D / (NW * 32);
        float O[kEach], M[kEach], sum[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = threadIdx.x + e * NW * 32;
            if (i < cols * D) O[e] = merged(i, M[e], sum[e]);
        }
        __syncthreads();                                 // the warps' states are read
        float *state_o = reinterpret_cast<float *>(ring), *state_m = s_m, *state_l = s_l;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = threadIdx.x + e * NW * 32;
            if (i >= cols * D) continue;
            state_o[i] = O[e];
            if (i % D == 0) {
                state_m[i / D] = M[e];
                state_l[i / D] = sum[e];
            }
        }
        cluster_sync();
        for (int i = (int)threadIdx.x + part * NW * 32; i < cols * D; i += kParts * NW * 32) {
            const int h = i / D;
            float pm[kParts], pl[kParts], po[kParts], top = -INFINITY;
#pragma unroll
            for (int r = 0; r < kParts; ++r) {
                pm[r] = remote_f32(state_m + h, r);
                pl[r] = remote_f32(state_l + h, r);
                po[r] = remote_f32(state_o + i, r);
            }
#pragma unroll
            for (int r = 0; r < kParts; ++r) top = fmaxf(top, pm[r]);
            float o = 0.f, l = 0.f;
#pragma unroll
            for (int r = 0; r < kParts; ++r) {
                const float f = pm[r] == -INFINITY ? 0.f : exp2f(pm[r] - top);
                l = fmaf(f, pl[r], l);
                o = fmaf(f, po[r], o);
            }
            put(i, l == 0.f ? 0.f : o / l);
        }
        cluster_sync();                                  // no CTA leaves while its state is read
    } else {
        const bool whole = w.nparts == 1;
        for (int i = threadIdx.x; i < cols * D; i += NW * 32) {
            float M, sum;
            const float O = merged(i, M, sum);
            if (whole) {
                // a NaN sum stays NaN; an empty context gives zeros
                put(i, sum == 0.f ? 0.f : O / sum);
            } else {
                const int64_t at = (col0 + i / D) * a.max_parts + part;
                a.part_o[at * D + i % D] = O;
                if (i % D == 0) a.part_ml[at] = make_float2(M, sum);
            }
        }
    }
}

// Merges the partitions of a column, one CTA a column: warp w
// takes partials w, w + kMergeWarps, ..., a lane four of 128 columns, four partials on
// their way at a time; the warps' sums meet in shared memory.
constexpr int kMergeWarps = 4;
template <int D, bool kChunks>
__global__ void __launch_bounds__(32 * kMergeWarps) pa_merge_fp4_kernel(const Fp4Args a) {
    constexpr int kVec = D / 4, kPer = (kVec + 31) / 32;         // 16-byte pieces of a row, and of a lane
    __shared__ float4 s_acc[kMergeWarps][kVec];
    __shared__ float s_sum[kMergeWarps], s_max[kMergeWarps];
    grid_dependency_wait();
    grid_dependents_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    Span w;
    const int per_seq = kChunks ? a.num_kv_heads * a.splits * a.cols : a.num_q_heads, b = (int)(row / per_seq);
    const int in_seq = (int)(row - (int64_t)b * per_seq), col = kChunks ? in_seq % a.cols : 0;
    int rows = 1, out_row;
    if constexpr (kChunks) {
        const int4 c = a.chunks[b];
        out_row = c.x < 0 ? -1 : c.y;
        rows = c.z;
        if (col >= a.heads * rows) return;
    } else {
        out_row = row_of(a, b, false);
    }
    span_of(a, a.context_lens[b], rows, 0, false, w);
    if (w.nparts <= 1 || out_row < 0) return;
    const float2 *ml = a.part_ml + row * a.max_parts;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + row * a.max_parts * D);
    float M = -INFINITY, sum = 0.f;
    float4 acc[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = warp; p0 < w.nparts; p0 += 4 * kMergeWarps) {
        float4 v[4][kPer];
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + i * kMergeWarps;
#pragma unroll
            for (int c = 0; c < kPer; ++c)
                v[i][c] = p < w.nparts && lane + 32 * c < kVec ? po[(int64_t)p * kVec + lane + 32 * c] : make_float4(0.f, 0.f, 0.f, 0.f);
            x[i] = p < w.nparts ? ml[p] : make_float2(-INFINITY, 0.f);
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, x[i].x);
        const float g = M == -INFINITY ? 0.f : exp2f(M - top);
        M = top;
        sum *= g;
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] = make_float4(acc[c].x * g, acc[c].y * g, acc[c].z * g, acc[c].w * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = x[i].x == -INFINITY ? 0.f : exp2f(x[i].x - M);
            sum = fmaf(f, x[i].y, sum);
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                acc[c].x = fmaf(f, v[i][c].x, acc[c].x);
                acc[c].y = fmaf(f, v[i][c].y, acc[c].y);
                acc[c].z = fmaf(f, v[i][c].z, acc[c].z);
                acc[c].w = fmaf(f, v[i][c].w, acc[c].w);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kPer; ++c)
        if (lane + 32 * c < kVec) s_acc[warp][lane + 32 * c] = acc[c];
    if (lane == 0) {
        s_sum[warp] = sum;
        s_max[warp] = M;
    }
    __syncthreads();
    if ((int)threadIdx.x >= kVec) return;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) top = fmaxf(top, s_max[k]);
    sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) {
        const float f = s_max[k] == -INFINITY ? 0.f : exp2f(s_max[k] - top);
        const float4 v = s_acc[k][threadIdx.x];
        sum = fmaf(f, s_sum[k], sum);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t out_head = kChunks ? at_of<true>(a, out_row, in_seq / a.cols * a.heads, col) : (int64_t)out_row * a.num_q_heads + in_seq;
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + out_head * D + 4 * threadIdx.x) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Query heads of one CTA: the group, or its largest divisor up to 8.
int heads_per_cta(int group) {
    int h = std::min(group, kHeads);
    while (group % h != 0) --h;
    return h;
}

struct Plan {
    int part_blocks, max_parts;
    int cluster;                 // CTAs of a cluster; > 1: max_parts is 1
    int warps;                   // of a CTA: 4, or without clusters 1, 8 or 16
    bool ordered;                // longest sequences first
    double time;                 // estimated, in microseconds (partition_size 0)
};

// Microseconds that each warp's pair of blocks takes with `ctas_per_sm` CTAs of `warps` warps on an SM.  A
// warp alone on its scheduler takes 0.8 us a pair (of 128 elements; its products wait for one
// another), and the SM 0.44 us for every four warps where many share it.
double pair_time(double ctas_per_sm, int warps, int head_dim) {
    const double k = warps / 4.0 * std::max(1.0, ctas_per_sm), f = head_dim == 64 ? 0.68 : head_dim == 256 ? 1.5 : 1.0;
    return f * (k <= 1 ? 0.8 : k <= 2 ? 1.05 : std::max(1.65, 0.44 * k));
}

// How contexts are cut, by the table's width, as only the GPU knows the lengths.  Compared are
// whole contexts (3.5 us and their pairs) by CTAs of 4, 8 or 16 warps, clusters of 2, 4 or 8 CTAs that fit the GPU at once
// (4.6 us, and 2.5 ns a CTA more) and parts enough to fill the GPU with a merge behind them (5 us
// and 5.8 ns a CTA, up to a thousand).  Parts have 8 blocks at least, 40 where the sequences alone
// make a CTA an SM, and 128 at most, or 256 where there are CTAs enough; a number of CTAs that
// is short of filling the GPU by an eighth is left.
// A few CTAs have more warps: the SM then has as much to do as in clusters, and less to merge.
// Contexts between half of and all of 1024 tokens, 8 KV heads of 128: 16 of them by 4 warps 10.1 us, by
// 16 8.5, in clusters of 2 or 4 9.9, of 8 14.8; 32 by 4 warps 12.9, by 8 12.3; of 2048: 8 by 4 warps
// 16.1, in clusters of 4 9.7; 16 by 4 warps 16.5, by 16 12.4, in clusters of 4 13.6, in 5 parts 14.8; 32 by 4
// warps 21.4, by 8 19.2, in clusters of 2 20.6, in 3 parts 24.4; of 8192: one in clusters of 8 11.4, in 64 parts
// 10.4; 32 by 4 warps 70.8, in clusters of 2 60.4, in 3 parts 59.2.
//
// Where there are more than five CTAs per SM and their parts short, CTAs have one warp, 16
// of which an SM holds: a short part's time is its start and its end.  Contexts between half of
// and all of 32 tokens: 800 CTAs 5.8 us against 9.8, 2048 7.8 / 21.0; of 128: 9.3 / 11.3, 13.7 / 23.6;
// of 512: 800 CTAs 21.2 / 18.3.  (Those of 512 CTAs or fewer gain nothing: 128 tokens 7.7 / 6.3.)
bool plan_of(int num_seqs, int axis, int max_blocks, int window, int partition_size, int head_dim, Plan *p) {
    if (partition_size != 0 && (partition_size < kBlockSize || partition_size > kMaxPartition || partition_size % kBlockSize))
        return false;
    int span = max_blocks;
    if (window > 0) span = std::min(span, (window - 1) / kBlockSize + 2);
    p->cluster = 1;
    p->warps = 4;
    // what the GPU holds at once: four CTAs of four warps an SM, two with heads of 256
    const int64_t sms = device_sms(), ctas = std::max<int64_t>(1, (int64_t)num_seqs * axis), target = (head_dim == 256 ? 2 : 4) * sms;
    if (partition_size != 0) {
        p->part_blocks = partition_size / kBlockSize;
    } else {
        const int most = ctas >= target ? 256 : 128, largest = kMaxPartition / kBlockSize;
        int64_t parts = std::max<int64_t>((target - ctas / 8 + ctas - 1) / ctas, (span + most - 1) / most);
        parts = std::max<int64_t>(1, std::min<int64_t>(parts, 4 * ctas > target ? span / 40 : (span + 7) / 8));
        // a grid beyond 32 CTAs an SM is made of the largest parts only: a wide table's last ones are often empty
        parts = std::min(parts, std::max<int64_t>(std::max<int64_t>((target + ctas - 1) / ctas, 8 * target / ctas),
                                                  (span + largest - 1) / largest));
        auto cost = [&](int64_t n, int warps, double base) {             // in n parts, by CTAs of `warps` warps
            return base + (double)((span + 2 * warps * n - 1) / (2 * warps * n)) * pair_time((double)ctas * n / sms, warps, head_dim);
        };
        double best = parts > 1 ? cost(parts, 4, 5.0 + 0.0058 * std::min((double)ctas * parts, 1024.0)) : INFINITY;
        for (int w = 4; w <= (head_dim == 256 ? 8 : 16); w *= 2)
            if (span <= largest && (w == 4 || ctas * w <= 4 * target) && cost(1, w, 3.5 + 0.02 * (w - 4)) <= best) {
                best = cost(1, w, 3.5 + 0.02 * (w - 4));
                parts = 1;
                p->warps = w;
            }
        for (int c = 2; c <= 8 && ctas * c <= target; c *= 2)
            if ((span + c - 1) / c < largest && c <= span && cost(c, 4, 4.6 + 0.0025 * ctas * c) < best) {
                best = cost(c, 4, 4.6 + 0.0025 * ctas * c);
                p->cluster = c;
            }
        if (p->cluster > 1) p->warps = 4;
        p->time = best;
        p->part_blocks = p->cluster > 1 ? (span + p->cluster - 1) / p->cluster + 1 : std::max(1, (int)((span + parts - 1) / parts));
    }
    p->max_parts = p->cluster > 1 ? 1 : std::max(1, (span + p->part_blocks - 1) / p->part_blocks);
    const int64_t all = ctas * p->max_parts;
    if (p->cluster == 1 && p->part_blocks <= (2 * all > 5 * target ? 24 : 4 * all > 5 * target ? 16 : 0)) p->warps = 1;
    // Longest first saves a share of the longest CTA's time, which grows with the span, and costs each CTA 1.4 us of
    // ranking, which adds up with the waves.  In order of length against the table's: 32 heads of their own,
    // contexts of up to 512 tokens, 128 sequences 52.6 us against 47.1, 256 107.7 / 87.4; of up to 2048, 64
    // 68.9 / 75.1, 128 121.0 / 122.9, 192 170.7 / 167.3, 256 228.9 / 215.3; of up to 16384, 64 373 / 443; 8 KV
    // heads, of up to 1024, 128 26.6 / 28.4, 256 51.1 / 49.6, of up to 4096, 256 121.9 / 133.1.  With heads of 64 and
    // 256 (25 shapes) it takes the faster order or is within 7% of it.
    // (Nor where CTAs are short: 2048 of one warp on 32 tokens 9.1 us in order of length, 7.8 in theirs.)
    p->ordered = p->warps == 4 && p->cluster == 1 && p->max_parts == 1 && num_seqs > 1 && num_seqs <= kOrdered && ctas > target &&
                 span * target > 20 * ctas;
    return true;
}

bool head_dim_ok(int head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }

size_t rows_bytes(int64_t rows, int head_dim) { return ((size_t)rows * head_dim * sizeof(float) + 255) & ~size_t(255); }

size_t workspace_of(int num_seqs, int num_q_heads, int head_dim, int max_parts) {
    if (max_parts <= 1) return 0;
    const int64_t rows = (int64_t)num_seqs * num_q_heads * max_parts;
    return rows_bytes(rows, head_dim) + (size_t)rows * sizeof(float2);
}

template <int D, int NW, int STAGES, int kParts>
pa_status launch_decode(const Fp4Args &a, cudaStream_t st) {
    using S = Shape<D, NW, STAGES>;
    auto kernel = pa_decode_fp4_kernel<D, NW, STAGES, kParts, false>;
    if constexpr (D == 128)                              // what prefill takes
        if (a.chunks != nullptr) kernel = pa_decode_fp4_kernel<D, NW, STAGES, kParts, true>;
    cudaError_t e = allow_smem(kernel, S::smem(kMaxPartition / kBlockSize));
    if (e != cudaSuccess) return cuda_failure(e, "cudaFuncSetAttribute(4-bit decode)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.num_seqs * a.num_kv_heads * a.splits * a.max_parts * kParts));
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = S::smem(a.part_blocks);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kParts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kParts > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_decode_fp4_kernel launch");
    count_launches(1);
    return PA_OK;
}

template <int D>
pa_status launch_all(const Fp4Args &a, const Plan &p, cudaStream_t st) {
    pa_status (*launch)(const Fp4Args &, cudaStream_t) = launch_decode<D, 4, 2, 1>;
    if (p.cluster == 2) launch = launch_decode<D, 4, 2, 2>;
    if (p.cluster == 4) launch = launch_decode<D, 4, 2, 4>;
    if (p.cluster == 8) launch = launch_decode<D, 4, 2, 8>;
    if (p.warps == 1) launch = launch_decode<D, 1, 2, 1>;
    if (p.warps == 8) launch = launch_decode<D, 8, 2, 1>;
    if constexpr (D < 256)
        if (p.warps == 16) launch = launch_decode<D, 16, 2, 1>;
    const pa_status s = launch(a, st);
    if (s != PA_OK || p.max_parts <= 1) return s;
    auto merge = pa_merge_fp4_kernel<D, false>;
    if constexpr (D == 128)
        if (a.chunks != nullptr) merge = pa_merge_fp4_kernel<D, true>;
    const cudaError_t e = launch_chained(merge, dim3((unsigned)(a.num_seqs * a.num_kv_heads * a.splits * a.cols)),
                                         dim3(32 * kMergeWarps), 0, st, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_merge_fp4_kernel launch");
    count_launches(1);
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_fp4_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                                int max_blocks_per_seq, int block_size, int window, int partition_size) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || !head_dim_ok(head_dim) ||
        max_blocks_per_seq < 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize || block_size != kBlockSize || window < 0)
        return (size_t)-1;
    const int group = num_q_heads / num_kv_heads;
    Plan p;
    if (!plan_of(num_seqs, num_kv_heads * (group / heads_per_cta(group)), max_blocks_per_seq, window, partition_size, head_dim, &p))
        return (size_t)-1;
    return workspace_of(num_seqs, num_q_heads, head_dim, p.max_parts);
}

namespace pa {
namespace {

// The window that `rows` rows one after another have together.
int window_of(int window, int rows) { return window > 0 ? std::min(window, INT_MAX - rows) + rows - 1 : 0; }

// max_blocks: entries of a table's row; width: of them, those that contexts reach.
pa_status run_decode(void *out, const void *query, const void *key_cache, const void *value_cache, const int32_t *block_tables,
                     const int32_t *context_lens, const int32_t *query_start, const int4 *chunks, int num_seqs,
                     int num_query_tokens, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                     int max_blocks_per_seq, int width, int num_blocks, float scale, int window, int partition_size,
                     void *workspace, size_t workspace_bytes, int32_t *device_status, void *stream) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        block_size != kBlockSize || max_blocks_per_seq < 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize ||
        num_blocks <= 0 || window < 0 || !(scale == scale) ||
        (query_start == nullptr && chunks == nullptr && num_query_tokens != num_seqs))
        return PA_ERR_INVALID_ARG;
    const int group = num_q_heads / num_kv_heads, heads = heads_per_cta(group), splits = group / heads;
    Plan p;
    const int rows = chunks != nullptr ? kHeads / heads : 1;     // of a CTA at most
    if (!plan_of(num_seqs, num_kv_heads * splits, width, window_of(window, rows), partition_size, head_dim, &p))
        return PA_ERR_INVALID_ARG;
    if (!head_dim_ok(head_dim)) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_query_tokens == 0) return PA_OK;
    if (!out || !query || !key_cache || !value_cache || !context_lens || (!block_tables && max_blocks_per_seq > 0))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(query_start)) & 3u))
        return PA_ERR_INVALID_ARG;
    if ((int64_t)num_seqs * num_q_heads * rows * p.max_parts * p.cluster >= ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;
    const size_t need = workspace_of(num_seqs, num_q_heads * rows, head_dim, p.max_parts);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))) return PA_ERR_WORKSPACE;
    Fp4Args a = {};
    a.out = out;
    a.query = query;
    a.key_cache = static_cast<const uint8_t *>(key_cache);
    a.value_cache = static_cast<const uint8_t *>(value_cache);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.chunks = chunks;
    if (need > 0) {
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) +
                                               rows_bytes((int64_t)num_seqs * num_q_heads * rows * p.max_parts, head_dim));
    }
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.num_rows = num_query_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.heads = heads;
    a.cols = heads * rows;
    a.splits = splits;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.part_blocks = p.part_blocks;
    a.max_parts = p.max_parts;
    a.window = window;
    a.reach = window > 0 ? std::min(window, INT_MAX - kHeads) : INT_MAX - kHeads;    // (with a CTA's rows taken off it is an int)
    a.ordered = p.ordered;
    a.scale_log2 = scale * 1.4426950408889634f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return head_dim == 64 ? launch_all<64>(a, p, st) : head_dim == 128 ? launch_all<128>(a, p, st) : launch_all<256>(a, p, st);
}

}  // namespace

int decode_fp4_chunk_rows(int num_q_heads, int num_kv_heads) { return kHeads / heads_per_cta(num_q_heads / num_kv_heads); }

double decode_fp4_chunks_time(int num_chunks, int num_q_heads, int num_kv_heads, int head_dim, int width, int window,
                              size_t *workspace_bytes) {
    const int group = num_q_heads / num_kv_heads, heads = heads_per_cta(group), rows = kHeads / heads;
    Plan p;
    plan_of(num_chunks, num_kv_heads * (group / heads), width, window_of(window, rows), 0, head_dim, &p);
    *workspace_bytes = workspace_of(num_chunks, num_q_heads * rows, head_dim, p.max_parts);
    // and 4 us for the start and the end of each wave of CTAs, which the choice among cuts does not need
    return p.time + 4.0 * num_chunks * num_kv_heads * (group / heads) / (4.0 * device_sms());
}

pa_status decode_fp4_chunks(void *out, const void *query, const void *key_cache, const void *value_cache,
                            const int32_t *block_tables, const int32_t *chunk_lens, const int4 *chunks, int num_chunks,
                            int num_query_tokens, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                            int width, int num_blocks, float scale, int window, void *workspace, size_t workspace_bytes,
                            int32_t *device_status, void *stream) {
    return run_decode(out, query, key_cache, value_cache, block_tables, chunk_lens, nullptr, chunks, num_chunks,
                      num_query_tokens, num_q_heads, num_kv_heads, head_dim, kBlockSize, max_blocks_per_seq, width, num_blocks,
                      scale, window, 0, workspace, workspace_bytes, device_status, stream);
}

}  // namespace pa

extern "C" pa_status pa_decode_fp4(void *out, const void *query, const void *key_cache, const void *value_cache,
                                   const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start,
                                   int num_seqs, int num_query_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                   int block_size, int max_blocks_per_seq, int num_blocks, float scale, int window,
                                   int partition_size, void *workspace, size_t workspace_bytes, int32_t *device_status,
                                   void *stream) {
    return run_decode(out, query, key_cache, value_cache, block_tables, context_lens, query_start, nullptr, num_seqs,
                      num_query_tokens, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                      max_blocks_per_seq, num_blocks, scale, window, partition_size, workspace, workspace_bytes,
                      device_status, stream);
}
