// Paged decode attention over E4M3 pools with one scale per block of 16 tokens
// and KV head ("KV cache: la memoria de trabajo que sostiene la inferencia LLM",
// section "Trucos para que el cuaderno sea más fino": quantising the cache), one
// query token per sequence.  The mathematics of the scales is in pa_block8.cuh.
//
// One CTA handles one (sequence, KV head, partition).  Each warp owns every
// NW-th block of the partition and streams it through its own ring of STAGES
// slots: a block's K and V tiles are 16 rows x 128 codes = 2 KiB each, one TMA
// box (128-byte swizzle).  The group's query heads are the N columns of
// mma.sync m16n8k16 tiles in transposed form, S^T[16 tokens x 8 heads] = K Q^T
// and O^T[128 x 8 heads] += V^T P^T, so one pass over K/V serves the group; a
// group of more than 8 heads is split over CTAs that follow one another and
// find the tiles in L2.  Codes widen to f16 exactly.
//
// Few sequences: a context is cut into parts so that the GPU is full.  Up to
// eight parts form a thread-block cluster, cut each context evenly and merge
// through distributed shared memory, so that the call is one launch without
// scratch memory; more parts (or a partition size of the caller's) leave partials
// in the workspace for a second kernel.
//
// Bound by memory: 64 ragged contexts of up to 2048 tokens with 32 KV heads, 560 MB,
// 89 us (6.3 TB/s, 0.93 of a copy); 256 of up to 4096 with 64 query heads on 8, 1.24
// GB, 195 us (0.94); eight of 32768, 2.15 GB, 305 us (7.1 TB/s).  Four warps with
// rings of two blocks each were the best shape there: 4x3 6x2 6x3 8x1 8x2 3x2 2x2 2x3
// were up to 18 % slower on one of the three.  One short request is latency: 6 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "pa_block8.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kD = 128;
constexpr int kTileBytes = kBlockSize * kD;      // codes of one block of one KV head
constexpr int kStageBytes = 2 * kTileBytes;      // K and V
constexpr int kHeads = 8;                        // query heads of a CTA at most
// a head's reference maximum moves only when a block exceeds it by more than
// 2^8: the weights stay in [0, 256], which f16 holds
constexpr float kLazyLog2 = 8.f;

struct Block8Args {
    void *out;
    const void *query;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;  // sequence b's row is query_start[b]; nullptr: row b
    const float *k_scales;       // [num_blocks][num_kv_heads]
    const float *v_scales;
    float *part_o;               // [(b * Hq + h) * max_parts + part][128]
    float2 *part_ml;             // (reference, sum)
    int32_t *status;
    int num_seqs, num_rows, num_q_heads, num_kv_heads;
    int heads;                   // query heads of a CTA
    int splits;                  // CTAs of a (sequence, KV head, partition)
    int max_blocks, num_blocks;
    int part_blocks, max_parts;
    int window;
    float scale_log2;
};

// A block of the partition as the warps read it: where its tiles are, and its scales.
struct __align__(16) Entry {
    int row;                     // first pool row of the block's tile of this KV head
    float ck;                    // key scale * softmax scale * log2(e)
    float lv;                    // log2 of the value scale
    float rv;                    // 1 / value scale
};

struct Span {
    int L, start, blk0, nblk, nparts;
};

// Blocks of a context of `len` tokens: [*first, *blocks), the first position
// attended in *start; *L the length, clamped.
__device__ __forceinline__ void range_of(const Block8Args &a, int len, bool say, int *L, int *start, int *first,
                                         int *blocks) {
    const int lmax = a.max_blocks * kBlockSize;
    if (len < 0 || len > lmax) {
        if (say) report(a.status, PA_DEV_BAD_CONTEXT_LEN);
        len = len < 0 ? 0 : lmax;
    }
    *L = len;
    *start = a.window > 0 && len > a.window ? len - a.window : 0;
    *first = *start / kBlockSize;
    *blocks = (len + kBlockSize - 1) / kBlockSize;
}

// Part `part` of `parts` of a context, cut evenly.
__device__ __forceinline__ void even_span(const Block8Args &a, int len, int part, int parts, bool say, Span &w) {
    int first, blocks;
    range_of(a, len, say, &w.L, &w.start, &first, &blocks);
    const int n = max(blocks - first, 0);
    w.blk0 = first + (int)((int64_t)part * n / parts);
    w.nblk = first + (int)((int64_t)(part + 1) * n / parts) - w.blk0;
    w.nparts = 1;
}

// Partition `part` of a context of `len` tokens; false when it lies past the end.
__device__ __forceinline__ bool span_of(const Block8Args &a, int len, int part, bool say, Span &w) {
    int first, blocks;
    range_of(a, len, say, &w.L, &w.start, &first, &blocks);
    w.nparts = blocks <= first ? 1 : (blocks - first + a.part_blocks - 1) / a.part_blocks;
    if (part >= w.nparts) return false;
    w.blk0 = first + part * a.part_blocks;
    w.nblk = max(min(w.blk0 + a.part_blocks, blocks) - w.blk0, 0);
    return true;
}

// The row of query and output that is sequence b's, or -1: it brings none, or more
// than the one that a decode step has.
__device__ __forceinline__ int row_of(const Block8Args &a, int b, bool say) {
    if (a.query_start == nullptr) return b;
    const int at = a.query_start[b], end = a.query_start[b + 1];
    if (end == at) return -1;
    const bool outside = at < 0 || end < at || end > a.num_rows;
    if (!outside && end == at + 1) return at;
    if (say) report(a.status, outside ? PA_DEV_BAD_CONTEXT_LEN : PA_DEV_BAD_QUERY_LEN);
    return -1;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
// byte offset of code `col` of tile row `row` (128-byte swizzle)
__device__ __forceinline__ uint32_t code_at(int row, int col) {
    return (uint32_t)(row * 128 + (((col >> 4) ^ (row & 7)) << 4) + (col & 15));
}

// One warp's attention state over its blocks: 8 query heads (columns; those
// past the group have a zero query and are not stored).  Lane (g, t) = (lane /
// 4, lane % 4) holds scores of tokens g and g + 8 for heads 2t and 2t + 1.
//  * S^T: the contraction may visit the head dimension in any order as long as
//    K and Q agree, so a lane reads 8 consecutive codes of rows g and g + 8 and
//    the query's fragments are laid out to match.
//  * O^T: the A operand needs two tokens of one head-dim element in a register,
//    so a lane reads 4 codes of rows 2t, 2t + 1, 2t + 8, 2t + 9 and pairs them
//    with byte permutes; m-tile 2c + j holds elements 32c + 4g + 2j (row g) and
//    + 1 (row g + 8).
struct Warp8 {
    uint32_t qb[8][2];
    float o[8][4];
    float m0, m1, l0, l1;
    float qs0, qs1;              // powers of two of heads 2t and 2t + 1: what their scores are multiplied by
    int lane, g, t;
    uint32_t koff[4], voff_a[4], voff_b[4];

    // This lane's part of the query: elements 32 c + 8 t .. + 7 of row g.
    __device__ __forceinline__ void load(const Block8Args &a, int row, int first_head, int lane_, uint4 (&w)[4]) {
        lane = lane_;
        g = lane >> 2;
        t = lane & 3;
        const uint4 *q = reinterpret_cast<const uint4 *>(
            static_cast<const __nv_bfloat16 *>(a.query) + ((int64_t)row * a.num_q_heads + first_head + g) * kD);
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = g < a.heads ? q[4 * c + t] : make_uint4(0u, 0u, 0u, 0u);
    }

    __device__ __forceinline__ void init(const Block8Args &a, const uint4 (&w)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            koff[c] = code_at(g, 32 * c + 8 * t);
            voff_a[c] = code_at(2 * t, 32 * c + 4 * g);
            voff_b[c] = code_at(2 * t + 1, 32 * c + 4 * g);
        }
        uint32_t amax = 0;                               // as bits: magnitudes compare like integers
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (uint32_t x : {w[c].x, w[c].y, w[c].z, w[c].w})
                amax = max(amax, max((x << 16) & 0x7fffffffu, x & 0x7fff0000u));
        if (amax >= 0x47800000u) {                       // 65536 or more: looked at again, as NaN is none of them
            bool beyond = false;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                beyond |= bf16x2_beyond_f16(w[c].x) | bf16x2_beyond_f16(w[c].y) | bf16x2_beyond_f16(w[c].z) | bf16x2_beyond_f16(w[c].w);
            if (beyond) report(a.status, PA_DEV_RANGE);  // the f16 query is not the query
        }
        amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = max(amax, __shfl_xor_sync(kFull, amax, 2));
        // A row is brought up by a power of two so that its largest magnitude lies in
        // [2^14, 2^15): f16 then holds every element exactly but those below 2^-29 of it,
        // which are off by at most 2^-39 of it.
        const int up = min(max(14 + 127 - (int)(amax >> 23), 0), 126);
        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
        const int down = (127 - up) << 23;               // 2^-up, of row g
        qs0 = __int_as_float(__shfl_sync(kFull, down, 8 * t));
        qs1 = __int_as_float(__shfl_sync(kFull, down, 8 * t + 4));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            qb[2 * c][0] = pack_f16x2(bf16lo(w[c].x) * f, bf16hi(w[c].x) * f);
            qb[2 * c][1] = pack_f16x2(bf16lo(w[c].y) * f, bf16hi(w[c].y) * f);
            qb[2 * c + 1][0] = pack_f16x2(bf16lo(w[c].z) * f, bf16hi(w[c].z) * f);
            qb[2 * c + 1][1] = pack_f16x2(bf16lo(w[c].w) * f, bf16hi(w[c].w) * f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
    }

    // One block, of which the rows [nlo, nvalid) are attended (at least one).
    __device__ __forceinline__ void block(uint32_t ktile, uint32_t vtile, int nlo, int nvalid, const Entry &e) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint2 r0 = lds64(ktile + koff[c]);
            const uint2 r1 = lds64(ktile + koff[c] + 1024);      // row g + 8: same swizzle phase
            uint32_t x[4];
            e4m3x4_to_f16x2x2(r0.x, x[0], x[2]);
            e4m3x4_to_f16x2x2(r1.x, x[1], x[3]);
            mma_f16_16816(s, x, qb[2 * c][0], qb[2 * c][1]);
            e4m3x4_to_f16x2x2(r0.y, x[0], x[2]);
            e4m3x4_to_f16x2x2(r1.y, x[1], x[3]);
            mma_f16_16816(s, x, qb[2 * c + 1][0], qb[2 * c + 1][1]);
        }
        const bool v0 = g >= nlo && g < nvalid, v1 = g + 8 >= nlo && g + 8 < nvalid;
        const float ck0 = e.ck * qs0, ck1 = e.ck * qs1;
        s[0] = v0 ? fmaf(s[0], ck0, e.lv) : -INFINITY;
        s[1] = v0 ? fmaf(s[1], ck1, e.lv) : -INFINITY;
        s[2] = v1 ? fmaf(s[2], ck0, e.lv) : -INFINITY;
        s[3] = v1 ? fmaf(s[3], ck1, e.lv) : -INFINITY;
        float mx0 = fmaxf(s[0], s[2]), mx1 = fmaxf(s[1], s[3]);
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, k));
            mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, k));
        }
        const bool need0 = mx0 > m0 + kLazyLog2, need1 = mx1 > m1 + kLazyLog2;
        if (__any_sync(kFull, need0 || need1)) {
            const float a0 = need0 ? exp2f(m0 - mx0) : 1.f;      // 0 while m0 is -inf
            const float a1 = need1 ? exp2f(m1 - mx1) : 1.f;
            m0 = need0 ? mx0 : m0;
            m1 = need1 ? mx1 : m1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i][0] *= a0;
                o[i][1] *= a1;
                o[i][2] *= a0;
                o[i][3] *= a1;
            }
        }
        const float w0 = ex2_fast(s[0] - m0), w1 = ex2_fast(s[1] - m1);
        const float w2 = ex2_fast(s[2] - m0), w3 = ex2_fast(s[3] - m1);
        l0 = fmaf(w0 + w2, e.rv, l0);
        l1 = fmaf(w1 + w3, e.rv, l1);
        // the weights enter the second product as f16, rounded once: 11 bits
        // move an output by at most 2^-11 of the largest value it weighs, where
        // bf16's 8 bits would be as coarse as the output's own rounding
        const uint32_t b0 = movmatrix_trans(pack_f16x2(w0, w1));
        const uint32_t b1 = movmatrix_trans(pack_f16x2(w2, w3));
        if (nlo > 0 || nvalid < kBlockSize) zero_rows(vtile, nlo, nvalid);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t wa = lds32(vtile + voff_a[c]), wb = lds32(vtile + voff_b[c]);
            const uint32_t wc = lds32(vtile + voff_a[c] + 1024), wd = lds32(vtile + voff_b[c] + 1024);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t sel = j == 0 ? 0x5140u : 0x7362u;
                uint32_t x[4];
                e4m3x4_to_f16x2x2(__byte_perm(wa, wb, sel), x[0], x[1]);     // tokens 2t, 2t + 1
                e4m3x4_to_f16x2x2(__byte_perm(wc, wd, sel), x[2], x[3]);     // tokens 2t + 8, 2t + 9
                mma_f16_16816(o[2 * c + j], x, b0, b1);
            }
        }
    }

    // Rows that are not attended may hold any code, NaN among them, and would
    // reach the sum as 0 * NaN.
    __device__ __forceinline__ void zero_rows(uint32_t tile, int nlo, int nvalid) {
        for (int i = lane; i < (kBlockSize - (nvalid - nlo)) * 8; i += 32) {
            int r = i / 8;
            r = r < nlo ? r : r - nlo + nvalid;
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(tile + (uint32_t)(r * 128 + (i % 8) * 16)),
                         "r"(0u)
                         : "memory");
        }
        __syncwarp();
    }

    // The state as acc[heads][128], m[heads], l[heads].
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
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float2 *>(acc + h * kD + 32 * (i >> 1) + 4 * g + 2 * (i & 1)) =
                    make_float2(o[i][e], o[i][2 + e]);
            if (g == 0) {
                m[h] = e ? m1 : m0;
                l[h] = e ? l1 : l0;
            }
        }
    }
};

template <int NW, int STAGES>
struct Shape {
    static constexpr int kRing = NW * STAGES * kStageBytes;
    static_assert(STAGES * kStageBytes >= kHeads * kD * 4, "a warp's state is merged over its ring");
    static size_t smem(int part_blocks) {
        return 1024 + kRing + (size_t)part_blocks * sizeof(Entry) + NW * STAGES * 8 + 2 * NW * kHeads * sizeof(float);
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
// (121 registers without clusters, four CTAs of four warps per SM; held to 96 for a fifth, by
// a launch bound or otherwise, the 70B-shaped batch took 200 to 204 us instead of 193.)
template <int NW, int STAGES, int kParts>
__global__ void __launch_bounds__(NW * 32)
    pa_decode_block8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                            const Block8Args a) {
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
    const int b = idx / axis;
    idx -= b * axis;
    const int kvh = idx / a.splits;
    const int first_head = kvh * a.heads * a.splits + (idx - kvh * a.splits) * a.heads;
    // What depends on the CTA's place alone is loaded together, so that a CTA
    // waits one memory round trip before its first tile is requested: the length,
    // the table entries of the warp's first blocks (a window moves the partition
    // with the length; then the table follows it) and the query.  The scales,
    // which follow the table, arrive while the first tiles do.  All of it is the
    // warp's own business: no barrier before the merge.
    const int len = a.context_lens[b];
    const int32_t *row_table = a.block_tables + (int64_t)b * a.max_blocks;
    const bool early = kParts == 1 && a.window == 0;     // the partition does not move with the length
    const int ahead = part * a.part_blocks + warp + NW * lane;
    int first_phys = early && warp + NW * lane < a.part_blocks && ahead < a.max_blocks ? row_table[ahead] : -1;
    const bool say = threadIdx.x == 0 && part == 0 && idx == 0;
    const int row = row_of(a, b, say);
    if (row < 0) return;                                 // (a cluster's CTAs all leave)
    Warp8 state;
    uint4 query[4];
    state.load(a, row, first_head, lane, query);
    Span w;
    if constexpr (kParts > 1) even_span(a, len, part, kParts, say, w);
    else if (!span_of(a, len, part, say, w)) return;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Entry *entries = reinterpret_cast<Entry *>(ring + Shape<NW, STAGES>::kRing);
    uint64_t *bars = reinterpret_cast<uint64_t *>(entries + a.part_blocks);
    float *s_m = reinterpret_cast<float *>(bars + NW * STAGES);
    float *s_l = s_m + NW * kHeads;
    __shared__ int s_fail[NW];
    const int count = w.nblk > warp ? (w.nblk - warp + NW - 1) / NW : 0;
    uint64_t *my_bars = bars + warp * STAGES;
    uint8_t *my_ring = ring + warp * STAGES * kStageBytes;
    if (lane == 0) {
        s_fail[warp] = 0;
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
#pragma unroll
        for (int s = 0; s < STAGES; ++s) mbar_init(&my_bars[s], 1);
        fence_mbar_init();
    }
    auto entry_of = [&](int phys) {
        if ((unsigned)phys >= (unsigned)a.num_blocks) {
            report(a.status, PA_DEV_BAD_BLOCK_ID);
            phys = 0;
        }
        return (int64_t)phys * a.num_kv_heads + kvh;
    };
    const int32_t *table = row_table + w.blk0 + warp;
    if (!early) first_phys = lane < count ? table[NW * lane] : -1;
    const int64_t first_at = lane < count ? entry_of(first_phys) : 0;
    const int first_row = (int)(first_at * kBlockSize);

    const uint64_t policy = l2_policy_evict_first();     // tiles are read once: they leave L2 first
    auto issue_row = [&](int it, int pool_row) {
        const int s = it % STAGES;
        uint8_t *kt = my_ring + s * kStageBytes;
        mbar_arrive_expect_tx(&my_bars[s], kStageBytes);
        tma_load_2d_hint(kt, &kmap, 0, pool_row, &my_bars[s], policy);
        tma_load_2d_hint(kt + kTileBytes, &vmap, 0, pool_row, &my_bars[s], policy);
    };
    auto issue = [&](int it) { issue_row(it, entries[warp + it * NW].row); };
#pragma unroll
    for (int it = 0; it < STAGES; ++it) {
        const int at = __shfl_sync(kFull, first_row, it);
        if (lane == 0 && it < count) issue_row(it, at);
    }
    state.init(a, query);                                // under the tiles' latency
    for (int k = lane; k < count; k += 32) {
        const int64_t at = k == lane ? first_at : entry_of(table[NW * k]);
        const float sv = value_scale(a.v_scales[at], a.status);
        entries[warp + k * NW] = Entry{(int)(at * kBlockSize), a.k_scales[at] * a.scale_log2, log2_scale(sv), 1.f / sv};
    }
    __syncwarp();
    bool ok = true;
    int it = 0;
    for (; it < count; ++it) {
        const int s = it % STAGES;
        if (!__all_sync(kFull, mbar_wait_bounded(&my_bars[s], (it / STAGES) & 1))) {
            ok = false;
            break;
        }
        const int tok = (w.blk0 + warp + it * NW) * kBlockSize;
        const uint32_t kt = smem_u32(my_ring + s * kStageBytes);
        state.block(kt, kt + kTileBytes, max(0, w.start - tok), min(kBlockSize, w.L - tok), entries[warp + it * NW]);
        __syncwarp();
        if (lane == 0 && it + STAGES < count) {
            fence_proxy_async_smem();
            issue(it + STAGES);
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
    state.finish(a.heads, acc, s_m + warp * kHeads, s_l + warp * kHeads);
    __syncthreads();
    bool failed = false;
#pragma unroll
    for (int k = 0; k < NW; ++k) failed |= s_fail[k] != 0;
    auto merged = [&](int i, float &M, float &sum) {     // element i of the CTA's state
        const int h = i / kD;
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
            O = fmaf(f, reinterpret_cast<const float *>(ring + k * STAGES * kStageBytes)[i], O);
        }
        // after a wait that gave up the row is NaN, through its partial sums too: what an earlier
        // call left in the workspace must not pass for an output
        if (failed) sum = __int_as_float(0x7fffffff);
        return O;
    };
    const int64_t head0 = (int64_t)b * a.num_q_heads + first_head;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)row * a.num_q_heads + first_head) * kD;
    if constexpr (kParts > 1) {
        // The parts' states side by side in the cluster's shared memory: each CTA
        // merges its share of the elements.  A part that gave up keeps its place at
        // the barriers; its sum makes the row NaN.
        constexpr int kEach = kHeads * kD / (NW * 32);
        float O[kEach], M[kEach], sum[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = threadIdx.x + e * NW * 32;
            if (i < a.heads * kD) O[e] = merged(i, M[e], sum[e]);
        }
        __syncthreads();                                 // the warps' states are read
        float *state_o = reinterpret_cast<float *>(ring), *state_m = s_m, *state_l = s_l;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = threadIdx.x + e * NW * 32;
            if (i >= a.heads * kD) continue;
            state_o[i] = O[e];
            if (i % kD == 0) {
                state_m[i / kD] = M[e];
                state_l[i / kD] = sum[e];
            }
        }
        cluster_sync();
        for (int i = (int)threadIdx.x + part * NW * 32; i < a.heads * kD; i += kParts * NW * 32) {
            const int h = i / kD;
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
            out[i] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
        }
        cluster_sync();                                  // no CTA leaves while its state is read
    } else {
        const bool whole = w.nparts == 1;
        for (int i = threadIdx.x; i < a.heads * kD; i += NW * 32) {
            float M, sum;
            const float O = merged(i, M, sum);
            if (whole) {
                // a NaN sum stays NaN; an empty context gives zeros
                out[i] = __float2bfloat16_rn(sum == 0.f ? 0.f : O / sum);
            } else {
                const int64_t at = (head0 + i / kD) * a.max_parts + part;
                a.part_o[at * kD + i % kD] = O;
                if (i % kD == 0) a.part_ml[at] = make_float2(M, sum);
            }
        }
    }
}

// Merges the partitions of a (sequence, query head) row, one CTA a row: warp w
// takes partials w, w + kMergeWarps, ..., a lane four of the 128 columns, four
// partials on their way at a time; the warps' sums meet in shared memory.  (One
// warp a row took 16 us for the 128 partials of one 32768-token context.)
constexpr int kMergeWarps = 4;
__global__ void __launch_bounds__(32 * kMergeWarps) pa_merge_block8_kernel(const Block8Args a) {
    __shared__ float4 s_acc[kMergeWarps][32];
    __shared__ float s_sum[kMergeWarps], s_max[kMergeWarps];
    grid_dependency_wait();
    grid_dependents_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    Span w;
    const int b = (int)(row / a.num_q_heads), out_row = row_of(a, b, false);
    span_of(a, a.context_lens[b], 0, false, w);
    if (w.nparts <= 1 || out_row < 0) return;
    const float2 *ml = a.part_ml + row * a.max_parts;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + row * a.max_parts * kD);
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = warp; p0 < w.nparts; p0 += 4 * kMergeWarps) {
        float4 v[4];
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + i * kMergeWarps;
            v[i] = p < w.nparts ? po[(int64_t)p * 32 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
            x[i] = p < w.nparts ? ml[p] : make_float2(-INFINITY, 0.f);
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, x[i].x);
        const float g = M == -INFINITY ? 0.f : exp2f(M - top);
        M = top;
        sum *= g;
        acc = make_float4(acc.x * g, acc.y * g, acc.z * g, acc.w * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = x[i].x == -INFINITY ? 0.f : exp2f(x[i].x - M);
            sum = fmaf(f, x[i].y, sum);
            acc.x = fmaf(f, v[i].x, acc.x);
            acc.y = fmaf(f, v[i].y, acc.y);
            acc.z = fmaf(f, v[i].z, acc.z);
            acc.w = fmaf(f, v[i].w, acc.w);
        }
    }
    s_acc[warp][lane] = acc;
    if (lane == 0) {
        s_sum[warp] = sum;
        s_max[warp] = M;
    }
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) top = fmaxf(top, s_max[k]);
    sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) {
        const float f = s_max[k] == -INFINITY ? 0.f : exp2f(s_max[k] - top);
        const float4 v = s_acc[k][lane];
        sum = fmaf(f, s_sum[k], sum);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t out_head = (int64_t)out_row * a.num_q_heads + (row - (int64_t)b * a.num_q_heads);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + out_head * kD + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
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
    bool narrow;                 // CTAs of one warp
};

// How contexts are cut.  partition_size 0: parts enough for four CTAs per SM
// (sequences are ragged, and a CTA's start and end overlap others' streaming),
// none of fewer than 8 blocks, nor of more than 128, or 256 where there are CTAs
// enough (70B-shaped batch 196 us whole, 207 in halves; eight 32768-token
// contexts 303 us in 2048-token parts, 324 in 4096, 462 in 16384).  With more than
// one CTA per SM from the sequences alone, parts have 40 blocks at least, and a
// number of CTAs that is short of four by an eighth is left (256 CTAs on 512 tokens
// 9.6 us whole, 15.0 in 4 parts, on 2048 25.8 / 22.5 in 3; 320 CTAs on 512 10.9 /
// 13.3 in 2, on 2048 27.5 / 26.8; 592 CTAs on 512 15.3 / 20.7, on 2048 39.9 / 43.5).
// The parts follow the table's width, as only the GPU knows the lengths, and a wide
// table's last parts are often empty: a grid beyond 32 CTAs per SM is made of the
// largest parts only (tables of 8192 entries: 64 7B-shaped contexts 97 us, 89 with tables
// of their size; 1024 contexts of up to 64 tokens with 8 KV heads 126 / 24; 8 of 2048 with 8
// KV heads 23.5 / 15.7; in 4096-token parts the first two took 178 and 621 when this
// form took 106 and 267).  Parts cut by each context's own length, or taken in
// stretches by a loop in the kernel, cost 5 to 12 % where the table fits.
// Up to 8 parts of a small call are clusters: the GPU time is the same, the host
// issues one launch instead of two (5 us, 8 otherwise); in larger calls clusters
// lose (32 ragged sequences 28.6 us, 26.5 with a merge kernel).
//
// Where there are more than five CTAs per SM (which holds four of four warps) and their
// parts short, CTAs have one warp, 16 of which an SM holds: a short part's time is
// its start (length, table, scales, first tiles one after another) and its end.
// Contexts between half of and all of 64 tokens: 960 CTAs 5.7 us against 7.5, 8192 24 / 48; of
// 256: 720 CTAs 13.5 / 12.9, 960 14.1 / 14.7, 2048 22.5 / 25.7, 8192 69 / 83; of 384: 960
// 18.8 / 18.2, 2048 31.0 / 31.8, 8192 99 / 104; 2048 CTAs on 512 tokens 39.6 / 38.6, on 768 57 / 53.
bool plan_of(int num_seqs, int axis, int max_blocks, int window, int partition_size, Plan *p) {
    if (partition_size != 0 && (partition_size < kBlockSize || partition_size > kMaxPartition || partition_size % kBlockSize))
        return false;
    int span = max_blocks;
    if (window > 0) span = std::min(span, (window - 1) / kBlockSize + 2);
    p->cluster = 1;
    p->narrow = false;
    const int64_t ctas = std::max<int64_t>(1, (int64_t)num_seqs * axis), target = 4LL * device_sms();
    if (partition_size != 0) {
        p->part_blocks = partition_size / kBlockSize;
    } else {
        const int most = ctas >= target ? 256 : 128;
        int64_t parts = std::max<int64_t>((target - ctas / 8 + ctas - 1) / ctas, (span + most - 1) / most);
        parts = std::max<int64_t>(1, std::min<int64_t>(parts, 4 * ctas > target ? span / 40 : (span + 7) / 8));
        const int cluster = parts <= 2 ? 2 : parts <= 4 ? 4 : 8;
        if (parts > 1 && parts <= 8 && ctas * cluster <= target) {
            p->cluster = cluster;
            p->max_parts = 1;
            p->part_blocks = (span + p->cluster - 1) / p->cluster + 1;
            return true;
        }
        const int largest = kMaxPartition / kBlockSize;
        parts = std::min(parts, std::max<int64_t>(std::max<int64_t>((target + ctas - 1) / ctas, 8 * target / ctas),
                                                  (span + largest - 1) / largest));
        p->part_blocks = std::max(1, (int)((span + parts - 1) / parts));
    }
    p->max_parts = std::max(1, (span + p->part_blocks - 1) / p->part_blocks);
    const int64_t all = ctas * p->max_parts;
    p->narrow = p->part_blocks <= (all > 10LL * device_sms() ? 24 : all > 5LL * device_sms() ? 16 : 0);
    return true;
}

size_t rows_bytes(int64_t rows) { return ((size_t)rows * kD * sizeof(float) + 255) & ~size_t(255); }

size_t workspace_of(int num_seqs, int num_q_heads, int max_parts) {
    if (max_parts <= 1) return 0;
    const int64_t rows = (int64_t)num_seqs * num_q_heads * max_parts;
    return rows_bytes(rows) + (size_t)rows * sizeof(float2);
}

template <int NW, int STAGES, int kParts>
pa_status launch_decode(const Block8Args &a, const void *kc, const void *vc, int64_t rows, cudaStream_t st) {
    CUtensorMap kmap, vmap;
    if (!encode_block8_map(&kmap, kc, rows, true) || !encode_block8_map(&vmap, vc, rows, true))
        return cuda_failure(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
    const size_t smem = Shape<NW, STAGES>::smem(a.part_blocks);
    auto kernel = pa_decode_block8_kernel<NW, STAGES, kParts>;
    cudaError_t e = allow_smem(kernel, Shape<NW, STAGES>::smem(kMaxPartition / kBlockSize));
    if (e != cudaSuccess) return cuda_failure(e, "cudaFuncSetAttribute(block-scaled decode)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.num_seqs * a.num_kv_heads * a.splits * a.max_parts * kParts));
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kParts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kParts > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, kmap, vmap, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_decode_block8_kernel launch");
    count_launches(1);
    return PA_OK;
}

}  // namespace

bool encode_block8_map(CUtensorMap *map, const void *pool, int64_t rows, bool swizzled) {
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
    cuuint64_t dims[2] = {kD, (cuuint64_t)rows};
    cuuint64_t strides[1] = {kD};
    cuuint32_t box[2] = {kD, kBlockSize};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(pool), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_block_fp8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                                      int max_blocks_per_seq, int block_size, int window,
                                                      int partition_size) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || head_dim != kD ||
        max_blocks_per_seq < 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize || block_size != kBlockSize || window < 0)
        return (size_t)-1;
    const int group = num_q_heads / num_kv_heads;
    Plan p;
    if (!plan_of(num_seqs, num_kv_heads * (group / heads_per_cta(group)), max_blocks_per_seq, window, partition_size, &p))
        return (size_t)-1;
    return workspace_of(num_seqs, num_q_heads, p.max_parts);
}

extern "C" pa_status pa_decode_block_fp8_rows(void *out, const void *query, const void *key_cache, const void *value_cache,
                                              const float *k_scales, const float *v_scales, const int32_t *block_tables,
                                              const int32_t *context_lens, const int32_t *query_start, int num_seqs,
                                              int num_query_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                              int block_size, int max_blocks_per_seq, int num_blocks, float scale,
                                              int window, int partition_size, void *workspace, size_t workspace_bytes,
                                              int32_t *device_status, void *stream) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        block_size != kBlockSize || max_blocks_per_seq < 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize ||
        num_blocks <= 0 || window < 0 || !(scale == scale) || (query_start == nullptr && num_query_tokens != num_seqs))
        return PA_ERR_INVALID_ARG;
    const int group = num_q_heads / num_kv_heads, heads = heads_per_cta(group), splits = group / heads;
    Plan p;
    if (!plan_of(num_seqs, num_kv_heads * splits, max_blocks_per_seq, window, partition_size, &p))
        return PA_ERR_INVALID_ARG;
    if (head_dim != kD) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_query_tokens == 0) return PA_OK;
    if (!out || !query || !key_cache || !value_cache || !k_scales || !v_scales || !context_lens ||
        (!block_tables && max_blocks_per_seq > 0))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales) |
          reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(query_start)) & 3u))
        return PA_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)num_blocks * num_kv_heads * kBlockSize;
    if (rows >= ((int64_t)1 << 31) ||
        (int64_t)num_seqs * num_q_heads * p.max_parts * p.cluster >= ((int64_t)1 << 31))
        return PA_ERR_UNSUPPORTED;
    const size_t need = workspace_of(num_seqs, num_q_heads, p.max_parts);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))) return PA_ERR_WORKSPACE;
    Block8Args a = {};
    a.out = out;
    a.query = query;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.num_rows = num_query_tokens;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    if (need > 0) {
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) +
                                               rows_bytes((int64_t)num_seqs * num_q_heads * p.max_parts));
    }
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.heads = heads;
    a.splits = splits;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.part_blocks = p.part_blocks;
    a.max_parts = p.max_parts;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto launch = p.cluster == 1   ? p.narrow ? launch_decode<1, 3, 1> : launch_decode<4, 2, 1>
                        : p.cluster == 2 ? launch_decode<4, 2, 2>
                        : p.cluster == 4 ? launch_decode<4, 2, 4>
                                         : launch_decode<4, 2, 8>;
    pa_status s = launch(a, key_cache, value_cache, rows, st);
    if (s != PA_OK || p.max_parts <= 1) return s;
    cudaError_t e = launch_chained(pa_merge_block8_kernel, dim3((unsigned)(num_seqs * num_q_heads)),
                                   dim3(32 * kMergeWarps), 0, st, a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_merge_block8_kernel launch");
    count_launches(1);
    return PA_OK;
}

extern "C" pa_status pa_decode_block_fp8(void *out, const void *query, const void *key_cache, const void *value_cache,
                                         const float *k_scales, const float *v_scales, const int32_t *block_tables,
                                         const int32_t *context_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                                         int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                                         float scale, int window, int partition_size, void *workspace,
                                         size_t workspace_bytes, int32_t *device_status, void *stream) {
    return pa_decode_block_fp8_rows(out, query, key_cache, value_cache, k_scales, v_scales, block_tables, context_lens,
                                    nullptr, num_seqs, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                    max_blocks_per_seq, num_blocks, scale, window, partition_size, workspace,
                                    workspace_bytes, device_status, stream);
}
