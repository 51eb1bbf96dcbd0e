// The bookkeeping of one serving step on the GPU: block tables, slots and
// positions of the step's tokens from the request lengths ("PagedAttention por
// dentro: bloques, tabla de páginas, evicción y el estado del arte del KV cache
// en 2026", section "La tabla de páginas (block table)": a sequence holding N
// tokens writes the next one into its last block while N mod 16 != 0, else into
// a block taken from the pool).
//
// With L_b tokens held and T_b new ones, sequence b takes
//   need_b = ceil((L_b + T_b) / 16) - ceil(L_b / 16)
// blocks.  The sequences are served in order; b is served while the running
// sums of need and T stay within the free blocks and the token capacity, so the
// served ones are a prefix of the batch (apart from sequences that bring
// nothing).  The sum of need before b is where b's blocks begin in the free
// stack, the sum of T before b where its tokens begin in the flat list.
//
// One launch, no scratch memory: the two running sums are cheap (8 bytes per
// sequence, from L2), so every CTA computes them for itself, kSeqs sequences at
// a time, and then writes its own range of tokens, finding a token's sequence
// by bisection among the kSeqs ends in shared memory.  A new block's table
// entry is written by the thread of its first token.  The sequences' outputs
// are written by one CTA for each group of kSeqs.
//
// Latency: 64 sequences of one token 3.0 us, an empty launch's 2 to 3; 4096 sequences
// with 109 thousand tokens 7.1 us (1.4 MB), most of it the sums, which every CTA goes
// through once.
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kPlanItems = 4;                       // sequences per thread and round

struct PlanArgs {
    int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *new_lens;
    const int32_t *free_blocks;
    const int32_t *num_free;
    int32_t *context_lens_out;
    int32_t *query_start;
    int64_t *slot_mapping;
    int32_t *positions;
    int32_t *num_free_out;
    int32_t *status;
    int num_seqs;
    int max_blocks;
    int num_blocks;
    int free_capacity;
    int token_capacity;
    int tokens_per_cta;
};

__device__ __forceinline__ int blocks_of(int tokens) {
    return (int)(((unsigned)tokens + (kBlockSize - 1)) / kBlockSize);
}

// kPlanThreads: 256 where one round of 1024 sequences holds the batch (64
// sequences 3.1 us, 4.1 with 512), else 512 (4096 sequences 7.5 us, 8.8 with 256).
template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) pa_plan_step_kernel(const PlanArgs a) {
    constexpr int kSeqs = kPlanThreads * kPlanItems, kPlanWarps = kPlanThreads / 32;
    // ends, first blocks and held tokens of the round's sequences; one that is not
    // served ends nowhere
    __shared__ int s_end[kSeqs], s_off[kSeqs], s_len[kSeqs];
    __shared__ int64_t s_warp[2][kPlanWarps];
    __shared__ int s_total[2], s_used[2];           // alternate between rounds
    grid_dependency_wait();
    grid_dependents_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool last = blockIdx.x + 1 == gridDim.x;  // goes through every round, and reports
    int free = *a.num_free;
    if (free < 0 || free > a.free_capacity) {
        if (last && tid == 0) report(a.status, PA_DEV_BAD_BLOCK_ID);
        free = free < 0 ? 0 : a.free_capacity;
    }
    const int t_lo = (int)min((int64_t)a.token_capacity, (int64_t)blockIdx.x * a.tokens_per_cta);
    const int t_hi = (int)min((int64_t)a.token_capacity, (int64_t)t_lo + a.tokens_per_cta);
    int64_t carry_need = 0, carry_new = 0;          // sums over the rounds before, served or not
    int total = 0, used = 0;                        // tokens and blocks of the served sequences
    if (tid < 2) s_total[tid] = s_used[tid] = 0;
    if (blockIdx.x == 0 && tid == 0) a.query_start[0] = 0;
    __syncthreads();
    int round = 0;
    // a round's lengths are loaded while the round before is worked on
    int next_len[kPlanItems], next_add[kPlanItems];
    static_assert(kPlanItems == 4, "one 16-byte load");
    const bool vec = ((reinterpret_cast<uintptr_t>(a.context_lens) | reinterpret_cast<uintptr_t>(a.new_lens)) & 15u) == 0;
    auto fetch = [&](int64_t base) {
        const int64_t b0 = base + tid * kPlanItems;
        if (vec && b0 + kPlanItems <= a.num_seqs) {
            const int4 x = *reinterpret_cast<const int4 *>(a.context_lens + b0);
            const int4 y = *reinterpret_cast<const int4 *>(a.new_lens + b0);
            next_len[0] = x.x, next_len[1] = x.y, next_len[2] = x.z, next_len[3] = x.w;
            next_add[0] = y.x, next_add[1] = y.y, next_add[2] = y.z, next_add[3] = y.w;
            return;
        }
#pragma unroll
        for (int j = 0; j < kPlanItems; ++j) {
            next_len[j] = b0 + j < a.num_seqs ? a.context_lens[b0 + j] : 0;
            next_add[j] = b0 + j < a.num_seqs ? a.new_lens[b0 + j] : 0;
        }
    };
    fetch(0);
    for (int64_t base = 0; base < a.num_seqs; base += kSeqs, ++round) {
        // a CTA whose tokens are written and that has no later round's sequences to
        // write is done (the last one counts the free blocks that are left)
        if (t_hi <= total && !last && (unsigned)round > blockIdx.x) return;
        int len[kPlanItems], add[kPlanItems], need[kPlanItems];
        int64_t sum_need = 0, sum_new = 0;
#pragma unroll
        for (int j = 0; j < kPlanItems; ++j) {
            len[j] = next_len[j];
            add[j] = next_add[j];
        }
        fetch(base + kSeqs);
#pragma unroll
        for (int j = 0; j < kPlanItems; ++j) {
            if (len[j] < 0 || add[j] < 0 ||
                (int64_t)len[j] + add[j] > (int64_t)a.max_blocks * kBlockSize) {
                if (last) report(a.status, PA_DEV_BAD_CONTEXT_LEN);
                add[j] = 0;
            }
            need[j] = add[j] > 0 ? blocks_of(len[j] + add[j]) - blocks_of(len[j]) : 0;
            sum_need += need[j];
            sum_new += add[j];
        }
        // exclusive sums over the round's threads
        int64_t at_need = sum_need, at_new = sum_new;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, at_need, o);
            const int64_t y = __shfl_up_sync(0xffffffffu, at_new, o);
            if (lane >= o) {
                at_need += x;
                at_new += y;
            }
        }
        if (lane == 31) {
            s_warp[0][warp] = at_need;
            s_warp[1][warp] = at_new;
        }
        __syncthreads();
        int64_t before_need = carry_need, before_new = carry_new;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            const int64_t x = s_warp[0][w], y = s_warp[1][w];
            if (w < warp) {
                before_need += x;
                before_new += y;
            }
            carry_need += x;
            carry_new += y;
        }
        at_need += before_need - sum_need;
        at_new += before_new - sum_new;
        bool served[kPlanItems];
        int last_new = 0, last_need = 0;
        bool cut = false;
#pragma unroll
        for (int j = 0; j < kPlanItems; ++j) {
            served[j] = at_need + need[j] <= free && at_new + add[j] <= a.token_capacity;
            cut |= !served[j] && add[j] > 0;
            const int k = tid * kPlanItems + j;
            s_off[k] = served[j] ? (int)at_need : 0;
            s_len[k] = len[j];
            at_need += need[j];
            at_new += add[j];
            s_end[k] = served[j] ? (int)at_new : 0x7fffffff;
            if (served[j]) {
                last_new = (int)at_new;
                last_need = (int)at_need;
            }
        }
        if (cut && last) report(a.status, PA_DEV_NO_BLOCKS);
        // the sums never fall, so the served prefix's totals are their maxima
        const int slot = round & 1;
        last_new = __reduce_max_sync(0xffffffffu, last_new);
        last_need = __reduce_max_sync(0xffffffffu, last_need);
        if (lane == 0) {
            atomicMax(&s_total[slot], last_new);
            atomicMax(&s_used[slot], last_need);
        }
        __syncthreads();
        const int total_before = total;
        total = max(total, s_total[slot]);
        used = max(used, s_used[slot]);
        if (tid == 0) s_total[slot ^ 1] = s_used[slot ^ 1] = 0;
        // round r's sequences are written by CTA r, those past the grid by the last
        if (blockIdx.x == min((unsigned)round, gridDim.x - 1)) {
#pragma unroll
            for (int j = 0; j < kPlanItems; ++j) {
                const int64_t b = base + tid * kPlanItems + j;
                if (b < a.num_seqs) {
                    a.context_lens_out[b] = len[j] + (served[j] ? add[j] : 0);
                    a.query_start[b + 1] = min(s_end[tid * kPlanItems + j], total);
                }
            }
        }
        // two tokens of a thread at a time: their searches and loads overlap
        const int i_end = min(t_hi, total);
        for (int i0 = max(t_lo, total_before) + tid; i0 < i_end; i0 += 2 * kPlanThreads) {
            int k[2] = {0, 0}, pos[2];
            int32_t *entry[2];
            int32_t phys[2];
            bool fresh[2];
#pragma unroll
            for (int step = kSeqs / 2; step >= 1; step >>= 1)        // the first sequence that ends behind the token
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (s_end[k[u] + step - 1] <= i0 + u * kPlanThreads) k[u] += step;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = i0 + u * kPlanThreads;
                if (i >= i_end) continue;
                const int len = s_len[k[u]];
                pos[u] = len + i - (k[u] > 0 ? s_end[k[u] - 1] : total_before);
                const int blk = pos[u] / kBlockSize, have = blocks_of(len);
                entry[u] = a.block_tables + (base + k[u]) * a.max_blocks + blk;
                fresh[u] = blk >= have;
                phys[u] = fresh[u] ? a.free_blocks[free - 1 - (s_off[k[u]] + blk - have)] : *entry[u];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = i0 + u * kPlanThreads;
                if (i >= i_end) continue;
                if (fresh[u] && pos[u] % kBlockSize == 0) *entry[u] = phys[u];
                const bool good = (unsigned)phys[u] < (unsigned)a.num_blocks;
                if (!good) report(a.status, PA_DEV_BAD_BLOCK_ID);
                a.slot_mapping[i] = good ? (int64_t)phys[u] * kBlockSize + pos[u] % kBlockSize : -1;
                a.positions[i] = pos[u];
            }
        }
        __syncthreads();                             // the round's arrays are read
    }
    for (int i = max(t_lo, total) + tid; i < t_hi; i += kPlanThreads) {
        a.slot_mapping[i] = -1;
        a.positions[i] = 0;
    }
    if (last && tid == 0) *a.num_free_out = free - used;
}

bool overlap(const void *p, size_t n, const void *q, size_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && x < y + m && y < x + n;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_plan_step(int32_t *block_tables, const int32_t *context_lens,
                                  const int32_t *new_lens, const int32_t *free_blocks,
                                  const int32_t *num_free, int32_t *context_lens_out,
                                  int32_t *query_start, int64_t *slot_mapping, int32_t *positions,
                                  int32_t *num_free_out, int num_seqs, int max_blocks_per_seq,
                                  int block_size, int num_blocks, int free_capacity,
                                  int token_capacity, int32_t *device_status, void *stream) {
    if (num_seqs < 0 || max_blocks_per_seq < 0 || block_size != kBlockSize || num_blocks <= 0 ||
        free_capacity < 0 || token_capacity < 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize)
        return PA_ERR_INVALID_ARG;
    if (token_capacity > 1 << 30) return PA_ERR_UNSUPPORTED;   // token indexes stay within 32 bits
    if (!query_start || !num_free || !num_free_out || (num_seqs > 0 && (!context_lens || !new_lens || !context_lens_out)) ||
        (num_seqs > 0 && max_blocks_per_seq > 0 && !block_tables) || (free_capacity > 0 && !free_blocks) ||
        (token_capacity > 0 && (!slot_mapping || !positions)))
        return PA_ERR_INVALID_ARG;
    const size_t n = (size_t)num_seqs, t = (size_t)token_capacity;
    const struct { const void *p; size_t bytes, align; } out[6] = {
        {block_tables, n * max_blocks_per_seq * 4, 4}, {context_lens_out, n * 4, 4},
        {query_start, n * 4 + 4, 4}, {slot_mapping, t * 8, 8}, {positions, t * 4, 4}, {num_free_out, 4, 4}};
    const struct { const void *p; size_t bytes; } in[4] = {
        {context_lens, n * 4}, {new_lens, n * 4}, {free_blocks, (size_t)free_capacity * 4}, {num_free, 4}};
    // every CTA reads all of the inputs while others write: nothing may overlap
    for (int i = 0; i < 6; ++i) {
        if (reinterpret_cast<uintptr_t>(out[i].p) % out[i].align) return PA_ERR_INVALID_ARG;
        for (int j = 0; j < 4; ++j)
            if (overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return PA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return PA_ERR_INVALID_ARG;
    }
    for (int j = 0; j < 4; ++j)
        if (reinterpret_cast<uintptr_t>(in[j].p) & 3u) return PA_ERR_INVALID_ARG;
    PlanArgs a;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.new_lens = new_lens;
    a.free_blocks = free_blocks;
    a.num_free = num_free;
    a.context_lens_out = context_lens_out;
    a.query_start = query_start;
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.num_free_out = num_free_out;
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.free_capacity = free_capacity;
    a.token_capacity = token_capacity;
    const int threads = num_seqs <= 256 * kPlanItems ? 256 : 512;
    // one token per thread up to 128 CTAs, then longer ranges: every CTA goes
    // through the lengths, and more of them get in one another's way (216 CTAs
    // took 10.6 us where 108 take 7.5)
    const int per_thread = std::max(1, (int)(((int64_t)token_capacity + 128 * threads - 1) / (128 * threads)));
    a.tokens_per_cta = per_thread * threads;
    const int grid = std::max(1, (int)(((int64_t)token_capacity + a.tokens_per_cta - 1) / a.tokens_per_cta));
    cudaError_t e = launch_chained(threads == 256 ? pa_plan_step_kernel<256> : pa_plan_step_kernel<512>,
                                   dim3((unsigned)grid), dim3((unsigned)threads), 0,
                                   static_cast<cudaStream_t>(stream), a);
    if (e != cudaSuccess) return cuda_failure(e, "pa_plan_step_kernel launch");
    count_launches(1);
    return PA_OK;
}
