// Block tables and slot maps from request lengths, on the device.
//
// Request n has ctx tokens stored and gets `new` more; with B tokens a block it
// owns blocks 0 .. ceil(ctx / B) - 1 and needs them up to ceil((ctx + new) / B) - 1.
// The new ones are taken from the free list in request order: entry
// free_head + (exclusive prefix sum of the new-block counts) + j.  Per token the
// plan writes its absolute position and its slot (block * B + offset), per
// request the block that holds its last stored token before (src) and after
// (dst) this call.
//
// One CTA scans the requests (a running prefix over tiles of 1024) and writes
// everything per request; the tokens follow in the same CTA when they are few,
// else in a second launch over the whole device, whose threads find their
// request by binary search in cu_seqlens.
#include "kda_gdr.h"

namespace kda {
namespace {

constexpr int kRowThreads = 1024;
constexpr int kTokenThreads = 256;
constexpr int kTokensPerThread = 4;
// Up to this many tokens the scanning CTA writes them itself.
constexpr int kInlineTokens = 4096;

__device__ __forceinline__ int64_t blocks_of(int64_t tokens, int32_t B) { return (tokens + B - 1) / B; }
__device__ __forceinline__ int32_t clamp_i32(int64_t x) { return (int32_t)(x > 0x7fffffff ? 0x7fffffff : x); }

// Inclusive block-wide sums of two values; `tot` receives the totals.
__device__ __forceinline__ void scan2(int64_t &x, int64_t &y, int64_t (*part)[32], int64_t (&tot)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, x, off), b = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) { x += a; y += b; }
    }
    if (lane == 31) { part[0][warp] = x; part[1][warp] = y; }
    __syncthreads();
    if (warp == 0) {
        int64_t u = part[0][lane], w = part[1][lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, u, off), b = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) { u += a; w += b; }
        }
        part[0][lane] = u;
        part[1][lane] = w;
    }
    __syncthreads();
    if (warp > 0) { x += part[0][warp - 1]; y += part[1][warp - 1]; }
    tot[0] = part[0][31];
    tot[1] = part[1][31];
    __syncthreads();   // part may be reused
}

// Token t of the packed batch: its request by binary search, position and slot.
// Tokens past the last request get -1.
__device__ __forceinline__ void write_token(const BlockPlanArgs &a, int t)
{
    int lo = 0, hi = a.num_seqs;       // smallest n with cu[n + 1] > t, or num_seqs
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    int32_t pos = -1;
    int64_t slot = -1;
    if (lo < a.num_seqs) {
        const int64_t p = (int64_t)(t - a.cu[lo]) + (a.ctx_lens ? max(a.ctx_lens[lo], 0) : 0);
        pos = clamp_i32(p);
        if (p / a.block < a.table_cols) {
            const int32_t blk = a.block_table[(size_t)lo * a.table_cols + p / a.block];
            if (blk >= 0) slot = (int64_t)blk * a.block + p % a.block;
        }
    }
    if (a.positions) a.positions[t] = pos;
    if (a.token_slots) a.token_slots[t] = slot;
}

__global__ void __launch_bounds__(kRowThreads)
plan_rows_kernel(BlockPlanArgs a, bool tokens_too)
{
    __shared__ int64_t part[2][32];
    __shared__ int64_t sFirst[kRowThreads];
    __shared__ int32_t sHave[kRowThreads], sWant[kRowThreads];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t head = max(*a.free_head, 0);
    int64_t run_tok = 0, run_blk = head;
    if (tid == 0) a.cu[0] = 0;
    auto from_free = [&](int64_t i) { return i < a.num_free ? a.free_blocks[i] : -1; };
    for (int base = 0; base < a.num_seqs; base += kRowThreads) {
        const int n = base + tid;
        int64_t fresh = 0, ctx = 0, have = 0, want = 0, add = 0;
        if (n < a.num_seqs) {
            add = max(a.new_lens[n], 0);
            ctx = a.ctx_lens ? max(a.ctx_lens[n], 0) : 0;
            have = blocks_of(ctx, a.block);
            want = blocks_of(ctx + add, a.block);
            fresh = want - have;
        }
        int64_t tok = add, blk = fresh, tot[2];
        scan2(tok, blk, part, tot);
        const int64_t first = run_blk + blk - fresh;
        if (n < a.num_seqs) {
            a.cu[n + 1] = clamp_i32(run_tok + tok);
            const int32_t *row = a.block_table + (size_t)n * a.table_cols;
            auto block_at = [&](int64_t j) {   // before this call's entries are visible
                if (j >= a.table_cols) return -1;
                return j >= have ? from_free(first + j - have) : row[j];
            };
            if (a.src) a.src[n] = ctx > 0 ? block_at((ctx - 1) / a.block) : -1;
            if (a.dst) a.dst[n] = ctx + add > 0 ? block_at((ctx + add - 1) / a.block) : -1;
        }
        // New table entries: a warp per request, lanes over its blocks.
        sFirst[tid] = first;
        sHave[tid] = clamp_i32(have);
        sWant[tid] = (int32_t)min(want, (int64_t)a.table_cols);
        __syncthreads();
        for (int i = warp; i < kRowThreads && base + i < a.num_seqs; i += kRowThreads / 32) {
            int32_t *row = a.block_table + (size_t)(base + i) * a.table_cols;
            for (int j = sHave[i] + lane; j < sWant[i]; j += 32) row[j] = from_free(sFirst[i] + j - sHave[i]);
        }
        run_tok += tot[0];
        run_blk += tot[1];
        __syncthreads();
    }
    if (tid == 0) *a.free_head_out = clamp_i32(run_blk);
    if (tokens_too)
        for (int t = tid; t < a.total_tokens; t += kRowThreads) write_token(a, t);
}

__global__ void __launch_bounds__(kTokenThreads)
plan_tokens_kernel(BlockPlanArgs a)
{
    const int64_t stride = (int64_t)gridDim.x * kTokenThreads;
    for (int64_t t = (int64_t)blockIdx.x * kTokenThreads + threadIdx.x; t < a.total_tokens; t += stride)
        write_token(a, (int)t);
}

}  // namespace

cudaError_t launch_block_plan(const BlockPlanArgs &a, cudaStream_t stream)
{
    const bool tokens = a.total_tokens > 0 && (a.positions || a.token_slots);
    const bool inline_tokens = tokens && a.total_tokens <= kInlineTokens;
    plan_rows_kernel<<<1, kRowThreads, 0, stream>>>(a, inline_tokens);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !tokens || inline_tokens) return err;
    const int64_t per = (int64_t)kTokenThreads * kTokensPerThread;
    plan_tokens_kernel<<<(unsigned)((a.total_tokens + per - 1) / per), kTokenThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
