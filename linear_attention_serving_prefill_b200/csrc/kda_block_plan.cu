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
// A call writes a few bytes per request and 12 per token, so it is bound by
// launch and memory latency until there are some 10^5 tokens.  One CTA scans the
// requests (tiles of 2048, two a thread) and writes everything per request: the new
// table entries of a tile as one flat list, whose threads find their request by
// binary search in the tile's prefix sums, so that long and short requests cost
// alike.  The tokens follow in the same CTA when they are few, else in a second
// launch over the whole device, four consecutive ones a thread.
#include "kda_gdr.h"

namespace kda {
namespace {

constexpr int kRowThreads = 1024;
constexpr int kPer = 2;                       // requests of a tile per thread
constexpr int kTile = kRowThreads * kPer;
constexpr int kTokenThreads = 256;
constexpr int kRun = 4;                       // consecutive tokens per thread
// Up to this many tokens the scanning CTA writes them itself: two waves of its
// threads take less than a second launch.
constexpr int kInlineTokens = 2 * kRowThreads * kRun;

// Division by the block size: a shift when it is a power of two (shift >= 0).
struct BlockSize {
    uint32_t size;
    int shift;
    __device__ __forceinline__ uint32_t div(uint32_t x) const { return shift >= 0 ? x >> shift : x / size; }
};

__device__ __forceinline__ int64_t blocks_of(int64_t tokens, BlockSize B)
{
    return tokens > 0x7fffffff ? (tokens + B.size - 1) / B.size : (int64_t)B.div((uint32_t)tokens + B.size - 1);
}
__device__ __forceinline__ int32_t clamp_i32(int64_t x) { return (int32_t)(x > 0x7fffffff ? 0x7fffffff : x); }

// Tokens t .. t + kRun - 1 (those below total_tokens): request by binary search among
// lo .. hi for the first (smallest n with cu[n + 1] > t), by walking for the others.
// Tokens past the last request get -1.
__device__ __forceinline__ void write_tokens(const BlockPlanArgs &a, BlockSize B, int64_t t0, uint32_t lo,
                                             uint32_t hi, bool vec)
{
    while (lo < hi) {
        const uint32_t mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > t0) hi = mid; else lo = mid + 1;
    }
    int32_t pos[kRun];
    int64_t slot[kRun];
    int n = (int)lo;
    int64_t end = n < a.num_seqs ? a.cu[n + 1] : 0;
    int64_t shift = n < a.num_seqs ? (int64_t)(a.ctx_lens ? max(a.ctx_lens[n], 0) : 0) - a.cu[n] : 0;
    uint32_t have = 0xffffffffu;      // block whose table entry is in blk
    int32_t blk = -1;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        const int64_t t = t0 + i;
        while (n < a.num_seqs && t >= end) {
            if (++n < a.num_seqs) {
                end = a.cu[n + 1];
                shift = (int64_t)(a.ctx_lens ? max(a.ctx_lens[n], 0) : 0) - a.cu[n];
                have = 0xffffffffu;
            }
        }
        pos[i] = -1;
        slot[i] = -1;
        if (n < a.num_seqs && t < a.total_tokens) {
            const uint32_t p = (uint32_t)(t + shift);      // below 2^32: two int32 sums
            const uint32_t b = B.div(p);
            if (b != have) {
                have = b;
                blk = b < (uint32_t)a.table_cols ? a.block_table[(size_t)n * a.table_cols + b] : -1;
            }
            pos[i] = clamp_i32(p);
            if (blk >= 0) slot[i] = (int64_t)blk * B.size + (p - b * B.size);
        }
    }
    if (vec && t0 + kRun <= a.total_tokens) {
        if (a.positions) *(int4 *)(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        if (a.token_slots) {
            *(longlong2 *)(a.token_slots + t0) = make_longlong2(slot[0], slot[1]);
            *(longlong2 *)(a.token_slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i)
        if (t0 + i < a.total_tokens) {
            if (a.positions) a.positions[t0 + i] = pos[i];
            if (a.token_slots) a.token_slots[t0 + i] = slot[i];
        }
}

__global__ void __launch_bounds__(kRowThreads)
plan_rows_kernel(BlockPlanArgs a, BlockSize B, bool tokens_too, bool vec)
{
    __shared__ int64_t part[2][32];
    __shared__ int32_t part_w[32];
    __shared__ int64_t sFirst[kTile];        // free-list entry of a request's first new block
    __shared__ int32_t sHave[kTile];         // its first new block
    __shared__ int32_t sPrefix[kTile + 1];   // table entries written before it, in this tile
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t head = max(*a.free_head, 0);
    int64_t run_tok = 0, run_blk = head;
    if (tid == 0) a.cu[0] = 0;
    auto from_free = [&](int64_t i) { return i < a.num_free ? a.free_blocks[i] : -1; };
    // (Unsigned: requests and a tile's table entries may reach 2^31 - 1, and both counters step past their end.)
    for (uint32_t base = 0; base < (uint32_t)a.num_seqs; base += kTile) {
        int64_t add[kPer], ctx[kPer], have[kPer], want[kPer];
        int64_t tok = 0, blk = 0;             // of this thread's requests
        int32_t wr = 0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const uint32_t n = base + tid * kPer + u;
            const bool in = n < (uint32_t)a.num_seqs;
            add[u] = in ? max(a.new_lens[n], 0) : 0;
            ctx[u] = in && a.ctx_lens ? max(a.ctx_lens[n], 0) : 0;
        }
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            have[u] = blocks_of(ctx[u], B);
            want[u] = blocks_of(ctx[u] + add[u], B);
            tok += add[u];
            blk += want[u] - have[u];
            wr += (int32_t)max((int64_t)0, min(want[u], (int64_t)a.table_cols) - have[u]);
        }
        // Block-wide inclusive scan of the three sums.
        int64_t it = tok, ib = blk;
        int32_t iw = wr;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, it, off), y = __shfl_up_sync(0xffffffffu, ib, off);
            const int32_t z = __shfl_up_sync(0xffffffffu, iw, off);
            if (lane >= off) { it += x; ib += y; iw += z; }
        }
        if (lane == 31) { part[0][warp] = it; part[1][warp] = ib; part_w[warp] = iw; }
        __syncthreads();
        if (warp == 0) {
            int64_t x = part[0][lane], y = part[1][lane];
            int32_t z = part_w[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t p = __shfl_up_sync(0xffffffffu, x, off), q = __shfl_up_sync(0xffffffffu, y, off);
                const int32_t r = __shfl_up_sync(0xffffffffu, z, off);
                if (lane >= off) { x += p; y += q; z += r; }
            }
            part[0][lane] = x; part[1][lane] = y; part_w[lane] = z;
        }
        __syncthreads();
        const int64_t before_t = warp ? part[0][warp - 1] : 0, before_b = warp ? part[1][warp - 1] : 0;
        const int32_t before_w = warp ? part_w[warp - 1] : 0, total_w = part_w[31];
        int64_t t = run_tok + before_t + it - tok, first = run_blk + before_b + ib - blk;
        int32_t w = before_w + iw - wr;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int e = tid * kPer + u;
            const uint32_t n = base + e;
            t += add[u];
            sFirst[e] = first;
            sHave[e] = clamp_i32(have[u]);
            sPrefix[e] = w;
            if (n < (uint32_t)a.num_seqs) {
                a.cu[n + 1] = clamp_i32(t);
                const int32_t *row = a.block_table + (size_t)n * a.table_cols;
                auto block_at = [&](int64_t j) {
                    if (j >= a.table_cols) return -1;
                    return j >= have[u] ? from_free(first + j - have[u]) : row[j];
                };
                // The last block's index: one below the block count.
                if (a.src) a.src[n] = have[u] > 0 ? block_at(have[u] - 1) : -1;
                if (a.dst) a.dst[n] = want[u] > 0 ? block_at(want[u] - 1) : -1;
            }
            first += want[u] - have[u];
            w += (int32_t)max((int64_t)0, min(want[u], (int64_t)a.table_cols) - have[u]);
        }
        if (tid == kRowThreads - 1) sPrefix[kTile] = w;
        run_tok += part[0][31];
        run_blk += part[1][31];
        __syncthreads();
#pragma unroll 4
        for (uint32_t e = tid; e < (uint32_t)total_w; e += kRowThreads) {
            int lo = 0, hi = kTile - 1;       // the request whose entries hold e
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if ((uint32_t)sPrefix[mid + 1] > e) hi = mid; else lo = mid + 1;
            }
            const int32_t i = (int32_t)(e - sPrefix[lo]);
            a.block_table[(size_t)(base + lo) * a.table_cols + sHave[lo] + i] = from_free(sFirst[lo] + i);
        }
        __syncthreads();
    }
    if (tid == 0) *a.free_head_out = clamp_i32(run_blk);
    if (tokens_too)
        for (int64_t t = (int64_t)tid * kRun; t < a.total_tokens; t += kRowThreads * kRun)
            write_tokens(a, B, t, 0, a.num_seqs, vec);
}

__global__ void __launch_bounds__(kTokenThreads)
plan_tokens_kernel(BlockPlanArgs a, BlockSize B, bool vec)
{
    constexpr int kCta = kTokenThreads * kRun;
    __shared__ int range[2];
    const int64_t t0 = (int64_t)blockIdx.x * kCta;
    // Requests of the CTA's first and last token; its threads search between them.
    if ((threadIdx.x & 31) == 0 && threadIdx.x < 64) {
        const int64_t t = threadIdx.x == 0 ? t0 : t0 + kCta - 1;
        uint32_t lo = 0, hi = a.num_seqs;
        while (lo < hi) {
            const uint32_t mid = (lo + hi) >> 1;
            if (a.cu[mid + 1] > t) hi = mid; else lo = mid + 1;
        }
        range[threadIdx.x >> 5] = (int)lo;
    }
    __syncthreads();
    const int64_t t = t0 + (int64_t)threadIdx.x * kRun;
    if (t < a.total_tokens) write_tokens(a, B, t, range[0], range[1], vec);
}

}  // namespace

cudaError_t launch_block_plan(const BlockPlanArgs &a, cudaStream_t stream)
{
    const bool tokens = a.total_tokens > 0 && (a.positions || a.token_slots);
    const bool inline_tokens = tokens && a.total_tokens <= kInlineTokens;
    const bool vec = (((uintptr_t)a.positions | (uintptr_t)a.token_slots) & 15) == 0;
    BlockSize B{(uint32_t)a.block, -1};
    if ((a.block & (a.block - 1)) == 0)
        for (B.shift = 0; (1 << B.shift) < a.block; ++B.shift) {}
    plan_rows_kernel<<<1, kRowThreads, 0, stream>>>(a, B, inline_tokens, vec);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !tokens || inline_tokens) return err;
    const int64_t per = (int64_t)kTokenThreads * kRun;
    plan_tokens_kernel<<<(unsigned)((a.total_tokens + per - 1) / per), kTokenThreads, 0, stream>>>(a, B, vec);
    return cudaGetLastError();
}

}  // namespace kda
