// Gated delta rule, token by token on a register-resident state:
//
//   Sb = e^{g} S;  d = beta (v - Sb^T k);  S <- Sb + k d^T;
//   o = scale S^T q = scale (Sb^T q + (k . q) d)
//
// with one log-decay g per token and value head; value head h reads key head
// h / (H / Hk).  This path serves every storage type and head size (the fp32
// check mode among them), packed sequences as well as a few tokens each
// (speculative verify and replay).
//
// Columns of S never mix, so a warp owns 16 value columns for all dk key
// channels: lane (rq, c) keeps the row pairs 8 i + 2 rq, + 1 of the columns 2 c and
// 2 c + 1 (64 registers at dk = 128), both reductions of a token are two xor
// shuffles over the four row groups, and no token step crosses warps.  Packed fp32
// pairs run along the rows, so that the pairs of k and q come as they lie in
// shared memory.  The decays are not applied token by token: the registers hold
// S / run with one running factor run = prod e^{g}, folded in before it leaves
// [2^-32, 2^32], so a token costs three packed products per row pair and column.
// q, k, v, g and beta of kGroup tokens at a time are staged in shared memory as
// fp32; the next group's global loads are in flight while the current one runs.
//
// A long sequence is bound by the latency of one token's chain (0.35 us at dk = 128,
// 0.30 us at dk = 64: two reductions, their shuffles and the update, one after the other);
// a verify pass of a few tokens by reading the states (64 x 96 states, 4 tokens: 139 us,
// 3.1 TB/s).
#include "kda_common.cuh"
#include "kda_gdr.h"

namespace kda {
namespace {

constexpr int kGroup = 8;           // tokens staged together

// The log-decay is clamped where e^{g} is 0 in fp32 anyway; NaN passes through.
__device__ __forceinline__ float clamp_log_decay(float g) { return g < kGClampSoftplus ? kGClampSoftplus : g; }

// 8 consecutive elements as fp32.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = *(const float4 *)p, b = *(const float4 *)(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 u = *(const uint4 *)p;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Sum over the four row groups.
__device__ __forceinline__ float group_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Two fp32 outputs to adjacent storage elements.
__device__ __forceinline__ void store_pair(float *p, float2 x) { *(float2 *)p = x; }
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float2 x) {
    *(__nv_bfloat162 *)p = __floats2bfloat162_rn(x.x, x.y);
}

// kMinBlocks: 4 (128 registers, a few of them spilled at dk = 128) holds more states per SM
// and wins where each sequence has a few tokens and loading the states counts; 1 wins over
// long sequences.  bf16, dk = dv = 128, 4 / 1: verify of 64 x 4 tokens, 32 heads 139 / 146 us;
// replay of 256 x up to 8 tokens 265 / 285 us.  dv = 64, prefill of 2048 tokens, 16 heads:
// 1112 / 836 us.
template <int DK, int DV, typename T, int kMinBlocks>
__global__ void __launch_bounds__(DV >= 64 ? 128 : 64, kMinBlocks)
gdr_recurrent_kernel(GdrArgs a)
{
    constexpr int kWarps = DV >= 64 ? 4 : 2, kThreads = 32 * kWarps;
    constexpr int kCols = 16 * kWarps;           // value columns of this CTA
    constexpr int R = DK / 8;                    // row pairs per lane
    constexpr int kLd = DK / 4 + 4;              // row-group stride: distinct banks for the four groups
    constexpr int kPieces = kGroup * DK / 8;     // 8-element pieces of one staged operand
    constexpr int kPer = (kPieces + kThreads - 1) / kThreads;
    constexpr int kVPieces = kGroup * kCols / 8;
    constexpr int kVPer = (kVPieces + kThreads - 1) / kThreads;
    __shared__ __align__(16) float sK[kGroup][4 * kLd], sQ[kGroup][4 * kLd];
    __shared__ __align__(16) float sV[kGroup][kCols];
    __shared__ float sA[kGroup], sB[kGroup], sKQ[kGroup];

    constexpr int kParts = DV / kCols;
    const int part = blockIdx.x % kParts;
    const int64_t chain = blockIdx.x / kParts;
    const int n = (int)(chain / a.H), h = (int)(chain % a.H);
    const int hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rq = lane >> 3, col = part * kCols + 16 * warp + 2 * (lane & 7);

    int64_t t0;
    int len;
    if (a.cu) {
        const int lo = max(a.cu[n], 0), hi = min(a.cu[n + 1], a.total_tokens);
        t0 = lo;
        len = max(hi - lo, 0);
    } else {
        t0 = (int64_t)n * a.Tq;
        len = a.num_tokens ? min(max(a.num_tokens[n], 0), a.Tq) : a.Tq;
    }
    // Pool rows: outside [0, pool_size) the state starts from zero / is not written.
    int src = a.src ? a.src[n] : (a.cu ? -1 : n);
    int dst = a.dst ? a.dst[n] : (a.cu ? -1 : src);
    if (!a.state || src < 0 || src >= a.pool_size) src = -1;
    if (!a.state || !a.update || dst < 0 || dst >= a.pool_size) dst = -1;
    if (len == 0 && dst < 0) return;
    const size_t own = (size_t)(2 * rq) * DV + col;    // row 2 rq, this lane's column pair
    auto row_of = [&](int slot) { return a.state + ((size_t)slot * a.H + h) * DK * DV + own; };

    float2 s0[R], s1[R];     // row pairs of columns col and col + 1, over run
    float run = 1.f;
    {
        const float *p = src >= 0 ? row_of(src) : nullptr;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float2 x = make_float2(0.f, 0.f), y = x;
            if (p) {
                x = *(const float2 *)(p + (size_t)8 * i * DV);
                y = *(const float2 *)(p + (size_t)(8 * i + 1) * DV);
            }
            s0[i] = make_float2(x.x, y.x);
            s1[i] = make_float2(x.y, y.y);
        }
    }
    auto fold = [&] {        // run into the state
#pragma unroll
        for (int i = 0; i < R; ++i) {
            s0[i] = __fmul2_rn(s0[i], make_float2(run, run));
            s1[i] = __fmul2_rn(s1[i], make_float2(run, run));
        }
        run = 1.f;
    };
    auto write_row = [&](int slot) {
        float *p = row_of(slot);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            *(float2 *)(p + (size_t)8 * i * DV) = make_float2(run * s0[i].x, run * s1[i].x);
            *(float2 *)(p + (size_t)(8 * i + 1) * DV) = make_float2(run * s0[i].y, run * s1[i].y);
        }
    };

    const T *q = (const T *)a.q, *k = (const T *)a.k, *v = (const T *)a.v;
    T *o = (T *)a.o;
    // Tokens left in the current block, and its index (no blocks: more than there are tokens).
    const int ctx = a.ctx ? max(a.ctx[n], 0) : 0;
    int64_t to_block = a.block > 0 ? a.block - ctx % a.block : (int64_t)1 << 40;
    int blk = a.block > 0 ? ctx / a.block : 0;
    float pk[kPer][8], pq[kPer][8], pv[kVPer][8], pa = 0.f, pb = 0.f;
    auto fetch = [&](int base) {     // tokens base .. base + kGroup - 1 into registers
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int e = tid + u * kThreads, t = e / (DK / 8), c = (e % (DK / 8)) * 8;
            if (e < kPieces && base + t < len) {
                const size_t at = ((size_t)(t0 + base + t) * a.Hk + hk) * DK + c;
                load8(k + at, pk[u]);
                load8(q + at, pq[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kVPer; ++u) {
            const int e = tid + u * kThreads, t = e / (kCols / 8), c = (e % (kCols / 8)) * 8;
            if (e < kVPieces && base + t < len)
                load8(v + ((size_t)(t0 + base + t) * a.H + h) * DV + part * kCols + c, pv[u]);
        }
        if (tid < kGroup && base + tid < len) {
            pa = a.g[(size_t)(t0 + base + tid) * a.H + h];
            pb = a.beta[(size_t)(t0 + base + tid) * a.H + h];
        }
    };
    fetch(0);
    for (int base = 0; base < len; base += kGroup) {
        const int m = min(kGroup, len - base);
        __syncthreads();             // the previous group is no longer read
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int e = tid + u * kThreads, t = e / (DK / 8), c = (e % (DK / 8)) * 8;   // channels c .. c + 7
            float dot = 0.f;
            if (e < kPieces) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {   // channels c + i, + 1: row group (c + i) / 2 % 4
                    const int at = ((i >> 1) & 3) * kLd + (c >> 2);
                    *(float2 *)&sK[t][at] = make_float2(pk[u][i], pk[u][i + 1]);
                    *(float2 *)&sQ[t][at] = make_float2(pq[u][i], pq[u][i + 1]);
                    dot = fmaf(pk[u][i], pq[u][i], fmaf(pk[u][i + 1], pq[u][i + 1], dot));
                }
            }
            // The DK / 8 lanes of one token are neighbours of one warp.
#pragma unroll
            for (int off = 1; off < DK / 8; off <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            if (e < kPieces && e % (DK / 8) == 0) sKQ[t] = dot;
        }
#pragma unroll
        for (int u = 0; u < kVPer; ++u) {
            const int e = tid + u * kThreads, t = e / (kCols / 8), c = (e % (kCols / 8)) * 8;
            if (e < kVPieces) {
                *(float4 *)&sV[t][c] = make_float4(pv[u][0], pv[u][1], pv[u][2], pv[u][3]);
                *(float4 *)&sV[t][c + 4] = make_float4(pv[u][4], pv[u][5], pv[u][6], pv[u][7]);
            }
        }
        if (tid < kGroup) { sA[tid] = expf(clamp_log_decay(pa)); sB[tid] = pb; }
        __syncthreads();
        if (base + kGroup < len) fetch(base + kGroup);
        for (int t = 0; t < m; ++t) {
            run *= sA[t];
            if (!(run >= 0x1p-32f && run <= 0x1p32f)) fold();
            const float inv = __frcp_rn(run);
            float2 n0[2] = {}, n1[2] = {}, r0[2] = {}, r1[2] = {};
#pragma unroll
            for (int i = 0; i < R; i += 2) {
                const float4 k4 = *(const float4 *)&sK[t][rq * kLd + 2 * i];
                const float4 q4 = *(const float4 *)&sQ[t][rq * kLd + 2 * i];
                const float2 ka = make_float2(k4.x, k4.y), kb = make_float2(k4.z, k4.w);
                const float2 qa = make_float2(q4.x, q4.y), qb = make_float2(q4.z, q4.w);
                n0[0] = __ffma2_rn(ka, s0[i], n0[0]);
                n1[0] = __ffma2_rn(ka, s1[i], n1[0]);
                r0[0] = __ffma2_rn(qa, s0[i], r0[0]);
                r1[0] = __ffma2_rn(qa, s1[i], r1[0]);
                n0[1] = __ffma2_rn(kb, s0[i + 1], n0[1]);
                n1[1] = __ffma2_rn(kb, s1[i + 1], n1[1]);
                r0[1] = __ffma2_rn(qb, s0[i + 1], r0[1]);
                r1[1] = __ffma2_rn(qb, s1[i + 1], r1[1]);
            }
            auto total = [&](const float2 (&x)[2]) {
                const float2 y = __fadd2_rn(x[0], x[1]);
                return run * group_sum(y.x + y.y);
            };
            const float seen0 = total(n0), seen1 = total(n1), read0 = total(r0), read1 = total(r1);
            const float2 vv = *(const float2 *)&sV[t][col - part * kCols];
            const float b = sB[t];
            const float d0 = b * (vv.x - seen0), d1 = b * (vv.y - seen1);
            if (o && rq == 0) {
                const float kq = sKQ[t];
                store_pair(o + ((size_t)(t0 + base + t) * a.H + h) * DV + col,
                           make_float2(a.scale * fmaf(kq, d0, read0), a.scale * fmaf(kq, d1, read1)));
            }
            const float e0 = d0 * inv, e1 = d1 * inv;
#pragma unroll
            for (int i = 0; i < R; i += 2) {
                const float4 k4 = *(const float4 *)&sK[t][rq * kLd + 2 * i];
                const float2 ka = make_float2(k4.x, k4.y), kb = make_float2(k4.z, k4.w);
                s0[i] = __ffma2_rn(ka, make_float2(e0, e0), s0[i]);
                s1[i] = __ffma2_rn(ka, make_float2(e1, e1), s1[i]);
                s0[i + 1] = __ffma2_rn(kb, make_float2(e0, e0), s0[i + 1]);
                s1[i + 1] = __ffma2_rn(kb, make_float2(e1, e1), s1[i + 1]);
            }
            if (--to_block == 0) {       // a completed block: its row keeps this state
                const int row = blk < a.table_cols ? a.table[(size_t)n * a.table_cols + blk] : -1;
                if (row >= 0 && row < a.pool_size) write_row(row);
                to_block = a.block;
                ++blk;
            }
        }
    }
    if (dst >= 0 && (len > 0 || dst != src)) write_row(dst);
}

template <int DK, int DV, typename T>
cudaError_t launch_typed(const GdrArgs &a, cudaStream_t stream)
{
    constexpr int kThreads = DV >= 64 ? 128 : 64;
    const int64_t blocks = (int64_t)a.num_seqs * a.H * (DV / (kThreads / 2));
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (sizeof(T) == 2 && DV >= 64 && !a.cu)
        gdr_recurrent_kernel<DK, DV, T, sizeof(T) == 2 && DV >= 64 ? 4 : 1><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    else
        gdr_recurrent_kernel<DK, DV, T, 1><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int DK, typename T>
cudaError_t launch_dv(const GdrArgs &a, cudaStream_t stream)
{
    switch (a.dv) {
    case 32: return launch_typed<DK, 32, T>(a, stream);
    case 64: return launch_typed<DK, 64, T>(a, stream);
    case 128: return launch_typed<DK, 128, T>(a, stream);
    default: return cudaErrorInvalidValue;
    }
}

template <typename T>
cudaError_t launch_dk(const GdrArgs &a, cudaStream_t stream)
{
    switch (a.dk) {
    case 32: return launch_dv<32, T>(a, stream);
    case 64: return launch_dv<64, T>(a, stream);
    case 128: return launch_dv<128, T>(a, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_gdr_recurrent(const GdrArgs &a, cudaStream_t stream)
{
    return a.bf16 ? launch_dk<__nv_bfloat16>(a, stream) : launch_dk<float>(a, stream);
}

}  // namespace kda
