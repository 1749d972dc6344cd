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
// shared memory; they are kept as 64-bit registers (as float2 the same code needed
// 540 instead of 320 instructions a token: 148 and 122 us for the verify pass
// below).  The decays are not applied token by token: the registers hold
// S / run with one running factor run = prod e^{g}, folded in before it leaves
// [2^-32, 2^32], so a token costs three packed products per row pair and column.
//
// Two kernels: packed sequences stage 8 tokens at a time, the next 8 on their way in
// registers; a few tokens of each of many sequences (verify, replay) overlap one
// state's steps with the next state's load.
//
// A long sequence is bound by the latency of one token's chain (two reductions, their
// shuffles and the update, one after the other): 0.31 us a token at dk = dv = 128, 0.25 us
// at 64.  A verify pass (64 x 96 states of 128 x 128, 4 tokens, 403 MB) takes 118 us and a
// replay (100 x 32 key heads, 96 heads, up to 6 tokens) 237 us, 3.4 and 5.4 TB/s: the steps'
// shared-memory loads and shuffles, at the 16 warps per SM that the states leave room for (the
// loads and stores alone: 72 and 205 us).
// Slower, both measured: four tokens at a time from one pass over the state and a small
// triangular solve (verify 119, replay 271 us, packed 0.38 us a token), and that with four
// columns and half the rows per lane (115, 266 us, 0.42 us); the same products on m16n8k16 warp
// instructions with S in three bf16 parts (119, 297 us).
#include "kda_common.cuh"
#include "kda_gdr.h"

namespace kda {
namespace {

constexpr int kGroup = 8, kFew = 4;  // tokens staged together: packed sequences, a few tokens each
constexpr int kSms = 148;

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

// Two adjacent elements as fp32.
__device__ __forceinline__ float2 load_pair(const float *p) { return *(const float2 *)p; }
__device__ __forceinline__ float2 load_pair(const __nv_bfloat16 *p) {
    const uint32_t u = *(const uint32_t *)p;
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
template <int BYTES> __device__ __forceinline__ void copy_async(void *to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                 ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "n"(BYTES) : "memory");
}

// Two fp32 outputs to adjacent storage elements.
__device__ __forceinline__ void store_pair(float *p, float2 x) { *(float2 *)p = x; }
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float2 x) {
    *(__nv_bfloat162 *)p = __floats2bfloat162_rn(x.x, x.y);
}

// Packed fp32 pairs as 64-bit registers.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float x, float y) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 both(Pair p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The columns col, col + 1 of one state for a lane: row pairs 8 i + 2 rq, + 1, over run.
template <int DK, int DV> struct Columns {
    static constexpr int R = DK / 8, kLd = DK / 4 + 4;   // row pairs; stride of a row group in a staged vector
    Pair s0[R], s1[R];
    float run;

    __device__ __forceinline__ void set(int i, float2 x, float2 y) {   // rows of pair i
        s0[i] = pair(x.x, y.x);
        s1[i] = pair(x.y, y.y);
    }
    // p: row 2 rq, column col of a state.
    __device__ __forceinline__ void load(const float *p) {
        run = 1.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (p)
                set(i, *(const float2 *)(p + (size_t)8 * i * DV), *(const float2 *)(p + (size_t)(8 * i + 1) * DV));
            else
                s0[i] = s1[i] = 0;
        }
    }
    __device__ __forceinline__ void store(float *p) const {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float2 x = both(s0[i]), y = both(s1[i]);
            *(float2 *)(p + (size_t)8 * i * DV) = make_float2(run * x.x, run * y.x);
            *(float2 *)(p + (size_t)(8 * i + 1) * DV) = make_float2(run * x.y, run * y.y);
        }
    }
    // One token: k and q this lane's row group of the staged vectors, kq their product, b beta;
    // returns the outputs before their scale.
    __device__ __forceinline__ float2 token(const float *k, const float *q, float decay, float b, float kq, float2 v) {
        run *= decay;
        if (!(run >= 0x1p-32f && run <= 0x1p32f)) {      // into the state
            const Pair f = pair(run, run);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                s0[i] = mul2(s0[i], f);
                s1[i] = mul2(s1[i], f);
            }
            run = 1.f;
        }
        Pair n0[2] = {}, n1[2] = {}, r0[2] = {}, r1[2] = {};
#pragma unroll
        for (int i = 0; i < R; i += 2) {
            const ulonglong2 kk = *(const ulonglong2 *)(k + 2 * i), qq = *(const ulonglong2 *)(q + 2 * i);
            n0[0] = fma2(kk.x, s0[i], n0[0]);
            n1[0] = fma2(kk.x, s1[i], n1[0]);
            r0[0] = fma2(qq.x, s0[i], r0[0]);
            r1[0] = fma2(qq.x, s1[i], r1[0]);
            n0[1] = fma2(kk.y, s0[i + 1], n0[1]);
            n1[1] = fma2(kk.y, s1[i + 1], n1[1]);
            r0[1] = fma2(qq.y, s0[i + 1], r0[1]);
            r1[1] = fma2(qq.y, s1[i + 1], r1[1]);
        }
        auto total = [&](const Pair (&x)[2]) {
            const float2 y = both(x[0]), z = both(x[1]);
            return run * group_sum((y.x + z.x) + (y.y + z.y));
        };
        const float seen0 = total(n0), seen1 = total(n1), read0 = total(r0), read1 = total(r1);
        const float d0 = b * (v.x - seen0), d1 = b * (v.y - seen1);
        const float inv = __frcp_rn(run);
        const Pair e0 = pair(d0 * inv, d0 * inv), e1 = pair(d1 * inv, d1 * inv);
#pragma unroll
        for (int i = 0; i < R; i += 2) {
            const ulonglong2 kk = *(const ulonglong2 *)(k + 2 * i);
            s0[i] = fma2(kk.x, e0, s0[i]);
            s1[i] = fma2(kk.x, e1, s1[i]);
            s0[i + 1] = fma2(kk.y, e0, s0[i + 1]);
            s1[i + 1] = fma2(kk.y, e1, s1[i + 1]);
        }
        return make_float2(fmaf(kq, d0, read0), fmaf(kq, d1, read1));
    }
};

// Channels c .. c + 7 of a vector into its staged form: four row groups, channels 8 i + 2 rq, + 1
// of group rq in a row of kLd.
template <int kLd> __device__ __forceinline__ void stage8(float *to, int c, const float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) *(float2 *)&to[(i >> 1) * kLd + (c >> 2)] = make_float2(x[i], x[i + 1]);
}

template <int DV> constexpr int kWarpsOf = DV >= 64 ? 4 : 2;

// Packed sequences.
template <int DK, int DV, typename T>
__global__ void __launch_bounds__(32 * kWarpsOf<DV>, 1)
gdr_recurrent_kernel(GdrArgs a)
{
    using Cols = Columns<DK, DV>;
    constexpr int kWarps = kWarpsOf<DV>, kThreads = 32 * kWarps, kLd = Cols::kLd;
    constexpr int kCols = 16 * kWarps;           // value columns of this CTA
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

    const int64_t t0 = max(a.cu[n], 0);
    const int len = max(min(a.cu[n + 1], a.total_tokens) - (int)t0, 0);
    // Pool rows: outside [0, pool_size) the state starts from zero / is not written.
    int src = a.src ? a.src[n] : -1, dst = a.dst ? a.dst[n] : -1;
    if (!a.state || src < 0 || src >= a.pool_size) src = -1;
    if (!a.state || dst < 0 || dst >= a.pool_size) dst = -1;
    if (len == 0 && dst < 0) return;
    const size_t own = (size_t)(2 * rq) * DV + col;    // row 2 rq, this lane's column pair
    auto row_of = [&](int slot) { return a.state + ((size_t)slot * a.H + h) * DK * DV + own; };

    Cols S;
    S.load(src >= 0 ? row_of(src) : nullptr);

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
                stage8<kLd>(sK[t], c, pk[u]);
                stage8<kLd>(sQ[t], c, pq[u]);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = fmaf(pk[u][i], pq[u][i], dot);
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
            const float2 y = S.token(&sK[t][rq * kLd], &sQ[t][rq * kLd], sA[t], sB[t], sKQ[t],
                                     *(const float2 *)&sV[t][col - part * kCols]);
            if (rq == 0)
                store_pair(o + ((size_t)(t0 + base + t) * a.H + h) * DV + col, make_float2(a.scale * y.x, a.scale * y.y));
            if (--to_block == 0) {       // a completed block: its row keeps this state
                const int row = blk < a.table_cols ? a.table[(size_t)n * a.table_cols + blk] : -1;
                if (row >= 0 && row < a.pool_size) S.store(row_of(row));
                to_block = a.block;
                ++blk;
            }
        }
    }
    if (dst >= 0 && (len > 0 || dst != src)) S.store(row_of(dst));
}

// One of PARTS column parts of a sequence's state in the decode layout.
struct Item { int n, h, part, src, dst, len; };
template <int PARTS> __device__ __forceinline__ Item item_at(const GdrArgs &a, uint32_t it) {
    Item x;
    x.part = it % PARTS;
    const uint32_t chain = it / PARTS;
    x.n = chain / (uint32_t)a.H;
    x.h = chain - x.n * a.H;
    x.len = a.num_tokens ? min(max(a.num_tokens[x.n], 0), a.Tq) : a.Tq;
    // Pool rows: outside [0, pool_size) the state starts from zero / is not written.
    x.src = a.src ? a.src[x.n] : x.n;
    x.dst = a.dst ? a.dst[x.n] : x.src;
    if (x.src < 0 || x.src >= a.pool_size) x.src = -1;
    if (!a.update || x.dst < 0 || x.dst >= a.pool_size || (x.len == 0 && x.dst == x.src)) x.dst = -1;
    return x;
}

// A few tokens of each of many sequences.  A CTA walks over states; while it applies one
// state's tokens, the next state's columns and tokens are on their way into shared memory
// (cp.async; a thread fetches what it keeps, so the state needs no barrier), so that loads
// and steps overlap although a state fills the registers.  BLOCKS: the state after a block's last
// token goes to that block's row.
template <int DK, int DV, typename T, bool BLOCKS>
__global__ void __launch_bounds__(32 * kWarpsOf<DV>, 16 / kWarpsOf<DV>)
gdr_few_kernel(GdrArgs a, uint32_t items)
{
    using Cols = Columns<DK, DV>;
    constexpr int kWarps = kWarpsOf<DV>, kThreads = 32 * kWarps, kLd = Cols::kLd, R = Cols::R;
    constexpr int kCols = 16 * kWarps, kParts = DV / kCols;
    constexpr int kPieces = kFew * DK / 8;
    constexpr int kEl = 16 / sizeof(T);          // elements of a 16-byte copy
    __shared__ __align__(16) float2 sS[2 * R][kThreads];
    __shared__ __align__(16) T rK[kFew][DK], rQ[kFew][DK], rV[2][kFew][kCols];
    __shared__ __align__(16) float sK[kFew][4 * kLd], sQ[kFew][4 * kLd];
    __shared__ float rG[kFew], rB[kFew], sA[kFew], sB[kFew], sKQ[kFew];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t group = a.H / a.Hk;
    const int rq = lane >> 3, own_col = 16 * warp + 2 * (lane & 7);
    const T *q = (const T *)a.q, *k = (const T *)a.k, *v = (const T *)a.v;
    T *o = (T *)a.o;

    auto state_at = [&](const Item &x, int slot) {   // row 2 rq, this lane's column pair
        return a.state + ((size_t)slot * a.H + x.h) * DK * DV + (size_t)(2 * rq) * DV + x.part * kCols + own_col;
    };
    int buf = 0;                   // rV's half that the next copies go to
    auto fetch_tokens = [&](const Item &x, int base) {
        const int hk = (uint32_t)x.h / group, m = min(kFew, x.len - base);
        const size_t t0 = (size_t)x.n * a.Tq + base;
        for (int e = tid; e < m * (DK / kEl); e += kThreads) {
            const int t = e / (DK / kEl), c = (e % (DK / kEl)) * kEl;
            const size_t at = ((t0 + t) * a.Hk + hk) * DK + c;
            copy_async<16>(&rK[t][c], k + at);
            copy_async<16>(&rQ[t][c], q + at);
        }
        for (int e = tid; e < m * (kCols / kEl); e += kThreads) {
            const int t = e / (kCols / kEl), c = (e % (kCols / kEl)) * kEl;
            copy_async<16>(&rV[buf][t][c], v + ((t0 + t) * a.H + x.h) * DV + x.part * kCols + c);
        }
        if (tid < m) {
            copy_async<4>(&rG[tid], a.g + (t0 + tid) * a.H + x.h);
            copy_async<4>(&rB[tid], a.beta + (t0 + tid) * a.H + x.h);
        }
    };
    auto fetch = [&](const Item &x) {
        if (x.len == 0 && x.dst < 0) return;
        if (x.src >= 0) {
            const float *p = state_at(x, x.src);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                copy_async<8>(&sS[2 * i][tid], p + (size_t)8 * i * DV);
                copy_async<8>(&sS[2 * i + 1][tid], p + (size_t)(8 * i + 1) * DV);
            }
        }
        fetch_tokens(x, 0);
    };

    uint32_t it = blockIdx.x;
    Item x = item_at<kParts>(a, it);          // (no more CTAs than items)
    fetch(x);
    for (;;) {
        const bool more = items - it > gridDim.x;
        Item next = x;
        if (more) next = item_at<kParts>(a, it + gridDim.x);
        Cols S;
        S.run = 1.f;
        auto position = [&](int t) { return (uint32_t)(a.ctx ? max(a.ctx[x.n], 0) : 0) + t; };
        uint32_t to_block = 0;     // tokens left in the current block
        if (BLOCKS) to_block = a.block - position(0) % a.block;
        for (int base = 0; base == 0 || base < x.len; base += kFew) {
            const int m = min(kFew, x.len - base);
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (base == 0) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float2 zero = make_float2(0.f, 0.f);
                    S.set(i, x.src >= 0 ? sS[2 * i][tid] : zero, x.src >= 0 ? sS[2 * i + 1][tid] : zero);
                }
            }
            __syncthreads();       // every thread's copies are here; the previous tokens are no longer read
            for (int e0 = 0; e0 < kPieces; e0 += kThreads) {
                const int e = e0 + tid, t = e / (DK / 8), c = (e % (DK / 8)) * 8;
                float dot = 0.f;
                if (e < kPieces && t < m) {
                    float xk[8], xq[8];
                    load8(&rK[t][c], xk);
                    load8(&rQ[t][c], xq);
                    stage8<kLd>(sK[t], c, xk);
                    stage8<kLd>(sQ[t], c, xq);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot = fmaf(xk[i], xq[i], dot);
                }
#pragma unroll
                for (int off = 1; off < DK / 8; off <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
                if (e < kPieces && t < m && e % (DK / 8) == 0) sKQ[t] = dot;
            }
            if (tid < m) { sA[tid] = expf(clamp_log_decay(rG[tid])); sB[tid] = rB[tid]; }
            buf ^= 1;
            __syncthreads();       // staged; the buffers of the copies are free
            if (base + kFew < x.len) fetch_tokens(x, base + kFew);
            else if (more) fetch(next);
            const size_t t0 = (size_t)x.n * a.Tq + base;
#pragma unroll 1
            for (int t = 0; t < m; ++t) {
                const float2 y = S.token(&sK[t][rq * kLd], &sQ[t][rq * kLd], sA[t], sB[t], sKQ[t],
                                         load_pair(&rV[buf ^ 1][t][own_col]));
                if (o && rq == 0)
                    store_pair(o + ((t0 + t) * a.H + x.h) * DV + x.part * kCols + own_col,
                               make_float2(a.scale * y.x, a.scale * y.y));
                if (BLOCKS) {
                    if (--to_block == 0) {
                        const uint32_t blk = position(base + t) / (uint32_t)a.block;
                        const int row = blk < (uint32_t)a.table_cols ? a.table[(size_t)x.n * a.table_cols + blk] : -1;
                        if (row >= 0 && row < a.pool_size) S.store(state_at(x, row));
                        to_block = a.block;
                    }
                }
            }
        }
        if (x.dst >= 0) S.store(state_at(x, x.dst));
        if (!more) break;
        it += gridDim.x;
        x = next;
    }
}

template <int DK, int DV, typename T>
cudaError_t launch_typed(const GdrArgs &a, cudaStream_t stream)
{
    constexpr int kThreads = 32 * kWarpsOf<DV>;
    const int64_t items = (int64_t)a.num_seqs * a.H * (DV / (kThreads / 2));
    if (items == 0) return cudaSuccess;
    if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (a.cu) {
        gdr_recurrent_kernel<DK, DV, T><<<(unsigned)items, kThreads, 0, stream>>>(a);
    } else {
        const int64_t resident = (int64_t)kSms * (16 / kWarpsOf<DV>);
        auto *kernel = a.block > 0 ? gdr_few_kernel<DK, DV, T, true> : gdr_few_kernel<DK, DV, T, false>;
        kernel<<<(unsigned)(items < resident ? items : resident), kThreads, 0, stream>>>(a, (uint32_t)items);
    }
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
