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
// channels: lane (rq, c) keeps rows 4 i + rq of the column pair 2 c, 2 c + 1 (64
// registers at dk = 128), both reductions of a token are two xor shuffles over
// the four row groups, and no token step crosses warps.  q, k, v, g and beta of
// kGroup tokens at a time are staged in shared memory as fp32 (k and q permuted
// so that a lane's rows are contiguous); the next group's global loads are in
// flight while the current one runs.
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

__device__ __forceinline__ float2 shfl_add(float2 x, int mask) {
    x.x += __shfl_xor_sync(0xffffffffu, x.x, mask);
    x.y += __shfl_xor_sync(0xffffffffu, x.y, mask);
    return x;
}

// Two fp32 outputs to adjacent storage elements.
__device__ __forceinline__ void store_pair(float *p, float2 x) { *(float2 *)p = x; }
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float2 x) {
    *(__nv_bfloat162 *)p = __floats2bfloat162_rn(x.x, x.y);
}

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(DV >= 64 ? 128 : 64)
gdr_recurrent_kernel(GdrArgs a)
{
    constexpr int kWarps = DV >= 64 ? 4 : 2, kThreads = 32 * kWarps;
    constexpr int kCols = 16 * kWarps;           // value columns of this CTA
    constexpr int R = DK / 4;                    // rows per lane
    constexpr int kLd = R + 4;                   // row-group stride: distinct banks for the four groups
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
    const size_t own = (size_t)rq * DV + col;    // row rq, this lane's column pair
    auto row_of = [&](int slot) { return a.state + ((size_t)slot * a.H + h) * DK * DV + own; };

    float2 s[R];
    if (src >= 0) {
        const float *p = row_of(src);
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = *(const float2 *)(p + (size_t)4 * i * DV);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = make_float2(0.f, 0.f);
    }
    auto write_row = [&](int slot) {
        float *p = row_of(slot);
#pragma unroll
        for (int i = 0; i < R; ++i) *(float2 *)(p + (size_t)4 * i * DV) = s[i];
    };

    const T *q = (const T *)a.q, *k = (const T *)a.k, *v = (const T *)a.v;
    T *o = (T *)a.o;
    const int ctx = a.ctx ? a.ctx[n] : 0;
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
            const int e = tid + u * kThreads, t = e / (DK / 8), c = (e % (DK / 8)) * 8;
            float dot = 0.f;
            if (e < kPieces) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {   // channel c + i: row group (c + i) % 4
                    const int at = ((c + i) & 3) * kLd + ((c + i) >> 2);
                    sK[t][at] = pk[u][i];
                    sQ[t][at] = pq[u][i];
                    dot = fmaf(pk[u][i], pq[u][i], dot);
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
            const float al = sA[t];
            const float2 al2 = make_float2(al, al);
            float2 seen[2] = {{0.f, 0.f}, {0.f, 0.f}}, read[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                const float4 k4 = *(const float4 *)&sK[t][rq * kLd + i];
                const float4 q4 = *(const float4 *)&sQ[t][rq * kLd + i];
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i + j] = __fmul2_rn(s[i + j], al2);
                    seen[j & 1] = __ffma2_rn(make_float2(kk[j], kk[j]), s[i + j], seen[j & 1]);
                    read[j & 1] = __ffma2_rn(make_float2(qq[j], qq[j]), s[i + j], read[j & 1]);
                }
            }
            float2 sn = __fadd2_rn(seen[0], seen[1]), rd = __fadd2_rn(read[0], read[1]);
            sn = shfl_add(sn, 8);
            rd = shfl_add(rd, 8);
            sn = shfl_add(sn, 16);
            rd = shfl_add(rd, 16);
            const float2 vv = *(const float2 *)&sV[t][col - part * kCols];
            const float b = sB[t];
            const float2 d = make_float2(b * (vv.x - sn.x), b * (vv.y - sn.y));
            if (o && rq == 0) {
                const float kq = sKQ[t];
                store_pair(o + ((size_t)(t0 + base + t) * a.H + h) * DV + col,
                           make_float2(a.scale * fmaf(kq, d.x, rd.x), a.scale * fmaf(kq, d.y, rd.y)));
            }
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                const float4 k4 = *(const float4 *)&sK[t][rq * kLd + i];
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[i + j] = __ffma2_rn(make_float2(kk[j], kk[j]), d, s[i + j]);
            }
            if (a.block > 0) {       // a completed block: its row keeps this state
                const int pos = ctx + base + t + 1;
                if (pos > 0 && pos % a.block == 0 && pos / a.block <= a.table_cols) {
                    const int row = a.table[(size_t)n * a.table_cols + pos / a.block - 1];
                    if (row >= 0 && row < a.pool_size) write_row(row);
                }
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
    gdr_recurrent_kernel<DK, DV, T><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
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
