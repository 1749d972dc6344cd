// Gated delta rule, one token per sequence (decode).  The state is read once
// into registers (128-bit loads, whole rows per warp), both dk reductions run
// on the decayed copy, and the updated state is written once:
//
//   seen = e^{g} S^T k,  read = e^{g} S^T q,  d = beta (v - seen),
//   S <- e^{g} S + k d^T,  o = scale (read + (k . q) d)
//
// so a step moves 8 dk dv bytes per (sequence, head) and is bound by HBM.
// Thread (rg, cg) of a CTA holds rows rg, rg + RG, ... of float4 column group cg of
// the CTA's COLS value columns: all of them in a large batch (whole rows per warp),
// 32 in a small one, so that more SMs share the latency of few states.  256 sequences of 96
// heads of 128 x 128 (3.24 GB): 523 us, 6.2 TB/s, 95 % of a plain copy's rate.
#include "kda_common.cuh"
#include "kda_gdr.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 148;

// BLOCKS: a token that completes a block leaves the state in that block's row too (as a value of the
// arguments instead, 534 to 536 instead of 524 us).
template <int DK, int DV, int COLS, typename T, bool BLOCKS>
__global__ void __launch_bounds__(kThreads)
gdr_step_kernel(GdrArgs a)
{
    constexpr int CG = COLS / 4, RG = kThreads / CG, RPT = DK / RG, kParts = DV / COLS;
    static_assert(RPT >= 1 && RG * CG == kThreads, "bad decode tiling");
    __shared__ float sK[DK], sQ[DK];
    __shared__ float4 sSeen[RG][CG], sRead[RG][CG], sD[CG];
    __shared__ float sKQ;

    const int part = blockIdx.x % kParts, bh = blockIdx.x / kParts;
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
    int src = a.src ? a.src[b] : b;
    int dst = a.dst ? a.dst[b] : src;
    if (src < 0 || src >= a.pool_size) src = -1;
    if (!a.update || dst < 0 || dst >= a.pool_size) dst = -1;
    const bool live = !a.num_tokens || a.num_tokens[b] > 0;
    int kept = -1;            // row of the block that this token completes
    if (BLOCKS && live) {
        const uint32_t pos = a.ctx ? max(a.ctx[b], 0) : 0, blk = pos / (uint32_t)a.block;
        if ((pos + 1) % (uint32_t)a.block == 0 && blk < (uint32_t)a.table_cols) kept = a.table[(size_t)b * a.table_cols + blk];
        if (kept >= a.pool_size || kept == dst) kept = -1;
    }
    if (!live && (dst < 0 || dst == src)) return;
    const size_t one = (size_t)DK * DV / 4, row = DV / 4;
    float4 *pool = (float4 *)a.state + part * CG + cg;

    // Every state load first; the inputs' loads and the decay overlap them.
    float4 s[RPT];
    if (src >= 0) {
        const float4 *S = pool + ((size_t)src * a.H + h) * one;
#pragma unroll
        for (int i = 0; i < RPT; ++i) s[i] = S[(size_t)(rg + i * RG) * row];
    } else {
#pragma unroll
        for (int i = 0; i < RPT; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (live) {
        const size_t tok = (size_t)b * a.H + h, ktok = (size_t)b * a.Hk + hk;
        if (tid < DK) {
            sK[tid] = to_f32(((const T *)a.k)[ktok * DK + tid]);
            sQ[tid] = to_f32(((const T *)a.q)[ktok * DK + tid]);
        }
        const float g = a.g[tok];
        const float al = expf(g < kGClampSoftplus ? kGClampSoftplus : g);
        __syncthreads();
        if (tid < 32) {
            float acc = 0.f;
            for (int c = tid; c < DK; c += 32) acc = fmaf(sK[c], sQ[c], acc);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
            if (tid == 0) sKQ = acc;
        }
        float4 sn = make_float4(0.f, 0.f, 0.f, 0.f), rd = sn;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kc = sK[rg + i * RG], qc = sQ[rg + i * RG];
            s[i].x *= al; s[i].y *= al; s[i].z *= al; s[i].w *= al;
            sn.x = fmaf(kc, s[i].x, sn.x); sn.y = fmaf(kc, s[i].y, sn.y);
            sn.z = fmaf(kc, s[i].z, sn.z); sn.w = fmaf(kc, s[i].w, sn.w);
            rd.x = fmaf(qc, s[i].x, rd.x); rd.y = fmaf(qc, s[i].y, rd.y);
            rd.z = fmaf(qc, s[i].z, rd.z); rd.w = fmaf(qc, s[i].w, rd.w);
        }
        sSeen[rg][cg] = sn;
        sRead[rg][cg] = rd;
        __syncthreads();
        if (tid < CG) {
            float4 ts = sSeen[0][tid], tr = sRead[0][tid];
#pragma unroll
            for (int r = 1; r < RG; ++r) {
                const float4 x = sSeen[r][tid], y = sRead[r][tid];
                ts.x += x.x; ts.y += x.y; ts.z += x.z; ts.w += x.w;
                tr.x += y.x; tr.y += y.y; tr.z += y.z; tr.w += y.w;
            }
            const float bt = a.beta[tok], kq = sKQ;
            const T *v = (const T *)a.v + tok * DV + part * COLS + 4 * tid;
            float4 d;
            d.x = bt * (to_f32(v[0]) - ts.x);
            d.y = bt * (to_f32(v[1]) - ts.y);
            d.z = bt * (to_f32(v[2]) - ts.z);
            d.w = bt * (to_f32(v[3]) - ts.w);
            sD[tid] = d;
            if (a.o) {
                T *o = (T *)a.o + tok * DV + part * COLS + 4 * tid;
                o[0] = from_f32<T>(a.scale * fmaf(kq, d.x, tr.x));
                o[1] = from_f32<T>(a.scale * fmaf(kq, d.y, tr.y));
                o[2] = from_f32<T>(a.scale * fmaf(kq, d.z, tr.z));
                o[3] = from_f32<T>(a.scale * fmaf(kq, d.w, tr.w));
            }
        }
        __syncthreads();
    }
    const float4 d = live ? sD[cg] : make_float4(0.f, 0.f, 0.f, 0.f);
    auto store = [&](int slot) {
        float4 *S = pool + ((size_t)slot * a.H + h) * one;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kc = live ? sK[rg + i * RG] : 0.f;
            S[(size_t)(rg + i * RG) * row] =
                make_float4(fmaf(kc, d.x, s[i].x), fmaf(kc, d.y, s[i].y), fmaf(kc, d.z, s[i].z),
                            fmaf(kc, d.w, s[i].w));
        }
    };
    if (dst >= 0) store(dst);
    if (BLOCKS && kept >= 0) store(kept);
}

template <int DK, int DV, typename T>
cudaError_t launch_typed(const GdrArgs &a, cudaStream_t stream)
{
    const int64_t blocks = (int64_t)a.num_seqs * a.H;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    // Few states: 32 columns per CTA.  Device time of 32 / 96 / 160 / 192 / 288 states of
    // 128 x 128, split: 3.2 / 5.9 / 7.2 / 8.3 / 10.6 us; whole: 4.2 / 6.2 / 8.5 / 8.7 / 9.9 us.
    auto launch = [&](auto *kernel, int64_t ctas) { kernel<<<(unsigned)ctas, kThreads, 0, stream>>>(a); };
    if (DV > 32 && blocks < 3 * kSms / 2)
        launch(a.block > 0 ? gdr_step_kernel<DK, DV, 32, T, true> : gdr_step_kernel<DK, DV, 32, T, false>,
               blocks * (DV / 32));
    else
        launch(a.block > 0 ? gdr_step_kernel<DK, DV, DV, T, true> : gdr_step_kernel<DK, DV, DV, T, false>, blocks);
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

cudaError_t launch_gdr_step(const GdrArgs &a, cudaStream_t stream)
{
    return a.bf16 ? launch_dk<__nv_bfloat16>(a, stream) : launch_dk<float>(a, stream);
}

}  // namespace kda
