// Chunked gated delta rule on tcgen05 tensor cores (bf16 operands, fp32
// accumulation, dk = dv = 128), one kernel.
//
// Within a chunk of 64 tokens (r, s; G the inclusive running log-decay from the
// chunk start, one number per token) the recurrence unrolls to
//   A = strictly_lower(Diag(beta) (K K^T) o D),   P = lower((Q K^T) o D),
//   D_rs = e^{G_r - G_s},   T = (I + A)^{-1},
//   U = T Diag(beta) V,   W = T Diag(beta e^G) K,   E = U - W S,
//   O = scale (Diag(e^G) Q S + P E),   S <- e^{G_C} S + (Diag(e^{G_C - G}) K)^T E.
// Every decay is one scalar per token (pair), so it folds into T's columns, E's
// columns and Q's rows; K and V enter the products as their TMA tiles.  All
// factors e^{G_r - G_s}, r >= s, are formed without a reciprocal and are at most
// 1 for g <= 0.
//
// One CTA of 23 warps owns a (sequence, value head) and walks its chunks with the
// fp32 state transposed in tensor memory.  Nothing goes through HBM but q, k, v,
// g, beta, o and the state rows.  Roles:
//   chain (warps 0-7)    E^T from its accumulator to bf16 operands (E for the
//                        outputs, e^{G_C - G} E for the state); S^T to its bf16
//                        copy, then the fp32 master times the next e^{G_C};
//   intra (warps 8-15)   two groups, even and odd chunks: A and P from the accumulator
//                        with their decays, T by 16 x 16 forward substitution and two
//                        block doublings (tf32 mma), T's two bf16 operands;
//   aux   (warps 16-19)  Q <- e^G Q in place, W^T from its accumulator to a bf16
//                        operand, O^T to o;
//   issue (warps 20, 21) the products of the state chain; A, P and W's products;
//   load  (warp 22)      TMA tiles, and the decay tables of a chunk (a warp scan).
// Products (TMEM accumulators in brackets), chunk c:
//   [AP] = [K; Q] K^T;  [W^T] = K^T (-T Diag(beta e^G))^T;  [E^T] = V^T (T Diag(beta))^T
//   [E^T] += S^T (-W)^T;  [O^T] = S^T (e^G Q)^T
//   [S^T] += (e^{G_C - G} E)^T K;  [O^T] += E^T P^T
// K^T, V^T and W^T are MN-major operands, so no tile is ever transposed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstring>

#include "kda_common.cuh"
#include "kda_gdr.h"
#include "kda_prefill_tc.h"
#include "tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kD = 128, kC = 64;              // head size, chunk
constexpr uint64_t kWaitNs = 2000000000ull;   // per-wait limit: 2 s
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kChainThreads = 256, kGroupThreads = 128, kAuxThreads = 128;
constexpr int kIntraWarp = 8, kAuxWarp = 16, kIssueWarp = 20, kIssue2Warp = 21, kLoadWarp = 22;
constexpr int kThreads = (kLoadWarp + 1) * 32;

// Shared memory (offsets from a 1024-aligned base).  A K/Q stage is
// [k K0 | q K0 | k K1 | q K1], 8 KiB each (64 rows x 128 B, 128-byte swizzle): the
// 128-row operand [K; Q] per half of 64 channels.  V: two halves of 8 KiB.
constexpr uint32_t kKQStage = 32768, kVStage = 16384;
constexpr int kKQStages = 3, kVStages = 2;
constexpr uint32_t kOffV = kKQStages * kKQStage;
constexpr uint32_t kOffW = kOffV + kVStages * kVStage;   // W^T: 128 channels x 64 tokens
constexpr uint32_t kOffP = kOffW + 16384;                // P: 64 x 64, two buffers
constexpr uint32_t kOffT1 = kOffP + 2 * 8192;            // -T Diag(beta e^G): 64 x 64
constexpr uint32_t kOffT2 = kOffT1 + 8192;               // T Diag(beta)
constexpr uint32_t kOffM = kOffT2 + 8192;                // per intra group: fp32 blocks, see kMBlock
// A's 32 x 32 diagonal blocks (then T's) and its lower-left block, rows padded to 36.
constexpr int kLd = 36, kMBlock = 32 * kLd;
constexpr uint32_t kMGroup = 3 * kMBlock * 4;
constexpr uint32_t kOffO = (kOffM + 2 * kMGroup + 1023) / 1024 * 1024;   // output staging, 4 KiB a warp
constexpr uint32_t kSmem = kOffO + 4 * 4096 + 1024;

// TMEM columns.
constexpr uint32_t kTS = 0;      // S^T, fp32 [dv][dk]
constexpr uint32_t kTSb = 128;   // its bf16 copy
constexpr uint32_t kTE = 192;    // E^T accumulator [dv][token]
constexpr uint32_t kTEo = 256;   // E^T bf16, for the outputs
constexpr uint32_t kTEs = 288;   // e^{G_C - G} E^T bf16, for the state
constexpr uint32_t kTO = 320;    // O^T accumulator
constexpr uint32_t kTAP = 384;   // A and P accumulators (rows 0-63, 64-127)
constexpr uint32_t kTW = 448;    // W^T accumulator [dk][token]

struct Bars {
    uint64_t kq_full[kKQStages], kq_empty[kKQStages], gate_full[kKQStages];
    uint64_t v_full[kVStages], v_empty[kVStages];   // v_empty: E^T = V^T T.. done (T too)
    uint64_t ap_full[2], o_full[2], w_full[2], prep[2];
    uint64_t ap_tfree, t_ready, w_tfree, w_ready;
    uint64_t s_ready, e_ready, decayed, e_full, s_full, o_free;
    uint64_t drain[2];
};

// Decay tables of a chunk (base-2 logarithms), one per K/Q stage.
struct __align__(16) Gate {
    float G[kC];      // running log-decay
    float f[kC];      // 2^(G at the end of the token's 16-token tile - G)
    float eG[kC];     // 2^G
    float beta[kC];
    float nbe[kC];    // -beta 2^G
    float tail[kC];   // 2^(G_C - G)
    float eGC;        // 2^G_C
    int steep;        // some tile decays by more than 2^-100: no factored form there
    int pad[2];
};

struct Params {
    GdrArgs a;
    bool ordered;
    uint16_t order[kGdrMaxOrder];   // sequence of launch position i, longest first
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}
__device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t y;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
    return y;
}
// D (+)= A B, one 16 x 8 x 8 tile: a = (row g, k t), (g + 8, t), (g, t + 4), (g + 8, t + 4);
// b = (k t, col g), (t + 4, g); d = (g, 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1), with
// g = lane / 4, t = lane % 4.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Barrier over one intra group; true when any of its threads passed true.
__device__ __forceinline__ bool group_sync_any(int group, bool pred) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.red.or.pred q, %2, 128, p;\n"
                 " selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r) : "r"((uint32_t)pred), "r"(1 + group) : "memory");
    return r != 0;
}
__device__ __forceinline__ void tma_tile(void *smem_dst, const CUtensorMap *map, int x, int h, int t0,
                                         uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(t0),
          "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *map, const void *smem_src, int x, int h, int t0) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(t0), "r"(smem_u32(smem_src))
                 : "memory");
}
__device__ __forceinline__ void named_timeout(int32_t *status) {
    atomicCAS(status, 0, (int32_t)KDA_TC_TIMEOUT_CODE);
}

// Off-diagonal block of the inverse of a lower-triangular matrix from its inverted diagonal
// blocks: Z = (T_ii A_ij) T_jj (the caller negates), all blocks W x W with leading dimension
// kLd.  This warp forms the 16 rows from rr, of them NT 8-column tiles from column n0.
template <int W, int NT>
__device__ __forceinline__ void block_product(const float *Ti, const float *A, const float *Tj, int rr, int n0,
                                              int lane, float (&z)[NT][4]) {
    const int g = lane >> 2, t = lane & 3;
    float y[W / 8][4];
#pragma unroll
    for (int n = 0; n < W / 8; ++n) y[n][0] = y[n][1] = y[n][2] = y[n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < W; k += 8) {
        if (k >= rr + 16) break;    // T_ii is lower triangular
        uint32_t a[4];
        const float *p = Ti + (rr + g) * kLd + k + t;
        a[0] = tf32(p[0]); a[1] = tf32(p[8 * kLd]); a[2] = tf32(p[4]); a[3] = tf32(p[8 * kLd + 4]);
        const float *q = A + (k + t) * kLd + g;
#pragma unroll
        for (int n = 0; n < W / 8; ++n) mma_tf32(y[n], a, tf32(q[8 * n]), tf32(q[4 * kLd + 8 * n]));
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) z[n][0] = z[n][1] = z[n][2] = z[n][3] = 0.f;
    // Y's accumulators are the A operand with the contraction index permuted: slot t is
    // column 2t, slot t + 4 is column 2t + 1; B reads its rows in the same order.
#pragma unroll
    for (int k = 0; k < W / 8; ++k) {
        const uint32_t a[4] = {tf32(y[k][0]), tf32(y[k][2]), tf32(y[k][1]), tf32(y[k][3])};
        const float *q = Tj + (8 * k + 2 * t) * kLd + n0 + g;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (8 * k + 7 >= n0 + 8 * n) mma_tf32(z[n], a, tf32(q[8 * n]), tf32(q[kLd + 8 * n]));
    }
}

__global__ void __launch_bounds__(kThreads, 1)
gdr_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                 const __grid_constant__ Params prm)
{
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    __shared__ Bars bars;
    __shared__ Gate gates[kKQStages];
    __shared__ uint32_t tbase;
    const GdrArgs &a = prm.a;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pos = blockIdx.x / a.H, h = blockIdx.x % a.H, hk = h / (a.H / a.Hk);
    const int n = prm.ordered ? prm.order[pos] : pos;
    const int tbeg = max(a.cu[n], 0), len = max(min(a.cu[n + 1], a.total_tokens) - tbeg, 0);
    const int ctx = a.ctx ? max(a.ctx[n], 0) : 0;
    int src = a.src ? a.src[n] : -1, dst = a.dst ? a.dst[n] : -1;
    if (!a.state || src < 0 || src >= a.pool_size) src = -1;
    if (!a.state || dst < 0 || dst >= a.pool_size) dst = -1;
    auto row_of = [&](int slot) { return a.state + ((size_t)slot * a.H + h) * kD * kD; };

    if (len == 0) {   // the state passes through
        if (dst >= 0 && dst != src) {
            float4 *to = (float4 *)row_of(dst);
            const float4 *from = src >= 0 ? (const float4 *)row_of(src) : nullptr;
            for (int e = tid; e < kD * kD / 4; e += kThreads)
                to[e] = from ? from[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }
    // Chunks end at multiples of 64 of the absolute position when block rows are
    // wanted (block sizes are multiples of 64), so that each block ends a chunk.
    const int off = a.block > 0 ? ctx % kC : 0;
    const int nch = (int)(((int64_t)off + len + kC - 1) / kC);
    auto begin_of = [&](int c) { return c == 0 ? 0 : c * kC - off; };
    auto len_of = [&](int c) { return min((c + 1) * kC - off, len) - begin_of(c); };

    if (tid == 0) {
        for (int s = 0; s < kKQStages; ++s) {
            mbar_init(&bars.kq_full[s], 1);
            mbar_init(&bars.kq_empty[s], 1);
            mbar_init(&bars.gate_full[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars.v_full[s], 1);
            mbar_init(&bars.v_empty[s], 1);
            mbar_init(&bars.ap_full[s], 1);
            mbar_init(&bars.o_full[s], 1);
            mbar_init(&bars.w_full[s], 1);
            mbar_init(&bars.prep[s], kGroupThreads);
            mbar_init(&bars.drain[s], 1);
        }
        mbar_init(&bars.ap_tfree, kGroupThreads);
        mbar_init(&bars.t_ready, kGroupThreads);
        mbar_init(&bars.w_tfree, kAuxThreads);
        mbar_init(&bars.w_ready, kAuxThreads);
        mbar_init(&bars.s_ready, kChainThreads);
        mbar_init(&bars.e_ready, kChainThreads);
        mbar_init(&bars.decayed, kChainThreads);
        mbar_init(&bars.e_full, 1);
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.o_free, kAuxThreads);
        fence_mbar_init();
    }
    // The upper right quadrants of P and T's operands are zero in every chunk.
    for (int e = tid; e < 4 * 32 * 4; e += kThreads) {
        const uint32_t img = e < 256 ? kOffP + (e >> 7) * 8192 : (e < 384 ? kOffT1 : kOffT2);
        *(uint4 *)(sm + img + sw128_offset((e >> 2) & 31, 32 + 8 * (e & 3), 64)) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == 0) { tmem_alloc(&tbase, 512); tmem_relinquish(); }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tb = tbase;
    const uint32_t lq = 32 * (warp & 3);   // this warp's TMEM lanes

    // Bounded wait of a whole warp; on expiry the timeout is recorded and the role
    // leaves its loop (the others run into their own limits).
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        // The timer is read only once a try has failed: a hand-off that is ready costs
        // one try_wait.
        bool r = mbar_try_wait(bar, parity & 1);
        if (!__all_sync(0xffffffffu, r)) {
            r = mbar_wait(bar, parity & 1, globaltimer_ns() + kWaitNs);
            if (!r) named_timeout(a.status);
            return __all_sync(0xffffffffu, r) != 0;
        }
        return true;
    };

    if (warp < kIntraWarp) {
        // ------------------------------------------------------------- chain --
        const int j = tid & 127, hh = warp >> 2;   // value channel; half of tokens / key channels
        uint32_t ra[32], rb[32];
        bool ok = wait(&bars.gate_full[0], 0);
        const float *S0 = src >= 0 ? row_of(src) + (size_t)(64 * hh) * kD + j : nullptr;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint32_t x[32], y[16];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = S0 ? __float_as_uint(S0[(size_t)(32 * p + i) * kD]) : 0u;
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            tmem_st16(tmem_addr(tb, lq, kTSb + 32 * hh + 16 * p), y);
            const float d = gates[0].eGC;
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * d);
            tmem_st32(tmem_addr(tb, lq, kTS + 64 * hh + 32 * p), x);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars.s_ready);
        mbar_arrive(&bars.decayed);
        for (int c = 0; c < nch && ok; ++c) {
            // E^T of this half's 32 tokens -> bf16, plain and with the decay to the chunk end.
            ok = wait(&bars.e_full, c);
            if (!ok) break;
            tc_fence_after_sync();
            tmem_ld32(tmem_addr(tb, lq, kTE + 32 * hh), ra);
            tmem_ld_wait();
            {
                const float4 *tail = (const float4 *)&gates[c % kKQStages].tail[32 * hh];
                uint32_t eo[16], es[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 d = tail[i];
                    const float e0 = __uint_as_float(ra[4 * i]), e1 = __uint_as_float(ra[4 * i + 1]);
                    const float e2 = __uint_as_float(ra[4 * i + 2]), e3 = __uint_as_float(ra[4 * i + 3]);
                    es[2 * i] = pack(e0 * d.x, e1 * d.y);
                    es[2 * i + 1] = pack(e2 * d.z, e3 * d.w);
                    eo[2 * i] = pack(e0, e1);
                    eo[2 * i + 1] = pack(e2, e3);
                }
                tmem_st16(tmem_addr(tb, lq, kTEs + 16 * hh), es);
                tmem_st16(tmem_addr(tb, lq, kTEo + 16 * hh), eo);
            }
            tmem_st_wait();
            tc_fence_before_sync();
            mbar_arrive(&bars.e_ready);
            ok = wait(&bars.s_full, c);
            if (!ok) break;
            tc_fence_after_sync();
            const bool last = c + 1 == nch;
            tmem_ld32(tmem_addr(tb, lq, kTS + 64 * hh), ra);
            tmem_ld32(tmem_addr(tb, lq, kTS + 64 * hh + 32), rb);
            tmem_ld_wait();
            if (!last) {
                uint32_t y[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = pack(__uint_as_float(ra[2 * i]), __uint_as_float(ra[2 * i + 1]));
                tmem_st16(tmem_addr(tb, lq, kTSb + 32 * hh), y);
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = pack(__uint_as_float(rb[2 * i]), __uint_as_float(rb[2 * i + 1]));
                tmem_st16(tmem_addr(tb, lq, kTSb + 32 * hh + 16), y);
                tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(&bars.s_ready);
            }
            // State rows: a block that ends here, and the last state.
            const int64_t done = (int64_t)ctx + begin_of(c) + len_of(c);
            int row = -1;
            if (a.block > 0 && done % a.block == 0 && done / a.block <= a.table_cols)
                row = a.table[(size_t)n * a.table_cols + done / a.block - 1];
            if (row >= a.pool_size) row = -1;
            for (int w = 0; w < 2; ++w) {
                const int to = w == 0 ? row : (last ? dst : -1);
                if (to < 0) continue;
                float *Sf = row_of(to) + (size_t)(64 * hh) * kD + j;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    Sf[(size_t)i * kD] = __uint_as_float(ra[i]);
                    Sf[(size_t)(32 + i) * kD] = __uint_as_float(rb[i]);
                }
            }
            if (last) break;
            // Off the critical path: the master times the next chunk's decay.
            ok = wait(&bars.gate_full[(c + 1) % kKQStages], (c + 1) / kKQStages);
            if (!ok) break;
            const float d = gates[(c + 1) % kKQStages].eGC;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                ra[i] = __float_as_uint(__uint_as_float(ra[i]) * d);
                rb[i] = __float_as_uint(__uint_as_float(rb[i]) * d);
            }
            tmem_st32(tmem_addr(tb, lq, kTS + 64 * hh), ra);
            tmem_st32(tmem_addr(tb, lq, kTS + 64 * hh + 32), rb);
            tmem_st_wait();
            tc_fence_before_sync();
            mbar_arrive(&bars.decayed);
        }
    } else if (warp < kAuxWarp) {
        // ------------------------------------------------------------- intra --
        const int group = (warp - kIntraWarp) >> 2, wq = warp & 3, half = wq & 1;
        const int it = 32 * wq + lane, r = it & 63;
        const bool is_p = wq >= 2;
        float *D0 = (float *)(sm + kOffM + group * kMGroup), *D1 = D0 + kMBlock, *X = D1 + kMBlock;
        bool ok = true;
        // A partial chunk's rows past its last token (another sequence's, or unwritten
        // ones) become zeros in K and V, before any product reads the tiles.
        auto prepare = [&](int c) {
            const int m = len_of(c);
            if (m < kC) {
                ok = ok && wait(&bars.kq_full[c % kKQStages], c / kKQStages) &&
                     wait(&bars.v_full[c % kVStages], c / kVStages);
                uint8_t *kt = sm + (c % kKQStages) * kKQStage, *vt = sm + kOffV + (c % kVStages) * kVStage;
                for (int e = it; e < (kC - m) * 8; e += kGroupThreads) {
                    const uint32_t at = (uint32_t)(m + (e >> 3)) * 128u + (uint32_t)(e & 7) * 16u;
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    *(uint4 *)(kt + at) = zero;
                    *(uint4 *)(kt + 16384 + at) = zero;
                    *(uint4 *)(vt + at) = zero;
                    *(uint4 *)(vt + 8192 + at) = zero;
                }
                fence_proxy_async_smem();
            }
            mbar_arrive(&bars.prep[c & 1]);
        };
        if (group < nch) prepare(group);
        for (int c = group; c < nch; c += 2) {
            const Gate &gt = gates[c % kKQStages];
            ok = ok && wait(&bars.gate_full[c % kKQStages], c / kKQStages);
            if (c >= 2) {   // P's buffer and this group's blocks: read by chunk c - 2's products
                ok = ok && wait(&bars.o_full[c & 1], (c >> 1) - 1);
                ok = ok && wait(&bars.w_full[c & 1], (c >> 1) - 1);
            }
            const float Gr = gt.G[r], br = is_p ? 1.f : gt.beta[r];
            // Row factors: the decay from a tile's end to this row (below 1 for earlier
            // tiles; up to 2^100 for its own, where f undoes it).
            const float n0 = br * ex2(Gr - gt.G[32 * half + 15]), n1 = br * ex2(Gr - gt.G[32 * half + 31]);
            const float far0 = half ? br * ex2(Gr - gt.G[15]) : 0.f, far1 = half ? br * ex2(Gr - gt.G[31]) : 0.f;
            const int lim = (is_p ? r : r - 1) - 32 * half;    // last column kept of the near 32
            const bool steep = gt.steep != 0;
            ok = ok && wait(&bars.ap_full[c & 1], c >> 1);
            tc_fence_after_sync();
            uint8_t *img = sm + kOffP + (c & 1) * 8192;
#pragma unroll
            for (int part = 0; part < 2; ++part) {   // 0: the near 32 columns; 1: columns 0-31 of rows 32-63
                if (part == 1 && !half) break;
                uint32_t v[32];
                const int s0 = part == 0 ? 32 * half : 0;
                tmem_ld32(tmem_addr(tb, lq, kTAP + s0), v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 f4 = *(const float4 *)&gt.f[s0 + i];
                    const float fs[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float row = part == 0 ? (i < 16 ? n0 : n1) : (i < 16 ? far0 : far1);
                        float x = __uint_as_float(v[i + u]);
                        if (part == 0 && steep) x = x * br * ex2(Gr - gt.G[s0 + i + u]);
                        else x = x * (row * fs[u]);
                        v[i + u] = part == 1 || i + u <= lim ? __float_as_uint(x) : 0u;
                    }
                }
                if (is_p) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint4 w;
                        w.x = pack(__uint_as_float(v[8 * i]), __uint_as_float(v[8 * i + 1]));
                        w.y = pack(__uint_as_float(v[8 * i + 2]), __uint_as_float(v[8 * i + 3]));
                        w.z = pack(__uint_as_float(v[8 * i + 4]), __uint_as_float(v[8 * i + 5]));
                        w.w = pack(__uint_as_float(v[8 * i + 6]), __uint_as_float(v[8 * i + 7]));
                        *(uint4 *)(img + sw128_offset(r, s0 + 8 * i, 64)) = w;
                    }
                } else {
                    float *m = (part == 1 ? X : (half ? D1 : D0)) + (r & 31) * kLd;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *(uint4 *)&m[i] = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            tc_fence_before_sync();
            mbar_arrive(&bars.ap_tfree);
            // The next chunk of this group: its product may start unless its tiles need zeros.
            if (c + 2 < nch && len_of(c + 2) == kC) mbar_arrive(&bars.prep[c & 1]);
            if (group_sync_any(group, !ok)) break;
            // Inverse of the two 32 x 32 diagonal blocks, one warp each: half a warp solves a
            // 16 x 16 block, lane j its column j, four unknowns at a time; then the block
            // between them.
            if (!is_p) {
                float *Dw = half ? D1 : D0;
                float *B = Dw + 16 * (lane >> 4) * (kLd + 1);
                const int j = lane & 15, g = lane >> 2, t = lane & 3;
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.f : 0.f;
#pragma unroll
                for (int m0 = 0; m0 < 16; m0 += 4) {
#pragma unroll
                    for (int i = m0 + 1; i < 16; ++i) {
                        const float4 l = *(const float4 *)&B[i * kLd + m0];
                        const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            if (m0 + m < i) x[i] = fmaf(-lv[m], x[m0 + m], x[i]);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) B[i * kLd + j] = x[i];
                __syncwarp();
                float z[2][4];
                block_product<16, 2>(Dw + 16 * (kLd + 1), Dw + 16 * kLd, Dw, 0, 0, lane, z);
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float *p = Dw + (16 + g) * kLd + 8 * q + 2 * t;
                    *(float2 *)p = make_float2(-z[q][0], -z[q][1]);
                    *(float2 *)(p + 8 * kLd) = make_float2(-z[q][2], -z[q][3]);
                }
            }
            // T's operands: free once the products of chunk c - 1 have read them.
            if (c > 0) {
                ok = ok && wait(&bars.w_full[(c - 1) & 1], (c - 1) >> 1);
                ok = ok && wait(&bars.v_empty[(c - 1) & 1], (c - 1) >> 1);
            }
            if (group_sync_any(group, !ok)) break;
            {   // rows 32-63, columns 0-31: 16 x 16 per warp, straight to the operands
                const int rr = 16 * half, nc = 16 * (wq >> 1), g = lane >> 2, t = lane & 3;
                float z[2][4];
                block_product<32, 2>(D1, X, D0, rr, nc, lane, z);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int col = nc + 8 * q + 2 * t;
                    const float2 nb = *(const float2 *)&gt.nbe[col], be = *(const float2 *)&gt.beta[col];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t at = sw128_offset(32 + rr + g + 8 * u, col, 64);
                        *(uint32_t *)(sm + kOffT1 + at) = pack(-z[q][2 * u] * nb.x, -z[q][2 * u + 1] * nb.y);
                        *(uint32_t *)(sm + kOffT2 + at) = pack(-z[q][2 * u] * be.x, -z[q][2 * u + 1] * be.y);
                    }
                }
            }
            {   // the diagonal blocks: half of the threads per operand, a row each
                const float *m = (r < 32 ? D0 : D1) + (r & 31) * kLd;
                const float *colf = (is_p ? gt.beta : gt.nbe) + (r & 32);
                uint8_t *to = sm + (is_p ? kOffT2 : kOffT1);
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    const float4 x = *(const float4 *)&m[i], y = *(const float4 *)&m[i + 4];
                    const float4 p = *(const float4 *)&colf[i], q = *(const float4 *)&colf[i + 4];
                    *(uint4 *)(to + sw128_offset(r, (r & 32) + i, 64)) =
                        make_uint4(pack(x.x * p.x, x.y * p.y), pack(x.z * p.z, x.w * p.w),
                                   pack(y.x * q.x, y.y * q.y), pack(y.z * q.z, y.w * q.w));
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bars.t_ready);
            if (c + 2 < nch && len_of(c + 2) < kC) prepare(c + 2);
        }
    } else if (warp < kIssueWarp) {
        // --------------------------------------------------------------- aux --
        const int wq = warp & 3, it = 32 * wq + lane;
        uint8_t *ost = sm + kOffO + 4096 * wq;     // [64 tokens][32 channels] of this warp
        __nv_bfloat16 *o = (__nv_bfloat16 *)a.o;
        uint32_t xa[32], xb[32];
        auto output = [&](int c) {
            if (!wait(&bars.o_full[c & 1], c >> 1)) return false;
            tc_fence_after_sync();
            tmem_ld32(tmem_addr(tb, lq, kTO), xa);
            tmem_ld32(tmem_addr(tb, lq, kTO + 32), xb);
            tmem_ld_wait();
            tc_fence_before_sync();
            mbar_arrive(&bars.o_free);
            const int m = len_of(c), t0 = tbeg + begin_of(c);
            if (lane == 0) bulk_wait_read<0>();    // the previous chunk's store has read the tile
            __syncwarp();
            __nv_bfloat16 *ot = (__nv_bfloat16 *)ost + lane;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                ot[i * 32] = __float2bfloat16_rn(a.scale * __uint_as_float(xa[i]));
                ot[(i + 32) * 32] = __float2bfloat16_rn(a.scale * __uint_as_float(xb[i]));
            }
            if (m == kC) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) { tma_store(&tm_o, ost, 32 * wq, h, t0); bulk_commit(); }
            } else {       // a partial chunk: only its own rows
                __syncwarp();
                for (int e = lane; e < m * 4; e += 32)
                    *(uint4 *)(o + ((size_t)(t0 + (e >> 2)) * a.H + h) * kD + 32 * wq + 8 * (e & 3)) =
                        *(const uint4 *)(ost + e * 16);
                __syncwarp();
            }
            return true;
        };
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
            const int s = c % kKQStages;
            const Gate &gt = gates[s];
            // Q <- e^G Q in place, once A and P have read the raw tile.
            ok = wait(&bars.gate_full[s], c / kKQStages) && wait(&bars.kq_full[s], c / kKQStages) &&
                 wait(&bars.ap_full[c & 1], c >> 1);
            if (!ok) break;
            {
                const int row = it >> 1;
                uint8_t *p = sm + s * kKQStage + 8192 + (it & 1) * 16384 + row * 128;
                const float d = gt.eG[row];
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = *(const uint4 *)(p + ((i ^ (row & 7)) << 4));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t *u = (uint32_t *)&w[i];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = unpack(u[k]);
                        u[k] = pack(f.x * d, f.y * d);
                    }
                    *(uint4 *)(p + ((i ^ (row & 7)) << 4)) = w[i];
                }
            }
            // W^T (negated) of key channel 32 wq + lane: 64 tokens -> one 128-byte row.
            ok = wait(&bars.w_full[c & 1], c >> 1);
            if (!ok) break;
            tc_fence_after_sync();
            tmem_ld32(tmem_addr(tb, lq, kTW), xa);
            tmem_ld32(tmem_addr(tb, lq, kTW + 32), xb);
            tmem_ld_wait();
            tc_fence_before_sync();
            mbar_arrive(&bars.w_tfree);
            if (c > 0) ok = wait(&bars.e_full, c - 1);   // the image: read by chunk c - 1's product
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint4 w;
                w.x = pack(__uint_as_float(xa[8 * i]), __uint_as_float(xa[8 * i + 1]));
                w.y = pack(__uint_as_float(xa[8 * i + 2]), __uint_as_float(xa[8 * i + 3]));
                w.z = pack(__uint_as_float(xa[8 * i + 4]), __uint_as_float(xa[8 * i + 5]));
                w.w = pack(__uint_as_float(xa[8 * i + 6]), __uint_as_float(xa[8 * i + 7]));
                *(uint4 *)(sm + kOffW + sw128_offset(it, 8 * i, 128)) = w;
                w.x = pack(__uint_as_float(xb[8 * i]), __uint_as_float(xb[8 * i + 1]));
                w.y = pack(__uint_as_float(xb[8 * i + 2]), __uint_as_float(xb[8 * i + 3]));
                w.z = pack(__uint_as_float(xb[8 * i + 4]), __uint_as_float(xb[8 * i + 5]));
                w.w = pack(__uint_as_float(xb[8 * i + 6]), __uint_as_float(xb[8 * i + 7]));
                *(uint4 *)(sm + kOffW + sw128_offset(it, 32 + 8 * i, 128)) = w;
            }
            fence_proxy_async_smem();
            mbar_arrive(&bars.w_ready);
            if (c > 0) ok = output(c - 1);
        }
        if (ok) output(nch - 1);
        if (lane == 0) bulk_wait<0>();   // every store has completed before the CTA exits
        __syncwarp();
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------------------- issue --
        const bool leader = elect_one();
        const uint32_t id64 = idesc_bf16_f32(128, 64), id128 = idesc_bf16_f32(128, 128);
        const uint32_t wimg = smem_u32(sm + kOffW), t2 = smem_u32(sm + kOffT2);
        auto issue_u = [&](int c) {       // [E^T] = V^T (T Diag(beta))^T
            if (!wait(&bars.v_full[c & 1], c >> 1) || !wait(&bars.t_ready, c)) return false;
            tc_fence_after_sync();
            if (leader) {
                const uint64_t dv = desc_mnmajor_sw128(smem_u32(sm + kOffV + (c % kVStages) * kVStage), 8192);
                const uint64_t dt = desc_kmajor_sw128(t2);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_ss(tmem_addr(tb, 0, kTE), dv + ks * (2048 >> 4), dt + ks * (32 >> 4), id64 | kIdescMnA, ks > 0);
                mma_commit(&bars.v_empty[c & 1]);
            }
            __syncwarp();
            return true;
        };
        bool ok = issue_u(0);
        for (int c = 0; c < nch && ok; ++c) {
            const int s = c % kKQStages;
            const uint32_t st = smem_u32(sm + s * kKQStage), sb = tmem_addr(tb, 0, kTSb);
            const uint64_t dW = desc_mnmajor_sw128(wimg, 16384), dQ = desc_kmajor_sw128(st + 8192);
            const uint64_t dK = desc_mnmajor_sw128(st, 16384), dP = desc_kmajor_sw128(smem_u32(sm + kOffP + (c & 1) * 8192));
            ok = wait(&bars.kq_full[s], c / kKQStages) && wait(&bars.w_ready, c) && wait(&bars.s_ready, c);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ts(tmem_addr(tb, 0, kTE), sb + 8 * ks, dW + ks * (2048 >> 4), id64 | kIdescMnB, true);
                mma_commit(&bars.e_full);
            }
            __syncwarp();
            if (c > 0 && !wait(&bars.o_free, c - 1)) break;
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ts(tmem_addr(tb, 0, kTO), sb + 8 * ks, dQ + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4), id64, ks > 0);
            }
            __syncwarp();
            ok = wait(&bars.e_ready, c) && wait(&bars.decayed, c);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_ts(tmem_addr(tb, 0, kTS), tmem_addr(tb, 0, kTEs + 8 * ks), dK + ks * (2048 >> 4),
                           id128 | kIdescMnB, true);
                mma_commit(&bars.s_full);
                mma_commit(&bars.kq_empty[s]);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_ts(tmem_addr(tb, 0, kTO), tmem_addr(tb, 0, kTEo + 8 * ks), dP + ks * (32 >> 4), id64, true);
                mma_commit(&bars.o_full[c & 1]);
            }
            __syncwarp();
            if (c + 1 < nch) ok = issue_u(c + 1);
        }
        if (leader) {
            mma_commit(&bars.drain[1]);
            mbar_wait(&bars.drain[1], 0, globaltimer_ns() + kWaitNs);
        }
        __syncwarp();
    } else if (warp == kIssue2Warp) {
        // --------------------------------------------- issue: A, P and W --
        const bool leader = elect_one();
        const uint32_t t1 = smem_u32(sm + kOffT1);
        auto issue_ap = [&](int c) {
            const int s = c % kKQStages;
            if (!wait(&bars.kq_full[s], c / kKQStages) || !wait(&bars.prep[c & 1], c >> 1)) return false;
            if (c > 0 && !wait(&bars.ap_tfree, c - 1)) return false;
            tc_fence_after_sync();
            if (leader) {
                const uint64_t d = desc_kmajor_sw128(smem_u32(sm + s * kKQStage));
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint64_t dk = d + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
                    mma_ss(tmem_addr(tb, 0, kTAP), dk, dk, idesc_bf16_f32(128, 64), ks > 0);
                }
                mma_commit(&bars.ap_full[c & 1]);
            }
            __syncwarp();
            return true;
        };
        bool ok = issue_ap(0) && (nch < 2 || issue_ap(1));
        for (int c = 0; c < nch && ok; ++c) {
            ok = wait(&bars.t_ready, c) && (c == 0 || wait(&bars.w_tfree, c - 1));
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {   // [W^T] = K^T (-T Diag(beta e^G))^T
                const uint64_t dk = desc_mnmajor_sw128(smem_u32(sm + (c % kKQStages) * kKQStage), 16384);
                const uint64_t dt = desc_kmajor_sw128(t1);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_ss(tmem_addr(tb, 0, kTW), dk + ks * (2048 >> 4), dt + ks * (32 >> 4),
                           idesc_bf16_f32(128, 64) | kIdescMnA, ks > 0);
                mma_commit(&bars.w_full[c & 1]);
            }
            __syncwarp();
            if (c + 2 < nch) ok = issue_ap(c + 2);
        }
        if (leader) {   // every product of this role has finished before the CTA may exit
            mma_commit(&bars.drain[0]);
            mbar_wait(&bars.drain[0], 0, globaltimer_ns() + kWaitNs);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------- load --
        const bool leader = elect_one();
        float g[2] = {0.f, 0.f}, be[2] = {0.f, 0.f};   // tokens 2 lane, 2 lane + 1 of the next chunk
        auto fetch = [&](int c) {
            const int m = len_of(c);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * lane + u;
                const size_t at = (size_t)(tbeg + begin_of(c) + t) * a.H + h;
                g[u] = t < m ? a.g[at] : 0.f;
                be[u] = t < m ? a.beta[at] : 0.f;
            }
        };
        fetch(0);
        int kq_loaded = 0, v_loaded = 0;
        for (int c = 0; c < nch; ++c) {
            const int s = c % kKQStages;
            if (c >= kKQStages && !wait(&bars.kq_empty[s], c / kKQStages - 1)) break;
            const int t0 = tbeg + begin_of(c);
            if (leader) {
                uint8_t *st = sm + s * kKQStage;
                mbar_arrive_expect_tx(&bars.kq_full[s], kKQStage);
                tma_tile(st, &tm_k, 0, hk, t0, &bars.kq_full[s]);
                tma_tile(st + 16384, &tm_k, 64, hk, t0, &bars.kq_full[s]);
                tma_tile(st + 8192, &tm_q, 0, hk, t0, &bars.kq_full[s]);
                tma_tile(st + 24576, &tm_q, 64, hk, t0, &bars.kq_full[s]);
            }
            ++kq_loaded;
            __syncwarp();
            if (c >= kVStages && !wait(&bars.v_empty[c & 1], (c >> 1) - 1)) break;
            if (leader) {
                uint8_t *vt = sm + kOffV + (c % kVStages) * kVStage;
                mbar_arrive_expect_tx(&bars.v_full[c & 1], kVStage);
                tma_tile(vt, &tm_v, 0, h, t0, &bars.v_full[c & 1]);
                tma_tile(vt + 8192, &tm_v, 64, h, t0, &bars.v_full[c & 1]);
            }
            ++v_loaded;
            __syncwarp();
            // Decay tables: two tokens per lane, an inclusive scan over the warp.
            float x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) x[u] = (g[u] < kGClampSoftplus ? kGClampSoftplus : g[u]) * kLog2e;
            const float pair = x[0] + x[1];
            float sum = pair;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += y;
            }
            const float tile_end = __shfl_sync(0xffffffffu, sum, lane | 7);
            const float GC = __shfl_sync(0xffffffffu, sum, 31);
            const float G0 = sum - x[1], G1 = sum;
            Gate &gt = gates[s];
            const float e0 = ex2(G0), e1 = ex2(G1);
            *(float2 *)&gt.G[2 * lane] = make_float2(G0, G1);
            *(float2 *)&gt.f[2 * lane] = make_float2(ex2(tile_end - G0), ex2(tile_end - G1));
            *(float2 *)&gt.eG[2 * lane] = make_float2(e0, e1);
            *(float2 *)&gt.beta[2 * lane] = make_float2(be[0], be[1]);
            *(float2 *)&gt.nbe[2 * lane] = make_float2(-be[0] * e0, -be[1] * e1);
            *(float2 *)&gt.tail[2 * lane] = make_float2(ex2(GC - G0), ex2(GC - G1));
            // Factored decays need every tile's range inside the fp32 exponent.
            const float tile_begin = __shfl_sync(0xffffffffu, G0, lane & 24);
            const bool steep = __any_sync(0xffffffffu, !(tile_begin - tile_end <= 100.f) || x[0] > 0.f || x[1] > 0.f);
            if (lane == 0) { gt.eGC = ex2(GC); gt.steep = steep; }
            __syncwarp();
            if (leader) mbar_arrive(&bars.gate_full[s]);
            if (c + 1 < nch) fetch(c + 1);
        }
        // Every tile has landed before the CTA may exit.
        if (leader) {
            for (int c = max(0, kq_loaded - kKQStages); c < kq_loaded; ++c)
                mbar_wait(&bars.kq_full[c % kKQStages], (c / kKQStages) & 1, globaltimer_ns() + kWaitNs);
            for (int c = max(0, v_loaded - kVStages); c < v_loaded; ++c)
                mbar_wait(&bars.v_full[c % kVStages], (c / kVStages) & 1, globaltimer_ns() + kWaitNs);
        }
        __syncwarp();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tb, 512);
}

}  // namespace

cudaError_t launch_gdr_tensor_core(const GdrArgs &a, cudaStream_t stream)
{
    const int64_t ctas = (int64_t)a.num_seqs * a.H;
    if (a.dk != kD || a.dv != kD || !a.bf16 || !a.cu || ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (ctas == 0) return cudaSuccess;
    cudaError_t err = cudaFuncSetAttribute(gdr_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (err != cudaSuccess) return err;
    CUtensorMap mq, mk, mv, mo;
    memset(&mq, 0, sizeof(mq));
    mk = mv = mo = mq;   // with no tokens no tile is read or written
    if (a.total_tokens > 0 &&
        (!tc_rows_map(&mq, a.q, a.total_tokens, a.Hk) || !tc_rows_map(&mk, a.k, a.total_tokens, a.Hk) ||
         !tc_rows_map(&mv, a.v, a.total_tokens, a.H) || !tc_out_map(&mo, a.o, a.total_tokens, a.H, 32)))
        return cudaErrorInvalidValue;
    // Longest sequences first (they set the end of the launch); the host offsets only
    // order the CTAs, each of which reads its own bounds on the device.
    Params p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    if (a.cu_host && a.num_seqs > 1 && a.num_seqs <= kGdrMaxOrder) {
        p.ordered = true;
        for (int i = 0; i < a.num_seqs; ++i) {     // insertion by length, ties by index
            const int32_t L = a.cu_host[i + 1] - a.cu_host[i];
            int at = i;
            while (at > 0) {
                const int m = p.order[at - 1];
                if (a.cu_host[m + 1] - a.cu_host[m] >= L) break;
                p.order[at] = p.order[at - 1];
                --at;
            }
            p.order[at] = (uint16_t)i;
        }
    }
    gdr_chunk_kernel<<<(unsigned)ctas, kThreads, kSmem, stream>>>(mq, mk, mv, mo, p);
    return cudaGetLastError();
}

}  // namespace kda
