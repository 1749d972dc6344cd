// Chunked gated delta rule on tcgen05 tensor cores (bf16 operands, fp32
// accumulation, dk = dv = 128), one kernel.
//
// A chunk holds up to 64 tokens (r, s).  With G_r the log-decay accumulated from
// the chunk's second token to token r (G = 0 at the first), and the incoming state
// already multiplied by the first token's e^{g}, the unrolled recurrence is
//   E_r + sum_{s<r} beta_r (k_r . k_s) e^{G_r - G_s} E_s = beta_r (v_r - e^{G_r} S^T k_r),
//   o_r = scale (e^{G_r} S^T q_r + sum_{s<=r} (q_r . k_s) e^{G_r - G_s} E_s),
//   S <- e^{G_C} S + sum_s e^{G_C - G_s} k_s E_s^T.
// In the variables F_r = e^{-G_r} E_r every decay leaves the sums:
//   T = (I + strictly_lower(Diag(beta) K K^T))^{-1},  P = lower(Q K^T),
//   R_r = beta_r (e^{-G_r} v_r - S^T k_r),  F = T R,
//   o_r = scale e^{G_r} (Q S + P F)_r,  S <- e^{G_C} (S + K^T F),
// so one factor per token remains in R, one at the outputs and one at the state, and K and Q
// enter the products as their TMA tiles.  e^{-G} has to stay in the floating-point range: a
// chunk ends early, before the token at which e^{-G} would pass 2^192; up to 2^100 nothing is
// shifted, between them the chunk's scale is shifted down so that e^{-G} <= 2^100 (which leaves room
// for |v| up to 2^20).  What its first tokens read and write is then up to 2^-92 of its size and has
// 2^-34 of bf16's exponents left: values from 2^-20 on keep their bits behind steep decays and small
// betas too.  With a limit of 200 (208), v and S of the order of 2^-18 came out off by a third of
// their size (by 19 times) in single output rows.  32768 tokens x 96 heads of rates e^-5 .. e: 1.75 ms
// (200: 1.67, 208: 1.62, 184: 1.84, 168: 2.05, 100: 3.5).
// Relative accuracy is that of the decayed form otherwise: each term is scaled by a
// power it keeps to its use.
//
// Precision.  K and Q are exact operands.  The others on the state's path, S, R, T and F, are
// each the sum of two bf16 numbers (17 bits), and a product of two such sums leaves out only
// low x low: the state comes out within 4e-6 of the recurrence in 64 bits (2-norm), where
// single bf16 operands gave 2.5e-3.  Of the outputs' own products P and S take their high part
// alone: outputs within 2.4e-3, of which their rounding to bf16 is 1.7e-3 (S's low part too:
// 2.2e-3, and 3.25 instead of 3.15 us a chunk).
//
// One CTA of 32 warps owns a (sequence, value head) and walks its chunks with the fp32 state
// transposed in tensor memory.  Nothing goes through HBM but q, k, v, g, beta, o and the
// state rows.  Roles:
//   chain (warps 0-15)   S^T K^T to R^T, F^T, and S^T times its factor, each from its
//                        accumulator to two bf16 operands; the fp32 master;
//   intra (warps 16-23)  two groups, even and odd chunks: A and P from the accumulator,
//                        T by forward substitution in 8 x 8 blocks (fp32) and three block
//                        doublings (warp products of split fp16), T's two bf16 operands;
//   aux   (warps 24-27)  O^T to o;
//   issue (warp 28)      the products of the state chain;
//   load  (warps 29, 30) the K and Q tiles for A and P and their product; K, Q and V for the
//                        chain;
//   info  (warp 31)      chunk bounds and factors (a warp scan).
// K and Q are loaded twice (the second time from L2): A and P are formed up to three chunks
// ahead of the state, and a tile that stayed for both uses would sit idle in between.
// One chain takes 3.05 us a chunk alone and 3.1 us at 96 CTAs (32768 tokens x 96 heads of slow decay: 1.58 ms):
// the state's way through three products and three passes of the chain warps, about 6000 cycles,
// next to the other roles, which take as long (A and P wait for one accumulator).  Tried and
// slower: fewer, wider chain warps; register splits between roles; deeper tile rings in place of
// the second load; TMA stores of o; unrolled waits and loops (instruction cache).
// Products (TMEM accumulators in brackets), chunk c:
//   [AP] = [K; Q] K^T;  [DF] = S^T K^T;  [O^T] = S^T Q^T;  [DF] = R^T T^T;
//   [S^T] += F^T K;  [O^T] += F^T P^T
// K is an MN-major operand of the state's product, so no tile is ever transposed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstring>

#include "kda_common.cuh"
#include "kda_gdr.h"
#include "kda_gdr_split.h"
#include "kda_prefill_tc.h"
#include "tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kD = 128, kC = 64;              // head size, chunk
// A wait gives up after kTries tries, each of which sleeps at most kSuspendNs (or until the
// phase completes): between tens of milliseconds and two seconds, against hand-offs that
// take microseconds.
constexpr uint32_t kTries = 1u << 20, kSuspendNs = 2000;
constexpr uint64_t kDrainNs = 2000000000ull;   // limit of the waits at the end of a role
constexpr int64_t kRange = 192ll << 32, kSafe = 100ll << 32;   // log2 bounds of e^{-G}, fixed point

constexpr int kChainThreads = 512, kGroupThreads = 128, kAuxThreads = 128;
constexpr int kIntraWarp = 16, kAuxWarp = 24, kIssueWarp = 28, kLoadWarp = 29, kLoad2Warp = 30, kInfoWarp = 31;
constexpr int kThreads = (kInfoWarp + 1) * 32;
// Sequences of up to so many tokens take the recurrence itself: 16 of one token, 32 heads 23 us, as
// a chunk 41 us; of four tokens 41.5 and 41.0 us.
constexpr int kFewTokens = 3;

// Shared memory (offsets from a 1024-aligned base).  A K/Q stage is
// [k K0 | q K0 | k K1 | q K1], 8 KiB each (64 rows x 128 B, 128-byte swizzle): the
// 128-row operand [K; Q] per half of 64 channels.  V: two halves of 8 KiB.
constexpr uint32_t kKQStage = 32768, kVStage = 16384;
constexpr int kKQStages = 2, kVStages = 2, kInfos = 8, kPBufs = 3;
constexpr uint32_t kOffEarly = kKQStages * kKQStage;     // the K/Q tile for A and P
constexpr uint32_t kOffV = kOffEarly + kKQStage;
constexpr uint32_t kOffP = kOffV + kVStages * kVStage;   // P: 64 x 64, three buffers
constexpr uint32_t kOffT = kOffP + kPBufs * 8192;        // T: 64 x 64, high and low parts
constexpr uint32_t kOffM = kOffT + 2 * 8192;             // per intra group, see below
// A's four 16 x 16 diagonal blocks in fp32 (rows padded to 20), then fp16 blocks of 32 rows
// (padded to 40), high and low parts: the two 32 x 32 diagonal blocks of T, transposed (A's own
// block between two diagonal ones sits in the unused lower left); A's rows 32-63, columns 0-31.
constexpr int kLdB = 20, kLdT = 40;
constexpr uint32_t kMDiag = 16 * kLdB * 4, kMTT = 32 * kLdT * 2;
constexpr uint32_t kMLow = 3 * kMTT;                     // from a high part to its low part
constexpr uint32_t kMGroup = 4 * kMDiag + 2 * kMLow;
constexpr uint32_t kOffO = (kOffM + 2 * kMGroup + 1023) / 1024 * 1024;   // output staging, 1 KiB a warp
constexpr uint32_t kSmem = kOffO + 4 * 1024 + 1024;

// TMEM columns.
constexpr uint32_t kTS = 0;      // S^T, fp32 [dv][dk]
constexpr uint32_t kTSb = 128;   // its bf16 parts: high, low (64 columns each)
constexpr uint32_t kTDF = 256;   // accumulator [dv][token]: S^T K^T, then F^T
constexpr uint32_t kTRF = 320;   // R^T, then F^T, bf16: high, low (32 columns each)
constexpr uint32_t kTO = 384;    // O^T accumulator
constexpr uint32_t kTAP = 448;   // A and P accumulators (rows 0-63, 64-127)

struct Bars {
    uint64_t early_full, kq_full[kKQStages], kq_empty[kKQStages], info_full[kInfos], info_free[kInfos];
    uint64_t v_full[kVStages], v_empty[kVStages];
    uint64_t ap_full[2], o_full[kPBufs], t_free[2];
    uint64_t ap_tfree, t_ready;
    uint64_t s_ready, d_full, r_ready, f_full, f_ready, s_full, o_free;
    uint64_t drain[2];
};

// Bounds and factors of a chunk.  Ring slots are reused after kInfos chunks: chunk c's is written
// once the outputs of chunk c - 6 are out, for which every role is past chunk c - 8.
struct __align__(16) Info {
    float beta[kC];   // 0 past the chunk's last token
    float ev[kC];     // beta e^{-G}
    float eo[kC];     // scale e^{G}
    float in, out;    // factors of the state: before the chunk (first token's e^g), after it (e^{G_C})
    int start, len;   // first token in the sequence, tokens
    int last;         // the sequence ends with this chunk
    int row;          // pool row of a block that ends with it, or -1
    int pad[2];
};

// One CTA per head and item.  Few chains leave most of the device idle, so long sequences are then
// cut into segments of whole chunks.  A segment maps its incoming state S to M S + L (columns never
// mix), so a first launch finds, for every segment but the last, L (the chain from zeros) and M (the
// chain from the identity, with v = 0); a short second one composes the incoming states; a third
// runs all segments with them.  Segment 0 needs no M: its L starts from the sequence's own state.
enum Kind : uint8_t { kOutputs, kOffset, kMap };
struct Item {
    uint16_t seq, buf;      // first workspace buffer of the sequence: S, L of segments 0 .., M of segments 1 ..
    uint8_t part, parts;    // segment, of how many
    Kind kind;
};
constexpr int kSms = kSplitSms;
static_assert(kSplitChunk == kC, "segments are whole chunks");

struct Params {
    GdrArgs a;
    float *ws;
    bool ordered;
    union {
        uint16_t order[kGdrMaxOrder];   // sequence of launch position i, longest first
        Item items[kSms];               // of launch position i, in a split
    };
};

// Segment of a sequence of len tokens, in tokens.
__device__ __forceinline__ int segment_of(int len, int parts) { return ((len + kC - 1) / kC + parts - 1) / parts * kC; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// g / ln 2 in fixed point, 32 bits behind the point, clamped far outside any fp32 exponent.
__device__ __forceinline__ int64_t fixed_log2(float g) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;   // 1 / ln 2
    g = fminf(fmaxf(g, -4096.f), 4096.f);                      // (NaN becomes -4096: see `bad`)
    const float p = g * kHi;
    return __float2ll_rn(p * 0x1p32f) + __float2ll_rn(fmaf(g, kLo, fmaf(g, kHi, -p)) * 0x1p32f);
}
// 2^x for a fixed-point x within fp32's exponents.
__device__ __forceinline__ float pow2(int64_t x) {
    return ex2((float)(uint32_t)x * 0x1p-32f) * __int_as_float(((int)(x >> 32) + 127) << 23);
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}
// 16 fp32 columns of this warp's lanes.
__device__ __forceinline__ void tmem_st16f(uint32_t taddr, const float (&x)[16]) {
    tmem_st16(taddr, reinterpret_cast<const uint32_t (&)[16]>(x));
}
// 16 lanes x 16 columns of TMEM as two 16 x 8 accumulator tiles: r[4 j ..] holds, of column
// group 8 j, (lane g, columns 2t, 2t + 1) and (lane g + 8, the same columns), with
// g = thread / 4, t = thread % 4.
__device__ __forceinline__ void tmem_ld_tiles16(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// Four 8 x 8 16-bit tiles, each stored transposed; lane 8 m + i gives the address of row i of
// tile m.
__device__ __forceinline__ void stmatrix4_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 ::"r"(saddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}
// x = hi + lo in bf16 (fp16) pairs: hi the rounded value, lo the rounded rest.
__device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack(a, b);
    const float2 r = __fadd2_rn(make_float2(a, b), make_float2(-__uint_as_float(hi << 16), -__uint_as_float(hi & 0xFFFF0000u)));
    lo = pack(r.x, r.y);
}
__device__ __forceinline__ void split_half(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_half(a, b);
    const float2 h = __half22float2(*(const __half2 *)&hi);
    lo = pack_half(a - h.x, b - h.y);
}
// D += A B, one 16 x 8 x 16 fp16 tile: a = (row g, k 2t..), (g + 8, 2t..), (g, 2t + 8..),
// (g + 8, 2t + 8..); b = (k 2t.., col g), (2t + 8.., g); d = (g, 2t), (g, 2t + 1), (g + 8, 2t),
// (g + 8, 2t + 1), with g = lane / 4, t = lane % 4.  (The fp16 form: the tf32 one has the same
// mantissa and took 72 cycles per half as deep a tile.)
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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
__device__ __forceinline__ void tma_prefetch(const CUtensorMap *map, int x, int h, int t0) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(t0) : "memory");
}
// Four 8 x 8 16-bit tiles; lane 8 m + i gives the address of row i of tile m.
template <bool TRANS> __device__ __forceinline__ void ldmatrix4(uint32_t saddr, uint32_t (&r)[4]) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr) : "memory");
}

// Off-diagonal block of the inverse of a lower-triangular matrix, transposed: Z^T = (T_jj^T
// A_ij^T) T_ii^T (the caller negates), W x W blocks with leading dimension kLdT, T's stored
// transposed, every matrix in two fp16 parts (22 bits) kMLow bytes apart, of whose products
// all but low x low are taken.  Where beta |k|^2 <= b, an entry of A, of T or of a product between
// them is at most b |k_s| / |k_r|: 1 for unit keys and beta <= 1, inside fp16 for norms within 2^14 of
// one another.  The smallest low part is 2^-24, which the ratio of the norms multiplies in the state:
// 1.2e-5 at 2^8, 4e-5 at 2^10, 5e-4 at 2^14.
// This warp forms rows j0 .. j0 + 15 (columns of the block) and, of them, columns
// i0 .. i0 + 15 (rows of the block).
template <int W>
__device__ __forceinline__ void block_product(uint32_t TjT, uint32_t A, uint32_t TiT, int j0, int i0, int lane,
                                              float (&z)[2][4]) {
    float v[W / 8][4];
#pragma unroll
    for (int n = 0; n < W / 8; ++n) v[n][0] = v[n][1] = v[n][2] = v[n][3] = 0.f;
    // Tiles of the A operand: rows 0-7 and 8-15 at k, the same at k + 8; of B (rows n of
    // A_ij): 0-7 at k and k + 8, 8-15 at k and k + 8.
    const uint32_t pa = TjT + 2 * ((j0 + (lane & 15)) * kLdT + (lane >> 4) * 8);
    const uint32_t pb = A + 2 * (((lane & 7) + (lane >> 4) * 8) * kLdT + ((lane >> 3) & 1) * 8);
#pragma unroll 1
    for (int k = j0; k < W; k += 16) {     // T_jj^T is upper triangular
        uint32_t ah[4], al[4];
        ldmatrix4<false>(pa + 2 * k, ah);
        ldmatrix4<false>(pa + 2 * k + kMLow, al);
#pragma unroll
        for (int n = 0; n < W / 8; n += 2) {
            uint32_t bh[4], bl[4];
            ldmatrix4<false>(pb + 2 * (8 * n * kLdT + k), bh);
            ldmatrix4<false>(pb + 2 * (8 * n * kLdT + k) + kMLow, bl);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                mma_f16(v[n + u], ah, bl[2 * u], bl[2 * u + 1]);
                mma_f16(v[n + u], al, bh[2 * u], bh[2 * u + 1]);
                mma_f16(v[n + u], ah, bh[2 * u], bh[2 * u + 1]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) z[n][0] = z[n][1] = z[n][2] = z[n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < W; k += 16) {
        if (k > i0) break;                 // T_ii is lower triangular
        const int n = k / 8;
        uint32_t ah[4], al[4], bh[4], bl[4];
        split_half(v[n][0], v[n][1], ah[0], al[0]);
        split_half(v[n][2], v[n][3], ah[1], al[1]);
        split_half(v[n + 1][0], v[n + 1][1], ah[2], al[2]);
        split_half(v[n + 1][2], v[n + 1][3], ah[3], al[3]);
        const uint32_t p = TiT + 2 * ((k + (lane & 15)) * kLdT + i0 + (lane >> 4) * 8);
        ldmatrix4<true>(p, bh);
        ldmatrix4<true>(p + kMLow, bl);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            mma_f16(z[u], ah, bl[2 * u], bl[2 * u + 1]);
            mma_f16(z[u], al, bh[2 * u], bh[2 * u + 1]);
            mma_f16(z[u], ah, bh[2 * u], bh[2 * u + 1]);
        }
    }
}

// Waits until the phase with the given parity completes, for kTries tries at most, in a loop
// of a few instructions (there are forty waits, and the roles' code has to stay in the
// instruction cache together).
__device__ __forceinline__ bool try_phase(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, %3;\n"
        "TRY%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n @p bra DONE%=;\n"
        " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra TRY%=;\n"
        "DONE%=:\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kTries), "n"(kSuspendNs)
        : "memory");
    return ok != 0;
}

// SPLIT: the launches over segments (their few more values in registers cost 3 % where there are
// none: 3.16 and 3.07 us a chunk).  COMPACT: for launches that fill the device, whose SMs wait for
// instructions (a cache line per 2.1 cycles and GPC at 148 CTAs): the inverse's first step as a loop,
// longer by 600 cycles and shorter by 1.4 KB.  us a chunk with it / without, at 96, 120, 128, 136
// and 148 CTAs: 3.47 / 3.11, 3.48 / 3.24, 3.49 / 3.4, 3.64 / 3.8, 3.71 / 3.90.
constexpr int kCompactCtas = 129;
template <bool SPLIT, bool COMPACT>
__global__ void __launch_bounds__(kThreads, 1)
gdr_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params prm)
{
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    __shared__ Bars bars;
    __shared__ Info infos[kInfos];
    __shared__ uint32_t tbase;
    const GdrArgs &a = prm.a;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pos = blockIdx.x / a.H, h = blockIdx.x % a.H, hk = h / (a.H / a.Hk);
    Item it = {0, 0, 0, 1, kOutputs};
    if (SPLIT) it = prm.items[pos];
    const int n = SPLIT ? it.seq : prm.ordered ? prm.order[pos] : pos;
    int tbeg = max(a.cu[n], 0), len = max(min(a.cu[n + 1], a.total_tokens) - tbeg, 0);
    // This segment; those behind the sequence's end (the host's lengths may differ) do nothing.
    const int whole = len;
    int from = 0;
    bool final = true;
    if (SPLIT) {
        const int seg = segment_of(len, it.parts);
        from = (int)min((int64_t)len, (int64_t)it.part * seg);
        final = len - from <= seg;
        if (it.part > 0 && from == len || it.kind != kOutputs && final) return;
        tbeg += from;
        len = final ? len - from : seg;
    }
    const int64_t before = (int64_t)(a.ctx ? max(a.ctx[n], 0) : 0) + from;   // tokens before this segment
    int src = a.src ? a.src[n] : -1, dst = final && a.dst ? a.dst[n] : -1;
    if (!a.state || src < 0 || src >= a.pool_size) src = -1;
    if (!a.state || dst < 0 || dst >= a.pool_size) dst = -1;
    auto row_of = [&](int slot) { return a.state + ((size_t)slot * a.H + h) * kD * kD; };
    auto buffer = [&](int b) { return prm.ws + ((size_t)(it.buf + b) * a.H + h) * kD * kD; };
    // The state before this segment (nullptr: zeros, or the identity) and where the one after it goes.
    auto state_in = [&]() -> const float * {
        if (SPLIT && it.part > 0) return it.kind == kOutputs ? buffer(it.part) : nullptr;
        if (src < 0) return nullptr;
        return SPLIT && it.parts > 1 && it.kind == kOutputs ? buffer(0) : row_of(src);
    };
    auto state_out = [&]() -> float * {
        if (SPLIT && it.kind != kOutputs) return buffer(it.kind == kMap ? it.parts - 1 + it.part : 1 + it.part);
        return dst >= 0 ? row_of(dst) : nullptr;
    };

    if (len == 0) {   // the state passes through
        float4 *to = (float4 *)state_out();
        const float4 *from = (const float4 *)state_in();
        if (to && to != from) {
#pragma unroll 1
            for (int e = tid; e < kD * kD / 4; e += kThreads)
                to[e] = from ? from[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }
    if (len <= kFewTokens) {   // token by token, S in fp32: column j, rows r0 .. r0 + 15 per thread
        float *vec = (float *)sm;                       // k, q of two tokens
        float2 *part = (float2 *)(vec + 4 * kD);        // [token & 1][row group][column]: S^T k, S^T q
        const int j = tid & 127, grp = tid >> 7, r0 = 16 * grp;
        const __nv_bfloat16 *kq_in = (const __nv_bfloat16 *)(grp == 0 ? a.k : a.q);
        const float *S0 = state_in();
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = S0 ? S0[(size_t)(r0 + i) * kD + j] : 0.f;
        auto store = [&](float *to) {
#pragma unroll
            for (int i = 0; i < 16; ++i) to[(size_t)(r0 + i) * kD + j] = x[i];
        };
#pragma unroll 1
        for (int t = 0; t < len; ++t) {
            const size_t tok = tbeg + t, at = tok * a.H + h;
            float *vk = vec + (t & 1) * 2 * kD;
            if (tid < 2 * kD) vk[tid] = __bfloat162float(kq_in[(tok * a.Hk + hk) * kD + j]);
            const float g = a.g[at], b = a.beta[at], v = __bfloat162float(((const __nv_bfloat16 *)a.v)[at * kD + j]);
            const float decay = expf(g < kGClampSoftplus ? kGClampSoftplus : g);
            __syncthreads();
            float seen = 0.f, read = 0.f, kq = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) kq = fmaf(vk[lane + 32 * i], vk[kD + lane + 32 * i], kq);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, off);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] *= decay;
                seen = fmaf(vk[r0 + i], x[i], seen);
                read = fmaf(vk[kD + r0 + i], x[i], read);
            }
            float2 *p = part + (t & 1) * 8 * kD + j;
            p[grp * kD] = make_float2(seen, read);
            __syncthreads();
            seen = read = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 y = p[i * kD];
                seen += y.x;
                read += y.y;
            }
            const float d = b * (v - seen);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = fmaf(vk[r0 + i], d, x[i]);
            if (grp == 0) ((__nv_bfloat16 *)a.o)[at * kD + j] = __float2bfloat16_rn(a.scale * fmaf(kq, d, read));
            const int64_t done = before + t + 1;
            if (a.block > 0 && done % a.block == 0 && done / a.block <= a.table_cols) {
                const int row = a.table[(size_t)n * a.table_cols + done / a.block - 1];
                if (row >= 0 && row < a.pool_size) store(row_of(row));
            }
        }
        if (float *to = state_out()) store(to);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < kKQStages; ++s) {
            mbar_init(&bars.kq_full[s], 1);
            mbar_init(&bars.kq_empty[s], 1);
        }
        mbar_init(&bars.early_full, 1);
        for (int s = 0; s < 2; ++s) mbar_init(&bars.drain[s], 1);
        for (int s = 0; s < kPBufs; ++s) mbar_init(&bars.o_full[s], 1);
        for (int s = 0; s < kInfos; ++s) {
            mbar_init(&bars.info_full[s], 1);
            mbar_init(&bars.info_free[s], kAuxThreads);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars.v_full[s], 1);
            mbar_init(&bars.v_empty[s], kChainThreads);
            mbar_init(&bars.ap_full[s], 1);
            mbar_init(&bars.t_free[s], 1);
        }
        mbar_init(&bars.ap_tfree, kGroupThreads);
        mbar_init(&bars.t_ready, kGroupThreads);
        mbar_init(&bars.s_ready, kChainThreads);
        mbar_init(&bars.d_full, 1);
        mbar_init(&bars.r_ready, kChainThreads);
        mbar_init(&bars.f_full, 1);
        mbar_init(&bars.f_ready, kChainThreads);
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.o_free, kAuxThreads);
        fence_mbar_init();
    }
    if (warp == 0) { tmem_alloc(&tbase, 512); tmem_relinquish(); }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tb = tbase;
    const uint32_t lq = 32 * (warp & 3);   // this warp's TMEM lanes

    // Bounded wait of a whole warp; once one has given up every later one fails at once, the
    // role leaves its loop and the timeout is recorded at the end (the other roles run into
    // the same limit).
    bool alive = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        alive = alive && __all_sync(0xffffffffu, try_phase(bar, parity & 1));
        return alive;
    };
    auto wait_info = [&](int c) { return wait(&bars.info_full[c % kInfos], c / kInfos); };
    // Buffer and phase of chunk c among the P buffers, advanced chunk by chunk.
    int stage = 0;
    uint32_t phase = 0;
    auto next_stage = [&] {
        if (++stage == kPBufs) { stage = 0; phase ^= 1; }
    };

    if (warp < kIntraWarp) {
        // ------------------------------------------------------------- chain --
        const int j = tid & 127, hh = warp >> 2;   // value channel; quarter of tokens / key channels
        const bool map = SPLIT && it.kind == kMap;
        const float *S0 = state_in();
        if (S0) S0 += (size_t)(32 * hh) * kD + j;
        // 16 columns of an accumulator as two bf16 operands of 8 columns each.
        auto put16 = [&](const float (&x)[16], uint32_t hi, uint32_t lo) {
            float h[8], l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t a, b;
                split(x[2 * i], x[2 * i + 1], a, b);
                h[i] = __uint_as_float(a);
                l[i] = __uint_as_float(b);
            }
            tmem_st8(tmem_addr(tb, lq, hi), h);
            tmem_st8(tmem_addr(tb, lq, lo), l);
        };
        auto hand_over = [&](uint64_t *bar) {
            tmem_st_wait();
            tc_fence_before_sync();
            mbar_arrive(bar);
        };
        bool ok = wait_info(0);
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
            float x[16];
            const float f = infos[0].in;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = S0 ? S0[(size_t)(16 * p + i) * kD] * f : map && 32 * hh + 16 * p + i == j ? f : 0.f;
            }
            tmem_st16f(tmem_addr(tb, lq, kTS + 32 * hh + 16 * p), x);
            put16(x, kTSb + 16 * hh + 8 * p, kTSb + 64 + 16 * hh + 8 * p);
        }
        hand_over(&bars.s_ready);
#pragma unroll 1
        for (int c = 0; ok; ++c) {
            float x[16];
            const Info &in = infos[c % kInfos];
            const bool last = in.last != 0;
            const float out = in.out;
            // V of this thread's channel and quarter of the tokens.
            ok = wait(&bars.v_full[c & 1], c >> 1);
            float2 w[8] = {};      // beta e^{-G} V^T
            if (!map) {
                const uint8_t *vt = sm + kOffV + (c & 1) * kVStage + (j >> 6) * 8192 + 16 * hh * 128;
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const uint32_t a0 = *(const uint16_t *)(vt + sw128_offset(i, j & 63, 64));
                    const uint32_t a1 = *(const uint16_t *)(vt + sw128_offset(i + 1, j & 63, 64));
                    w[i / 2] = __fmul2_rn(*(const float2 *)&in.ev[16 * hh + i],
                                          make_float2(__uint_as_float(a0 << 16), __uint_as_float(a1 << 16)));
                }
            }
            mbar_arrive(&bars.v_empty[c & 1]);
            if (in.len < kC) {
                // K's rows past the last token (another sequence's, or unwritten ones) become
                // zeros: F's zeros there do not undo an infinity or a NaN.
                ok = ok && wait(&bars.kq_full[c & 1], c >> 1);
                uint8_t *kt = sm + (c & 1) * kKQStage;
#pragma unroll 1
                for (int e = tid; e < (kC - in.len) * 16; e += kChainThreads)
                    *(uint4 *)(kt + (e & 8) * 2048 + (in.len + (e >> 4)) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            // R^T = beta (e^{-G} V^T - S^T K^T).
            ok = ok && wait(&bars.d_full, c);
            if (!ok) break;
            tc_fence_after_sync();
            tmem_ld16f(tmem_addr(tb, lq, kTDF + 16 * hh), x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 be = *(const float2 *)&in.beta[16 * hh + i];
                const float2 t = __ffma2_rn(make_float2(-be.x, -be.y), make_float2(x[i], x[i + 1]), w[i / 2]);
                x[i] = t.x;
                x[i + 1] = t.y;
            }
            if (in.len < kC) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = 16 * hh + i < in.len ? x[i] : 0.f;
            }
            put16(x, kTRF + 8 * hh, kTRF + 32 + 8 * hh);
            hand_over(&bars.r_ready);
            // F^T = R^T T^T.
            ok = wait(&bars.f_full, c);
            if (!ok) break;
            tc_fence_after_sync();
            tmem_ld16f(tmem_addr(tb, lq, kTDF + 16 * hh), x);
            tmem_ld_wait();
            put16(x, kTRF + 8 * hh, kTRF + 32 + 8 * hh);
            hand_over(&bars.f_ready);
            const int row = in.row;
            if (!last) ok = wait_info(c + 1);
            // (One after the other: their product may leave the exponent range.)
            const float next = infos[(c + 1) % kInfos].in;
            ok = ok && wait(&bars.s_full, c);
            if (!ok) break;
            tc_fence_after_sync();
            if (row >= 0 || last) {   // rows that keep the state after this chunk
#pragma unroll 1
                for (int w = 0; w < 4; ++w) {
                    float *to = w >= 2 ? (last ? state_out() : nullptr) : row >= 0 ? row_of(row) : nullptr;
                    const int p = w & 1;
                    if (!to) continue;
                    tmem_ld16f(tmem_addr(tb, lq, kTS + 32 * hh + 16 * p), x);
                    tmem_ld_wait();
                    float *Sf = to + (size_t)(32 * hh + 16 * p) * kD + j;
#pragma unroll
                    for (int i = 0; i < 16; ++i) Sf[(size_t)i * kD] = x[i] * out;
                }
                if (last) break;
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                tmem_ld16f(tmem_addr(tb, lq, kTS + 32 * hh + 16 * p), x);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 t = __fmul2_rn(__fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(out, out)),
                                                make_float2(next, next));
                    x[i] = t.x;
                    x[i + 1] = t.y;
                }
                tmem_st16f(tmem_addr(tb, lq, kTS + 32 * hh + 16 * p), x);
                put16(x, kTSb + 16 * hh + 8 * p, kTSb + 64 + 16 * hh + 8 * p);
            }
            hand_over(&bars.s_ready);
        }
    } else if (warp < kAuxWarp) {
        // ------------------------------------------------------------- intra --
        const int group = (warp - kIntraWarp) >> 2, wq = warp & 3, half = wq & 1;
        const int it = 32 * wq + lane, r = it & 63;
        const bool is_p = wq >= 2;
        float *diag = (float *)(sm + kOffM + group * kMGroup);
        uint8_t *tt = sm + kOffM + group * kMGroup + 4 * kMDiag, *X = tt + 2 * kMTT;   // T^T: two blocks; A
        bool ok = true;
        if (group == 1) { ok = wait_info(0); next_stage(); }
        bool more = group == 0 || (ok && !infos[0].last);
#pragma unroll 1
        for (int c = group; more; c += 2) {
            ok = ok && wait_info(c);
            const Info &in = infos[c % kInfos];
            // This group's blocks (every thread has read chunk c - 2's) and P's buffer (read by
            // the outputs of chunk c - 3).
            if (c >= 2) ok = ok && wait(&bars.t_free[c & 1], (c >> 1) - 1);
            if (c >= kPBufs) ok = ok && wait(&bars.o_full[stage], phase ^ 1);
            const float br = in.beta[r];
            ok = ok && wait(&bars.ap_full[c & 1], c >> 1);
            tc_fence_after_sync();
            // Columns 0 .. 32 half + 31 of this row, a 16-token tile at a time: A to its blocks in
            // fp32, P to its operand.
            uint8_t *img = sm + kOffP + stage * 8192;
#pragma unroll 1
            for (int k = 0; k < 2 * (1 + half); ++k) {
                const int s0 = (32 * half + 16 * k) & 63;   // the diagonal blocks first
                // Last column kept (15 or more: all; none in rows past the last token).
                const int lim = (r >= in.len ? -1 : is_p ? r : r - 1) - s0;
                float v[16];
                tmem_ld16f(tmem_addr(tb, lq, kTAP + s0), v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = i <= lim ? v[i] : 0.f;
                if (is_p) {
#pragma unroll
                    for (int i = 0; i < 16; i += 8)
                        *(uint4 *)(img + sw128_offset(r, s0 + i, 64)) =
                            make_uint4(pack(v[i], v[i + 1]), pack(v[i + 2], v[i + 3]), pack(v[i + 4], v[i + 5]),
                                       pack(v[i + 6], v[i + 7]));
                } else {
                    const int sub = (r >> 4) & 1, rel = s0 - 32 * half;   // this row's 16-block, the tile's
                    if (rel == 16 * sub) {          // the diagonal block
                        float *m = diag + (2 * half + sub) * (kMDiag / 4) + (r & 15) * kLdB;
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            *(float4 *)&m[i] = make_float4(v[i] * br, v[i + 1] * br, v[i + 2] * br, v[i + 3] * br);
                    } else if (rel < 16 * sub) {    // left of it: fp16 (rel < 0: rows 32-63, columns 0-31)
                        uint4 *m = (uint4 *)((rel < 0 ? X : tt + half * kMTT) + 2 * ((r & 31) * kLdT + (s0 & 31)));
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) split_half(v[2 * i] * br, v[2 * i + 1] * br, hi[i], lo[i]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            m[i] = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                            m[kMLow / 16 + i] = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                        }
                    }
                    if (k == 1) {          // the inverses may start
                        __threadfence_block();
                        asm volatile("barrier.arrive %0, 128;" ::"r"(3 + group) : "memory");
                    }
                }
            }
            if (is_p) fence_proxy_async_smem();
            tc_fence_before_sync();
            mbar_arrive(&bars.ap_tfree);
            // Inverse of the two 32 x 32 diagonal blocks, one warp each (those of P, whose readback is
            // shorter; on the warps of A 3.16 instead of 3.11 us/chunk at 96 heads): four 8 x 8 blocks
            // by substitution, then the blocks between them, 8 x 8 and 16 x 16.  COMPACT: the 16 x 16
            // blocks by substitution, half a warp each, lane j its column j, four unknowns at a time.
            if (is_p) {
                asm volatile("barrier.sync %0, 128;" ::"r"(3 + group) : "memory");
                uint8_t *Tw = tt + half * kMTT;
                const int g = lane >> 2, t = lane & 3;
                if constexpr (COMPACT) {
                    const int sub = lane >> 4;
                    const float *B = diag + (2 * half + sub) * (kMDiag / 4);
                    const int j = lane & 15;
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.f : 0.f;
                    // x: rows m0 .. m0 + 15 (those past the block's last are never used); stored transposed,
                    // lane j's column as row j of the block.
                    uint8_t *p = Tw + 2 * ((16 * sub + j) * kLdT + 16 * sub);
#pragma unroll 1
                    for (int m0 = 0; m0 < 16; m0 += 4, B += 4 * kLdB + 4, p += 8) {
#pragma unroll
                        for (int i = 1; i < 16; ++i) {
                            const float4 l = *(const float4 *)&B[i * kLdB];
                            const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                if (m < i) x[i] = fmaf(-lv[m], x[m], x[i]);
                        }
                        uint32_t hi[2], lo[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) split_half(x[2 * u], x[2 * u + 1], hi[u], lo[u]);
                        *(uint2 *)p = make_uint2(hi[0], hi[1]);
                        *(uint2 *)(p + kMLow) = make_uint2(lo[0], lo[1]);
#pragma unroll
                        for (int i = 0; i < 12; ++i) x[i] = x[i + 4];
                    }
                    __syncwarp();
                } else {
                    const float *B = diag + 2 * half * (kMDiag / 4);       // its two 16 x 16 blocks
                    {   // four 8 x 8 blocks, a column j per lane
                        const int j = lane & 7, sub = lane >> 4, q = (lane >> 3) & 1;
                        const float *L = B + sub * (kMDiag / 4) + 8 * q * (kLdB + 1);
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = i == j ? 1.f : 0.f;
#pragma unroll
                        for (int m0 = 0; m0 < 8; m0 += 4) {
#pragma unroll
                            for (int i = m0 + 1; i < 8; ++i) {
                                const float4 l = *(const float4 *)&L[i * kLdB + m0];
                                const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                                for (int m = 0; m < 4; ++m)
                                    if (m0 + m < i) x[i] = fmaf(-lv[m], x[m0 + m], x[i]);
                            }
                        }
                        // Transposed: lane j's column is row j of the block; left of a lower one zeros.
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) split_half(x[2 * u], x[2 * u + 1], hi[u], lo[u]);
                        uint4 *p = (uint4 *)(Tw + 2 * ((16 * sub + 8 * q + j) * kLdT + 16 * sub));
                        const uint4 zero = make_uint4(0, 0, 0, 0);
                        if (q) p[0] = p[kMLow / 16] = zero;
                        p[q] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        p[q + kMLow / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    __syncwarp();
                    {   // the blocks between them, both 16 x 16 at once: two diagonal tiles of each operand
                        const uint32_t p = smem_u32(Tw) + 2 * ((lane & 7) * kLdT + ((lane >> 3) & 1) * (16 * kLdT + 16)) + (lane >> 4) * kMLow;
                        uint32_t tj[4], ti[4], ah[2], al[2];     // (high, high, low, low) of the two blocks
                        ldmatrix4<false>(p, tj);
                        ldmatrix4<true>(p + 2 * 8 * (kLdT + 1), ti);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float2 l = *(const float2 *)&B[u * (kMDiag / 4) + (8 + g) * kLdB + 2 * t];
                            split_half(l.x, l.y, ah[u], al[u]);
                        }
                        float v[4] = {}, z[4] = {};
                        const uint32_t th[4] = {tj[0], 0, 0, tj[1]}, tl[4] = {tj[2], 0, 0, tj[3]};
                        mma_f16(v, th, al[0], al[1]);
                        mma_f16(v, tl, ah[0], ah[1]);
                        mma_f16(v, th, ah[0], ah[1]);
                        uint32_t vh[4] = {}, vl[4] = {};
                        split_half(v[0], v[1], vh[0], vl[0]);
                        split_half(v[2], v[3], vh[3], vl[3]);
                        mma_f16(z, vh, ti[2], ti[3]);
                        mma_f16(z, vl, ti[0], ti[1]);
                        mma_f16(z, vh, ti[0], ti[1]);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint32_t *to = (uint32_t *)(Tw + 2 * ((16 * u + g) * kLdT + 16 * u + 8 + 2 * t));
                            split_half(-z[2 * u], -z[2 * u + 1], to[0], to[kMLow / 4]);
                        }
                    }
                    __syncwarp();
                }
                float z[2][4];
                const uint32_t tw = smem_u32(Tw);
                block_product<16>(tw, tw + 2 * 16 * kLdT, tw + 2 * (16 * kLdT + 16), 0, 0, lane, z);
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t *to = (uint32_t *)(Tw + 2 * ((g + 8 * u) * kLdT + 16 + 8 * q + 2 * t));
                        split_half(-z[q][2 * u], -z[q][2 * u + 1], to[0], to[kMLow / 4]);
                    }
            }
            // T's operands: free once chunk c - 1's product has read them.
            if (c > 0) ok = ok && wait(&bars.t_free[(c - 1) & 1], (c - 1) >> 1);
            if (group_sync_any(group, !ok)) break;
            // T's operand in two parts, rows i, columns j: tiles of T^T stored transposed.
            const uint32_t timg = smem_u32(sm + kOffT);
            {   // rows 32-63, columns 0-31: 16 x 16 per warp
                const int i0 = 16 * half, j0 = 16 * (wq >> 1);
                float z[2][4];
                block_product<32>(smem_u32(tt), smem_u32(X), smem_u32(tt + kMTT), j0, i0, lane, z);
                const uint32_t at = timg + sw128_offset(32 + i0 + 8 * (lane >> 4) + (lane & 7), j0 + 8 * ((lane >> 3) & 1), 64);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) split(-z[u >> 1][2 * (u & 1)], -z[u >> 1][2 * (u & 1) + 1], hi[u], lo[u]);
                stmatrix4_trans(at, hi[0], hi[1], hi[2], hi[3]);
                stmatrix4_trans(at + 8192, lo[0], lo[1], lo[2], lo[3]);
            }
            // The diagonal blocks: half a block per warp, eight rows i at a time; tiles of T^T are
            // columns j of the image in blocks of eight.
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                const int i = (is_p ? 16 : 0) + 8 * u;
                const uint32_t tw = smem_u32(tt + half * kMTT) + 2 * (lane * kLdT + i);
                uint32_t p[4], q[4];
                ldmatrix4<false>(tw, p);
                ldmatrix4<false>(tw + kMLow, q);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 x = __half22float2(*(const __half2 *)&p[m]), y = __half22float2(*(const __half2 *)&q[m]);
                    const float2 t = 8 * m <= i ? __fadd2_rn(x, y) : make_float2(0.f, 0.f);
                    split(t.x, t.y, p[m], q[m]);
                }
                const uint32_t at = timg + sw128_offset(32 * half + i + (lane & 7), 32 * half + 8 * (lane >> 3), 64);
                stmatrix4_trans(at, p[0], p[1], p[2], p[3]);
                stmatrix4_trans(at + 8192, q[0], q[1], q[2], q[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&bars.t_ready);
            more = !in.last;
            if (more) {
                ok = ok && wait_info(c + 1);
                more = ok && !infos[(c + 1) % kInfos].last;
            }
            next_stage();
            next_stage();
        }
    } else if (warp < kIssueWarp) {
        // --------------------------------------------------------------- aux --
        const int wq = warp & 3;
        uint8_t *ost = sm + kOffO + 1024 * wq;     // a tile of [16 tokens][32 channels]
        __nv_bfloat16 *o = (__nv_bfloat16 *)a.o;
        const uint32_t osa = smem_u32(ost) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll 1
        for (int c = 0;; ++c) {
            if (!wait_info(c) || !wait(&bars.o_full[stage], phase)) break;
            next_stage();
            const Info &in = infos[c % kInfos];
            const bool last = in.last != 0;
            const int rows = !SPLIT || it.kind == kOutputs ? in.len : 0;
            tc_fence_after_sync();
            // 16 tokens at a time: four 8 x 8 blocks (channels x tokens) become eight token rows of 32
            // channels, 16-byte pieces swizzled by token pair; a lane then stores two of them.
#pragma unroll 1
            for (int q = 0; q < kC; q += 16) {
                uint32_t u[8], v[8];
                tmem_ld_tiles16(tmem_addr(tb, lq, kTO + q), u);
                tmem_ld_tiles16(tmem_addr(tb, lq + 16, kTO + q), v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 d = *(const float2 *)&in.eo[q + 8 * j + 2 * (lane & 3)];
                    auto scaled = [&](const uint32_t *x) {
                        return pack(__uint_as_float(x[0]) * d.x, __uint_as_float(x[1]) * d.y);
                    };
                    stmatrix4_trans(osa + j * 512, scaled(u + 4 * j), scaled(u + 4 * j + 2), scaled(v + 4 * j),
                                    scaled(v + 4 * j + 2));
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int t = q + 8 * j + (lane >> 2);
                    const uint4 w = *(const uint4 *)(ost + j * 512 + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4));
                    if (t < rows)
                        *(uint4 *)(o + ((size_t)(tbeg + in.start + t) * a.H + h) * kD + 32 * wq + 8 * (lane & 3)) = w;
                }
                __syncwarp();
            }
            tc_fence_before_sync();
            mbar_arrive(&bars.o_free);
            mbar_arrive(&bars.info_free[c % kInfos]);
            if (last) break;
        }
    } else {
    if (warp == kIssueWarp) {
        // ------------------------------------------------------------- issue --
        const bool leader = elect_one();
        const uint32_t id64 = idesc_bf16_f32(128, 64), id128 = idesc_bf16_f32(128, 128);
        const uint64_t dT = desc_kmajor_sw128(smem_u32(sm + kOffT));
        const uint32_t sb = tmem_addr(tb, 0, kTSb), rf = tmem_addr(tb, 0, kTRF);
        const uint32_t tdf = tmem_addr(tb, 0, kTDF), to = tmem_addr(tb, 0, kTO);
        bool ok = true;
#pragma unroll 1
        for (int c = 0; ok; ++c) {
            const int s = c & 1;
            const uint32_t st = smem_u32(sm + s * kKQStage);
            const uint64_t dK = desc_kmajor_sw128(st), dQ = desc_kmajor_sw128(st + 8192);
            const uint64_t dKn = desc_mnmajor_sw128(st, 16384);
            const uint64_t dP = desc_kmajor_sw128(smem_u32(sm + kOffP + stage * 8192));
            ok = wait_info(c) && wait(&bars.kq_full[s], c >> 1) && wait(&bars.s_ready, c);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {   // [DF] = S^T K^T
#pragma unroll
                for (int ks = 0; ks < 16; ++ks)
                    mma_ts(tdf, sb + 8 * ks, dK + ((((ks >> 2) & 1) * 16384 + (ks & 3) * 32) >> 4), id64, ks > 0);
                mma_commit(&bars.d_full);
            }
            __syncwarp();
            ok = wait(&bars.t_ready, c) && wait(&bars.r_ready, c);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {   // [DF] = R^T T^T: high x low, low x high, high x high
#pragma unroll
                for (int ks = 0; ks < 12; ++ks) {
                    const int s16 = ks & 3;
                    mma_ts(tdf + 16 * s16, rf + 8 * s16 + (ks >= 4 && ks < 8 ? 32 : 0),
                           dT + (((ks < 4 ? 8192 : 0) + s16 * (2048 + 32)) >> 4),
                           idesc_bf16_f32(128, 64 - 16 * s16), ks > 0);
                }
                mma_commit(&bars.f_full);
                mma_commit(&bars.t_free[s]);
            }
            __syncwarp();
            if (c > 0 && !wait(&bars.o_free, c - 1)) break;
            tc_fence_after_sync();
            if (leader) {   // [O^T] = S^T Q^T
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ts(to, sb + 8 * ks, dQ + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4), id64, ks > 0);
            }
            __syncwarp();
            ok = wait(&bars.f_ready, c);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {   // [S^T] += F^T K;  [O^T] += F^T P^T
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ts(tmem_addr(tb, 0, kTS), rf + 8 * ks, dKn + (ks & 3) * (2048 >> 4), id128 | kIdescMnB, true);
                mma_commit(&bars.s_full);
                mma_commit(&bars.kq_empty[s]);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ts(to + 16 * (ks & 3), rf + 8 * ks, dP + (ks & 3) * ((2048 + 32) >> 4),
                           idesc_bf16_f32(128, 64 - 16 * (ks & 3)), true);
                mma_commit(&bars.o_full[stage]);
            }
            __syncwarp();
            next_stage();
            if (infos[c % kInfos].last) break;
        }
        if (leader) {   // every product of this role has finished before the CTA may exit
            mma_commit(&bars.drain[0]);
            mbar_wait(&bars.drain[0], 0, globaltimer_ns() + kDrainNs);
        }
        __syncwarp();
    } else if (warp == kLoadWarp) {
        // -------------------------------------------------------------- load --
        const bool leader = elect_one();
        int loaded = 0;
        // The tiles of tokens t .. t + 63 into L2, a chunk ahead of their loads.
        auto prefetch = [&](int t) {
            if (!leader || t >= len) return;
            for (int x = 0; x < kD; x += 64) {
                tma_prefetch(&tm_k, x, hk, tbeg + t);
                tma_prefetch(&tm_q, x, hk, tbeg + t);
                tma_prefetch(&tm_v, x, h, tbeg + t);
            }
        };
        prefetch(kC);
#pragma unroll 1
        for (int c = 0;; ++c) {
            if (!wait_info(c)) break;
            const Info &in = infos[c % kInfos];
            const int start = in.start, next = start + in.len;
            const bool last = in.last != 0;
            if (c > 0 && !wait(&bars.ap_full[(c - 1) & 1], (c - 1) >> 1)) break;
            if (leader) {
                uint8_t *st = sm + kOffEarly;
                const int t0 = tbeg + start;
                mbar_arrive_expect_tx(&bars.early_full, kKQStage);
                tma_tile(st, &tm_k, 0, hk, t0, &bars.early_full);
                tma_tile(st + 16384, &tm_k, 64, hk, t0, &bars.early_full);
                tma_tile(st + 8192, &tm_q, 0, hk, t0, &bars.early_full);
                tma_tile(st + 24576, &tm_q, 64, hk, t0, &bars.early_full);
            }
            ++loaded;
            __syncwarp();
            prefetch(next + kC);
            // [AP] = [K; Q] K^T, once the previous chunk's A and P have been read.
            if (!wait(&bars.early_full, c) || (c > 0 && !wait(&bars.ap_tfree, c - 1))) break;
            tc_fence_after_sync();
            if (leader) {
                const uint64_t d = desc_kmajor_sw128(smem_u32(sm + kOffEarly));
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint64_t x = d + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
                    mma_ss(tmem_addr(tb, 0, kTAP), x, x, idesc_bf16_f32(128, 64), ks > 0);
                }
                mma_commit(&bars.ap_full[c & 1]);
            }
            __syncwarp();
            if (last) break;
        }
        if (leader) {   // tiles landed and products finished before the CTA may exit
            if (loaded > 0) mbar_wait(&bars.early_full, (loaded - 1) & 1, globaltimer_ns() + kDrainNs);
            mma_commit(&bars.drain[1]);
            mbar_wait(&bars.drain[1], 0, globaltimer_ns() + kDrainNs);
        }
        __syncwarp();
    } else if (warp == kLoad2Warp) {
        // ---------------------------------------------- load: the other products --
        const bool leader = elect_one();
        int loaded = 0;
#pragma unroll 1
        for (int c = 0;; ++c) {
            const int s = c & 1;
            if (!wait_info(c)) break;
            if (c >= 2 && !(wait(&bars.kq_empty[s], (c >> 1) - 1) && wait(&bars.v_empty[s], (c >> 1) - 1))) break;
            const int t0 = tbeg + infos[c % kInfos].start;
            if (leader) {
                uint8_t *st = sm + s * kKQStage, *vt = sm + kOffV + s * kVStage;
                mbar_arrive_expect_tx(&bars.v_full[s], kVStage);
                tma_tile(vt, &tm_v, 0, h, t0, &bars.v_full[s]);
                tma_tile(vt + 8192, &tm_v, 64, h, t0, &bars.v_full[s]);
                mbar_arrive_expect_tx(&bars.kq_full[s], kKQStage);
                tma_tile(st, &tm_k, 0, hk, t0, &bars.kq_full[s]);
                tma_tile(st + 16384, &tm_k, 64, hk, t0, &bars.kq_full[s]);
                tma_tile(st + 8192, &tm_q, 0, hk, t0, &bars.kq_full[s]);
                tma_tile(st + 24576, &tm_q, 64, hk, t0, &bars.kq_full[s]);
            }
            ++loaded;
            __syncwarp();
            if (infos[c % kInfos].last) break;
        }
        if (leader)
#pragma unroll 1
            for (int c = max(0, loaded - 2); c < loaded; ++c) {
                mbar_wait(&bars.kq_full[c & 1], (c >> 1) & 1, globaltimer_ns() + kDrainNs);
                mbar_wait(&bars.v_full[c & 1], (c >> 1) & 1, globaltimer_ns() + kDrainNs);
            }
        __syncwarp();
    } else {
        // -------------------------------------------------------------- info --
        int start = 0;
        // Tokens left in the current block, and its index (no blocks: more than there are).
        int to_block = a.block > 0 ? a.block - (int)(before % a.block) : 0x7fffffff;
        int blk = a.block > 0 ? (int)(before / a.block) : 0;
        // Columns of the blocks that this call completes end here.
        const int64_t done = SPLIT && a.block > 0 ? min((before - from + whole) / a.block, (int64_t)a.table_cols) : 0;
        // g and beta of tokens 2 lane, 2 lane + 1 of this chunk, and of the next if this one is full.
        float g[2], be[2], gn[2], bn[2];
        auto fetch = [&](int from, float (&g)[2], float (&be)[2]) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = from + 2 * lane + u;
                const size_t x = (size_t)(tbeg + t) * a.H + h;
                g[u] = t < len ? a.g[x] : 0.f;
                be[u] = t < len ? a.beta[x] : 0.f;
            }
        };
        fetch(0, g, be);
#pragma unroll 1
        for (int c = 0; start < len; ++c) {
            if (c >= 6 && !wait(&bars.info_free[(c - 6) % kInfos], (c - 6) / kInfos)) break;
            // Bounds: 64 tokens, the sequence's end, the end of a block that wants its row, and the
            // range of e^{-G}; then the factors.
            fetch(start + kC, gn, bn);
            int m = min(kC, len - start);
            m = min(m, to_block);
            // The scan is in 64 bits (fixed point, 32 of them behind the point): near its end a
            // chunk's G is large and its differences are not.
            const int64_t x0 = fixed_log2(g[0]), x1 = fixed_log2(g[1]);
            const int64_t first = __shfl_sync(0xffffffffu, x0, 0);   // applied to the incoming state
            int64_t sum = lane == 0 ? x1 : x0 + x1;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += y;
            }
            const int64_t before = __shfl_up_sync(0xffffffffu, sum, 1);
            const int64_t G0 = lane == 0 ? 0 : before + x0, G1 = sum;
            // (A positive log-decay: G need not fall, so it stays within kSafe either way.)
            const int64_t range = __any_sync(0xffffffffu, !(g[0] <= 0.f) || !(g[1] <= 0.f)) ? kSafe : kRange;
            const uint32_t out0 = __ballot_sync(0xffffffffu, G0 > range || G0 < -range);
            const uint32_t out1 = __ballot_sync(0xffffffffu, G1 > range || G1 < -range);
            if (out0) m = min(m, 2 * (__ffs(out0) - 1));
            if (out1) m = min(m, 2 * (__ffs(out1) - 1) + 1);
            const int64_t GC = __shfl_sync(0xffffffffu, (m - 1) & 1 ? G1 : G0, (m - 1) >> 1);
            const int64_t shift = max((int64_t)0, -GC - kSafe);
            const bool in0 = 2 * lane < m, in1 = 2 * lane + 1 < m;
            // A NaN among the log-decays reaches its token's factors, and the state's.
            const float bad0 = g[0] == g[0] ? 0.f : g[0], bad1 = g[1] == g[1] ? 0.f : g[1];
            Info &in = infos[c % kInfos];
            *(float2 *)&in.beta[2 * lane] = make_float2(in0 ? be[0] : 0.f, in1 ? be[1] : 0.f);
            *(float2 *)&in.ev[2 * lane] = make_float2(in0 ? be[0] * pow2(-G0 - shift) + bad0 : 0.f,
                                                      in1 ? be[1] * pow2(-G1 - shift) + bad1 : 0.f);
            *(float2 *)&in.eo[2 * lane] = make_float2(in0 ? a.scale * pow2(G0 + shift) + bad0 : 0.f,
                                                      in1 ? a.scale * pow2(G1 + shift) + bad1 : 0.f);
            const float bad = __uint_as_float(__reduce_or_sync(
                0xffffffffu, (in0 ? __float_as_uint(bad0) : 0u) | (in1 ? __float_as_uint(bad1) : 0u)));
            // The state's two factors multiply it again and again: to the last bit.
            const float factor = (float)exp2((double)(lane == 0 ? first - shift : GC + shift) * 0x1p-32) + bad;
            // Segments run at once, so a row that the sequence writes again (its last state, a later
            // block under the same row) is left to the later token.
            bool again = false;
            if (SPLIT && it.kind == kOutputs && a.block > 0 && m == to_block && blk < a.table_cols) {
                const int32_t *rows = a.table + (size_t)n * a.table_cols;
                const int row = rows[blk];
                again = a.dst && a.dst[n] == row;
                for (int64_t j = (int64_t)blk + 1 + lane; j < done; j += 32) again = again || rows[j] == row;
                again = __any_sync(0xffffffffu, again);
            }
            if (lane == 1) in.out = factor;
            if (lane == 0) {
                in.in = factor;
                in.start = start;
                in.len = m;
                in.last = start + m >= len;
                in.row = -1;
                if (a.block > 0 && (!SPLIT || it.kind == kOutputs) && m == to_block && blk < a.table_cols) {
                    const int row = a.table[(size_t)n * a.table_cols + blk];
                    if (row >= 0 && row < a.pool_size && !again) in.row = row;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.info_full[c % kInfos]);
            start += m;
            to_block -= m;
            if (to_block == 0 && a.block > 0) { to_block = a.block; ++blk; }
            if (m == kC) {
                g[0] = gn[0]; g[1] = gn[1];
                be[0] = bn[0]; be[1] = bn[1];
            } else if (start < len) {
                fetch(start, g, be);
            }
        }
    }
    }
    if (!alive && lane == 0) atomicCAS(a.status, 0, (int32_t)KDA_TC_TIMEOUT_CODE);
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tb, 512);
}

// Composes the segments' incoming states: S_{p+1} = M_p S_p + L_p, over L_p (S_1 is L_0), 16 value
// columns per CTA in fp32; and keeps a copy of the sequence's own state, which a later segment's
// row may overwrite.  3.3 us a segment; wider column blocks per warp (fewer reads of M), scalar
// products and an earlier load of L changed that by 5 % either way.
constexpr int kJoinCols = 16, kJoinThreads = 256, kLdM = kD + 4;
constexpr uint32_t kJoinSmem = (2 * kD * kLdM + kD * kJoinCols) * 4;
struct Joins {
    GdrArgs a;
    float *ws;
    Item items[kSms / 2];      // the split sequences
};
__global__ void __launch_bounds__(kJoinThreads)
gdr_join_kernel(const __grid_constant__ Joins prm)
{
    extern __shared__ __align__(16) float smj[];
    float *sS = smj + 2 * kD * kLdM;                 // [k][column]
    const GdrArgs &a = prm.a;
    const Item it = prm.items[blockIdx.x / a.H];
    const int h = blockIdx.x % a.H, tid = threadIdx.x, c = 2 * (tid & 7), r = tid >> 3;   // rows r + 32 i
    const int col = blockIdx.y * kJoinCols + c, P = it.parts;
    const int len = max(min(a.cu[it.seq + 1], a.total_tokens) - max(a.cu[it.seq], 0), 0), seg = segment_of(len, P);
    auto buffer = [&](int b) { return prm.ws + ((size_t)(it.buf + b) * a.H + h) * kD * kD; };
    auto at = [&](float *p, int i) { return (float2 *)(p + (size_t)(r + 32 * i) * kD + col); };
    // Segments 1 .. last + 1 have tokens: S_2 .. S_{last + 1} are formed, with M_1 .. M_last.
    const int last = seg > 0 ? min(P - 2, (len - 1) / seg - 1) : 0;
    auto fetch = [&](int p) {
        const float *M = buffer(P - 1 + p);
        const uint32_t to = smem_u32(smj + (p & 1) * kD * kLdM);
        for (int e = tid; e < kD * kD / 4; e += kJoinThreads)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         ::"r"(to + (e / 32 * kLdM + e % 32 * 4) * 4), "l"(M + 4 * e) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (last >= 1) fetch(1);
    const int src = a.src ? a.src[it.seq] : -1;
    if (a.state && src >= 0 && src < a.pool_size) {
        float *row = a.state + ((size_t)src * a.H + h) * kD * kD;
#pragma unroll
        for (int i = 0; i < 4; ++i) *at(buffer(0), i) = *at(row, i);
    }
    if (last < 1) return;
    float2 S[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) S[i] = *at(buffer(1), i);
    for (int p = 1; p <= last; ++p) {
        __syncthreads();                             // S and M_{p - 1} are no longer read
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *(float2 *)&sS[(r + 32 * i) * kJoinCols + c] = S[i];
            S[i] = *at(buffer(1 + p), i);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (p < last) fetch(p + 1);
        const float *M = smj + (p & 1) * kD * kLdM + r * kLdM;
#pragma unroll 4
        for (int k = 0; k < kD; k += 4) {
            float2 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = *(const float2 *)&sS[(k + u) * kJoinCols + c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 m = *(const float4 *)&M[32 * i * kLdM + k];
                S[i] = __ffma2_rn(make_float2(m.x, m.x), x[0], S[i]);
                S[i] = __ffma2_rn(make_float2(m.y, m.y), x[1], S[i]);
                S[i] = __ffma2_rn(make_float2(m.z, m.z), x[2], S[i]);
                S[i] = __ffma2_rn(make_float2(m.w, m.w), x[3], S[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) *at(buffer(1 + p), i) = S[i];
    }
}

}  // namespace

template <bool SPLIT>
static cudaError_t launch_chunks(int ctas, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                 const Params &p, cudaStream_t stream)
{
    auto *kernel = ctas >= kCompactCtas ? gdr_chunk_kernel<SPLIT, true> : gdr_chunk_kernel<SPLIT, false>;
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (err != cudaSuccess) return err;
    kernel<<<(unsigned)ctas, kThreads, kSmem, stream>>>(q, k, v, p);
    return cudaGetLastError();
}

size_t gdr_tensor_core_workspace(int32_t total_tokens, int32_t num_seqs, int32_t H)
{
    // Of a sequence's 2 P - 2 buffers per head all but one belong to a CTA of the first launch.
    return may_split({num_seqs, total_tokens, H, nullptr}) ? (size_t)2 * kSms * kD * kD * sizeof(float) : 0;
}

cudaError_t launch_gdr_tensor_core(const GdrArgs &a, void *workspace, cudaStream_t stream)
{
    const int64_t ctas = (int64_t)a.num_seqs * a.H;
    if (a.dk != kD || a.dv != kD || !a.bf16 || !a.cu || ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (ctas == 0) return cudaSuccess;
    cudaError_t err;
    CUtensorMap mq, mk, mv;
    memset(&mq, 0, sizeof(mq));
    mk = mv = mq;   // with no tokens no tile is read
    if (a.total_tokens > 0 &&
        (!tc_rows_map(&mq, a.q, a.total_tokens, a.Hk) || !tc_rows_map(&mk, a.k, a.total_tokens, a.Hk) ||
         !tc_rows_map(&mv, a.v, a.total_tokens, a.H)))
        return cudaErrorInvalidValue;
    Params p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    const SplitBatch batch = {a.num_seqs, a.total_tokens, a.H, a.cu_host};
    if (const int chunks = plan_split(batch)) {
        Joins joins;
        memset(&joins, 0, sizeof(joins));
        joins.a = a;
        joins.ws = p.ws = (float *)workspace;
        Params first = p;
        int all = 0, firsts = 0, splits = 0, buf = 0;
        for (int n = 0; n < a.num_seqs; ++n) {
            const int P = parts_of(chunks_of(batch, n), chunks);
            Item it = {(uint16_t)n, (uint16_t)buf, 0, (uint8_t)P, kOutputs};
            for (int s = 0; s < P; ++s) {
                it.part = (uint8_t)s;
                it.kind = kOutputs;
                p.items[all++] = it;
                if (s + 1 == P) break;
                it.kind = kOffset;
                first.items[firsts++] = it;
                it.kind = kMap;
                if (s > 0) first.items[firsts++] = it;
            }
            if (P == 1) continue;
            joins.items[splits++] = it;
            buf += 2 * P - 2;
        }
        err = cudaFuncSetAttribute(gdr_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kJoinSmem);
        if (err != cudaSuccess) return err;
        err = launch_chunks<true>(firsts * a.H, mq, mk, mv, first, stream);
        if (err != cudaSuccess) return err;
        gdr_join_kernel<<<dim3(splits * a.H, kD / kJoinCols), kJoinThreads, kJoinSmem, stream>>>(joins);
        err = cudaGetLastError();
        return err == cudaSuccess ? launch_chunks<true>(all * a.H, mq, mk, mv, p, stream) : err;
    }
    // Longest sequences first (they set the end of the launch); the host offsets only
    // order the CTAs, each of which reads its own bounds on the device.
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
    return launch_chunks<false>((int)ctas, mq, mk, mv, p, stream);
}

}  // namespace kda
