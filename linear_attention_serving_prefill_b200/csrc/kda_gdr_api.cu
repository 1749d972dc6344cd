// C-ABI layer of the gated delta rule and the block plan: argument validation
// and dispatch.  Nothing here allocates device memory; every call is
// asynchronous on the caller's stream.
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "kda_gdr.h"
#include "kda_internal.h"

namespace {

bool head_dim_ok(int32_t d) { return d == 32 || d == 64 || d == 128; }
bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

kda_status check_sizes(int32_t Hk, int32_t H, int32_t dk, int32_t dv, kda_dtype dt)
{
    if (H <= 0 || Hk <= 0 || H % Hk != 0) return KDA_ERR_INVALID_ARG;
    if (dt != KDA_DTYPE_BF16 && dt != KDA_DTYPE_F32) return KDA_ERR_INVALID_ARG;
    if (dk <= 0 || dv <= 0) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_prefill(int32_t total_tokens, int32_t num_seqs, int32_t Hk, int32_t H, int32_t dk,
                         int32_t dv, kda_dtype dt, kda_algo algo)
{
    if (total_tokens < 0 || num_seqs < 0) return KDA_ERR_INVALID_ARG;
    if (algo != KDA_ALGO_AUTO && algo != KDA_ALGO_CUDA_CORE && algo != KDA_ALGO_TENSOR_CORE &&
        algo != KDA_ALGO_TENSOR_CORE_SPLIT)
        return KDA_ERR_INVALID_ARG;
    const kda_status st = check_sizes(Hk, H, dk, dv, dt);
    if (st != KDA_OK) return st;
    if (algo == KDA_ALGO_TENSOR_CORE_SPLIT) return KDA_ERR_UNSUPPORTED;
    if (algo == KDA_ALGO_TENSOR_CORE && (dt != KDA_DTYPE_BF16 || dk != 128 || dv != 128))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

bool use_tensor_core(int32_t dk, int32_t dv, kda_dtype dt, kda_algo algo)
{
    return algo != KDA_ALGO_CUDA_CORE && dt == KDA_DTYPE_BF16 && dk == 128 && dv == 128;
}

kda_status status_of(cudaError_t err) { return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" size_t kda_gdr_prefill_workspace_size(int32_t total_tokens, int32_t num_seqs, int32_t Hk,
                                                 int32_t H, int32_t dk, int32_t dv, kda_dtype dt,
                                                 kda_algo algo)
{
    if (check_prefill(total_tokens, num_seqs, Hk, H, dk, dv, dt, algo) != KDA_OK) return 0;
    return use_tensor_core(dk, dv, dt, algo) ? kda::gdr_tensor_core_workspace(total_tokens, num_seqs, H) : 0;
}

extern "C" kda_status kda_gdr_prefill(const void *q, const void *k, const void *v, const float *g,
                                      const float *beta, const int32_t *cu_seqlens_dev,
                                      const int32_t *cu_seqlens_host, int32_t num_seqs,
                                      int32_t total_tokens, int32_t Hk, int32_t H, int32_t dk,
                                      int32_t dv, kda_dtype dt, float scale, float *state,
                                      int32_t pool_size, const int32_t *src_slots,
                                      const int32_t *dst_slots, const int32_t *ctx_lens,
                                      const int32_t *block_table, int32_t block_table_cols,
                                      int32_t block_size, void *o, void *workspace,
                                      size_t workspace_bytes, kda_algo algo, void *stream)
{
    const kda_status st = check_prefill(total_tokens, num_seqs, Hk, H, dk, dv, dt, algo);
    if (st != KDA_OK) return st;
    if (!isfinite(scale) || pool_size < 0 || block_size < 0 || block_size % 64 != 0 ||
        block_table_cols < 0)
        return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0) return KDA_OK;
    if (!cu_seqlens_dev) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !g || !beta || !o)) return KDA_ERR_INVALID_ARG;
    if (!state && (src_slots || dst_slots || block_size > 0)) return KDA_ERR_INVALID_ARG;
    if (block_size > 0 && (!block_table || block_table_cols == 0)) return KDA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)o, (const void *)state, (const void *)workspace})
        if (p && !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    for (const void *p : {(const void *)g, (const void *)beta, (const void *)cu_seqlens_dev,
                          (const void *)src_slots, (const void *)dst_slots, (const void *)ctx_lens,
                          (const void *)block_table})
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    if (cu_seqlens_host) {
        if (cu_seqlens_host[0] != 0 || cu_seqlens_host[num_seqs] != total_tokens)
            return KDA_ERR_INVALID_ARG;
        for (int32_t i = 0; i < num_seqs; ++i)
            if (cu_seqlens_host[i + 1] < cu_seqlens_host[i]) return KDA_ERR_INVALID_ARG;
    }
    const size_t need = kda_gdr_prefill_workspace_size(total_tokens, num_seqs, Hk, H, dk, dv, dt, algo);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;

    kda::GdrArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.num_seqs = num_seqs; a.total_tokens = total_tokens;
    a.Hk = Hk; a.H = H; a.dk = dk; a.dv = dv; a.bf16 = (dt == KDA_DTYPE_BF16);
    a.scale = scale;
    a.state = state; a.pool_size = pool_size; a.src = src_slots; a.dst = dst_slots;
    a.o = o;
    a.cu = cu_seqlens_dev; a.cu_host = cu_seqlens_host; a.ctx = ctx_lens;
    a.table = block_size > 0 ? block_table : nullptr;
    a.table_cols = block_table_cols; a.block = block_size;
    a.update = true;
    if (!use_tensor_core(dk, dv, dt, algo))
        return status_of(kda::launch_gdr_recurrent(a, (cudaStream_t)stream));
    if (!kda::device_status_word(&a.status)) return KDA_ERR_CUDA;
    return status_of(kda::launch_gdr_tensor_core(a, workspace, (cudaStream_t)stream));
}

namespace {

// Rows of completed blocks: none (kda_gdr_decode), or as the caller names them.
struct Blocks {
    const int32_t *ctx, *table;
    int32_t cols, size;
};

kda_status decode(const void *q, const void *k, const void *v, const float *g, const float *beta,
                  int32_t B, int32_t Tq, int32_t Hk, int32_t H, int32_t dk, int32_t dv, kda_dtype dt,
                  float scale, float *state, int32_t pool_size, const int32_t *src_slots,
                  const int32_t *dst_slots, const int32_t *num_tokens, int32_t update_state,
                  const Blocks *blocks, void *o, void *stream)
{
    if (B < 0 || Tq < 1 || Tq > 64 || pool_size < 0) return KDA_ERR_INVALID_ARG;
    const kda_status st = check_sizes(Hk, H, dk, dv, dt);
    if (st != KDA_OK) return st;
    if (!isfinite(scale) || (update_state != 0 && update_state != 1)) return KDA_ERR_INVALID_ARG;
    if (!update_state && dst_slots) return KDA_ERR_INVALID_ARG;
    if (blocks && (blocks->size <= 0 || blocks->cols < 0)) return KDA_ERR_INVALID_ARG;
    if (B == 0) return KDA_OK;
    if (!o && !update_state) return KDA_ERR_INVALID_ARG;   // verify without outputs does nothing
    if (!q || !k || !v || !g || !beta || !state) return KDA_ERR_INVALID_ARG;
    if (!src_slots && pool_size < B) return KDA_ERR_INVALID_ARG;
    if (blocks && (!blocks->table || blocks->cols == 0)) return KDA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)o, (const void *)state})
        if (p && !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    for (const void *p : {(const void *)g, (const void *)beta, (const void *)src_slots,
                          (const void *)dst_slots, (const void *)num_tokens,
                          (const void *)(blocks ? blocks->ctx : nullptr),
                          (const void *)(blocks ? blocks->table : nullptr)})
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    if ((int64_t)B * Tq > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;

    kda::GdrArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.num_seqs = B; a.total_tokens = B * Tq; a.Tq = Tq;
    a.Hk = Hk; a.H = H; a.dk = dk; a.dv = dv; a.bf16 = (dt == KDA_DTYPE_BF16);
    a.scale = scale;
    a.state = state; a.pool_size = pool_size; a.src = src_slots; a.dst = dst_slots;
    a.num_tokens = num_tokens; a.update = update_state != 0; a.o = o;
    if (blocks) {
        a.ctx = blocks->ctx; a.table = blocks->table;
        a.table_cols = blocks->cols; a.block = blocks->size;
    }
    return status_of(Tq == 1 ? kda::launch_gdr_step(a, (cudaStream_t)stream)
                             : kda::launch_gdr_recurrent(a, (cudaStream_t)stream));
}

}  // namespace

extern "C" kda_status kda_gdr_decode(const void *q, const void *k, const void *v, const float *g,
                                     const float *beta, int32_t B, int32_t Tq, int32_t Hk,
                                     int32_t H, int32_t dk, int32_t dv, kda_dtype dt, float scale,
                                     float *state, int32_t pool_size, const int32_t *src_slots,
                                     const int32_t *dst_slots, const int32_t *num_tokens,
                                     int32_t update_state, void *o, void *stream)
{
    return decode(q, k, v, g, beta, B, Tq, Hk, H, dk, dv, dt, scale, state, pool_size, src_slots,
                  dst_slots, num_tokens, update_state, nullptr, o, stream);
}

extern "C" kda_status kda_gdr_decode_blocks(
    const void *q, const void *k, const void *v, const float *g, const float *beta, int32_t B,
    int32_t Tq, int32_t Hk, int32_t H, int32_t dk, int32_t dv, kda_dtype dt, float scale,
    float *state, int32_t pool_size, const int32_t *src_slots, const int32_t *dst_slots,
    const int32_t *num_tokens, const int32_t *ctx_lens, const int32_t *block_table,
    int32_t block_table_cols, int32_t block_size, void *o, void *stream)
{
    const Blocks blocks = {ctx_lens, block_table, block_table_cols, block_size};
    return decode(q, k, v, g, beta, B, Tq, Hk, H, dk, dv, dt, scale, state, pool_size, src_slots,
                  dst_slots, num_tokens, 1, &blocks, o, stream);
}

extern "C" kda_status kda_block_plan(const int32_t *new_lens, const int32_t *ctx_lens,
                                     int32_t num_seqs, const int32_t *free_blocks,
                                     int32_t num_free, const int32_t *free_head,
                                     int32_t *block_table, int32_t block_table_cols,
                                     int32_t block_size, int32_t total_tokens, int32_t *cu_seqlens,
                                     int32_t *positions, int64_t *token_slots, int32_t *src_slots,
                                     int32_t *dst_slots, int32_t *free_head_out, void *stream)
{
    if (num_seqs < 0 || num_free < 0 || block_table_cols < 0 || block_size <= 0 || total_tokens < 0)
        return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens || !free_head || !free_head_out) return KDA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!new_lens || !block_table || block_table_cols == 0))
        return KDA_ERR_INVALID_ARG;
    if (num_free > 0 && !free_blocks) return KDA_ERR_INVALID_ARG;
    if ((int64_t)num_seqs * block_table_cols > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    for (const void *p : {(const void *)new_lens, (const void *)ctx_lens, (const void *)free_blocks,
                          (const void *)free_head, (const void *)block_table,
                          (const void *)cu_seqlens, (const void *)positions,
                          (const void *)src_slots, (const void *)dst_slots,
                          (const void *)free_head_out})
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    if (token_slots && !aligned(token_slots, 8)) return KDA_ERR_INVALID_ARG;

    kda::BlockPlanArgs a{};
    a.new_lens = new_lens; a.ctx_lens = ctx_lens; a.num_seqs = num_seqs;
    a.free_blocks = free_blocks; a.num_free = num_free; a.free_head = free_head;
    a.block_table = block_table; a.table_cols = block_table_cols; a.block = block_size;
    a.total_tokens = total_tokens;
    a.cu = cu_seqlens; a.positions = positions; a.token_slots = token_slots;
    a.src = src_slots; a.dst = dst_slots; a.free_head_out = free_head_out;
    return status_of(kda::launch_block_plan(a, (cudaStream_t)stream));
}
