// Internal launch interface of the gated delta rule (one log-decay per token and
// head) and of the block plan; the C-ABI layer is kda_gdr_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Longest-first launch order is passed by value for up to this many sequences.
constexpr int kGdrMaxOrder = 512;

struct GdrArgs {
    const void *q, *k, *v;          // [tokens, Hk, dk], [tokens, Hk, dk], [tokens, H, dv]
    const float *g, *beta;          // [tokens, H]
    int32_t num_seqs, total_tokens, Hk, H, dk, dv;
    bool bf16;                      // storage dtype of q, k, v, o
    float scale;
    float *state;                   // pool [pool_size, H, dk, dv] or nullptr
    int32_t pool_size;
    const int32_t *src, *dst;       // pool rows per sequence, see the C ABI
    void *o;                        // [tokens, H, dv] (decode: nullptr = no outputs)
    // Prefill: packed sequences.
    const int32_t *cu;              // device [num_seqs + 1]; nullptr = decode layout
    const int32_t *cu_host;         // host copy or nullptr (launch order, segments)
    // Rows of the blocks that the call completes.
    const int32_t *ctx;             // tokens before this call, or nullptr = 0
    const int32_t *table;           // [num_seqs, table_cols] or nullptr
    int32_t table_cols, block;      // block = 0: none
    // Decode: Tq tokens per sequence, of which num_tokens[n] count.
    int32_t Tq;
    const int32_t *num_tokens;
    bool update;                    // write the states back
    int32_t *status;                // device status word (tensor-core path)
};

// Token-by-token recurrence on states held in registers: every dtype and size,
// prefill layout (a.cu) or Tq tokens per sequence.
cudaError_t launch_gdr_recurrent(const GdrArgs &a, cudaStream_t stream);

// One token per sequence (a.Tq == 1), one pass over each state.
cudaError_t launch_gdr_step(const GdrArgs &a, cudaStream_t stream);

// Chunked prefill on tensor cores (bf16, dk = dv = 128; a.cu and a.status set), with a workspace
// of gdr_tensor_core_workspace bytes, 16-byte aligned.
size_t gdr_tensor_core_workspace(int32_t total_tokens, int32_t num_seqs, int32_t H);
cudaError_t launch_gdr_tensor_core(const GdrArgs &a, void *workspace, cudaStream_t stream);

struct BlockPlanArgs {
    const int32_t *new_lens, *ctx_lens;
    int32_t num_seqs;
    const int32_t *free_blocks;
    int32_t num_free;
    const int32_t *free_head;
    int32_t *block_table;
    int32_t table_cols, block, total_tokens;
    int32_t *cu, *positions;
    int64_t *token_slots;
    int32_t *src, *dst, *free_head_out;
};
cudaError_t launch_block_plan(const BlockPlanArgs &a, cudaStream_t stream);

}  // namespace kda
