// speculative.h -- internal interface between speculative_api.cu and the kernels of a
// speculative decoding step (rotary positions, tree attention, verification, compaction).
#pragma once

#include "launch.h"

namespace pkv {

// ---- rotary positions ------------------------------------------------------------
constexpr int kRotaryUnit = 16;  // values a thread turns: 8 pairs

struct RotaryParams {
    void *out;
    const void *x;
    int64_t out_row, out_head, x_row, x_head;  // strides in elements
    const int32_t *positions;
    const uint64_t *frequencies;  // [rotary_dim / 2], turns a position in units of 2^-64
    int32_t num_tokens, num_heads, head_dim, rotary_dim;
    float magnitude;
};
cudaError_t launch_rotary(const RotaryParams &p, bool interleaved, int sm_count, cudaStream_t stream);

struct RotaryWriteParams {
    void *q_out;  // bf16 [tokens][heads][128]
    const void *q, *key, *value;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;  // strides in elements
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;  // FP8 pool only
    const int32_t *positions, *slot_mapping;
    const uint64_t *frequencies;
    int64_t num_slots;
    int32_t num_tokens, n_q, n_kv, rotary_dim;
    float magnitude;
};
cudaError_t launch_rotary_write(const RotaryWriteParams &p, bool interleaved, bool fp8, int sm_count,
                                cudaStream_t stream);

// ---- attention of a tree's rows over the cache ---------------------------------------
constexpr int kMaxTreeNodes = 64;  // nodes of a sequence's tree: the bits of a mask

struct TreeParams {
    const void *q;  // bf16 [total_rows][n_q][128]
    void *out;      // [total_rows][n_q][128], f32 or bf16
    const uint64_t *mask;  // [total_rows]
    const int32_t *cu_q_lens, *block_tables, *context_lens;
    const float *k_scale, *v_scale;  // FP8 pool only
    uint32_t *status;
    int32_t num_seqs, n_q, n_kv, group, max_blocks, num_blocks, total_rows, max_q_len;
    int32_t whole_nodes;   // 128 / group where that is whole (Q by copies of whole nodes), else 0
    uint32_t group_magic;  // 2^32 / group rounded up (0 for a group of 1)
    float scale_log2;
    int32_t out_bf16;
    // The split: all (sequence, KV head, 128-row tile) units' key tiles in `ranges` equal ranges, one a CTA.
    int32_t ranges, part_rows;  // part_rows: rows of a partial (the most a row tile holds)
    int4 *record;               // [ranges]: the split unit that begins in the range (first row of q, KV head, parts (0: none),
                                // row tile x 256 + its rows)
    float2 *part_ml;            // [ranges][2][part_rows] (m, l), log2 domain, scale folded in
    float *part_o;              // the same x [128], unnormalised
};
cudaError_t tree_prepare_device();
cudaError_t launch_tree_attention(const CUtensorMap &kmap, const CUtensorMap &vmap, const CUtensorMap &qmap, const TreeParams &p, bool fp8,
                                  cudaStream_t stream);

// ---- verification of drafted tokens, compaction of the accepted path -----------------
struct SpecVerifyParams {
    int32_t *tokens_out, *path;  // [num_seqs][max_q_len]
    int32_t *counts;             // [num_seqs]
    const float *target, *draft;  // rows of vocab probabilities
    int64_t target_row, draft_row;
    const int32_t *tokens, *parents, *cu_q_lens;
    const float *uniforms;
    uint32_t *status;
    int32_t num_seqs, max_q_len, total_rows, vocab;
    int32_t segment;  // vocabulary entries a warp sums
};
cudaError_t launch_speculative_verify(const SpecVerifyParams &p, int cluster, cudaStream_t stream);
constexpr int kVerifyWarps = 16;
constexpr int kVerifyMaxCluster = 8;

struct CompactParams {
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;
    const int32_t *block_tables, *context_lens, *cu_q_lens, *path, *counts;
    uint32_t *status;
    int32_t num_seqs, max_blocks, num_blocks, n_kv, path_len;
};
cudaError_t launch_kv_compact_path(const CompactParams &p, bool fp8, cudaStream_t stream);

}  // namespace pkv
