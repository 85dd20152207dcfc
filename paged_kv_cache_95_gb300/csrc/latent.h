// latent.h -- internal interface between latent_api.cu and the latent-attention kernels.
#pragma once

#include "launch.h"

namespace pkv {

constexpr int kLatentDim = 512;                      // values of the shared latent a token
constexpr int kRopeDim = 64;                         // values of the rotated key a token
constexpr int kLatentRow = kLatentDim + kRopeDim;    // a bf16 pool row
constexpr int kNopeDim = 128;                        // expanded head: key part from the latent
constexpr int kExpandedQk = kNopeDim + kRopeDim;     // expanded head: query / key values
constexpr int kExpandedV = 128;                      // expanded head: value values

// ---- cache write and read-back ------------------------------------------------
struct LatentWriteParams {
    const void *latent;  // bf16 rows of 512, latent_stride elements apart
    const void *rope;    // bf16 rows of 64, rope_stride elements apart
    int64_t latent_stride, rope_stride;
    void *cache;         // bf16 [slots][576], or E4M3 codes [slots][512]
    void *rope_cache;    // FP8 pool: bf16 [slots][64]
    float *cache_scale;  // FP8 pool: [slots]
    const int32_t *slot_mapping;
    int64_t num_slots;
    int32_t num_tokens;
};
cudaError_t launch_latent_write(const LatentWriteParams &p, bool fp8, int sm_count, cudaStream_t stream);

struct LatentGatherParams {
    void *out;  // bf16 [total_rows][576]
    const void *cache, *rope_cache;
    const float *cache_scale;
    const int32_t *block_tables;
    const int32_t *cu_lens;
    uint32_t *status;
    int32_t num_seqs, max_blocks, num_blocks, total_rows;
};
cudaError_t launch_latent_gather(const LatentGatherParams &p, bool fp8, cudaStream_t stream);

// ---- absorbed attention -----------------------------------------------------------
struct LatentDecodeParams {
    void *out;  // [rows][heads][512], f32 or bf16
    const void *q_latent, *q_rope;
    int64_t ql_row, ql_head, qr_row, qr_head;  // strides in elements
    const void *cache, *rope_cache;            // rope_cache, cache_scale: FP8 pool only
    const float *cache_scale;
    const int32_t *block_tables;
    const int32_t *context_lens;
    uint32_t *status;
    int32_t num_seqs, q_per_seq, heads, max_blocks, num_blocks;
    float scale_log2;
    int32_t out_bf16;
    // The split: the q_per_seq x heads columns of a sequence in col_tiles tiles of cols_per_tile
    // (the last may hold fewer), the keys of all sequences in `ranges` ranges of tiles.
    int32_t col_tiles, cols_per_tile, ranges;
    int2 *record;            // [ranges]: the split sequence that begins in the range, and its parts (0: none)
    float2 *part_ml;         // [ranges][2][col_tiles * cols_per_tile] (m, l), log2 domain, scale folded in
    float *part_o;           // the same x [512], unnormalised
};
constexpr int kLatentMaxRanges = 160;  // at least the SMs (152); the merge keeps 5 records a lane
constexpr int kLatentMaxCols = 64;     // columns a CTA takes
constexpr int kLatentTile = 32;        // keys of the smallest tile
cudaError_t latent_decode_prepare_device();
struct LatentDecodeMaps {
    CUtensorMap kv, rope;  // rope: FP8 pool only
};
cudaError_t launch_latent_decode(const LatentDecodeMaps &maps, const LatentDecodeParams &p, bool fp8, cudaStream_t stream);

// ---- expanded attention of a prefill chunk --------------------------------------------
struct LatentPrefillParams {
    void *out;  // [rows][heads][128], f32 or bf16
    const void *q, *v;                      // (keys and the first row tile's q come by their tensor maps)
    int64_t q_row, q_head, k_row, k_head;  // strides in elements
    const int32_t *cu_q_lens, *cu_k_lens;
    uint32_t *status;
    int32_t num_seqs, heads, max_q_len, total_q, total_k;
    float scale_log2;
    int32_t out_bf16;
    int32_t pairs;   // of row tiles in the longest chunk
    int32_t splits;  // parts of a pair's key tiles (1: no partials)
    float2 *part_ml;  // [splits][total_q][heads] (m, l), log2 domain, scale folded in
    float *part_o;    // the same x [128], unnormalised
};
constexpr int kLatentMaxSplits = 32;  // the merge keeps a split a lane
struct LatentPrefillMaps {
    CUtensorMap q, k, rope;
};
cudaError_t latent_prefill_prepare_device();
cudaError_t launch_latent_prefill(const LatentPrefillMaps &maps, const LatentPrefillParams &p, cudaStream_t stream);

}  // namespace pkv
