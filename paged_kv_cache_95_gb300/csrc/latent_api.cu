// latent_api.cu -- the extern "C" entry points of the latent-attention operators
// declared in include/pagedkv.h: argument validation before anything is enqueued,
// then the kernel launches on the caller's stream.  No allocation, no
// synchronisation.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/pagedkv.h"
#include "latent.h"
#include "tensor_map.h"

namespace {

using pkv::kBlockSize;

constexpr size_t kStatusBytes = 256;
constexpr int kMaxDevices = 64;
constexpr int kDefaultSms = 152;  // sizes asked for without a GPU
constexpr int32_t kMaxRowsPerSeq = 16;
constexpr int32_t kMaxHeads = 1024;
constexpr int64_t kMinSplitTiles = 6;  // key tiles from which a pair's are split (4 tiles: 10.1 us whole, 11.8 in parts)
constexpr int32_t kMaxChunk = 65535 * 256;  // query rows of a prefill chunk: 256 a step of the launch grid

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The current device (-1: none) and its SM count (0: none), looked up once per device.
std::atomic<int> g_sms[kMaxDevices];
int current_device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : -1;
}
int current_sms() {
    const int dev = current_device();
    if (dev < 0) return 0;
    int v = g_sms[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    g_sms[dev].store(v, std::memory_order_relaxed);
    return v;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Kernel attributes, set once per device; false on failure.
std::once_flag g_prepared[kMaxDevices];
cudaError_t g_prepare_err[kMaxDevices];
bool prepare_device() {
    const int dev = current_device();
    if (dev < 0) return false;
    std::call_once(g_prepared[dev], [&] {
        g_prepare_err[dev] = pkv::latent_decode_prepare_device();
        if (g_prepare_err[dev] == cudaSuccess) g_prepare_err[dev] = pkv::latent_prefill_prepare_device();
    });
    return g_prepare_err[dev] == cudaSuccess;
}

// Rows [rows][heads][width] bf16 at free (row, head) strides (in elements); a box is 64
// values of one head of box_rows rows, 128-byte swizzle: [row][128 B].
bool encode_rows(CUtensorMap *map, const void *base, int32_t rows, int32_t heads, int32_t width, int64_t row_stride,
                 int64_t head_stride, uint32_t box_rows) {
    const pkv::EncodeTiledFn fn = pkv::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
    const cuuint32_t box[3] = {64, 1, box_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for rows without heads: [rows][64].
bool encode_rows_2d(CUtensorMap *map, const void *base, int32_t rows, int64_t row_stride, uint32_t box_rows) {
    const pkv::EncodeTiledFn fn = pkv::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {64, static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_stride) * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A bf16 pool [num_blocks][16][576] viewed so that one box is a whole block in the order
// the tensor core wants it: dims inner -> outer are 64 values (128 bytes), 8 slots, the 9
// chunks of 64 values, the two groups of 8 slots, the block; it lands as
// [slot group][chunk][8 slots][128 B], eighteen 1 KB swizzle atoms.
bool encode_latent_map(CUtensorMap *map, const void *base, int32_t num_blocks) {
    const pkv::EncodeTiledFn fn = pkv::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[5] = {64, 8, 9, 2, static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t strides[4] = {pkv::kLatentRow * 2, 128, pkv::kLatentRow * 16, pkv::kLatentRow * 32};
    const cuuint32_t box[5] = {64, 8, 9, 2, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An FP8 pool: the codes [num_blocks][16][512] the same way (128 codes a chunk, 4 chunks), the
// rotated keys [num_blocks][16][64] bf16 as [16 slots][128 B].
bool encode_latent_maps_fp8(pkv::LatentDecodeMaps *maps, const void *codes, const void *rope, int32_t num_blocks) {
    const pkv::EncodeTiledFn fn = pkv::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[5] = {128, 8, 4, 2, static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t strides[4] = {pkv::kLatentDim, 128, pkv::kLatentDim * 8, pkv::kLatentDim * 16};
    const cuuint32_t box[5] = {128, 8, 4, 2, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const cuuint64_t rdims[3] = {64, 16, static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t rstrides[2] = {128, 2048};
    const cuuint32_t rbox[3] = {64, 16, 1};
    return fn(&maps->kv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(codes), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
           fn(&maps->rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(rope), rdims, rstrides, rbox, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a decode call is split: one CTA per SM, column tiles of at most 64 columns of equal
// size, and as many ranges of keys as there are SMs for a column tile (never more than
// tiles).  Workspace: [status 256 B | records | part_ml | part_o].
struct DecodePlan {
    int32_t col_tiles, cols_per_tile, ranges;
    size_t off_ml, off_o, total;
};
DecodePlan plan_decode(int32_t num_seqs, int32_t q_per_seq, int32_t heads, int32_t max_blocks, int sms) {
    DecodePlan pl{};
    const int32_t cols = heads * q_per_seq;
    pl.col_tiles = (cols + pkv::kLatentMaxCols - 1) / pkv::kLatentMaxCols;
    pl.cols_per_tile = (cols + pl.col_tiles - 1) / pl.col_tiles;
    const int64_t tiles = static_cast<int64_t>(num_seqs) *
                          ((static_cast<int64_t>(max_blocks) * kBlockSize + pkv::kLatentTile - 1) / pkv::kLatentTile);
    const int64_t ranges = std::min<int64_t>(std::max(1, sms / pl.col_tiles), tiles);
    pl.ranges = static_cast<int32_t>(std::min<int64_t>(ranges, pkv::kLatentMaxRanges));
    const size_t rows = static_cast<size_t>(pl.ranges) * 2 * pl.col_tiles * pl.cols_per_tile;
    pl.off_ml = kStatusBytes + align_up(static_cast<size_t>(pl.ranges) * 8, 256);
    pl.off_o = pl.off_ml + align_up(rows * 8, 256);
    pl.total = pl.off_o + rows * pkv::kLatentDim * 4;
    return pl;
}

// How a prefill call is split: pairs of row tiles (256 rows) over the grid, and where those do not fill the GPU their key
// tiles in parts (the lengths are device data: the parts follow from the totals).  Workspace: [status 256 B | part_ml |
// part_o].
struct PrefillPlan {
    int32_t pairs, splits;
    size_t off_o, total;
};
PrefillPlan plan_prefill(int32_t num_seqs, int32_t heads, int32_t max_q_len, int32_t total_q, int32_t total_k, int sms) {
    PrefillPlan pl{};
    pl.pairs = (std::min(max_q_len, total_q) + 255) / 256;
    const int64_t units = static_cast<int64_t>(heads) *
                          std::min<int64_t>(static_cast<int64_t>(num_seqs) * pl.pairs, (static_cast<int64_t>(total_q) + 255) / 256 + num_seqs);
    const int64_t tiles = (static_cast<int64_t>(total_k) / num_seqs + 127) / 128;
    // A part costs its tiles (1 us each) and its share of the merge (0.4 us): sqrt(2.5 tiles) parts are least.  100 rows x 8
    // heads over 1000 / 2000 / 4000 keys: 14.1 -> 11.7, 22.3 -> 12.9, 38.5 -> 14.3 us; 512 rows x 16 heads over 4000: 64.7 -> 31.
    const int64_t best = static_cast<int64_t>(std::sqrt(2.5 * static_cast<double>(tiles)));
    const int64_t splits = units > 0 && tiles >= kMinSplitTiles ? std::min<int64_t>({sms / units, best, pkv::kLatentMaxSplits}) : 1;
    pl.splits = static_cast<int32_t>(std::max<int64_t>(splits, 1));
    const size_t rows = pl.splits > 1 ? static_cast<size_t>(pl.splits) * total_q * heads : 0;
    pl.off_o = kStatusBytes + align_up(rows * 8, 256);
    pl.total = pl.off_o + rows * pkv::kExpandedV * 4;
    return pl;
}

int check_latent(const pkv_latent_desc *d, int32_t dtype) {
    if (!d || d->num_blocks < 1) return PKV_ERR_INVALID_ARG;
    if (d->block_size != kBlockSize || d->latent_dim != pkv::kLatentDim || d->rope_dim != pkv::kRopeDim ||
        d->dtype != dtype)
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// A strided bf16 input: 16-byte vectors at every row, offsets that 64 bits hold.
bool good_stride(int64_t s) { return s >= 0 && s % 8 == 0 && s < (int64_t{1} << 38); }

// The softmax scale in the log2 domain, which has to be finite too.
bool log2_scale(float scale, float *out) {
    *out = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    return std::isfinite(*out);
}

// Lengths that the kernels may round up to whole tiles within 32 bits.
constexpr int64_t kMaxLength = INT32_MAX - 4096;

int write_impl(const void *latent, int64_t latent_stride, const void *rope, int64_t rope_stride, void *cache,
               void *rope_cache, float *cache_scale, const int32_t *slot_mapping, int32_t num_tokens,
               const pkv_latent_desc *desc, bool fp8, void *stream) {
    if (int rc = check_latent(desc, fp8 ? PKV_DTYPE_FP8_E4M3 : PKV_DTYPE_BF16)) return rc;
    if (num_tokens < 0 || !good_stride(latent_stride) || !good_stride(rope_stride)) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!latent || !rope || !cache || !slot_mapping) return PKV_ERR_INVALID_ARG;
    if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(cache, 16) || !aligned(slot_mapping, 4))
        return PKV_ERR_INVALID_ARG;
    if (fp8 && (!rope_cache || !cache_scale || !aligned(rope_cache, 16) || !aligned(cache_scale, 16)))
        return PKV_ERR_INVALID_ARG;
    const int sms = current_sms();
    if (sms < 1) return PKV_ERR_CUDA;
    pkv::LatentWriteParams p{};
    p.latent = latent;
    p.rope = rope;
    p.latent_stride = latent_stride;
    p.rope_stride = rope_stride;
    p.cache = cache;
    p.rope_cache = rope_cache;
    p.cache_scale = cache_scale;
    p.slot_mapping = slot_mapping;
    p.num_slots = static_cast<int64_t>(desc->num_blocks) * kBlockSize;
    p.num_tokens = num_tokens;
    return pkv::launch_latent_write(p, fp8, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK
                                                                                                   : PKV_ERR_CUDA;
}

// Sizes shared by the absorbed form's entry points and its workspace query.
int check_decode_sizes(int32_t num_seqs, int32_t q_per_seq, int32_t heads, int32_t max_blocks) {
    if (num_seqs < 1 || num_seqs > 65535 || q_per_seq < 1 || q_per_seq > kMaxRowsPerSeq || heads < 1 || max_blocks < 1)
        return PKV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_blocks) * kBlockSize > kMaxLength) return PKV_ERR_INVALID_ARG;
    if (heads > kMaxHeads) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

int decode_impl(void *out, int32_t out_dtype, const void *q_latent, int64_t ql_row, int64_t ql_head,
                const void *q_rope, int64_t qr_row, int64_t qr_head, const void *cache, const void *rope_cache,
                const float *cache_scale, const int32_t *block_tables, const int32_t *context_lens, int32_t num_seqs,
                int32_t q_per_seq, int32_t heads, int32_t max_blocks, float scale, const pkv_latent_desc *desc,
                bool fp8, void *workspace, size_t workspace_bytes, void *stream) {
    if (int rc = check_latent(desc, fp8 ? PKV_DTYPE_FP8_E4M3 : PKV_DTYPE_BF16)) return rc;
    if (int rc = check_decode_sizes(num_seqs, q_per_seq, heads, max_blocks)) return rc;
    if (!out || !q_latent || !q_rope || !cache || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
    if (fp8 && (!rope_cache || !cache_scale || !aligned(rope_cache, 16) || !aligned(cache_scale, 16)))
        return PKV_ERR_INVALID_ARG;
    if (out_dtype != PKV_DTYPE_FLOAT32 && out_dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    pkv::LatentDecodeParams p{};
    if (!log2_scale(scale, &p.scale_log2)) return PKV_ERR_INVALID_ARG;
    if (!good_stride(ql_row) || !good_stride(ql_head) || !good_stride(qr_row) || !good_stride(qr_head))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q_latent, 16) || !aligned(q_rope, 16) || !aligned(cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256)) return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < latent_attention_workspace_size(num_seqs, q_per_seq, heads, max_blocks, desc))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    p.out = out;
    p.q_latent = q_latent;
    p.q_rope = q_rope;
    p.ql_row = ql_row;
    p.ql_head = ql_head;
    p.qr_row = qr_row;
    p.qr_head = qr_head;
    p.cache = cache;
    p.rope_cache = rope_cache;
    p.cache_scale = cache_scale;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.status = static_cast<uint32_t *>(workspace);
    p.num_seqs = num_seqs;
    p.q_per_seq = q_per_seq;
    p.heads = heads;
    p.max_blocks = max_blocks;
    p.num_blocks = desc->num_blocks;
    p.out_bf16 = out_dtype == PKV_DTYPE_BF16;
    const int sms = current_sms();
    if (sms < 1 || !prepare_device()) return PKV_ERR_CUDA;
    const DecodePlan pl = plan_decode(num_seqs, q_per_seq, heads, max_blocks, sms);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.col_tiles = pl.col_tiles;
    p.cols_per_tile = pl.cols_per_tile;
    p.ranges = pl.ranges;
    p.record = reinterpret_cast<int2 *>(ws + kStatusBytes);
    p.part_ml = reinterpret_cast<float2 *>(ws + pl.off_ml);
    p.part_o = reinterpret_cast<float *>(ws + pl.off_o);
    pkv::LatentDecodeMaps maps{};
    if (fp8 ? !encode_latent_maps_fp8(&maps, cache, rope_cache, desc->num_blocks)
            : !encode_latent_map(&maps.kv, cache, desc->num_blocks))
        return PKV_ERR_CUDA;
    return pkv::launch_latent_decode(maps, p, fp8, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK
                                                                                                     : PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

int latent_reshape_and_cache(const void *latent, int64_t latent_stride, const void *rope, int64_t rope_stride,
                             void *cache, const int32_t *slot_mapping, int32_t num_tokens, const pkv_latent_desc *desc,
                             void *stream) {
    return write_impl(latent, latent_stride, rope, rope_stride, cache, nullptr, nullptr, slot_mapping, num_tokens, desc,
                      false, stream);
}

int latent_reshape_and_cache_fp8(const void *latent, int64_t latent_stride, const void *rope, int64_t rope_stride,
                                 void *cache, void *rope_cache, float *cache_scale, const int32_t *slot_mapping,
                                 int32_t num_tokens, const pkv_latent_desc *desc, void *stream) {
    return write_impl(latent, latent_stride, rope, rope_stride, cache, rope_cache, cache_scale, slot_mapping,
                      num_tokens, desc, true, stream);
}

int latent_gather(void *out, const void *cache, const void *rope_cache, const float *cache_scale,
                  const int32_t *block_tables, const int32_t *cu_lens, int32_t num_seqs, int32_t max_blocks_per_seq,
                  int32_t total_rows, const pkv_latent_desc *desc, uint32_t *status, void *stream) {
    if (!desc) return PKV_ERR_INVALID_ARG;
    const bool fp8 = desc->dtype == PKV_DTYPE_FP8_E4M3;
    if (int rc = check_latent(desc, fp8 ? PKV_DTYPE_FP8_E4M3 : PKV_DTYPE_BF16)) return rc;
    if (num_seqs < 1 || max_blocks_per_seq < 1 || total_rows < 0) return PKV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_blocks_per_seq) * kBlockSize > kMaxLength || total_rows > kMaxLength)
        return PKV_ERR_INVALID_ARG;
    if (total_rows == 0) return PKV_OK;
    if (!out || !cache || !block_tables || !cu_lens) return PKV_ERR_INVALID_ARG;
    if (fp8 ? (!rope_cache || !cache_scale || !aligned(rope_cache, 16) || !aligned(cache_scale, 16))
            : (rope_cache || cache_scale))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(cache, 16) || !aligned(block_tables, 4) || !aligned(cu_lens, 4) ||
        !aligned(status, 4))
        return PKV_ERR_INVALID_ARG;
    pkv::LatentGatherParams p{};
    p.out = out;
    p.cache = cache;
    p.rope_cache = rope_cache;
    p.cache_scale = cache_scale;
    p.block_tables = block_tables;
    p.cu_lens = cu_lens;
    p.status = status;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = desc->num_blocks;
    p.total_rows = total_rows;
    return pkv::launch_latent_gather(p, fp8, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

size_t latent_attention_workspace_size(int32_t num_seqs, int32_t q_per_seq, int32_t num_q_heads,
                                       int32_t max_blocks_per_seq, const pkv_latent_desc *desc) {
    if (!desc || check_latent(desc, desc->dtype == PKV_DTYPE_FP8_E4M3 ? PKV_DTYPE_FP8_E4M3 : PKV_DTYPE_BF16) != PKV_OK)
        return 0;
    if (check_decode_sizes(num_seqs, q_per_seq, num_q_heads, max_blocks_per_seq) != PKV_OK) return 0;
    const int sms = current_sms();
    return plan_decode(num_seqs, q_per_seq, num_q_heads, max_blocks_per_seq, sms > 0 ? sms : kDefaultSms).total;
}

int latent_attention_decode(void *out, int32_t out_dtype, const void *q_latent, int64_t q_latent_row_stride,
                            int64_t q_latent_head_stride, const void *q_rope, int64_t q_rope_row_stride,
                            int64_t q_rope_head_stride, const void *cache, const int32_t *block_tables,
                            const int32_t *context_lens, int32_t num_seqs, int32_t q_per_seq, int32_t num_q_heads,
                            int32_t max_blocks_per_seq, float scale, const pkv_latent_desc *desc, void *workspace,
                            size_t workspace_bytes, void *stream) {
    return decode_impl(out, out_dtype, q_latent, q_latent_row_stride, q_latent_head_stride, q_rope, q_rope_row_stride,
                       q_rope_head_stride, cache, nullptr, nullptr, block_tables, context_lens, num_seqs, q_per_seq,
                       num_q_heads, max_blocks_per_seq, scale, desc, false, workspace, workspace_bytes, stream);
}

int latent_attention_decode_fp8(void *out, int32_t out_dtype, const void *q_latent, int64_t q_latent_row_stride,
                                int64_t q_latent_head_stride, const void *q_rope, int64_t q_rope_row_stride,
                                int64_t q_rope_head_stride, const void *cache, const void *rope_cache,
                                const float *cache_scale, const int32_t *block_tables, const int32_t *context_lens,
                                int32_t num_seqs, int32_t q_per_seq, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                float scale, const pkv_latent_desc *desc, void *workspace, size_t workspace_bytes,
                                void *stream) {
    return decode_impl(out, out_dtype, q_latent, q_latent_row_stride, q_latent_head_stride, q_rope, q_rope_row_stride,
                       q_rope_head_stride, cache, rope_cache, cache_scale, block_tables, context_lens, num_seqs,
                       q_per_seq, num_q_heads, max_blocks_per_seq, scale, desc, true, workspace, workspace_bytes,
                       stream);
}

size_t latent_attention_prefill_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t max_q_len,
                                               int32_t total_q_rows, int32_t total_k_rows) {
    if (num_seqs < 1 || num_seqs > 65535 || num_heads < 1 || num_heads > kMaxHeads || max_q_len < 0 ||
        total_q_rows < 0 || total_k_rows < 0)
        return 0;
    const int sms = current_sms();
    return plan_prefill(num_seqs, num_heads, max_q_len, total_q_rows, total_k_rows, sms > 0 ? sms : kDefaultSms).total;
}

int latent_attention_prefill_chunk(void *out, int32_t out_dtype, const void *q, int64_t q_row_stride,
                                   int64_t q_head_stride, const void *k_nope, const void *v, int64_t k_row_stride,
                                   int64_t k_head_stride, const void *k_rope, int64_t k_rope_stride,
                                   const int32_t *cu_q_lens, const int32_t *cu_k_lens, int32_t num_seqs,
                                   int32_t num_heads, int32_t max_q_len, int32_t total_q_rows, int32_t total_k_rows,
                                   float scale, void *workspace, size_t workspace_bytes, void *stream) {
    if (num_seqs < 1 || num_seqs > 65535 || num_heads < 1 || max_q_len < 0 || total_q_rows < 0 || total_k_rows < 0)
        return PKV_ERR_INVALID_ARG;
    if (total_q_rows > kMaxLength || total_k_rows > kMaxLength) return PKV_ERR_INVALID_ARG;
    if (num_heads > kMaxHeads || std::min(max_q_len, total_q_rows) > kMaxChunk) return PKV_ERR_UNSUPPORTED;
    if (out_dtype != PKV_DTYPE_FLOAT32 && out_dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    pkv::LatentPrefillParams p{};
    if (!log2_scale(scale, &p.scale_log2)) return PKV_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256)) return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < kStatusBytes) return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (max_q_len == 0 || total_q_rows == 0) return PKV_OK;
    if (!out || !q || !k_nope || !v || !k_rope || !cu_q_lens || !cu_k_lens || total_k_rows < 1)
        return PKV_ERR_INVALID_ARG;
    // Rows and heads are boxes of a tensor map: distinct, 16 bytes apart at least.
    if (!good_stride(q_row_stride) || !good_stride(q_head_stride) || !good_stride(k_row_stride) ||
        !good_stride(k_head_stride) || !good_stride(k_rope_stride) || q_row_stride < 8 || q_head_stride < 8 ||
        k_row_stride < 8 || k_head_stride < 8 || k_rope_stride < 8)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_nope, 16) || !aligned(v, 16) || !aligned(k_rope, 16) ||
        !aligned(cu_q_lens, 4) || !aligned(cu_k_lens, 4))
        return PKV_ERR_INVALID_ARG;
    p.out = out;
    p.q = q;
    p.v = v;
    p.q_row = q_row_stride;
    p.q_head = q_head_stride;
    p.k_row = k_row_stride;
    p.k_head = k_head_stride;
    p.cu_q_lens = cu_q_lens;
    p.cu_k_lens = cu_k_lens;
    p.status = static_cast<uint32_t *>(workspace);
    p.num_seqs = num_seqs;
    p.heads = num_heads;
    p.max_q_len = max_q_len;
    p.total_q = total_q_rows;
    p.total_k = total_k_rows;
    p.out_bf16 = out_dtype == PKV_DTYPE_BF16;
    if (p.scale_log2 == 0.f) p.scale_log2 = 1e-37f;  // the kernel hides a key by an infinite score: never 0 x infinity
    const int sms = current_sms();
    if (sms < 1 || !prepare_device()) return PKV_ERR_CUDA;
    PrefillPlan pl = plan_prefill(num_seqs, num_heads, max_q_len, total_q_rows, total_k_rows, sms);
    if (workspace_bytes < pl.total) pl.splits = 1;  // the status word alone
    p.pairs = pl.pairs;
    p.splits = pl.splits;
    p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + kStatusBytes);
    p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + pl.off_o);
    pkv::LatentPrefillMaps maps;
    if (!encode_rows(&maps.q, q, total_q_rows, num_heads, pkv::kExpandedQk, q_row_stride, q_head_stride, 128) ||
        !encode_rows(&maps.k, k_nope, total_k_rows, num_heads, pkv::kNopeDim, k_row_stride, k_head_stride, 128) ||
        !encode_rows_2d(&maps.rope, k_rope, total_k_rows, k_rope_stride, 128))
        return PKV_ERR_CUDA;
    return pkv::launch_latent_prefill(maps, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK
                                                                                                : PKV_ERR_CUDA;
}

}  // extern "C"
