// speculative_api.cu -- the extern "C" entry points of a speculative decoding step's operators
// declared in include/pagedkv.h: argument validation before anything is enqueued, then the kernel
// launches on the caller's stream.  No allocation, no synchronisation.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/pagedkv.h"
#include "speculative.h"
#include "tensor_map.h"

namespace {

using pkv::kBlockSize;
using pkv::kHeadDim;

constexpr int kMaxDevices = 64;

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

int check_pool(const pkv_cache_desc *c, bool fp8) {
    if (!c || c->num_blocks < 1 || c->num_kv_heads < 1) return PKV_ERR_INVALID_ARG;
    if (c->block_size != kBlockSize || c->head_dim != kHeadDim ||
        c->dtype != (fp8 ? PKV_DTYPE_FP8_E4M3 : PKV_DTYPE_BF16))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// A strided bf16 tensor: 16-byte vectors at every row, offsets that 64 bits hold.
bool good_stride(int64_t s) { return s >= 0 && s % 8 == 0 && s < (int64_t{1} << 38); }

int check_rotation(int32_t head_dim, int32_t rotary_dim, int32_t layout, float magnitude) {
    if (layout != PKV_ROTARY_HALF && layout != PKV_ROTARY_INTERLEAVED) return PKV_ERR_INVALID_ARG;
    if (rotary_dim < 1 || rotary_dim > head_dim || !std::isfinite(magnitude)) return PKV_ERR_INVALID_ARG;
    if (head_dim % pkv::kRotaryUnit != 0 || rotary_dim % pkv::kRotaryUnit != 0) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// The softmax scale in the log2 domain, which has to be finite too.
bool log2_scale(float scale, float *out) {
    *out = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    return std::isfinite(*out);
}

constexpr size_t kStatusBytes = 256;
constexpr int32_t kMaxTreeHeads = 1024;
constexpr int kDefaultSms = 152;  // sizes asked for without a GPU
// Lengths that the kernels may round up to whole tiles within 32 bits.
constexpr int64_t kMaxLength = INT32_MAX - 4096;

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Tree attention: one range of key tiles for each SM.  Workspace: [status 256 B | records | part_ml | part_o].
struct TreePlan {
    int32_t ranges, part_rows;
    size_t off_ml, off_o, total;
};
TreePlan plan_tree(int32_t group, int32_t max_q_len, int sms) {
    TreePlan pl{};
    pl.ranges = sms;
    pl.part_rows = static_cast<int32_t>(std::min<int64_t>(128, static_cast<int64_t>(group) * max_q_len));
    const size_t rows = static_cast<size_t>(pl.ranges) * 2 * pl.part_rows;
    pl.off_ml = kStatusBytes + align_up(static_cast<size_t>(pl.ranges) * 16, 256);
    pl.off_o = pl.off_ml + align_up(rows * 8, 256);
    pl.total = pl.off_o + rows * kHeadDim * 4;
    return pl;
}

int check_tree_sizes(int32_t num_seqs, int32_t num_q_heads, int32_t max_q_len, const pkv_cache_desc *cache) {
    const bool fp8 = cache && cache->dtype == PKV_DTYPE_FP8_E4M3;
    if (int rc = check_pool(cache, fp8)) return rc;
    if (num_seqs < 1 || num_seqs > 65535 || max_q_len < 1 || max_q_len > PKV_MAX_TREE_NODES) return PKV_ERR_INVALID_ARG;
    if (num_q_heads < 1 || num_q_heads % cache->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (num_q_heads > kMaxTreeHeads) return PKV_ERR_UNSUPPORTED;
    // K/V tiles are addressed by the 32-bit index block * n_kv + head.
    if (static_cast<int64_t>(cache->num_blocks) * cache->num_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

std::once_flag g_tree_prepared[kMaxDevices];
cudaError_t g_tree_prep_err[kMaxDevices];

int finish(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

int rotary_write(void *q_out, const void *q, int64_t q_row, int64_t q_head, const void *key, int64_t k_row,
                 int64_t k_head, const void *value, int64_t v_row, int64_t v_head, void *k_cache, void *v_cache,
                 float *k_scale, float *v_scale, const int32_t *positions, const int32_t *slot_mapping,
                 const uint64_t *frequencies, int32_t num_tokens, int32_t num_q_heads, int32_t rotary_dim,
                 int32_t layout, float magnitude, const pkv_cache_desc *cache, bool fp8, void *stream) {
    if (int rc = check_pool(cache, fp8)) return rc;
    if (int rc = check_rotation(kHeadDim, rotary_dim, layout, magnitude)) return rc;
    if (num_tokens < 0 || num_q_heads < 0) return PKV_ERR_INVALID_ARG;
    if (cache->num_kv_heads > 65536 || num_q_heads > 65536) return PKV_ERR_UNSUPPORTED;
    if (!good_stride(k_row) || !good_stride(k_head) || !good_stride(v_row) || !good_stride(v_head))
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!good_stride(q_row) || !good_stride(q_head))) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!key || !value || !k_cache || !v_cache || !positions || !slot_mapping || !frequencies ||
        (num_q_heads > 0 && (!q || !q_out)))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(positions, 4) || !aligned(slot_mapping, 4) || !aligned(frequencies, 8) ||
        (num_q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16))))
        return PKV_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale || !aligned(k_scale, 16) || !aligned(v_scale, 16))) return PKV_ERR_INVALID_ARG;
    // in place: every row where it was
    if (num_q_heads > 0 && q == q_out &&
        ((num_q_heads > 1 && q_head != kHeadDim) || (num_tokens > 1 && q_row != static_cast<int64_t>(num_q_heads) * kHeadDim)))
        return PKV_ERR_INVALID_ARG;
    const int sms = current_sms();
    if (sms < 1) return PKV_ERR_CUDA;
    pkv::RotaryWriteParams p{};
    p.q_out = q_out;
    p.q = q;
    p.key = key;
    p.value = value;
    p.q_row = q_row;
    p.q_head = q_head;
    p.k_row = k_row;
    p.k_head = k_head;
    p.v_row = v_row;
    p.v_head = v_head;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.frequencies = frequencies;
    p.num_slots = static_cast<int64_t>(cache->num_blocks) * kBlockSize;
    p.num_tokens = num_tokens;
    p.n_q = num_q_heads;
    p.n_kv = cache->num_kv_heads;
    p.rotary_dim = rotary_dim;
    p.magnitude = magnitude;
    return finish(pkv::launch_rotary_write(p, layout == PKV_ROTARY_INTERLEAVED, fp8, sms,
                                           static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int rotary_frequencies(uint64_t *frequencies, float *magnitude, int32_t rotary_dim, double base,
                       const pkv_rotary_scaling *scaling) {
    if (!frequencies || !magnitude || rotary_dim < 2 || rotary_dim % 2 != 0) return PKV_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base)) return PKV_ERR_INVALID_ARG;
    const int kind = scaling ? scaling->kind : PKV_ROTARY_SCALING_NONE;
    if (kind < PKV_ROTARY_SCALING_NONE || kind > PKV_ROTARY_SCALING_BY_WAVELENGTH) return PKV_ERR_INVALID_ARG;
    const double pi = 3.14159265358979323846;
    double factor = 1.0, length = 0.0, low = 0.0, high = 0.0;
    if (kind != PKV_ROTARY_SCALING_NONE) {
        factor = scaling->factor;
        if (!(factor > 0.0) || !std::isfinite(factor)) return PKV_ERR_INVALID_ARG;
        // (a base of 1 or below would turn every pair alike, or faster than the first)
        if (kind == PKV_ROTARY_SCALING_NTK &&
            (rotary_dim == 2 || !(base * std::pow(factor, rotary_dim / (rotary_dim - 2.0)) > 1.0)))
            return PKV_ERR_INVALID_ARG;
    }
    if (kind == PKV_ROTARY_SCALING_BY_PARTS || kind == PKV_ROTARY_SCALING_BY_WAVELENGTH) {
        length = scaling->original_length;
        low = scaling->low;
        high = scaling->high;
        if (!(length >= 1.0) || !(low > 0.0) || !(high > low) || !std::isfinite(high)) return PKV_ERR_INVALID_ARG;
    }
    const double d = rotary_dim;
    if (kind == PKV_ROTARY_SCALING_NTK) base *= std::pow(factor, d / (d - 2.0));
    if (!std::isfinite(base)) return PKV_ERR_INVALID_ARG;
    // by parts: the pairs that turn `high` and `low` times over the original length
    const double at_high = d * std::log(length / (2.0 * pi * high)) / (2.0 * std::log(base));
    const double at_low = d * std::log(length / (2.0 * pi * low)) / (2.0 * std::log(base));
    const double from = std::max(0.0, std::floor(at_high)), to = std::min(d - 1.0, std::ceil(at_low));
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        double w = std::exp(-2.0 * i / d * std::log(base));  // radians a position
        if (kind == PKV_ROTARY_SCALING_LINEAR) {
            w /= factor;
        } else if (kind == PKV_ROTARY_SCALING_BY_PARTS) {
            const double ramp = std::min(1.0, std::max(0.0, (i - from) / std::max(to - from, 0.001)));
            w = w / factor * ramp + w * (1.0 - ramp);
        } else if (kind == PKV_ROTARY_SCALING_BY_WAVELENGTH) {
            const double keep = std::min(1.0, std::max(0.0, (length * w / (2.0 * pi) - low) / (high - low)));
            w = (1.0 - keep) * w / factor + keep * w;
        }
        // turns modulo 1 in units of 2^-64 (a factor below 1 may turn a pair more than once a position)
        double turns = w / (2.0 * pi);
        turns -= std::floor(turns);
        const double scaled = turns * 18446744073709551616.0;
        frequencies[i] = scaled >= 18446744073709551615.0 ? 0 : static_cast<uint64_t>(scaled + 0.5);
    }
    *magnitude = kind == PKV_ROTARY_SCALING_BY_PARTS && factor > 1.0 ? static_cast<float>(0.1 * std::log(factor) + 1.0)
                                                                     : 1.f;
    return PKV_OK;
}

int rotary_embedding(void *out, int64_t out_row_stride, int64_t out_head_stride, const void *x, int64_t x_row_stride,
                     int64_t x_head_stride, const int32_t *positions, const uint64_t *frequencies, int32_t num_tokens,
                     int32_t num_heads, int32_t head_dim, int32_t rotary_dim, int32_t layout, float magnitude,
                     void *stream) {
    if (num_tokens < 0 || num_heads < 1 || head_dim < 1) return PKV_ERR_INVALID_ARG;
    if (int rc = check_rotation(head_dim, rotary_dim, layout, magnitude)) return rc;
    if (head_dim > 1024 || num_heads > 65536) return PKV_ERR_UNSUPPORTED;
    if (!good_stride(out_row_stride) || !good_stride(out_head_stride) || !good_stride(x_row_stride) ||
        !good_stride(x_head_stride))
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!out || !x || !positions || !frequencies) return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(x, 16) || !aligned(positions, 4) || !aligned(frequencies, 8))
        return PKV_ERR_INVALID_ARG;
    // in place: every row where it was (other overlaps are the caller's error)
    if (out == x && (out_row_stride != x_row_stride || out_head_stride != x_head_stride)) return PKV_ERR_INVALID_ARG;
    const int sms = current_sms();
    if (sms < 1) return PKV_ERR_CUDA;
    pkv::RotaryParams p{};
    p.out = out;
    p.x = x;
    p.out_row = out_row_stride;
    p.out_head = out_head_stride;
    p.x_row = x_row_stride;
    p.x_head = x_head_stride;
    p.positions = positions;
    p.frequencies = frequencies;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.head_dim = head_dim;
    p.rotary_dim = rotary_dim;
    p.magnitude = magnitude;
    return finish(pkv::launch_rotary(p, layout == PKV_ROTARY_INTERLEAVED, sms, static_cast<cudaStream_t>(stream)));
}

int rotary_reshape_and_cache(void *q_out, const void *q, int64_t q_row_stride, int64_t q_head_stride, const void *key,
                             int64_t k_row_stride, int64_t k_head_stride, const void *value, int64_t v_row_stride,
                             int64_t v_head_stride, void *k_cache, void *v_cache, const int32_t *positions,
                             const int32_t *slot_mapping, const uint64_t *frequencies, int32_t num_tokens,
                             int32_t num_q_heads, int32_t rotary_dim, int32_t layout, float magnitude,
                             const pkv_cache_desc *cache, void *stream) {
    return rotary_write(q_out, q, q_row_stride, q_head_stride, key, k_row_stride, k_head_stride, value, v_row_stride,
                        v_head_stride, k_cache, v_cache, nullptr, nullptr, positions, slot_mapping, frequencies,
                        num_tokens, num_q_heads, rotary_dim, layout, magnitude, cache, false, stream);
}

int rotary_reshape_and_cache_fp8(void *q_out, const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                 const void *key, int64_t k_row_stride, int64_t k_head_stride, const void *value,
                                 int64_t v_row_stride, int64_t v_head_stride, void *k_cache, void *v_cache,
                                 float *k_scale, float *v_scale, const int32_t *positions, const int32_t *slot_mapping,
                                 const uint64_t *frequencies, int32_t num_tokens, int32_t num_q_heads,
                                 int32_t rotary_dim, int32_t layout, float magnitude, const pkv_cache_desc *cache,
                                 void *stream) {
    return rotary_write(q_out, q, q_row_stride, q_head_stride, key, k_row_stride, k_head_stride, value, v_row_stride,
                        v_head_stride, k_cache, v_cache, k_scale, v_scale, positions, slot_mapping, frequencies,
                        num_tokens, num_q_heads, rotary_dim, layout, magnitude, cache, true, stream);
}

size_t paged_attention_tree_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t max_q_len,
                                           const pkv_cache_desc *cache) {
    if (check_tree_sizes(num_seqs, num_q_heads, max_q_len, cache) != PKV_OK) return 0;
    const int sms = current_sms();
    return plan_tree(num_q_heads / cache->num_kv_heads, max_q_len, sms > 0 ? sms : kDefaultSms).total;
}

int paged_attention_tree(void *out, int32_t out_dtype, const void *q, const uint64_t *tree_mask, const int32_t *cu_q_lens,
                         int32_t max_q_len, int32_t total_q_rows, const void *k_cache, const void *v_cache,
                         const float *k_scale, const float *v_scale, const int32_t *block_tables,
                         const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq,
                         float scale, const pkv_cache_desc *cache, void *workspace, size_t workspace_bytes, void *stream) {
    if (int rc = check_tree_sizes(num_seqs, num_q_heads, max_q_len, cache)) return rc;
    const bool fp8 = cache->dtype == PKV_DTYPE_FP8_E4M3;
    if (out_dtype != PKV_DTYPE_FLOAT32 && out_dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    if (total_q_rows < 0 || max_blocks_per_seq < 1 || static_cast<int64_t>(max_blocks_per_seq) * kBlockSize > kMaxLength)
        return PKV_ERR_INVALID_ARG;
    pkv::TreeParams p{};
    if (!log2_scale(scale, &p.scale_log2)) return PKV_ERR_INVALID_ARG;
    if (total_q_rows == 0) return PKV_OK;
    if (!out || !q || !tree_mask || !cu_q_lens || !k_cache || !v_cache || !block_tables || !context_lens)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(tree_mask, 8) || !aligned(cu_q_lens, 4) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    if (fp8 ? (!k_scale || !v_scale || !aligned(k_scale, 16) || !aligned(v_scale, 16)) : (k_scale || v_scale))
        return PKV_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256)) return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < paged_attention_tree_workspace_size(num_seqs, num_q_heads, max_q_len, cache))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    const int sms = current_sms(), dev = current_device();
    if (sms < 1) return PKV_ERR_CUDA;
    std::call_once(g_tree_prepared[dev], [&] { g_tree_prep_err[dev] = pkv::tree_prepare_device(); });
    if (g_tree_prep_err[dev] != cudaSuccess) return PKV_ERR_CUDA;
    const int32_t n_kv = cache->num_kv_heads;
    const int32_t group = num_q_heads / n_kv, whole_nodes = 128 % group == 0 ? 128 / group : 0;
    CUtensorMap kmap, vmap, qmap{};
    if (!(fp8 ? pkv::encode_pool_map_fp8(&kmap, k_cache, cache->num_blocks, n_kv)
              : pkv::encode_pool_tile_map(&kmap, k_cache, cache->num_blocks, n_kv)) ||
        !(fp8 ? pkv::encode_pool_map_fp8(&vmap, v_cache, cache->num_blocks, n_kv)
              : pkv::encode_pool_tile_map(&vmap, v_cache, cache->num_blocks, n_kv)) ||
        (whole_nodes && !pkv::encode_query_group_map(&qmap, q, total_q_rows, num_q_heads, group)))
        return PKV_ERR_CUDA;
    const TreePlan pl = plan_tree(group, max_q_len, sms);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.q = q;
    p.out = out;
    p.mask = tree_mask;
    p.cu_q_lens = cu_q_lens;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.status = reinterpret_cast<uint32_t *>(ws);
    p.num_seqs = num_seqs;
    p.n_q = num_q_heads;
    p.n_kv = n_kv;
    p.group = group;
    p.whole_nodes = whole_nodes;
    p.group_magic = p.group > 1 ? static_cast<uint32_t>(((uint64_t{1} << 32) + p.group - 1) / p.group) : 0;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = cache->num_blocks;
    p.total_rows = total_q_rows;
    p.max_q_len = max_q_len;
    p.out_bf16 = out_dtype == PKV_DTYPE_BF16;
    p.ranges = pl.ranges;
    p.part_rows = pl.part_rows;
    p.record = reinterpret_cast<int4 *>(ws + kStatusBytes);
    p.part_ml = reinterpret_cast<float2 *>(ws + pl.off_ml);
    p.part_o = reinterpret_cast<float *>(ws + pl.off_o);
    return finish(pkv::launch_tree_attention(kmap, vmap, qmap, p, fp8, static_cast<cudaStream_t>(stream)));
}

int speculative_verify(int32_t *tokens_out, int32_t *path, int32_t *counts, const float *target_probs,
                       int64_t target_row_stride, const float *draft_probs, int64_t draft_row_stride,
                       const int32_t *tokens, const int32_t *parents, const float *uniforms, const int32_t *cu_q_lens,
                       int32_t num_seqs, int32_t max_q_len, int32_t total_q_rows, int32_t vocab_size, uint32_t *status,
                       void *stream) {
    if (num_seqs < 1 || num_seqs > 65535 || max_q_len < 1 || max_q_len > pkv::kMaxTreeNodes || total_q_rows < 0 ||
        vocab_size < 1)
        return PKV_ERR_INVALID_ARG;
    if (vocab_size > (1 << 24)) return PKV_ERR_UNSUPPORTED;
    if (draft_probs && parents) return PKV_ERR_UNSUPPORTED;  // the drafter's probabilities: chains only
    if (target_row_stride < vocab_size || target_row_stride >= int64_t{1} << 38 ||
        (draft_probs && (draft_row_stride < vocab_size || draft_row_stride >= int64_t{1} << 38)))
        return PKV_ERR_INVALID_ARG;
    if (!tokens_out || !path || !counts || !cu_q_lens) return PKV_ERR_INVALID_ARG;
    if (total_q_rows > 0 && (!target_probs || !tokens || !uniforms)) return PKV_ERR_INVALID_ARG;
    if (!aligned(tokens_out, 4) || !aligned(path, 4) || !aligned(counts, 4) || !aligned(cu_q_lens, 4) ||
        !aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(tokens, 4) || !aligned(parents, 4) ||
        !aligned(uniforms, 4) || !aligned(status, 4))
        return PKV_ERR_INVALID_ARG;
    const int sms = current_sms();
    if (sms < 1) return PKV_ERR_CUDA;
    pkv::SpecVerifyParams p{};
    p.tokens_out = tokens_out;
    p.path = path;
    p.counts = counts;
    p.target = target_probs;
    p.draft = draft_probs;
    p.target_row = target_row_stride;
    p.draft_row = draft_row_stride;
    p.tokens = tokens;
    p.parents = parents;
    p.cu_q_lens = cu_q_lens;
    p.uniforms = uniforms;
    p.status = status;
    p.num_seqs = num_seqs;
    p.max_q_len = max_q_len;
    p.total_rows = total_q_rows;
    p.vocab = vocab_size;
    // CTAs a sequence: one for every 4096 entries, up to a portable cluster of 8, as long as all run at once, two an
    // SM (with the drafter's rows: 64 of 128000 take 19.5 us in 4 CTAs each, 26 in 2 or 8; 160 of 128000 46 in 1, 48 in 2, 56 in 8;
    // 256 of 128000 55 in 1, 57 in 2, 85 in 8; 256 of 32000 20 in 1, 28 in 2; 16 of 50257 10.2 in 8, 11.0 in 4, 15.2 in 1).
    int cluster = 1;
    while (cluster < pkv::kVerifyMaxCluster && static_cast<int64_t>(cluster) * 4096 < vocab_size &&
           static_cast<int64_t>(cluster) * num_seqs <= sms)
        cluster *= 2;
    const int32_t warps = cluster * pkv::kVerifyWarps;
    p.segment = (vocab_size + warps * 128 - 1) / (warps * 128) * 128;
    return finish(pkv::launch_speculative_verify(p, cluster, static_cast<cudaStream_t>(stream)));
}

int kv_compact_path(void *k_cache, void *v_cache, float *k_scale, float *v_scale, const int32_t *block_tables,
                    const int32_t *context_lens, const int32_t *cu_q_lens, const int32_t *path, const int32_t *counts,
                    int32_t num_seqs, int32_t max_blocks_per_seq, int32_t path_len, const pkv_cache_desc *cache,
                    uint32_t *status, void *stream) {
    const bool fp8 = cache && cache->dtype == PKV_DTYPE_FP8_E4M3;
    if (int rc = check_pool(cache, fp8)) return rc;
    if (num_seqs < 1 || max_blocks_per_seq < 1 || path_len < 1 || path_len > pkv::kMaxTreeNodes)
        return PKV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_blocks_per_seq) * kBlockSize > INT32_MAX) return PKV_ERR_INVALID_ARG;
    if (cache->num_kv_heads > 65536) return PKV_ERR_UNSUPPORTED;
    if (!k_cache || !v_cache || !block_tables || !context_lens || !cu_q_lens || !path || !counts)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(cu_q_lens, 4) || !aligned(path, 4) || !aligned(counts, 4) || !aligned(status, 4))
        return PKV_ERR_INVALID_ARG;
    if (fp8 ? (!k_scale || !v_scale || !aligned(k_scale, 16) || !aligned(v_scale, 16)) : (k_scale || v_scale))
        return PKV_ERR_INVALID_ARG;
    pkv::CompactParams p{};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.cu_q_lens = cu_q_lens;
    p.path = path;
    p.counts = counts;
    p.status = status;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = cache->num_blocks;
    p.n_kv = cache->num_kv_heads;
    p.path_len = path_len;
    return finish(pkv::launch_kv_compact_path(p, fp8, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
