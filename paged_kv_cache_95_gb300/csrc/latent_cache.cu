// latent_cache.cu -- the latent pool's write (slot mapping, optional E4M3
// quantisation) and its read-back in sequence order.
//
// A cached token is one row [c (512) | r (64)] that every head shares, so both
// kernels are plain row moves, HBM bound: 1152 bytes a token each way for a bf16
// pool, 1152 against 512 + 128 + 4 for an FP8 pool.
#include <cuda_runtime.h>

#include "latent.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kVecRow = kLatentRow * 2 / 16;     // 72 vectors of 8 bf16 in a row
constexpr int kVecLatent = kLatentDim * 2 / 16;  // 64 of them the latent
constexpr int kVecRope = kRopeDim * 2 / 16;      // 8 the rotated key

// One thread moves one 16-byte vector of a row: reads and writes are contiguous
// runs of 1024 and 128 bytes a token.
__global__ void __launch_bounds__(256) latent_write_kernel(const LatentWriteParams p) {
    griddep_launch_dependents();
    griddep_wait();  // the previous kernel on the stream may still read the pool
    const int64_t total = static_cast<int64_t>(p.num_tokens) * kVecRow;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
        const int64_t t = i / kVecRow;
        const int c = static_cast<int>(i - t * kVecRow);
        const int64_t slot = __ldg(p.slot_mapping + t);
        if (slot < 0 || slot >= p.num_slots) continue;  // padding token or out-of-range slot: no write
        const uint16_t *src = c < kVecLatent
                                  ? static_cast<const uint16_t *>(p.latent) + t * p.latent_stride + c * 8
                                  : static_cast<const uint16_t *>(p.rope) + t * p.rope_stride + (c - kVecLatent) * 8;
        static_cast<uint4 *>(p.cache)[slot * kVecRow + c] = __ldg(reinterpret_cast<const uint4 *>(src));
    }
}

// One warp per token: 16 latent values a lane (two 16-byte loads, one 16-byte
// store of codes), lanes 0..7 move the rotated key.
__global__ void __launch_bounds__(256) latent_write_fp8_kernel(const LatentWriteParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t stride = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    for (int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; t < p.num_tokens; t += stride) {
        const int64_t slot = __ldg(p.slot_mapping + t);
        if (slot < 0 || slot >= p.num_slots) continue;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.latent) + t * p.latent_stride);
        const uint4 x0 = __ldg(src + 2 * lane), x1 = __ldg(src + 2 * lane + 1);
        uint4 r = make_uint4(0u, 0u, 0u, 0u);
        if (lane < kVecRope)
            r = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.rope) + t * p.rope_stride) + lane);
        const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        float v[16];
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            a = fmaxf(a, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        a = fmaxf(a, 0x1p-100f);
        const float inv = __fdiv_rn(448.f, a);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = f32x2_to_e4m3x2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv)) |
                   (f32x2_to_e4m3x2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv)) << 16);
        static_cast<uint4 *>(p.cache)[slot * 32 + lane] = make_uint4(c[0], c[1], c[2], c[3]);
        if (lane < kVecRope) static_cast<uint4 *>(p.rope_cache)[slot * kVecRope + lane] = r;
        if (lane == 0) p.cache_scale[slot] = __fdiv_rn(a, 448.f);
    }
}

// The slot that holds output row r0 + lane, for lanes 0..3 (-1: none, the row becomes zeros; -2: past the
// last sequence, the row is left as it was).  The warp finds r0's sequence 32 lengths at a time: one round trip
// to L2 for up to 32 sequences, where a bisection is one a halving.
__device__ __forceinline__ int64_t gather_slot(const LatentGatherParams &p, int r0, int lane) {
    const int end = __ldg(p.cu_lens + p.num_seqs);
    int lo = 0;  // cu_lens[lo] <= r0; one of the n sequences from lo on has it
    for (int n = p.num_seqs; n > 1;) {
        const int step = (n + 31) / 32;
        const int64_t next = lo + static_cast<int64_t>(lane + 1) * step;
        const int ahead = __popc(__ballot_sync(0xffffffffu, next < lo + n && __ldg(p.cu_lens + next) <= r0));
        lo += ahead * step;
        n = min(step, n - ahead * step);
    }
    const int r = r0 + lane;
    if (lane >= 4 || r >= p.total_rows || r >= end) return -2;
    while (lo + 1 < p.num_seqs && __ldg(p.cu_lens + lo + 1) <= r) ++lo;
    const int pos = r - __ldg(p.cu_lens + lo);
    if (pos < 0 || pos >= static_cast<int64_t>(p.max_blocks) * kBlockSize) {
        if (p.status) atomicOr(p.status, kStatusBadContextLen);
        return -1;
    }
    const int blk = __ldg(p.block_tables + static_cast<size_t>(lo) * p.max_blocks + pos / kBlockSize);
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
        if (p.status) atomicOr(p.status, kStatusBadBlockId);
        return -1;
    }
    return static_cast<int64_t>(blk) * kBlockSize + pos % kBlockSize;
}

// A warp moves four rows: lanes 0..3 find their slots, then every lane has nine
// 16-byte loads in flight (35K rows 14.5 us, 5.55 TB/s; loads and stores that are not
// streaming 15.2, a bisection for the sequence 14.8).
__global__ void __launch_bounds__(256) latent_gather_kernel(const LatentGatherParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int r0 = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 4;
    if (r0 >= p.total_rows) return;
    const int64_t mine = gather_slot(p, r0, lane);
    const uint4 *pool = static_cast<const uint4 *>(p.cache);
    uint4 *out = static_cast<uint4 *>(p.out) + static_cast<size_t>(r0) * kVecRow;
    uint4 v[9];
#pragma unroll
    for (int k = 0; k < 9; ++k) {
        const int i = k * 32 + lane, row = i / kVecRow;
        const int64_t slot = __shfl_sync(0xffffffffu, mine, row);
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (slot >= 0) v[k] = __ldcs(pool + slot * kVecRow + (i - row * kVecRow));
    }
#pragma unroll
    for (int k = 0; k < 9; ++k) {
        const int i = k * 32 + lane, row = i / kVecRow;
        if (__shfl_sync(0xffffffffu, mine, row) != -2) __stcs(out + i, v[k]);
    }
}

__device__ __forceinline__ uint32_t dequant_pair(uint32_t two_codes, float scale) {
    const float2 f = unpack_f16x2(e4m3x2_to_f16x2(two_codes));
    return pack_bf16x2(f.x * scale, f.y * scale);
}

// FP8 pool: a lane takes 16 codes of each of the warp's four rows (one 16-byte load,
// two 16-byte stores a row) and one vector of the four rotated keys.
__global__ void __launch_bounds__(256) latent_gather_fp8_kernel(const LatentGatherParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int r0 = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 4;
    if (r0 >= p.total_rows) return;
    const int64_t mine = gather_slot(p, r0, lane);
    const float my_scale = mine >= 0 ? __ldg(p.cache_scale + mine) : 0.f;
    uint4 *out = static_cast<uint4 *>(p.out) + static_cast<size_t>(r0) * kVecRow;
    uint4 c[4], rope = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t slot = __shfl_sync(0xffffffffu, mine, k);
        c[k] = make_uint4(0u, 0u, 0u, 0u);
        if (slot >= 0) c[k] = __ldg(static_cast<const uint4 *>(p.cache) + slot * 32 + lane);
    }
    const int64_t rope_slot = __shfl_sync(0xffffffffu, mine, lane / kVecRope);
    if (rope_slot >= 0)
        rope = __ldg(static_cast<const uint4 *>(p.rope_cache) + rope_slot * kVecRope + lane % kVecRope);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t slot = __shfl_sync(0xffffffffu, mine, k);
        const float s = __shfl_sync(0xffffffffu, my_scale, k);
        if (slot == -2) continue;
        uint4 *o = out + k * kVecRow + 2 * lane;
        o[0] = make_uint4(dequant_pair(c[k].x, s), dequant_pair(c[k].x >> 16, s), dequant_pair(c[k].y, s),
                          dequant_pair(c[k].y >> 16, s));
        o[1] = make_uint4(dequant_pair(c[k].z, s), dequant_pair(c[k].z >> 16, s), dequant_pair(c[k].w, s),
                          dequant_pair(c[k].w >> 16, s));
    }
    if (rope_slot != -2) out[(lane / kVecRope) * kVecRow + kVecLatent + lane % kVecRope] = rope;
}

}  // namespace

cudaError_t launch_latent_write(const LatentWriteParams &p, bool fp8, int sm_count, cudaStream_t stream) {
    if (p.num_tokens == 0) return cudaSuccess;
    const int threads = 256;
    const int64_t work = static_cast<int64_t>(p.num_tokens) * (fp8 ? 32 : kVecRow);
    int64_t blocks = (work + threads - 1) / threads;
    const int64_t cap = static_cast<int64_t>(sm_count > 0 ? sm_count : 1) * 8;
    if (blocks > cap) blocks = cap;
    return launch_pdl(fp8 ? latent_write_fp8_kernel : latent_write_kernel, dim3(static_cast<unsigned>(blocks)),
                      dim3(threads), 0, stream, p);
}

cudaError_t launch_latent_gather(const LatentGatherParams &p, bool fp8, cudaStream_t stream) {
    if (p.total_rows == 0) return cudaSuccess;
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(p.total_rows) + 31) / 32);  // 8 warps x 4 rows
    return launch_pdl(fp8 ? latent_gather_fp8_kernel : latent_gather_kernel, dim3(blocks), dim3(256), 0, stream, p);
}

}  // namespace pkv
