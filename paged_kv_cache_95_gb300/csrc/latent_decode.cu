// latent_decode.cu -- absorbed latent attention over the paged pool (decode and verify).
//
//     s_j = scale (<q_latent, c_j> + <q_rope, r_j>),  out = sum_j softmax(s)_j c_j
//
// One warp per (row, head): the query lies in registers (16 latent values and 2
// rotated ones a lane), the keys are walked one by one with a running maximum and
// sum in fp32 (log2 domain).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "latent.h"
#include "ptx.cuh"

namespace pkv {

namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool FP8>
__global__ void __launch_bounds__(128) latent_decode_kernel(const LatentDecodeParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.q_per_seq;
    if (unit >= rows * p.heads) return;
    const int64_t row = unit / p.heads;
    const int h = static_cast<int>(unit - row * p.heads);
    const int b = static_cast<int>(row / p.q_per_seq), i = static_cast<int>(row - static_cast<int64_t>(b) * p.q_per_seq);
    const int cap = p.max_blocks * kBlockSize;
    int ctx = __ldg(p.context_lens + b);
    uint32_t bad = ctx < 1 || ctx > cap ? kStatusBadContextLen : 0u;
    if (ctx >= 1 && ctx < p.q_per_seq) bad |= kStatusBadQLen;
    ctx = min(ctx, cap);
    const int keys = ctx < 1 || ctx < p.q_per_seq ? 0 : ctx - p.q_per_seq + 1 + i;

    float q[18], o[16] = {};
    {
        const uint4 *ql = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q_latent) + row * p.ql_row +
                                                          h * p.ql_head);
        const uint4 a = __ldg(ql + 2 * lane), c = __ldg(ql + 2 * lane + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) q[2 * k] = bf16_lo(w[k]), q[2 * k + 1] = bf16_hi(w[k]);
        const uint32_t r = __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.q_rope) +
                                                                    row * p.qr_row + h * p.qr_head) + lane);
        q[16] = bf16_lo(r), q[17] = bf16_hi(r);
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < keys; ++j) {
        const int blk = __ldg(p.block_tables + static_cast<size_t>(b) * p.max_blocks + j / kBlockSize);
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
            bad |= kStatusBadBlockId;
            continue;
        }
        const size_t slot = static_cast<size_t>(blk) * kBlockSize + j % kBlockSize;
        float c[16];
        uint32_t rw;
        if (FP8) {
            const uint4 a = __ldg(static_cast<const uint4 *>(p.cache) + slot * 32 + lane);
            const float sc = __ldg(p.cache_scale + slot);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = unpack_f16x2(e4m3x2_to_f16x2(w[k])), g = unpack_f16x2(e4m3x2_to_f16x2(w[k] >> 16));
                c[4 * k] = f.x * sc, c[4 * k + 1] = f.y * sc, c[4 * k + 2] = g.x * sc, c[4 * k + 3] = g.y * sc;
            }
            rw = __ldg(static_cast<const uint32_t *>(p.rope_cache) + slot * 32 + lane);
        } else {
            const uint4 *src = static_cast<const uint4 *>(p.cache) + slot * 72;
            const uint4 a = __ldg(src + 2 * lane), d = __ldg(src + 2 * lane + 1);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) c[2 * k] = bf16_lo(w[k]), c[2 * k + 1] = bf16_hi(w[k]);
            rw = __ldg(reinterpret_cast<const uint32_t *>(src + 64) + lane);
        }
        float s = q[16] * bf16_lo(rw) + q[17] * bf16_hi(rw);
#pragma unroll
        for (int k = 0; k < 16; ++k) s += q[k] * c[k];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s);
        const float alpha = exp2f(m - mn), e = exp2f(s - mn);
        l = l * alpha + e;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = o[k] * alpha + e * c[k];
        m = mn;
    }
    if (bad && lane == 0 && p.status) atomicOr(p.status, bad);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const size_t at = static_cast<size_t>(unit) * kLatentDim + 16 * lane;
    if (p.out_bf16) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(o[2 * k] * inv, o[2 * k + 1] * inv);
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            dst[k] = make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv, o[4 * k + 3] * inv);
    }
}

}  // namespace

cudaError_t launch_latent_decode(const LatentDecodeParams &p, bool fp8, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(p.num_seqs) * p.q_per_seq * p.heads;
    const dim3 grid(static_cast<unsigned>((units + 3) / 4));
    return launch_pdl(fp8 ? latent_decode_kernel<true> : latent_decode_kernel<false>, grid, dim3(128), 0, stream, p);
}

}  // namespace pkv
