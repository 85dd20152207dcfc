// latent_prefill.cu -- expanded latent attention of a causal prefill chunk.
//
//     s_j = scale (<q_nope, k_nope_j> + <q_rope, r_j>), j <= k_len - q_len + i,
//     out_i = sum_j softmax(s)_j v_j
//
// One warp per (row, head): 4 + 2 query values and 4 output values a lane, the keys
// walked one by one with a running maximum and sum in fp32 (log2 domain).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "latent.h"
#include "ptx.cuh"

namespace pkv {

namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__global__ void __launch_bounds__(128) latent_prefill_kernel(const LatentPrefillParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
    const int q0 = __ldg(p.cu_q_lens + b), q_len = __ldg(p.cu_q_lens + b + 1) - q0;
    const int k0 = __ldg(p.cu_k_lens + b), k_len = __ldg(p.cu_k_lens + b + 1) - k0;
    bool ok = q_len >= 0 && q_len <= k_len && q_len <= p.max_q_len && q0 >= 0 && k0 >= 0 &&
              static_cast<int64_t>(q0) + q_len <= p.total_q && static_cast<int64_t>(k0) + k_len <= p.total_k;
    if (!ok && i == 0 && h == 0 && lane == 0 && p.status) atomicOr(p.status, kStatusBadQLen);
    if (i >= q_len || q0 < 0 || static_cast<int64_t>(q0) + i >= p.total_q) return;
    const size_t row = static_cast<size_t>(q0) + i;
    float q[6], o[4] = {}, m = -INFINITY, l = 0.f;
    const uint16_t *qp = static_cast<const uint16_t *>(p.q) + row * p.q_row + h * p.q_head;
    const uint2 qn = __ldg(reinterpret_cast<const uint2 *>(qp) + lane);
    const uint32_t qr = __ldg(reinterpret_cast<const uint32_t *>(qp + kNopeDim) + lane);
    q[0] = bf16_lo(qn.x), q[1] = bf16_hi(qn.x), q[2] = bf16_lo(qn.y), q[3] = bf16_hi(qn.y);
    q[4] = bf16_lo(qr), q[5] = bf16_hi(qr);
    const int keys = ok ? k_len - q_len + 1 + i : 0;
    for (int j = 0; j < keys; ++j) {
        const size_t kr = static_cast<size_t>(k0) + j;
        const uint2 kn = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.k_nope) + kr * p.k_row +
                                                               h * p.k_head) + lane);
        const uint32_t r = __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.k_rope) + kr * p.r_row) +
                                 lane);
        const uint2 vv = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.v) + kr * p.k_row +
                                                               h * p.k_head) + lane);
        float s = q[0] * bf16_lo(kn.x) + q[1] * bf16_hi(kn.x) + q[2] * bf16_lo(kn.y) + q[3] * bf16_hi(kn.y) +
                  q[4] * bf16_lo(r) + q[5] * bf16_hi(r);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s);
        const float alpha = exp2f(m - mn), e = exp2f(s - mn);
        l = l * alpha + e;
        o[0] = o[0] * alpha + e * bf16_lo(vv.x), o[1] = o[1] * alpha + e * bf16_hi(vv.x);
        o[2] = o[2] * alpha + e * bf16_lo(vv.y), o[3] = o[3] * alpha + e * bf16_hi(vv.y);
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const size_t at = (row * p.heads + h) * kExpandedV + 4 * lane;
    if (p.out_bf16)
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
            make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
            make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillParams &p, cudaStream_t stream) {
    const dim3 grid((p.max_q_len + 3) / 4, p.heads, p.num_seqs);
    return launch_pdl(latent_prefill_kernel, grid, dim3(128), 0, stream, p);
}

}  // namespace pkv
