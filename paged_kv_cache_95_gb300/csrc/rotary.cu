// rotary.cu -- rotary positions: alone, and on the way into the paged cache.
//
// Pair i of a head's first rotary_dim values turns by the angle position * w_i:
//     (a, b) -> m (a cos - b sin, b cos + a sin)
// with the pairs (i, i + rotary_dim / 2) or (2 i, 2 i + 1) and one magnitude m.
//
// Angles: w_i comes as a fraction of a turn in units of 2^-64, so the product with the
// position in 64-bit whole numbers is the angle modulo one turn, exactly, however far the
// position (a position below zero turns back).  It is rounded once, to fp32 half turns
// (relative 2^-24), and goes to sincospif.
//
// One thread takes 8 pairs of a token (two 16-byte vectors of a head's row), computes their
// sines and cosines once and turns that part of many heads' rows: with 8 heads a thread
// the sines and cosines are a third of the instructions, and those a quarter of what the
// memory time leaves room for.  HBM bound: every row is read once and written once.
// 8192 tokens x 40 heads: 28.2 us, 5.95 TB/s (88% of a plain copy); 16384 tokens x 48 rows into an FP8 pool:
// 63.3 us, 5.85 TB/s, into a bf16 pool 59.4 us (the copy rate).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ptx.cuh"
#include "speculative.h"

namespace pkv {

namespace {

// (Blocks of 256 threads leave SMs waiting for their last ones: 16384 tokens of 32 + 8 + 8 heads into an FP8 pool take 78 us,
// 64 in blocks of 64, of which HBM needs 54; into a bf16 pool either takes the 59 us of HBM.)
constexpr int kRotaryThreads = 64;
constexpr int kBatch = 4;  // rows that a thread has on their way at once

struct Turn {
    float c[8], s[8];
};

template <bool INTERLEAVED>
__device__ __forceinline__ Turn load_turn(const uint64_t *frequencies, int unit, int rotary_dim, int32_t position,
                                          float magnitude) {
    Turn t;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pair = !INTERLEAVED ? 8 * unit + i : i < 4 ? 4 * unit + i : rotary_dim / 4 + 4 * unit + i - 4;
        const uint64_t turns = __ldg(reinterpret_cast<const unsigned long long *>(frequencies) + pair) *
                               static_cast<uint64_t>(static_cast<int64_t>(position));
        const float half_turns = __ll2float_rn(static_cast<long long>(turns)) * 0x1p-63f;
        float s, c;
        sincospif(half_turns, &s, &c);
        t.s[i] = s * magnitude;
        t.c[i] = c * magnitude;
    }
    return t;
}

// The 16 values of a unit as fp32: v[0..7] the first vector, v[8..15] the second.
__device__ __forceinline__ void widen(const uint4 &a, const uint4 &b, float (&v)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void narrow(const float (&v)[16], uint4 &a, uint4 &b) {
    a = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    b = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                   pack_bf16x2(v[14], v[15]));
}

template <bool INTERLEAVED>
__device__ __forceinline__ void turn_pairs(float (&v)[16], const Turn &t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &x = v[INTERLEAVED ? 2 * i : i], &y = v[INTERLEAVED ? 2 * i + 1 : 8 + i];
        const float a = x, b = y;
        x = a * t.c[i] - b * t.s[i];
        y = b * t.c[i] + a * t.s[i];
    }
}

// Where a unit's two vectors of 8 values lie in a head's row: one in each half of the rotated values (pairs (i, i +
// rotary_dim / 2) want it so; interleaved pairs lie within a vector), or of the values behind them.  (Neighbouring lanes'
// vectors are neighbours then.  As one piece of 32 bytes a unit 8192 tokens x 40 heads took 30.7 us interleaved, 26.6 so.)
__device__ __forceinline__ int2 unit_places(int unit, int rotary_dim, int head_dim) {
    const int at = 8 * unit;
    if (2 * at < rotary_dim) return make_int2(at, rotary_dim / 2 + at);
    return make_int2(rotary_dim / 2 + at, head_dim / 2 + at);
}

// Thread (token, s, unit) turns the unit of heads s, s + split, ...
template <bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryParams p, int split) {
    griddep_launch_dependents();
    griddep_wait();
    const int units = p.head_dim / kRotaryUnit;
    const int64_t index = static_cast<int64_t>(blockIdx.x) * kRotaryThreads + threadIdx.x;
    const int64_t ts = index / units;
    const int unit = static_cast<int>(index - ts * units);
    const int64_t token = ts / split;
    const int s = static_cast<int>(ts - token * split);
    if (token >= p.num_tokens) return;
    const bool turned = kRotaryUnit * unit < p.rotary_dim;
    const int2 at = unit_places(unit, p.rotary_dim, p.head_dim);
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x) + token * p.x_row;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + token * p.out_row;
    Turn t;
    if (turned) t = load_turn<INTERLEAVED>(p.frequencies, unit, p.rotary_dim, __ldg(p.positions + token), p.magnitude);
    else if (x == out && p.x_head == p.out_head) return;  // in place: nothing to copy
    for (int h0 = s; h0 < p.num_heads; h0 += kBatch * split) {
        uint4 a[kBatch], b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = h0 + i * split;
            if (h < p.num_heads) {
                a[i] = *reinterpret_cast<const uint4 *>(x + h * p.x_head + at.x);
                b[i] = *reinterpret_cast<const uint4 *>(x + h * p.x_head + at.y);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = h0 + i * split;
            if (h >= p.num_heads) break;
            if (turned) {
                float v[16];
                widen(a[i], b[i], v);
                turn_pairs<INTERLEAVED>(v, t);
                narrow(v, a[i], b[i]);
            }
            *reinterpret_cast<uint4 *>(out + h * p.out_head + at.x) = a[i];
            *reinterpret_cast<uint4 *>(out + h * p.out_head + at.y) = b[i];
        }
    }
}

// The append: a token's rows are its query heads, key heads and value heads in this order;
// thread (token, s, unit of 8 a head) takes the unit of rows s, s + split, ...  A row's 8 units
// are 8 neighbouring lanes, which share the maximum of an E4M3 row by shuffles.
// E4M3: as kv_reshape_and_cache_fp8 has it, from the turned values in fp32 (one rounding, to the code).  (Ten blocks an SM, 96
// registers: with 99, nine blocks, 16384 tokens take 69.6 us for 63.5.)
template <bool INTERLEAVED, bool FP8>
__global__ void __launch_bounds__(kRotaryThreads, FP8 ? 10 : 1) rotary_write_kernel(const RotaryWriteParams p, int split) {
    constexpr int kUnits = kHeadDim / kRotaryUnit;
    static_assert(kUnits == 8, "a row's units are 8 lanes");
    griddep_launch_dependents();
    griddep_wait();  // the kernel before may still read the pool
    const int64_t index = static_cast<int64_t>(blockIdx.x) * kRotaryThreads + threadIdx.x;
    const int unit = static_cast<int>(index) & (kUnits - 1);
    const int64_t ts = index / kUnits;
    const int64_t token = ts / split;
    const int s = static_cast<int>(ts - token * split);
    if (token >= p.num_tokens) return;  // (whole groups of 8 lanes)
    const uint32_t group = 0xffu << (threadIdx.x & 24);
    const bool turned = kRotaryUnit * unit < p.rotary_dim;
    const int2 at = unit_places(unit, p.rotary_dim, kHeadDim);
    const int64_t slot = __ldg(p.slot_mapping + token);
    const bool kept = slot >= 0 && slot < p.num_slots;  // else padding, or no slot of the pool: not written
    const int64_t block = slot / kBlockSize, place = slot - block * kBlockSize;
    const int rows = p.n_q + 2 * p.n_kv;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + token * p.q_row;
    const __nv_bfloat16 *key = static_cast<const __nv_bfloat16 *>(p.key) + token * p.k_row;
    const __nv_bfloat16 *value = static_cast<const __nv_bfloat16 *>(p.value) + token * p.v_row;
    __nv_bfloat16 *q_out = static_cast<__nv_bfloat16 *>(p.q_out) + token * p.n_q * kHeadDim;
    const int end = kept ? rows : p.n_q;

    uint4 a[kBatch], b[kBatch];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * split;
            if (r >= end) break;
            const __nv_bfloat16 *src = r < p.n_q            ? q + r * p.q_head
                                       : r < p.n_q + p.n_kv ? key + (r - p.n_q) * p.k_head
                                                            : value + (r - p.n_q - p.n_kv) * p.v_head;
            a[i] = *reinterpret_cast<const uint4 *>(src + at.x);
            b[i] = *reinterpret_cast<const uint4 *>(src + at.y);
        }
    };
    load(s);  // (on their way while the sines are computed)
    Turn t;
    if (turned) t = load_turn<INTERLEAVED>(p.frequencies, unit, p.rotary_dim, __ldg(p.positions + token), p.magnitude);
    for (int r0 = s; r0 < end; r0 += kBatch * split) {
        if (r0 != s) load(r0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * split;
            if (r >= end) break;
            const bool is_q = r < p.n_q, is_v = r >= p.n_q + p.n_kv;
            float v[16];
            if (FP8 || (turned && !is_v)) widen(a[i], b[i], v);
            if (turned && !is_v) turn_pairs<INTERLEAVED>(v, t);
            if (is_q || !FP8) {
                if (turned && !is_v) narrow(v, a[i], b[i]);
                __nv_bfloat16 *dst;
                if (is_q) {
                    dst = q_out + static_cast<int64_t>(r) * kHeadDim;
                } else {
                    const int h = is_v ? r - p.n_q - p.n_kv : r - p.n_q;
                    dst = static_cast<__nv_bfloat16 *>(is_v ? p.v_cache : p.k_cache) +
                          ((block * p.n_kv + h) * kBlockSize + place) * kHeadDim;
                }
                *reinterpret_cast<uint4 *>(dst + at.x) = a[i];
                *reinterpret_cast<uint4 *>(dst + at.y) = b[i];
            } else {
                float most = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(v[k]));
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(group, most, off));
                most = fmaxf(most, 0x1p-100f);
                const float inv = __fdiv_rn(448.f, most);
                uint32_t code[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    code[k] = f32x2_to_e4m3x2(__fmul_rn(v[4 * k], inv), __fmul_rn(v[4 * k + 1], inv)) |
                              (f32x2_to_e4m3x2(__fmul_rn(v[4 * k + 2], inv), __fmul_rn(v[4 * k + 3], inv)) << 16);
                const int h = is_v ? r - p.n_q - p.n_kv : r - p.n_q;
                const int64_t row = (block * p.n_kv + h) * kBlockSize + place;
                uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + row * kHeadDim;
                *reinterpret_cast<uint2 *>(dst + at.x) = make_uint2(code[0], code[1]);
                *reinterpret_cast<uint2 *>(dst + at.y) = make_uint2(code[2], code[3]);
                if (unit == 0) (is_v ? p.v_scale : p.k_scale)[row] = __fdiv_rn(most, 448.f);
            }
        }
    }
}

// Threads that share a token's rows: enough for every SM, at most one a row, at most 8 rows each.
int row_split(int64_t units, int rows, int sm_count) {
    const int64_t want = static_cast<int64_t>(sm_count > 0 ? sm_count : 1) * 2048;
    const int64_t few = std::max<int64_t>((want + units - 1) / units, (rows + 7) / 8);
    return static_cast<int>(std::min<int64_t>(few, rows));
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, bool interleaved, int sm_count, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(p.num_tokens) * (p.head_dim / kRotaryUnit);
    const int split = row_split(units, p.num_heads, sm_count);
    const int64_t blocks = (units * split + kRotaryThreads - 1) / kRotaryThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(interleaved ? rotary_kernel<true> : rotary_kernel<false>, dim3(static_cast<unsigned>(blocks)),
                      dim3(kRotaryThreads), 0, stream, p, split);
}

cudaError_t launch_rotary_write(const RotaryWriteParams &p, bool interleaved, bool fp8, int sm_count,
                                cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(p.num_tokens) * (kHeadDim / kRotaryUnit);
    const int split = row_split(units, p.n_q + 2 * p.n_kv, sm_count);
    const int64_t blocks = (units * split + kRotaryThreads - 1) / kRotaryThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    auto kernel = interleaved ? (fp8 ? rotary_write_kernel<true, true> : rotary_write_kernel<true, false>)
                              : (fp8 ? rotary_write_kernel<false, true> : rotary_write_kernel<false, false>);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kRotaryThreads), 0, stream, p, split);
}

}  // namespace pkv
