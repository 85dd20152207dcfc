// latent_prefill.cu -- expanded latent attention of a causal prefill chunk on the
// 5th-generation tensor cores (tcgen05.mma, accumulators in tensor memory).
//
//     s_j = scale (<q_nope, k_nope_j> + <q_rope, r_j>), j <= k_len - q_len + i,
//     out_i = sum_j softmax(s)_j v_j
//
// One CTA takes two adjacent tiles of 128 query rows of one head and walks the keys in
// tiles of 128 once for both (where such pairs do not fill the GPU, each walks a part of the
// keys, and a second kernel joins the parts (m, l, O)); per key tile and row tile S = Q K^T (M = N = 128, 192 values:
// two chunks of k_nope, one of the rotated key that all heads share) and O += P V (P from
// tensor memory).  Tensor memory: S / P of row tile t in columns [128 t, +128), O in
// [256 + 128 t, +128).
//
// What bounds it: a key tile costs two row tiles 2 x (768 + 512) cycles of the tensor pipe;
// its operands read 2 x 128 KB of shared memory and its 80 KB of keys and values are
// written there, 2690 cycles at 128 B a clock.  Shared memory is the nearer limit: the S
// MMAs (8 KB of operands in 64 cycles) leave nothing for the copies and take 85 cycles each
// beside them; a tile takes 3300-3600 cycles, in which the pipe is hardly ever idle.  One SM's
// TMA unit delivers 24 B a clock (measured), too little for 80 KB in 2560 cycles, so K comes by
// TMA and V by cp.async, which also fills rows past the sequence's end with zeros (a weight of
// 0 times a stranger's NaN would be NaN).
//
// Warps:
//  * 0-3 softmax of row tile 0, 4-7 of row tile 1, a row a thread: 64 scores at a time, one
//    pass, weights P = 2^(s - m) against a reference m straight back over the consumed scores
//    as bf16 (relative 2^-8).  m is the row's first largest score; only where the weights of 64
//    scores add up to more than 64 x 2^8 is the largest one looked for, m raised by a whole power
//    of two, and what was made with the old one (weights, l, O) rescaled exactly: bf16 and fp32
//    hold weights above 1 as they hold those below (462 -> 452 us on 8192 tokens x 32 heads
//    against a maximum over every 64 scores).  The sum l stays in fp32.  (l of the rounded
//    weights, which would round as the numerator does, is two instructions more a weight: 461 ->
//    480 us; a quarter of the exponentials as polynomials on the FMA pipe 480 -> 506; scores 32 at
//    a time with the next ones on their way spill: 452 -> 480.)
//  * 8 TMA: the first row tile's Q, K.  10-13 cp.async: the second's Q, V.  Chunks of 16 KB:
//    three a key tile of K ([128 keys][64 values]) and two of V ([64 keys][128 dims]), each kind
//    in a ring of 4, each refilled as the MMAs that read it end.  (One ring of 8 for both let the
//    next K wait for this V: 474 us.)
//  * 9 issues the MMAs in the order S0(k), P1 V(k-1), S1(k), P0 V(k): while one row tile's
//    softmax runs the tensor pipe has the other's P V and next S (with a warp a tile they
//    fell into step, both softmaxes at once and the pipe idle: 5400 cycles a key tile).
//    S(k + 1) follows P V (k): it overwrites the P that P V reads, and the MMAs of one
//    thread run in order.
//
// 8192 tokens x 32 heads: 450 us, 1.53 PFLOP/s (487, 1.41, in a run of seconds under the power cap).  Short chunks (4 of 162-417 rows behind
// 179-791 cached ones, 32 heads): 35.1 us; 224 CTAs of 4 to 9 key tiles on 152 SMs, each with
// 5-6 us of launch, first copies and epilogue.  (CTAs that take the next unit themselves,
// its copies issued early: no gain there, and the long prompt's loop got 6% slower.)
//
// Every mbarrier wait is bounded; a role whose wait runs out raises a CTA-wide abort
// flag, the others stop at their next wait, and the CTA records PKV_STATUS_TIMEOUT and
// frees its tensor memory before it returns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "latent.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kRows = 128;                    // query rows a tile
constexpr int kKeys = 128;                    // keys a tile
constexpr int kTmaWarp = 8, kMmaWarp = 9, kLoadWarp = 10;
constexpr int kLoadThreads = 128;
constexpr int kThreads = 14 * 32;
constexpr uint32_t kChunk = 128 * 128;        // 16 KB: 128 rows x 64 values
constexpr int kSlotsK = 4, kPerTileK = 3;     // ring of K chunks; a key tile has k_nope 0, 1, k_rope
constexpr int kSlotsV = 4, kPerTileV = 2;     // ring of V chunks; a key tile has keys 0-63, 64-127
constexpr uint32_t kOffQ = 0;                 // [row tile][3 chunks]
constexpr uint32_t kOffK = 6 * kChunk;
constexpr uint32_t kOffV = kOffK + kSlotsK * kChunk;  // a chunk: [dim half][64 keys][128 B]
constexpr uint32_t kOffBar = kOffV + kSlotsV * kChunk;
enum { kBarQ = 0, kBarFullK, kBarFullV = kBarFullK + kSlotsK, kBarEmptyK = kBarFullV + kSlotsV,
       kBarEmptyV = kBarEmptyK + kSlotsK, kBarS = kBarEmptyV + kSlotsV, kBarP = kBarS + 2, kBarO = kBarP + 2,
       kBarMerge = kBarO + 2, kNumBars };
constexpr uint32_t kOffTmem = kOffBar + 8 * kNumBars;
constexpr uint32_t kOffAbort = kOffTmem + 4;
constexpr uint32_t kSmemBytes = kOffAbort + 4;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
constexpr uint32_t kTmemCols = 512, kTmemO = 256;
constexpr float kRaise = 8.f, kTooMuch = 64.f * 256.f;

// kind::f16, D f32, A and B bf16, M = 128.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);
constexpr uint32_t kIdescQK = kIdesc | ((128u >> 3) << 17);
constexpr uint32_t kIdescPV = kIdesc | ((128u >> 3) << 17) | (1u << 16);  // B (V) MN-major, 128 dims

__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// 16 bytes global -> shared; zeros where !valid (the source is not read then).
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

template <bool kParts>  // the key tiles of a pair of row tiles in p.splits parts
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap rmap,
                          const LatentPrefillParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Pairs of row tiles in reverse: later rows see more keys, so the longest CTAs start first.  Split `sp` of a pair takes
    // the sp-th part of its key tiles.
    const int h = blockIdx.x, b = blockIdx.y, sp = kParts ? blockIdx.z / p.pairs : 0,
              pair = p.pairs - 1 - static_cast<int>(kParts ? blockIdx.z % p.pairs : blockIdx.z);

    if (tid == 0) {
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&rmap);
    }
    griddep_launch_dependents();
    griddep_wait();  // the producers of q, keys and values before us on the stream
    if (sbase & 1023u) {  // operands need the 1 KB swizzle alignment
        if (tid == 0) atomicOr(p.status, kStatusTimeout);
        return;
    }
    const int q0 = __ldg(p.cu_q_lens + b), q_len = __ldg(p.cu_q_lens + b + 1) - q0;
    const int k_first = __ldg(p.cu_k_lens + b), k_all = __ldg(p.cu_k_lens + b + 1) - k_first;
    const int r_lo = 2 * pair * kRows;  // this CTA's first row of the chunk
    auto part_at = [&](int64_t row) { return (static_cast<size_t>(sp) * p.total_q + row) * p.heads + h; };
    auto part_of = [&](int64_t row) -> float2 & { return p.part_ml[part_at(row)]; };
    if (q_len < 0 || q_len > k_all || q_len > p.max_q_len || q0 < 0 || k_first < 0 ||
        static_cast<int64_t>(q0) + q_len > p.total_q || static_cast<int64_t>(k_first) + k_all > p.total_k) {
        if (pair == 0 && h == 0 && sp == 0 && tid == 0) atomicOr(p.status, kStatusBadQLen);
        // The rows that can be addressed read as zeros; the last pair of the grid takes those past max_q_len too.
        if (q0 >= 0) {
            const int64_t end = min(static_cast<int64_t>(q_len), static_cast<int64_t>(p.total_q) - q0);
            const int64_t hi = pair == p.pairs - 1 ? end : min(end, static_cast<int64_t>(r_lo) + 2 * kRows);
            if (kParts) {  // (the merge writes the zeros)
                for (int64_t i = r_lo + tid; i < hi; i += kThreads) part_of(q0 + i) = make_float2(-INFINITY, 0.f);
                return;
            }
            const int chunks = p.out_bf16 ? 16 : 32;  // 16-byte pieces of a row
            for (int64_t idx = tid; idx < (hi - r_lo) * chunks; idx += kThreads) {
                const size_t row = static_cast<size_t>(q0) + r_lo + idx / chunks;
                reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) +
                                          (row * p.heads + h) * kExpandedV * (p.out_bf16 ? 2 : 4))[idx % chunks] =
                    make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }
    // Row tile t: rows i0 .. i0 + rows - 1 of the chunk, keys 0 .. k_all - q_len + i0 + rows - 1, in key tiles.
    auto tile_rows = [&](int t) { return max(0, min(kRows, q_len - r_lo - t * kRows)); };
    auto tiles_of = [&](int t) {
        const int rows = tile_rows(t);
        return rows > 0 ? (k_all - q_len + r_lo + t * kRows + rows + kKeys - 1) / kKeys : 0;
    };
    // This part's key tiles; the keys from its first one on are as if they were the sequence's.
    const int per = kParts ? (max(tiles_of(0), tiles_of(1)) + p.splits - 1) / p.splits : 0, skipped = sp * per * kKeys;
    auto tile_nt = [&](int t) { return kParts ? max(0, min(tiles_of(t) - sp * per, per)) : tiles_of(t); };
    const int k0 = k_first + skipped, k_len = k_all - skipped, c = k_len - q_len;
    const int n_tiles = max(tile_nt(0), tile_nt(1));
    if (n_tiles == 0) {
        if (kParts)
            for (int i = tid; i < min(2 * kRows, q_len - r_lo); i += kThreads) part_of(q0 + r_lo + i) = make_float2(-INFINITY, 0.f);
        return;
    }

    auto bar = [&](int i) { return sbase + kOffBar + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffTmem);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + kOffAbort);
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i)
            mbar_init(bar(i), i == kBarQ || (i >= kBarFullV && i < kBarEmptyK) ? kLoadThreads / 32
                              : (i >= kBarP && i < kBarO) || i == kBarMerge ? 4
                                                               : 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // A warp's bounded wait, each lane for a barrier of its own; it gives up soon after another role did (timer and
    // flag every 64 tries).
    auto lanes_wait = [&](uint32_t b, uint32_t parity) -> bool {
        uint64_t t_first = 0;
        for (uint32_t tries = 0; !__all_sync(0xffffffffu, mbar_try_wait(b, parity)); ++tries) {
            if ((tries & 63u) != 63u) continue;
            const uint64_t now = globaltimer_ns();
            if (t_first == 0) t_first = now;
            if (__any_sync(0xffffffffu, *abort_flag != 0 || now - t_first > kWaitLimitNs)) {
                *abort_flag = 1u;
                return false;
            }
        }
        return true;
    };
    auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool { return lanes_wait(b, parity); };
    // K chunk j (three a key tile) lies in slot j % 4 as its use j / 4, V chunk j (two) the same.
    auto full_k = [&](int j) { return bar(kBarFullK + j % kSlotsK); };
    auto full_v = [&](int j) { return bar(kBarFullV + j % kSlotsV); };
    auto empty_k = [&](int j) { return bar(kBarEmptyK + j % kSlotsK); };
    auto empty_v = [&](int j) { return bar(kBarEmptyV + j % kSlotsV); };

    // One row tile (short chunks, a chunk's last rows) leaves the other's warps and tensor memory free: its keys are split,
    // even tiles to the first group, odd ones to the second, and the first joins their O: a tile of keys in 1900 instead of
    // 3100 cycles (4 chunks of up to 110 rows over 5.6K keys, 32 heads: 81 -> 55 us).  Else each group has a row tile.
    auto roles = [&](auto split) {
        constexpr bool kSplit = decltype(split)::value;
        auto steps = [&](int t) { return kSplit ? (n_tiles + 1 - t) >> 1 : tile_nt(t); };  // key tiles that group t takes
        auto key_tile = [&](int t, int i) { return kSplit ? 2 * i + t : i; };
        if (warp == kTmaWarp) {
            bool ok = true;
            for (int j = 0; ok && j < kPerTileK * n_tiles; ++j) {
                if (j >= kSlotsK && !(ok = warp_wait(empty_k(j), ((j / kSlotsK) - 1) & 1))) break;
                const int kt = j / kPerTileK, i = j - kPerTileK * kt;
                const uint32_t dst = sbase + kOffK + (j % kSlotsK) * kChunk;
                if (elect_one()) {
                    // The first row tile's Q comes with the first K, chunk by chunk: S starts after 32 KB.
                    mbar_arrive_expect_tx(full_k(j), kt == 0 ? 2 * kChunk : kChunk);
                    if (kt == 0) tma_load_3d(sbase + kOffQ + i * kChunk, &qmap, full_k(j), 64 * i, h, q0 + r_lo);
                    if (i < 2)
                        tma_load_3d(dst, &kmap, full_k(j), 64 * i, h, k0 + kt * kKeys);
                    else
                        tma_load_2d(dst, &rmap, full_k(j), 0, k0 + kt * kKeys);
                }
                __syncwarp();
            }
        } else if (warp >= kLoadWarp) {
            const int t = tid - kLoadWarp * 32;
            // The second row tile's Q: 8 threads a 64-value chunk of a row, 16 rows at a time (zeros past the last row).
            if (tile_rows(1) > 0) {
                const int row = t >> 3, v = t & 7, r1 = q0 + r_lo + kRows + row;
                const uint16_t *src = static_cast<const uint16_t *>(p.q) + static_cast<int64_t>(r1) * p.q_row + h * p.q_head + v * 8;
                const uint32_t dst = sbase + kOffQ + 3 * kChunk + row * 128 + ((v ^ (row & 7)) << 4);
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        cp_async_16_or_zero(dst + i * kChunk + r * 16 * 128, src + 64 * i + r * 16 * p.q_row, r1 + 16 * r < p.total_q);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            // V, 16 threads a row, 8 rows at a time; rows past the sequence's keys become zeros.
            const int row = t >> 4, v = t & 15;
            const uint32_t to = (v >> 3) * (kChunk / 2) + row * 128 + (((v & 7) ^ row) << 4);
            bool ok = true;
            for (int kt = 0; ok && kt < n_tiles; ++kt) {
                for (int i = 0; i < kPerTileV; ++i) {
                    const int j = kPerTileV * kt + i, key = kt * kKeys + 64 * i + row;
                    if (j >= kSlotsV) ok = ok && warp_wait(empty_v(j), ((j / kSlotsV) - 1) & 1);
                    if (!ok) break;
                    const uint16_t *src = static_cast<const uint16_t *>(p.v) + (static_cast<int64_t>(k0) + key) * p.k_row +
                                          h * p.k_head + v * 8;
                    const uint32_t dst = sbase + kOffV + (j % kSlotsV) * kChunk + to;
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        cp_async_16_or_zero(dst + r * 8 * 128, src + r * 8 * p.k_row, key + 8 * r < k_len);
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    // What came before (Q, then the chunk before) has landed: made visible to the tensor core, an arrival a warp.
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(j == 0 ? bar(kBarQ) : full_v(j - 1));
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(full_v(kPerTileV * n_tiles - 1));
        } else if (warp == kMmaWarp) {
            // The warp runs whole on warp-uniform values, one elected lane issues: descriptors stay in uniform registers.
            const int nt0 = steps(0), nt1 = steps(1);
            const uint64_t q_desc = sw128_desc(sbase + kOffQ, 16, 1024);
            const uint64_t k_desc = sw128_desc(sbase + kOffK, 16, 1024);
            const uint64_t v_desc = sw128_desc(sbase + kOffV, kChunk / 2, 1024);  // 128 dims: two halves side by side
            bool ok = true;
            // Besides the weights the warp waits for K chunks only where it needs them first: the softmax warps look that
            // V(k) and the first chunk of K(k + 1) have landed before they hand over P(k) (a wait costs this warp 100
            // cycles and more even when it need not wait); the others are given until the MMAs before them are issued.
            ok = ok && warp_wait(full_k(0), 0);
            auto score = [&](int t, int i) {
                const int kt = key_tile(t, i);
                const bool first_reader = kSplit || t == 0 || kt >= nt0, last_reader = kSplit || t == 1 || kt >= nt1;
                tc_fence_after();
                const uint64_t qd = q_desc + static_cast<uint32_t>(kSplit ? 0 : 3 * t) * (kChunk >> 4);
                const int j = kPerTileK * kt;
                auto chunk = [&](int i) {
                    const uint64_t kd = k_desc + static_cast<uint32_t>((j + i) % kSlotsK) * (kChunk >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(tmem + 128 * t, qd + i * (kChunk >> 4) + 2 * kk, kd + 2 * kk, kIdescQK, i > 0 || kk > 0);
                    if (last_reader) umma_commit(empty_k(j + i));
                };
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    if (first_reader && (kSplit || i > 0)) {
                        ok = ok && warp_wait(full_k(j + i), ((j + i) / kSlotsK) & 1);
                        tc_fence_after();
                    }
                    if (ok && elect_one()) {
                        chunk(i);
                        if (i == 2) umma_commit(bar(kBarS + t));
                    }
                    __syncwarp();
                }
            };
            auto value = [&](int t, int step) {
                const int kt = key_tile(t, step);
                const bool of_v = kSplit && (lane == 1 || lane == 2);  // (else the softmax warps looked)
                const int jv = kPerTileV * kt + (lane & 1);
                if (!(ok = ok && lanes_wait(of_v ? full_v(jv) : bar(kBarP + t), (of_v ? jv / kSlotsV : step) & 1))) return;
                tc_fence_after();
                const uint32_t o = tmem + kTmemO + 128 * t, w = tmem + 128 * t;
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = kPerTileV * kt + i;
                        const uint64_t vd = v_desc + static_cast<uint32_t>(j % kSlotsV) * (kChunk >> 4);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            umma_bf16_tmem_a(o, w + 32 * i + 8 * ks, vd + ks * (2048 >> 4), kIdescPV, step > 0 || i + ks > 0);
                        if (kSplit || t == 1 || kt >= nt1) umma_commit(empty_v(j));  // its last reader
                    }
                    if (step == (t == 0 ? nt0 : nt1) - 1) umma_commit(bar(kBarO + t));
                }
                __syncwarp();
            };
            for (int i = 0; ok && i <= max(nt0, nt1); ++i) {
                if (i < nt0) score(0, i);
                if (ok && i >= 1 && i - 1 < nt1) value(1, i - 1);
                if (!kSplit && i == 0 && nt1 > 0) ok = ok && warp_wait(bar(kBarQ), 0);
                if (ok && i < nt1) score(1, i);
                if (ok && i < nt0) value(0, i);
            }
        } else {
            // ---------------- softmax: a row a thread ----------------
            const int t = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
            const int nt = steps(t), nt0 = tile_nt(0), rows = tile_rows(kSplit ? 0 : t), i0 = r_lo + (kSplit ? 0 : t * kRows);
            const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
            const uint32_t s_at = tmem + lanes + 128 * t, o_at = tmem + lanes + kTmemO + 128 * t;
            const float sl2 = p.scale_log2;
            const bool neg = sl2 < 0.f;  // then the largest score is the smallest product
            const float hidden = neg ? INFINITY : -INFINITY;
            const int limit = c + i0 + r;  // last visible key
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f), l3 = l2;  // the sum, in four parts
            bool alive = true;
            for (int i = 0; alive && i < nt; ++i) {
                const int kt = key_tile(t, i);
                if (!(alive = warp_wait(bar(kBarS + t), i & 1))) break;
                tc_fence_after();
                const bool mask = kt * kKeys + kKeys - 1 > c + i0;  // some row does not see some key
                auto load = [&](int cc, uint32_t(&v)[64]) {
                    tmem_ld_32x32b_x64(s_at + 64 * cc, v);
                    if (mask) {
                        const int last = limit - kt * kKeys - 64 * cc;
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (e > last) v[e] = __float_as_uint(hidden);
                    }
                };
                // The largest score of 64 (log2 domain).
                auto largest = [&](const uint32_t(&v)[64]) {
                    float x[4] = {hidden, hidden, hidden, hidden};
                    if (neg) {
#pragma unroll
                        for (int e = 0; e < 64; ++e) x[e & 3] = fminf(x[e & 3], __uint_as_float(v[e]));
                        return fminf(fminf(x[0], x[1]), fminf(x[2], x[3])) * sl2;
                    }
#pragma unroll
                    for (int e = 0; e < 64; e += 2)
                        x[(e >> 1) & 3] = fmax3(x[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * sl2;
                };
#pragma unroll 1
                for (int cc = 0; cc < 2; ++cc) {
                    uint32_t v[64], w[32];
                    load(cc, v);
                    float2 a2, a3;  // the chunk's sum, in four parts
                    // The reference is looked at only where it has to be: for a row's first keys, and again where weights against
                    // the old one add up to more than 64 x 2^8.
                    for (bool raise = __any_sync(0xffffffffu, m == -INFINITY);;) {
                        if (raise) {
                            // Raise the references that are passed to the largest score from here on, and rescale what was made
                            // with the old one: the weights before, l, O.
                            float mx = largest(v);
                            if (cc == 0) {
                                uint32_t u[64];
                                load(1, u);
                                mx = fmaxf(mx, largest(u));
                            }
                            float alpha = 1.f;
                            if (mx > m + kRaise) {
                                // The first largest score as it is, then steps of whole powers of two: the weights of the
                                // largest scores are exact in bf16, and a row of one key is its value.  (From 2^256 on
                                // nothing is left of what was: the new score itself, for a step from a mask's -1e10 or
                                // less is rounded by more than the scores that follow.)
                                const float up = ceilf(mx - m);
                                alpha = fast_exp2(-up);
                                m = up < 256.f ? m + up : mx;
                            }
                            l2 = fmul2(l2, make_float2(alpha, alpha));
                            l3 = fmul2(l3, make_float2(alpha, alpha));
                            tmem_wait_st();  // the weights that are read back now
#pragma unroll 1
                            for (int k = 0; k < 2 * cc; ++k) {
                                uint32_t wt[16];
                                tmem_ld_32x32b_x16(s_at + 16 * k, wt);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    wt[e] = pack_bf16x2(__uint_as_float(wt[e] << 16) * alpha, __uint_as_float(wt[e] & 0xffff0000u) * alpha);
                                tmem_st_32x32b_x16(s_at + 16 * k, wt);
                            }
                            if (i > 0) {  // every earlier P V of this tile completed before S (kt) did
#pragma unroll 1
                                for (int k = 0; k < 8; ++k) {
                                    uint32_t u[16];
                                    tmem_ld_32x32b_x16(o_at + 16 * k, u);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
                                    tmem_st_32x32b_x16(o_at + 16 * k, u);
                                }
                            }
                            tmem_wait_st();
                            load(cc, v);  // (kept in tensor memory meanwhile, not in registers)
                        }
                        const float mu = m == -INFINITY ? 0.f : m;
                        const float2 sv = make_float2(sl2, sl2), nm = make_float2(-mu, -mu);
                        a2 = a3 = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float2 x = ffma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sv, nm);
                            const float2 pr = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                            if (e & 1)
                                a3 = fadd2(a3, pr);
                            else
                                a2 = fadd2(a2, pr);
                            w[e] = pack_bf16x2(pr.x, pr.y);
                        }
                        if (raise || !__any_sync(0xffffffffu, (a2.x + a2.y) + (a3.x + a3.y) > kTooMuch)) break;
                        raise = true;
                        load(cc, v);
                    }
                    l2 = fadd2(l2, a2);
                    l3 = fadd2(l3, a3);
                    tmem_st_32x32b_x32(s_at + 32 * cc, w);
                }
                tmem_wait_st();
                if (!kSplit && quarter == 0 && (t == 0 || kt >= nt0)) {
                    // V(kt) and, for the S that follows, the first chunk of K(kt + 1): a lane a chunk.
                    const int jv = kPerTileV * kt + (lane & 1), jk = kPerTileK * (kt + 1);
                    const bool of_k = lane == 2 && kt + 1 < n_tiles;
                    alive = lanes_wait(of_k ? full_k(jk) : full_v(jv), (of_k ? jk / kSlotsK : jv / kSlotsV) & 1);
                }
                tc_fence_before();
                __syncwarp();
                if (alive && lane == 0) mbar_arrive(bar(kBarP + t));
            }
            // ---------------- epilogue: out = O / l ----------------
            if (nt > 0 && alive && warp_wait(bar(kBarO + t), 0)) {
                tc_fence_after();
                float l = (l2.x + l2.y) + (l3.x + l3.y), w0 = 1.f, w1 = 0.f;
                // Split keys: the second group's (m, l) in the place of a second row tile's Q, its O in K's ring, which every S is
                // done with ([128 rows][32 vectors], a row's vectors turned by the row).
                const uint32_t other_ml = sbase + kOffQ + 3 * kChunk + 8 * r, other_o = sbase + kOffK + 512 * r;
                if (kSplit && t == 1) {
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(o_at + 32 * k, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            sts128(other_o + (((8 * k + e) ^ lane) << 4), make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
                    }
                    sts32(other_ml, __float_as_uint(m));
                    sts32(other_ml + 4, __float_as_uint(l));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarMerge));
                    return;
                }
                if (kSplit) {
                    if (!warp_wait(bar(kBarMerge), 0)) return;
                    const float2 ml = lds_f32x2(other_ml);
                    const float all = fmaxf(m, ml.x);
                    // (A side that a row sees nothing of weighs 0.  One whose scores are all NaN has m = -infinity too, but its l
                    // is NaN, and so is its weight; the difference of two infinities is NaN as well.)
                    w0 = m == -INFINITY ? l : fast_exp2(m - all);
                    w1 = ml.x == -INFINITY ? ml.y : fast_exp2(ml.x - all);
                    l = w0 * l + w1 * ml.y;
                    m = all;
                }
                const float inv = kParts ? 1.f : l > 0.f ? 1.f / l : 0.f;
                // bf16: a warp's 32 rows through its part of Q's place, then out in runs of 256 bytes (by TMA, at 24 bytes a clock,
                // two full row tiles took 2 us longer).
                const uint32_t stage = sbase + kOffQ + 3 * t * kChunk;
                const bool bf16 = p.out_bf16 && !kParts;
                float *out = kParts ? p.part_o + part_at(q0 + i0 + r) * kExpandedV
                                    : static_cast<float *>(p.out) + ((static_cast<size_t>(q0) + i0 + r) * p.heads + h) * kExpandedV;
                if (kParts && r < rows) part_of(q0 + i0 + r) = make_float2(m, l);
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(o_at + 32 * k, v);
                    if (kSplit) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint4 u = lds128(other_o + (((8 * k + e) ^ lane) << 4));
                            auto join = [&](int x, uint32_t y) {
                                v[4 * e + x] = __float_as_uint(w0 * __uint_as_float(v[4 * e + x]) + (w1 == 0.f ? 0.f : w1 * __uint_as_float(y)));
                            };
                            join(0, u.x), join(1, u.y), join(2, u.z), join(3, u.w);
                        }
                    }
                    auto f = [&](int e) { return __uint_as_float(v[e]) * inv; };
                    if (bf16) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 w = make_uint4(pack_bf16x2(f(8 * e), f(8 * e + 1)), pack_bf16x2(f(8 * e + 2), f(8 * e + 3)),
                                                       pack_bf16x2(f(8 * e + 4), f(8 * e + 5)), pack_bf16x2(f(8 * e + 6), f(8 * e + 7)));
                            sts128(stage + (k >> 1) * kChunk + r * 128 + (((4 * (k & 1) + e) ^ (r & 7)) << 4), w);
                        }
                    } else if (r < rows) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            reinterpret_cast<float4 *>(out)[8 * k + e] = make_float4(f(4 * e), f(4 * e + 1), f(4 * e + 2), f(4 * e + 3));
                    }
                }
                if (bf16) {
                    __syncwarp();
                    const int c = lane & 15;
                    uint4 *dst = static_cast<uint4 *>(p.out) + ((static_cast<size_t>(q0) + i0) * p.heads + h) * (kExpandedV / 8) + c;
#pragma unroll 4
                    for (int k = 0; k < 16; ++k) {
                        const int row = quarter * 32 + 2 * k + (lane >> 4);
                        const uint4 w = lds128(stage + (c >> 3) * kChunk + row * 128 + (((c & 7) ^ (row & 7)) << 4));
                        if (row < rows) dst[static_cast<size_t>(row) * p.heads * (kExpandedV / 8)] = w;
                    }
                }
            } else if (kParts && nt == 0 && r < rows) {
                part_of(q0 + i0 + r) = make_float2(-INFINITY, 0.f);
            }
        }
    };
    if (tile_rows(1) == 0 && n_tiles > 1)
        roles(std::true_type{});
    else
        roles(std::false_type{});

    // ---- teardown: every role is done (or gave up); free tensor memory ----
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag && tid == 0) {
        atomicOr(p.status, kStatusTimeout);
        // Copies and MMAs that are still in flight: let them finish before the CTA's memory is freed.
        const uint64_t until = globaltimer_ns() + kWaitLimitNs;
        while (globaltimer_ns() < until) {
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the splits of a (row, head): out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s, a warp each, four values a lane.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(kMergeWarps * 32) latent_prefill_merge_kernel(const LatentPrefillParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5), all = static_cast<int64_t>(p.total_q) * p.heads;
    griddep_launch_dependents();
    griddep_wait();
    if (at >= min(all, static_cast<int64_t>(__ldg(p.cu_q_lens + p.num_seqs)) * p.heads)) return;
    const float2 ml = lane < p.splits ? p.part_ml[lane * all + at] : make_float2(-INFINITY, 0.f);
    const float4 *src = reinterpret_cast<const float4 *>(p.part_o) + at * (kExpandedV / 4) + lane;
    float m = ml.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    // (A part without a weight may hold anything; l is NaN where a query or a key was.)
    const float w = ml.x == -INFINITY && ml.y == 0.f ? 0.f : exp2f(ml.x - (m == -INFINITY ? 0.f : m));
    float sum = ml.x == -INFINITY && ml.y == 0.f ? 0.f : w * ml.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint32_t used = __ballot_sync(0xffffffffu, !(ml.x == -INFINITY && ml.y == 0.f));
#pragma unroll 4
    for (int k = 0; k < p.splits; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        if (!((used >> k) & 1u)) continue;
        const float4 v = src[k * all * (kExpandedV / 4)];
        o.x += wk * v.x, o.y += wk * v.y, o.z += wk * v.z, o.w += wk * v.w;
    }
    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // NaN stays
    if (p.out_bf16)
        reinterpret_cast<uint2 *>(p.out)[at * (kExpandedV / 4) + lane] = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    else
        reinterpret_cast<float4 *>(p.out)[at * (kExpandedV / 4) + lane] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

}  // namespace

cudaError_t latent_prefill_prepare_device() {
    const int bytes = static_cast<int>(kSmemBytes);
    const cudaError_t e = cudaFuncSetAttribute(latent_prefill_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(latent_prefill_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

cudaError_t launch_latent_prefill(const LatentPrefillMaps &maps, const LatentPrefillParams &p, cudaStream_t stream) {
    const cudaError_t e = launch_pdl(p.splits > 1 ? latent_prefill_kernel<true> : latent_prefill_kernel<false>, dim3(p.heads, p.num_seqs, p.pairs * p.splits), dim3(kThreads), kSmemBytes,
                                     stream, maps.q, maps.k, maps.rope, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    const int64_t blocks = (static_cast<int64_t>(p.total_q) * p.heads + kMergeWarps - 1) / kMergeWarps;
    return launch_pdl(latent_prefill_merge_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kMergeWarps * 32), 0, stream, p);
}

}  // namespace pkv
