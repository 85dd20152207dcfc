// latent_decode.cu -- absorbed latent attention over the paged pool (decode and verify)
// on the 5th-generation tensor cores.
//
//     s_j = scale (<q_latent, c_j> + <q_rope, r_j>),  out = sum_j softmax(s)_j c_j
//
// Every (query row, head) pair of a sequence is a column that reads the same cached
// rows, so a CTA takes up to 64 columns and reads each key once for all of them.
//
// Work split: the keys of all sequences are one line of tiles, cut into equal ranges,
// one CTA per SM and column tile (context lengths are device data, so every CTA sums
// them itself; a sequence's start counts a few tiles more, for its Q and the epilogue).
// A range covers whole sequences and at most two parts of one; whole sequences are
// written out, parts go to the workspace as (m, l, O) and the merge kernel folds them.
// No CTA waits for another.
//
// Per tile (bf16: 32 keys, four stages of 36 KB; up to 16 columns 64 keys, two stages;
// FP8: 64 keys, 40 KB, four stages, with 64 columns three):
//  * S [columns x keys] = Q K^T: M = 64 (FP8 with 64 columns 128), N = keys; Q stays in
//    shared memory (128-byte swizzle).  Over an FP8 pool Q is pairs of E4M3 codes, P three E5M2 codes a weight.
//  * half of the blocks are copied by TMA, half by cp.async: one SM's TMA unit delivers 24
//    bytes a clock however much is in flight (measured, from L2 as from HBM), both paths
//    together 47; HBM's share of an SM is 23-28, so a ring on TMA alone never catches up.
//  * softmax by 8 warps (a warp: a quarter of the columns, half of the keys): running reference m,
//    raised only when a score passes it by 2^8 (one vote a tile), sum l in fp32;
//    P = 2^(s - m) rounded to bf16 (l adds the rounded weights, so numerator and
//    denominator round alike) into shared memory as the B operand, two buffers in turn.
//  * O^T [512 dims x columns] += V^T P^T: the same bytes as K, read as an MN-major A
//    operand: M = 128 (4 tiles of dims), N = columns, 16 keys a step (FP8: 32).  Transposed,
//    because O has 512 x 64 values: as 128 lanes x 256 columns it leaves tensor memory
//    for two S buffers, and M is full for any number of heads.
// S and P V are issued by two warps, so neither waits behind the other's inputs (one
// issuer that waits for the next tile's copy before a P V leaves no copy in flight);
// P V frees a stage block by block.
//
// What bounds it (cycles of one CTA, 1.9 GHz): a tile of 32 keys takes 1550-1650.  With 32
// columns that is HBM's rate (23 bytes a clock and SM: 6.6 TB/s; the ragged batch of 64
// sequences and 32 heads 39.0 us, 25.5 of them bytes); with 64 the tensor pipe, 36 MMAs of
// 28 cycles for S and 16 of 52 for P V, whose operands come from shared memory (8 x 32K
// tokens of 64 heads 63.9 us, 128 heads over 32 sequences 72.6).  FP8: 64 keys a tile,
// with 32 columns the ring's four stages held from S to P V (32.3 us, 14.5 of bytes; 30.2 with P
// as two codes), with 64 the tensor pipe and three stages (4 rows x 64 heads over 16 sequences
// 100.9 us, 39.9 of operations; 90.8 with two codes).  Around
// the tiles: launch, plan and first copies 5 us, Q of another sequence and the epilogue of
// the one before 2-4 us (72 KB of Q come in at 47 bytes a clock, 128 KB of O go out), the
// merge 4-6 us.
//
// Every mbarrier wait is bounded; a role whose wait runs out raises a CTA-wide abort
// flag, the others stop at their next wait, and the CTA records PKV_STATUS_TIMEOUT and
// frees its tensor memory before it returns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "latent.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kSoftWarps = 8;                 // warps w and w + 4 share rows 16 (w % 4) .. and split the keys
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kProducerWarp = kSoftWarps;
constexpr int kScoreWarp = kSoftWarps + 1;    // issues S = Q K^T
constexpr int kValueWarp = kSoftWarps + 2;    // issues O^T += V^T P^T
constexpr int kLoadWarp = kSoftWarps + 3;     // two pairs of copying warps, one pair a stage
constexpr int kThreads = (kSoftWarps + 7) * 32;
constexpr float kLeastScale = 0x1p-100f / 448.f;  // of an FP8 row, as latent_write_fp8_kernel makes it of zeros
constexpr int kMaxLeft = 1 << 20;  // of a tile's record; past the tile and 16 rows the keys are all the same
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;  // O^T in columns [0, 4 NCOL), the scores of tile i from 256 + (i & 1) kScoreCols on

// Shared memory for NCOL columns over a bf16 or an FP8 pool.
template <int NCOL, bool FP8, int TILE>
struct Layout {
    static constexpr int kTile = TILE, kTileBlocks = TILE / kBlockSize;  // keys a tile
    static constexpr int kTmaBlocks = kTileBlocks / 2;  // blocks of a tile that TMA copies; the others go through cp.async
    static constexpr int kGroups = TILE / 16;           // 8-key groups of the half tile that a warp takes
    // A block of 16 slots: [2 groups of 8 slots][chunks of 128 bytes][8 slots][128 B]; chunks are 64 bf16 values
    // (9 of them, the last the rotated key) or 128 codes (4; the rotated keys follow the stage's codes).
    static constexpr uint32_t kChunks = FP8 ? 4 : 9;
    static constexpr uint32_t kGroup = kChunks * 1024;
    static constexpr uint32_t kBlock = 2 * kGroup;
    static constexpr uint32_t kRopeBlock = FP8 ? kBlockSize * 128 : 0;
    static constexpr uint32_t kStage = kTileBlocks * (kBlock + kRopeBlock);
    // FP8: the E4M3 heads and remainders of Q are rows of one product, two of P's codes (up to 32 columns) columns of one:
    // an MMA of few columns is bound by its other operand, M = 128 takes 43 cycles with N = 32 and 52 with 64, and N = 64
    // takes 35 with M = 64 and 52 with 128.  A remainder's row is 8 behind its head's, in rows that M = 64 has anyway
    // and in the same thread after the load; for 64 columns 16 behind, M = 128.  P is three E5M2 codes a weight, what
    // each leaves in the next: the second's column is NCOL behind the first's (for 64 columns O has no room: a product of
    // its own), the third's product adds to the first's columns.
    static constexpr bool kStack = FP8 && NCOL <= 32;
    static constexpr int kOCols = kStack ? 2 * NCOL : NCOL;  // columns of a dim tile's O
    static constexpr int kStages = FP8 ? (kStack ? 4 : 3) : 128 / TILE;
    // What beginning another sequence costs a range, in tiles: its Q, the epilogue of the one before.
    static constexpr int kLead = FP8 ? 5 : 128 / TILE;
    // M = 64: rows 16 q .. 16 q + 15 of S lie in tensor-memory lanes 32 q .., which only warps w % 4 = q reach, one
    // scheduler's.  A quarter of the columns goes to each: column c is row 16 (c / kPerQuarter) + c % kPerQuarter.
    static constexpr int kPerQuarter = NCOL / 4, kRowsPerThread = NCOL == 64 ? 2 : 1;
    // Score columns of a tile (FP8: the latent's and the rotated key's products apart, the scale goes with the first).
    static constexpr uint32_t kScoreCols = FP8 ? 128 : 64;
    // Q: 9 chunks of [64 rows][128 B]; FP8: 4 chunks of [heads and remainders][128 B] (E4M3), one of the rotated part in
    // bf16.
    static constexpr int kQRows = FP8 && NCOL == 64 ? 128 : 64;
    static constexpr uint32_t kQChunk = kQRows * 128;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kQRope = kQ + (FP8 ? 4 : 8) * kQChunk;
    static constexpr uint32_t kKv = kQRope + 64 * 128;
    // P, two buffers in turn: [NCOL][64 bf16], or [NCOL][64 first | 64 second codes]; rows of 64 bytes (32 keys, or stacked
    // [first, second][NCOL][64 codes]) lie side by side.
    static constexpr uint32_t kP = kKv + kStages * kStage;
    static constexpr bool kPHalf = kStack || (!FP8 && TILE == 32);
    static constexpr uint32_t kPBuf = kPHalf ? 64 : NCOL * 128;
    static constexpr uint32_t kP3 = kP + (kPHalf ? 1 : 2) * kOCols * 128;  // FP8: third codes, [NCOL][two buffers of 64]
    static constexpr uint32_t kScale = kP3 + (FP8 ? NCOL * 128 : 0);  // FP8: [stage][scale, its log2, its inverse in kUnit][64 keys]
    static constexpr uint32_t kQf = kScale + (FP8 ? kStages * 3 * TILE * 4 : 0);  // FP8: [a piece's first tile & 1][64] factors of the columns
    // kv_full[stage], kv_empty[stage][block], s_full[2], s_empty[2], p_full[2], pv_done[2], q_full
    static constexpr int kBarKvFull = 0, kBarKvEmpty = kStages, kBarSFull = kBarKvEmpty + kStages * kTileBlocks,
                         kBarSEmpty = kBarSFull + 2, kBarPFull = kBarSEmpty + 2, kBarPvDone = kBarPFull + 2,
                         kBarQFull = kBarPvDone + 2, kNumBars = kBarQFull + 1;
    static constexpr uint32_t kBar = kQf + (FP8 ? 2 * 64 * 4 : 0);
    static constexpr uint32_t kTmemSlot = kBar + 8 * kNumBars;
    static constexpr uint32_t kAbort = kTmemSlot + 4;
    static constexpr uint32_t kXch = (kAbort + 4 + 15) / 16 * 16;  // [tile & 1][key half][64] maxima, later sums
    static constexpr uint32_t kAlpha = kXch + 4 * 64 * 4;          // [64] factors of O's columns
    static constexpr uint32_t kPlan = kAlpha + 64 * 4;             // warp totals, then the range's start
    // What softmax has to know of a stage's tile, by the warps that copy it: {keys left and the invalid blocks, tiles
    // left, sequence, next tile's sequence}.  (Walking the tiles itself cost softmax 240 cycles a tile, of 1600.)
    static constexpr uint32_t kInfo = kPlan + 18 * 8;
    static constexpr uint32_t kDead = kInfo + kStages * 16;  // [tile & 1]: a softmax warp's wait ran out
    static constexpr uint32_t kQAt = (kDead + 8 + 15) / 16 * 16;  // [NCOL] a column's places in a sequence's q_latent, q_rope
    static constexpr uint32_t kBytes = kQAt + NCOL * 16;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
    static_assert(kKv % 1024 == 0 && kP % 1024 == 0 && kStage % 1024 == 0, "swizzle atoms");
    static_assert(kScale % 16 == 0 && kBar % 8 == 0 && kPlan % 8 == 0 && kInfo % 16 == 0, "alignment");
    // A weight may pass the reference by 2^kRaise before the reference follows.  FP8 keeps a weight as three E5M2 codes:
    // 2^9 at the reference, so 2^15 at most (57344 is the largest code), and half of the smallest step is 2^-17, 2^-26 of
    // the reference: a million keys that small come to 2^-6 of it.  (Pairs of E4M3 codes, 2^2 at the reference and steps of
    // 2^-9, lost every key below 2^-12 of the largest: with one key of 0.3 of the weight and 14000 more up to 94% of
    // the output.  A raise of 2^4: on the verify of 64 columns a reference was raised in every second tile, 1900 cycles each.)
    static constexpr float kRaise = FP8 ? 6.f : 8.f, kLift = FP8 ? 9.f : 0.f;
    // FP8: the sum l takes a weight times 1 / s_j, 2^109 for a row of zeros (s = 2^-100 / 448): in units of 2^15, a thousand
    // of those would be infinite at 2^9.  (At the other end s is 2^120, and l 2^-126.)  O leaves in the same units.
    static constexpr float kUnit = FP8 ? 0x1p-15f : 1.f;
};

// Instruction descriptor: D f32; A and B bf16 (kind::f16), or A E4M3 and B E4M3 or E5M2 (kind::f8f6f4).
enum class Kind : uint32_t { kBf16 = (1u << 7) | (1u << 10), kE4m3 = 0, kE4m3E5m2 = 1u << 10 };
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool a_mn, Kind kind = Kind::kBf16) {
    return (1u << 4) | static_cast<uint32_t>(kind) | (a_mn ? 1u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// Shared-memory matrix descriptor of a 128-byte-swizzled operand; operands a few KB further on
// differ in the address field alone (`+ (bytes >> 4)`).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ bool bar_red_or(uint32_t id, uint32_t nthreads, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(static_cast<uint32_t>(pred)), "r"(nthreads)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Keys of sequence b that its rows see (0: none, its rows are zeros).
__device__ __forceinline__ int keys_of(const LatentDecodeParams &p, int b) {
    const int ctx = __ldg(p.context_lens + b);
    return ctx < 1 || ctx < p.q_per_seq ? 0 : min(ctx, p.max_blocks * kBlockSize);
}
template <typename L>
__device__ __forceinline__ int tiles_of(const LatentDecodeParams &p, int b) {
    return (keys_of(p, b) + L::kTile - 1) / L::kTile;
}

// The line of tiles that the ranges cut: every sequence with keys counts kLead tiles more, at its start.
template <typename L>
__device__ __forceinline__ int cost_of(const LatentDecodeParams &p, int b) {
    const int t = tiles_of<L>(p, b);
    return t > 0 ? t + L::kLead : 0;
}

// A walk over the tiles of a range.
template <typename L>
struct Walk {
    int b, t, keys, nt;  // tile t of the nt tiles of sequence b
    __device__ void at(const LatentDecodeParams &p, int b0, int t0) {
        b = b0;
        t = t0;
        keys = keys_of(p, b);
        nt = (keys + L::kTile - 1) / L::kTile;
    }
    __device__ void next(const LatentDecodeParams &p) {  // only while another tile follows
        if (++t < nt) return;
        do at(p, b + 1, 0);
        while (nt == 0 && b + 1 < p.num_seqs);
    }
};

template <int NCOL, bool FP8, int TILE>
__global__ void __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap ropemap,
                         const LatentDecodeParams p) {
    using L = Layout<NCOL, FP8, TILE>;
    constexpr int kStages = L::kStages, kTile = L::kTile, kTileBlocks = L::kTileBlocks, kTmaBlocks = L::kTmaBlocks,
                  kGroups = L::kGroups;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x / p.col_tiles, ct = blockIdx.x % p.col_tiles;
    const int cols = p.heads * p.q_per_seq;
    const int c0 = ct * p.cols_per_tile, nc = min(p.cols_per_tile, cols - c0);

    if (tid == 0) {
        prefetch_tensormap(&kvmap);
        if (FP8) prefetch_tensormap(&ropemap);
    }
    if (sbase & 1023u) {  // operands need the 1 KB swizzle alignment
        griddep_wait();
        if (tid == 0) atomicOr(p.status, kStatusTimeout);
        if (tid == 0 && ct == 0) p.record[range] = make_int2(0, 0);
        return;
    }
    auto bar = [&](int i) { return sbase + L::kBar + 8 * i; };
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + L::kAbort);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmemSlot);
    int64_t *plan = reinterpret_cast<int64_t *>(smem + L::kPlan);
    unsigned long long *first_tile = reinterpret_cast<unsigned long long *>(plan + 16), *tile_count = first_tile + 1;
    if (tid == 0) {
        for (int i = 0; i < L::kNumBars; ++i)
            mbar_init(bar(i), i < L::kBarKvEmpty ? kTmaBlocks + 2
                              : (i >= L::kBarSEmpty && i < L::kBarPvDone) || i == L::kBarQFull ? kSoftWarps : 1);
        *abort_flag = 0u;
        *reinterpret_cast<uint2 *>(smem + L::kDead) = make_uint2(0u, 0u);
        *first_tile = ~0ull;
        *tile_count = 0;
        fence_mbar_init();
    }
    longlong2 *q_at = reinterpret_cast<longlong2 *>(smem + L::kQAt);
    if (tid < nc) {
        const int i = (c0 + tid) / p.heads, h = c0 + tid - i * p.heads;
        q_at[tid] = make_longlong2(i * p.ql_row + h * p.ql_head, i * p.qr_row + h * p.qr_head);
    }
    if (warp == kScoreWarp) {  // (no other kernel's CTA waits for ours: the columns come free)
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    // While the kernel before us drains: the lengths, tables and queries on their way into L2 (a prefetch reads
    // nothing: what that kernel still writes to them is written there), each CTA a share.
    {
        const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + tid, all = static_cast<int64_t>(gridDim.x) * kThreads;
        const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.q_per_seq * p.heads;
        const int64_t tables = static_cast<int64_t>(p.num_seqs) * p.max_blocks;
        if (id * 32 < p.num_seqs) prefetch_l2(p.context_lens + id * 32);
        if (id * 32 < tables) prefetch_l2(p.block_tables + id * 32);
        for (int64_t k = id; k < rows * 9 && k < 4 * all; k += all) {  // 8 lines of latent part and one of rotated a row
            const int64_t r = k / 9, line = k - 9 * r, qr = r / p.heads, h = r - qr * p.heads;
            prefetch_l2(line < 8 ? static_cast<const uint16_t *>(p.q_latent) + qr * p.ql_row + h * p.ql_head + line * 64
                                 : static_cast<const uint16_t *>(p.q_rope) + qr * p.qr_row + h * p.qr_head);
        }
    }
    griddep_wait();  // the producers of q and of the cache before us on the stream

    // ---- the range: total tiles, then where tile `start` lies ----
    const int seg = (p.num_seqs + kThreads - 1) / kThreads;
    const int b_lo = min(p.num_seqs, tid * seg), b_hi = min(p.num_seqs, b_lo + seg);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += cost_of<L>(p, b);
    int64_t upto = mine;  // inclusive prefix
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += o;
    }
    if (lane == 31) plan[warp] = upto;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += plan[w];
        total += plan[w];
    }
    upto += before;
    // Of few and short sequences not every SM takes a range: a part costs about as much in the epilogue and the merge as an
    // eighth of a tile per part of its sequence, so sqrt(8 tiles sequences) ranges are least (one sequence of 4000 tokens, 64
    // heads: 129 ranges 29.2 us, 32 17.7; 8000: 35.2, 20.0; two of 8000: 27.4, 20.8); up to 24 tiles a sequence each has its own.
    const int64_t few = 24 * static_cast<int64_t>(p.num_seqs);
    const int64_t best = static_cast<int64_t>(sqrtf(8.f * static_cast<float>(total) * static_cast<float>(p.num_seqs)));
    const int64_t ranges = min(static_cast<int64_t>(p.ranges), total <= few ? total : max(few, best));
    auto cut = [&](int r) -> int64_t {  // r total / ranges (64-bit division only where 32 bits do not hold it)
        if (r > ranges || ranges == 0) return 0;
        if (total < (1 << 24)) return static_cast<uint32_t>(r) * static_cast<uint32_t>(total) / static_cast<uint32_t>(ranges);
        return r * total / ranges;
    };
    const int64_t start = range < ranges ? cut(range) : 0, stop = range < ranges ? cut(range + 1) : 0;
    // The tiles in [start, stop), by the threads whose sequences lie there (a range may hold none, when it falls
    // into a lead): how many, and the first one.
    int64_t tiles = 0;
    if (upto - mine < stop && start < upto) {
        int64_t acc = upto - mine;
        for (int b = b_lo; b < b_hi && acc < stop; ++b) {
            const int t = tiles_of<L>(p, b);
            if (t == 0) continue;
            const int64_t lo = max(static_cast<int64_t>(0), start - acc - L::kLead);
            const int64_t hi = min(static_cast<int64_t>(t), stop - acc - L::kLead);
            if (hi > lo) {
                tiles += hi - lo;
                atomicMin(first_tile, (static_cast<unsigned long long>(b) << 32) | lo);
            }
            acc += t + L::kLead;
        }
    }
    if (tiles > 0) atomicAdd(tile_count, static_cast<unsigned long long>(tiles));
    // Sequences without keys get zero rows, and every length is checked, shared out over the ranges.
    auto empty_sequences = [&](int thread, int threads) {
        for (int b = range; b < p.num_seqs; b += p.ranges) {
            const int ctx = __ldg(p.context_lens + b);
            if (thread == 0 && ct == 0) {
                uint32_t st = ctx < 1 || ctx > p.max_blocks * kBlockSize ? kStatusBadContextLen : 0u;
                if (ctx >= 1 && ctx < p.q_per_seq) st |= kStatusBadQLen;
                if (st) atomicOr(p.status, st);
            }
            if (keys_of(p, b) == 0) {
                const size_t at = (static_cast<size_t>(b) * cols + c0) * kLatentDim * (p.out_bf16 ? 2 : 4);
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + at);
                for (int i = thread; i < nc * (p.out_bf16 ? 64 : 128); i += threads) o[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int n = static_cast<int>(*tile_count);
    const int b0 = static_cast<int>(*first_tile >> 32), t0 = static_cast<int>(*first_tile & 0xffffffffu);
    if (tid == 0 && ct == 0) p.record[range] = make_int2(0, 0);  // (its last piece may write it below)
    const uint32_t tmem = *tmem_slot;
    if (n == 0) {
        empty_sequences(tid, kThreads);
        if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
        return;
    }

    // A warp's bounded wait; it gives up soon after another role did.  The timer and the flag are
    // read only every 64 tries: a read of %globaltimer between two tries delays the waiter by
    // several hundred cycles.
    // (Each lane may name a barrier of its own: one wait for several costs what one does.)
    auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool {
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

    // The pool passes through L2 once (column tiles of one range read it at about the same time): its lines go first.
    const uint64_t policy = l2_evict_first();

    if (warp == kProducerWarp) {
        // ---------------- TMA producer: lane j copies block j of a tile ----------------
        Walk<L> w;
        w.at(p, b0, t0);
        auto block_id = [&]() -> int {  // -1: past the context, or an invalid id (never copied)
            const int jb = w.t * kTileBlocks + lane;
            if (lane >= kTileBlocks || jb * kBlockSize >= w.keys) return -1;
            const int id = __ldg(p.block_tables + static_cast<size_t>(w.b) * p.max_blocks + jb);
            return static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks) ? id : -1;
        };
        int id = block_id();
        for (int i = 0; i < n; ++i) {
            const int cur = id;
            if (i + 1 < n) {
                w.next(p);
                id = block_id();
            }
            const int st = i % kStages;
            bool ok = true;
#pragma unroll
            for (int j = 0; j < kTmaBlocks; ++j) {  // P V frees a stage block by block
                if (i >= kStages) ok = ok && warp_wait(bar(L::kBarKvEmpty + st * kTileBlocks + j), ((i / kStages) - 1) & 1);
                if (ok && lane == j) {
                    const uint32_t full = bar(L::kBarKvFull + st), stage = sbase + L::kKv + st * L::kStage;
                    mbar_arrive_expect_tx(full, cur >= 0 ? L::kBlock + L::kRopeBlock : 0);
                    if (cur >= 0) {
                        tma_load_5d(stage + j * L::kBlock, &kvmap, full, 0, 0, 0, 0, cur, policy);
                        if constexpr (FP8)
                            tma_load_3d(stage + kTileBlocks * L::kBlock + j * L::kRopeBlock, &ropemap, full, 0, 0, cur);
                    }
                }
            }
            if (!ok) break;
            // FP8: the next tile on its way into L2 while its place is taken (98.4 -> 97.4 us on the verify of 64 columns;
            // a bf16 ring is bound by HBM: no gain).
            if (FP8 && i + 1 < n && lane < kTileBlocks && id >= 0) {
                bulk_prefetch_l2(static_cast<const uint8_t *>(p.cache) + static_cast<size_t>(id) * L::kBlock, L::kBlock);
                if constexpr (FP8)
                    bulk_prefetch_l2(static_cast<const uint8_t *>(p.rope_cache) + static_cast<size_t>(id) * L::kRopeBlock, L::kRopeBlock);
            }
            __syncwarp();
        }
    } else if (warp >= kLoadWarp) {
        // ---------------- copying warps: the blocks from kTmaBlocks on of every second tile ----------------
        // (A pair that waits for its place is at most one use of the stage ahead of the barrier, whose parity tells no
        // more: its tile before has landed, so P V of the tile two uses back is done.  More pairs need as many stages.)
        static_assert(kStages >= 2, "a stage a pair of copying warps");
        const int g = (warp - kLoadWarp) >> 1, t = ((warp - kLoadWarp) & 1) * 32 + lane;  // 64 threads a tile
        // Where the 16-byte vectors t + 64 k of 8 slots (72 a slot, or 32) go; the second 8 slots follow kGroup
        // bytes on.
        constexpr int kVec = FP8 ? 32 : 72, kSteps = kVec * 8 / 64;
        uint32_t to[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int v = t + 64 * k, r = v / kVec, c = v - r * kVec;
            to[k] = (c >> 3) * 1024 + r * 128 + (((c & 7) ^ r) << 4);
        }
        Walk<L> w;
        w.at(p, b0, t0);
        if (g == 1 && n > 1) w.next(p);
        auto block_id = [&]() -> int {  // lane j: block j's id, read while the tile before is copied
            const int jb = w.t * kTileBlocks + lane;
            return lane < kTileBlocks && jb * kBlockSize < w.keys
                       ? __ldg(p.block_tables + static_cast<size_t>(w.b) * p.max_blocks + jb)
                       : -1;
        };
        int id_next = block_id();
        for (int i = g; i < n; i += 2) {
            const int st = i % kStages;
            const bool exists = lane < kTileBlocks && (w.t * kTileBlocks + lane) * kBlockSize < w.keys;
            const int id = static_cast<unsigned>(id_next) < static_cast<unsigned>(p.num_blocks) ? id_next : -1;
            const uint32_t bad = __ballot_sync(0xffffffffu, exists && id < 0);
            int4 info = make_int4(min(w.keys - w.t * kTile, kMaxLeft) | static_cast<int>(bad << 24), w.nt - 1 - w.t, w.b, w.b);
            float sc = 1.f;
            if constexpr (FP8) {
                // Key t's scale, once for all columns (the stage's last reader, softmax, is behind every one of its
                // blocks' P V): 1 for a slot without a key, whose scale may be anything.
                const int blk = __shfl_sync(0xffffffffu, id, t >> 4);
                if (blk >= 0 && w.t * kTile + t < w.keys) sc = __ldg(p.cache_scale + static_cast<size_t>(blk) * kBlockSize + (t & 15));
                // A slot of a cleared pool has scale 0, whose logarithm and inverse are infinite: the least that a write
                // makes instead (NaN stays).
                if (fabsf(sc) < kLeastScale) sc = kLeastScale;
            }
            bool ok = true;
#pragma unroll
            for (int j = kTmaBlocks; j < kTileBlocks; ++j) {
                const int blk = __shfl_sync(0xffffffffu, id, j);
                if (i >= kStages) ok = ok && warp_wait(bar(L::kBarKvEmpty + st * kTileBlocks + j), ((i / kStages) - 1) & 1);
                if (ok && blk >= 0) {
                    const uint32_t stage = sbase + L::kKv + st * L::kStage, dst = stage + j * L::kBlock;
                    const uint8_t *src = static_cast<const uint8_t *>(p.cache) + static_cast<size_t>(blk) * L::kBlock + 16 * t;
#pragma unroll
                    for (int k = 0; k < 2 * kSteps; ++k)
                        cp_async_16(dst + (k / kSteps) * L::kGroup + to[k % kSteps], src + 1024 * k, policy);
                    if constexpr (FP8) {  // 8 vectors of rotated key a slot, and the 16 scales
                        const uint8_t *rope = static_cast<const uint8_t *>(p.rope_cache) + static_cast<size_t>(blk) * L::kRopeBlock + 16 * t;
                        const uint32_t rdst = stage + kTileBlocks * L::kBlock + j * L::kRopeBlock + (t >> 3) * 128 +
                                              (((t & 7) ^ (t >> 3)) << 4);
                        cp_async_16(rdst, rope);
                        cp_async_16(rdst + 1024, rope + 1024);
                    }
                }
            }
            if (!ok) break;
            if constexpr (FP8) {
                float *at = reinterpret_cast<float *>(smem + L::kScale) + st * 3 * kTile + t;
                at[0] = sc;
                at[kTile] = __log2f(sc);
                at[2 * kTile] = __fdividef(L::kUnit, sc);
            }
            if (i + 1 < n) w.next(p);
            info.w = w.b;
            if (i + 2 < n) w.next(p);
            id_next = block_id();
            if (t == 0) *reinterpret_cast<int4 *>(smem + L::kInfo + 16 * st) = info;
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();  // generic writes -> the tensor core
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kBarKvFull + st));
        }
    } else if (warp == kScoreWarp) {
        // ---------------- S = Q K^T ----------------
        // (Both tensor warps run their loop whole, on warp-uniform values, and one elected lane
        // issues: the descriptors stay in uniform registers.  Issued from a one-lane branch an
        // MMA took 74-98 cycles to issue, against 36-52 in the pipe.)
        Walk<L> w;
        w.at(p, b0, t0);
        const uint64_t q_desc = sw128_desc(sbase + L::kQ, 16, 1024);
        const uint64_t k_desc = sw128_desc(sbase + L::kKv, 16, L::kGroup);
        const uint64_t r_desc = sw128_desc(sbase + L::kKv + kTileBlocks * L::kBlock, 16, 1024);
        int pieces = 0;
        for (int i = 0; i < n; ++i) {
            const int st = i % kStages;
            // The tile; S's buffer, free after softmax (i - 2) has read it; a sequence's first tile: its Q.
            const bool of_s = lane == 1 && i >= 2, of_q = lane == 2 && (i == 0 || w.t == 0);
            if (!warp_wait(bar(of_s   ? L::kBarSEmpty + (i & 1)
                               : of_q ? L::kBarQFull
                                      : L::kBarKvFull + st),
                           (of_s ? (i >> 1) - 1 : of_q ? pieces : i / kStages) & 1))
                break;
            pieces += i == 0 || w.t == 0;
            tc_fence_after();
            const uint32_t d = tmem + kTmemS + L::kScoreCols * (i & 1);
            const uint64_t kd = k_desc + static_cast<uint32_t>(st) * (L::kStage >> 4);
            const uint64_t rd = r_desc + static_cast<uint32_t>(st) * (L::kStage >> 4);
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < (FP8 ? 4 : 8); ++c)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t qd = q_desc + ((c * L::kQChunk + kk * 32) >> 4), k = kd + ((c * 1024 + kk * 32) >> 4);
                        if constexpr (FP8)  // heads and remainders against the same codes
                            umma_f8(d, qd, k, idesc(L::kQRows, kTile, false, Kind::kE4m3), c + kk > 0);
                        else
                            umma_bf16(d, qd, k, idesc(64, kTile, false), c + kk > 0);
                    }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_bf16(FP8 ? d + 64 : d, q_desc + ((L::kQRope - L::kQ + kk * 32) >> 4),
                              (FP8 ? rd : kd + (8 * 1024 >> 4)) + ((kk * 32) >> 4), idesc(64, kTile, false), !FP8 || kk > 0);
                umma_commit(bar(L::kBarSFull + (i & 1)));
            }
            __syncwarp();
            if (i + 1 < n) w.next(p);
        }
    } else if (warp == kValueWarp) {
        // ---------------- O^T += V^T P^T ----------------
        Walk<L> w;
        w.at(p, b0, t0);
        const uint64_t v_desc = sw128_desc(sbase + L::kKv, 1024, L::kGroup);
        const uint64_t p_desc = sw128_desc(sbase + L::kP, 16, 1024);
        for (int i = 0; i < n; ++i) {
            const int st = i % kStages;
            const uint32_t keep = i > 0 && w.t > 0;  // a piece's first P V overwrites O
            if (!warp_wait(bar(L::kBarPFull + (i & 1)), (i >> 1) & 1)) break;
            tc_fence_after();
            const uint64_t vd = v_desc + static_cast<uint32_t>(st) * (L::kStage >> 4);
            const uint64_t pd = p_desc + static_cast<uint32_t>(i & 1) * (L::kPBuf >> 4);
            if (elect_one()) {
                if constexpr (!FP8) {
#pragma unroll
                    for (int ks = 0; ks < kTileBlocks; ++ks) {
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            umma_bf16(tmem + m * NCOL, vd + ((ks * L::kBlock + m * 2048) >> 4), pd + ((ks * 32) >> 4),
                                      idesc(128, NCOL, true), ks > 0 ? 1u : keep);
                        umma_commit(bar(L::kBarKvEmpty + st * kTileBlocks + ks));
                    }
                } else {  // 32 keys a step; a weight's three codes against the same key
                    const uint64_t p3 = p_desc + ((L::kP3 - L::kP + static_cast<uint32_t>(i & 1) * 64) >> 4);
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint64_t v = vd + ((ks * 2 * L::kBlock + m * 1024) >> 4), w8 = pd + ((ks * 32) >> 4);
                            const uint32_t o = tmem + m * L::kOCols;
                            umma_f8(o, v, w8, idesc(128, L::kOCols, true, Kind::kE4m3E5m2), ks > 0 ? 1u : keep);
                            if constexpr (!L::kStack) umma_f8(o, v, w8 + (64 >> 4), idesc(128, NCOL, true, Kind::kE4m3E5m2), 1u);
                            umma_f8(o, v, p3 + ((ks * 32) >> 4), idesc(128, NCOL, true, Kind::kE4m3E5m2), 1u);
                        }
                        umma_commit(bar(L::kBarKvEmpty + st * kTileBlocks + 2 * ks));
                        umma_commit(bar(L::kBarKvEmpty + st * kTileBlocks + 2 * ks + 1));
                    }
                }
                umma_commit(bar(L::kBarPvDone + (i & 1)));
            }
            __syncwarp();
            if (i + 1 < n) w.next(p);
        }
    } else {
        // ---------------- softmax, rescaling and epilogue: 8 warps ----------------
        const int quarter = warp & 3, half = warp >> 2;
        // The 16-lane load spreads a quarter's rows over the warp: a thread holds rows lane / 4 and (64 columns)
        // lane / 4 + 8 of it, of each 8 keys of its half tile (columns 8 j + 2 (lane % 4) + 0, 1).
        constexpr int kR = L::kRowsPerThread;
        const int col0 = quarter * L::kPerQuarter + (lane >> 2);  // the column of row k is col0 + 8 k
        const bool live = (lane >> 2) < L::kPerQuarter;
        const bool has = live && (lane & 3) == 0;  // speaks for its columns
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        int q_row[kR];
#pragma unroll
        for (int k = 0; k < kR; ++k) q_row[k] = col0 + 8 * k < nc ? (c0 + col0 + 8 * k) / p.heads : p.q_per_seq - 1;
        // P: where this thread's pair of keys of 8-key group j goes, p_at[.] (+ 1024 for row k = 1).  bf16: a pair is 4
        // bytes, group j the 16-byte chunk 4 half + j.  FP8: 2 bytes, chunk 2 half + j / 2, second codes 64 bytes on or
        // (stacked) NCOL rows, third codes in rows of their own.
        auto p_at = [&](int j) {
            const int v = FP8 ? 2 * half + (j >> 1) : kGroups * half + j;
            return sbase + L::kP + col0 * 128 + ((v ^ (col0 & 7)) << 4) + (FP8 ? 8 * (j & 1) + 2 * (lane & 3) : 4 * (lane & 3));
        };
        float *xch = reinterpret_cast<float *>(smem + L::kXch);
        float *alpha_s = reinterpret_cast<float *>(smem + L::kAlpha);
        auto soft_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); };
        bool alive = true;

        // Sequence b's Q, a row a warp, zeros behind the last one, in the operand's swizzle.  FP8: the
        // latent part times a power of two that takes its largest value into (224, 448], as E4M3
        // heads and remainders (a bf16 value has 8 bits, two codes hold 4 each: exact down to steps
        // of 2^-9); the factor that undoes it in shared memory, in two buffers by the parity of the tile that
        // reads it, the piece's first: where a piece is one tile a warp writes the next piece's factors while another still
        // has to read this one's.  (A write to the same buffer comes two tiles on at least, behind the barrier of a tile.)
        float *qf_s = reinterpret_cast<float *>(smem + L::kQf);
        auto load_q = [&](int b, int first_tile) {
            const uint16_t *ql0 = static_cast<const uint16_t *>(p.q_latent) + static_cast<int64_t>(b) * p.q_per_seq * p.ql_row;
            const uint16_t *qp0 = static_cast<const uint16_t *>(p.q_rope) + static_cast<int64_t>(b) * p.q_per_seq * p.qr_row;
            auto q_of = [&](int r, const uint16_t *&ql, const uint16_t *&qp) {  // (r < nc)
                const longlong2 to = q_at[r];
                ql = ql0 + to.x;
                qp = qp0 + to.y;
            };
            // FP8: a row's data, read while the row before is converted (the loop stays rolled: unrolled, its code took
            // longer to fetch than to run).
            uint4 a, d, rope;
            auto fetch = [&](int r) {
                a = d = rope = make_uint4(0u, 0u, 0u, 0u);
                if (r < nc) {
                    const uint16_t *ql, *qp;
                    q_of(r, ql, qp);
                    a = __ldg(reinterpret_cast<const uint4 *>(ql) + 2 * lane);
                    d = __ldg(reinterpret_cast<const uint4 *>(ql) + 2 * lane + 1);
                    if (lane < 8) rope = __ldg(reinterpret_cast<const uint4 *>(qp) + lane);
                }
            };
            if constexpr (FP8) fetch(warp);
#pragma unroll 1
            for (int r = warp; r < NCOL; r += kSoftWarps) {
                const int rq = r / L::kPerQuarter * 16 + r % L::kPerQuarter;
                auto at = [&](int chunk, int v) { return sbase + L::kQ + chunk * L::kQChunk + rq * 128 + ((v ^ (rq & 7)) << 4); };
                constexpr uint32_t kRest = L::kQRows == 128 ? 16 * 128 : 8 * 128;  // from a head to its remainder
                if constexpr (!FP8) {
                    const uint16_t *ql = ql0, *qp = qp0;
                    if (r < nc) q_of(r, ql, qp);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const int v = lane + 32 * k;
                        if (v >= 72) continue;
                        if (r < nc)
                            cp_async_16(at(v >> 3, v & 7), v < 64 ? ql + v * 8 : qp + (v - 64) * 8);
                        else
                            sts128(at(v >> 3, v & 7), make_uint4(0u, 0u, 0u, 0u));
                    }
                } else {
                    const uint32_t u[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
                    const uint4 rotated = rope;
                    if (r + kSoftWarps < NCOL) fetch(r + kSoftWarps);
                    float v[16], most = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        v[2 * k] = bf16_lo(u[k]), v[2 * k + 1] = bf16_hi(u[k]);
                        most = fmax3(most, fabsf(v[2 * k]), fabsf(v[2 * k + 1]));
                    }
                    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));  // (none is negative)
                    // most = f 2^e, 1 <= f < 2: times 2^(8 - e), or 2^(7 - e) when f 2^8 passes 448 (both exponents
                    // kept within fp32's; an all-zero row keeps factor 1).
                    const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;
                    int lift = most > 0.f ? ((__float_as_uint(most) & 0x7fffffu) > 0x600000u ? 7 : 8) - e : 0;
                    lift = max(-126, min(126, lift));
                    const float up = __uint_as_float(static_cast<uint32_t>(lift + 127) << 23);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t h0 = f32x2_to_e4m3x2(v[4 * k] * up, v[4 * k + 1] * up);
                        const uint32_t h1 = f32x2_to_e4m3x2(v[4 * k + 2] * up, v[4 * k + 3] * up);
                        const float2 f0 = unpack_f16x2(e4m3x2_to_f16x2(h0)), f1 = unpack_f16x2(e4m3x2_to_f16x2(h1));
                        hi[k] = h0 | h1 << 16;
                        lo[k] = f32x2_to_e4m3x2(v[4 * k] * up - f0.x, v[4 * k + 1] * up - f0.y) |
                                f32x2_to_e4m3x2(v[4 * k + 2] * up - f1.x, v[4 * k + 3] * up - f1.y) << 16;
                    }
                    const uint32_t head = at(lane >> 3, lane & 7) + (L::kQRows == 128 ? r / 16 * (16 * 128) : 0);
                    sts128(head, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                    sts128(head + kRest, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                    if (lane < 8) sts128(at(4, lane), rotated);
                    // (E4M3 has no infinity: a row that holds one scores NaN.)
                    if (lane == 0) qf_s[64 * (first_tile & 1) + r] = __uint_as_float(most == INFINITY ? 0x7fffffffu : static_cast<uint32_t>(127 - lift) << 23);
                }
            }
        };
        auto publish_q = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kBarQFull));
        };

        load_q(b0, 0);
        empty_sequences(tid, kSoftThreads);
        publish_q();
        if constexpr (FP8) soft_sync();  // the factors of Q's rows are written
        float q_scale[kR] = {};          // FP8: those of this thread's columns, times the softmax scale
        float m_ref[kR];
        float2 l[kR];
        bool piece_mid = t0 > 0;  // the piece does not hold its sequence's first key
        bool first = true;        // of its piece
        for (int i = 0; i < n; ++i) {
            // FP8: c_j = code s_j, so the score is s_j <q, code_j> + <q_rope, r_j>, and the weight that multiplies the
            // codes is s_j 2^score = 2^(score + log2 s_j); the sum l takes it times 1 / s_j (in kUnit).
            const uint32_t sc_at = sbase + L::kScale + ((i % kStages) * 3 * kTile + kTile / 2 * half + 2 * (lane & 3)) * 4;
            // S; the tile's record and scales; P's buffer, free after P V (i - 2).
            const bool of_kv = lane == 1, of_p = lane == 2 && i >= 2;
            alive = alive && warp_wait(bar(of_kv  ? L::kBarKvFull + i % kStages
                                           : of_p ? L::kBarPvDone + (i & 1)
                                                  : L::kBarSFull + (i & 1)),
                                       (of_kv ? i / kStages : of_p ? (i >> 1) - 1 : i >> 1) & 1);
            const int4 info = alive ? lds_i32x4(sbase + L::kInfo + 16 * (i % kStages)) : make_int4(0, 0, 0, 0);
            const int left = info.x & 0xffffff;  // keys of the tile that exist (may pass its size)
            const uint32_t bad = static_cast<uint32_t>(info.x) >> 24;  // its blocks with an invalid id: flagged, their keys masked
            const bool ends = info.y == 0, last = i == n - 1 || ends;
            if (bad && tid == 0) atomicOr(p.status, kStatusBadBlockId);
            if (first) {
#pragma unroll
                for (int k = 0; k < kR; ++k) {
                    m_ref[k] = -INFINITY;
                    l[k] = make_float2(0.f, 0.f);
                    if constexpr (FP8) q_scale[k] = live ? qf_s[64 * (i & 1) + col0 + 8 * k] * p.scale_log2 : 0.f;
                }
            }
            float2 x[kR][kGroups];  // [k][j]: row k, keys kTile / 2 half + 8 j + 2 (lane % 4) + 0, 1
            float mx[kR];
#pragma unroll
            for (int k = 0; k < kR; ++k) mx[k] = -INFINITY;
            if (alive) {
                tc_fence_after();
                uint32_t v[4 * kGroups];
                const uint32_t s_at = tmem + lanes + kTmemS + L::kScoreCols * (i & 1) + kTile / 2 * half;
                const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
                auto pair = [](const uint32_t(&r)[4 * kGroups], int j, int k) {
                    return make_float2(__uint_as_float(r[4 * j + 2 * k]), __uint_as_float(r[4 * j + 2 * k + 1]));
                };
                if constexpr (!FP8) {
                    if constexpr (kGroups == 4)
                        tmem_ld_16x256b_x4(s_at, v);
                    else
                        tmem_ld_16x256b_x2(s_at, v);
#pragma unroll
                    for (int j = 0; j < kGroups; ++j)
#pragma unroll
                        for (int k = 0; k < kR; ++k) x[k][j] = fmul2(pair(v, j, k), sl2);
                } else {
                    uint32_t u[16];
                    if constexpr (L::kQRows == 128) {  // rows 32 q + 16 ..: the remainders
                        tmem_ld_16x256b_x4_pair(s_at, v, s_at + (16u << 16), u);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(u[e]));
                        tmem_ld_16x256b_x4(s_at + 64, u);
                    } else {
                        tmem_ld_16x256b_x4_pair(s_at, v, s_at + 64, u);
                    }
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) {
                        const float2 sc = lds_f32x2(sc_at + 32 * j), lg = lds_f32x2(sc_at + kTile * 4 + 32 * j);
#pragma unroll
                        for (int k = 0; k < kR; ++k)
                            x[k][j] = ffma2(L::kStack ? fadd2(pair(v, j, 0), pair(v, j, 1)) : pair(v, j, k), fmul2(sc, make_float2(q_scale[k], q_scale[k])),
                                            ffma2(pair(u, j, k), sl2, lg));
                    }
                }
                tc_fence_before();
                // Row q_row sees keys up to keys - q_per_seq + q_row; bad blocks see none.
                if (left - p.q_per_seq + 1 < kTile || bad) {
#pragma unroll
                    for (int j = 0; j < kGroups; ++j)
#pragma unroll
                        for (int k = 0; k < kR; ++k) {
                            const int key = kTile / 2 * half + 8 * j + 2 * (lane & 3), end = left - p.q_per_seq + q_row[k];
                            const bool hide = (bad >> (key >> 4)) & 1u;
                            if (hide || key > end) x[k][j].x = -INFINITY;
                            if (hide || key + 1 > end) x[k][j].y = -INFINITY;
                        }
                }
#pragma unroll
                for (int k = 0; k < kR; ++k) {
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) mx[k] = fmax3(mx[k], x[k][j].x, x[k][j].y);
                    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
                    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
                }
            }
            __syncwarp();
            if (alive && lane == 0) mbar_arrive(bar(L::kBarSEmpty + (i & 1)));
            // The last S of a piece is complete: its Q can make way for the next sequence's.
            const bool more = last && i + 1 < n;
            if (more && alive) load_q(info.w, i + 1);

            float *xm = xch + (i & 1) * 128;
            bool pass = false;
#pragma unroll
            for (int k = 0; k < kR; ++k) {
                if (has) xm[half * 64 + col0 + 8 * k] = mx[k];
                pass = pass || (live && mx[k] > m_ref[k] + L::kRaise);
            }
            // A warp whose wait ran out does not know the tile: all of them leave here.
            volatile uint32_t *dead = reinterpret_cast<volatile uint32_t *>(smem + L::kDead) + (i & 1);
            if (!alive && lane == 0) *dead = 1u;
            if (bar_red_or(1, kSoftThreads, pass || !alive)) {
                if (*dead) break;
                if (live) {
#pragma unroll
                    for (int k = 0; k < kR; ++k) {
                        float alpha = 1.f;
                        const float mt = fmaxf(xm[col0 + 8 * k], xm[64 + col0 + 8 * k]);
                        if (mt > m_ref[k] + L::kRaise) {
                            alpha = fast_exp2(m_ref[k] - mt);  // 0 from -inf
                            m_ref[k] = mt;
                            l[k] = fmul2(l[k], make_float2(alpha, alpha));
                        }
                        if (has && half == 0) alpha_s[col0 + 8 * k] = alpha;
                    }
                }
                if (!first) {  // (the first P V of a piece overwrites O)
                    soft_sync();
                    alive = alive && warp_wait(bar(L::kBarPvDone + ((i - 1) & 1)), ((i - 1) >> 1) & 1);
                    if (alive) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 2 * L::kOCols; c += 16) {  // dim tiles 2 half, 2 half + 1
                            uint32_t o[16];
                            const uint32_t at = tmem + lanes + 2 * half * L::kOCols + c;
                            tmem_ld_32x32b_x16(at, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha_s[(c + e) % NCOL]);
                            tmem_st_32x32b_x16(at, o);
                        }
                        tmem_wait_st();
                    }
                }
            }
            // Weights, rounded to bf16 (relative 2^-8; l adds what P V will read), or to three E5M2 codes by way of fp16
            // (2^-11; each code is off by 2^-3 of what it rounds, so three by 2^-9, or by 2^-17; l adds the unrounded
            // weights).
            uint32_t pk[kR][kGroups], pk3[kR][FP8 ? kGroups : 1];
#pragma unroll
            for (int k = 0; k < kR; ++k) {
                const float mu = m_ref[k] == -INFINITY ? 0.f : m_ref[k] - L::kLift;
#pragma unroll
                for (int j = 0; j < kGroups; ++j) {
                    const float2 y = fadd2(x[k][j], make_float2(-mu, -mu));
                    const float2 w2 = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    if constexpr (FP8) {
                        l[k] = ffma2(w2, lds_f32x2(sc_at + 2 * kTile * 4 + 32 * j), l[k]);
                        e5m2_codes(pack_f16x2(w2.x, w2.y), pk[k][j], pk3[k][j]);
                    } else {
                        pk[k][j] = pack_bf16x2(w2.x, w2.y);
                        l[k] = fadd2(l[k], make_float2(bf16_lo(pk[k][j]), bf16_hi(pk[k][j])));
                    }
                }
            }
            if (alive) {
                const uint32_t buf = (i & 1) * L::kPBuf;
                if (live) {
#pragma unroll
                    for (int j = 0; j < kGroups; ++j)
#pragma unroll
                        for (int k = 0; k < kR; ++k) {
                            const uint32_t at = (L::kPHalf ? p_at(j) ^ buf : p_at(j) + buf) + 1024 * k;
                            if constexpr (FP8) {
                                sts16(at, pk[k][j]);
                                sts16(L::kStack ? at + NCOL * 128 : at ^ 64u, pk[k][j] >> 16);
                                sts16((p_at(j) ^ ((i & 1) * 64u)) + (L::kP3 - L::kP) + 1024 * k, pk3[k][j]);
                            } else {
                                sts32(at, pk[k][j]);
                            }
                        }
                }
                // Rows that no key fills (past the context, of an invalid block) hold whatever was there:
                // their weights are 0, their values have to be finite.
                if (left < kTile || bad) {
                    alive = warp_wait(bar(L::kBarKvFull + i % kStages), (i / kStages) & 1);
                    const uint32_t kv = sbase + L::kKv + (i % kStages) * L::kStage;
                    constexpr int kVec = FP8 ? 32 : 64;  // (all of a latent's 16-byte chunks: the swizzle is moot)
                    for (int idx = tid; alive && idx < kTile * kVec; idx += kSoftThreads) {
                        const int key = idx / kVec, v = idx % kVec;
                        if (key >= left || ((bad >> (key >> 4)) & 1u))
                            sts128(kv + (key >> 3) * L::kGroup + (v >> 3) * 1024 + (key & 7) * 128 + (v & 7) * 16,
                                   make_uint4(0u, 0u, 0u, 0u));
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
            }
            __syncwarp();
            if (alive && lane == 0) mbar_arrive(bar(L::kBarPFull + (i & 1)));
            if (more && alive) publish_q();

            if (last) {
                // ---- the piece's columns: whole sequences to out, parts to the workspace ----
                const bool whole = !piece_mid && ends;
                // (The merge's CTAs come now, when the SMs empty: launched at the start they crowd onto the first that do.)
                if (i == n - 1) griddep_launch_dependents();
                // Slot 0: the range's first piece when it starts inside its sequence; else slot 1.
                const size_t slot = (static_cast<size_t>(range) * 2 + (piece_mid ? 0 : 1)) * (p.col_tiles * p.cols_per_tile) + c0;
                soft_sync();  // the maxima have been read
#pragma unroll
                for (int k = 0; k < kR; ++k) {
                    float sum = l[k].x + l[k].y;
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    if (has) xch[half * 64 + col0 + 8 * k] = sum;
                }
                soft_sync();
                if (tid < NCOL) alpha_s[tid] = [&] {
                    const float sum = xch[tid] + xch[64 + tid];
                    return !whole ? 1.f : sum > 0.f ? L::kUnit / sum : sum;  // (0, or NaN: never a finite row from a sum that is none)
                }();
                if (tid == 0 && ct == 0 && !whole && !piece_mid) {
                    // The merge's record: this sequence begins here and ends in the range that holds its last tile,
                    // at `end - 1` on the line: the largest r with r total / ranges <= end - 1.
                    const int64_t end = stop + info.y;
                    const int last_range = static_cast<int>((end * ranges - 1) / total);
                    p.record[range] = make_int2(info.z, last_range - range + 1);
                }
                if (!whole && has && half == 0) {
#pragma unroll
                    for (int k = 0; k < kR; ++k) {
                        const int r = col0 + 8 * k;
                        if (r < nc) p.part_ml[slot + r] = make_float2(m_ref[k], xch[r] + xch[64 + r]);
                    }
                }
                soft_sync();
                alive = alive && warp_wait(bar(L::kBarPvDone + (i & 1)), (i >> 1) & 1);
                if (alive) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 2 * NCOL; c += 16) {
                        uint32_t o[16];
                        const uint32_t o_at = tmem + lanes + (2 * half + c / NCOL) * L::kOCols + c % NCOL;
                        tmem_ld_32x32b_x16(o_at, o);
                        if constexpr (L::kStack) {
                            uint32_t rest[16];
                            tmem_ld_32x32b_x16(o_at + NCOL, rest);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(rest[e]));
                        }
                        const int col = c % NCOL, dim = (2 * half + c / NCOL) * 128 + 32 * quarter + lane;
                        if (!whole) {
                            float *dst = p.part_o + (slot + col) * kLatentDim + dim;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (col + e < nc) dst[static_cast<size_t>(e) * kLatentDim] = __uint_as_float(o[e]) * L::kUnit;
                        } else if (p.out_bf16) {
                            // lanes 2 d and 2 d + 1 swap a value: each then stores two dims of one column
                            uint32_t *dst = static_cast<uint32_t *>(p.out) +
                                            ((static_cast<size_t>(info.z) * cols + c0 + col) * kLatentDim + (dim & ~1)) / 2;
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float a = __uint_as_float(o[e]) * alpha_s[col + e];
                                const float d = __uint_as_float(o[e + 1]) * alpha_s[col + e + 1];
                                const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : d, 1);
                                const int ce = e + (lane & 1);
                                if (col + ce < nc)
                                    dst[static_cast<size_t>(ce) * (kLatentDim / 2)] =
                                        lane & 1 ? pack_bf16x2(other, d) : pack_bf16x2(a, other);
                            }
                        } else {
                            float *dst = static_cast<float *>(p.out) + (static_cast<size_t>(info.z) * cols + c0 + col) * kLatentDim + dim;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (col + e < nc)
                                    dst[static_cast<size_t>(e) * kLatentDim] = __uint_as_float(o[e]) * alpha_s[col + e];
                        }
                    }
                    tc_fence_before();
                }
                piece_mid = false;
                soft_sync();  // the factors have been read
            }
            first = last;
        }
    }

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
    if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
}

// Folds the parts of the y-th split sequence, one column (of the x-th eight) a warp, 512 / z
// of its dims (z = 1 or 4).  Its parts are the last piece (slot 1) of the range in which it begins,
// which recorded it, and the first pieces (slot 0) of the ranges from there on.  Two round
// trips to L2: the records, then everything else.
constexpr int kMergeWarps = 8;
constexpr int kRecords = kLatentMaxRanges / 32;
constexpr int kMergeResident = 2 * 152;  // CTAs
template <int STEPS, int BATCH>  // steps of 32 lanes x 4 dims, batches of parts read at once
__global__ void __launch_bounds__(kMergeWarps * 32, BATCH > 2 ? 2 : 3) latent_merge_kernel(const LatentDecodeParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * kMergeWarps + warp;
    griddep_launch_dependents();
    griddep_wait();
    if (col >= p.heads * p.q_per_seq) return;
    // The y-th range in which a split sequence begins: {sequence, parts}.
    int first = -1, b = 0, parts = 0, seen = 0;
    int2 rec[kRecords];
#pragma unroll
    for (int k = 0; k < kRecords; ++k) rec[k] = 32 * k + lane < p.ranges ? p.record[32 * k + lane] : make_int2(0, 0);
#pragma unroll
    for (int k = 0; k < kRecords; ++k) {
        uint32_t mask = __ballot_sync(0xffffffffu, rec[k].y > 0);
        const int want = static_cast<int>(blockIdx.y) - seen;
        seen += __popc(mask);
        if (first < 0 && want < __popc(mask)) {
            for (int j = want; j > 0; --j) mask &= mask - 1;
            const int at = __ffs(mask) - 1;
            first = 32 * k + at;
            b = __shfl_sync(0xffffffffu, rec[k].x, at);
            parts = __shfl_sync(0xffffffffu, rec[k].y, at);
        }
    }
    if (first < 0) return;
    const size_t padded = static_cast<size_t>(p.col_tiles) * p.cols_per_tile;
    // Part k among the (range, slot, column) partials: slot 1 of that range, then slot 0 of those behind it.
    const size_t part0 = (static_cast<size_t>(first) * 2 + 1) * padded + col;
    const size_t part1 = static_cast<size_t>(first + 1) * 2 * padded + col;
    auto slot = [&](int k) { return k == 0 ? part0 : part1 + static_cast<size_t>(k - 1) * 2 * padded; };
    constexpr int kBatch = BATCH;
    float4 v[kBatch][STEPS], o[STEPS];
    const int lane4 = blockIdx.z * STEPS * 32 + lane;
    auto load = [&](int j) {
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const float4 *src = reinterpret_cast<const float4 *>(p.part_o + slot(j + e) * kLatentDim) + lane4;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) v[e][s] = j + e < parts ? src[32 * s] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    float2 ml[kRecords];
    float w[kRecords], m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kRecords; ++k)
        ml[k] = 32 * k + lane < parts ? p.part_ml[slot(32 * k + lane)] : make_float2(-INFINITY, 0.f);
    load(0);
#pragma unroll
    for (int k = 0; k < kRecords; ++k) m = fmaxf(m, ml[k].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
#pragma unroll
    for (int k = 0; k < kRecords; ++k) {
        w[k] = ml[k].x == -INFINITY ? 0.f : exp2f(ml[k].x - m);
        sum += w[k] * ml[k].y;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float inv = sum > 0.f ? 1.f / sum : sum;  // (0 or NaN)
#pragma unroll
    for (int s = 0; s < STEPS; ++s) o[s] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0;;) {
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            float wk = 0.f;  // weight of part j + e, kept by lane (j + e) % 32
#pragma unroll
            for (int k = 0; k < kRecords; ++k)
                if ((j + e) >> 5 == k) wk = w[k];
            wk = __shfl_sync(0xffffffffu, wk, (j + e) & 31);
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
                o[s].x += wk * v[e][s].x, o[s].y += wk * v[e][s].y, o[s].z += wk * v[e][s].z, o[s].w += wk * v[e][s].w;
        }
        j += kBatch;
        if (j >= parts) break;
        load(j);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const size_t at = (static_cast<size_t>(b) * p.heads * p.q_per_seq + col) * kLatentDim + 4 * (lane4 + 32 * s);
        if (p.out_bf16)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
                make_uint2(pack_bf16x2(o[s].x * inv, o[s].y * inv), pack_bf16x2(o[s].z * inv, o[s].w * inv));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
                make_float4(o[s].x * inv, o[s].y * inv, o[s].z * inv, o[s].w * inv);
    }
}

}  // namespace

// Keys a tile.  Over a bf16 pool Q and two tiles of 64 keys fill the shared memory, and a tile stays through S,
// softmax and P V: tiles of 32 keys in four stages are held shorter (8 x 32K tokens of 64 heads 70.9 -> 67.3 us,
// 128 heads 81.8 -> 77.3, the ragged batch of 32 heads 43.6 -> 41.9).  With up to 16 columns 64 keys halve the parts
// of a short context (one sequence of 1000 tokens 12.5 -> 10.4 us).
template <int NCOL, bool FP8>
constexpr int kTileOf = !FP8 && NCOL >= 32 ? 32 : 64;

template <int NCOL, bool FP8>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(latent_decode_kernel<NCOL, FP8, kTileOf<NCOL, FP8>>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Layout<NCOL, FP8, kTileOf<NCOL, FP8>>::kBytes));
}

cudaError_t latent_decode_prepare_device() {
    cudaError_t e = prepare_one<16, false>();
    if (e == cudaSuccess) e = prepare_one<32, false>();
    if (e == cudaSuccess) e = prepare_one<64, false>();
    if (e == cudaSuccess) e = prepare_one<16, true>();
    if (e == cudaSuccess) e = prepare_one<32, true>();
    if (e == cudaSuccess) e = prepare_one<64, true>();
    return e;
}

template <int NCOL, bool FP8>
cudaError_t launch_one(const LatentDecodeMaps &maps, const LatentDecodeParams &p, cudaStream_t stream) {
    return launch_pdl(latent_decode_kernel<NCOL, FP8, kTileOf<NCOL, FP8>>, dim3(p.ranges * p.col_tiles), dim3(kThreads),
                      Layout<NCOL, FP8, kTileOf<NCOL, FP8>>::kBytes, stream, maps.kv, maps.rope, p);
}

template <bool FP8>
cudaError_t launch_cols(const LatentDecodeMaps &maps, const LatentDecodeParams &p, cudaStream_t stream) {
    return p.cols_per_tile <= 16   ? launch_one<16, FP8>(maps, p, stream)
           : p.cols_per_tile <= 32 ? launch_one<32, FP8>(maps, p, stream)
                                   : launch_one<64, FP8>(maps, p, stream);
}

cudaError_t launch_latent_decode(const LatentDecodeMaps &maps, const LatentDecodeParams &p, bool fp8, cudaStream_t stream) {
    const cudaError_t e = fp8 ? launch_cols<true>(maps, p, stream) : launch_cols<false>(maps, p, stream);
    if (e != cudaSuccess || p.ranges <= 1) return e;
    // Few sequences over many ranges have many parts each: then as many warps share a column's dims as leave all CTAs resident
    // (two an SM; 32 sequences of 1000 tokens, 64 heads: four warps in 1024 CTAs 27.4 us, one 21.2), and read as many parts at
    // once as registers hold (8 sequences of 32K tokens: 8 65.5 us, 12 63.9, 16 65.1); over few ranges 16 (one sequence of 1000
    // tokens, 16 parts: 10.3 us, 12 and 4 10.9).
    const int split = std::min(p.num_seqs, p.ranges - 1), x = (p.heads * p.q_per_seq + kMergeWarps - 1) / kMergeWarps;
    auto merge = [&](auto kernel, int z) { return launch_pdl(kernel, dim3(x, split, z), dim3(kMergeWarps * 32), 0, stream, p); };
    if (p.ranges > 4 * split) {
        if (x * split * 4 <= kMergeResident) return p.ranges <= 32 ? merge(latent_merge_kernel<1, 16>, 4) : merge(latent_merge_kernel<1, 12>, 4);
        return x * split * 2 <= kMergeResident ? merge(latent_merge_kernel<2, 6>, 2) : merge(latent_merge_kernel<4, 4>, 1);
    }
    return merge(latent_merge_kernel<4, 2>, 1);
}

}  // namespace pkv
