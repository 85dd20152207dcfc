// tree_attention.cu -- attention of a tree of drafted tokens over the paged cache, on the
// 5th-generation tensor cores (tcgen05.mma, accumulators in tensor memory).
//
// Sequence b has n nodes whose K and V stand behind its c = ctx - n cached tokens.  Node i's
// row of head h sees the keys j < c and the nodes j - c whose bits are set in its mask:
//     s_j = scale <q[i][h], K_j,g>,  g = floor(h / G),   out[i][h] = sum softmax(s)_j V_j,g
//
// Every row of a (sequence, KV head) sees the same prefix, so the G heads of its n nodes are the
// rows of one MMA tile (row r = node r / G, head r % G; 128 rows, more in several tiles) and
// each K and V tile is read once for all of them: HBM bound up to 128 rows.  Masks touch
// the last key tiles only: a thread holds a row, its mask shifted to a key chunk gives the
// chunk's 32 visible bits.
//
// Split.  The units (sequence, KV head, row tile) have as many key tiles (64 keys) as their
// sequence; all tiles in this order are cut into equal ranges, one for each SM's one CTA (the
// lengths are device data: every CTA finds its range from them).  A CTA walks the pieces of
// units in its range; a unit that lies in several ranges leaves (m, l, O) partials, which
// a second kernel joins.
//
// A CTA's warps (hand-offs through mbarriers, every wait bounded):
//  * 8 fetches K and 12 V by TMA (one copy for each of a tile's four paged blocks) into rings that run
//    ahead of the pieces.  (One warp for both takes 2700 cycles for 64 keys, of which HBM leaves 1400;
//    V by 16-byte asynchronous copies instead: what any warp reads then waits behind them, a
//    piece's 128 rows of Q 6 us.)
//  * 11 fetches the pieces' Q rows into two places in turn, a piece ahead (FP8: behind the last scales of the piece before): by two
//    TMA copies where a tile holds whole nodes (G divides 128), else row by row, which takes the warp
//    9000 cycles for 128 rows (FP8, 64 sequences of 512 .. 4096 tokens: 221 us, 168 with the copies; over a bf16 pool
//    these rows come while the piece before runs: 5 query heads a KV head 118 us for the 115 of 4); the first
//    piece's rows then come by the softmax warps, before the rings fill (behind full rings any
//    read takes 5 us).  FP8: it also makes them codes, and fetches every tile's scales.
//  * 9 issues S = Q K^T, 10 P V (run whole, one elected lane issues: descriptors stay in uniform
//    registers; one warp for both took 3500 cycles for 128 keys, of which HBM leaves 2800).  Tensor
//    memory: S of tile j in [64 (j & 3), +64), O of the even and of the odd tiles in [256, +128) and
//    [384, +128).  With four places for S the next scores are there when a tile's weights are
//    done (with tiles of 128 keys in two places a tile waited for the P V of the one before
//    it: 3400 cycles for 128 keys).
//  * 0-3 and 4-7 are two groups of softmax threads, for the even and the odd tiles; thread r of
//    a group holds row r: maximum, weights 2^(s - m) and their sum need no exchange.  The
//    exponent reference m is raised when a maximum passes it by more than 2^8 (then the row's O is
//    rescaled).  P goes back over S as bf16 heads (truncated) and remainders (rounded), P V =
//    P_hi V + P_lo V: weights to 2^-16.  At a piece's end the groups' (m, l, O) are joined, each
//    group storing half of the values.
//  * Keys past ctx and of blocks with an invalid id are masked by index and their V rows zeroed in
//    shared memory, so stale bytes reach no result.
//
// FP8 pool (E4M3 codes, one scale per key and head).  K's codes are the B operand as they are; a row of Q
// is two rows of E4M3 codes, what the first leaves in the second, scaled by the power of two that
// puts the row's largest value in [2^7, 2^8): exact down to 2^-9 of that value, 2^-17 of it below.
// V's codes come into a ring of their own; 13-15 take every third tile each
// and expand it to fp16 (exact) into the V ring.  K's scale multiplies the scores, V's the weights,
// which enter P V as fp16 heads and remainders (2^-22, as in the FP8 decode).  The reference m counts the exponent of
// a tile's largest V scale in, so that weights times scales stay below 2^15.
//
// Measured (152 SMs, HBM 6.8 TB/s): 64 sequences of 512 .. 4096 tokens, trees of 5 .. 16 nodes, 32 heads over 8: 123 us for
// 640 MB (94 at the copy rate); 8 of 32768, 16 nodes, 64 heads: 189 us for 1.08 GB (159); FP8, the ragged batch with trees of 16
// .. 32 nodes: 192 us for 381 MB (56), not HBM: with one piece of 256 tiles a CTA a tile takes 0.80 us (bf16 0.73, the copy
// rate): S and P V about 1000 cycles each from issue to hand-off, the softmax 2000 for two tiles at once, four places of S, all
// that tensor memory holds; and a piece's change takes 6 to 8 us (bf16 1.6 to 2.6): by the order of warp 11's work Q of the next
// piece is asked for behind this one's last scales, and its codes and first scales come after that.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "ptx.cuh"
#include "speculative.h"

namespace pkv {

namespace {

constexpr int kRows = 128;         // of a row tile
constexpr int kKeys = 64;          // of a tile
constexpr int kTileBlocks = kKeys / kBlockSize;
constexpr int kGroupWarps = 4;     // softmax warps of a group
constexpr int kPlaces = 4;         // of S in tensor memory
constexpr int kWarpK = 8, kWarpS = 9, kWarpPv = 10, kWarpQ = 11, kWarpV = 12, kWarpExpand = 13;

constexpr uint32_t kHalfTile = kRows * 128;      // 16 KB: 128 rows x 128 bytes
constexpr uint32_t kVTile = kKeys * 256;         // 16 KB: 64 bf16 rows of V
constexpr uint32_t kBlkBytes = 4096;             // one paged (block, head) tile of bf16 values
constexpr uint32_t kCodeBytes = 2048;            // the same of codes
constexpr uint32_t kTmemCols = 512, kTmemO = 256;
// FP8: weights times V scales are held 2^6 up, below 2^15 (fp16 ends at 2^16): what fp16 drops is then 2^-31 of the largest.
constexpr int kUp = 6;

template <bool FP8>
struct Layout {
    static constexpr int kExpandWarps = FP8 ? 3 : 0;
    static constexpr int kThreads = (kWarpExpand + kExpandWarps) * 32;
    // (bf16: more than the 128 KB on their way that HBM's latency asks for keep the pieces' Q waiting, 131 us for 140 with 5 + 5,
    // fewer the tensor cores: 16384-token contexts 199 us, 205 with 4 + 3)
    static constexpr int kStagesK = FP8 ? 6 : 4, kStagesV = 4;
    static constexpr int kStagesRaw = FP8 ? 5 : 0;     // of V's codes
    static constexpr int kStagesScale = FP8 ? 12 : 0;  // of both scales, which stay until the softmax is done with the tile
    static constexpr uint32_t kBlk = FP8 ? kCodeBytes : kBlkBytes;  // of the pool
    static constexpr uint32_t kKTile = kTileBlocks * kBlk;
    // Two places of [value half][128 rows][128 B], FP8: [codes, remainders' codes][128 rows][128 B]
    static constexpr uint32_t kOffQ = 0, kQTile = 2 * kHalfTile;
    static constexpr uint32_t kOffK = kOffQ + 2 * kQTile;
    static constexpr uint32_t kOffV = kOffK + kStagesK * kKTile;
    static constexpr uint32_t kOffRaw = kOffV + kStagesV * kVTile;
    static constexpr uint32_t kOffScale = kOffRaw + kStagesRaw * kTileBlocks * kCodeBytes;  // FP8: [tile][K, V][64]
    static constexpr uint32_t kOffOnes = kOffScale + kStagesScale * 2 * kKeys * 4;  // FP8: a tile's K scales, all 1
    static constexpr uint32_t kOffRow = kOffOnes + (FP8 ? kKeys * 4 : 0);  // FP8: factors of Q's rows, two places
    static constexpr uint32_t kOffBad = kOffRow + (FP8 ? 2 * kRows * 4 : 0);  // [tile modulo 16]: blocks with an invalid id
    static constexpr uint32_t kOffMl = kOffBad + (FP8 ? 2 : 1) * 16 * 4;  // (m, l) of the groups' rows
    static constexpr uint32_t kOffBar = kOffMl + 2 * kRows * 8;
    static constexpr int kBarRaw = 2 * kStagesK + 2 * kStagesV, kBarScale = kBarRaw + 2 * kStagesRaw;
    static constexpr int kBarQ = kBarScale + 2 * kStagesScale, kBarS = kBarQ + 6;
    static constexpr int kBarOFree = kBarS + 3 * kPlaces, kBarOReady = kBarOFree + 1, kBars = kBarOFree + 5;
    static constexpr uint32_t kOffPlan = kOffBar + 8 * kBars;
    static constexpr uint32_t kOffSequences = kOffPlan + 96;
    static constexpr uint32_t kBytes = kOffSequences + 32 * sizeof(int) * 3;
    static_assert(kBytes <= 232448, "shared memory of a CTA");
    static_assert(kOffK % 1024 == 0 && kKTile % 1024 == 0 && kOffV % 1024 == 0 && kOffPlan % 8 == 0, "alignment");
};

// Instruction descriptors: D f32; M = 128, N = 64 (S) or 128 (P V).
constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((64u >> 3) << 17) | ((128u >> 4) << 24);  // bf16
constexpr uint32_t kIdescS8 = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);                         // E4M3
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);  // bf16, V MN-major
constexpr uint32_t kIdescPV16 = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);               // the same in fp16

// Shared-memory matrix descriptor for a 128-byte-swizzled canonical layout.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Whether the phase with the given parity is complete, at once.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// The bounded wait of mbar_wait, asleep up to 20 us at a time (a poller takes issue slots from the softmax).
__device__ __forceinline__ bool mbar_sleep_wait(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
    }
}

// A whole warp waits for a barrier's phase, within a bound, and gives up at once after another role gave up.
// (What is complete already costs one test; then come some polls, asleep in code that is not repeated at every wait: the
// roles' loops share the instruction caches.  Without the polls a waking costs what makes FP8 225 us for 191.)
__device__ __noinline__ bool warp_wait_on(uint32_t bar, uint32_t parity, uint32_t abort_at) {
#pragma unroll 1
    for (int i = 0; i < 40; ++i)
        if (__any_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    bool ok = false;
    if ((threadIdx.x & 31) == 0) {
        uint32_t gave_up;
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(gave_up) : "r"(abort_at) : "memory");
        if (!gave_up) {
            ok = mbar_sleep_wait(bar, parity);
            if (!ok) asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort_at), "r"(1u) : "memory");
        }
    }
    return __any_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort_at) {
    return __any_sync(0xffffffffu, mbar_test_wait(bar, parity)) || warp_wait_on(bar, parity, abort_at);
}
// The same without a call, for the softmax warps: what they hold would have to be saved around one.
__device__ __forceinline__ bool softmax_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag) {
#pragma unroll 1
    for (int i = 0; i < 20; ++i)
        if (__any_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    bool ok = false;
    if ((threadIdx.x & 31) == 0 && !*abort_flag) {
        ok = mbar_sleep_wait(bar, parity);
        if (!ok) *abort_flag = 1u;
    }
    return __any_sync(0xffffffffu, ok);
}

// The softmax warps of both groups.
__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(2 * kGroupWarps * 32) : "memory");
}

// P - head for a pair, head = the packed fp16 pair `h`: exact, since head is P rounded.
__device__ __forceinline__ float2 minus_f16x2(float2 p, uint32_t h) {
    float2 d;
    asm("{\n\t.reg .b16 lo, hi, m;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b16 m, 0xBC00;\n\t"
        "fma.rn.f32.f16 %0, lo, m, %3;\n\tfma.rn.f32.f16 %1, hi, m, %4;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(h), "f"(p.x), "f"(p.y));
    return d;
}

// P - head for a pair, head = the packed bf16 pair `h`: exact, since head is P truncated.
__device__ __forceinline__ float2 minus_bf16x2(float2 p, uint32_t h) {
    float2 d;
    asm("{\n\t.reg .b16 lo, hi, m;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b16 m, 0xBF80;\n\t"
        "fma.rn.f32.bf16 %0, lo, m, %3;\n\tfma.rn.f32.bf16 %1, hi, m, %4;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(h), "f"(p.x), "f"(p.y));
    return d;
}

// x / group for a row x of a sequence (magic: 2^32 / group rounded up: exact for 64 nodes of up to 1024 heads, one too many at
// times for the rows of a sequence whose length is refused).
__device__ __forceinline__ int by_group(int x, int group, uint32_t magic) {
    if (magic == 0) return x;  // (a group of 1)
    const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(x), magic));
    return q * group > x ? q - 1 : q;
}

// A sequence as the split sees it (device data: checked).  units is 0 for one without rows, or whose
// rows lie outside the tensors; one whose lengths do not fit has one tile that no row sees, so its rows become zeros.
struct Sequence {
    int row0, n, ctx, row_tiles, units, tiles;
    uint32_t wrong;  // status bits
};
struct Lengths {
    int row0, n, ctx;
};
__device__ __forceinline__ void count_tiles(const TreeParams &p, Sequence &s) {
    s.row_tiles = static_cast<int>((static_cast<int64_t>(s.n) * p.group + kRows - 1) / kRows);
    s.units = s.n > 0 ? s.row_tiles * p.n_kv : 0;
    s.tiles = max(1, (s.ctx + kKeys - 1) / kKeys);
}
__device__ __noinline__ Sequence load_sequence(const TreeParams &p, int b) {
    Sequence s;
    s.row0 = __ldg(p.cu_q_lens + b);
    s.n = __ldg(p.cu_q_lens + b + 1) - s.row0;
    s.ctx = __ldg(p.context_lens + b);
    s.wrong = 0;
    const int64_t most = static_cast<int64_t>(p.max_blocks) * kBlockSize;
    if (s.n < 0 || s.row0 < 0 || s.n > p.total_rows - s.row0) {
        s.wrong = kStatusBadQLen;
        s.n = 0;
    } else if (s.n > 0) {
        if (s.ctx < 1 || s.ctx > most) s.wrong = kStatusBadContextLen;
        if (s.n > p.max_q_len || (s.ctx >= 1 && s.ctx < s.n)) s.wrong |= kStatusBadQLen;
        if (s.wrong) s.ctx = 0;
    }
    count_tiles(p, s);
    return s;
}

// A CTA's range of tiles: the unit it starts in, and its length.
struct Plan {
    int64_t begin, total;  // of the range; tiles of the whole call
    int b, unit, tile, count;
    int ranges;  // that are not empty
    Sequence s;  // b's
};

// The pieces of a range, one after the other; every role walks them by itself.  The sequences (rows, nodes, context) of
// the 32 with plan.b stand in shared memory: behind full rings a read of memory takes 5 us.
struct Walk {
    Sequence s;
    int b, g, row_tile, t0, t1, left;
    bool far;  // past those
    __device__ __forceinline__ void start(const TreeParams &p, const Plan &plan) {
        far = false;
        b = plan.b;
        t0 = plan.tile;
        left = plan.count;
        s = plan.s;
        g = left > 0 ? plan.unit / s.row_tiles : 0;
        row_tile = plan.unit - g * s.row_tiles;
        t1 = min(s.tiles, t0 + left);
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next(const TreeParams &p, const Lengths *known) {
        left -= t1 - t0;
        if (left <= 0) return;
        t0 = 0;
        if (++row_tile == s.row_tiles) {
            row_tile = 0;
            if (++g == p.n_kv) {
                g = 0;
                do {
                    if ((++b & 31) == 0) far = true;
                    if (!far) {
                        s.row0 = known[b & 31].row0;
                        s.n = known[b & 31].n;
                        s.ctx = known[b & 31].ctx;
                        count_tiles(p, s);
                    } else {
                        s = load_sequence(p, b);
                    }
                } while (s.units == 0);
            }
        }
        t1 = min(s.tiles, left);
    }
    __device__ __forceinline__ int rows(const TreeParams &p) const { return min(kRows, s.n * p.group - row_tile * kRows); }
};

// The range of this CTA, by the softmax warps, a thread a sequence: tiles of all sequences, then the sequence that the range
// starts in.  (By one warp, 32 sequences after the other: 304 sequences of 512 tokens took 133 us for 127, 1000 of 100 tokens
// 313 for 293; a lone sequence 0.3 us less.  On the way of every call, with cold instruction caches: short code, and dividends
// that fit 32 bits divided in them.)
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}
constexpr int kPlanThreads = 2 * kGroupWarps * 32;
__device__ __noinline__ void make_plan(const TreeParams &p, Plan *slot, Lengths *known, int64_t *sums) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Sequence s{};
    int64_t upto = 0;  // this thread's tiles and those of the lanes before
    auto load = [&](int b) -> int64_t {  // tiles of all of a sequence's units
        s.tiles = 1;
        s.units = 0;
        if (b < p.num_seqs) s = load_sequence(p, b);
        return static_cast<int64_t>(s.units) * s.tiles;
    };
    auto sum_warps = [&](int64_t x) {  // a warp's sum to its place, and x's scan
        upto = x;
#pragma unroll 1
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        if (lane == 31) sums[warp] = upto;
        softmax_sync();
    };
    int64_t mine = 0, all = 0;
    uint32_t wrong = 0;
#pragma unroll 1
    for (int b = tid; b < p.num_seqs; b += kPlanThreads) {
        all += mine = load(b);
        wrong |= s.wrong;
    }
    if (wrong && blockIdx.x == 0 && p.status) atomicOr(p.status, wrong);
    sum_warps(all);
    int64_t total = 0;
#pragma unroll 1
    for (int w = 0; w < 2 * kGroupWarps; ++w) total += sums[w];
    Plan plan{};
    plan.total = total;
    // (no range of one tile while there are more: a second tile costs 0.7 us, the joining of twice the parts more; one
    // sequence of 128 tokens and 8 KV heads takes 10.3 us for 12.0, of 1000 tokens 13.9 for 15.0, 4 tiles a range 14.1 and 15.0)
    plan.ranges = static_cast<int>(min(static_cast<int64_t>(p.ranges), (total + 1) / 2));
    if (static_cast<int>(blockIdx.x) >= plan.ranges) {
        if (tid == 0) *slot = plan;
        return;
    }
    plan.begin = divide(total * blockIdx.x, plan.ranges);
    plan.count = static_cast<int>(divide(total * (blockIdx.x + 1), plan.ranges) - plan.begin);
    int64_t before = 0;  // tiles of the sequences before these
#pragma unroll 1
    for (int b0 = 0; b0 < p.num_seqs && before <= plan.begin; b0 += kPlanThreads) {
        if (p.num_seqs > kPlanThreads) {  // (else they are there)
            softmax_sync();
            mine = load(b0 + tid);
            sum_warps(mine);
        }
#pragma unroll 1
        for (int w = 0; w < 2 * kGroupWarps; ++w) {
            if (w == warp) {
                const uint32_t past = __ballot_sync(0xffffffffu, before + upto > plan.begin);
                if (past && before <= plan.begin) {  // the range starts in one of this warp's sequences
                    known[lane] = {s.row0, s.n, s.ctx};
                    if (lane == __ffs(past) - 1) {
                        const int64_t inside = plan.begin - (before + upto - mine);
                        plan.b = b0 + tid;
                        plan.unit = static_cast<int>(divide(inside, s.tiles));
                        plan.tile = static_cast<int>(inside - static_cast<int64_t>(plan.unit) * s.tiles);
                        plan.s = s;
                        *slot = plan;
                    }
                }
            }
            before += sums[w];
        }
    }
}

// Sixteen E4M3 codes to fp16 (exact): a holds values 0 .. 7, b 8 .. 15.
__device__ __forceinline__ void e4m3x16_to_f16(const uint4 &c, uint4 &a, uint4 &b) {
    e4m3x4_to_f16x2x2(c.x, a.x, a.y);
    e4m3x4_to_f16x2x2(c.y, a.z, a.w);
    e4m3x4_to_f16x2x2(c.z, b.x, b.y);
    e4m3x4_to_f16x2x2(c.w, b.z, b.w);
}

// A pair of fp16 values to E4M3 codes (in the low 16 bits), to the nearest.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t x) {
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t x, uint32_t y) {
    uint32_t z;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t x, uint32_t y) {
    uint32_t z;
    asm("max.u16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}

// The Q rows first .. first + rows - 1 of a (sequence, KV head) into the tile at dst, unless they are there: the eight rows
// 8 part .., 8 (part + parts) .., .. by one warp.  FP8: as two rows of E4M3 codes (dst, dst + 16 KB), and the factor that undoes the
// row's power of two.  (Not inlined: two roles call it.)
template <bool FP8>
__device__ __noinline__ void load_q(const TreeParams &p, int row0, int first, int rows, int head0, uint32_t dst, float *factor,
                                    int part, int parts, bool there) {
    const int lane = threadIdx.x & 31, G = p.group;
    const uint32_t magic = p.group_magic;
    const __nv_bfloat16 *base = static_cast<const __nv_bfloat16 *>(p.q) + 8 * (lane & 15) +
                                (static_cast<int64_t>(row0) * p.n_q + head0) * kHeadDim;
    // Row r's 16-byte chunk c: half c / 8 (FP8: of the raw values too, whose place the codes take).
    auto place = [&](int r, int c) { return dst + (c >> 3) * kHalfTile + r * 128 + (((c & 7) ^ (r & 7)) << 4); };
#pragma unroll 1
    for (int r0 = there ? rows : 8 * part; r0 < rows; r0 += 8 * parts) {
#pragma unroll 1
        for (int i = 0; i < 8; i += 2) {  // (16 lanes a row; rows past the last are read as the last)
            const int r = r0 + i + (lane >> 4), at = first + min(r, rows - 1), node = by_group(at, G, magic);
            cp_async_16(place(r, lane & 15), base + (static_cast<int64_t>(node) * p.n_q + (at - node * G)) * kHeadDim);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (FP8) {
        __syncwarp();
#pragma unroll 1
        for (int r0 = 8 * part; r0 < rows; r0 += 8 * parts) {  // four lanes a row, 32 values each
            const int r = r0 + (lane >> 2), c = lane & 3;
            uint32_t u[16], most2 = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 raw = lds128(place(r, 4 * c + k));
                u[4 * k] = raw.x;
                u[4 * k + 1] = raw.y;
                u[4 * k + 2] = raw.z;
                u[4 * k + 3] = raw.w;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) most2 = max_u16x2(most2, u[k] & 0x7fff7fffu);
            most2 = max_u16x2(most2, __shfl_xor_sync(0xffffffffu, most2, 1));
            most2 = max_u16x2(most2, __shfl_xor_sync(0xffffffffu, most2, 2));  // (and every lane has its values)
            const uint32_t most = max(most2 << 16, most2 & 0xffff0000u);  // as fp32
            // 2^e puts the largest value in [2^7, 2^8) (both powers are normal numbers)
            const int e = min(126, max(-119, 7 - (static_cast<int>(most >> 23) - 127)));
            // (a scale below 0 negates the row: the softmax's is above)
            const float up = __uint_as_float((static_cast<uint32_t>(127 + e) << 23) | (p.scale_log2 < 0.f ? 0x80000000u : 0u));
            const float2 up2 = make_float2(up, up);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t x[2];  // (fp16 holds the 8 bits down to 2^-17, of which E4M3 keeps those down to 2^-10)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = u[8 * h + 2 * k + i];
                        const float2 y = fmul2(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), up2);
                        x[i] = pack_f16x2(y.x, y.y);
                    }
                    hi[k] = f16x2_to_e4m3x2(x[0]) | (f16x2_to_e4m3x2(x[1]) << 16);
                    uint32_t f0, f1;
                    e4m3x4_to_f16x2x2(hi[k], f0, f1);
                    lo[k] = f16x2_to_e4m3x2(sub_f16x2(x[0], f0)) | (f16x2_to_e4m3x2(sub_f16x2(x[1], f1)) << 16);
                }
                // (a row with an infinity has no finite scores: codes of NaN, as one of 448 would not say)
                if (most == 0x7f800000u) hi[0] = hi[1] = hi[2] = hi[3] = 0x7f7f7f7fu;
                const uint32_t to = dst + r * 128 + (((2 * c + h) ^ (r & 7)) << 4);
                sts128(to, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                sts128(to + kHalfTile, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
            if (c == 0) factor[r] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// The end of a piece: the groups' parts joined, values 64 a .. 64 a + 63 stored by group a; by a softmax warp whose lanes'
// tensor memory begins at lane_base.  It runs behind the group's first tile of the next piece, whose scores are
// there long before the last P V of this one.  False where the wait for that ran out.  (Not inlined: one copy, for the
// instruction caches.)
struct End {
    int64_t to;  // this lane's row among the heads' rows of out, or among the partials
    int piece, rows;
    bool had0, had1, direct;  // the groups' tiles; a whole unit
};
template <bool FP8>
__device__ __noinline__ bool finish_piece(const TreeParams &p, const End end, uint32_t sbase, uint32_t lane_base, bool alive) {
    using L = Layout<FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, a = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const float2 *ml = reinterpret_cast<const float2 *>(smem + L::kOffMl);
    const uint32_t o_free = sbase + L::kOffBar + 8 * L::kBarOFree, o_ready = sbase + L::kOffBar + 8 * L::kBarOReady;
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + L::kOffPlan + 88);
    softmax_sync();  // (m, l) of both groups
    alive = alive && softmax_wait(o_ready, end.piece & 1, abort_flag);
    tc_fence_after();
    if (alive && quarter * 32 < end.rows) {
        const float2 x0 = ml[r], x1 = ml[kRows + r];
        const float top = fmaxf(x0.x, x1.x);
        const float mu = top == -INFINITY ? 0.f : top;
        float f0 = fast_exp2(x0.x - mu), f1 = fast_exp2(x1.x - mu);
        const float sum = f0 * x0.y + f1 * x1.y;
        if (end.direct) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (a row that sees nothing is zero)
            f0 *= inv;
            f1 *= inv;
        } else if (a == 0 && r < end.rows) {
            p.part_ml[end.to] = make_float2(top, sum);
        }
        // Through the piece's place of Q, 4 KB a warp (128 bytes of 32 rows), so that a store writes whole lines: 4 rows of
        // 128 bytes (a row a thread they take the SM 2000 cycles).
        const bool narrow = end.direct && p.out_bf16;
        const uint32_t stage = sbase + L::kOffQ + (end.piece & 1) * L::kQTile + warp * 4096;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {  // 32 values; bf16 leaves as 64, fp32 as 32
            uint32_t o[32], x[32];
            const uint32_t from = lane_base + kTmemO + 64 * a + 32 * half;
            if (end.had0) {
                tmem_ld_32x32b_x32(from, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f0);
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0u;
            }
            if (end.had1) {
                tmem_ld_32x32b_x32(from + 128, x);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(fmaf(__uint_as_float(x[k]), f1, __uint_as_float(o[k])));
            }
            if (half == 1) {  // O has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free);
            }
            const uint32_t at = stage + lane * 128;
            if (narrow) {
                auto two = [&](int k) { return pack_bf16x2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])); };
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sts128(at + (((4 * half + k) ^ (lane & 7)) << 4),
                           make_uint4(two(8 * k), two(8 * k + 2), two(8 * k + 4), two(8 * k + 6)));
                if (half == 0) continue;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sts128(at + ((k ^ (lane & 7)) << 4), make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
            }
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const int rr = 4 * i + (lane >> 3), ch = lane & 7;
                const int64_t to = __shfl_sync(0xffffffffu, end.to, rr) * kHeadDim + 64 * a;
                const uint4 y = lds128(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
                if (quarter * 32 + rr < end.rows) {
                    if (narrow)
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + to + 8 * ch) = y;
                    else
                        *reinterpret_cast<uint4 *>((end.direct ? static_cast<float *>(p.out) : p.part_o) + to + 32 * half + 4 * ch) = y;
                }
            }
            __syncwarp();
        }
        fence_proxy_async_smem();  // (the place's next Q comes behind)
    } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
    }
    softmax_sync();  // (m, l) have been read, and the place of Q
    if (threadIdx.x == 0) mbar_arrive(sbase + L::kOffBar + 8 * (L::kBarQ + 2 + (end.piece & 1)));
    return alive;
}

template <bool FP8>
__global__ void __launch_bounds__(Layout<FP8>::kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ TreeParams p) {
    using L = Layout<FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.group;
    auto bar = [&](int i) { return sbase + L::kOffBar + 8 * i; };
    auto k_full = [&](int st) { return bar(st); };
    auto k_empty = [&](int st) { return bar(L::kStagesK + st); };
    auto v_full = [&](int st) { return bar(2 * L::kStagesK + st); };
    auto v_empty = [&](int st) { return bar(2 * L::kStagesK + L::kStagesV + st); };
    auto raw_full = [&](int st) { return bar(L::kBarRaw + st); };
    auto raw_empty = [&](int st) { return bar(L::kBarRaw + L::kStagesRaw + st); };
    auto scale_full = [&](int st) { return bar(L::kBarScale + st); };
    auto scale_empty = [&](int st) { return bar(L::kBarScale + L::kStagesScale + st); };
    auto q_full = [&](int place) { return bar(L::kBarQ + place); };
    auto q_empty = [&](int place) { return bar(L::kBarQ + 2 + place); };
    auto q_raw = [&](int place) { return bar(L::kBarQ + 4 + place); };  // FP8: before it is codes
    // of tile j: place j % kPlaces, phase j / kPlaces
    auto s_full = [&](int j) { return bar(L::kBarS + j % kPlaces); };
    auto p_full = [&](int j) { return bar(L::kBarS + kPlaces + j % kPlaces); };
    auto pv_done = [&](int j) { return bar(L::kBarS + 2 * kPlaces + j % kPlaces); };
    auto phase = [](int j) -> uint32_t { return (j / kPlaces) & 1; };
    const uint32_t o_free = bar(L::kBarOFree), o_ready = bar(L::kBarOReady);  // O has been read; a piece's last P V is done
    const uint32_t q_first = bar(L::kBarOReady + 1);                          // the first piece's Q is there
    const uint32_t drained = bar(L::kBarOReady + 2);                          // one of each issuing warp
    Plan *plan_slot = reinterpret_cast<Plan *>(smem + L::kOffPlan);
    Lengths *known = reinterpret_cast<Lengths *>(smem + L::kOffSequences);  // of the 32 sequences with the range's first
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffPlan + 80);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + L::kOffPlan + 88);
    static_assert(sizeof(Plan) <= 80, "plan area");

    if (tid == 0) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
        if (p.whole_nodes) prefetch_tensormap(&qmap);
        for (int st = 0; st < L::kStagesK; ++st) {
            mbar_init(k_full(st), 1);
            mbar_init(k_empty(st), 1);
        }
        for (int st = 0; st < L::kStagesV; ++st) {
            mbar_init(v_full(st), 1);
            mbar_init(v_empty(st), 1);
        }
        for (int st = 0; st < L::kStagesRaw; ++st) {
            mbar_init(raw_full(st), 1);
            mbar_init(raw_empty(st), 1);
        }
        for (int st = 0; st < L::kStagesScale; ++st) {
            mbar_init(scale_full(st), 32);  // a lane's share each
            mbar_init(scale_empty(st), kGroupWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_raw(i), 1);
            mbar_init(q_empty(i), 2);  // the last S of a piece, and its end
        }
        for (int i = 0; i < kPlaces; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), kGroupWarps);
            mbar_init(pv_done(i), 1);
        }
        mbar_init(o_free, 2 * kGroupWarps);
        mbar_init(drained, 1);
        mbar_init(drained + 8, 1);
        mbar_init(q_first, 1);
        mbar_init(o_ready, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (FP8 && tid < kKeys) reinterpret_cast<float *>(smem + L::kOffOnes)[tid] = 1.f;
    if (warp == kWarpS) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    griddep_launch_dependents();
    griddep_wait();
    if (warp < 2 * kGroupWarps) make_plan(p, plan_slot, known, reinterpret_cast<int64_t *>(smem + L::kOffMl));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Plan plan = *plan_slot;
    const uint32_t tmem = *tmem_slot;

    auto warp_wait = [&](uint32_t b, uint32_t parity) { return pkv::warp_wait(b, parity, sbase + L::kOffPlan + 88); };

    Walk w;
    w.start(p, plan);
    // A lane's block id of the eight tiles from t on (-1: none), read eight tiles ahead: a read behind full rings takes longer
    // than a tile.
    constexpr int kAhead = 32 / kTileBlocks;
    auto block_ids = [&](int t) -> int {
        const int at = t * kTileBlocks + lane;
        return at < (w.s.ctx + kBlockSize - 1) / kBlockSize ? __ldg(p.block_tables + static_cast<int64_t>(w.b) * p.max_blocks + at) : -1;
    };
    if (warp == kWarpK || warp == kWarpV) {
        // ---------------- copies: one for each of a tile's blocks ----------------
        const bool is_k = warp == kWarpK;
        const bool raw = FP8 && !is_k;
        const int stages = is_k ? L::kStagesK : raw ? L::kStagesRaw : L::kStagesV;
        const uint32_t ring = sbase + (is_k ? L::kOffK : raw ? L::kOffRaw : L::kOffV);
        const uint32_t full0 = is_k ? k_full(0) : raw ? raw_full(0) : v_full(0);
        const uint32_t empty0 = is_k ? k_empty(0) : raw ? raw_empty(0) : v_empty(0);
        const CUtensorMap *map = is_k ? &kmap : &vmap;
        int j = 0, st = 0, use = 0;  // tile of the range; its stage, and the stage's use
        bool ok = true;
#pragma unroll 1
        for (; ok && w.more(); w.next(p, known)) {
            const int blocks = (w.s.ctx + kBlockSize - 1) / kBlockSize, g = w.g;
            // (K and V of one row tile are read once: 64 ragged sequences 131 us, 140 where they push out what others left in L2)
            const uint64_t policy = w.s.row_tiles == 1 ? l2_evict_first() : l2_evict_normal();
            int ids = -1, next = block_ids(w.t0);
#pragma unroll 1
            for (int t = w.t0; t < w.t1; ++t, ++j) {
                // (an invalid id fetches block 0; its keys are masked)
                const int turn = (t - w.t0) & (kAhead - 1);
                if (turn == 0) {
                    ids = next;
                    if (t + kAhead < w.t1) next = block_ids(t + kAhead);
                }
                const int now = __shfl_sync(0xffffffffu, ids, turn * kTileBlocks + (lane & (kTileBlocks - 1)));
                const int id = static_cast<unsigned>(now) < static_cast<unsigned>(p.num_blocks) ? now : 0;
                // (behind full rings a read takes 5 us: the first piece's Q before them)
                if (j == 2 && !(ok = warp_wait(q_first, 0))) break;
                if (use > 0 && !(ok = warp_wait(empty0 + 8 * st, (use - 1) & 1))) break;
                const int load = max(0, min(kTileBlocks, blocks - t * kTileBlocks));
                const uint32_t full = full0 + 8 * st;
                if (is_k || FP8) {
                    // Blocks with an invalid id, for the softmax (which is behind by less than 12 tiles: the place is free)
                    // and, FP8, for the expansion.
                    const uint32_t bad = __ballot_sync(0xffffffffu, lane < load && now != id);
                    if (lane == 0) {
                        sts32(sbase + L::kOffBad + 4 * (j & 15) + (is_k ? 0 : 64), bad);
                        if (is_k && bad && p.status) atomicOr(p.status, kStatusBadBlockId);
                    }
                    __syncwarp();  // (before whichever lane is elected arrives)
                }
                int block[kTileBlocks];
#pragma unroll
                for (int k = 0; k < kTileBlocks; ++k) block[k] = __shfl_sync(0xffffffffu, id, k);
                if (elect_one()) {
                    if (load > 0)
                        mbar_arrive_expect_tx(full, load * L::kBlk);
                    else
                        mbar_arrive(full);
                    const uint32_t dst = ring + st * kTileBlocks * L::kBlk;
#pragma unroll
                    for (int k = 0; k < kTileBlocks; ++k) {
                        if (k < load) {
                            if constexpr (FP8)
                                tma_load_4d(dst + k * L::kBlk, map, full, 0, 0, g, block[k], policy);
                            else
                                tma_load_5d(dst + k * L::kBlk, map, full, 0, 0, 0, 0, block[k] * p.n_kv + g, policy);
                        }
                    }
                }
                __syncwarp();
                if (++st == stages) {
                    st = 0;
                    ++use;
                }
            }
        }
        // (given up: the copies still on their way land before the CTA ends)
        if (!ok && lane == 0)
#pragma unroll 1
            for (int i = max(0, j - stages); i < j; ++i) mbar_wait(full0 + 8 * (i % stages), (i / stages) & 1);
    } else if (FP8 && warp >= kWarpExpand) {
        // ---------------- V's codes of every third tile expanded to fp16 ----------------
        const int x = warp - kWarpExpand;
        const int row = lane >> 3, c = lane & 7;  // of a block: rows row + 4 i, codes 16 c .. 16 c + 15
        int j = 0;
        bool ok = true;
#pragma unroll 1
        for (; ok && w.more(); w.next(p, known)) {
            int t = w.t0 + (x + 2 * j) % 3;  // the piece's first tile whose number j + t - t0 is x modulo 3
#pragma unroll 1
            for (; t < w.t1; t += 3) {
                const int i = j + t - w.t0, raw_st = i % (FP8 ? L::kStagesRaw : 1), st = i % L::kStagesV;
                const int keys = w.s.ctx - t * kKeys;
                ok = warp_wait(raw_full(raw_st), (i / (FP8 ? L::kStagesRaw : 1)) & 1);
                if (ok && i >= L::kStagesV) ok = warp_wait(v_empty(st), ((i / L::kStagesV) - 1) & 1);
                if (!ok) break;
                const uint32_t bad = reinterpret_cast<const volatile uint32_t *>(smem + L::kOffBad)[16 + (i & 15)];
                uint4 code[4];  // a block ahead
                auto read = [&](int k) {
                    const uint32_t src = sbase + L::kOffRaw + (raw_st * kTileBlocks + k) * kCodeBytes + row * 128;
#pragma unroll
                    for (int n = 0; n < 4; ++n) code[n] = lds128(src + n * 512 + ((c ^ ((row + 4 * n) & 7)) << 4));
                };
                read(0);
#pragma unroll 1
                for (int k = 0; k < kTileBlocks; ++k) {
                    const bool good = ((bad >> k) & 1) == 0;
                    const uint32_t dst = sbase + L::kOffV + st * kVTile + k * kBlkBytes + (c >> 2) * 1024;
                    uint4 a[4], b[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        e4m3x16_to_f16(code[n], a[n], b[n]);
                        if (!good || k * kBlockSize + row + 4 * n >= keys) a[n] = b[n] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    if (k + 1 < kTileBlocks) read(k + 1);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {  // 16-byte chunks 2 c and 2 c + 1 of the row's 16
                        const int r = row + 4 * n;
                        const uint32_t at = dst + (r >> 3) * 2048 + (r & 7) * 128;
                        sts128(at + (((2 * (c & 3)) ^ (r & 7)) << 4), a[n]);
                        sts128(at + (((2 * (c & 3) + 1) ^ (r & 7)) << 4), b[n]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(v_full(st));
                    mbar_arrive(raw_empty(raw_st));
                }
            }
            j += w.t1 - w.t0;
        }
    } else if (warp == kWarpQ) {
        // ---------------- the Q rows of the pieces from the second on ----------------
        int4 rec = make_int4(0, 0, 0, 0);  // a unit that begins in the last piece and goes on in the next ranges: for the second kernel
        auto note = [&]() {
            if (w.t0 > 0 || w.left != w.t1 - w.t0 || w.t1 == w.s.tiles) return;
            const int64_t end = plan.begin + plan.count - w.t1 + w.s.tiles;  // behind the unit's last tile
            const int64_t cta = (end * plan.ranges + plan.total - 1) / plan.total - 1;
            rec = make_int4(w.s.row0, w.g, static_cast<int>(cta) - static_cast<int>(blockIdx.x) + 1, w.row_tile * 256 + w.rows(p));
        };
        int j = 0, sent = 0;
        bool ok = true;
        auto arrives = [&](int piece) { return FP8 ? q_raw(piece & 1) : q_full(piece & 1); };  // what the copies complete
#pragma unroll 1
        for (int piece = 0; ok && w.more(); w.next(p, known), ++piece) {
            note();
            const int place = piece & 1;
            const uint32_t dst = sbase + L::kOffQ + place * L::kQTile;
            if (piece > 1 && !(ok = warp_wait(q_empty(place), ((piece >> 1) - 1) & 1))) break;
            if (p.whole_nodes) {
                // One copy for each value half: a tile's rows are the G heads of 128 / G nodes.  (Row by row by 16-byte
                // asynchronous copies the warp takes 9000 cycles for 128 rows.)
                if (elect_one()) {
                    mbar_arrive_expect_tx(arrives(piece), L::kQTile);
                    tma_load_3d(dst, &qmap, arrives(piece), 0, w.g * G, w.s.row0 + w.row_tile * p.whole_nodes);
                    tma_load_3d(dst + kHalfTile, &qmap, arrives(piece), 64, w.g * G, w.s.row0 + w.row_tile * p.whole_nodes);
                    if (piece == 0) mbar_arrive(q_first);
                }
                __syncwarp();
                sent = piece + 1;
            }
            if (piece > 0 && (FP8 || !p.whole_nodes)) {  // (the first piece's by the softmax warps)
                if (p.whole_nodes && !(ok = warp_wait(q_raw(place), (piece >> 1) & 1))) break;
                load_q<FP8>(p, w.s.row0, w.row_tile * kRows, w.rows(p), w.g * G, dst,
                            reinterpret_cast<float *>(smem + L::kOffRow) + place * kRows, 0, 1, p.whole_nodes != 0);
                if (lane == 0) mbar_arrive(q_full(place));
            }
            if constexpr (FP8) {
                const int64_t at = static_cast<int64_t>(w.g) * kBlockSize + 4 * (lane & 3);
                const float *from = ((lane >> 2) & 1) ? p.v_scale : p.k_scale;
                const uint32_t to = sbase + L::kOffScale + (((lane >> 2) & 1) * kKeys + (lane >> 3) * kBlockSize + 4 * (lane & 3)) * 4;
                int ids = -1, next = block_ids(w.t0);
                if (piece == 0 && !(ok = warp_wait(q_first, 0))) break;
#pragma unroll 1
                for (int t = w.t0; t < w.t1; ++t, ++j) {
                    const int turn = (t - w.t0) & (kAhead - 1), place = j % L::kStagesScale;
                    if (turn == 0) {
                        ids = next;
                        if (t + kAhead < w.t1) next = block_ids(t + kAhead);
                    }
                    const int now = __shfl_sync(0xffffffffu, ids, turn * kTileBlocks + (lane >> 3));
                    const int id = static_cast<unsigned>(now) < static_cast<unsigned>(p.num_blocks) ? now : 0;
                    if (j >= L::kStagesScale && !(ok = warp_wait(scale_empty(place), ((j / L::kStagesScale) - 1) & 1))) break;
                    if ((t * kTileBlocks + (lane >> 3)) * kBlockSize < w.s.ctx)
                        cp_async_16(to + place * 2 * kKeys * 4, from + static_cast<int64_t>(id) * p.n_kv * kBlockSize + at);
                    cp_async_mbar_arrive_noinc(scale_full(place));
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        // (given up: the copies still on their way land before the CTA ends)
        if (!ok && lane == 0)
#pragma unroll 1
            for (int i = max(0, sent - 2); i < sent; ++i) mbar_wait(arrives(i), (i >> 1) & 1);
        if (lane == 0) p.record[blockIdx.x] = rec;
    } else if (warp == kWarpS) {
        // ---------------- S = Q K^T ----------------
        int j = 0;
        bool ok = true;
#pragma unroll 1
        for (int piece = 0; ok && w.more(); w.next(p, known), ++piece) {
            const int place = piece & 1;
            if (!(ok = warp_wait(q_full(place), (piece >> 1) & 1))) break;
#pragma unroll 1
            for (int t = w.t0; t < w.t1; ++t, ++j) {
                const int st = j % L::kStagesK;
                ok = warp_wait(k_full(st), (j / L::kStagesK) & 1);
                if (ok && j >= kPlaces) ok = warp_wait(pv_done(j), phase(j - kPlaces));  // the weights there have been read
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t kb = sbase + L::kOffK + st * L::kKTile, qb = sbase + L::kOffQ + place * L::kQTile;
                    const uint32_t d = tmem + kKeys * (j % kPlaces);
                    if constexpr (FP8) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)  // 32 values per step: codes, then the remainders'
                            umma_f8(d, sw128_desc(qb + (kk >> 2) * kHalfTile + (kk & 3) * 32, 16, 1024),
                                    sw128_desc(kb + (kk & 3) * 32, 16, 1024), kIdescS8, kk > 0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)  // 16 values per step: half kk / 4, 32 B into the row
                            umma_bf16(d, sw128_desc(qb + (kk >> 2) * kHalfTile + (kk & 3) * 32, 16, 1024),
                                      sw128_desc(kb + (kk >> 2) * 1024 + (kk & 3) * 32, 16, 2048), kIdescS, kk > 0);
                    }
                    umma_commit(s_full(j));
                    umma_commit(k_empty(st));
                    if (t + 1 == w.t1) umma_commit(q_empty(place));
                }
                __syncwarp();
            }
        }
    } else if (warp == kWarpPv) {
        // ---------------- O += P V ----------------
        int j = 0;
        bool ok = true;
#pragma unroll 1
        for (int piece = 0; ok && w.more(); w.next(p, known), ++piece) {
#pragma unroll 1
            for (int t = w.t0; t < w.t1; ++t, ++j) {
                const int st = j % L::kStagesV;
                ok = warp_wait(v_full(st), (j / L::kStagesV) & 1);
                // O of the piece before has been read
                if (ok && piece > 0 && t - w.t0 < 2) ok = warp_wait(o_free, (piece - 1) & 1);
                ok = ok && warp_wait(p_full(j), phase(j));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t vb = sbase + L::kOffV + st * kVTile, d = tmem + kTmemO + 128 * (j & 1);
                    const uint32_t first = t - w.t0 < 2 ? 0u : 1u;
#pragma unroll
                    for (int s4 = 0; s4 < 4; ++s4) {  // keys 16 s4 ..: [8 columns heads | 8 remainders]
                        const uint32_t at = tmem + kKeys * (j % kPlaces) + 16 * s4;
                        const uint64_t bd = sw128_desc(vb + s4 * kBlkBytes, 1024, 2048);
                        umma_bf16_tmem_a(d, at, bd, FP8 ? kIdescPV16 : kIdescPV, s4 > 0 ? 1u : first);
                        umma_bf16_tmem_a(d, at + 8, bd, FP8 ? kIdescPV16 : kIdescPV, 1u);
                    }
                    umma_commit(pv_done(j));
                    umma_commit(v_empty(st));
                    if (t + 1 == w.t1) umma_commit(o_ready);
                }
                __syncwarp();
            }
        }
    } else {
        // ---------------- softmax: group a takes the tiles j with j & 1 == a, thread r the row r ----------------
        const int a = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_o = lane_base + kTmemO + 128 * a;
        float2 *ml = reinterpret_cast<float2 *>(smem + L::kOffMl);
        bool alive = true;
        if (w.more() && (FP8 || !p.whole_nodes)) {  // the first piece's Q, by all of these warps
            if (p.whole_nodes) alive = softmax_wait(q_raw(0), 0, abort_flag);
            load_q<FP8>(p, w.s.row0, w.row_tile * kRows, w.rows(p), w.g * G, sbase + L::kOffQ,
                        reinterpret_cast<float *>(smem + L::kOffRow), warp, 2 * kGroupWarps, p.whole_nodes != 0);
            softmax_sync();
            if (tid == 0) {
                mbar_arrive(q_full(0));
                if (!p.whole_nodes) mbar_arrive(q_first);
            }
        }
        int j0 = 0;  // tiles before the piece

        End end{};
        bool pending = false;  // a piece's end is still to come
        auto finish = [&]() {
            alive = finish_piece<FP8>(p, end, sbase, lane_base, alive);
            pending = false;
        };
#pragma unroll 1
        for (int piece = 0; w.more(); w.next(p, known), ++piece) {
            const int rows = w.rows(p), first_row = w.row_tile * kRows, g = w.g;
            const bool busy = quarter * 32 < rows;  // (warp-uniform: a warp without rows only keeps step)
            const int prefix = w.s.ctx - w.s.n;
            const int node = by_group(first_row + r, G, p.group_magic);
            const int64_t row = static_cast<int64_t>(w.s.row0) + node;
            uint64_t mask = 0;
            if (r < rows && w.s.ctx > 0) {
                mask = __ldg(reinterpret_cast<const unsigned long long *>(p.mask) + row);  // (not looked at before the tree's tiles)
            }
            __syncwarp();  // (the loads from tensor memory want the whole warp)
            float sl2 = p.scale_log2;
            float m = -INFINITY, l = 0.f;
            const int t_first = w.t0 + ((j0 ^ a) & 1);
#pragma unroll 1
            for (int t = t_first; t < w.t1; t += 2) {
                const int j = j0 + t - w.t0;
                if constexpr (FP8) {
                    // (both barriers by one vote while both are complete: the hand-offs are on a tile's way, 197 us for 180)
                    const uint32_t scale_bar = scale_full(j % L::kStagesScale), scale_phase = (j / L::kStagesScale) & 1;
                    if (!__any_sync(0xffffffffu, mbar_test_wait(s_full(j), phase(j)) & mbar_test_wait(scale_bar, scale_phase)))
                        alive = alive && softmax_wait(scale_bar, scale_phase, abort_flag) && softmax_wait(s_full(j), phase(j), abort_flag);
                } else {
                    alive = alive && softmax_wait(s_full(j), phase(j), abort_flag);
                }
                if (!alive) continue;
                tc_fence_after();
                const uint32_t t_s = lane_base + kKeys * (j % kPlaces);
                const uint32_t bad = reinterpret_cast<const volatile uint32_t *>(smem + L::kOffBad)[j & 15];
                if (busy) {
                    if constexpr (FP8) {
                        // (a factor of 0 counts as the least normal number: a hidden key's -inf times it stays one)
                        if (t == t_first) {
                            sl2 = fabsf(p.scale_log2) * reinterpret_cast<const float *>(smem + L::kOffRow)[(piece & 1) * kRows + r];
                            if (sl2 < 0x1p-126f) sl2 = 0x1p-126f;
                        }
                    }
                    const uint32_t scales = sbase + L::kOffScale + (j % (FP8 ? L::kStagesScale : 1)) * 2 * kKeys * 4;
                    float2 sl2v = make_float2(sl2, sl2);  // (bf16)
                    uint32_t most_v = 0;  // FP8: the largest V scale (its bits) of the keys that the row sees
                    uint32_t k_scales = scales;
                    // Tiles that not every row sees whole: the scores are scaled and the hidden ones -inf before the pass below,
                    // which then scales them by 1.  (A loop of its own, once or twice a sequence: in the pass, whose code the
                    // instruction caches have to hold beside six other roles', selects cost every tile.)
                    if (__builtin_expect(t * kKeys + kKeys > prefix || bad, 0)) {
                        const int at = t * kKeys - prefix;  // node of the tile's first key
                        const uint64_t nodes = w.s.n < 64 ? mask & ((1ull << w.s.n) - 1) : mask;
                        uint64_t seen = at >= 0 ? (at < 64 ? nodes >> at : 0) : at > -64 ? ((1ull << -at) - 1) | (nodes << -at) : ~0ull;
#pragma unroll 1
                        for (int k = 0; k < kTileBlocks; ++k)
                            if ((bad >> k) & 1) seen &= ~(0xffffull << (16 * k));
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[16];
                            tmem_ld_32x32b_x16(t_s + 16 * c, x);
                            const uint32_t bits = static_cast<uint32_t>(seen >> (16 * c));
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float f = FP8 ? lds_f32(scales + 4 * (16 * c + k)) : sl2;
                                x[k] = (bits >> k) & 1 ? __float_as_uint(__uint_as_float(x[k]) * f) : 0xff800000u;
                                if (FP8 && ((bits >> k) & 1))
                                    most_v = max(most_v, __float_as_uint(lds_f32(scales + 4 * (kKeys + 16 * c + k))) & 0x7fffffffu);
                            }
                            tmem_st_32x32b_x16(t_s + 16 * c, x);
                        }
                        tmem_wait_st();
                        sl2v = make_float2(1.f, 1.f);
                        if constexpr (FP8) {
                            k_scales = sbase + L::kOffOnes;
                            // V scales that belong to no key may be anything: 0 (every warp writes the same)
#pragma unroll 1
                            for (int k = lane; k < kKeys; k += 32)
                                if (t * kKeys + k >= w.s.ctx || ((bad >> (k >> 4)) & 1)) sts32(scales + 4 * (kKeys + k), 0u);
                            fence_proxy_async_smem();  // (the next copy there comes behind)
                            __syncwarp();
                        }
                    }
                    // The row's largest score in the log2 domain.  (FP8: 32 keys at a time, scaled by each key's K scale, the first
                    // 32 put back; the row's factor comes behind.  All 64 at once leave no registers for the scales: spilled
                    // ones come back through the L1 that 200 KB of shared memory leave, 403 us for 211.)
                    constexpr int kPass = FP8 ? 32 : kKeys;
                    uint32_t v[kPass];
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < kKeys / kPass; ++c) {
                        if constexpr (FP8)
                            tmem_ld_32x32b_x32(t_s + kPass * c, v);
                        else
                            tmem_ld_32x32b_x64(t_s, v);
#pragma unroll
                        for (int i = 0; i < kPass / 4; ++i) {
                            float2 f0 = sl2v, f1 = sl2v;
                            if constexpr (FP8) {
                                const uint4 f = lds128(k_scales + 128 * c + 16 * i);
                                f0 = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
                                f1 = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
                            }
                            const float2 x = fmul2(make_float2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), f0);
                            const float2 y = fmul2(make_float2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), f1);
                            mx[2 * (i & 1)] = fmax3(mx[2 * (i & 1)], x.x, x.y);
                            mx[2 * (i & 1) + 1] = fmax3(mx[2 * (i & 1) + 1], y.x, y.y);
                            if constexpr (FP8) {
                                v[4 * i] = __float_as_uint(x.x);
                                v[4 * i + 1] = __float_as_uint(x.y);
                                v[4 * i + 2] = __float_as_uint(y.x);
                                v[4 * i + 3] = __float_as_uint(y.y);
                            }
                        }
                        if (FP8 && c == 0) tmem_st_32x32b_x32(t_s, reinterpret_cast<uint32_t (&)[32]>(v));
                    }
                    float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if constexpr (FP8) {
                        // and the exponent of the largest V scale of the tile's keys (a sum of weights of scales below 2^-90 would
                        // leave fp32); where the rows do not see the same keys, of those that this one sees
                        if (k_scales == scales) {
                            const float2 sv = lds_f32x2(scales + (kKeys + 2 * lane) * 4);
                            most_v = __reduce_max_sync(0xffffffffu,
                                                       max(__float_as_uint(sv.x) & 0x7fffffffu, __float_as_uint(sv.y) & 0x7fffffffu));
                        }
                        mt = fmaf(mt, sl2, static_cast<float>(min(max(static_cast<int>(most_v >> 23) - 127 - kUp, -90), 100)));
                        tmem_wait_st();
                    }
                    float alpha = 1.f;
                    if (mt > m + 8.f) {
                        alpha = fast_exp2(m - mt);  // (0 where m is -inf)
                        m = mt;
                    }
                    // O rescaled, behind the P V of this group's tile before
                    if (__builtin_expect(t >= w.t0 + 2 && __any_sync(0xffffffffu, alpha != 1.f), 0)) {
                        alive = softmax_wait(pv_done(j - 2), phase(j - 2), abort_flag);
                        tc_fence_after();
                        if (alive) {
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint32_t o[16];
                                tmem_ld_32x32b_x16(t_o + 16 * c, o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                                tmem_st_32x32b_x16(t_o + 16 * c, o);
                            }
                        }
                    }
                    // P = 2^(s - m) over S, and the row's sum
                    const float mu = m == -INFINITY ? 0.f : m;
                    const float2 nmu = make_float2(-mu, -mu);
                    float2 rs0 = make_float2(0.f, 0.f), rs1 = make_float2(0.f, 0.f);
                    const float2 slope = FP8 ? make_float2(sl2, sl2) : sl2v;
#pragma unroll 1
                    for (int c = kKeys / kPass - 1; c >= 0; --c) {
                        if (FP8 && c == 0) tmem_ld_32x32b_x32(t_s, reinterpret_cast<uint32_t (&)[32]>(v));
#pragma unroll
                        for (int h = 0; h < kPass / 16; ++h) {  // 16 keys: 8 columns of heads, 8 of remainders
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const int k = 16 * h + 2 * e;
                                const float2 x = ffma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), slope, nmu);
                                const float2 y = ffma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), slope, nmu);
                                float2 px = make_float2(fast_exp2(x.x), fast_exp2(x.y)), py = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                                rs0 = fadd2(rs0, px);
                                rs1 = fadd2(rs1, py);
                                if constexpr (FP8) {  // (the sum keeps the plain weights)
                                    const uint4 f = lds128(scales + (kKeys + kPass * c + k) * 4);
                                    px = fmul2(px, make_float2(__uint_as_float(f.x), __uint_as_float(f.y)));
                                    py = fmul2(py, make_float2(__uint_as_float(f.z), __uint_as_float(f.w)));
                                    pk[e] = pack_f16x2(px.x, px.y);
                                    pk[e + 1] = pack_f16x2(py.x, py.y);
                                    const float2 ex = minus_f16x2(px, pk[e]), ey = minus_f16x2(py, pk[e + 1]);
                                    pk[8 + e] = pack_f16x2(ex.x, ex.y);
                                    pk[9 + e] = pack_f16x2(ey.x, ey.y);
                                } else {
                                    pk[e] = __byte_perm(__float_as_uint(px.x), __float_as_uint(px.y), 0x7632);
                                    pk[e + 1] = __byte_perm(__float_as_uint(py.x), __float_as_uint(py.y), 0x7632);
                                    const float2 ex = minus_bf16x2(px, pk[e]), ey = minus_bf16x2(py, pk[e + 1]);
                                    pk[8 + e] = pack_bf16x2(ex.x, ex.y);
                                    pk[9 + e] = pack_bf16x2(ey.x, ey.y);
                                }
                            }
                            tmem_st_32x32b_x16(t_s + kPass * c + 16 * h, pk);
                        }
                    }
                    const float2 rs = fadd2(rs0, rs1);
                    l = l * alpha + (rs.x + rs.y);
                    tmem_wait_st();
                }
                // V rows of keys that are not the sequence's, or of a bad block: zeros before the P V reads them (FP8: by the
                // expansion)
                const int past = w.s.ctx - t * kKeys;
                if (__builtin_expect(!FP8 && (past < kKeys || bad), 0)) {
                    alive = softmax_wait(v_full(j % L::kStagesV), (j / L::kStagesV) & 1, abort_flag);
                    if (!alive) continue;
                    const uint32_t vb = sbase + L::kOffV + (j % L::kStagesV) * kVTile;
#pragma unroll 1
                    for (int i = r; i < kKeys * 16; i += kGroupWarps * 32) {
                        const int key = i >> 4, ch = i & 15;  // (all 16 chunks of a row: the swizzle is moot)
                        if (key >= past || ((bad >> (key >> 4)) & 1u))
                            sts128(vb + (key >> 4) * kBlkBytes + ((key >> 3) & 1) * 2048 + (ch >> 3) * 1024 + (key & 7) * 128 +
                                       (ch & 7) * 16,
                                   make_uint4(0u, 0u, 0u, 0u));
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(p_full(j));
                    if constexpr (FP8) mbar_arrive(scale_empty(j % L::kStagesScale));
                }
                if (pending) finish();
            }
            // ---- the piece's end ----
            const int tiles = w.t1 - w.t0;
            if (pending) finish();
            ml[a * kRows + r] = make_float2(m, l);
            pending = true;
            end.piece = piece;
            end.rows = busy ? rows : 0;
            end.had0 = tiles > 1 || (j0 & 1) == 0;
            end.had1 = tiles > 1 || (j0 & 1) == 1;
            end.direct = tiles == w.s.tiles;
            end.to = end.direct ? row * p.n_q + static_cast<int64_t>(g) * G + (first_row + r - node * G)
                                : (static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 > 0 ? 0 : 1)) * p.part_rows + r;
            j0 += tiles;
        }
        if (pending) finish();
    }

    // ---- every role is done (or gave up): tensor memory is freed ----
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag) {
        if (tid == 0 && p.status) atomicOr(p.status, kStatusTimeout);
        if ((warp == kWarpS || warp == kWarpPv) && elect_one()) {  // MMAs on their way end before the columns are freed
            const uint32_t b = drained + (warp == kWarpS ? 0 : 8);
            umma_commit(b);
            mbar_wait(b, 0);
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == kWarpS) tmem_dealloc(tmem, kTmemCols);
}

// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the parts of a split unit: a warp takes a
// row, lane k its values 4 k .. 4 k + 3.  The unit's first part lies in the range that it begins in (slot
// 1), the others in slot 0 of the ranges behind.
constexpr int kMergeRows = 8;  // rows (warps) of a CTA
__global__ void __launch_bounds__(kMergeRows * 32) tree_merge_kernel(const TreeParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int c = blockIdx.x, lane = threadIdx.x & 31, r = blockIdx.y * kMergeRows + (threadIdx.x >> 5);
    const int4 rec = p.record[c];
    const int parts = rec.z;
    if (parts < 2 || r >= (rec.w & 255)) return;
    auto part = [&](int i) -> int64_t { return (static_cast<int64_t>(c + i) * 2 + (i == 0 ? 1 : 0)) * p.part_rows + r; };
    // Lane k holds (m, l) of the parts k, 32 + k, ..; the first 32 are read once.
    const float2 none = make_float2(-INFINITY, 0.f), x0 = lane < parts ? __ldcg(p.part_ml + part(lane)) : none;
    float top = x0.x;
    for (int i = lane + 32; i < parts; i += 32) top = fmaxf(top, __ldcg(p.part_ml + part(i)).x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float mu = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = 0; i0 < parts; i0 += 32) {
        const float2 x = i0 == 0 ? x0 : i0 + lane < parts ? __ldcg(p.part_ml + part(i0 + lane)) : none;
        const float mine = fast_exp2(x.x - mu);
        sum = fmaf(mine, x.y, sum);
        const int here = min(32, parts - i0);
#pragma unroll 8
        for (int i = 0; i < here; ++i) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part_o + part(i0 + i) * kHeadDim) + lane);
            const float f = __shfl_sync(0xffffffffu, mine, i);
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int at = (rec.w >> 8) * kRows + r, node = by_group(at, p.group, p.group_magic);
    const int64_t head = (static_cast<int64_t>(rec.x) + node) * p.n_q + static_cast<int64_t>(rec.y) * p.group + (at - node * p.group);
    if (p.out_bf16)
        reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + head * kHeadDim)[lane] =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    else
        reinterpret_cast<float4 *>(static_cast<float *>(p.out) + head * kHeadDim)[lane] =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

}  // namespace

cudaError_t tree_prepare_device() {
    const cudaError_t e = cudaFuncSetAttribute(tree_attention_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(Layout<false>::kBytes));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(tree_attention_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Layout<true>::kBytes));
}

cudaError_t launch_tree_attention(const CUtensorMap &kmap, const CUtensorMap &vmap, const CUtensorMap &qmap, const TreeParams &p, bool fp8,
                                  cudaStream_t stream) {
    const cudaError_t e = fp8 ? launch_pdl(tree_attention_kernel<true>, dim3(p.ranges), dim3(Layout<true>::kThreads),
                                           Layout<true>::kBytes, stream, kmap, vmap, qmap, p)
                              : launch_pdl(tree_attention_kernel<false>, dim3(p.ranges), dim3(Layout<false>::kThreads),
                                           Layout<false>::kBytes, stream, kmap, vmap, qmap, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(tree_merge_kernel, dim3(p.ranges, (p.part_rows + kMergeRows - 1) / kMergeRows), dim3(kMergeRows * 32), 0,
                      stream, p);
}

}  // namespace pkv
