// speculate.cu -- what follows the attention of drafted tokens: their verification against
// the target's probabilities, and the accepted path's rows moved to consecutive slots.
//
// Verification.  Sequence b's tree has the nodes 0 .. n - 1 (node 0 is the token sampled last;
// a parent comes before its children); p_i is the target's distribution behind node i.  From
// node 0 on, the children of the current node are looked at in their order:
//   chain with the drafter's q:  child j, token x, is accepted when u_j q_i(x) < p_i(x);
//   without q:                   when u_j r < p_i(x), r = 1 - the p_i of the siblings refused
//                                before it (a token refused once has no probability left).
// An accepted child is the next current node.  Where none is left, the last token comes from
// the current node's weights w(v) -- max(p_i(v) - q_i(v), 0) where a drafted child was refused,
// else p_i(v) without the refused children's tokens -- as the least v with
//   w(0) + .. + w(v) > u_0 sum w.
// (Leviathan et al., "Fast Inference from Transformers via Speculative Decoding"; the tree form
// draws from p_i and follows the draw as long as it is among the children.)
//
// The products next to a border (24 bits each) and the few sums of the walk are fp64: exact, or
// nearly.  The sums over the vocabulary are pairs of fp32 (high part and remainder; a lane's n
// entries are off by n^2 2^-50 at most, a join of two sums by 2^-46): the same token as sums in fp64
// but for borders closer than that, without the slow fp64 pipe (two additions a clock and SM: 64 rows
// of 128000 would take it 14 us, and the search within a segment of 2000 entries 10 us).
//
// One cluster of up to 8 CTAs takes a sequence: each warp sums one segment of the vocabulary, the
// segment sums are exchanged through distributed shared memory, and the CTA whose segment
// holds the drawn token reads that segment (a few KB, in cache) a second time.  HBM bound for
// batches (one row of p and one of q a sequence), latency bound for few sequences: three
// dependent reads (lengths, tokens, probabilities) come before the row.
// 64 sequences x 128000 entries with the drafter's: 20.3 us (65 MB; HBM alone 9.7: 3 us until the row is known, 11 to
// read it, 5 from the last sum to the token); 16 trees of up to 32 nodes x 50257 entries: 10.5 us.
#include <cuda_runtime.h>

#include <cmath>

#include "ptx.cuh"
#include "speculative.h"

namespace pkv {

namespace {

constexpr int kVerifyThreads = kVerifyWarps * 32;
constexpr int kSegments = kVerifyWarps * kVerifyMaxCluster;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A pair into another CTA's copy of this CTA's shared-memory address.
__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t rank, float2 v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(v.x), "f"(v.y) : "memory");
}

// A probability as it counts: NaN and below 0 as 0, above 1 as 1 (so sums stay finite).
__device__ __forceinline__ float weigh(float p) { return fminf(fmaxf(p, 0.f), 1.f); }

// Pairs (x the sum rounded to fp32, y what that leaves) of weights: each sum is right to 2^-46.
__device__ __forceinline__ float2 renormal(float h, float l) {
    const float x = __fadd_rn(h, l);
    return make_float2(x, __fsub_rn(l, __fsub_rn(x, h)));
}
__device__ __forceinline__ float2 plus(float2 a, float2 b) {
    const float sum = __fadd_rn(a.x, b.x), part = __fsub_rn(sum, a.x);
    const float rest = __fadd_rn(__fsub_rn(a.x, __fsub_rn(sum, part)), __fsub_rn(b.x, part));
    return renormal(sum, __fadd_rn(rest, __fadd_rn(a.y, b.y)));
}
__device__ __forceinline__ float2 pair(double x) {
    const float h = static_cast<float>(x);
    return make_float2(h, static_cast<float>(x - static_cast<double>(h)));
}
__device__ __forceinline__ bool above(float2 a, float2 b) { return a.x > b.x || (a.x == b.x && a.y > b.y); }
__device__ __forceinline__ float2 shuffle_up(float2 a, int off) {
    return make_float2(__shfl_up_sync(0xffffffffu, a.x, off), __shfl_up_sync(0xffffffffu, a.y, off));
}
// This lane's value and those of the lanes before, over a power of two of lanes.
__device__ __forceinline__ float2 scan_lanes(float2 a, int lane, int lanes) {
#pragma unroll
    for (int off = 1; off < lanes; off <<= 1) {
        const float2 y = shuffle_up(a, off), z = plus(a, y);
        a = make_float2(lane >= off ? z.x : a.x, lane >= off ? z.y : a.y);
    }
    return a;
}

// The weight of entry v (exact: p > q, so p - (p - q rounded) - q has no rounding).
__device__ __forceinline__ float2 weight(const float *p, const float *q, int v) {
    const float x = weigh(__ldg(p + v));
    if (!q) return make_float2(x, 0.f);
    const float y = weigh(__ldg(q + v));
    if (!(x > y)) return make_float2(0.f, 0.f);
    const float d = __fsub_rn(x, y);
    return make_float2(d, __fsub_rn(__fsub_rn(x, d), y));
}

struct VerifyShared {
    float2 sums[kSegments];  // of every segment of the cluster
    double p[kMaxTreeNodes];
    float u[kMaxTreeNodes];
    bool accepted[kMaxTreeNodes];  // with the drafter's probabilities: u q < p
    int32_t token[kMaxTreeNodes], parent[kMaxTreeNodes];
    int32_t path[kMaxTreeNodes];
    int32_t refused[kMaxTreeNodes];  // tokens that have no weight left
    int32_t count, refusals, found;
    double goal, below;  // of the draw: u_0 sum w, and the weights before the segment
    float2 warp_sums[kVerifyWarps];
    int32_t passes[kVerifyWarps], some[kVerifyWarps];  // entries: the first that passes the goal, the last with weight
};

__global__ void __launch_bounds__(kVerifyThreads, 2) speculative_verify_kernel(const SpecVerifyParams p) {
    __shared__ VerifyShared sh;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int b = blockIdx.x / ctas;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    cluster_arrive();  // (every CTA of the cluster runs before another writes to it)
    griddep_launch_dependents();
    griddep_wait();
    const int row0 = __ldg(p.cu_q_lens + b);
    int n = __ldg(p.cu_q_lens + b + 1) - row0;
    if (n < 0 || n > p.max_q_len || row0 < 0 || n > p.total_rows - row0) {
        if (rank == 0 && tid == 0 && p.status) atomicOr(p.status, kStatusBadQLen);
        n = 0;
    }

    // ---- the nodes: tokens, parents, and the probabilities behind their parents ----
    if (tid < kMaxTreeNodes && tid < n) {
        const int j = tid;
        const int32_t token = __ldg(p.tokens + row0 + j);
        int32_t up = j - 1;
        if (p.parents && j > 0) up = __ldg(p.parents + row0 + j);
        const bool ok = j > 0 && up >= 0 && up < j && token >= 0 && token < p.vocab;
        sh.u[j] = __ldg(p.uniforms + row0 + j);
        sh.token[j] = token;
        sh.parent[j] = j > 0 && up >= 0 && up < j ? up : -1;
        const int64_t at = static_cast<int64_t>(row0) + (ok ? up : 0);
        const double pj = ok ? static_cast<double>(weigh(__ldg(p.target + at * p.target_row + token))) : 0.0;
        sh.p[j] = pj;
        if (p.draft) {
            const double qj = ok ? static_cast<double>(weigh(__ldg(p.draft + at * p.draft_row + token))) : 0.0;
            sh.accepted[j] = static_cast<double>(sh.u[j]) * qj < pj;
        }
    }
    cluster_wait();
    __syncthreads();

    // ---- the walk: warp 0, every lane alike ----
    if (warp == 0 && p.draft) {  // a chain up to its first refusal
        const uint64_t refused = ~((static_cast<uint64_t>(__ballot_sync(0xffffffffu, lane < n && (lane == 0 || sh.accepted[lane]))) |
                                    static_cast<uint64_t>(__ballot_sync(0xffffffffu, lane + 32 < n && sh.accepted[lane + 32])) << 32));
        const int count = refused ? __ffsll(static_cast<long long>(refused)) - 1 : 64;
        if (lane < count) sh.path[lane] = lane;
        if (lane + 32 < count) sh.path[lane + 32] = lane + 32;
        if (lane == 0) {
            sh.count = count;
            sh.refusals = count < n ? 1 : 0;
        }
    } else if (warp == 0) {
        int cur = 0, count = n > 0 ? 1 : 0, refusals = 0;
        if (lane == 0) sh.path[0] = 0;
        // nodes lane and lane + 32
        const int up0 = lane < n ? sh.parent[lane] : -1, up1 = lane + 32 < n ? sh.parent[lane + 32] : -1;
        while (n > 0) {
            uint64_t children = static_cast<uint64_t>(__ballot_sync(0xffffffffu, up0 == cur)) |
                                (static_cast<uint64_t>(__ballot_sync(0xffffffffu, up1 == cur)) << 32);
            double rest = 1.0;
            int next = -1;
            refusals = 0;
            while (children) {
                const int j = __ffsll(static_cast<long long>(children)) - 1;
                children &= children - 1;
                const int32_t token = sh.token[j];
                double pj = sh.p[j];
                // a token refused before has no probability left
                const bool gone = (lane < refusals && sh.refused[lane] == token) ||
                                  (lane + 32 < refusals && sh.refused[lane + 32] == token);
                if (__any_sync(0xffffffffu, gone)) pj = 0.0;
                if (static_cast<double>(sh.u[j]) * rest < pj) {
                    next = j;
                    break;
                }
                __syncwarp();
                if (lane == 0) sh.refused[refusals] = token;
                ++refusals;
                __syncwarp();
                rest -= pj;
            }
            if (next < 0) break;
            cur = next;
            if (lane == 0) sh.path[count] = cur;
            ++count;
        }
        if (lane == 0) {
            sh.count = count;
            sh.refusals = refusals;
        }
    }
    __syncthreads();
    const int count = sh.count;

    // ---- everything but the last token ----
    if (rank == 0)
        for (int i = tid; i < p.max_q_len; i += kVerifyThreads) {
            const int64_t o = static_cast<int64_t>(b) * p.max_q_len + i;
            p.path[o] = i < count ? sh.path[i] : -1;
            if (i + 1 < count) p.tokens_out[o] = sh.token[sh.path[i + 1]];
            if (i >= count) p.tokens_out[o] = -1;
        }
    if (rank == 0 && tid == 0) p.counts[b] = count;
    const int cur = count > 0 ? sh.path[count - 1] : 0;
    const int64_t row = static_cast<int64_t>(row0) + cur;
    const float *target = p.target + row * p.target_row;
    const float *draft = p.draft && sh.refusals > 0 ? p.draft + row * p.draft_row : nullptr;
    int refusals = p.draft ? 0 : sh.refusals;
    const int segments = ctas * kVerifyWarps;
    const int seg = rank * kVerifyWarps + warp;
    // (64 bits: the last segments may lie wholly behind the vocabulary)
    const int lo = static_cast<int>(min(static_cast<int64_t>(seg) * p.segment, static_cast<int64_t>(p.vocab)));
    const int hi = static_cast<int>(min(static_cast<int64_t>(seg + 1) * p.segment, static_cast<int64_t>(p.vocab)));
    auto refused_from = [&](int v) {  // bit i: v + i, i < 4
        uint32_t gone = 0;
        for (int i = 0; i < refusals; ++i) {
            const uint32_t at = static_cast<uint32_t>(sh.refused[i]) - static_cast<uint32_t>(v);
            if (at < 4) gone |= 1u << at;
        }
        return gone;
    };

    for (int attempt = 0; attempt < 2 && count > 0; ++attempt) {
        // ---- the segment's sum ----
        float2 h = make_float2(0.f, 0.f), l = make_float2(0.f, 0.f);  // two sums, of even and odd entries
        bool here = false;  // a refused token lies in this segment
        for (int i = lane; i < refusals; i += 32) here = here || (sh.refused[i] >= lo && sh.refused[i] < hi);
        here = __any_sync(0xffffffffu, here);
        // h + l += max(x - y, 0), with what each rounding loses going to l
        auto add = [&](float2 x, float2 y) {
            const float2 minus = make_float2(-1.f, -1.f);
            y = make_float2(weigh(y.x), weigh(y.y));
            x = make_float2(fmaxf(weigh(x.x), y.x), fmaxf(weigh(x.y), y.y));
            const float2 d = ffma2(y, minus, x), e = ffma2(y, minus, ffma2(d, minus, x));
            const float2 sum = fadd2(h, d), part = ffma2(h, minus, sum);
            const float2 rest = fadd2(ffma2(ffma2(part, minus, sum), minus, h), ffma2(part, minus, d));
            l = fadd2(l, fadd2(rest, e));
            h = sum;
        };
        auto one = [&](int v) {
            const float x = __ldg(target + v), y = draft ? __ldg(draft + v) : 0.f;
            if (!here || !(refused_from(v) & 1)) add(make_float2(x, 0.f), make_float2(y, 0.f));
        };
        // Four entries a load where both rows begin alike against 16 bytes (lo is a multiple of 4), from the first boundary on.
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(target) >> 2) & 3;
        const bool wide = !draft || (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(draft) >> 2) & 3) == off;
        if (wide) {
            const int head = min(lo + static_cast<int>((4 - off) & 3), hi), full = head + ((hi - head) & ~3);
            // Two loads ahead of the sums (loads of one turn, then its sums: 64 x 128000 with drafts 22.4 us for 20.2; three or four
            // ahead gain 2 us where a warp takes 8000 entries and lose 2 where it takes 400).
            constexpr int kAhead = 2;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            float4 x[kAhead], y[kAhead];
            auto load = [&](int i, int v) {
                x[i] = v < full ? __ldg(reinterpret_cast<const float4 *>(target + v)) : zero;
                y[i] = v < full && draft ? __ldg(reinterpret_cast<const float4 *>(draft + v)) : zero;
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) load(i, head + 4 * lane + 128 * i);
#pragma unroll 1
            for (int v0 = head + 4 * lane; v0 < full; v0 += 128 * kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int v = v0 + 128 * i;
                    float4 now = x[i];
                    const float4 less = y[i];
                    load(i, v + 128 * kAhead);
                    if (here) {
                        const uint32_t gone = refused_from(v);
                        if (gone & 1) now.x = 0.f;
                        if (gone & 2) now.y = 0.f;
                        if (gone & 4) now.z = 0.f;
                        if (gone & 8) now.w = 0.f;
                    }
                    add(make_float2(now.x, now.y), make_float2(less.x, less.y));
                    add(make_float2(now.z, now.w), make_float2(less.z, less.w));
                }
            }
            if (lo + lane < head) one(lo + lane);
            if (full + lane < hi) one(full + lane);
        } else {
#pragma unroll 2
            for (int v = lo + lane; v < hi; v += 32) one(v);
        }
        float2 sum = plus(renormal(h.x, l.x), renormal(h.y, l.y));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            sum = plus(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, off), __shfl_xor_sync(0xffffffffu, sum.y, off)));
        if (lane < static_cast<int>(ctas)) store_remote(smem_u32(&sh.sums[seg]), lane, sum);
        cluster_arrive();
        cluster_wait();

        // ---- the segment that the draw falls into (warp 0 of every CTA, alike) ----
        if (warp == 0) {
            // (in fp64: one warp's few additions, each one instruction)
            double x[4], upto = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 y = 4 * lane + i < segments ? sh.sums[4 * lane + i] : make_float2(0.f, 0.f);
                x[i] = static_cast<double>(y.x) + static_cast<double>(y.y);
                upto += x[i];
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {  // of this lane's segments and those before
                const double y = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += y;
            }
            const double goal = static_cast<double>(sh.u[0]) * __shfl_sync(0xffffffffu, upto, 31);
            double before = __shfl_up_sync(0xffffffffu, upto, 1);
            if (lane == 0) before = 0.0;
            // the first segment whose sum passes the goal, and (where a rounding leaves none) the last with weight
            int first = 1 << 20, last = -1;
            double first_below = 0.0, last_below = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const double with = before + x[i];
                if (x[i] > 0.0) {
                    last = 4 * lane + i;
                    last_below = before;
                    if (first == 1 << 20 && with > goal) {
                        first = 4 * lane + i;
                        first_below = before;
                    }
                }
                before = with;
            }
            const int least = __reduce_min_sync(0xffffffffu, first);
            const int most = __reduce_max_sync(0xffffffffu, last);
            const int found = least < 1 << 20 ? least : most;
            if (found < 0 ? lane == 0 : found / 4 == lane) {
                sh.found = found;
                sh.goal = goal;
                sh.below = least < 1 << 20 ? first_below : last_below;
            }
        }
        __syncthreads();
        if (sh.found >= 0) break;
        // No weight at all: the target's own probabilities (a second time: there is no token).
        if (!draft && refusals == 0) break;
        draft = nullptr;
        refusals = 0;
        cluster_arrive();  // (the sums have been read everywhere before they are written again)
        cluster_wait();
    }
    if (count == 0) return;
    const int64_t o = static_cast<int64_t>(b) * p.max_q_len + count - 1;
    if (sh.found < 0) {
        if (rank == 0 && tid == 0) p.tokens_out[o] = -1;
        return;
    }
    if (sh.found / kVerifyWarps != static_cast<int>(rank)) return;

    // ---- the token within the segment, by its CTA: four entries a thread, 2048 at a time ----
    const float2 goal = pair(sh.goal);
    const int from = static_cast<int>(min(static_cast<int64_t>(sh.found) * p.segment, static_cast<int64_t>(p.vocab)));
    const int to = static_cast<int>(min(static_cast<int64_t>(sh.found + 1) * p.segment, static_cast<int64_t>(p.vocab)));
    float2 below = pair(sh.below);
    int token = -1;
    for (int v0 = from; v0 < to; v0 += 4 * kVerifyThreads) {
        const int v = v0 + 4 * tid;
        const uint32_t gone = refused_from(v);
        float2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = v + i < to && !((gone >> i) & 1) ? weight(target, draft, v + i) : make_float2(0.f, 0.f);
        const float2 scan = scan_lanes(plus(plus(w[0], w[1]), plus(w[2], w[3])), lane, 32);
        if (lane == 31) sh.warp_sums[warp] = scan;
        __syncthreads();
        const float2 warps_upto = scan_lanes(sh.warp_sums[lane & (kVerifyWarps - 1)], lane & (kVerifyWarps - 1), kVerifyWarps);
        auto warps = [&](int i) {
            return make_float2(__shfl_sync(0xffffffffu, warps_upto.x, i), __shfl_sync(0xffffffffu, warps_upto.y, i));
        };
        const float2 before_warp = warps(max(warp - 1, 0)), before_lane = shuffle_up(scan, 1);
        float2 at = below;
        if (warp > 0) at = plus(at, before_warp);
        if (lane > 0) at = plus(at, before_lane);
        below = plus(below, warps(kVerifyWarps - 1));
        int pass = -1, some = -1;  // of this thread's entries
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            at = plus(at, w[i]);
            if (w[i].x > 0.f) {
                some = v + i;
                if (pass < 0 && above(at, goal)) pass = v + i;
            }
        }
        const uint32_t passes = __ballot_sync(0xffffffffu, pass >= 0), with = __ballot_sync(0xffffffffu, some >= 0);
        const int first = __shfl_sync(0xffffffffu, pass, passes ? __ffs(passes) - 1 : 0);
        const int last = __shfl_sync(0xffffffffu, some, with ? 31 - __clz(with) : 0);
        if (lane == 0) {
            sh.passes[warp] = passes ? first : -1;
            sh.some[warp] = with ? last : -1;
        }
        __syncthreads();
        // the first entry that passes, or (should a rounding leave none) the last with weight
        const int pass_w = sh.passes[lane & (kVerifyWarps - 1)], some_w = sh.some[lane & (kVerifyWarps - 1)];
        const uint32_t hit = __ballot_sync(0xffffffffu, lane < kVerifyWarps && pass_w >= 0);
        const uint32_t any = __ballot_sync(0xffffffffu, lane < kVerifyWarps && some_w >= 0);
        if (hit)
            token = __shfl_sync(0xffffffffu, pass_w, __ffs(hit) - 1);
        else if (any)
            token = __shfl_sync(0xffffffffu, some_w, 31 - __clz(any));
        if (hit) break;
    }
    if (tid == 0) p.tokens_out[o] = token;
}

// ---- compaction ----------------------------------------------------------------------
// One CTA moves 256 of the 16-byte pieces of a token's rows (K and V, every head) along the
// path: node path[i] to place i, i = 1, 2, ..  Parents come before their children, so
// path[i] >= i: a place that is written is never read for a later node, and a thread that reads eight
// nodes before it writes them keeps that order.
constexpr int kCompactBatch = 8;
__global__ void __launch_bounds__(256) kv_compact_path_kernel(const CompactParams p, int row_vecs) {
    __shared__ int32_t from[kMaxTreeNodes], to[kMaxTreeNodes];  // blocks (-1: nothing moves)
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int count = __ldg(p.counts + b);
    const int n = __ldg(p.cu_q_lens + b + 1) - __ldg(p.cu_q_lens + b);
    const int ctx = __ldg(p.context_lens + b);
    if (count <= 1) return;
    if (n < count || n > kMaxTreeNodes || count > p.path_len || ctx < n || ctx > p.max_blocks * kBlockSize) {
        if (blockIdx.y == 0 && tid == 0 && p.status)
            atomicOr(p.status, ctx < 1 || ctx > p.max_blocks * kBlockSize ? kStatusBadContextLen : kStatusBadQLen);
        return;
    }
    if (tid > 0 && tid < count) {
        const int node = __ldg(p.path + static_cast<int64_t>(b) * p.path_len + tid);
        const int32_t *table = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
        from[tid] = to[tid] = -1;
        if (node < tid || node >= n) {
            if (blockIdx.y == 0 && p.status) atomicOr(p.status, kStatusBadQLen);
        } else if (node > tid) {
            const int s = ctx - n + node, d = ctx - n + tid;
            const int sb = __ldg(table + s / kBlockSize), db = __ldg(table + d / kBlockSize);
            if (static_cast<unsigned>(sb) < static_cast<unsigned>(p.num_blocks) &&
                static_cast<unsigned>(db) < static_cast<unsigned>(p.num_blocks)) {
                from[tid] = sb;
                to[tid] = db;
            } else if (blockIdx.y == 0 && p.status) {
                atomicOr(p.status, kStatusBadBlockId);
            }
        }
    }
    __syncthreads();
    // This thread's piece: cache (K, V), head, vector; the scales of an FP8 pool are one more piece of 4 bytes.
    const int per_cache = p.n_kv * row_vecs;
    const int64_t item = static_cast<int64_t>(blockIdx.y) * blockDim.x + tid;
    if (item >= 2 * per_cache) return;
    const bool is_v = item >= per_cache;
    const int r = static_cast<int>(item - (is_v ? per_cache : 0));
    const int h = r / row_vecs, vec = r - h * row_vecs;
    uint4 *cache = static_cast<uint4 *>(is_v ? p.v_cache : p.k_cache);
    float *scale = vec == 0 ? (is_v ? p.v_scale : p.k_scale) : nullptr;
    const int start = ctx - n;
    const int32_t *path = p.path + static_cast<int64_t>(b) * p.path_len;
    for (int i0 = 1; i0 < count; i0 += kCompactBatch) {
        uint4 x[kCompactBatch];
        float sc[kCompactBatch];
#pragma unroll
        for (int k = 0; k < kCompactBatch; ++k) {
            const int i = i0 + k;
            if (i >= count || from[i] < 0) continue;
            const int64_t row = (static_cast<int64_t>(from[i]) * p.n_kv + h) * kBlockSize +
                                ((start + __ldg(path + i)) & (kBlockSize - 1));
            x[k] = cache[row * row_vecs + vec];
            if (scale) sc[k] = scale[row];
        }
#pragma unroll
        for (int k = 0; k < kCompactBatch; ++k) {
            const int i = i0 + k;
            if (i >= count || from[i] < 0) continue;
            const int64_t row = (static_cast<int64_t>(to[i]) * p.n_kv + h) * kBlockSize + ((start + i) & (kBlockSize - 1));
            cache[row * row_vecs + vec] = x[k];
            if (scale) scale[row] = sc[k];
        }
    }
}

}  // namespace

cudaError_t launch_speculative_verify(const SpecVerifyParams &p, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * cluster);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, speculative_verify_kernel, p);
}

cudaError_t launch_kv_compact_path(const CompactParams &p, bool fp8, cudaStream_t stream) {
    const int row_vecs = kHeadDim * (fp8 ? 1 : 2) / 16;
    const int64_t items = 2LL * p.n_kv * row_vecs;
    return launch_pdl(kv_compact_path_kernel, dim3(p.num_seqs, static_cast<unsigned>((items + 255) / 256)), dim3(256), 0,
                      stream, p, row_vecs);
}

}  // namespace pkv
