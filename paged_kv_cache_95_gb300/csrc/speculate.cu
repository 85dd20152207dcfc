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
// nearly.  The sums over the vocabulary are error-free pairs of fp32 (high part and
// remainder, 2^-48), joined in fp64: the same token as sums in fp64 but for borders closer than
// that, without the slow fp64 pipe (two additions a clock and SM: 64 rows of 128000 would take
// it 14 us).
//
// One cluster of up to 8 CTAs takes a sequence: each warp sums one segment of the vocabulary, the
// segment sums are exchanged through distributed shared memory, and the one warp whose segment
// holds the drawn token reads that segment (a few KB, in cache) a second time.  HBM bound for
// batches (one row of p and one of q a sequence), latency bound for few sequences: three
// dependent reads (lengths, tokens, probabilities) come before the row.
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
// A double into another CTA's copy of this CTA's shared-memory address.
__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t rank, double v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(v) : "memory");
}

// A probability as it counts: NaN and below 0 as 0, above 1 as 1 (so sums stay finite).
__device__ __forceinline__ float weigh(float p) { return fminf(fmaxf(p, 0.f), 1.f); }

// hi + lo += x without error in hi (the error of each addition goes to lo).
__device__ __forceinline__ void add_exact(float &hi, float &lo, float x) {
    const float sum = __fadd_rn(hi, x);
    const float part = __fsub_rn(sum, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, part)), __fsub_rn(x, part)));
    hi = sum;
}

// The weight of entry v in fp64 (exact: a difference of two fp32 numbers of [0, 1] that are
// not tiny against each other; else its rounding is below 2^-53 of the larger).
__device__ __forceinline__ double weight64(const float *p, const float *q, int v) {
    const double w = static_cast<double>(weigh(__ldg(p + v)));
    if (!q) return w;
    const double d = w - static_cast<double>(weigh(__ldg(q + v)));
    return d > 0.0 ? d : 0.0;
}

struct VerifyShared {
    double sums[kSegments];  // of every segment of the cluster
    double p[kMaxTreeNodes], q[kMaxTreeNodes];
    float u[kMaxTreeNodes];
    int32_t token[kMaxTreeNodes], parent[kMaxTreeNodes];
    int32_t path[kMaxTreeNodes];
    int32_t refused[kMaxTreeNodes];  // tokens that have no weight left
    int32_t count, refusals, found;
    double goal;  // what the draw leaves to the segment: u_0 sum w less the weights before it
};

__global__ void __launch_bounds__(kVerifyThreads) speculative_verify_kernel(const SpecVerifyParams p) {
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
        sh.p[j] = ok ? static_cast<double>(weigh(__ldg(p.target + at * p.target_row + token))) : 0.0;
        sh.q[j] = ok && p.draft ? static_cast<double>(weigh(__ldg(p.draft + at * p.draft_row + token))) : 0.0;
    }
    cluster_wait();
    __syncthreads();

    // ---- the walk: warp 0, every lane alike ----
    if (warp == 0) {
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
                if (!p.draft) {  // a token refused before has no probability left
                    const bool gone = (lane < refusals && sh.refused[lane] == token) ||
                                      (lane + 32 < refusals && sh.refused[lane + 32] == token);
                    if (__any_sync(0xffffffffu, gone)) pj = 0.0;
                }
                if (static_cast<double>(sh.u[j]) * (p.draft ? sh.q[j] : rest) < pj) {
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
    auto is_refused = [&](int v) {
        bool gone = false;
        for (int i = 0; i < refusals; ++i) gone = gone || sh.refused[i] == v;
        return gone;
    };

    for (int attempt = 0; attempt < 2 && count > 0; ++attempt) {
        // ---- the segment's sum ----
        float h0 = 0.f, l0 = 0.f, h1 = 0.f, l1 = 0.f;
        bool here = false;  // a refused token lies in this segment
        for (int i = lane; i < refusals; i += 32) here = here || (sh.refused[i] >= lo && sh.refused[i] < hi);
        here = __any_sync(0xffffffffu, here);
        auto add = [&](float pv, float qv, float &h, float &l) {
            pv = weigh(pv);
            qv = weigh(qv);
            if (pv > qv) {
                add_exact(h, l, pv);
                if (draft) add_exact(h, l, -qv);
            }
        };
        const bool wide = ((reinterpret_cast<uintptr_t>(target) | (draft ? reinterpret_cast<uintptr_t>(draft) : 0)) & 15) == 0;
        if (!here && wide) {  // (lo is a multiple of 4)
            const int full = lo + ((hi - lo) & ~3);
#pragma unroll 4
            for (int v = lo + 4 * lane; v < full; v += 128) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(target + v));
                const float4 y = draft ? __ldg(reinterpret_cast<const float4 *>(draft + v)) : make_float4(0.f, 0.f, 0.f, 0.f);
                add(x.x, y.x, h0, l0);
                add(x.y, y.y, h1, l1);
                add(x.z, y.z, h0, l0);
                add(x.w, y.w, h1, l1);
            }
            const int v = full + lane;
            if (v < hi) add(__ldg(target + v), draft ? __ldg(draft + v) : 0.f, h0, l0);
        } else {
#pragma unroll 4
            for (int v = lo + lane; v < hi; v += 32) {
                const float x = __ldg(target + v), y = draft ? __ldg(draft + v) : 0.f;
                if (!here || !is_refused(v)) add(x, y, h0, l0);
            }
        }
        double sum = (static_cast<double>(h0) + static_cast<double>(h1)) + (static_cast<double>(l0) + static_cast<double>(l1));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane < static_cast<int>(ctas)) store_remote(smem_u32(&sh.sums[seg]), lane, sum);
        cluster_arrive();
        cluster_wait();

        // ---- the segment that the draw falls into (warp 0 of every CTA, alike) ----
        if (warp == 0) {
            double x[4], total = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = 4 * lane + i;
                x[i] = s < segments ? sh.sums[s] : 0.0;
                total += x[i];
            }
            double upto = total;  // of this lane's segments and those before
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += y;
            }
            total = __shfl_sync(0xffffffffu, upto, 31);
            const double goal = static_cast<double>(sh.u[0]) * total;
            double before = __shfl_up_sync(0xffffffffu, upto, 1);
            if (lane == 0) before = 0.0;
            // the first segment whose sum passes the goal, and (where a rounding leaves none) the last with weight
            int first = 1 << 20, last = -1;
            double first_below = 0.0, last_below = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = 4 * lane + i;
                if (x[i] > 0.0) {
                    last = s;
                    last_below = before;
                }
                if (first == 1 << 20 && x[i] > 0.0 && before + x[i] > goal) {
                    first = s;
                    first_below = before;
                }
                before += x[i];
            }
            const int least = __reduce_min_sync(0xffffffffu, first);
            const int most = __reduce_max_sync(0xffffffffu, last);
            const int found = least < 1 << 20 ? least : most;
            if (found < 0 ? lane == 0 : found / 4 == lane) {
                sh.found = found;
                sh.goal = goal - (least < 1 << 20 ? first_below : last_below);
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
    if (sh.found != seg) return;

    // ---- the token within the segment, by this warp ----
    const double goal = sh.goal;
    auto entry = [&](int v) { return v < hi && !(refusals > 0 && is_refused(v)) ? weight64(target, draft, v) : 0.0; };
    // Lane l's share is the l-th run of `run` entries; the run that passes the goal is then spread over the lanes.
    const int run = (p.segment / 32 + 3) / 4 * 4;
    const int mine = lo + lane * run;
    double s0 = 0.0, s1 = 0.0;
    for (int v = mine; v < mine + run; v += 2) {
        s0 += entry(v);
        s1 += entry(v + 1);
    }
    const double share = s0 + s1;
    double scan = share;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, scan, off);
        if (lane >= off) scan += y;
    }
    const uint32_t some = __ballot_sync(0xffffffffu, share > 0.0);
    const uint32_t pass = __ballot_sync(0xffffffffu, share > 0.0 && scan > goal);
    const int who = pass ? __ffs(pass) - 1 : some ? 31 - __clz(some) : 0;
    double below = __shfl_sync(0xffffffffu, scan - share, who);
    int token = -1;
    for (int v0 = lo + who * run; v0 < lo + (who + 1) * run; v0 += 32) {
        const int v = v0 + lane;
        const double w = v < lo + (who + 1) * run ? entry(v) : 0.0;
        double at = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, at, off);
            if (lane >= off) at += y;
        }
        const uint32_t has = __ballot_sync(0xffffffffu, w > 0.0);
        const uint32_t hit = __ballot_sync(0xffffffffu, w > 0.0 && below + at > goal);
        if (hit) {
            token = v0 + __ffs(hit) - 1;
            break;
        }
        if (has) token = v0 + 31 - __clz(has);  // (the last with weight, should a rounding leave none)
        below += __shfl_sync(0xffffffffu, at, 31);
    }
    if (lane == 0) p.tokens_out[o] = token;
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
