// Append and release on the device block pool: block tables, context lengths,
// slot map, query starts and copy-on-write pairs of a serving step, made on
// the GPU from the sequences' lengths.
//
// The result is that of the host pool's calls one sequence after another
// ([P2 "PagedAttention原理与KV Cache显存优化", §3.3-§3.4 and §4.2: a new block
// when the cached count is a multiple of the block size, blocks freed at count
// 0]; [P4 "PagedAttention 实现细节", §3.3: the copy-on-write rule]); the
// kernels reach it in parallel:
//   append   sequence s takes cow_s + ceil((L + n) / bs) - ceil(L / bs) blocks,
//            which are consecutive in the order the free list is handed out, so
//            an exclusive scan over the sequences gives every take its place
//            in the list. Of the sequences that write into a shared block, all
//            copy it but the last one in order, and that one too while somebody
//            else still holds the block (count > writers).
//   release  a block is freed at its last drop, the largest (sequence, entry)
//            place that holds it, if all its holders drop it; a scan of those
//            marks over the places gives each freed block its place at the
//            list's back.
// Everything is checked before anything changes.
//
// One launch of one thread-block cluster: the phases are separated by the
// cluster's hardware barrier, which needs no counter in memory and cannot be
// left waiting by a CTA that is not resident. All that a step moves is a few
// bytes per sequence, block and token, so latency bounds it, not bandwidth.
#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_dpool.cuh"
#include "pa_internal.h"

namespace pa {
namespace dpool {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;  // the largest portable cluster
constexpr int kPer = PA_DPOOL_MAX_SEQS / kThreads;  // sequences per thread, at most
static_assert(kPer * kThreads == PA_DPOOL_MAX_SEQS, "a thread holds a run of whole sequences");

struct AppendParams {
    int32_t *state;
    int32_t *tables;
    int32_t *ctx;
    const int32_t *new_lens;
    int32_t *q_start;
    int32_t *slots;
    int64_t *cow_pairs;
    int32_t *num_cow;
    int num_seqs;
    int max_blocks;
    int max_tokens;
    int num_blocks;
    int block_size;
    unsigned int *err;
};

struct ReleaseParams {
    int32_t *state;
    int32_t *tables;
    int32_t *ctx;
    const int32_t *finished;
    int num_seqs;
    int max_blocks;
    int num_blocks;
    int block_size;
    unsigned int *err;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Whether `state` is a sound pool of these sizes.
__device__ __forceinline__ bool header_ok(const Pool &p, int nb, int bs) {
    return __ldcg(p.hdr + 5) == kMagic && __ldcg(p.hdr) == nb && __ldcg(p.hdr + 1) == bs;
}

template <typename T> __device__ __forceinline__ T warp_inclusive(T v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Exclusive scan of one value per thread over the CTA; *total receives the
// sum. `sums` holds kWarps + 1 values; the call ends with a CTA barrier.
template <typename T> __device__ T block_exclusive(T v, T *sums, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T inc = warp_inclusive(v, lane);
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const T w = sums[lane];
        const T wi = warp_inclusive(w, lane);
        sums[lane] = wi - w;
        if (lane == 31) sums[kWarps] = wi;
    }
    __syncthreads();
    const T r = sums[warp] + inc - v;
    *total = sums[kWarps];
    __syncthreads();
    return r;
}

// The largest s in [0, n) with pre[s] <= k (pre non-decreasing, pre[0] = 0 <= k).
__device__ __forceinline__ int find_run(const int *pre, int n, int k) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= k) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ------------------------------------------------------------------ append

__global__ void __launch_bounds__(kThreads, 1) append_kernel(const AppendParams q) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x;
    const int S = q.num_seqs, MB = q.max_blocks, nb = q.num_blocks, bs = q.block_size;
    // every CTA works out every sequence; the ones a CTA's output threads
    // answer for (marks, per-sequence outputs) are those of its slice
    const bool mine = tid / (kThreads / ctas) == rank;
    const int gtid = rank * kThreads + tid, gstep = ctas * kThreads;

    extern __shared__ int dyn[];
    int *tok_pre = dyn;                  // [S + 1] new tokens before sequence s
    int *take_pre = tok_pre + S + 1;     // [S + 1] blocks taken before sequence s
    int *ctx_cow = take_pre + S + 1;     // [S] context length, sign bit: its last block is copied
    __shared__ long long sums[kWarps + 1];

    const Pool p = views(q.state, nb);
    int bad = 0;  // PA_DEVERR_* bits
    auto refuse = [&]() {  // nothing is applied: outputs that make the step's other calls do nothing
        for (int i = gtid; i <= S; i += gstep) q.q_start[i] = 0;
        for (int i = gtid; i < q.max_tokens; i += gstep) q.slots[i] = -1;
        for (int i = gtid; i < 2 * S; i += gstep) q.cow_pairs[i] = -1;
        if (gtid == 0) *q.num_cow = 0;
    };
    if (!header_ok(p, nb, bs)) {  // the same in every CTA: the header changes behind the cluster's barriers
        if (gtid == 0) record_error(q.err, PA_DEVERR_POOL);
        refuse();
        return;
    }
    const int policy = __ldcg(p.hdr + 2), head = __ldcg(p.hdr + 3), count = __ldcg(p.hdr + 4);

    // ---- lengths, and who writes into which partly filled block
    const int per = (S + kThreads - 1) / kThreads;
    const int s0 = tid * per, s1 = min(S, s0 + per);
    int ctx[kPer], nw[kPer], blk[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = s0 + i;
        ctx[i] = nw[i] = 0;
        blk[i] = -1;
        if (s >= s1) continue;
        const int c = __ldcg(q.ctx + s), n = __ldg(q.new_lens + s);
        if (c < 0 || n < 0 || c > (long long)MB * bs) {
            bad |= PA_DEVERR_CONTEXT;
            continue;
        }
        if ((long long)c + n > (long long)MB * bs) {
            bad |= PA_DEVERR_POOL;
            continue;
        }
        ctx[i] = c;
        nw[i] = n;
        if (n > 0 && c % bs != 0) {
            const int b = __ldcg(q.tables + (size_t)s * MB + c / bs);
            if (b < 0 || b >= nb) {
                bad |= PA_DEVERR_BLOCK_ID;
                continue;
            }
            if (__ldcg(p.ref + b) < 1) {
                bad |= PA_DEVERR_POOL;
                continue;
            }
            blk[i] = b;
            if (mine) {
                atomicAdd(p.writers + b, 1);
                atomicMax(p.last_writer + b, s);
            }
        }
    }
    cluster.sync();

    // ---- takes and their places; the same in every CTA
    long long tok = 0;
    int takes = 0, cows = 0;
    bool cow[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        cow[i] = false;
        if (blk[i] >= 0) {
            const int r = __ldcg(p.ref + blk[i]), w = __ldcg(p.writers + blk[i]);
            if (w > r) bad |= PA_DEVERR_POOL;  // more tables hold the block than its count says
            cow[i] = r > 1 && !(w == r && __ldcg(p.last_writer + blk[i]) == s0 + i);
        }
        tok += nw[i];
        takes += (int)cow[i] + ceil_div(ctx[i] + nw[i], bs) - ceil_div(ctx[i], bs);
        cows += cow[i];
    }
    // takes and cows are below 2^30 (sequences x table entries): one 64-bit scan for both
    long long all_tok, all_tc;
    long long tok_at = block_exclusive<long long>(tok, sums, &all_tok);
    const long long tc_at = block_exclusive<long long>(((long long)takes << 32) | (unsigned)cows, sums, &all_tc);
    int take_at = (int)(tc_at >> 32), cow_at = (int)(unsigned)tc_at;
    const int all_takes = (int)(all_tc >> 32), all_cows = (int)(unsigned)all_tc;
    if (all_tok > q.max_tokens || all_takes > count) bad |= PA_DEVERR_POOL;
    if (bad) record_error(q.err, (unsigned)bad);
    bad = __syncthreads_or(bad);  // nonzero in every thread of every CTA, or in none
    if (!bad) {
        int t = (int)tok_at, k = take_at;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int s = s0 + i;
            if (s >= s1) continue;
            tok_pre[s] = t;
            take_pre[s] = k;
            ctx_cow[s] = cow[i] ? (ctx[i] | (int)0x80000000) : ctx[i];
            t += nw[i];
            k += (int)cow[i] + ceil_div(ctx[i] + nw[i], bs) - ceil_div(ctx[i], bs);
        }
        if (tid == 0) {
            tok_pre[S] = (int)all_tok;
            take_pre[S] = all_takes;
        }
    }
    cluster.sync();  // every CTA has read lengths, counts and marks, and its shared arrays are written

#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (mine && blk[i] >= 0) {
            p.writers[blk[i]] = 0;
            p.last_writer[blk[i]] = -1;
        }
    if (bad) {
        refuse();
        return;
    }

    // ---- apply. Block k of the step's takes:
    const long long first = policy == PA_POOL_FIFO ? head : (long long)head + count - 1;
    auto block_of = [&](int k) -> int {
        const long long at = policy == PA_POOL_FIFO ? first + k : first - k;
        return __ldcg(p.ring + at % nb);
    };
    if (mine) {
        int t = (int)tok_at, k = take_at;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int s = s0 + i;
            if (s >= s1) continue;
            q.q_start[s] = t;
            q.ctx[s] = ctx[i] + nw[i];
            if (cow[i]) {
                const int id = block_of(k);
                atomicSub(p.ref + blk[i], 1);
                reinterpret_cast<longlong2 *>(q.cow_pairs)[cow_at] = make_longlong2(blk[i], id);
                ++cow_at;
            }
            t += nw[i];
            k += (int)cow[i] + ceil_div(ctx[i] + nw[i], bs) - ceil_div(ctx[i], bs);
        }
    }
    for (int i = all_cows + gtid; i < S; i += gstep)
        reinterpret_cast<longlong2 *>(q.cow_pairs)[i] = make_longlong2(-1, -1);
    for (int k = gtid; k < all_takes; k += gstep) {
        const int s = find_run(take_pre, S, k);
        const int c = ctx_cow[s] & 0x7fffffff, cw = ctx_cow[s] < 0;
        const int id = block_of(k);
        // the copy of the last block (if any) is the sequence's first take
        const int j = k - take_pre[s] < cw ? c / bs : ceil_div(c, bs) + k - take_pre[s] - cw;
        q.tables[(size_t)s * MB + j] = id;
        p.ref[id] = 1;
    }
    for (int t = gtid; t < q.max_tokens; t += gstep) {
        int slot = -1;
        if (t < all_tok) {
            const int s = find_run(tok_pre, S, t);
            const int c = ctx_cow[s] & 0x7fffffff, cw = ctx_cow[s] < 0;
            const int pos = c + t - tok_pre[s];
            const int j = pos / bs, have = ceil_div(c, bs);
            int id;
            if (j >= have) id = block_of(take_pre[s] + cw + j - have);
            else if (cw) id = block_of(take_pre[s]);
            else id = __ldcg(q.tables + (size_t)s * MB + j);  // kept: no thread writes this entry
            slot = id * bs + (pos - j * bs);
        }
        q.slots[t] = slot;
    }
    if (gtid == 0) {
        q.q_start[S] = (int)all_tok;
        *q.num_cow = all_cows;
        if (policy == PA_POOL_FIFO) p.hdr[3] = (int)(((long long)head + all_takes) % nb);
        p.hdr[4] = count - all_takes;
    }
}

// ----------------------------------------------------------------- release

__global__ void __launch_bounds__(kThreads, 1) release_kernel(const ReleaseParams q) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = q.num_seqs, MB = q.max_blocks, nb = q.num_blocks, bs = q.block_size;

    extern __shared__ int dyn[];
    int *item_pre = dyn;             // [S + 1] 32-entry items before sequence s
    int *entries = item_pre + S + 1; // [S] entries sequence s drops
    __shared__ int sums[kWarps + 1];
    __shared__ int s_bad[kCluster], s_freed[kCluster];  // of every CTA, written by each into all

    const Pool p = views(q.state, nb);
    int bad = 0;  // PA_DEVERR_* bits
    if (!header_ok(p, nb, bs)) {  // the same in every CTA, as in append_kernel
        if (rank == 0 && tid == 0) record_error(q.err, PA_DEVERR_POOL);
        return;
    }
    const int head = __ldcg(p.hdr + 3), count = __ldcg(p.hdr + 4);

    // ---- the items, in sequence order: 32 consecutive table entries of one
    // sequence each; a warp takes a run of consecutive items
    const int per = (S + kThreads - 1) / kThreads;
    const int s0 = tid * per, s1 = min(S, s0 + per);
    int n[kPer], items = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = s0 + i;
        n[i] = 0;
        if (s >= s1 || __ldg(q.finished + s) == 0) continue;
        const int c = __ldcg(q.ctx + s);
        if (c < 0 || c > (long long)MB * bs) {
            bad |= PA_DEVERR_CONTEXT;
            continue;
        }
        n[i] = ceil_div(c, bs);
        items += (n[i] + 31) / 32;
    }
    int all_items;
    int at = block_exclusive<int>(items, sums, &all_items);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = s0 + i;
        if (s >= s1) continue;
        item_pre[s] = at;
        entries[s] = n[i];
        at += (n[i] + 31) / 32;
    }
    if (tid == 0) item_pre[S] = all_items;
    __syncthreads();
    const int gwarp = rank * kWarps + warp, warps = ctas * kWarps;
    const int i0 = (int)((long long)all_items * gwarp / warps), i1 = (int)((long long)all_items * (gwarp + 1) / warps);
    const int seq0 = i0 < i1 ? find_run(item_pre, S, i0) : 0;
    // calls f(place, table entry pointer, block id) for this lane's entries, in order; f runs in all 32 lanes
    // (pointer null where the lane has no entry)
    auto each = [&](auto f) {
        int s = seq0;
        for (int it = i0; it < i1; ++it) {
            while (item_pre[s + 1] <= it) ++s;
            const int j = (it - item_pre[s]) * 32 + lane;
            int32_t *e = j < entries[s] ? q.tables + (size_t)s * MB + j : nullptr;
            const int id = e ? __ldcg(e) : -1;
            f(it * 32 + lane, e, id);
        }
    };

    // ---- drops per block and the last place that drops it
    each([&](int place, int32_t *e, int id) {
        if (!e) return;
        if (id < 0 || id >= nb) {
            bad |= PA_DEVERR_BLOCK_ID;
            return;
        }
        if (__ldcg(p.ref + id) < 1) bad |= PA_DEVERR_POOL;
        atomicAdd(p.delta + id, 1);
        atomicMax(p.last_old + id, place);
    });
    cluster.sync();

    // ---- freed blocks, counted in place order
    int freed = 0;
    auto valid = [&](int32_t *e, int id) { return e && id >= 0 && id < nb; };
    each([&](int place, int32_t *e, int id) {
        bool f = false;
        if (valid(e, id)) {
            const int d = __ldcg(p.delta + id), r = __ldcg(p.ref + id);
            if (d > r) bad |= PA_DEVERR_POOL;
            f = d == r && __ldcg(p.last_old + id) == place;
        }
        freed += __popc(__ballot_sync(0xffffffffu, f));
    });
    int cta_freed;
    int base = block_exclusive<int>(lane == 0 ? freed : 0, sums, &cta_freed);
    base = __shfl_sync(0xffffffffu, base, 0);
    if (bad) record_error(q.err, (unsigned)bad);
    bad = __syncthreads_or(bad);
    if (tid < ctas) {
        *cluster.map_shared_rank(s_bad + rank, tid) = bad;
        *cluster.map_shared_rank(s_freed + rank, tid) = cta_freed;
    }
    cluster.sync();
    int all_freed = 0;
    bad = 0;
    for (int r = 0; r < ctas; ++r) {
        bad |= s_bad[r];
        if (r < rank) base += s_freed[r];
        all_freed += s_freed[r];
    }
    if (!bad && (long long)count + all_freed > nb) {  // a free list that cannot be
        if (rank == 0 && tid == 0) record_error(q.err, PA_DEVERR_POOL);
        bad = 1;
    }

    // ---- apply: a block's last place lowers its count and, if it frees the block, hands it back
    if (!bad) {
        each([&](int place, int32_t *e, int id) {
            bool f = false;
            if (e && __ldcg(p.last_old + id) == place) {
                const int d = __ldcg(p.delta + id), r = __ldcg(p.ref + id);
                f = d == r;
                p.ref[id] = r - d;
            }
            const unsigned m = __ballot_sync(0xffffffffu, f);
            if (f) p.ring[((long long)head + count + base + __popc(m & ((1u << lane) - 1u))) % nb] = id;
            base += __popc(m);
        });
    }
    cluster.sync();  // every CTA is done with the marks and the lengths

    each([&](int, int32_t *e, int id) {
        if (!valid(e, id)) return;
        p.delta[id] = 0;
        p.last_old[id] = -1;
        if (!bad) *e = -1;
    });
    if (!bad && tid / (kThreads / ctas) == rank) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (s0 + i < s1 && __ldg(q.finished + s0 + i) != 0) q.ctx[s0 + i] = 0;
    }
    if (rank == 0 && tid == 0) {
        if (!bad) p.hdr[4] = count + all_freed;
    }
}

// -------------------------------------------------------------------- host

template <typename P>
static cudaError_t launch_cluster(void (*kern)(P), const P &q, int smem, AttrCache *attr, int smem_max,
                                  cudaStream_t stream) {
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem_max, attr);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, q);
}

static bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Sizes shared by the two calls.
static int check_sizes(int num_blocks, int block_size, int max_blocks_per_seq, int num_seqs) {
    if (num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 || num_seqs < 0 ||
        num_seqs > PA_DPOOL_MAX_SEQS || num_blocks > INT32_MAX / PA_DPOOL_ARRAYS)
        return PA_ERR_SHAPE;
    if ((long long)num_seqs * max_blocks_per_seq >= (1LL << 30) || (long long)num_blocks * block_size >= INT32_MAX ||
        (long long)max_blocks_per_seq * block_size >= INT32_MAX)
        return PA_ERR_SHAPE;
    return PA_OK;
}

}  // namespace dpool
}  // namespace pa

using namespace pa;

extern "C" int pa_dpool_append(void *state, int num_blocks, int block_size, int32_t *block_tables,
                               int max_blocks_per_seq, int32_t *context_lens, const int32_t *new_lens, int num_seqs,
                               int32_t *q_start, int32_t *slot_mapping, int max_tokens, int64_t *cow_pairs,
                               int32_t *num_cow, cudaStream_t stream) {
    int rc = dpool::check_sizes(num_blocks, block_size, max_blocks_per_seq, num_seqs);
    if (rc != PA_OK) return rc;
    if (max_tokens < 0) return PA_ERR_SHAPE;
    if (!state || !q_start || !num_cow || (max_tokens > 0 && !slot_mapping) ||
        (num_seqs > 0 && (!block_tables || !context_lens || !new_lens || !cow_pairs)))
        return PA_ERR_NULL;
    if (!dpool::aligned(state, 16) || !dpool::aligned(block_tables, 4) || !dpool::aligned(context_lens, 4) ||
        !dpool::aligned(new_lens, 4) || !dpool::aligned(q_start, 4) || !dpool::aligned(slot_mapping, 4) ||
        !dpool::aligned(cow_pairs, 16) || !dpool::aligned(num_cow, 4))
        return PA_ERR_ALIGN;
    dpool::AppendParams q{};
    if (device_error_word(&q.err) != cudaSuccess) return PA_ERR_CUDA;
    q.state = static_cast<int32_t *>(state);
    q.tables = block_tables;
    q.ctx = context_lens;
    q.new_lens = new_lens;
    q.q_start = q_start;
    q.slots = slot_mapping;
    q.cow_pairs = cow_pairs;
    q.num_cow = num_cow;
    q.num_seqs = num_seqs;
    q.max_blocks = max_blocks_per_seq;
    q.max_tokens = max_tokens;
    q.num_blocks = num_blocks;
    q.block_size = block_size;
    static AttrCache attr;
    constexpr int kMax = (3 * PA_DPOOL_MAX_SEQS + 2) * 4;
    cudaError_t e = dpool::launch_cluster(dpool::append_kernel, q, (3 * num_seqs + 2) * 4, &attr, kMax, stream);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" int pa_dpool_release(void *state, int num_blocks, int block_size, int32_t *block_tables,
                                int max_blocks_per_seq, int32_t *context_lens, const int32_t *finished, int num_seqs,
                                cudaStream_t stream) {
    int rc = dpool::check_sizes(num_blocks, block_size, max_blocks_per_seq, num_seqs);
    if (rc != PA_OK) return rc;
    if (!state || (num_seqs > 0 && (!block_tables || !context_lens || !finished))) return PA_ERR_NULL;
    if (!dpool::aligned(state, 16) || !dpool::aligned(block_tables, 4) || !dpool::aligned(context_lens, 4) ||
        !dpool::aligned(finished, 4))
        return PA_ERR_ALIGN;
    if (num_seqs == 0) return PA_OK;
    dpool::ReleaseParams q{};
    if (device_error_word(&q.err) != cudaSuccess) return PA_ERR_CUDA;
    q.state = static_cast<int32_t *>(state);
    q.tables = block_tables;
    q.ctx = context_lens;
    q.finished = finished;
    q.num_seqs = num_seqs;
    q.max_blocks = max_blocks_per_seq;
    q.num_blocks = num_blocks;
    q.block_size = block_size;
    static AttrCache attr;
    constexpr int kMax = (2 * PA_DPOOL_MAX_SEQS + 1) * 4;
    cudaError_t e = dpool::launch_cluster(dpool::release_kernel, q, (2 * num_seqs + 1) * 4, &attr, kMax, stream);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
