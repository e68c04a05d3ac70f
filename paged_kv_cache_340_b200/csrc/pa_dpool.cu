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
#include "pa_pdl.cuh"

namespace pa {
namespace dpool {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
// CTAs of the cluster: 8 is the largest portable size; where a call may have
// enough to do for more, 16; one where that is enough, since every barrier and
// phase then stays within an SM.
constexpr int kCluster = 8, kClusterLarge = 16;
constexpr int kBatch = 8;    // items of a warp whose accesses are in flight at once
constexpr int kClaimed = INT32_MIN;  // a block's count while release_kernel frees it (or 0, see there)
// The kernels are compiled for at most kPer sequences a thread, in registers:
// one, for up to 1024 sequences, and as many as PA_DPOOL_MAX_SEQS needs (whose
// registers spill).
constexpr int kPerMost = PA_DPOOL_MAX_SEQS / kThreads;
static_assert(kPerMost * kThreads == PA_DPOOL_MAX_SEQS, "a thread holds a run of whole sequences");

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

// Quotients by the block size of numbers from 0 on; a power of two is a shift, a
// division some 25 instructions.
struct ByBlock {
    int bs, shift;  // (-1: no power of two)
    __device__ __forceinline__ explicit ByBlock(int size) {
        bs = size;
        shift = (size & (size - 1)) == 0 ? 31 - __clz(size) : -1;
    }
    __device__ __forceinline__ int down(int x) const { return shift >= 0 ? x >> shift : x / bs; }
    __device__ __forceinline__ int up(int x) const {
        const int n = down(x);
        return n + (n * bs != x);
    }
};

struct Header {
    int nb, bs, policy, head, count, magic;
    __device__ __forceinline__ explicit Header(const Pool &p)
        : nb(__ldcg(p.hdr)), bs(__ldcg(p.hdr + 1)), policy(__ldcg(p.hdr + 2)), head(__ldcg(p.hdr + 3)),
          count(__ldcg(p.hdr + 4)), magic(__ldcg(p.hdr + 5)) {}
    // whether the state is a sound pool of these sizes
    __device__ __forceinline__ bool ok(int num_blocks, int block_size) const {
        return magic == kMagic && nb == num_blocks && bs == block_size;
    }
};

template <typename T> __device__ __forceinline__ T warp_inclusive(T v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Exclusive scans of two values per thread over the CTA, in place; *ta and *tb
// receive the sums. `sums` holds 2 (kWarps + 1) values; the call ends with a
// CTA barrier.
__device__ __forceinline__ void block_exclusive2(long long &a, long long &b, long long *sums, long long *ta,
                                                 long long *tb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long *sa = sums, *sb = sums + kWarps + 1;
    const long long ia = warp_inclusive(a, lane), ib = warp_inclusive(b, lane);
    if (lane == 31) {
        sa[warp] = ia;
        sb[warp] = ib;
    }
    __syncthreads();
    if (warp < 2) {
        long long *x = warp == 0 ? sa : sb;
        const long long w = x[lane], wi = warp_inclusive(w, lane);
        x[lane] = wi - w;
        if (lane == 31) x[kWarps] = wi;
    }
    __syncthreads();
    a = sa[warp] + ia - a;
    b = sb[warp] + ib - b;
    *ta = sa[kWarps];
    *tb = sb[kWarps];
    __syncthreads();
}

// The same of one value, returned.
__device__ __forceinline__ int block_exclusive(int v, int *sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int inc = warp_inclusive(v, lane);
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int w = sums[lane], wi = warp_inclusive(w, lane);
        sums[lane] = wi - w;
        if (lane == 31) sums[kWarps] = wi;
    }
    __syncthreads();
    const int r = sums[warp] + inc - v;
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

template <int kPer> __global__ void __launch_bounds__(kThreads, 1) append_kernel(const AppendParams q) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x;
    const int S = q.num_seqs, MB = q.max_blocks, nb = q.num_blocks, bs = q.block_size;
    const ByBlock by(bs);
    // every CTA works out every sequence; the ones a CTA's output threads
    // answer for (marks, per-sequence outputs) are those of its slice
    const bool mine = tid / (kThreads / ctas) == rank;
    const int gtid = rank * kThreads + tid, gstep = ctas * kThreads;

    extern __shared__ int dyn[];
    int *tok_pre = dyn;                  // [S + 1] new tokens before sequence s
    int *take_pre = tok_pre + S + 1;     // [S + 1] blocks taken before sequence s
    int *ctx_cow = take_pre + S + 1;     // [S] context length, sign bit: its last block is copied
    __shared__ long long sums[2 * (kWarps + 1)];
    // The writers of shared blocks are counted in a hash table of each CTA (every
    // CTA goes over every sequence), or in the pool's scratch where the sequences
    // are too many for one: a barrier of the cluster and two trips to L2 more (64
    // single tokens 8.1 us that way, 7.8 with the table; 1000 sequences 10.6, 10.0).
    constexpr bool kLocal = kPer == 1;
    constexpr int kHash = kLocal ? 2 * kThreads : 1;
    __shared__ int h_block[kHash], h_writers[kHash], h_last[kHash];

    wait_previous();
    allow_next();
    const Pool p = views(q.state, nb);
    const Header hdr(p);
    if constexpr (kLocal)
        for (int i = tid; i < kHash; i += kThreads) {
            h_block[i] = h_last[i] = -1;
            h_writers[i] = 0;
        }
    const int per = (S + kThreads - 1) / kThreads;
    const int s0 = tid * per, s1 = min(S, s0 + per);
    int ctx[kPer], nw[kPer], blk[kPer], ref[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {  // in flight with the header
        ctx[i] = nw[i] = 0;
        if (s0 + i < s1) {
            ctx[i] = __ldcg(q.ctx + s0 + i);
            nw[i] = __ldcg(q.new_lens + s0 + i);
        }
    }
    int bad = 0;  // PA_DEVERR_* bits
    auto refuse = [&]() {  // nothing is applied: outputs that make the step's other calls do nothing
        for (int i = gtid; i <= S; i += gstep) q.q_start[i] = 0;
        for (int i = gtid; i < q.max_tokens; i += gstep) q.slots[i] = -1;
        for (int i = gtid; i < 2 * S; i += gstep) q.cow_pairs[i] = -1;
        if (gtid == 0) *q.num_cow = 0;
    };
    if (!hdr.ok(nb, bs)) {  // the same in every CTA: the header changes behind the cluster's barriers
        if (gtid == 0) record_error(q.err, PA_DEVERR_POOL);
        refuse();
        return;
    }
    const int head = hdr.head, count = hdr.count;

    // ---- who writes into which partly filled block
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        blk[i] = -1;
        if (ctx[i] < 0 || nw[i] < 0 || ctx[i] > (long long)MB * bs) {
            bad |= PA_DEVERR_CONTEXT;
            ctx[i] = nw[i] = 0;
        } else if ((long long)ctx[i] + nw[i] > (long long)MB * bs) {
            bad |= PA_DEVERR_POOL;
            ctx[i] = nw[i] = 0;
        } else if (nw[i] > 0 && by.down(ctx[i]) * bs != ctx[i]) {
            blk[i] = __ldcg(q.tables + (size_t)(s0 + i) * MB + by.down(ctx[i]));
            if (blk[i] < 0 || blk[i] >= nb) {
                bad |= PA_DEVERR_BLOCK_ID;
                blk[i] = -1;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) ref[i] = blk[i] >= 0 ? __ldcg(p.ref + blk[i]) : 1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (ref[i] < 1) bad |= PA_DEVERR_POOL;
        if (ref[i] <= 1) {
            blk[i] = -1;  // this sequence's alone: written in place
        } else if (!kLocal && mine) {
            atomicAdd(p.writers + blk[i], 1);
            atomicMax(p.last_writer + blk[i], s0 + i);
        }
    }
    int place = 0;  // of this thread's block in the table
    if constexpr (kLocal) {
        __syncthreads();
        if (blk[0] >= 0) {
            place = (int)((unsigned)blk[0] * 2654435769u >> 16) & (kHash - 1);
            for (;; place = (place + 1) & (kHash - 1)) {  // at most half of the places are taken
                const int held = atomicCAS(h_block + place, -1, blk[0]);
                if (held == -1 || held == blk[0]) break;
            }
            atomicAdd(h_writers + place, 1);
            atomicMax(h_last + place, s0);
        }
        __syncthreads();
    } else {
        cluster.sync();
    }

    // ---- takes and their places; the same in every CTA
    long long tok_at = 0;
    int takes = 0, cows = 0;
    bool cow[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        cow[i] = false;
        if (blk[i] >= 0) {
            const int w = kLocal ? h_writers[place] : __ldcg(p.writers + blk[i]);
            const int last = kLocal ? h_last[place] : __ldcg(p.last_writer + blk[i]);
            if (w > ref[i]) bad |= PA_DEVERR_POOL;  // more tables hold the block than its count says
            cow[i] = !(w == ref[i] && last == s0 + i);
        }
        tok_at += nw[i];
        takes += (int)cow[i] + by.up(ctx[i] + nw[i]) - by.up(ctx[i]);
        cows += cow[i];
    }
    // takes and cows are below 2^30 (sequences x table entries): one 64-bit scan for both
    long long tc_at = ((long long)takes << 32) | (unsigned)cows, all_tok, all_tc;
    block_exclusive2(tok_at, tc_at, sums, &all_tok, &all_tc);
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
            k += (int)cow[i] + by.up(ctx[i] + nw[i]) - by.up(ctx[i]);
        }
        if (tid == 0) {
            tok_pre[S] = (int)all_tok;
            take_pre[S] = all_takes;
        }
    }
    cluster.sync();  // every CTA has read lengths, counts and marks, and its shared arrays are written

#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (!kLocal && mine && blk[i] >= 0) {
            p.writers[blk[i]] = 0;
            p.last_writer[blk[i]] = -1;
        }
    if (bad) {
        refuse();
        return;
    }

    // ---- apply. Block k of the step's takes:
    auto block_of = [&](int k) -> int {
        const int at = hdr.policy == PA_POOL_FIFO ? head + k : head + count - 1 - k;  // from 0 to below 2 nb
        return __ldcg(p.ring + (at < nb ? at : at - nb));
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
                atomicSub(p.ref + blk[i], 1);  // other sequences of the call may copy it too
                reinterpret_cast<longlong2 *>(q.cow_pairs)[cow_at] = make_longlong2(blk[i], id);
                ++cow_at;
            }
            t += nw[i];
            k += (int)cow[i] + by.up(ctx[i] + nw[i]) - by.up(ctx[i]);
        }
    }
    for (int i = all_cows + gtid; i < S; i += gstep)
        reinterpret_cast<longlong2 *>(q.cow_pairs)[i] = make_longlong2(-1, -1);
    for (int k = gtid; k < all_takes; k += gstep) {
        const int s = find_run(take_pre, S, k);
        const int c = ctx_cow[s] & 0x7fffffff, cw = ctx_cow[s] < 0;
        const int id = block_of(k);
        // the copy of the last block (if any) is the sequence's first take
        const int j = k - take_pre[s] < cw ? by.down(c) : by.up(c) + k - take_pre[s] - cw;
        q.tables[(size_t)s * MB + j] = id;
        p.ref[id] = 1;
    }
    // Slots, four consecutive tokens a thread: one search and, within a block,
    // one look at the list serve all four (a token a thread took 2.6 times as
    // long for 256 prompts of 262,000 tokens).
    const bool vec = (reinterpret_cast<uintptr_t>(q.slots) & 15) == 0;
    const int quads = (q.max_tokens + 3) / 4;
#pragma unroll 2
    for (int i = gtid; i < quads; i += gstep) {
        int v[4] = {-1, -1, -1, -1};
        int s = -1, next = 4 * i, j = 0, o = 0, id = 0;  // sequence, its end, block and offset of the token, block id
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = 4 * i + u;
            if (t >= all_tok) continue;
            bool look = true;
            if (t >= next) {  // the first token here, or of a new sequence
                if (s < 0) s = find_run(tok_pre, S, t);
                else
                    do ++s;
                    while (t >= tok_pre[s + 1]);
                next = tok_pre[s + 1];
                const int pos = (ctx_cow[s] & 0x7fffffff) + t - tok_pre[s];
                j = by.down(pos);
                o = pos - j * bs;
            } else if (++o == bs) {
                o = 0;
                ++j;
            } else {
                look = false;
            }
            if (look) {
                const int c = ctx_cow[s] & 0x7fffffff, cw = ctx_cow[s] < 0;
                const int have = by.up(c);
                if (j >= have) id = block_of(take_pre[s] + cw + j - have);
                else if (cw) id = block_of(take_pre[s]);
                else id = __ldcg(q.tables + (size_t)s * MB + j);  // kept: no thread writes this entry
            }
            v[u] = id * bs + o;
        }
        if (vec && 4 * i + 3 < q.max_tokens) {
            reinterpret_cast<int4 *>(q.slots)[i] = make_int4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (4 * i + u < q.max_tokens) q.slots[4 * i + u] = v[u];
        }
    }
    if (gtid == 0) {
        q.q_start[S] = (int)all_tok;
        *q.num_cow = all_cows;
        if (hdr.policy == PA_POOL_FIFO) p.hdr[3] = (int)(((long long)head + all_takes) % nb);
        p.hdr[4] = count - all_takes;
    }
}

// ----------------------------------------------------------------- release

template <int kPer> __global__ void __launch_bounds__(kThreads, 1) release_kernel(const ReleaseParams q) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = q.num_seqs, MB = q.max_blocks, nb = q.num_blocks, bs = q.block_size;
    const ByBlock by(bs);

    extern __shared__ int dyn[];
    int *item_pre = dyn;             // [S + 1] 32-entry items before sequence s
    int *entries = item_pre + S + 1; // [S] entries sequence s drops
    __shared__ int sums[kWarps + 1];
    __shared__ int s_bad[kClusterLarge], s_freed[kClusterLarge];  // of every CTA, written by each into all

    wait_previous();
    allow_next();
    const Pool p = views(q.state, nb);
    const Header hdr(p);
    const int per = (S + kThreads - 1) / kThreads;
    const int s0 = tid * per, s1 = min(S, s0 + per);
    int n[kPer];          // entries that each sequence drops
    unsigned gone = 0;    // bit i: sequence s0 + i is finished
#pragma unroll
    for (int i = 0; i < kPer; ++i) {  // in flight with the header
        n[i] = 0;
        if (s0 + i < s1) {
            n[i] = __ldcg(q.ctx + s0 + i);
            gone |= (unsigned)(__ldcg(q.finished + s0 + i) != 0) << i;
        }
    }
    int bad = 0;  // PA_DEVERR_* bits
    if (!hdr.ok(nb, bs)) {  // the same in every CTA, as in append_kernel
        if (rank == 0 && tid == 0) record_error(q.err, PA_DEVERR_POOL);
        return;
    }
    const int head = hdr.head, count = hdr.count;

    // ---- the items, in sequence order: 32 consecutive table entries of one
    // sequence each; a warp takes a run of consecutive items
    int items = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (!(gone >> i & 1u)) {
            n[i] = 0;
        } else if (n[i] < 0 || n[i] > (long long)MB * bs) {
            bad |= PA_DEVERR_CONTEXT;
            n[i] = 0;
        }
        n[i] = by.up(n[i]);
        items += (n[i] + 31) / 32;
    }
    int all_items;
    int at = block_exclusive(items, sums, &all_items);
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
    // A warp's items go in batches whose memory accesses are all in flight at
    // once; the entries of a single batch stay in registers, more than one are
    // read again in each pass.
    const bool single = i1 - i0 <= kBatch;
    // A claimed block's count. 0 is what it will be, and spares a scattered store
    // (64,000 entries: 22.5 -> 21.0 us); with several batches it has to be told from
    // a free block's when it is read again.
    const int claimed = single ? 0 : kClaimed;
    int entry[kBatch];         // this lane's table entry of each item of the batch (-1: none)
    int id[kBatch];            // its block (-1: none)
    int ref[kBatch];           // the block's count; for a shared block's last place, from the count of drops on, what is left of it
    unsigned own = 0;          // bit k: the block is this sequence's alone (count 1)
    unsigned last = 0;         // bit k: the last place that drops a shared block
    auto load = [&](int b0) {
        int s = b0 < i1 ? find_run(item_pre, S, b0) : 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int item = b0 + k;
            entry[k] = -1;
            if (item >= i1) continue;
            while (item_pre[s + 1] <= item) ++s;
            const int j = (item - item_pre[s]) * 32 + lane;
            if (j < entries[s]) entry[k] = s * MB + j;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) id[k] = entry[k] >= 0 ? __ldcg(q.tables + entry[k]) : -1;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (id[k] < 0 || id[k] >= nb) {
                if (entry[k] >= 0) bad |= PA_DEVERR_BLOCK_ID;
                id[k] = -1;
            }
    };
    auto place_of = [&](int b0, int k) { return (b0 + k) * 32 + lane; };

    // ---- drops. A block of count 1 is claimed in one step: it is freed, here,
    // unless the call is refused. A shared block counts its drops and the last
    // place that drops it.
    for (int b0 = i0; b0 < i1; b0 += kBatch) {
        load(b0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) ref[k] = id[k] >= 0 ? atomicCAS(p.ref + id[k], 1, claimed) : 0;
        own = 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (id[k] < 0) continue;
            if (ref[k] == 1) {
                own |= 1u << k;
            } else if (ref[k] > 1) {
                atomicAdd(p.delta + id[k], 1);
                atomicMax(p.last_old + id[k], place_of(b0, k));
            } else {
                bad |= PA_DEVERR_POOL;  // a free block, or one that is listed twice
                id[k] = -1;
            }
        }
    }
    cluster.sync();

    // The batch's entries again, where there are several batches; then bit k of
    // the result: the entry frees its block.
    auto look = [&](int b0) -> unsigned {
        if (!single) {
            load(b0);
            own = 0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) ref[k] = id[k] >= 0 ? __ldcg(p.ref + id[k]) : 0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (id[k] >= 0 && ref[k] == kClaimed) own |= 1u << k;
                else if (ref[k] < 1) id[k] = -1;
            }
        }
        unsigned f = own;
        last = 0;
        int drops[kBatch], at_last[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool shared = id[k] >= 0 && !(own >> k & 1u);
            drops[k] = shared ? __ldcg(p.delta + id[k]) : 0;
            at_last[k] = shared ? __ldcg(p.last_old + id[k]) : -1;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (at_last[k] == place_of(b0, k)) {
                last |= 1u << k;
                ref[k] -= drops[k];
                if (ref[k] < 0) bad |= PA_DEVERR_POOL;
                if (ref[k] == 0) f |= 1u << k;
            }
        return f;
    };

    // ---- freed blocks, counted in place order
    int freed = 0;
    unsigned f = 0;
    for (int b0 = i0; b0 < i1; b0 += kBatch) {
        f = look(b0);
        freed += __popc(f);
    }
    freed = __reduce_add_sync(0xffffffffu, freed);
    int cta_freed;
    int base = block_exclusive(lane == 0 ? freed : 0, sums, &cta_freed);
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

    // ---- apply: freed blocks to the list's back, in place order; or claims taken back
    const int back = head + count + base;  // below 2 nb, as is every place behind it
    base = 0;
    for (int b0 = i0; b0 < i1; b0 += kBatch) {
        if (!single) f = look(b0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const unsigned m = __ballot_sync(0xffffffffu, !bad && (f >> k & 1u));
            if (m >> lane & 1u) {
                const int to = back + base + __popc(m & ((1u << lane) - 1u));
                p.ring[to < nb ? to : to - nb] = id[k];
            }
            base += __popc(m);
            if ((own >> k & 1u) && (bad || !single)) p.ref[id[k]] = bad ? 1 : 0;
        }
    }
    cluster.sync();  // every CTA is done with the marks, shared counts, tables and lengths

    // ---- shared counts, marks, table entries and lengths
    for (int b0 = i0; b0 < i1; b0 += kBatch) {
        if (!single) {
            load(b0);
            last = 0;
            int at_last[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) at_last[k] = id[k] >= 0 ? __ldcg(p.last_old + id[k]) : -1;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (at_last[k] == place_of(b0, k)) {
                    last |= 1u << k;
                    ref[k] = __ldcg(p.ref + id[k]) - __ldcg(p.delta + id[k]);
                }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (last >> k & 1u) {
                if (!bad) p.ref[id[k]] = ref[k];
                p.delta[id[k]] = 0;
                p.last_old[id[k]] = -1;
            }
            if (!bad && entry[k] >= 0) q.tables[entry[k]] = -1;
        }
    }
    if (!bad && tid / (kThreads / ctas) == rank) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (gone >> i & 1u) q.ctx[s0 + i] = 0;
    }
    if (rank == 0 && tid == 0 && !bad) p.hdr[4] = count + all_freed;
}

// -------------------------------------------------------------------- host

// What a kernel has been set up for, per device context.
struct KernelCache {
    AttrCache smem, large;
};

// Launches one cluster of `ctas` CTAs (kClusterLarge where the device can hold one, else kCluster).
template <typename P>
static cudaError_t launch_cluster(void (*kern)(P), const P &q, int smem, KernelCache *cache, int smem_max,
                                  unsigned ctas, cudaStream_t stream) {
    const void *fn = reinterpret_cast<const void *>(kern);
    cudaError_t e = ensure_smem_attr(fn, smem_max, &cache->smem);
    if (e != cudaSuccess) return e;
    if (ctas == kClusterLarge) {
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev >= kCacheDevices) return cudaErrorInvalidDevice;
        void *ctx = current_context();
        bool fits = ctx != nullptr && cache->large.ctx[dev].load(std::memory_order_acquire) == ctx;
        if (!fits) {
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = kClusterLarge;
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kClusterLarge);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = (size_t)smem_max;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int n = 0;
            fits = cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess && n > 0;
            if (fits) cache->large.ctx[dev].store(current_context(), std::memory_order_release);
            else (void)cudaGetLastError();
        }
        if (!fits) ctas = kCluster;
    }
    return launch_after(kern, dim3(ctas), kThreads, (size_t)smem, ctas, stream, q);
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
    if (max_tokens < 0 || max_tokens > (1 << 30)) return PA_ERR_SHAPE;
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
    const int smem = (3 * num_seqs + 2) * 4;
    // One CTA: a round of four slots for every thread (64 single tokens 7.8 -> 7.2 us, 296 short ones
    // 8.7 -> 8.2). 16: over two rounds for every thread of 8.
    const unsigned ctas = num_seqs <= dpool::kThreads && max_tokens <= 4 * dpool::kThreads ? 1
                          : max_tokens > 65536                                            ? dpool::kClusterLarge
                                                                                          : dpool::kCluster;
    static dpool::KernelCache one, most;
    cudaError_t e =
        num_seqs <= dpool::kThreads
            ? dpool::launch_cluster(dpool::append_kernel<1>, q, smem, &one, (3 * dpool::kThreads + 2) * 4, ctas,
                                    stream)
            : dpool::launch_cluster(dpool::append_kernel<dpool::kPerMost>, q, smem, &most,
                                    (3 * PA_DPOOL_MAX_SEQS + 2) * 4, ctas, stream);
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
    const int smem = (2 * num_seqs + 1) * 4;
    // Items that the warps of a CTA hold at once. One CTA: no more of them (168 sequences 8.6 -> 7.2 us; two
    // batches took 9.7 -> 11.1 us for 560, four 11.0 -> 29.7 for 858). 16: more than 8 CTAs hold.
    constexpr long long kHeld = dpool::kBatch * dpool::kWarps;
    const long long most_items = (long long)num_seqs * ((max_blocks_per_seq + 31ll) / 32);
    const unsigned ctas = most_items <= kHeld ? 1
                          : (long long)num_seqs * max_blocks_per_seq > 32 * kHeld * dpool::kCluster ? dpool::kClusterLarge
                                                                                                    : dpool::kCluster;
    static dpool::KernelCache one, most;
    cudaError_t e =
        num_seqs <= dpool::kThreads
            ? dpool::launch_cluster(dpool::release_kernel<1>, q, smem, &one, (2 * dpool::kThreads + 1) * 4, ctas,
                                    stream)
            : dpool::launch_cluster(dpool::release_kernel<dpool::kPerMost>, q, smem, &most,
                                    (2 * PA_DPOOL_MAX_SEQS + 1) * 4, ctas, stream);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
