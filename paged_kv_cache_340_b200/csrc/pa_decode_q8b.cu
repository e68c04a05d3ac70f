// Paged decode attention over an int8 cache with one scale per (block, kv
// head): out = softmax(scale q K^T) V with K_t = kq_t * k_scale[block, h],
// V_t = vq_t * v_scale[block, h].
//
// The cache is read once and HBM bounds the call: an SM gets about 26 bytes a
// clock of it, so the work per byte must stay off the warps. Both products run
// on the 5th-generation tensor cores on the int8 codes as they lie in shared
// memory; no code of the cache ever passes through a register.
//   S^T = K Q^T   (M 128 = a tile's token rows, N = query columns, K = 128 bytes)
//   O^T = V^T P^T (M 128 = head dims, N = probability columns, K = 128 tokens)
// as tcgen05.mma kind::i8 with exact int32 sums. Query and probabilities enter
// as fixed point in base 256, three columns a head:
//   * q_d = qs * (65536 a + 256 b + c), signed digits, qs = 2^-21 of the power of
//     two of max|q|: elements down to 2^-11 (fp16) or 2^-14 (bf16) of it are exact.
//     Where the others lose too much (a few elements 100 times as large as they
//     are or more), what they lose is three more columns in a unit of its own.
//     (Without them scores were off by 2e-4 where four elements of 128 were 1000
//     times the others and met zeros in K: 2^-22 of max|q| for each of the others);
//   * w_t = p_t v_scale_t / (the tile's largest one) = (65536 a + 256 b + c) /
//     8388607, unsigned digits: 23 bits of the tile's largest weight, each off by
//     2^-24 of it (as fp32 holds that largest one), which makes digits the bits
//     of a sum's mantissa. The block scales are folded in here, and the tile's
//     largest weight is the unit, so a tile's sum is exact to 2^-17 of itself
//     whatever the others hold; tiles are joined in fp32.
// Scores, running maxima and sums are fp32 (log2 domain).
//
// A work item is a (sequence, kv head, up to 8 of its query heads[,
// partition]); the grid has one block per item. A resident CTA takes over
// blocks that have not started yet (clusterlaunchcontrol.try_cancel), some tiles
// ahead of its work, so K and V tiles of the next item stream in while the
// last one ends: a CTA per item lost about 3 us to each item's first lookups.
// A tile is 128 rows of 128 bytes of K and of V. A row is one token at
// head_dim 128 and two neighbouring tokens at 64: there each query head has two
// columns ("virtual heads"), one for the even and one for the odd tokens, its
// query padded with zeros over the other half, and the two are joined at the
// end.
//   * warp 7 claims the items, looks up what the other warps need of them and
//     writes the query's digits, a few items deep;
//   * warps 5 and 6 load the K and the V tiles, one lane a block, through the
//     table with 2-D TMA copies in the 128-byte swizzled layout, two stages
//     each; warp 5 also puts the tile's block scales beside them;
//   * warp 4 issues the products: S of tile t + 2 as soon as S of tile t has
//     been read, O of tile t when its weights have been written;
//   * warps 0-3: thread r owns row r of S^T (a token row) and row r of O^T (a
//     head dim). It forms the scores, keeps the running (max, sum) of its own
//     tokens per head, agrees on the tile's largest weight with the other
//     threads, writes the weights' digits, and adds up O in registers (which it
//     takes over from the other four warps: setmaxnreg).
// Rows past the sequence (or of a bad block) may hold anything: their weight is
// 0, and 0 times an int8 code is 0.
// Every wait is bounded (PA_DEVERR_TIMEOUT); tensor memory is always freed.
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_pdl.cuh"

namespace pa {
namespace q8b {

struct DecodeParams {
    void *out;
    // split along the tokens: each partition's largest score m (log2 units), l = sum of 2^(score - m) and
    // acc = sum of 2^(score - m) V
    float *ws_ml;   // [num_seqs, num_heads, max_parts, 2]
    float *ws_acc;  // [num_seqs, num_heads, max_parts, head_dim]
    const void *query;
    const float *k_scale;
    const float *v_scale;
    const int32_t *tables;
    const int32_t *ctx;
    const int32_t *seq_order;
    int max_blocks;
    int max_ctx;
    int num_seqs;
    int num_heads;
    int num_kv_heads;
    int group;
    int sub_groups;
    int num_blocks;
    int bs_shift;
    int partition_size;  // tokens; 0: the whole sequence
    int max_parts;
    int steal;  // whether a CTA takes over further blocks of the grid
    float scale_log2;
    pa_dtype out_dtype;
    unsigned int *err;
    // test hook (pa_decode_q8b_withhold_tile; its own instance of the kernel): the K tile `withhold_tile` of this
    // (sequence, kv head) is never asked for, and every wait gives up after wait_limit_ns
    int withhold_seq, withhold_kvh, withhold_tile;
    unsigned long long wait_limit_ns;
};

constexpr int kMaxContext = 1 << 30;
constexpr int kG = 8;                          // query heads per item, at most
constexpr int kRowBytes = 128;
constexpr int kTile = 128 * kRowBytes;         // 16 KB of K or V
constexpr int kClaimAhead = 4;                 // tiles still to be loaded when another item is claimed
// Splitting along the tokens: pieces of at most 16 tiles, which measured best of 8,
// 12, 16, 32 and 64 for 8 sequences of 32,768 to 131,072 tokens (163, 161, 158, 172, 195 us).
constexpr int kPiece = 16;
constexpr int kMaxBlocks = 16;                 // blocks of a tile, at most
// Virtual heads from which the softmax has two warpgroups: 16 (222 sequences of
// 4096 tokens, 8 kv heads of 64 with 8 query heads each: 273 -> 227 us); at 8 the
// third CTA that one warpgroup leaves room for is worth more (151 against 167 us).
constexpr int kTwoTeams = 16;
constexpr float kWUnit = 8388607.f;            // 2^23 - 1
constexpr float kNone = -3e38f;                // below every score: the maximum of no tokens
constexpr float kRaise = 16.f;                 // see the softmax

constexpr int kWide = 1 << 8;                  // see the item warp

// An item, as warp 7 hands it to the others.
struct Item {
    int ntiles;   // -1: no more items
    int s;
    int head0;    // its first query head
    int kvh;
    int first;    // its tokens: first .. end - 1
    int end;
    int part;
    int heads;    // its query heads that there are, plus kWide if what their digits lose has columns, too
    int ids[kMaxBlocks];  // blocks of the first tile (-1: none)
};

struct Scales {
    float k[kMaxBlocks], v[kMaxBlocks];
    unsigned valid;  // bit i: block i of the tile is one
    unsigned pad[3];
};

// V: virtual heads of an item (query heads, twice that at head_dim 64); kLone: one
// query head, which has digit rows for what its digits lose, too. The digit rows a
// product reads past the last one (up to kN) only give columns that nobody
// reads, so those rows are whatever lies behind.
template <int V, bool kLone> struct Shape {
    static constexpr int kQueries = kLone ? 2 * V : V;         // query columns, three digits each
    // softmax warpgroups: two halve the heads, and so a tile's time, where that bounds
    static constexpr int kTeams = V >= kTwoTeams ? 2 : 1;
    static constexpr int kSoftmaxThreads = 128 * kTeams, kThreads = kSoftmaxThreads + 128;
    static constexpr int kMmaWarp = 4 * kTeams, kLoadK = kMmaWarp + 1, kLoadV = kMmaWarp + 2, kItemWarp = kMmaWarp + 3;
    static constexpr int kN = (3 * V + 15) / 16 * 16;          // MMA columns
    // as shared memory allows: stages of K and of V, items known at a time
    static constexpr int kStages = kTeams == 2 && V <= 8 ? 3 : 2;
    static constexpr int kItems = kTeams == 2 ? (V <= 8 ? 3 : 4) : V <= 2 ? 4 : V <= 4 ? 3 : 2;
    // tiles whose scales are kept: the K warp fills tile t once S of tile t -
    // kStages is computed, and that was issued after O of the tile two before,
    // whose scales have been read
    static constexpr int kScales = kStages + 2;
    static constexpr int kDigits = (3 * V + 7) / 8 * 1024;     // bytes of the weights' 3 V digit rows, in 8-row groups
    static constexpr int kQDigits = (3 * kQueries + 7) / 8 * 1024;  // and the query's
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kStages * kTile;
    static constexpr int kOffQ = kOffV + kStages * kTile;      // [kItems] signed digits
    static constexpr int kOffP = kOffQ + kItems * kQDigits;     // unsigned digits; at an item's end at head_dim 64 the odd tokens' sums
    static constexpr int kOffScales = kOffP + kDigits;
    static constexpr int kOffItems = kOffScales + kScales * (int)sizeof(Scales);
    static constexpr int kOffQs = kOffItems + kItems * (int)sizeof(Item);  // float [kItems][kQueries]: log2 score per digit unit
    static constexpr int kOffMax = (kOffQs + kItems * kQueries * 4 + 15) / 16 * 16;  // float [2][4 warps][V], tiles in turn
    static constexpr int kOffSums = (kOffMax + 8 * V * 4 + 15) / 16 * 16;  // float [2][4 warps][V]: the threads' sums
    static constexpr int kOffClc = (kOffSums + 8 * V * 4 + 15) / 16 * 16;
    static constexpr int kOffBar = kOffClc + 16;
    static constexpr int kBars = 4 * kStages + 2 + 3 + 3 * kItems + 1;
    static constexpr int kEnd = kOffBar + kBars * 8 + 24;  // and tensor memory's address, flags, the hook's wait limit
    static constexpr int kReadEnd = kOffP + kN * kRowBytes;    // the last byte a product may read
    static constexpr int kSmemBytes = kEnd > kReadEnd ? kEnd : kReadEnd;
    // tensor memory: S in two buffers, O in one
    static constexpr int kSCol = 0, kOCol = 2 * kN;
    static constexpr int kCols = 3 * kN <= 64 ? 64 : 3 * kN <= 128 ? 128 : 256;
    // CTAs per SM: three, by shared memory; two with two softmax warpgroups
    static constexpr int kCtas = kTeams == 1 ? 3 : 2;
    // registers: of the launch, and after the last four warps have given theirs to the softmax. Split so that no warp
    // spills, which is a trip to L2 (111 sequences of up to 432 tokens, 32 heads x 6: 34.8 us; with 40 left to the last
    // four warps, 100 to 200 bytes of them spilled, 37.3)
    static constexpr int kRegs = 80, kRegsLow = 64, kRegsHigh = kTeams == 1 ? 96 : 88;
    static_assert(kRegsLow + kTeams * kRegsHigh <= (kTeams + 1) * kRegs, "registers taken over are registers given up");
    static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "CTAs per SM");
    static_assert(kCtas * kCols <= 512 && (kCtas + 1) * kRegs * kThreads > 65536, "tensor memory for every resident CTA");
    static_assert(sizeof(Item) <= 32 * 4, "an item is copied by a warp");
    static_assert(3 * kQueries <= kN, "a column for every digit");
    static_assert((V / 2) * 64 * 4 <= kDigits, "the odd tokens' sums fit the weights' digits");
};

// ------------------------------------------------------------- tensor cores

// Shared-memory matrix descriptor, 128-byte swizzle, 8-row groups 1024 bytes
// apart: its low word for an address, and its high word.
__device__ __forceinline__ uint32_t desc128(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | (1u << 16); }
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);

// Instruction descriptor of kind::i8, int32 sums, A signed, M 128.
__host__ __device__ constexpr uint32_t idesc_i8(bool b_signed, bool a_mn_major, int N) {
    return (2u << 4) | (1u << 7) | ((b_signed ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) |
           ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// a and b: the descriptors' low words; the high words are the same for all.
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], a, b, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"((int)kDescHigh)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// Whether the barrier's phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// kC columns of this warp's 32 tensor-memory lanes (4, or a multiple of 4 by eights).
template <int kC> __device__ __forceinline__ void tmem_load(uint32_t addr, int (&r)[kC]) {
    static_assert(kC % 4 == 0, "columns");
#pragma unroll
    for (int i = 0; i + 8 <= kC; i += 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]),
                       "=r"(r[i + 6]), "=r"(r[i + 7])
                     : "r"(addr + i));
    if constexpr (kC % 8 != 0)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[kC - 4]), "=r"(r[kC - 3]), "=r"(r[kC - 2]), "=r"(r[kC - 1])
                     : "r"(addr + kC - 4));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // the values exist from here on: no use of one may be moved above the wait
#pragma unroll
    for (int i = 0; i < kC; ++i) asm volatile("" : "+r"(r[i]));
}

// Barrier over the N softmax threads; true in all of them when `v` holds in all of them.
template <int N> __device__ __forceinline__ bool sync_and(bool v) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred pv, pa;\n\t"
        "setp.ne.u32 pv, %1, 0;\n\t"
        "barrier.cta.red.and.pred pa, 1, %2, pv;\n\t"
        "selp.u32 %0, 1, 0, pa;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)v), "n"(N)
        : "memory");
    return all != 0;
}

// Sums of N values per lane over the warp. While a lane has several, it keeps
// half of them and gives the others away, so lane i ends with the sum of value
// i * N / 32 in x[0].
template <int N, int Mask> __device__ __forceinline__ void warp_sums(float *x, int lane) {
    if constexpr (Mask >= 1) {
        if constexpr (N > 1) {
            const bool upper = (lane & Mask) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float give = upper ? x[i] : x[i + N / 2], keep = upper ? x[i + N / 2] : x[i];
                x[i] = keep + __shfl_xor_sync(0xffffffffu, give, Mask);
            }
            warp_sums<N / 2, Mask / 2>(x, lane);
        } else {
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], Mask);
            warp_sums<1, Mask / 2>(x, lane);
        }
    }
}

// The number whose base-256 digits' sums are hi, mid and lo (each below 2^22 in
// magnitude). One conversion instruction instead of two: they are issued at an
// eighth of the rate of sums. The first goes by adding 1.5 * 2^23 as bits.
__device__ __forceinline__ float number(int hi, int mid, int lo) {
    const float h = __int_as_float(0x4b400000 + hi) - 12582912.f;
    return fmaf(h, 65536.f, (float)(mid * 256 + lo));
}

// Two at a time: sums and products of pairs are one instruction each.
struct Pair {
    uint64_t v;
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit Pair(float a) : Pair(a, a) {}
    __device__ __forceinline__ void get(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
    return a;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
    return a;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(a.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return a;
}
__device__ __forceinline__ Pair number2(const int *c) {
    const Pair h = Pair(__int_as_float(0x4b400000 + c[0]), __int_as_float(0x4b400000 + c[3])) + Pair(-12582912.f);
    return fma2(h, Pair(65536.f), Pair((float)(c[1] * 256 + c[2]), (float)(c[4] * 256 + c[5])));
}

__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// TMA load of the box at row `row` of the map, which this call reads once: it is
// the first to leave L2 (4 % faster than without the hint on all of 64 x MHA,
// 256 x GQA and 8 long sequences, 75.6 / 92.0 / 156.7 us without).
__device__ __forceinline__ void load_once(void *dst, const CUtensorMap *map, int row, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(row), "l"(policy)
        : "memory");
}

// Registers per thread of this warpgroup, given up or taken over.
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// a[1], a[2], .., a[0]
template <typename T, int N> __device__ __forceinline__ void turn(T (&a)[N]) {
    const T first = a[0];
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) a[i] = a[i + 1];
    a[N - 1] = first;
}

// Asks for a block of the grid that has not started; the 16-byte answer completes on bar.
__device__ __forceinline__ void try_cancel(void *answer, uint64_t *bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
}

// Whether the answer is a block, and which.
__device__ __forceinline__ bool canceled(const void *answer, int &x, int &y, int &z) {
    uint32_t ok, cx, cy, cz;
    asm volatile(
        "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 a, [%4];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::y.b32.b128 %2, a;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::z.b32.b128 %3, a;\n\t}"
        : "=r"(ok), "=r"(cx), "=r"(cy), "=r"(cz)
        : "r"(smem_addr(answer))
        : "memory");
    x = (int)cx;
    y = (int)cy;
    z = (int)cz;
    return ok != 0;
}

// ------------------------------------------------------------------- kernel

template <typename T, int D, int G, bool kHook = false>
__global__ void __launch_bounds__(Shape<G * (128 / D), G == 1>::kThreads, Shape<G * (128 / D), G == 1>::kCtas)
    decode_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const DecodeParams p) {
    constexpr int kPar = 128 / D;   // tokens per row
    constexpr int kV = G * kPar;    // virtual heads: par * G + g
    using Sh = Shape<kV, G == 1>;
    constexpr int kN = Sh::kN, kStages = Sh::kStages, kScales = Sh::kScales, kTeams = Sh::kTeams;
    constexpr int kSoftmaxThreads = Sh::kSoftmaxThreads, kMmaWarp = Sh::kMmaWarp, kLoadV = Sh::kLoadV;
    constexpr int kSV = kV / kTeams, kOG = G / kTeams;  // virtual heads of a softmax thread, and heads whose O it adds up
    constexpr int kCols3 = (3 * kSV + 3) / 4 * 4;  // S columns read: three a virtual head
    constexpr int kOCols3 = (3 * kOG + 3) / 4 * 4; // O columns read: those of the lane's own tokens
    constexpr int kTok = 128 * kPar;              // tokens per tile
    constexpr int kItems = Sh::kItems;
    constexpr int kHalf = G > 1 ? G / 2 : 1;       // heads of a part of an item in two (see the item warp)

    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char *Ps = sm + Sh::kOffP;
    Scales *scales = reinterpret_cast<Scales *>(sm + Sh::kOffScales);
    Item *items = reinterpret_cast<Item *>(sm + Sh::kOffItems);
    float *qscale = reinterpret_cast<float *>(sm + Sh::kOffQs);
    float *wmax = reinterpret_cast<float *>(sm + Sh::kOffMax);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Sh::kOffBar);
    uint64_t *k_full = bars, *v_full = bars + kStages;              // a stage's tile (and its scales) is there
    uint64_t *k_empty = bars + 2 * kStages, *v_empty = bars + 3 * kStages;  // the product that read it is done
    uint64_t *s_full = bars + 4 * kStages;   // [2] S of the tile computed
    uint64_t *p_full = s_full + 2;           // weights of the tile written (its S and the O before it read)
    uint64_t *o_full = s_full + 3;           // O of the tile computed
    uint64_t *idle = s_full + 4;             // every product issued has finished
    uint64_t *clc = s_full + 5;              // the answer to a claim
    uint64_t *i_full = s_full + 6;           // [kItems] an item is described
    uint64_t *q_full = i_full + kItems;      // [kItems] and its query's digits are there
    uint64_t *i_empty = q_full + kItems;     // [kItems] everybody is done with it
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Sh::kBars);
    volatile int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    volatile int *loaded = reinterpret_cast<int *>(tmem_slot + 2);  // tiles that warp 5 has asked for

    uint64_t *const wl = kHook ? bars + Sh::kBars + 2 : nullptr;  // (nullptr: the library's bound)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs_shift = p.bs_shift;
    const int blocks = kTok >> bs_shift;      // per tile: 4, 8 or 16
    const int rows = 128 / blocks;            // 128-byte rows of a block
    // mbar_wait that also ends when another warp has given up (looked at only while it spins)
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = global_ns();
        for (uint32_t i = 1;; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((i & 63u) == 0u && (*abort_flag || global_ns() - t0 > (wl ? *wl : kWaitLimitNs))) return false;
        }
    };
    auto give_up = [&]() {
        record_error(p.err, PA_DEVERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (smem_addr(sm) & 1023u) {  // the swizzled layouts count on it
        wait_previous();
        if (tid == 0) record_error(p.err, PA_DEVERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(k_full + i, 2);
            mbar_init(v_full + i, 1);
            mbar_init(k_empty + i, 1);
            mbar_init(v_empty + i, 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_full + 1, 1);
        mbar_init(p_full, kSoftmaxThreads);
        mbar_init(o_full, 1);
        mbar_init(idle, 1);
        mbar_init(clc, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(i_full + i, 1);
            mbar_init(q_full + i, 1);
            mbar_init(i_empty + i, 4 * kTeams + 3);  // every warp but the item warp
        }
        *abort_flag = 0;
        *loaded = 0;
        if constexpr (kHook) *wl = p.wait_limit_ns;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(Sh::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    wait_previous();
    const uint32_t tmem = *tmem_slot;

    if (warp >= kMmaWarp) {
        regs_dec<Sh::kRegsLow>();
        if (warp == Sh::kItemWarp) {
            // ======================================================= item warp
            int x = blockIdx.x, y = blockIdx.y, z = blockIdx.z;
            bool more = true, sound = true;
            int tiles = 0;  // of all items so far
            // n: items handed on (a partition past its sequence's end is dropped here), claims: answers asked for
            for (int n = 0, claims = 0; sound;) {
                auto slot_free = [&]() {
                    if (n >= kItems)
                        sound = __all_sync(0xffffffffu, wait(i_empty + n % kItems, (n / kItems - 1) & 1));
                    return sound;
                };
                bool asked = false;  // and not answered
                auto claim = [&]() {  // asks for the next item
                    if (lane == 0) {
                        fence_proxy_async_smem();  // the last answer has been read
                        mbar_arrive_expect_tx(clc, 16);
                        try_cancel(sm + Sh::kOffClc, clc);
                    }
                    asked = true;
                };
                if (!more) {
                    allow_next();
                    if (!slot_free()) break;
                    if (lane == 0) {
                        items[n % kItems].ntiles = -1;
                        mbar_arrive(i_full + n % kItems);
                        mbar_arrive(q_full + n % kItems);
                    }
                    break;
                }
                // ---- the item
                int s = z;
                bool real = true;  // whether it has an output (else it is dropped)
                if (p.seq_order) {
                    s = p.seq_order[z];
                    if (s < 0 || s >= p.num_seqs) {
                        if (lane == 0) record_error(p.err, PA_DEVERR_CONTEXT);
                        s = 0;
                        real = false;
                    }
                }
                const int kvh = y / p.sub_groups, sub = y % p.sub_groups;
                const int head0 = kvh * p.group + sub * kG, g_valid = min(G, p.group - sub * kG);
                // the query's raw values, while the lengths come (heads past the last one: that one's)
                constexpr int kE = D / 32;
                using Raw = std::conditional_t<kE == 4, uint2, uint32_t>;  // a lane's kE values
                Raw raw[G];
#pragma unroll
                for (int g = 0; g < G; ++g)
                    raw[g] = reinterpret_cast<const Raw *>(static_cast<const T *>(p.query) +
                                                           ((size_t)s * p.num_heads + head0 + min(g, g_valid - 1)) * D)[lane];
                const int first = x * p.partition_size;
                const int lb = (first >> bs_shift) + lane;
                int id = lane < blocks && lb < p.max_blocks ? p.tables[(size_t)s * p.max_blocks + lb] : -1;
                int L = p.ctx[s];
                const int room = (int)min((long long)p.max_blocks << bs_shift, (long long)p.max_ctx);
                if (real && (L < 0 || L > room)) {
                    if (lane == 0) record_error(p.err, PA_DEVERR_CONTEXT);
                    L = L < 0 ? 0 : room;
                }
                if (p.partition_size) {
                    L = min(L, first + p.partition_size);
                    if (first >= L) real = false;  // no such partition: its entry is not read
                }
                if (!real) L = first;
                const int ntiles = L > first ? (L - first + kTok - 1) / kTok : 0;
                if (lb >= (L + (1 << bs_shift) - 1) >> bs_shift) id = -1;
                if (real && slot_free()) {
                    int slot = n % kItems;
                    Item *it = items + slot;
                    if (lane < kMaxBlocks) it->ids[lane] = id;
                    if (lane == 0) {
                        it->ntiles = ntiles;
                        it->s = s;
                        it->head0 = head0;
                        it->kvh = kvh;
                        it->first = first;
                        it->end = L;
                        it->part = x;
                        it->heads = g_valid;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(i_full + slot);  // the load warps can start
                    tiles += ntiles;
                    if (p.steal && __all_sync(0xffffffffu, tiles - *loaded <= kClaimAhead)) claim();
                    // ---- the query's digits
                    constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: a sum with it is a whole number below 2^22, in its bits
                    // the largest of two magnitudes in a word (16-bit ones order like the values, infinities and NaN on top)
                    auto larger = [](uint32_t m) { return max(m >> 16, m & 0xffffu); };
                    // a lane's largest |q| of a head
                    auto lanes = [&](const Raw &raw) -> uint32_t {
                        const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw);
                        if constexpr (kE == 4) return larger(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu));
                        else return larger(w[0] & 0x7fff7fffu);
                    };
                    auto as_float = [](uint32_t m) -> uint32_t {  // its fp32 bits
                        const unsigned short bits = (unsigned short)m;
                        return __float_as_uint((float)*reinterpret_cast<const T *>(&bits));
                    };
                    auto largest = [&](const Raw &raw) { return as_float(__reduce_max_sync(0xffffffffu, lanes(raw))); };
                    // The digits' unit for that largest magnitude, and its reciprocal; 0 and 0 below 2^-100, which
                    // counts as zero (the reciprocal would not be finite). Returns whether it is finite.
                    auto units = [](uint32_t bits, float &unit, float &inv) {
                        const uint32_t e = bits >> 23;
                        const bool live = e < 255u && e >= 27u;
                        unit = live ? __uint_as_float((e - 21u) << 23) : 0.f;
                        inv = live ? __uint_as_float((275u - e) << 23) : 0.f;
                        return e < 255u;
                    };
                    // the digits of whole numbers (with kWhole added) as query column col, in units of `unit`
                    auto put = [&](int col, const float (&t)[kE], float unit) {
                        unsigned char *Qs = sm + Sh::kOffQ + slot * Sh::kQDigits;
                        uint32_t u[kE];  // the digits, plus 128 each
#pragma unroll
                        for (int i = 0; i < kE; ++i) u[i] = __float_as_uint(t[i]) + 0x408080u;
                        uint32_t w[3];  // the lane's kE digits of each place
                        if constexpr (kE == 4) {
                            const uint32_t lo01 = __byte_perm(u[0], u[1], 0x5140), lo23 = __byte_perm(u[2], u[3], 0x5140);
                            w[0] = __byte_perm(__byte_perm(u[0], u[1], 0x0062), __byte_perm(u[2], u[3], 0x0062), 0x5410);
                            w[1] = __byte_perm(lo01, lo23, 0x7632);
                            w[2] = __byte_perm(lo01, lo23, 0x5410);
                        } else {
                            w[0] = __byte_perm(u[0], u[1], 0x0062);
                            w[1] = __byte_perm(u[0], u[1], 0x0051);
                            w[2] = __byte_perm(u[0], u[1], 0x0040);
                        }
#pragma unroll
                        for (int i = 0; i < 3; ++i) w[i] ^= 0x80808080u;
                        auto place = [&](int par) { return G == 1 ? col * kPar + par : par * G + col; };
#pragma unroll
                        for (int par = 0; par < kPar; ++par)
#pragma unroll
                            for (int i = 0; i < 3; ++i) {
                                const int r = place(par) * 3 + i;  // digit row; its 16-byte chunks are swizzled
                                auto at = [&](int half) {
                                    return Qs + r * kRowBytes + ((half * D + lane * kE) ^ ((r & 7) << 4));
                                };
                                if constexpr (kPar == 1) {
                                    *reinterpret_cast<uint32_t *>(at(0)) = w[i];
                                } else {
                                    *reinterpret_cast<uint16_t *>(at(par)) = (uint16_t)w[i];
                                    *reinterpret_cast<uint16_t *>(at(1 - par)) = 0;
                                }
                            }
                        if (lane < kPar) qscale[slot * Sh::kQueries + place(lane)] = unit * p.scale_log2;
                    };
                    uint32_t mag[G];
                    bool wide = false;
                    // How many lanes have an element below the exact ones, and one of 2^-7 of the largest or
                    // more: a byte a head, four heads a sum over the warp.
                    uint32_t below = 0, above = 0;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        constexpr int kExponent = std::is_same_v<T, __half> ? 10 : 7, kExact = std::is_same_v<T, __half> ? 11 : 14;
                        constexpr uint32_t kFew = std::is_same_v<T, __half> && kE == 4 ? 4 : 2;  // such lanes that do no harm
                        const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw[g]);
                        uint32_t least = w[0] & 0x7fff7fffu;
                        if constexpr (kE == 4) least = __vminu2(least, w[1] & 0x7fff7fffu);
                        const int most = lanes(raw[g]), top = __reduce_max_sync(0xffffffffu, most);
                        below += (int)min(least >> 16, least & 0xffffu) < top - (kExact << kExponent) ? 1u << 8 * (g % 4) : 0u;
                        above += most >= top - (7 << kExponent) ? 1u << 8 * (g % 4) : 0u;
                        mag[g] = as_float(top);
                        if (g % 4 == 3 || g == G - 1) {
                            below = __reduce_add_sync(0xffffffffu, below);
                            above = __reduce_add_sync(0xffffffffu, above);
                            // (a byte's top bit) more than a few are below, or one is and fewer than 16 are above
                            wide |= (((below + (0x7f - kFew) * 0x01010101u) | ((below + 0x7f7f7f7fu) & ~(above + 0x70707070u))) & 0x80808080u) != 0;
                            below = above = 0;
                        }
                    }
                    // Then whether a head's digits lose more than 2^-21 of the sum of its elements below 2^17 units (a
                    // sixteenth of the largest), by one sum over the warp, of 256ths of a unit lost and 256s of units
                    // there. (Queries whose elements are less than some 50 times apart hardly ever come here, so that
                    // these instructions are not at hand. A few lanes' elements lose 2^-18 of the largest at most.)
                    if (__builtin_expect(wide, 0)) {
                        wide = false;
#pragma unroll 1
                        for (int g = 0; g < G; ++g) {  // (head 0 of the arrays, which turn: the loop's code stays small)
                            float unit, inv, gone = 0.f, there = 0.f;
                            units(mag[0], unit, inv);
#pragma unroll
                            for (int i = 0; i < kE; ++i) {
                                const float q = (float)reinterpret_cast<const T *>(&raw[0])[i], t = fmaf(q, inv, kWhole);
                                gone += fabsf(fmaf(q, inv, kWhole - t));
                                there += fabsf(t - kWhole) < 131072.f ? fabsf(t - kWhole) : 0.f;
                            }
                            const uint32_t sums = __reduce_add_sync(0xffffffffu, (uint32_t)(gone * 256.f) << 17 | (uint32_t)there >> 8);
                            wide |= (sums >> 17) * 32u > (sums & 0x1ffffu);
                            turn(raw);
                            turn(mag);
                        }
                        wide = wide && ntiles > 0;
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        float unit, inv, t[kE];
                        const bool finite = units(mag[g], unit, inv);
#pragma unroll
                        for (int i = 0; i < kE; ++i) t[i] = fmaf((float)reinterpret_cast<const T *>(&raw[g])[i], inv, kWhole);
                        put(g, t, finite ? unit : NAN);  // (a query that is not finite makes its scores, and so its row, NaN)
                    }
                    // Then what they lose has digits of its own: beside the others where there is one head, else in
                    // place of half of the heads, which become an item of their own.
                    for (int left = wide ? it->heads : 0; __builtin_expect(left > 0, 0);) {
                        const int now = min(left, kHalf);
                        Raw part[kHalf];
#pragma unroll
                        for (int g = 0; g < kHalf; ++g)
                            part[g] = reinterpret_cast<const Raw *>(static_cast<const T *>(p.query) +
                                                                    ((size_t)it->s * p.num_heads + it->head0 + min(g, now - 1)) * D)[lane];
#pragma unroll 1
                        for (int g = 0; g < kHalf; ++g) {
                            float unit, inv, t[kE], rest[kE];
                            const bool finite = units(largest(part[0]), unit, inv);
                            uint32_t m = 0;
#pragma unroll
                            for (int i = 0; i < kE; ++i) {
                                const float q = inv > 0.f ? (float)reinterpret_cast<const T *>(&part[0])[i] : 0.f;
                                t[i] = fmaf(q, inv, kWhole);
                                rest[i] = fmaf(kWhole - t[i], unit, q);  // exact
                                m = max(m, __float_as_uint(fabsf(rest[i])));
                            }
                            put(g, t, finite ? unit : NAN);
                            units(__reduce_max_sync(0xffffffffu, m), unit, inv);
#pragma unroll
                            for (int i = 0; i < kE; ++i) t[i] = fmaf(rest[i], inv, kWhole);
                            put(g + kHalf, t, unit);
                            turn(part);
                        }
                        if (lane == 0) it->heads = now + kWide;
                        left -= now;
                        if (left <= 0) break;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(q_full + slot);
                        ++n;
                        if (!slot_free()) break;
                        const Item *before = it;
                        slot = n % kItems;
                        it = items + slot;
                        // (its fields are as before, but the head)
                        if (lane < (int)(sizeof(Item) / 4))
                            reinterpret_cast<int *>(it)[lane] = reinterpret_cast<const int *>(before)[lane];
                        __syncwarp();
                        if (lane == 0) it->head0 += kHalf;
                        tiles += it->ntiles;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(i_full + slot);
                    }
                    if (sound) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(q_full + slot);
                        ++n;
                    }
                }
                // ---- the next one, once few tiles are left to load
                more = false;
                if (p.steal) {
                    if (sound && !asked && tiles - *loaded > kClaimAhead) {
                        const uint64_t t0 = global_ns();
                        for (uint32_t i = 1; sound && tiles - *loaded > kClaimAhead; ++i) {
                            __nanosleep(64);
                            if (*abort_flag || ((i & 63u) == 0u && global_ns() - t0 > 4 * (wl ? *wl : kWaitLimitNs))) sound = false;
                        }
                    }
                    sound = __all_sync(0xffffffffu, sound && !*abort_flag);
                    if (sound) {
                        if (!asked) claim();
                        sound = __all_sync(0xffffffffu, wait(clc, claims & 1));
                    }
                    if (!sound) {  // an answer on its way lands before the CTA (and its shared memory) goes
                        if (asked) mbar_wait(clc, claims & 1, wl);
                        break;
                    }
                    ++claims;
                    more = canceled(sm + Sh::kOffClc, x, y, z);
                    __syncwarp();
                }
            }
            if (!sound && lane == 0) give_up();
            __syncwarp();
        } else if (warp != kMmaWarp) {
            // ======================================================= load warps
            // Lane i brings block i of the tile: `rows` rows of 128 bytes.
            const bool is_v = warp == kLoadV;
            const CUtensorMap *map = is_v ? &v_map : &k_map;
            uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
            unsigned char *ring = sm + (is_v ? Sh::kOffV : Sh::kOffK);
            int t = 0;  // tiles loaded, over all items
            const uint64_t policy = l2_evict_first_policy();
            bool sound = true;
            for (int n = 0; sound; ++n) {
                const int slot = n % kItems;
                sound = __all_sync(0xffffffffu, wait(i_full + slot, (n / kItems) & 1));
                if (!sound) break;
                const Item &it = items[slot];
                const int ntiles = it.ntiles;
                if (ntiles < 0) break;
                const int kvh = it.kvh, seq = it.s, b0 = it.first >> bs_shift;
                const int nblk = (it.end + (1 << bs_shift) - 1) >> bs_shift;
                const int32_t *trow = p.tables + (size_t)seq * p.max_blocks;
                int id = lane < kMaxBlocks ? it.ids[lane] : -1;
                __syncwarp();
                if (lane == 0) mbar_arrive(i_empty + slot);
                auto look = [&](int j) -> int {
                    const int lb = b0 + j * blocks + lane;
                    return (lane < blocks && lb < nblk) ? trow[lb] : -1;
                };
                auto scale_of = [&](const float *scale, int block) -> float {
                    return !is_v && block >= 0 && block < p.num_blocks
                               ? scale[(size_t)block * p.num_kv_heads + kvh] : 0.f;
                };
                int id_next = ntiles > 1 ? look(1) : -1;
                float ks = scale_of(p.k_scale, id), vs = scale_of(p.v_scale, id);
                for (int j = 0; j < ntiles; ++j, ++t) {
                    const int b = t % kStages;
                    if (t >= kStages) {
                        sound = __all_sync(0xffffffffu, wait(empty + b, (t / kStages - 1) & 1));
                        if (!sound) break;
                    }
                    const bool here = lane < blocks && b0 + j * blocks + lane < nblk;
                    const bool ok = here && id >= 0 && id < p.num_blocks;
                    if (here && !ok && !is_v) record_error(p.err, PA_DEVERR_BLOCK_ID);
                    const unsigned m = __ballot_sync(0xffffffffu, ok);
                    const bool withheld = kHook && !is_v && seq == p.withhold_seq && kvh == p.withhold_kvh &&
                                          j == p.withhold_tile;
                    if (lane == 0 && !withheld) mbar_arrive_expect_tx(full + b, __popc(m) * rows * kRowBytes);
                    __syncwarp();
                    if (ok && !withheld)
                        load_once(ring + b * kTile + lane * rows * kRowBytes, map, (id * p.num_kv_heads + kvh) * rows,
                                  full + b, policy);
                    if (!is_v) {
                        Scales &sc = scales[t % kScales];
                        if (lane < kMaxBlocks) {
                            sc.k[lane] = ks;
                            sc.v[lane] = vs;
                        }
                        if (lane == 0) sc.valid = m;
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(full + b);
                            *loaded = t + 1;
                        }
                    }
                    id = id_next;
                    ks = scale_of(p.k_scale, id);
                    vs = scale_of(p.v_scale, id);
                    id_next = look(j + 2);
                }
            }
            if (!sound && lane == 0) give_up();
            // copies in flight land before the CTA leaves
            for (int i = max(0, t - kStages); i < t; ++i) mbar_wait(full + i % kStages, (i / kStages) & 1, wl);
            __syncwarp();
        } else {
            // ========================================================= MMA warp
            if (lane == 0) {
                constexpr uint32_t kIdQK = idesc_i8(true, false, kN), kIdPV = idesc_i8(false, true, kN);
                const uint32_t base = smem_addr(sm);
                int n = -1, left = 0, slot = 0;  // the item whose S is issued next, and its tiles to come
                int issued = 0, done = 0;        // tiles whose S, whose O has been issued
                bool sound = true, more = true;
                while (sound) {
                    if (more && left == 0 && issued < done + 2) {
                        // The next item. It may be described only after an item has
                        // ended whose O is still to be issued here, so that goes first.
                        const int next = (n + 1) % kItems;
                        if (done == issued || mbar_test(q_full + next, ((n + 1) / kItems) & 1)) {
                            sound = wait(q_full + next, ((n + 1) / kItems) & 1);
                            if (!sound) break;
                            if (n >= 0) mbar_arrive(i_empty + slot);
                            ++n;
                            slot = next;
                            left = items[slot].ntiles;
                            if (left < 0) {
                                more = false;
                                left = 0;
                            }
                            continue;
                        }
                    }
                    // S or O, whichever has its operands first
                    bool take_s = left > 0 && issued < done + 2, take_o = done < issued;
                    if (!take_s && !take_o) break;  // no more items (with some, the next one was taken above)
                    const int bs = issued % kStages, bo = done % kStages;
                    if (take_s && take_o) {
                        uint64_t t0 = 0;
                        for (uint32_t i = 1;; ++i) {
                            take_s = mbar_test(k_full + bs, (issued / kStages) & 1);
                            take_o = !take_s && mbar_test(p_full, done & 1) && mbar_test(v_full + bo, (done / kStages) & 1);
                            if (take_s || take_o) break;
                            if (i == 64u) t0 = global_ns();
                            if ((i & 63u) == 0u && (*abort_flag || global_ns() - t0 > (wl ? *wl : kWaitLimitNs))) {
                                sound = false;
                                break;
                            }
                        }
                        if (!sound) break;
                    }
                    if (take_s) {
                        const int b = bs;
                        sound = wait(k_full + b, (issued / kStages) & 1);
                        if (!sound) break;
                        fence_after();
                        const uint32_t ka = desc128(base + Sh::kOffK) + b * (kTile / 16);
                        const uint32_t qa = desc128(base + Sh::kOffQ) + slot * (Sh::kQDigits / 16);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_i8(tmem + Sh::kSCol + (issued & 1) * kN, ka + kk * 2, qa + kk * 2, kIdQK,
                                   kk > 0);
                        mma_commit(s_full + (issued & 1));
                        mma_commit(k_empty + b);
                        ++issued;
                        --left;
                        continue;
                    }
                    const int b = bo;
                    sound = wait(p_full, done & 1) && wait(v_full + b, (done / kStages) & 1);
                    if (!sound) break;
                    fence_after();
                    const uint32_t va = desc128(base + Sh::kOffV) + b * (kTile / 16), pa_ = desc128(base + Sh::kOffP);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_i8(tmem + Sh::kOCol, va + kk * (32 * kRowBytes / 16), pa_ + kk * 2, kIdPV, kk > 0);
                    mma_commit(o_full);
                    mma_commit(v_empty + b);
                    ++done;
                }
                if (!sound) give_up();
                // tensor memory is freed below: every product issued must have finished
                mma_commit(idle);
                if (!mbar_wait(idle, 0, wl)) record_error(p.err, PA_DEVERR_TIMEOUT);
            }
            __syncwarp();
        }
    } else {
        // =================================================== softmax warps
        regs_inc<Sh::kRegsHigh>();
        const int r = tid & 127, quarter = warp & 3;
        const uint32_t tlane = tmem + ((uint32_t)(quarter * 32) << 16);
        const int block = r / rows;                           // this row's block within a tile
        const int v0 = (warp >> 2) * kSV;                     // this thread's first virtual head,
        const int g0 = (warp >> 2) * kOG;                     // its first head in O,
        const int vo = (kPar == 2 ? (quarter >> 1) * G : 0) + g0;  // and that one's virtual head (of the lane's head dim)
        float *red_m = reinterpret_cast<float *>(sm + Sh::kOffSums), *red_l = red_m + 4 * kV;  // [4 warps][kV]
        // at head_dim 64 the odd tokens' sums, [G][64], where the weights' digits were
        float *red_o = reinterpret_cast<float *>(Ps);
        int t = 0;                      // tiles done, over all items
        // The warps leave the loops together: one whose wait ran out says so at
        // the next barrier of all (each tile has one, each item's end and the end of all).
        bool ok = true, sound = true;
        for (int n = 0; ok; ++n) {
            const int slot = n % kItems;
            sound = __all_sync(0xffffffffu, sound && wait(q_full + slot, (n / kItems) & 1));
            const Item &it = items[slot];
            const int ntiles = sound ? it.ntiles : -1;
            if (ntiles < 0) {
                ok = sync_and<kSoftmaxThreads>(sound);
                break;
            }
            const int L = it.end, first = it.first, part = it.part;
            const size_t row0 = (size_t)it.s * p.num_heads + it.head0;  // output row of head 0
            const int g_valid = it.heads & (kWide - 1);
            float qs[kSV];
#pragma unroll
            for (int v = 0; v < kSV; ++v) qs[v] = qscale[slot * Sh::kQueries + v0 + v];
            float m_l[kSV], l[kSV];                // this thread's tokens: about their largest score, sum of 2^(score - it)
            float m_o[kOG], o[kOG], m_tile[kOG];   // O of the lane's dim: sum * 2^-m_o; the unit of the tile in tensor memory
#pragma unroll
            for (int v = 0; v < kSV; ++v) {
                m_l[v] = kNone;
                l[v] = 0.f;
            }
#pragma unroll
            for (int g = 0; g < kOG; ++g) {
                m_o[g] = m_tile[g] = kNone;
                o[g] = 0.f;
            }
            // adds the tile in tensor memory (its O columns, in units of 2^m_tile / kWUnit) to o
            auto add_tile = [&]() {
                int c[kOCols3];
                tmem_load<kOCols3>(tlane + Sh::kOCol + 3 * vo, c);
                float f2[2];
#pragma unroll
                for (int g = 0; g < kOG; ++g) {
                    if constexpr (kOG % 2 == 0) {
                        if (g % 2 == 0) number2(c + 3 * g).get(f2[0], f2[1]);
                    } else {
                        f2[g % 2] = number(c[3 * g], c[3 * g + 1], c[3 * g + 2]);
                    }
                    const float f = f2[g % 2];
                    if (m_tile[g] > m_o[g]) {  // the same in every thread of the warp
                        o[g] = fmaf(o[g], fast_exp2(m_o[g] - m_tile[g]), f);
                        m_o[g] = m_tile[g];
                    } else {
                        o[g] = fmaf(f, fast_exp2(m_tile[g] - m_o[g]), o[g]);
                    }
                }
            };
            for (int j = 0; j < ntiles; ++j, ++t) {
                float *wm = wmax + (t & 1) * 4 * kV;
                sound = __all_sync(0xffffffffu, sound && wait(s_full + (t & 1), (t >> 1) & 1));
                // log2 of the weight is score + lv. Their sum is rounded at the score's size,
                // so it only finds a unit for the tile; the weights are formed from their
                // distances to it, which are as small as the sums' from m_l (the sum's
                // rounding alone cost a softmax of one token 4e-5 at scores of 1000).
                float score[kSV], lv = 0.f;
                if (sound) {
                    fence_after();
                    const Scales &sc = scales[t % kScales];
                    const float ks = sc.k[block], vs = sc.v[block];
                    const unsigned valid = sc.valid;
                    lv = vs > 0.f ? log2f(vs) : -INFINITY;
                    const int tok = first + j * kTok + r * kPar;
                    // (the same in every thread)
                    const bool whole = first + (j + 1) * kTok <= L && valid == (1u << blocks) - 1u;
                    int c[kCols3];
                    tmem_load<kCols3>(tlane + Sh::kSCol + (t & 1) * kN + 3 * v0, c);
                    if constexpr (kSV % 2 == 0) {
#pragma unroll
                        for (int v = 0; v < kSV; v += 2)
                            (number2(c + 3 * v) * (Pair(qs[v], qs[v + 1]) * Pair(ks))).get(score[v], score[v + 1]);
                    } else {
#pragma unroll
                        for (int v = 0; v < kSV; ++v)
                            score[v] = number(c[3 * v], c[3 * v + 1], c[3 * v + 2]) * (qs[v] * ks);
                    }
                    if (__builtin_expect(it.heads >= kWide, 0)) {  // what the digits lose (looked up: no register lives for it)
                        if constexpr (G == 1) {
                            tmem_load<kCols3>(tlane + Sh::kSCol + (t & 1) * kN + 3 * kV, c);
#pragma unroll
                            for (int v = 0; v < kSV; ++v)
                                score[v] += number(c[3 * v], c[3 * v + 1], c[3 * v + 2]) * (qscale[slot * Sh::kQueries + kV + v] * ks);
                        } else {  // (kSV is a multiple of G)
#pragma unroll
                            for (int v = 0; v < kSV; ++v) {
                                if (v % G < kHalf) score[v] += score[v + kHalf];
                                else score[v] = -INFINITY;
                            }
                        }
                    }
                    if (!whole) {
#pragma unroll
                        for (int v = 0; v < kSV; ++v)
                            if (!(valid >> block & 1u) || tok + (v0 + v) / G >= L) score[v] = -INFINITY;
                    }
                    // The sum's reference is a score seen before, raised only when one is
                    // above it by kRaise: a term is then at most 2^kRaise.
                    float above = -INFINITY, over[kSV];  // score - m_l
                    auto sub = [&](float (&to)[kSV], const float (&a)[kSV], const float (&b)[kSV]) {
                        if constexpr (kSV % 2 == 0) {
#pragma unroll
                            for (int v = 0; v < kSV; v += 2)
                                fma2(Pair(b[v], b[v + 1]), Pair(-1.f), Pair(a[v], a[v + 1])).get(to[v], to[v + 1]);
                        } else {
#pragma unroll
                            for (int v = 0; v < kSV; ++v) to[v] = a[v] - b[v];
                        }
                    };
                    sub(over, score, m_l);
#pragma unroll
                    for (int v = 0; v < kSV; ++v) above = fmaxf(above, over[v]);
                    if (above > kRaise) {
#pragma unroll
                        for (int v = 0; v < kSV; ++v)
                            if (over[v] > kRaise) {
                                l[v] *= fast_exp2(-over[v]);
                                m_l[v] = score[v];
                                over[v] = 0.f;
                            }
                    }
                    if constexpr (kSV % 2 == 0) {
#pragma unroll
                        for (int v = 0; v < kSV; v += 2) {
                            (Pair(l[v], l[v + 1]) + Pair(fast_exp2(over[v]), fast_exp2(over[v + 1]))).get(l[v], l[v + 1]);
                        }
                    } else {
#pragma unroll
                        for (int v = 0; v < kSV; ++v) l[v] += fast_exp2(over[v]);
                    }
                    // the tile's largest weight per head, over this warp, and a little above
                    // it: more than the roundings of x, of the unit and of the distances to
                    // it, so that no weight is above its unit.
                    float x[kSV];
                    const float lx = lv + 0x1p-16f;
                    if constexpr (kSV % 2 == 0) {
#pragma unroll
                        for (int v = 0; v < kSV; v += 2) (Pair(score[v], score[v + 1]) + Pair(lx)).get(x[v], x[v + 1]);
                    } else {
#pragma unroll
                        for (int v = 0; v < kSV; ++v) x[v] = score[v] + lx;
                    }
                    float mw = 0.f;  // lane v has head v's
#pragma unroll
                    for (int v = 0; v < kSV; ++v) {
                        const float m = warp_max(x[v]);
                        mw = lane == v ? m : mw;
                    }
                    // (without a weight it is -inf, which gives NaN here and so kNone)
                    if (lane < kSV) wm[quarter * kV + v0 + lane] = fmaxf(fmaf(fabsf(mw), 0x1p-22f, mw), kNone);
                }
                ok = sync_and<kSoftmaxThreads>(sound);
                if (!ok) break;
                // over the four quarters of the tile: N heads from virtual head v on
                auto tile_max = [&]<int N>(float (&m)[N], int v) {
                    if constexpr (N % 4 == 0) {
#pragma unroll
                        for (int i = 0; i < N; i += 4) {
                            float4 w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const float4 *>(wm + k * kV + v + i);
                            m[i] = fmaxf(fmaxf(w[0].x, w[1].x), fmaxf(w[2].x, w[3].x));
                            m[i + 1] = fmaxf(fmaxf(w[0].y, w[1].y), fmaxf(w[2].y, w[3].y));
                            m[i + 2] = fmaxf(fmaxf(w[0].z, w[1].z), fmaxf(w[2].z, w[3].z));
                            m[i + 3] = fmaxf(fmaxf(w[0].w, w[1].w), fmaxf(w[2].w, w[3].w));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            m[i] = fmaxf(fmaxf(wm[v + i], wm[kV + v + i]), fmaxf(wm[2 * kV + v + i], wm[3 * kV + v + i]));
                    }
                };
                float mt[kSV];
                tile_max(mt, v0);
                if (j > 0) {  // O of the tile before is there: P and O are free once it is added up
                    sound = __all_sync(0xffffffffu, wait(o_full, (t - 1) & 1));
                    if (!sound) continue;  // (the next barrier tells the others)
                    fence_after();
                    add_tile();
                }
                if constexpr (kTeams == 1 && kPar == 1) {
#pragma unroll
                    for (int g = 0; g < kOG; ++g) m_tile[g] = mt[g];
                } else {
                    tile_max(m_tile, vo);
                }
                // ---- the weights' digits, row 3 v + i, byte r of the row (its 16-byte chunks swizzled)
                // (a whole number is the sum's mantissa: no conversion; bit 23 is 0 in its exponent)
                float w[kSV];
                if constexpr (kSV % 2 == 0) {
#pragma unroll
                    for (int v = 0; v < kSV; v += 2) {
                        (fma2(Pair(mt[v], mt[v + 1]), Pair(-1.f), Pair(score[v], score[v + 1])) + Pair(lv)).get(w[v], w[v + 1]);
                        fma2(Pair(fast_exp2(w[v]), fast_exp2(w[v + 1])), Pair(kWUnit), Pair(8388608.f)).get(w[v], w[v + 1]);
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < kSV; ++v) w[v] = fmaf(fast_exp2((score[v] - mt[v]) + lv), kWUnit, 8388608.f);
                }
#pragma unroll
                for (int v = 0; v < kSV; ++v) {
                    const unsigned u = __float_as_uint(w[v]);
                    const int d = 3 * v, d0 = 3 * v0;  // (3 v0 is a multiple of 8 with two teams, else 0)
                    static_assert(kTeams == 1 || 3 * kSV % 8 == 0 || kSV == 4, "swizzle phase");
                    const int ph = kTeams == 1 || 3 * kSV % 8 == 0 ? 0 : d0 & 7;
                    unsigned char *row = Ps + d0 * kRowBytes;
                    row[d * kRowBytes + (r ^ (((d + ph) & 7) << 4))] = (unsigned char)(u >> 16);
                    row[(d + 1) * kRowBytes + (r ^ (((d + 1 + ph) & 7) << 4))] = (unsigned char)(u >> 8);
                    row[(d + 2) * kRowBytes + (r ^ (((d + 2 + ph) & 7) << 4))] = (unsigned char)u;
                }
                fence_proxy_async_smem();
                fence_before();
                mbar_arrive(p_full);
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(i_empty + slot);  // its last S has been read
            // ---- the threads' sums, while the last product runs
            if (ntiles > 0) {
#pragma unroll
                for (int v = 0; v < kSV; ++v) {
                    const float mw = warp_max(m_l[v]);
                    l[v] *= fast_exp2(m_l[v] - mw);
                    if (lane == 0) red_m[quarter * kV + v0 + v] = mw;
                }
                warp_sums<kSV, 16>(l, lane);  // lane c * 32 / kSV holds head c's
                if (lane % (32 / kSV) == 0) red_l[quarter * kV + v0 + lane / (32 / kSV)] = l[0];
                ok = sync_and<kSoftmaxThreads>(sound);
                if (!ok) break;
            }
            // lane g * kEnt + i: entry i of head g (its four quarters, twice at head_dim 64)
            constexpr int kEnt = 4 * kPar;
            const int hg = min(lane / kEnt, kOG - 1), ent = lane % kEnt;
            const int at = (ent & 3) * kV + (ent >> 2) * G + g0 + hg;
            const float mi = ntiles > 0 ? red_m[at] : kNone;
            float m = mi;
#pragma unroll
            for (int i = kEnt / 2; i; i /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
            float sum = ntiles > 0 ? red_l[at] * fast_exp2(mi - m) : 0.f;  // (a NaN query's sum is NaN)
#pragma unroll
            for (int i = kEnt / 2; i; i /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, i);
            const float unit = p.partition_size ? 1.f / kWUnit : sum != 0.f ? 1.f / (sum * kWUnit) : 0.f;
            if (p.partition_size && quarter == 0 && ent == 0 && lane < kOG * kEnt && g0 + hg < g_valid)
                *reinterpret_cast<float2 *>(p.ws_ml + ((row0 + g0 + hg) * p.max_parts + part) * 2) = make_float2(m, sum);
            // ---- the last tile, and the output
            if (ntiles > 0) {
                sound = __all_sync(0xffffffffu, wait(o_full, (t - 1) & 1));
                if (sound) {
                    fence_after();
                    add_tile();
                }
            }
#pragma unroll
            for (int g = 0; g < kOG; ++g) {
                o[g] *= fast_exp2(m_o[g] - __shfl_sync(0xffffffffu, m, g * kEnt));
                if (kPar == 2 && ntiles > 0 && r >= D) red_o[(g0 + g) * D + r - D] = o[g];
            }
            if (kPar == 2 && ntiles > 0) {
                ok = sync_and<kSoftmaxThreads>(sound);
                if (!ok) break;
            }
            if (!sound) continue;
#pragma unroll
            for (int g = 0; g < kOG; ++g) {
                if (kPar == 2 && ntiles > 0 && r < D) o[g] += red_o[(g0 + g) * D + r];
                o[g] *= __shfl_sync(0xffffffffu, unit, g * kEnt);
            }
            if (r < D) {  // (a loop for each type: a choice within one costs its instructions' fetch eight times)
                const size_t row = row0 + g0;
                auto put = [&](auto *to, size_t step) {
#pragma unroll
                    for (int g = 0; g < kOG; ++g)
                        if (g0 + g < g_valid) to[g * step] = (std::remove_pointer_t<decltype(to)>)o[g];
                };
                if (p.partition_size) put(p.ws_acc + (row * p.max_parts + part) * D + r, (size_t)p.max_parts * D);
                else if (p.out_dtype == PA_F32) put(static_cast<float *>(p.out) + row * D + r, D);
                else put(static_cast<T *>(p.out) + row * D + r, D);
            }
            // (the sums are read before the next ones or weights are written: the next tile's barrier is in between)
        }
        if (!ok && tid == 0) give_up();
    }
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kCols) : "memory");
    }
}

// Joins the partitions: out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p.
// One CTA per (head, sequence); warp w takes partitions w, w + kJoinWarps, ..,
// a lane D / 32 dims, and the warps are joined in shared memory. A batch of
// kJoinWarps * kU partitions costs one trip to L2, which is all that bounds it:
// 16 warps for many partitions; 4 for up to 16 of them, where a batch's CTAs
// then fit the GPU at once (40 sequences of 8 heads: 25.2 us with 16 warps,
// decode included, 24.4 with 4).
template <int D, int kJoinWarps> __global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const DecodeParams p) {
    constexpr int kE = D / 32, kU = 4;
    using Vec = std::conditional_t<kE == 4, float4, float2>;
    __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps], sm_o[kJoinWarps][D];
    wait_previous();  // decode_kernel's partitions are written
    allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int s = blockIdx.y;
    if (p.seq_order) {
        s = p.seq_order[s];
        if (s < 0 || s >= p.num_seqs) return;  // recorded by decode_kernel
    }
    const long long room = min((long long)p.max_blocks << p.bs_shift, (long long)p.max_ctx);
    const int L = (int)min((long long)max(p.ctx[s], 0), room);
    const int n = (L + p.partition_size - 1) / p.partition_size;
    const size_t row = (size_t)s * p.num_heads + blockIdx.x;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml) + row * p.max_parts;
    const Vec *acc = reinterpret_cast<const Vec *>(p.ws_acc + row * p.max_parts * D) + lane;
    float m = kNone, l = 0.f, o[kE] = {};
    for (int i0 = warp; i0 < n; i0 += kJoinWarps * kU) {
        float2 v[kU];
        Vec a[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {  // kU partitions' loads in flight
            const int i = i0 + kJoinWarps * u;
            v[u] = i < n ? __ldcg(ml + i) : make_float2(kNone, 0.f);
            a[u] = i < n ? __ldcg(acc + (size_t)i * 32) : Vec{};
        }
        float mn = m;
#pragma unroll
        for (int u = 0; u < kU; ++u) mn = fmaxf(mn, v[u].x);
        const float r = fast_exp2(m - mn);
        l *= r;
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] *= r;
        m = mn;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const float w = fast_exp2(v[u].x - m);
            l = fmaf(w, v[u].y, l);  // (a NaN sum stays)
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] = fmaf(w, reinterpret_cast<const float *>(&a[u])[e], o[e]);
        }
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) sm_o[warp][lane * kE + e] = o[e];
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= D) return;
    float M = kNone;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, sm_m[w]);
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = fast_exp2(sm_m[w] - M);
        num = fmaf(f, sm_o[w][d], num);
        den = fmaf(f, sm_l[w], den);
    }
    store_out(p.out, row * D + d, den != 0.f ? num / den : 0.f, p.out_dtype);
}

template <typename T, int D, int G, bool kHook = false>
static cudaError_t launch_decode_t(const CUtensorMap &km, const CUtensorMap &vm, DecodeParams p, cudaStream_t stream) {
    using Sh = Shape<G * (128 / D), G == 1>;
    auto kern = decode_kernel<T, D, G, kHook>;
    static AttrCache attr;
    static std::atomic<int> regs{0};
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), Sh::kSmemBytes, &attr);
    if (e != cudaSuccess) return e;
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, reinterpret_cast<const void *>(kern));
        if (e != cudaSuccess) return e;
        // a launch with fewer registers than are taken over would wait for them for good
        if (at.numRegs != Sh::kRegs) return cudaErrorInvalidConfiguration;
        regs.store(at.numRegs, std::memory_order_relaxed);
    }
    const dim3 grid(p.max_parts, p.num_kv_heads * p.sub_groups, p.num_seqs);
    // blocks that all start at once leave none to take over
    p.steal = (long long)grid.x * grid.y * grid.z > (long long)Sh::kCtas * sm_count();
    return launch_after(kern, grid, Sh::kThreads, Sh::kSmemBytes, 1, stream, km, vm, p);
}

template <typename T>
static cudaError_t launch_decode(const CUtensorMap &km, const CUtensorMap &vm, const DecodeParams &p, int head_dim,
                                 cudaStream_t stream) {
    const int g = p.group;  // rounded up to a power of two, at most kG
#define PA_Q8B(DD) \
    (g == 1 ? launch_decode_t<T, DD, 1>(km, vm, p, stream) : g == 2 ? launch_decode_t<T, DD, 2>(km, vm, p, stream) \
     : g <= 4 ? launch_decode_t<T, DD, 4>(km, vm, p, stream) : launch_decode_t<T, DD, 8>(km, vm, p, stream))
    return head_dim == 128 ? PA_Q8B(128) : PA_Q8B(64);
#undef PA_Q8B
}

// Tokens of a partition (0: none). One piece per resident CTA, as far as the
// longest context tells (two or three pieces measured 0 to 30 % slower for 1 to 40
// sequences); longer work goes in pieces of kPiece tiles, which the CTAs take one
// after another, so that ragged lengths even out.
static int partition_of(int num_seqs, int rows_y, int group, int head_dim, int max_ctx) {
    const int tok = 128 * (128 / head_dim);
    const long long items = (long long)num_seqs * rows_y, tiles = ((long long)max_ctx + tok - 1) / tok;
    const int heads = (group > 4 ? 8 : group > 2 ? 4 : group) * (128 / head_dim);
    const long long ctas = (heads >= kTwoTeams ? 2ll : 3ll) * sm_count();
    if (items >= ctas || tiles < 2) return 0;
    long long per = (items * tiles + ctas - 1) / ctas;
    if (per > kPiece) per = kPiece;
    return per >= tiles ? 0 : (int)(per * tok);
}

// CTAs along the kv heads: a group above kG query heads takes several.
static long long rows_of(int num_heads, int num_kv_heads) {
    return (long long)num_kv_heads * ((num_heads / num_kv_heads + kG - 1) / kG);
}

static bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace q8b
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_q8b_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                int max_context_len) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        (head_dim != 64 && head_dim != 128) || max_context_len < 0 || max_context_len > q8b::kMaxContext ||
        num_heads % num_kv_heads != 0 ||
        q8b::rows_of(num_heads, num_kv_heads) > 65535)
        return 0;
    const int rows_y = (int)q8b::rows_of(num_heads, num_kv_heads);
    const int P = q8b::partition_of(num_seqs, rows_y, num_heads / num_kv_heads, head_dim, max_context_len);
    // at least 16 bytes, so that a workspace of the size asked for is always one
    return P ? pa_splitk_workspace_bytes(num_seqs, num_heads, head_dim, max_context_len, P) : 16;
}

namespace {

// pa_decode_q8b; hook.withhold_tile >= 0: its test form.
int decode_q8b_call(const q8b::DecodeParams &hook, void *out, const void *query, pa_dtype q_dtype, const int8_t *k_cache,
                             const int8_t *v_cache, const float *k_scale, const float *v_scale,
                             const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                             int num_seqs, int num_heads, int num_kv_heads, int head_dim, float scale, int block_size,
                             int num_blocks, int max_context_len, pa_dtype out_dtype, const int32_t *seq_order,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks < 0 || max_blocks_per_seq < 0 ||
        num_seqs > 65535 || num_kv_heads > 65535 || max_context_len < 0 || max_context_len > q8b::kMaxContext ||
        !std::isfinite(scale))
        return PA_ERR_SHAPE;
    if (q_dtype != PA_F16 && q_dtype != PA_BF16) return PA_ERR_DTYPE;
    if (out_dtype != q_dtype && out_dtype != PA_F32) return PA_ERR_DTYPE;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_HEAD_DIM;
    if (block_size != 16 && block_size != 32) return PA_ERR_BLOCK_SIZE;
    if (num_heads % num_kv_heads != 0) return PA_ERR_HEADS;
    const int group = num_heads / num_kv_heads;
    const long long rows_y = q8b::rows_of(num_heads, num_kv_heads);
    if (rows_y > 65535 || max_blocks_per_seq > INT_MAX / block_size ||
        (long long)num_blocks * num_kv_heads * block_size >= INT_MAX)
        return PA_ERR_SHAPE;
    if (num_seqs == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens)
        return PA_ERR_NULL;
    if (workspace &&
        workspace_bytes < pa_decode_q8b_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len))
        return PA_ERR_WORKSPACE;
    using q8b::aligned_to;
    if (!aligned_to(out, 16) || !aligned_to(query, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
        !aligned_to(k_scale, 16) || !aligned_to(v_scale, 16) || !aligned_to(workspace, 16) ||
        !aligned_to(block_tables, 4) || !aligned_to(context_lens, 4) || !aligned_to(seq_order, 4))
        return PA_ERR_ALIGN;
    q8b::DecodeParams p = hook;
    if (device_error_word(&p.err) != cudaSuccess) return PA_ERR_CUDA;
    p.out = out;
    p.query = query;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.tables = block_tables;
    p.ctx = context_lens;
    p.seq_order = seq_order;
    p.max_blocks = max_blocks_per_seq;
    p.max_ctx = max_context_len;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.num_blocks = num_blocks;
    p.sub_groups = (int)(rows_y / num_kv_heads);
    p.bs_shift = block_size == 16 ? 4 : 5;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out_dtype = out_dtype;
    p.max_parts = 1;
    const int P = workspace ? q8b::partition_of(num_seqs, (int)rows_y, group, head_dim, max_context_len) : 0;
    if (P) {
        p.partition_size = P;
        p.max_parts = (max_context_len + P - 1) / P;
        p.ws_ml = static_cast<float *>(workspace);
        p.ws_acc = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) +
                                             pa_splitk_acc_offset(num_seqs, num_heads, max_context_len, P));
    }
    // the pools as rows of 128 bytes, a block at a time
    const unsigned box = (unsigned)(block_size * head_dim / 128);
    const unsigned long long rows = (unsigned long long)num_blocks * num_kv_heads * box;
    CUtensorMap km, vm;
    if (!encode_rows_2d(&km, CU_TENSOR_MAP_DATA_TYPE_UINT8, k_cache, 128, rows ? rows : 1, 128, 128, box,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_rows_2d(&vm, CU_TENSOR_MAP_DATA_TYPE_UINT8, v_cache, 128, rows ? rows : 1, 128, 128, box,
                        CU_TENSOR_MAP_SWIZZLE_128B))
        return PA_ERR_CUDA;
    cudaError_t e;
    if (hook.withhold_tile >= 0) e = q8b::launch_decode_t<__half, 128, 1, true>(km, vm, p, stream);
    else
        e = q_dtype == PA_F16 ? q8b::launch_decode<__half>(km, vm, p, head_dim, stream)
                              : q8b::launch_decode<__nv_bfloat16>(km, vm, p, head_dim, stream);
    if (e == cudaSuccess && P) {
        const dim3 grid((unsigned)num_heads, (unsigned)num_seqs);
        const bool few = p.max_parts <= 16;  // a batch of 4 warps
        auto join = head_dim == 128 ? (few ? q8b::join_kernel<128, 4> : q8b::join_kernel<128, 16>)
                                    : (few ? q8b::join_kernel<64, 4> : q8b::join_kernel<64, 16>);
        e = launch_after(join, grid, few ? 128u : 512u, 0, 1, stream, p);
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" int pa_decode_q8b(void *out, const void *query, pa_dtype q_dtype, const int8_t *k_cache,
                             const int8_t *v_cache, const float *k_scale, const float *v_scale,
                             const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                             int num_seqs, int num_heads, int num_kv_heads, int head_dim, float scale, int block_size,
                             int num_blocks, int max_context_len, pa_dtype out_dtype, const int32_t *seq_order,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    q8b::DecodeParams none{};
    none.withhold_tile = -1;
    return decode_q8b_call(none, out, query, q_dtype, k_cache, v_cache, k_scale, v_scale, block_tables,
                           max_blocks_per_seq, context_lens, num_seqs, num_heads, num_kv_heads, head_dim, scale,
                           block_size, num_blocks, max_context_len, out_dtype, seq_order, workspace, workspace_bytes,
                           stream);
}

extern "C" int pa_decode_q8b_withhold_tile(void *out, const void *query, pa_dtype q_dtype, const int8_t *k_cache,
                                           const int8_t *v_cache, const float *k_scale, const float *v_scale,
                                           const int32_t *block_tables, int max_blocks_per_seq,
                                           const int32_t *context_lens, int num_seqs, int num_heads, int num_kv_heads,
                                           int head_dim, float scale, int block_size, int num_blocks,
                                           int max_context_len, pa_dtype out_dtype, int seq, int kv_head, int tile,
                                           unsigned long long wait_limit_ns, cudaStream_t stream) {
    if (q_dtype != PA_F16) return PA_ERR_DTYPE;  // the hook's instance
    if (head_dim != 128) return PA_ERR_HEAD_DIM;
    if (num_heads != num_kv_heads) return PA_ERR_HEADS;
    if (seq < 0 || seq >= num_seqs || kv_head < 0 || kv_head >= num_kv_heads || tile < 0 || wait_limit_ns < 100000ull ||
        wait_limit_ns > 1000000000ull)
        return PA_ERR_SHAPE;
    q8b::DecodeParams hook{};
    hook.withhold_seq = seq;
    hook.withhold_kvh = kv_head;
    hook.withhold_tile = tile;
    hook.wait_limit_ns = wait_limit_ns;
    return decode_q8b_call(hook, out, query, q_dtype, k_cache, v_cache, k_scale, v_scale, block_tables,
                           max_blocks_per_seq, context_lens, num_seqs, num_heads, num_kv_heads, head_dim, scale,
                           block_size, num_blocks, max_context_len, out_dtype, nullptr, nullptr, 0, stream);
}
