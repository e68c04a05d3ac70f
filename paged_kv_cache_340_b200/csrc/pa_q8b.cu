// int8 caches with one scale per (block, kv head): the quantizing write of new
// tokens and the copy-on-write block copy (the scheme is in pa.h; decode over
// such a cache is in pa_decode_q8b.cu).
//
// Both move each byte once, so HBM bounds them.
#include <cfloat>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_pdl.cuh"

namespace pa {
namespace q8b {

struct AppendParams {
    const void *key;
    const void *value;
    const int32_t *q_start;
    int8_t *k_cache;
    int8_t *v_cache;
    float *k_scale;
    float *v_scale;
    const int32_t *tables;
    const int32_t *ctx;
    int num_tokens;
    int num_seqs;
    int max_blocks;
    int num_blocks;
    int num_kv_heads;
    unsigned int *err;
};

constexpr int kWarps = 8;

template <typename T, int D, int BS, bool kByToken> struct AppendShape {
    static constexpr int kVec = 16 / sizeof(T);  // values of a lane's vector
    static constexpr int kLanes = D / kVec;      // lanes of a row
    static constexpr int kRows = 32 / kLanes;    // rows per warp load
    // Warps that share a block. Two above 16 loads of a warp, so that its rows
    // take at most 64 registers of a lane (a warp alone with 128 took 143 us where
    // the pair takes 109: prompts of 2048 fp32 tokens, 32 heads of 128, blocks of
    // 32); and above 8, which leaves room for a fourth CTA (100 ragged chunks, 6
    // fp32 heads of 64: 23.1 -> 21.0 us, 20 of up to 1000 bf16 tokens 15.9 ->
    // 14.7), but not for a few rows a block, which a warp takes in one load (256
    // single tokens: 8.6 us, 10.6 in pairs).
    static constexpr int kTeam = BS / kRows > (kByToken ? 16 : 8) ? 2 : 1;
    static constexpr int kIt = BS / kRows / kTeam;  // loads of a warp per full block
    static constexpr int kCtas = kIt <= 8 ? 4 : 3;
};

// The units of work are a sequence's blocks with new rows. Numbering them must
// need no scan: a sequence touches at most q_len / bs + 2 blocks, so counting
// from q_start[s] / bs + 2 s on gives every block a unit of its own, and a few
// units are empty. With few tokens a sequence, where that is fewer, a block's
// unit is its first new token instead: none is empty for single tokens (256 of
// them: 8.7 -> 7.1 us with blocks of 32, 6.6 -> 4.6 with 16).
template <int BS, bool kByToken> __device__ __forceinline__ int first_unit(int q0, int s) {
    return kByToken ? q0 : q0 / BS + 2 * s;
}

// The largest s with first_unit(q_start[s], s) <= u, searched by the warp 128
// ways at a time, so that up to 128 sequences take one round of loads.
template <int BS, bool kByToken> __device__ __forceinline__ int unit_seq(const int32_t *q_start, int n, int u, int lane) {
    constexpr int kWays = 4;  // probes a lane
    int lo = 0;
    while (n > 1) {
        const int step = (n + 32 * kWays - 1) / (32 * kWays);
        bool le[kWays];
#pragma unroll
        for (int i = 0; i < kWays; ++i) {
            const int k = (i * 32 + lane) * step;
            le[i] = k < n && first_unit<BS, kByToken>(q_start[lo + min(k, n - 1)], lo + k) <= u;
        }
        int last = 0;
#pragma unroll
        for (int i = 0; i < kWays; ++i) {
            const unsigned m = __ballot_sync(0xffffffffu, le[i]);
            if (m) last = i * 32 + 31 - __clz(m);
        }
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

__device__ __forceinline__ int code_of(float x, float inv) {
    // NaN converts to 0, +-inf saturates
    return max(-127, min(127, __float2int_rn(__fmul_rn(x, inv))));
}

// Four codes of finite values none of which is above 127 / inv: the rounded
// product plus 1.5 * 2^23 has the code in its low byte (the sum's rounding is
// the rounding to a whole number, half to even), so nothing is converted or
// clamped. (The product is rounded on its own: as two-wide mul.rn.f32x2 and
// add.rn.f32x2 the pair came out fused, with other codes next to a half.)
__device__ __forceinline__ uint32_t codes4(const float *x, float inv) {
    uint32_t t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], inv), 12582912.f));
    return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
}

// Four codes in a raised scale (ratio below 1, so codes4 serves).
__device__ __forceinline__ uint32_t recode4(uint32_t codes, float ratio) {
    float x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = (float)(int8_t)(codes >> (8 * c));
    return codes4(x, ratio);
}

// Magnitudes as unsigned numbers (the bits without the sign order like the
// values, infinities and NaN above every finite one), 16-bit types two at a time.
template <typename T> struct Magnitude {
    static constexpr bool k32 = sizeof(T) == 4;
    static constexpr uint32_t kInf = k32 ? 0x7f800000u : std::is_same_v<T, __half> ? 0x7c00u : 0x7f80u;
    static __device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t word) {
        return k32 ? max(m, word & 0x7fffffffu) : __vmaxu2(m, word & 0x7fff7fffu);
    }
    // the warp's largest
    static __device__ __forceinline__ uint32_t over_warp(uint32_t m) {
        return __reduce_max_sync(0xffffffffu, k32 ? m : max(m & 0xffffu, m >> 16));
    }
    static __device__ __forceinline__ float value(uint32_t m) {
        if constexpr (k32) return __uint_as_float(m);
        else if constexpr (std::is_same_v<T, __half>) return __half2float(__ushort_as_half((unsigned short)m));
        else return __uint_as_float(m << 16);
    }
};

// One CTA per unit and part of the heads, one warp per (head, K or V) at a
// time, 16 bytes a lane. The block's rows stay in registers between the search
// for the largest value and the quantization, so HBM sees each byte once; about
// 4 instructions a value leave the loads the bound (a first version with
// conversions and clamps and one (head, K or V) a warp took 99 us where this
// one takes 67 for eight fp16 prompts of 2048 tokens and 32 heads, 403 MB).
template <typename T, int D, int BS, bool kByToken>
__global__ void __launch_bounds__(kWarps * 32, AppendShape<T, D, BS, kByToken>::kCtas)
    append_kernel(const AppendParams p) {
    using Sh = AppendShape<T, D, BS, kByToken>;
    using Mag = Magnitude<T>;
    constexpr int kVec = Sh::kVec, kLanes = Sh::kLanes, kRows = Sh::kRows, kIt = Sh::kIt, kTeam = Sh::kTeam;
    wait_previous();
    allow_next();
    const int lane = threadIdx.x & 31;
    const int H = p.num_kv_heads;
    const int u = blockIdx.x;
    const int s = unit_seq<BS, kByToken>(p.q_start, p.num_seqs, u, lane);
    const int q0 = p.q_start[s], q1 = p.q_start[s + 1];
    const int ctx = p.ctx[s];
    if (q0 == q1) return;  // nothing to write (such a sequence has units only where they are counted by blocks)
    const bool first_warp = blockIdx.y == 0 && threadIdx.x < 32;
    if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > ctx || ctx > (long long)p.max_blocks * BS) {
        if (first_warp && lane == 0) record_error(p.err, PA_DEVERR_CONTEXT);
        return;
    }
    const int p0 = ctx - (q1 - q0);                        // position of the first new token
    const int unit = u - first_unit<BS, kByToken>(q0, s);  // of the sequence
    const int lb = kByToken ? (p0 + unit) / BS : p0 / BS + unit;  // its logical block
    const int a = max(p0, lb * BS), e = min(ctx, (lb + 1) * BS);
    if (kByToken ? u >= q1 || a != p0 + unit : a >= e) return;
    const int id = p.tables[(size_t)s * p.max_blocks + lb];
    if (id < 0 || id >= p.num_blocks) {
        if (first_warp && lane == 0) record_error(p.err, PA_DEVERR_BLOCK_ID);
        return;
    }
    const int o0 = a - lb * BS, n = e - a;  // the new rows are slots o0 .. o0 + n - 1 of the block
    const int warp = threadIdx.x >> 5, part = warp % kTeam;
    const int row = part * kRows + lane / kLanes, col = (lane % kLanes) * kVec;
    // the largest of the team's warps; two slots a warp, used in turn
    __shared__ uint32_t team_mag[2][kWarps];
    int turn = 0;
    auto over_team = [&](uint32_t m) -> uint32_t {
        if constexpr (kTeam > 1) {
            if (lane == 0) team_mag[turn][warp] = m;
            named_bar_sync(1 + warp / kTeam, kTeam * 32);
            m = max(team_mag[turn][warp], team_mag[turn][warp ^ 1]);
            turn ^= 1;
        }
        return m;
    };
    constexpr int kTeams = kWarps / kTeam;
    for (int which = blockIdx.y * kTeams + warp / kTeam; which < 2 * H; which += gridDim.y * kTeams) {
        const int h = which >> 1;
        const bool is_v = which & 1;
        const T *src = static_cast<const T *>(is_v ? p.value : p.key) + ((size_t)(q0 + a - p0) * H + h) * D + col;
        float *scale = (is_v ? p.v_scale : p.k_scale) + (size_t)id * H + h;
        int8_t *dst = (is_v ? p.v_cache : p.k_cache) + ((size_t)id * H + h) * (BS * D);
        const float old = o0 > 0 ? *scale : 0.f;

        auto load = [&](int i) -> uint4 {
            const int r = i * kTeam * kRows + row;
            return r < n ? *reinterpret_cast<const uint4 *>(src + (size_t)r * H * D) : make_uint4(0u, 0u, 0u, 0u);
        };
        uint4 held[kIt];
        uint32_t mag = 0;
#pragma unroll
        for (int i = 0; i < kIt; ++i) held[i] = load(i);
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            mag = Mag::larger(Mag::larger(mag, held[i].x), held[i].y);
            mag = Mag::larger(Mag::larger(mag, held[i].z), held[i].w);
        }
        mag = over_team(Mag::over_warp(mag));
        const bool finite = mag < Mag::kInf;  // the same in the whole team
        float amax = Mag::value(mag);
        if (!finite) {  // rare: the largest finite value instead
            amax = 0.f;
#pragma unroll
            for (int i = 0; i < kIt; ++i) {
                float x[kVec];
                Elt<T>::unpack(held[i], x);
#pragma unroll
                for (int c = 0; c < kVec; ++c) amax = fabsf(x[c]) <= FLT_MAX ? fmaxf(amax, fabsf(x[c])) : amax;
            }
            amax = __uint_as_float(over_team(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))));
        }
        float now = __fdiv_rn(amax, 127.f);
        if (now < FLT_MIN) now = 0.f;
        now = fmaxf(old, now);
        const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int r = i * kTeam * kRows + row;
            if (r >= n) continue;
            float x[kVec];
            Elt<T>::unpack(held[i], x);
            uint32_t w[kVec / 4];
#pragma unroll
            for (int c = 0; c < kVec; c += 4) {
                if (finite) {
                    w[c / 4] = codes4(x + c, inv);
                } else {
                    w[c / 4] = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[c / 4] |= (uint32_t)(code_of(x[c + k], inv) & 0xff) << (8 * k);
                }
            }
            int8_t *d = dst + (o0 + r) * D + col;
            if constexpr (kVec == 8) *reinterpret_cast<uint2 *>(d) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t *>(d) = w[0];
        }
        if (now > old) {
            if (lane == 0 && part == 0) *scale = now;
            // The older rows' codes in the raised scale, 16 a lane at a time (four took 7.9 us
            // for 64 single tokens where this takes 6.8, 19.5 for 231 short fp32 chunks, 17.3;
            // several vectors in flight were up to 2 us faster there and cost prompts 2 to 5 %,
            // by their registers).
            if (o0 > 0) {
                const float ratio = __fdiv_rn(old, now);
                uint4 *old_rows = reinterpret_cast<uint4 *>(dst);
                for (int i = part * 32 + lane; i < o0 * D / 16; i += 32 * kTeam) {
                    const uint4 w = old_rows[i];
                    old_rows[i] = make_uint4(recode4(w.x, ratio), recode4(w.y, ratio), recode4(w.z, ratio), recode4(w.w, ratio));
                }
            }
        } else if (o0 == 0 && lane == 0 && part == 0) {
            *scale = now;  // a fresh block of zeros
        }
    }
}

// The scales of copied blocks: one thread per (pair, K or V, head).
__global__ void __launch_bounds__(256)
    copy_scales_kernel(float *k_scale, float *v_scale, const int64_t *pairs, const int32_t *pair_count, int max_pairs,
                       int num_blocks, int num_kv_heads) {
    const int n = pair_count ? min(__ldg(pair_count), max_pairs) : max_pairs;
    const long long all = 2ll * n * num_kv_heads;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        const int pair = (int)(i / (2 * num_kv_heads));
        int h = (int)(i - 2ll * pair * num_kv_heads);
        float *pool = h < num_kv_heads ? k_scale : v_scale;
        if (h >= num_kv_heads) h -= num_kv_heads;
        const int64_t src = __ldg(pairs + 2 * pair), dst = __ldg(pairs + 2 * pair + 1);
        if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) continue;  // recorded by the codes' copy
        pool[dst * num_kv_heads + h] = pool[src * num_kv_heads + h];
    }
}

template <typename T, int D, int BS, bool kByToken>
static cudaError_t launch_append_as(const AppendParams &p, long long units, cudaStream_t stream) {
    // (head, K or V) pairs a warp takes one after another: two where 8 CTAs
    // an SM are left, which halves the lookups (1, 2, 3 and 4 took 69.4, 67.0,
    // 66.5 and 67.5 us for prompts of 2048 tokens and 32 heads)
    const int warps_y = (2 * p.num_kv_heads * AppendShape<T, D, BS, kByToken>::kTeam + kWarps - 1) / kWarps;
    long long per = units * warps_y / (8ll * sm_count());
    per = per < 1 ? 1 : per > 2 ? 2 : per;
    const dim3 grid((unsigned)units, (unsigned)((warps_y + per - 1) / per));
    return launch_after(append_kernel<T, D, BS, kByToken>, grid, kWarps * 32, 0, 1, stream, p);
}

template <typename T, int D, int BS> static cudaError_t launch_append_n(const AppendParams &p, cudaStream_t stream) {
    const long long units = (long long)p.num_tokens / BS + 2ll * p.num_seqs + 1;
    return p.num_tokens < units ? launch_append_as<T, D, BS, true>(p, p.num_tokens, stream)
                                : launch_append_as<T, D, BS, false>(p, units, stream);
}

template <typename T>
static cudaError_t launch_append_t(const AppendParams &p, int head_dim, int block_size, cudaStream_t stream) {
    return head_dim == 128 ? (block_size == 16 ? launch_append_n<T, 128, 16>(p, stream) : launch_append_n<T, 128, 32>(p, stream))
                           : (block_size == 16 ? launch_append_n<T, 64, 16>(p, stream) : launch_append_n<T, 64, 32>(p, stream));
}

static bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace q8b
}  // namespace pa

using namespace pa;

extern "C" int pa_append_q8b(const void *key, const void *value, pa_dtype src_dtype, const int32_t *q_start,
                             int num_tokens, int8_t *k_cache, int8_t *v_cache, float *k_scale, float *v_scale,
                             const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                             int num_seqs, int num_blocks, int num_kv_heads, int head_dim, int block_size,
                             cudaStream_t stream) {
    if (num_tokens < 0 || num_seqs < 0 || num_blocks < 0 || num_kv_heads <= 0 || max_blocks_per_seq < 0 ||
        num_seqs > 65535 || num_kv_heads > 65535)
        return PA_ERR_SHAPE;
    if (src_dtype != PA_F32 && src_dtype != PA_F16 && src_dtype != PA_BF16) return PA_ERR_DTYPE;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_HEAD_DIM;
    if (block_size != 16 && block_size != 32) return PA_ERR_BLOCK_SIZE;
    if ((long long)num_blocks * block_size > INT32_MAX || max_blocks_per_seq > INT32_MAX / block_size ||
        num_tokens > INT32_MAX - 4 * 65536)
        return PA_ERR_SHAPE;
    if (num_tokens == 0 || num_seqs == 0) return PA_OK;
    if (!key || !value || !q_start || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens)
        return PA_ERR_NULL;
    if (!q8b::aligned(key, 16) || !q8b::aligned(value, 16) || !q8b::aligned(k_cache, 16) ||
        !q8b::aligned(v_cache, 16) || !q8b::aligned(k_scale, 16) || !q8b::aligned(v_scale, 16) ||
        !q8b::aligned(q_start, 4) || !q8b::aligned(block_tables, 4) || !q8b::aligned(context_lens, 4))
        return PA_ERR_ALIGN;
    q8b::AppendParams p{};
    if (device_error_word(&p.err) != cudaSuccess) return PA_ERR_CUDA;
    p.key = key;
    p.value = value;
    p.q_start = q_start;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.tables = block_tables;
    p.ctx = context_lens;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.num_kv_heads = num_kv_heads;
    cudaError_t e = src_dtype == PA_F32   ? q8b::launch_append_t<float>(p, head_dim, block_size, stream)
                    : src_dtype == PA_F16 ? q8b::launch_append_t<__half>(p, head_dim, block_size, stream)
                                          : q8b::launch_append_t<__nv_bfloat16>(p, head_dim, block_size, stream);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" int pa_copy_blocks_q8b(int8_t *k_cache, int8_t *v_cache, float *k_scale, float *v_scale,
                                  const int64_t *src_dst_pairs, const int32_t *num_pairs, int max_pairs,
                                  int num_blocks, int num_kv_heads, int head_dim, int block_size,
                                  cudaStream_t stream) {
    if (max_pairs < 0 || num_blocks < 0 || num_kv_heads <= 0 || num_kv_heads > 65535) return PA_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_HEAD_DIM;
    if (block_size != 16 && block_size != 32) return PA_ERR_BLOCK_SIZE;
    if (max_pairs == 0) return PA_OK;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !src_dst_pairs) return PA_ERR_NULL;
    if (!q8b::aligned(k_cache, 16) || !q8b::aligned(v_cache, 16) || !q8b::aligned(k_scale, 16) ||
        !q8b::aligned(v_scale, 16) || !q8b::aligned(src_dst_pairs, 8) || !q8b::aligned(num_pairs, 4))
        return PA_ERR_ALIGN;
    unsigned int *err = nullptr;
    if (device_error_word(&err) != cudaSuccess) return PA_ERR_CUDA;
    cudaError_t e = launch_copy_blocks(k_cache, v_cache, src_dst_pairs, max_pairs, num_pairs, num_blocks,
                                       (size_t)num_kv_heads * block_size * head_dim, err, stream);
    if (e == cudaSuccess) {
        long long ctas = (2ll * max_pairs * num_kv_heads + 255) / 256;
        if (ctas > 8ll * sm_count()) ctas = 8ll * sm_count();
        q8b::copy_scales_kernel<<<(unsigned)ctas, 256, 0, stream>>>(k_scale, v_scale, src_dst_pairs, num_pairs,
                                                                    max_pairs, num_blocks, num_kv_heads);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
