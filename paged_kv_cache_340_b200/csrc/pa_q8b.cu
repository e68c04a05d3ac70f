// int8 caches with one scale per (block, kv head): the quantizing write of new
// tokens and the copy-on-write block copy (the scheme is in pa.h; decode over
// such a cache is in pa_decode_q8b.cu).
//
// Both move each byte once, so HBM bounds them.
#include <cfloat>

#include "pa_common.cuh"
#include "pa_internal.h"

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

// Sequence s touches at most q_len / bs + 2 blocks, so numbering its blocks
// from first_unit(q_start[s], s) on gives every block of every sequence a unit
// of its own without a scan; a few units are empty.
template <int BS> __device__ __forceinline__ int first_unit(int q0, int s) { return q0 / BS + 2 * s; }

// The largest s with first_unit(q_start[s], s) <= u, searched 32 ways at a time by the warp.
template <int BS> __device__ __forceinline__ int unit_seq(const int32_t *q_start, int n, int u, int lane) {
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int k = lane * step;
        const bool le = k < n && first_unit<BS>(__ldg(q_start + lo + k), lo + k) <= u;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

__device__ __forceinline__ int code_of(float x, float inv) {
    // NaN converts to 0, +-inf saturates
    return max(-127, min(127, __float2int_rn(__fmul_rn(x, inv))));
}

// One warp per (unit, head, K or V): the block's new rows, 16 bytes a lane.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const AppendParams p) {
    constexpr int kVec = 16 / sizeof(T);       // values of a lane's vector
    constexpr int kLanes = D / kVec;           // lanes of a row
    constexpr int kRows = 32 / kLanes;         // rows per warp load
    constexpr int kIt = BS / kRows;            // loads per full block
    // a block's rows stay in registers between the search for the largest
    // value and the quantization, unless that would take over 64 of them
    constexpr bool kHold = kIt <= 16;
    const int lane = threadIdx.x & 31;
    const int which = blockIdx.y * kWarps + (threadIdx.x >> 5);
    const int h = which >> 1, H = p.num_kv_heads;
    const bool is_v = which & 1;
    if (h >= H) return;
    const int u = blockIdx.x;
    const int s = unit_seq<BS>(p.q_start, p.num_seqs, u, lane);
    const int q0 = __ldg(p.q_start + s), q1 = __ldg(p.q_start + s + 1);
    const int ctx = __ldg(p.ctx + s);
    if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > ctx || ctx > (long long)p.max_blocks * BS) {
        if (lane == 0 && which == 0) record_error(p.err, PA_DEVERR_CONTEXT);
        return;
    }
    const int p0 = ctx - (q1 - q0);                        // position of the first new token
    const int lb = p0 / BS + u - first_unit<BS>(q0, s);    // this unit's logical block
    const int a = max(p0, lb * BS), e = min(ctx, (lb + 1) * BS);
    if (a >= e) return;
    const int id = __ldg(p.tables + (size_t)s * p.max_blocks + lb);
    if (id < 0 || id >= p.num_blocks) {
        if (lane == 0 && which == 0) record_error(p.err, PA_DEVERR_BLOCK_ID);
        return;
    }
    const int o0 = a - lb * BS, n = e - a;  // the new rows are slots o0 .. o0 + n - 1 of the block
    const int row = lane / kLanes, col = (lane % kLanes) * kVec;
    const T *src = static_cast<const T *>(is_v ? p.value : p.key) + ((size_t)(q0 + a - p0) * H + h) * D + col;
    float *scale = (is_v ? p.v_scale : p.k_scale) + (size_t)id * H + h;
    int8_t *dst = (is_v ? p.v_cache : p.k_cache) + ((size_t)id * H + h) * (BS * D);
    const float old = o0 > 0 ? *scale : 0.f;

    auto load = [&](int i) -> uint4 {
        const int r = i * kRows + row;
        return r < n ? __ldg(reinterpret_cast<const uint4 *>(src + (size_t)r * H * D)) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 held[kHold ? kIt : 1];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
        const uint4 v = load(i);
        if constexpr (kHold) held[i] = v;
        float x[kVec];
        Elt<T>::unpack(v, x);
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            const float m = fabsf(x[c]);
            amax = m <= FLT_MAX ? fmaxf(amax, m) : amax;  // finite values only
        }
    }
#pragma unroll
    for (int mk = 16; mk >= 1; mk >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, mk));
    float now = __fdiv_rn(amax, 127.f);
    if (now < FLT_MIN) now = 0.f;
    now = fmaxf(old, now);
    const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
        const int r = i * kRows + row;
        if (r >= n) continue;
        uint4 v;
        if constexpr (kHold) v = held[i];
        else v = load(i);
        float x[kVec];
        Elt<T>::unpack(v, x);
        uint32_t w[kVec / 4];
#pragma unroll
        for (int c = 0; c < kVec; c += 4)
            w[c / 4] = (uint32_t)(code_of(x[c], inv) & 0xff) | (uint32_t)(code_of(x[c + 1], inv) & 0xff) << 8 |
                       (uint32_t)(code_of(x[c + 2], inv) & 0xff) << 16 | (uint32_t)code_of(x[c + 3], inv) << 24;
        int8_t *d = dst + (o0 + r) * D + col;
        if constexpr (kVec == 8) *reinterpret_cast<uint2 *>(d) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(d) = w[0];
    }
    if (now > old) {
        if (lane == 0) *scale = now;
        if (o0 > 0) {  // the older rows' codes in the raised scale
            const float ratio = __fdiv_rn(old, now);
            for (int i = lane; i < o0 * D / 4; i += 32) {
                uint32_t w = reinterpret_cast<uint32_t *>(dst)[i], r = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    r |= (uint32_t)(code_of((float)(int8_t)(w >> (8 * c)), ratio) & 0xff) << (8 * c);
                reinterpret_cast<uint32_t *>(dst)[i] = r;
            }
        }
    } else if (o0 == 0 && lane == 0) {
        *scale = now;  // a fresh block of zeros
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

template <typename T>
static cudaError_t launch_append_t(const AppendParams &p, int head_dim, int block_size, cudaStream_t stream) {
    const dim3 grid((unsigned)(p.num_tokens / block_size + 2 * p.num_seqs + 1),
                    (unsigned)((2 * p.num_kv_heads + kWarps - 1) / kWarps));
    if (head_dim == 128) {
        if (block_size == 16) append_kernel<T, 128, 16><<<grid, kWarps * 32, 0, stream>>>(p);
        else append_kernel<T, 128, 32><<<grid, kWarps * 32, 0, stream>>>(p);
    } else {
        if (block_size == 16) append_kernel<T, 64, 16><<<grid, kWarps * 32, 0, stream>>>(p);
        else append_kernel<T, 64, 32><<<grid, kWarps * 32, 0, stream>>>(p);
    }
    return cudaGetLastError();
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
    if ((long long)num_blocks * block_size > INT32_MAX || num_tokens > INT32_MAX - 4 * 65536) return PA_ERR_SHAPE;
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
