// Paged decode attention over an int8 cache with one scale per (block, kv
// head): out = softmax(scale q K^T) V with K_t = kq_t * k_scale[block, h].
#include <climits>
#include <cmath>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace q8b {

struct DecodeParams {
    void *out;
    const void *query;
    const int8_t *k_cache;
    const int8_t *v_cache;
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
    int num_blocks;
    int block_size;
    float scale_log2;
    pa_dtype out_dtype;
    unsigned int *err;
};

constexpr int kWarps = 4;
constexpr int kG = 8;  // query heads per CTA, at most

// One CTA per (sequence, kv head, up to 8 of its query heads); each warp takes
// every fourth token, a lane D / 32 of its dims.
template <typename T, int D> __global__ void __launch_bounds__(kWarps * 32) decode_kernel(const DecodeParams p) {
    constexpr int kE = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = blockIdx.x;
    if (p.seq_order) {
        s = __ldg(p.seq_order + s);
        if (s < 0 || s >= p.num_seqs) {
            if (threadIdx.x == 0) record_error(p.err, PA_DEVERR_CONTEXT);
            return;
        }
    }
    const int subs = (p.group + kG - 1) / kG;
    const int kvh = blockIdx.y / subs, sub = blockIdx.y % subs;
    const int head0 = kvh * p.group + sub * kG, g_valid = min(kG, p.group - sub * kG);
    int L = __ldg(p.ctx + s);
    const long long room = min((long long)p.max_blocks * p.block_size, (long long)p.max_ctx);
    if (L < 0 || L > room) {
        if (threadIdx.x == 0) record_error(p.err, PA_DEVERR_CONTEXT);
        L = L < 0 ? 0 : (int)room;
    }
    float q[kG][kE], o[kG][kE], m[kG], l[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            q[g][e] = g < g_valid ? (float)static_cast<const T *>(p.query)[((size_t)s * p.num_heads + head0 + g) * D +
                                                                           lane * kE + e] * p.scale_log2
                                  : 0.f;
            o[g][e] = 0.f;
        }
    }
    for (int t = warp; t < L; t += kWarps) {
        const int id = __ldg(p.tables + (size_t)s * p.max_blocks + t / p.block_size);
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) record_error(p.err, PA_DEVERR_BLOCK_ID);
            continue;
        }
        const size_t unit = (size_t)id * p.num_kv_heads + kvh;
        const size_t at = (unit * p.block_size + t % p.block_size) * D + lane * kE;
        const float ks = __ldg(p.k_scale + unit), vs = __ldg(p.v_scale + unit);
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < kE; ++e) x = fmaf(q[g][e], (float)p.k_cache[at + e], x);
#pragma unroll
            for (int mk = 16; mk >= 1; mk >>= 1) x += __shfl_xor_sync(0xffffffffu, x, mk);
            x *= ks;
            const float mn = fmaxf(m[g], x);
            const float a = fast_exp2(m[g] - mn), w = fast_exp2(x - mn);
            m[g] = mn;
            l[g] = l[g] * a + w;
#pragma unroll
            for (int e = 0; e < kE; ++e) o[g][e] = fmaf(o[g][e], a, w * vs * (float)p.v_cache[at + e]);
        }
    }
    __shared__ float sm[kWarps][kG], sl[kWarps][kG], so[kWarps][kG][D];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        if (lane == 0) {
            sm[warp][g] = m[g];
            sl[warp][g] = l[g];
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) so[warp][g][lane * kE + e] = o[g][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g_valid * D; i += kWarps * 32) {
        const int g = i / D, d = i % D;
        float M = -INFINITY;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][g]);
        float num = 0.f, den = 0.f;
        if (M > -INFINITY)
            for (int w = 0; w < kWarps; ++w) {
                const float a = fast_exp2(sm[w][g] - M);
                num = fmaf(a, so[w][g][d], num);
                den = fmaf(a, sl[w][g], den);
            }
        store_out(p.out, ((size_t)s * p.num_heads + head0 + g) * D + d, den > 0.f ? num / den : 0.f, p.out_dtype);
    }
}

static bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace q8b
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_q8b_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                int max_context_len) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || max_context_len < 0) return 0;
    return 16;
}

extern "C" int pa_decode_q8b(void *out, const void *query, pa_dtype q_dtype, const int8_t *k_cache,
                             const int8_t *v_cache, const float *k_scale, const float *v_scale,
                             const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                             int num_seqs, int num_heads, int num_kv_heads, int head_dim, float scale, int block_size,
                             int num_blocks, int max_context_len, pa_dtype out_dtype, const int32_t *seq_order,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks < 0 || max_blocks_per_seq < 0 ||
        num_seqs > 65535 || num_kv_heads > 65535 || max_context_len < 0 || !std::isfinite(scale))
        return PA_ERR_SHAPE;
    if (q_dtype != PA_F16 && q_dtype != PA_BF16) return PA_ERR_DTYPE;
    if (out_dtype != q_dtype && out_dtype != PA_F32) return PA_ERR_DTYPE;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_HEAD_DIM;
    if (block_size != 16 && block_size != 32) return PA_ERR_BLOCK_SIZE;
    if (num_heads % num_kv_heads != 0) return PA_ERR_HEADS;
    const int group = num_heads / num_kv_heads;
    const long long rows_y = (long long)num_kv_heads * ((group + q8b::kG - 1) / q8b::kG);
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
    q8b::DecodeParams p{};
    if (device_error_word(&p.err) != cudaSuccess) return PA_ERR_CUDA;
    p.out = out;
    p.query = query;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
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
    p.block_size = block_size;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out_dtype = out_dtype;
    const dim3 grid((unsigned)num_seqs, (unsigned)rows_y);
    if (q_dtype == PA_F16) {
        if (head_dim == 128) q8b::decode_kernel<__half, 128><<<grid, q8b::kWarps * 32, 0, stream>>>(p);
        else q8b::decode_kernel<__half, 64><<<grid, q8b::kWarps * 32, 0, stream>>>(p);
    } else {
        if (head_dim == 128) q8b::decode_kernel<__nv_bfloat16, 128><<<grid, q8b::kWarps * 32, 0, stream>>>(p);
        else q8b::decode_kernel<__nv_bfloat16, 64><<<grid, q8b::kWarps * 32, 0, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
