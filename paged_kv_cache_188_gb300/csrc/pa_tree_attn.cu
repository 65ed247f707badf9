// pa_tree_attn.cu -- attention of drafted tokens (a tree or a chain per request)
// over the paged cache, bf16 or block-scaled e4m3.
//
//     s_j = scale <q_i, K_j>,   out_i = sum_j softmax(s)_j V_j
// over the context and the nodes whose bits the mask has.  One warp per (node,
// query head) walks the keys with a running maximum and sum: the simplest form.
#include <math.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kTreeMaxReqs = 4096;

struct TreeArgs {
    const __nv_bfloat16 *q;
    const uint8_t *k, *v;                        // the layer's rows
    const uint8_t *k_exp, *v_exp;                // the layer's exponents (e4m3 cache)
    const int32_t *qo_indptr, *req_to_token, *req_pool_indices, *seq_lens, *tree_mask;
    __nv_bfloat16 *out;
    int32_t *err;
    int T, R, Hq, Hkv, G, size, req_rows, max_ctx, mask_words, block_shift;
    float scale_log2;
};

template <int D, bool E8>
__device__ __forceinline__ void load_row(const uint8_t *rows, const uint8_t *exps, int64_t slot, int Hkv, int h, int shift,
                                         int lane, float (&x)[D / 32])
{
    constexpr int N = D / 32;
    const int64_t at = (slot * Hkv + h) * D + lane * N;
    if constexpr (E8) {
        const int e = exps[(slot >> shift) * Hkv + h];
        const float sc = e == 0 ? 0.f : __uint_as_float((uint32_t)e << 23);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            e4m3x2_floats(*reinterpret_cast<const uint16_t *>(rows + at + i), x[i], x[i + 1]);
            x[i] *= sc;
            x[i + 1] *= sc;
        }
    } else {
        const __nv_bfloat16 *r = reinterpret_cast<const __nv_bfloat16 *>(rows) + at;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __bfloat162float(r[i]);
    }
}

template <int D, bool E8>
__global__ void __launch_bounds__(256) tree_attn_kernel(const TreeArgs a)
{
    constexpr int N = D / 32;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, r = blockIdx.y;
    const int q0 = __ldg(a.qo_indptr + r), q1 = __ldg(a.qo_indptr + r + 1), n = q1 - q0;
    if (n <= 0 || q0 < 0 || q1 > a.T) {
        if (n != 0) set_error(a.err, PA_DEVERR_LEN);
        return;
    }
    int L = __ldg(a.seq_lens + r);
    const int row = __ldg(a.req_pool_indices + r);
    int bits = 0;
    if (row < 0 || row >= a.req_rows) bits |= PA_DEVERR_ROW;
    if (L < n || L > a.max_ctx || (a.tree_mask && n > 32 * (int64_t)a.mask_words)) bits |= PA_DEVERR_LEN;
    if (bits) {
        set_error(a.err, bits);
        L = 0;
    }
    const int c = L - n;
    const int32_t *tab = a.req_to_token + (int64_t)(bits ? 0 : row) * a.max_ctx;
    for (int64_t w = blockIdx.x * 8 + (threadIdx.x >> 5); w < (int64_t)n * a.Hq; w += gridDim.x * 8) {
        const int i = (int)(w / a.Hq), hq = (int)(w % a.Hq), h = hq / a.G;
        const int64_t at = ((int64_t)(q0 + i) * a.Hq + hq) * D + lane * N;
        float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) q[e] = __bfloat162float(a.q[at + e]), o[e] = 0.f;
        for (int j = 0; j < L; ++j) {
            if (j >= c) {
                const int k = j - c;
                const bool seen = a.tree_mask ? a.tree_mask[(int64_t)(q0 + i) * a.mask_words + (k >> 5)] >> (k & 31) & 1 : k <= i;
                if (!seen) continue;
            }
            const int slot = tab[j];
            if (slot < 0 || slot >= a.size) {
                set_error(a.err, PA_DEVERR_SLOT);
                continue;
            }
            float x[N], s = 0.f;
            load_row<D, E8>(a.k, a.k_exp, slot, a.Hkv, h, a.block_shift, lane, x);
#pragma unroll
            for (int e = 0; e < N; ++e) s = fmaf(q[e], x[e], s);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            s *= a.scale_log2;
            const float mn = fmaxf(m, s), mz = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m - mz), p = exp2f(s - mz);
            l = l * f + p;
            m = mn;
            if (p == 0.f && s == -INFINITY) continue;
            load_row<D, E8>(a.v, a.v_exp, slot, a.Hkv, h, a.block_shift, lane, x);
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = fmaf(p, x[e], o[e] * f);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) a.out[at + e] = __float2bfloat16_rn(l != 0.f ? o[e] / l : 0.f);
    }
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_tree_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim)
{
    if (n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || n_q_heads % n_kv_heads != 0) return 0;
    return kWorkspaceHeader;
}

extern "C" pa_status pa_paged_tree_attn(const void *q, int n_tokens, int n_q_heads, const void *k_buf, const void *v_buf,
                                        pa_kv_shape s, int layer_id, const int32_t *qo_indptr, int n_reqs,
                                        const int32_t *req_to_token, int req_rows, int max_ctx,
                                        const int32_t *req_pool_indices, const int32_t *seq_lens,
                                        const int32_t *tree_mask, int mask_words, float scale, const uint8_t *k_exp,
                                        const uint8_t *v_exp, int block, void *workspace, size_t workspace_bytes,
                                        void *out, cudaStream_t st)
{
    const bool e4m3 = block != 0;
    if (n_tokens < 0 || n_reqs < 0 || n_reqs > kTreeMaxReqs || n_q_heads <= 0 || s.n_layers <= 0 || s.size <= 0 ||
        s.n_kv_heads <= 0 || req_rows <= 0 || max_ctx <= 0 || mask_words < 0)
        return PA_ERR_SHAPE;
    if (layer_id < 0 || layer_id >= s.n_layers || n_q_heads % s.n_kv_heads != 0) return PA_ERR_SHAPE;
    if (e4m3 && !block_ok(block)) return PA_ERR_SHAPE;
    if (!e4m3 && (k_exp || v_exp)) return PA_ERR_SHAPE;
    if ((tree_mask != nullptr) != (mask_words > 0)) return PA_ERR_SHAPE;
    const int G = n_q_heads / s.n_kv_heads;
    if (G > 16 || (s.head_dim != 64 && s.head_dim != 128)) return PA_ERR_UNSUPPORTED;
    if ((int64_t)s.n_layers * s.size >= (int64_t)INT32_MAX - 16) return PA_ERR_SHAPE;
    // tiles of all segments (256 rows of nodes and heads over 128 cached tokens) in 32 bits
    if (((int64_t)n_tokens * G / 256 + n_reqs) * (((int64_t)max_ctx + 127) / 128) >= (int64_t)1 << 30) return PA_ERR_SHAPE;
    if (!workspace) return PA_ERR_NULL;
    if (!aligned256(workspace)) return PA_ERR_ALIGN;
    if (workspace_bytes < pa_tree_workspace_bytes(n_q_heads, s.n_kv_heads, s.head_dim)) return PA_ERR_WORKSPACE;
    if (n_tokens == 0 || n_reqs == 0) return PA_OK;
    if (!q || !k_buf || !v_buf || !qo_indptr || !req_to_token || !req_pool_indices || !seq_lens || !out) return PA_ERR_NULL;
    if (e4m3 && (!k_exp || !v_exp)) return PA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_buf) || !aligned16(v_buf) || !aligned16(out) || !aligned4(qo_indptr) ||
        !aligned4(req_to_token) || !aligned4(req_pool_indices) || !aligned4(seq_lens) || !aligned4(tree_mask))
        return PA_ERR_ALIGN;
    TreeArgs a{};
    const int64_t layer = (int64_t)layer_id * s.size * s.n_kv_heads * s.head_dim * (e4m3 ? 1 : 2);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const uint8_t *>(k_buf) + layer;
    a.v = static_cast<const uint8_t *>(v_buf) + layer;
    if (e4m3) {
        const int64_t off = block_layer_offset(layer_id, s.size, s.n_kv_heads, block);
        a.k_exp = k_exp + off;
        a.v_exp = v_exp + off;
        while ((1 << a.block_shift) < block) ++a.block_shift;
    }
    a.qo_indptr = qo_indptr;
    a.req_to_token = req_to_token;
    a.req_pool_indices = req_pool_indices;
    a.seq_lens = seq_lens;
    a.tree_mask = tree_mask;
    a.mask_words = mask_words;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.err = static_cast<int32_t *>(workspace);
    a.T = n_tokens;
    a.R = n_reqs;
    a.Hq = n_q_heads;
    a.Hkv = s.n_kv_heads;
    a.G = G;
    a.size = s.size;
    a.req_rows = req_rows;
    a.max_ctx = max_ctx;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    const dim3 grid(256, n_reqs);
    cudaError_t rc;
    if (e4m3) rc = s.head_dim == 64 ? launch_kernel(tree_attn_kernel<64, true>, grid, dim3(256), 0, st, a)
                                    : launch_kernel(tree_attn_kernel<128, true>, grid, dim3(256), 0, st, a);
    else rc = s.head_dim == 64 ? launch_kernel(tree_attn_kernel<64, false>, grid, dim3(256), 0, st, a)
                               : launch_kernel(tree_attn_kernel<128, false>, grid, dim3(256), 0, st, a);
    if (rc != cudaSuccess) return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
