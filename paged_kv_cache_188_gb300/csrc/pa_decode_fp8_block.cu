// pa_decode_fp8_block.cu -- the C-ABI entry point of decode attention over an
// e4m3 cache with a scale per (block of slots, kv head) (kernel in
// pa_decode_block.cuh).
#include "pa_decode_block_host.h"

using namespace pa;

extern "C" size_t pa_decode_fp8_block_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim)
{
    if (n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || n_q_heads % n_kv_heads != 0) return 0;
    return blk_ws(n_q_heads, n_kv_heads, head_dim).scores_off;
}

extern "C" pa_status pa_paged_decode_attn_fp8_block(const void *q, int batch, int n_q_heads, const void *k_buf,
                                                    const void *v_buf, pa_kv_shape s, int layer_id,
                                                    const int32_t *req_to_token, int req_rows, int max_ctx,
                                                    const int32_t *req_pool_indices, const int32_t *seq_lens, float scale,
                                                    const uint8_t *k_exp, const uint8_t *v_exp, int block, void *workspace,
                                                    size_t workspace_bytes, void *out, cudaStream_t st)
{
    const pa_status rc = check_block(q, batch, n_q_heads, k_buf, v_buf, s, layer_id, req_to_token, req_rows, max_ctx,
                                     req_pool_indices, seq_lens, true, block, k_exp, v_exp, workspace, workspace_bytes, out,
                                     false, nullptr);
    if (rc != PA_OK || batch == 0) return rc;
    BlkArgs a;
    if (!fill_block(a, q, batch, n_q_heads, k_buf, v_buf, s, layer_id, req_to_token, req_rows, max_ctx, req_pool_indices,
                    seq_lens, scale, true, block, k_exp, v_exp, workspace, workspace_bytes, out, nullptr))
        return PA_ERR_CUDA;
    return dispatch_block<true, false>(a, s.head_dim, st);
}
