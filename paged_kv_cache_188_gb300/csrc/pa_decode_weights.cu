// pa_decode_weights.cu -- the C-ABI entry point of decode attention that also
// adds each cached token's attention weight to a running table, over the bf16
// cache or the block-scaled e4m3 cache (kernel in pa_decode_block.cuh).
#include "pa_decode_block_host.h"

using namespace pa;

extern "C" size_t pa_decode_weights_workspace_bytes(int max_batch, int64_t max_tokens, int n_q_heads, int n_kv_heads,
                                                    int head_dim)
{
    if (max_batch < 0 || max_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 ||
        n_q_heads % n_kv_heads != 0)
        return 0;
    // every request's last tile may be partly filled
    const size_t tiles = (size_t)(max_tokens / kBlkTile) + (size_t)max_batch;
    return blk_ws(n_q_heads, n_kv_heads, head_dim).scores_off + tiles * blk_tile_bytes(n_q_heads);
}

extern "C" pa_status pa_paged_decode_attn_weights(const void *q, int batch, int n_q_heads, const void *k_buf,
                                                  const void *v_buf, pa_kv_shape s, int layer_id,
                                                  const int32_t *req_to_token, int req_rows, int max_ctx,
                                                  const int32_t *req_pool_indices, const int32_t *seq_lens, float scale,
                                                  const uint8_t *k_exp, const uint8_t *v_exp, int block, float *weights,
                                                  void *workspace, size_t workspace_bytes, void *out, cudaStream_t st)
{
    if (block == 0 && (k_exp || v_exp)) return PA_ERR_SHAPE;
    const pa_status rc = check_block(q, batch, n_q_heads, k_buf, v_buf, s, layer_id, req_to_token, req_rows, max_ctx,
                                     req_pool_indices, seq_lens, block != 0, block, k_exp, v_exp, workspace,
                                     workspace_bytes, out, true, weights);
    if (rc != PA_OK || batch == 0) return rc;
    BlkArgs a;
    if (!fill_block(a, q, batch, n_q_heads, k_buf, v_buf, s, layer_id, req_to_token, req_rows, max_ctx, req_pool_indices,
                    seq_lens, scale, block != 0, block, k_exp, v_exp, workspace, workspace_bytes, out, weights))
        return PA_ERR_CUDA;
    return block != 0 ? decode_block_weights(a, s.head_dim, st) : dispatch_block<false, true>(a, s.head_dim, st);
}
