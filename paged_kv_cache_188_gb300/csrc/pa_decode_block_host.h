// pa_decode_block_host.h -- checks, workspace layout and launch arguments
// shared by the entry points of pa_decode_block.cuh's kernels.
#pragma once
#include "pa_decode_block.cuh"

namespace pa {

// Workspace: header, tickets (one per worker, zero between calls), partials (two
// slots per worker), log-sum-exps, then the score tiles (weights calls).  Offsets
// depend on the head counts alone; the tickets' on nothing.
struct BlkWs {
    size_t tickets_off, ml_off, o_off, lse_off, scores_off;
};
inline BlkWs blk_ws(int Hq, int Hkv, int D)
{
    const int G = Hq / Hkv;
    BlkWs w;
    w.tickets_off = kWorkspaceHeader;
    w.ml_off = align_up(w.tickets_off + kBlkMaxWorkers * 4, 256);
    w.o_off = align_up(w.ml_off + (size_t)2 * kBlkMaxWorkers * G * 2 * 4, 256);
    w.lse_off = align_up(w.o_off + (size_t)2 * kBlkMaxWorkers * G * D * 4, 256);
    w.scores_off = align_up(w.lse_off + (size_t)kBlkMaxBatch * Hq * 4, 256);
    return w;
}
inline size_t blk_tile_bytes(int Hq) { return (size_t)Hq * kBlkTile * 4; }

// Everything that does not touch CUDA.  `weights_call`: scores are kept.
inline pa_status check_block(const void *q, int batch, int Hq, const void *k_buf, const void *v_buf, pa_kv_shape s,
                             int layer_id, const int32_t *req_to_token, int req_rows, int max_ctx,
                             const int32_t *req_pool_indices, const int32_t *seq_lens, bool e4m3, int block,
                             const uint8_t *k_exp, const uint8_t *v_exp, const void *workspace,
                             size_t workspace_bytes, const void *out, bool weights_call, const float *weights)
{
    if (batch < 0 || batch > kBlkMaxBatch || Hq <= 0 || s.n_layers <= 0 || s.size <= 0 || s.n_kv_heads <= 0 ||
        req_rows <= 0 || max_ctx <= 0)
        return PA_ERR_SHAPE;
    if (layer_id < 0 || layer_id >= s.n_layers) return PA_ERR_SHAPE;
    if (Hq % s.n_kv_heads != 0) return PA_ERR_SHAPE;
    if (e4m3 && !block_ok(block)) return PA_ERR_SHAPE;
    const int G = Hq / s.n_kv_heads;
    if (G > 16 || Hq > kBlkMaxHeads || (s.head_dim != 64 && s.head_dim != 128)) return PA_ERR_UNSUPPORTED;
    if ((int64_t)s.n_layers * s.size >= (int64_t)INT32_MAX - 16) return PA_ERR_SHAPE;
    // tiles of all segments in 32 bits
    if (((int64_t)max_ctx + kBlkTile - 1) / kBlkTile * s.n_kv_heads * (batch > 0 ? batch : 1) >= (int64_t)INT32_MAX / 2)
        return PA_ERR_SHAPE;
    if (!workspace) return PA_ERR_NULL;
    if (!aligned256(workspace)) return PA_ERR_ALIGN;
    if (workspace_bytes < blk_ws(Hq, s.n_kv_heads, s.head_dim).scores_off) return PA_ERR_WORKSPACE;
    // a weights call needs one tile per request at the least; the lengths are on the device
    if (weights_call && (workspace_bytes - blk_ws(Hq, s.n_kv_heads, s.head_dim).scores_off) / blk_tile_bytes(Hq) < (size_t)batch)
        return PA_ERR_WORKSPACE;
    if (batch == 0) return PA_OK;
    if (!q || !k_buf || !v_buf || !req_to_token || !req_pool_indices || !seq_lens || !out) return PA_ERR_NULL;
    if (e4m3 && (!k_exp || !v_exp)) return PA_ERR_NULL;
    if (weights_call && !weights) return PA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_buf) || !aligned16(v_buf) || !aligned16(out) || !aligned4(req_to_token) ||
        !aligned4(req_pool_indices) || !aligned4(seq_lens) || (weights_call && !aligned4(weights)))
        return PA_ERR_ALIGN;
    return PA_OK;
}

inline bool fill_block(BlkArgs &a, const void *q, int batch, int Hq, const void *k_buf, const void *v_buf, pa_kv_shape s,
                       int layer_id, const int32_t *req_to_token, int req_rows, int max_ctx,
                       const int32_t *req_pool_indices, const int32_t *seq_lens, float scale, bool e4m3, int block,
                       const uint8_t *k_exp, const uint8_t *v_exp, void *workspace, size_t workspace_bytes, void *out,
                       float *weights)
{
    memset(&a, 0, sizeof a);
    const int row_bytes = s.head_dim * (e4m3 ? 1 : 2), sw = row_bytes < 128 ? row_bytes : 128;
    const cuuint64_t inner = (cuuint64_t)s.n_kv_heads * s.head_dim, rows = (cuuint64_t)s.n_layers * s.size;
    const cuuint32_t box = sw / (e4m3 ? 1 : 2);
    if (!encode_tmap_rows(&a.tm_k16, k_buf, !e4m3, inner, rows, box, 16, sw) ||
        !encode_tmap_rows(&a.tm_k1, k_buf, !e4m3, inner, rows, box, 1, sw) ||
        !encode_tmap_rows(&a.tm_v16, v_buf, !e4m3, inner, rows, box, 16, sw) ||
        !encode_tmap_rows(&a.tm_v1, v_buf, !e4m3, inner, rows, box, 1, sw))
        return false;
    const BlkWs ws = blk_ws(Hq, s.n_kv_heads, s.head_dim);
    unsigned char *w = static_cast<unsigned char *>(workspace);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.req_to_token = req_to_token;
    a.req_pool_indices = req_pool_indices;
    a.seq_lens = seq_lens;
    if (e4m3) {
        const int64_t layer_exps = block_layer_offset(layer_id, s.size, s.n_kv_heads, block);
        a.k_exp = k_exp + layer_exps;
        a.v_exp = v_exp + layer_exps;
        while ((1 << a.block_shift) < block) ++a.block_shift;
    }
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.err = reinterpret_cast<int32_t *>(w);
    a.tickets = reinterpret_cast<int32_t *>(w + ws.tickets_off);
    a.ml_part = reinterpret_cast<float *>(w + ws.ml_off);
    a.o_part = reinterpret_cast<float *>(w + ws.o_off);
    a.lse = reinterpret_cast<float *>(w + ws.lse_off);
    a.scores = reinterpret_cast<float *>(w + ws.scores_off);
    a.weights = weights;
    a.batch = batch;
    a.Hq = Hq;
    a.Hkv = s.n_kv_heads;
    a.G = Hq / s.n_kv_heads;
    a.size = s.size;
    a.req_rows = req_rows;
    a.max_ctx = max_ctx;
    a.layer_row0 = layer_id * s.size;
    a.total_rows = s.n_layers * s.size;
    const size_t cap = (workspace_bytes - ws.scores_off) / blk_tile_bytes(Hq);
    a.cap_tiles = cap < (size_t)(1 << 30) ? (int)cap : 1 << 30;
    a.early_meta = early_metadata();
    a.wait_ns = wait_limit_ns();
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    return true;
}

// the weights kernels over an e4m3 cache (instances of their own translation unit)
pa_status decode_block_weights(const BlkArgs &a, int head_dim, cudaStream_t st);

}  // namespace pa
