// pa_accept.cu -- the accepted path of a request's drafted tokens stays in the
// cache, the other nodes go: in the page table, or by moving K/V rows.
//
// Table form: one CTA per request.  A node's rank is the number of path entries
// in front of it (a binary search), so that kept nodes go to their rank and the
// others to their index minus it.  Kept entries only ever move towards the front: a
// chunk's entries are all read before any is written, and later chunks' are never
// overwritten.
// Move form: a CTA per (request, layer, K or V).  A thread owns 16 bytes of the
// row and takes the path's entries in order, several read before they are written:
// position c + k never lies behind node e_k >= k, nor is it a later entry's node.
//
// Measured, in a graph: 64 requests' entries 3.8 us, which is a launch and four
// dependent reads; 32 requests' rows in 16 layers (19 MB read and written, 2.8 us at
// a copy's rate) 5.7 us.
#include <cuda_runtime.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kAcThreads = 128;
constexpr int kAcBatch = 8;             // rows a thread has on their way

struct AcceptArgs {
    int32_t *req_to_token;
    const int32_t *req_pool_indices, *seq_lens, *qo_indptr, *accepted, *n_accepted;
    int32_t *new_lens, *freed, *err;
    uint8_t *k, *v;
    int64_t layer_bytes;
    int T, R, req_rows, max_ctx, max_path, n_layers, size, row_bytes;
};

// A request's nodes [q0, q0 + n), context c and accepted number; false where it is left as it is, for a fault or because
// it has no nodes (a batch's padding, whose row and length may be anything); its length then is `len`.  Whole CTA;
// `report` by one CTA per request.
struct AcReq {
    int q0, n, c, kept, row, len;
};
__device__ __forceinline__ bool ac_request(const AcceptArgs &a, int r, bool report, AcReq &q)
{
    const int tid = threadIdx.x;
    q.q0 = __ldg(a.qo_indptr + r);
    const int q1 = __ldg(a.qo_indptr + r + 1), L = __ldcg(a.seq_lens + r);
    q.row = __ldg(a.req_pool_indices + r);
    q.kept = __ldcg(a.n_accepted + r);
    q.n = q1 - q.q0;
    q.c = L - q.n;
    q.len = max(0, min(L, a.max_ctx));
    int bits = 0;
    const bool range = q.n >= 0 && q.q0 >= 0 && q1 <= a.T;
    if (q.n != 0 && (!range || L < q.n || L > a.max_ctx || L < 0)) bits |= PA_DEVERR_LEN;
    if (q.n > 0 && (q.row < 0 || q.row >= a.req_rows)) bits |= PA_DEVERR_ROW;
    const bool count = q.kept >= 0 && q.kept <= a.max_path && q.kept <= max(q.n, 0);
    // earlier requests with nodes: of the same row, or whose range ends behind this one's start (two would list their slots
    // in the same entries)
    int again = 0, over = 0, wrong = !count;
    if (range && q.n > 0) {
        for (int b = tid; b < r; b += kAcThreads) {
            const int s = __ldg(a.qo_indptr + b), e = __ldg(a.qo_indptr + b + 1);
            again |= s < e && __ldg(a.req_pool_indices + b) == q.row;
            over |= s >= 0 && s < e && e <= a.T && e > q.q0;
        }
        const int32_t *path = a.accepted + (int64_t)r * a.max_path;
        if (count)
            for (int k = tid; k < q.kept; k += kAcThreads) {
                const int e = __ldcg(path + k);
                wrong |= e < 0 || e >= q.n || (k > 0 && e <= __ldcg(path + k - 1));
            }
    }
    if (__syncthreads_or(again | over | wrong)) {
        if (__syncthreads_or(again)) bits |= PA_DEVERR_ROW;
        if (__syncthreads_or(over)) bits |= PA_DEVERR_LEN;
        if (__syncthreads_or(wrong)) bits |= PA_DEVERR_TREE;
    }
    if (bits && report && tid == 0) set_error(a.err, bits);
    if (bits != 0 || q.n == 0) return false;
    q.len = q.c + q.kept;
    return true;
}

__global__ void __launch_bounds__(kAcThreads) kv_accept_table_kernel(const AcceptArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int r = blockIdx.x, tid = threadIdx.x;
    AcReq q;
    const bool ok = ac_request(a, r, true, q);     // every thread has read the length (new_lens may be seq_lens)
    if (tid == 0) a.new_lens[r] = q.len;
    if (!ok) return;
    int32_t *tab = a.req_to_token + (int64_t)q.row * a.max_ctx + q.c;
    const int32_t *path = a.accepted + (int64_t)r * a.max_path;
    for (int i0 = 0; i0 < q.n; i0 += kAcThreads) {
        const int i = i0 + tid;
        int slot = 0, rank = 0;
        bool keep = false;
        if (i < q.n) {
            slot = tab[i];
            int hi = q.kept;
            while (rank < hi) {                    // path entries below i
                const int mid = (rank + hi) >> 1;
                if (__ldcg(path + mid) < i) rank = mid + 1; else hi = mid;
            }
            keep = rank < q.kept && __ldcg(path + rank) == i;
        }
        __syncthreads();
        if (i < q.n) {
            if (keep) tab[rank] = slot;
            else a.freed[q.q0 + i - rank] = slot;
        }
    }
}

__global__ void __launch_bounds__(kAcThreads) kv_accept_move_kernel(const AcceptArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, layers2 = 2 * a.n_layers;
    const int r = (int)(blockIdx.x / layers2), y = (int)(blockIdx.x % layers2);
    AcReq q;
    const bool ok = ac_request(a, r, y == 0, q);
    if (y == 0 && tid == 0) a.new_lens[r] = q.len;
    if (!ok) return;
    const int32_t *tab = a.req_to_token + (int64_t)q.row * a.max_ctx + q.c;
    const int32_t *path = a.accepted + (int64_t)r * a.max_path;
    if (y == 0)
        for (int i = q.kept + tid; i < q.n; i += kAcThreads) a.freed[q.q0 + i - q.kept] = tab[i];
    uint8_t *rows = (y & 1 ? a.v : a.k) + (y >> 1) * a.layer_bytes;
    for (int col = tid * 16; col < a.row_bytes; col += kAcThreads * 16) {
        for (int k0 = 0; k0 < q.kept; k0 += kAcBatch) {
            uint4 x[kAcBatch];
            int dst[kAcBatch];
#pragma unroll
            for (int i = 0; i < kAcBatch; ++i) {
                dst[i] = -1;
                if (k0 + i < q.kept) {
                    const int e = __ldcg(path + k0 + i);
                    const int from = __ldg(tab + e), to = __ldg(tab + k0 + i);
                    if (from < 0 || from >= a.size || to < 0 || to >= a.size) {
                        set_error(a.err, PA_DEVERR_SLOT);
                    } else if (from != to) {
                        dst[i] = to;
                        x[i] = *reinterpret_cast<const uint4 *>(rows + (int64_t)from * a.row_bytes + col);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kAcBatch; ++i)
                if (dst[i] >= 0) *reinterpret_cast<uint4 *>(rows + (int64_t)dst[i] * a.row_bytes + col) = x[i];
        }
    }
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_kv_accept(int32_t *req_to_token, int req_rows, int max_ctx, const int32_t *req_pool_indices,
                                  const int32_t *seq_lens, const int32_t *qo_indptr, int n_tokens, int n_reqs,
                                  const int32_t *accepted, int max_path, const int32_t *n_accepted, int32_t *new_lens,
                                  int32_t *freed, void *k_buf, void *v_buf, pa_kv_shape s, int elem_bytes,
                                  int32_t *error_word, cudaStream_t st)
{
    const bool move = k_buf || v_buf;
    if (n_tokens < 0 || n_reqs < 0 || req_rows <= 0 || max_ctx <= 0 || max_path <= 0) return PA_ERR_SHAPE;
    if (move) {
        if (s.n_layers <= 0 || s.size <= 0 || s.n_kv_heads <= 0 || s.head_dim <= 0 || (elem_bytes != 1 && elem_bytes != 2))
            return PA_ERR_SHAPE;
        if ((int64_t)s.n_kv_heads * s.head_dim * elem_bytes > (1 << 24) ||
            (int64_t)n_reqs * s.n_layers * 2 >= (int64_t)INT32_MAX)
            return PA_ERR_SHAPE;
        if (s.n_kv_heads * s.head_dim * elem_bytes % 16 != 0) return PA_ERR_UNSUPPORTED;
    }
    if (n_reqs == 0) return PA_OK;
    if (!req_to_token || !req_pool_indices || !seq_lens || !qo_indptr || !accepted || !n_accepted || !new_lens)
        return PA_ERR_NULL;
    if (n_tokens > 0 && !freed) return PA_ERR_NULL;
    if (move && (!k_buf || !v_buf)) return PA_ERR_NULL;
    if (!aligned4(req_to_token) || !aligned4(req_pool_indices) || !aligned4(seq_lens) || !aligned4(qo_indptr) ||
        !aligned4(accepted) || !aligned4(n_accepted) || !aligned4(new_lens) || !aligned4(freed) || !aligned4(error_word) ||
        !aligned16(k_buf) || !aligned16(v_buf))
        return PA_ERR_ALIGN;
    // a request's length is written while other requests' are read, and in the move form its own as well
    if ((move || seq_lens != new_lens) && seq_lens < new_lens + n_reqs && new_lens < seq_lens + n_reqs)
        return PA_ERR_SHAPE;
    AcceptArgs a{};
    a.req_to_token = req_to_token;
    a.req_pool_indices = req_pool_indices;
    a.seq_lens = seq_lens;
    a.qo_indptr = qo_indptr;
    a.accepted = accepted;
    a.n_accepted = n_accepted;
    a.new_lens = new_lens;
    a.freed = freed;
    a.err = error_word;
    a.T = n_tokens;
    a.R = n_reqs;
    a.req_rows = req_rows;
    a.max_ctx = max_ctx;
    a.max_path = max_path;
    cudaError_t rc;
    if (move) {
        a.k = static_cast<uint8_t *>(k_buf);
        a.v = static_cast<uint8_t *>(v_buf);
        a.n_layers = s.n_layers;
        a.size = s.size;
        a.row_bytes = s.n_kv_heads * s.head_dim * elem_bytes;
        a.layer_bytes = (int64_t)s.size * a.row_bytes;
        rc = launch_kernel(kv_accept_move_kernel, dim3((unsigned)(n_reqs * 2 * s.n_layers)), dim3(kAcThreads), 0, st, a);
    } else {
        rc = launch_kernel(kv_accept_table_kernel, dim3((unsigned)n_reqs), dim3(kAcThreads), 0, st, a);
    }
    if (rc != cudaSuccess) return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
