// pa_evict.cu -- eviction from the cache by accumulated attention weight.
//
// For a request of n tokens over its budget: the last `recent` positions stay,
// and of the others the budget - recent with the largest weights; ties go to
// the lowest position, a NaN counts as minus infinity.  The table row and the
// weights are compacted in place in position order, the weights behind them
// zeroed, the evicted slots listed in position order.
//
// How: a cluster of CTAs per request.  The cut is found by a radix select over
// the weights' bits in an order-preserving integer form: four passes of eight
// bits, each a 256-bin count per CTA, summed over the cluster through
// distributed shared memory, all ranks' counts requested at once (a loop over
// them took 1700 cycles a pass; three passes of 11 bits read eight times as much
// from the other SMs and were slower, 17.5 us for 32K tokens; 1024 threads, or
// one addition per distinct bin of a warp, 12.3 and 11.0 us against 9.9).  Then
// one ordered pass: a token is kept if its key is above the cut, or equal to it
// and among the first `ties` of those; both running counts come from ballots, so
// positions need no sort.  Kept tokens only ever move towards the front, so a
// chunk's tokens are all read before any is written (one cluster barrier) and
// later chunks are never overwritten.
// Bound: latency (a handful of cluster barriers); 8 n bytes read, 8 per kept
// token and 8 per evicted one written.  32768 tokens to 8192: 10.1 us (the bytes
// alone 0.1); 64 requests of up to 16000 tokens to 2000: 12.6 us (0.5).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace cg = cooperative_groups;

constexpr int kEvThreads = 512;
constexpr int kEvPer = 8;                              // tokens per thread of a chunk
constexpr int kEvChunk = kEvThreads * kEvPer;          // tokens per CTA and chunk
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvMaxCluster = 8;
constexpr int kEvBins = 256;

struct EvictArgs {
    int32_t *req_to_token;
    float *weights;
    const int32_t *req_pool_indices, *seq_lens;
    int32_t *new_lens, *freed, *err;
    int req_rows, max_ctx, budget, recent;
};

// weights as unsigned integers in the same order; -0 = +0, NaN = -infinity
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (!(w == w)) return 0x007FFFFFu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(const EvictArgs a)
{
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / C;
    __shared__ int s_hist[2][kEvBins];
    __shared__ int s_sum[kEvWarps];
    __shared__ int2 s_cnt[2];                 // this CTA's (sure, ties) of a chunk
    __shared__ int s_sure[kEvWarps], s_ties[kEvWarps];
    __shared__ int s_bin, s_above;

    pdl_wait();
    pdl_launch_dependents();
    const int len = __ldcg(a.seq_lens + b), row = __ldg(a.req_pool_indices + b);
    int bits = 0;
    if (row < 0 || row >= a.req_rows) bits |= PA_DEVERR_ROW;
    if (len < 0 || len > a.max_ctx) bits |= PA_DEVERR_LEN;
    // two requests of one row would both compact it: the later one is refused
    // (requests without tokens, a batch's padding, do not count: looked at only
    // where a row comes twice)
    int again = 0;
    for (int c = tid; c < b; c += kEvThreads) again |= __ldg(a.req_pool_indices + c) == row;
    if (__syncthreads_or(again) && len > 0) {
        again = 0;
        for (int c = tid; c < b; c += kEvThreads)
            again |= __ldg(a.req_pool_indices + c) == row && __ldcg(a.seq_lens + c) > 0;
        if (__syncthreads_or(again)) bits |= PA_DEVERR_ROW;
    }
    const int n = len < 0 ? 0 : min(len, a.max_ctx);
    if (bits || n <= a.budget) {              // the same for every CTA of the cluster
        if (bits & PA_DEVERR_LEN) cl.sync();  // new_lens may be seq_lens: every CTA has read the length that changes
        if (rank == 0 && tid == 0) {
            a.new_lens[b] = n;
            if (bits) set_error(a.err, bits);
        }
        return;
    }
    int32_t *tab = a.req_to_token + (int64_t)row * a.max_ctx;
    float *wts = a.weights + (int64_t)row * a.max_ctx;
    int32_t *freed = a.freed + (int64_t)b * a.max_ctx;
    const int cand = n - a.recent, want = a.budget - a.recent;   // want < cand
    const int span = C * kEvChunk, chunks = (n + span - 1) / span;

    // token j of (chunk, e): warps hold 32 kEvPer consecutive tokens
    auto token = [&](int chunk, int e) { return chunk * span + rank * kEvChunk + (warp * kEvPer + e) * 32 + lane; };
    float w0[kEvPer];                          // the first chunk's weights and slots stay in registers
    int slot0[kEvPer];
#pragma unroll
    for (int e = 0; e < kEvPer; ++e) {
        const int j = token(0, e);
        w0[e] = j < n ? wts[j] : 0.f;
        slot0[e] = j < n ? tab[j] : 0;
    }
    // ---- the cut: the `want`-th largest key of the first `cand` tokens
    uint32_t prefix = 0;
    int left = want;                           // still to be taken among keys that match the prefix
    if (want > 0) {
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            int *hist = s_hist[pass & 1];
            if (tid < kEvBins) hist[tid] = 0;
            __syncthreads();
            for (int c = 0; c < chunks; ++c) {
#pragma unroll
                for (int e = 0; e < kEvPer; ++e) {
                    const int j = token(c, e);
                    const uint32_t key = weight_key(c == 0 ? w0[e] : j < n ? wts[j] : 0.f);
                    const bool in = j < cand && (pass == 0 || (key >> (shift + 8)) == (prefix >> (shift + 8)));
                    if (in) atomicAdd(hist + ((key >> shift) & 255u), 1);
                }
            }
            cl.sync();
            // thread t < 256 holds bin 255 - t
            int v = 0, incl = 0;
            if (tid < kEvBins) {
                int x[kEvMaxCluster];
#pragma unroll
                for (int r = 0; r < kEvMaxCluster; ++r) x[r] = r < C ? cl.map_shared_rank(hist, r)[kEvBins - 1 - tid] : 0;
#pragma unroll
                for (int r = 0; r < kEvMaxCluster; ++r) v += x[r];
                incl = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                if (lane == 31) s_sum[warp] = incl;
            }
            __syncthreads();
            if (tid < kEvBins) {
                int above = incl - v;                         // and the warps with higher bins
                for (int w = 0; w < warp; ++w) above += s_sum[w];
                if (above < left && left <= above + v) {
                    s_bin = kEvBins - 1 - tid;
                    s_above = above;
                }
            }
            __syncthreads();
            prefix |= (uint32_t)s_bin << shift;
            left -= s_above;
        }
    } else {
        prefix = 0xFFFFFFFFu;                  // no key is above it, and none of those equal is taken
    }
    // keys above `prefix` stay, and the first `left` equal to it

    // ---- the ordered pass
    int done_sure = 0, done_ties = 0;          // of the chunks before
    for (int c = 0; c < chunks; ++c) {
        float w[kEvPer];
        int slot[kEvPer];
        unsigned sure[kEvPer], ties[kEvPer];
        int ns = 0, nt = 0;
#pragma unroll
        for (int e = 0; e < kEvPer; ++e) {
            const int j = token(c, e);
            w[e] = c == 0 ? w0[e] : j < n ? wts[j] : 0.f;
            slot[e] = c == 0 ? slot0[e] : j < n ? tab[j] : 0;
            const uint32_t key = weight_key(w[e]);
            sure[e] = __ballot_sync(0xffffffffu, j < n && (j >= cand || key > prefix));
            ties[e] = __ballot_sync(0xffffffffu, j < cand && key == prefix);
            ns += __popc(sure[e]);
            nt += __popc(ties[e]);
        }
        if (lane == 0) {
            s_sure[warp] = ns;
            s_ties[warp] = nt;
        }
        __syncthreads();
        if (warp == 0) {
            int x = lane < kEvWarps ? s_sure[lane] : 0, y = lane < kEvWarps ? s_ties[lane] : 0;
            int xi = x, yi = y;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int p = __shfl_up_sync(0xffffffffu, xi, o), q = __shfl_up_sync(0xffffffffu, yi, o);
                if (lane >= o) xi += p, yi += q;
            }
            if (lane < kEvWarps) {
                s_sure[lane] = xi - x;
                s_ties[lane] = yi - y;
            }
            if (lane == 31) s_cnt[c & 1] = make_int2(xi, yi);
        }
        cl.sync();                             // every token of the chunk has been read, every count is there
        int bs = done_sure + s_sure[warp], bt = done_ties + s_ties[warp];
        int2 cnt[kEvMaxCluster];
#pragma unroll
        for (int r = 0; r < kEvMaxCluster; ++r) cnt[r] = r < C ? *cl.map_shared_rank(&s_cnt[c & 1], r) : make_int2(0, 0);
#pragma unroll
        for (int r = 0; r < kEvMaxCluster; ++r) {
            done_sure += cnt[r].x;
            done_ties += cnt[r].y;
            if (r < rank) bs += cnt[r].x, bt += cnt[r].y;
        }
        const unsigned below = (1u << lane) - 1u;
#pragma unroll
        for (int e = 0; e < kEvPer; ++e) {
            const int j = token(c, e);
            const int s = bs + __popc(sure[e] & below), t = bt + __popc(ties[e] & below);
            const int kept = s + min(t, left);             // kept tokens before j
            const bool keep = (sure[e] >> lane & 1u) || ((ties[e] >> lane & 1u) && t < left);
            if (j < n) {
                if (keep) {
                    tab[kept] = slot[e];
                    wts[kept] = w[e];
                } else {
                    freed[j - kept] = slot[e];
                }
                if (j >= a.budget) wts[j] = 0.f;
            }
            bs += __popc(sure[e]);
            bt += __popc(ties[e]);
        }
        __syncthreads();                       // s_sure, s_ties reuse
    }
    if (rank == 0 && tid == 0) a.new_lens[b] = a.budget;
    cl.sync();                                 // no CTA leaves while another reads its counts
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_kv_evict(int32_t *req_to_token, int req_rows, int max_ctx, const int32_t *req_pool_indices,
                                 const int32_t *seq_lens, int batch, float *weights, int budget, int recent,
                                 int32_t *new_lens, int32_t *freed, int32_t *error_word, cudaStream_t st)
{
    if (batch < 0 || req_rows <= 0 || max_ctx <= 0 || budget < 1 || recent < 0 || recent > budget) return PA_ERR_SHAPE;
    if (max_ctx > INT32_MAX - kEvMaxCluster * kEvChunk || batch > INT32_MAX / kEvMaxCluster) return PA_ERR_SHAPE;
    if (batch == 0) return PA_OK;
    if (!req_to_token || !req_pool_indices || !seq_lens || !weights || !new_lens || !freed) return PA_ERR_NULL;
    if (!aligned4(req_to_token) || !aligned4(req_pool_indices) || !aligned4(seq_lens) || !aligned4(weights) ||
        !aligned4(new_lens) || !aligned4(freed) || (error_word && !aligned4(error_word)))
        return PA_ERR_ALIGN;
    EvictArgs a{};
    a.req_to_token = req_to_token;
    a.weights = weights;
    a.req_pool_indices = req_pool_indices;
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.freed = freed;
    a.err = error_word;
    a.req_rows = req_rows;
    a.max_ctx = max_ctx;
    a.budget = budget;
    a.recent = recent;
    // as many CTAs per request as its longest row fills with one chunk each, at most 8
    int cs = 1;
    while (cs < kEvMaxCluster && (int64_t)cs * kEvChunk < max_ctx) cs *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(batch * cs));
    cfg.blockDim = dim3(kEvThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = launch_overlap() != PA_OVERLAP_OFF ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kv_evict_kernel, a) != cudaSuccess) return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
