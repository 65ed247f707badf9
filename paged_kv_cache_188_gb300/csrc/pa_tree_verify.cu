// pa_tree_verify.cu -- which drafted tokens are kept, and the token behind them,
// from the target's (and the draft's) probabilities and given random numbers.
//
// With cur = the root, w = p[cur], Z = 1, the nodes behind cur are tried in
// order: kept if u Z f[cur][x] < w[x] (f the draft's probabilities; 1 where the
// node was chosen, not drawn); a refused one takes its share off: w <- max(w - Z
// f[cur], 0), Z <- sum w (chosen: Z <- Z - w[x], w[x] <- 0).  The token that
// follows is drawn from what is left of w by its running sum.
//
// How: a cluster of CTAs per request.  What the tests need is two numbers per
// node, p and f of its token behind its parent, gathered for all nodes at once;
// the walk then runs in shared memory, a warp looking at 32 nodes at a time (the
// same in every CTA, so nothing is passed around).  Only a row that is drawn
// from, or that a refusal takes a share off, is read whole: the warps of the cluster take
// consecutive pieces of it, and the piece that holds the goal is looked through
// again.  Sums are whole numbers of 2^-48 in 64 bits: exact, so that they and
// the token do not depend on how the row is cut.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace cg = cooperative_groups;

constexpr int kVfThreads = 512;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfMaxNodes = 1024;
constexpr int kVfMaxCluster = 8;
constexpr int kVfAhead = 4;              // chunks of four probabilities that a lane has on their way

struct VerifyArgs {
    const float *p, *f;
    const int32_t *tokens, *parents, *qo_indptr;
    const float *u_accept, *u_sample;
    int32_t *accepted, *n_accepted, *next_token, *err;
    int V, T, R, max_path;
};

typedef unsigned long long u64;

// a probability: NaN and negative numbers are 0
__device__ __forceinline__ float prob(float x) { return x > 0.f ? x : 0.f; }
// in whole steps of 2^-48, nearest even (the product is exact or overflows)
__device__ __forceinline__ u64 steps(float x) { return __float2ull_rn(x * 0x1p48f); }

// The row that is summed: w of row `row` after the refusals behind it.
struct VfRow {
    const float *p, *f;     // 16-byte aligned address at or in front of the row's start; f NULL: chosen tokens
    int lead;               // elements between that address and the row
    int V, chunks;          // of four elements from that address
    int refused;            // f: number of Z in z; chosen: number of tokens in x
    const float *z;
    const int *x;
};

__device__ __forceinline__ float4 vf_load(const float *row, int c, int lead, int V)
{
    const int v0 = 4 * c - lead;
    if (v0 >= 0 && v0 + 4 <= V) return __ldg(reinterpret_cast<const float4 *>(row) + c);
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    float *e = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (v0 + i >= 0 && v0 + i < V) e[i] = __ldg(row + 4 * (int64_t)c + i);
    return r;
}

// w of the four elements of chunk c, from their probabilities
__device__ __forceinline__ void vf_weights(const VfRow &r, int c, const float4 &p4, const float4 &f4, float (&w)[4])
{
    w[0] = prob(p4.x), w[1] = prob(p4.y), w[2] = prob(p4.z), w[3] = prob(p4.w);
    if (r.f) {
        const float f[4] = {prob(f4.x), prob(f4.y), prob(f4.z), prob(f4.w)};
        for (int j = 0; j < r.refused; ++j) {
            const float z = r.z[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = prob(__fsub_rn(w[e], __fmul_rn(z, f[e])));
        }
    } else {
        for (int j = 0; j < r.refused; ++j) {
            const int d = r.x[j] - (4 * c - r.lead);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d == e) w[e] = 0.f;
        }
    }
}

// The sum of a warp's chunks c0 .. c1, every lane has it.
__device__ __forceinline__ u64 vf_sum(const VfRow &r, int c0, int c1, int lane)
{
    u64 sum = 0;
#pragma unroll 1
    for (int c = c0 + lane; c < c1; c += 32 * kVfAhead) {
        float4 p4[kVfAhead], f4[kVfAhead];
#pragma unroll
        for (int i = 0; i < kVfAhead; ++i) {
            const int cc = c + 32 * i;
            p4[i] = cc < c1 ? vf_load(r.p, cc, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f);
            f4[i] = cc < c1 && r.f ? vf_load(r.f, cc, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kVfAhead; ++i) {
            float w[4];
            vf_weights(r, c + 32 * i, p4[i], f4[i], w);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += steps(w[e]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// The first element of chunks c0 .. c1 at which the running sum, from `run` on, passes `goal`.
__device__ __forceinline__ int vf_find(const VfRow &r, int c0, int c1, u64 run, u64 goal, int lane)
{
#pragma unroll 1
    for (int cb = c0; cb < c1; cb += 32) {
        const int c = cb + lane;
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        if (c < c1)
            vf_weights(r, c, vf_load(r.p, c, r.lead, r.V),
                       r.f ? vf_load(r.f, c, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f), w);
        u64 s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = steps(w[e]);
        const u64 mine = s[0] + s[1] + s[2] + s[3];
        u64 incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, run + incl > goal);
        if (hit) {
            const int src = __ffs(hit) - 1;
            u64 at = run + incl - mine;
            int v = 4 * c - r.lead;
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                at += s[e];
                if (at > goal) break;
                ++v;
            }
            return __shfl_sync(0xffffffffu, v, src);
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    return -1;
}

__global__ void __launch_bounds__(kVfThreads) tree_verify_kernel(const VerifyArgs a)
{
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = blockIdx.x / C;
    __shared__ int s_parent[kVfMaxNodes], s_tok[kVfMaxNodes];
    __shared__ float s_p[kVfMaxNodes], s_f[kVfMaxNodes], s_u[kVfMaxNodes];
    __shared__ float s_z[kVfMaxNodes];             // Z of each refusal behind cur (f given)
    __shared__ int s_x[kVfMaxNodes];               // or its token (chosen)
    __shared__ u64 s_sum[kVfWarps], s_total[2];
    __shared__ int s_state[4];                     // cur, refusals behind it, next node to try, kept

    pdl_wait();
    pdl_launch_dependents();
    const int q0 = __ldg(a.qo_indptr + r), q1 = __ldg(a.qo_indptr + r + 1);
    int n = q1 - q0;
    int32_t *path = a.accepted + (int64_t)r * a.max_path;
    if (n <= 0 || n > kVfMaxNodes || q0 < 0 || q1 > a.T) {     // the same for every CTA of the cluster
        if (rank == 0) {
            for (int i = tid; i < a.max_path; i += kVfThreads) path[i] = -1;
            if (tid == 0) {
                a.n_accepted[r] = 0;
                a.next_token[r] = -1;
                if (n != 0) set_error(a.err, PA_DEVERR_LEN);
            }
        }
        return;
    }
    for (int i = tid; i < n; i += kVfThreads) {
        const int par = i > 0 ? __ldg(a.parents + q0 + i) : -1, x = __ldg(a.tokens + q0 + i);
        const bool ok = i > 0 && par >= 0 && par < i && x >= 0 && x < a.V;
        if (i > 0 && !ok && rank == 0) set_error(a.err, PA_DEVERR_TREE);
        const int64_t at = (int64_t)(q0 + (ok ? par : 0)) * a.V + (ok ? x : 0);
        s_parent[i] = ok ? par : -1;
        s_tok[i] = x;
        s_p[i] = ok ? prob(__ldg(a.p + at)) : 0.f;
        s_f[i] = ok && a.f ? prob(__ldg(a.f + at)) : 1.f;
        s_u[i] = __ldg(a.u_accept + q0 + i);
    }
    if (tid == 0) {
        s_state[0] = 0, s_state[1] = 0, s_state[2] = 1, s_state[3] = 1;
        s_z[0] = 1.f;
        if (rank == 0) path[0] = 0;
    }
    const float us = __ldg(a.u_sample + r);
    __syncthreads();

    int round = 0;
    float Z = 1.f;                                 // warp 0: of the weights behind the refusals so far
    VfRow w;
    int c0 = 0, c1 = 0;
    u64 mine = 0, total = 0, before = 0;
    while (true) {
        if (warp == 0) {
            // nodes from `next` on whose parent is cur, in order; stops at one that needs a Z which is yet to be summed
            int cur = s_state[0], refused = s_state[1], next = s_state[2], kept = s_state[3];
            bool pending = false, sum = false;     // pending: the last refusal's Z is not known
            while (kept < a.max_path) {
                int found = -1;
                for (int b = next & ~31; b < n && found < 0; b += 32) {
                    const int i = b + lane;
                    const unsigned hit = __ballot_sync(0xffffffffu, i >= next && i < n && s_parent[i] == cur);
                    if (hit) found = b + __ffs(hit) - 1;
                }
                if (found < 0) break;
                next = found;
                sum = pending;
                if (sum) break;
                ++next;
                // w[x] behind the refusals
                float have = s_p[found];
                const float f = s_f[found];
                if (a.f) {
                    for (int j = 0; j < refused; ++j) have = prob(__fsub_rn(have, __fmul_rn(s_z[j], f)));
                } else {
                    for (int j = 0; j < refused; ++j)
                        if (s_x[j] == s_tok[found]) have = 0.f;
                }
                const float share = __fmul_rn(s_u[found], a.f ? __fmul_rn(Z, f) : Z);
                if (share < have) {
                    if (lane == 0 && rank == 0) path[kept] = found;
                    ++kept;
                    cur = found;
                    refused = 0;
                    Z = 1.f;
                } else if (a.f) {
                    ++refused;                     // s_z[refused] is Z once it is summed
                    pending = true;
                } else {
                    if (lane == 0) s_x[refused] = s_tok[found];
                    ++refused;
                    Z = prob(__fsub_rn(Z, have));
                    __syncwarp();
                }
            }
            __syncwarp();
            if (lane == 0) {
                s_state[0] = cur, s_state[1] = refused, s_state[2] = sum ? next : n, s_state[3] = kept;
            }
        }
        __syncthreads();
        // ---- the sum of w: a refusal's Z, or the last one
        const int64_t row = (int64_t)(q0 + s_state[0]) * a.V;
        w.lead = (int)(row & 3);
        w.p = a.p + (row - w.lead);
        w.f = a.f && s_state[1] > 0 ? a.f + (row - w.lead) : nullptr;
        w.V = a.V;
        w.chunks = (w.lead + a.V + 3) / 4;
        w.refused = s_state[1];
        w.z = s_z;
        w.x = s_x;
        const int per = (w.chunks + C * kVfWarps - 1) / (C * kVfWarps);
        c0 = min(w.chunks, (rank * kVfWarps + warp) * per);
        c1 = min(w.chunks, c0 + per);
        bool plain = false;
        while (true) {
            mine = vf_sum(w, c0, c1, lane);
            if (lane == 0) s_sum[warp] = mine;
            __syncthreads();
            u64 block = 0;
            before = 0;
#pragma unroll
            for (int i = 0; i < kVfWarps; ++i) {
                const u64 x = s_sum[i];
                if (i < warp) before += x;
                block += x;
            }
            if (tid == 0) s_total[round & 1] = block;
            cl.sync();
            total = 0;
            u64 t[kVfMaxCluster];
#pragma unroll
            for (int i = 0; i < kVfMaxCluster; ++i) t[i] = i < C ? *cl.map_shared_rank(&s_total[round & 1], i) : 0;
#pragma unroll
            for (int i = 0; i < kVfMaxCluster; ++i) {
                if (i < rank) before += t[i];
                total += t[i];
            }
            ++round;
            if (total > 0 || plain || s_state[2] < n || w.refused == 0) break;
            // the refusals left nothing: the target's row itself
            plain = true;
            w.refused = 0;
            w.f = nullptr;
            __syncthreads();                       // s_sum reuse
        }
        if (s_state[2] >= n) break;
        Z = __fmul_rn(__ull2float_rn(total), 0x1p-48f);
        if (tid == 0) s_z[s_state[1]] = Z;
        __syncthreads();
    }
    // ---- the token: the first at which the running sum passes u total
    const int kept = s_state[3];
    if (rank == 0) {
        for (int i = kept + tid; i < a.max_path; i += kVfThreads) path[i] = -1;
        if (tid == 0) {
            a.n_accepted[r] = kept;
            if (total == 0) a.next_token[r] = -1;
        }
    }
    if (total > 0) {
        // floor(u total), u in steps of 2^-64 (exact for u of 2^-40 and more, as of 24 bits)
        const u64 goal = __umul64hi(us > 0.f ? (us < 1.f ? __float2ull_rz(us * 0x1p64f) : ~0ull) : 0ull, total);
        if (goal >= before && goal < before + mine) {
            const int v = vf_find(w, c0, c1, before, goal, lane);
            if (lane == 0) a.next_token[r] = v;
        }
    }
    cl.sync();                                     // no CTA leaves while another reads its sums
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_tree_verify(const float *target_probs, const float *draft_probs, int vocab, const int32_t *tokens,
                                    const int32_t *parents, int n_tokens, const int32_t *qo_indptr, int n_reqs,
                                    const float *u_accept, const float *u_sample, int32_t *accepted, int max_path,
                                    int32_t *n_accepted, int32_t *next_token, int32_t *error_word, cudaStream_t st)
{
    if (vocab <= 0 || vocab > (1 << 24) || n_tokens < 0 || n_reqs < 0 || n_reqs > 65536 || max_path <= 0) return PA_ERR_SHAPE;
    if (n_reqs == 0) return PA_OK;
    if (!qo_indptr || !u_sample || !accepted || !n_accepted || !next_token) return PA_ERR_NULL;
    if (n_tokens > 0 && (!target_probs || !tokens || !parents || !u_accept)) return PA_ERR_NULL;
    if (!aligned16(target_probs) || !aligned16(draft_probs) || !aligned4(tokens) || !aligned4(parents) ||
        !aligned4(qo_indptr) || !aligned4(u_accept) || !aligned4(u_sample) || !aligned4(accepted) || !aligned4(n_accepted) ||
        !aligned4(next_token) || !aligned4(error_word))
        return PA_ERR_ALIGN;
    VerifyArgs a{};
    a.p = target_probs;
    a.f = draft_probs;
    a.tokens = tokens;
    a.parents = parents;
    a.qo_indptr = qo_indptr;
    a.u_accept = u_accept;
    a.u_sample = u_sample;
    a.accepted = accepted;
    a.n_accepted = n_accepted;
    a.next_token = next_token;
    a.err = error_word;
    a.V = vocab;
    a.T = n_tokens;
    a.R = n_reqs;
    a.max_path = max_path;
    int cs = 1;
    while (cs < kVfMaxCluster && cs * 4096 < vocab) cs *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n_reqs * cs));
    cfg.blockDim = dim3(kVfThreads);
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
    if (cudaLaunchKernelEx(&cfg, tree_verify_kernel, a) != cudaSuccess) return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
