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
//
// Measured, in a graph: 64 chains of 5 drafted tokens, V = 131072 (67 MB of rows that
// are drawn from: 9.9 us at a copy's rate) 19.4 us: sums by 64-bit conversions 39.8,
// exact float additions 33, running sums of a piece's groups and 512 threads 19.  32
// trees of chosen tokens, V = 100003, 15.1 us; 16 of drawn ones 21.9 (refusals wait
// for one another, each a pass over rows that are kept in registers where they fit;
// read again each time 29.7).  One chain 7.4 us: the kernel's start, four dependent
// reads and a row's sum across the cluster.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace cg = cooperative_groups;

constexpr int kVfMaxNodes = 1024;
constexpr int kVfMaxCluster = 8;
constexpr int kVfAhead = 4;              // chunks of four probabilities that a lane has on their way
constexpr int kVfGroups = 8;             // running sums kept of a warp's piece, so that little of it is looked through again

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

// Whole steps of 2^-48, nearest even, without the conversion to 64 bits (83 cycles a warp: a row of 131072 took 13 us
// in it).  Below 2, adding a power of two leaves w rounded to that sum's last place in its low bits, and what is left
// over is exact: three such sums take 22, 22 and 4 bits.  The words are added as they are; what the powers of two
// contribute is taken off at the end.
struct Steps {
    uint32_t hi, mid, lo;
};
constexpr uint32_t kOneHi = 0x40000000u, kOneMid = 0x35400000u, kOneLo = 0x33400000u;   // 2, 1.5 2^-21, 1.5 2^-25
__device__ __forceinline__ void steps_add(Steps &s, float w)
{
    const float m1 = __uint_as_float(kOneHi), m2 = __uint_as_float(kOneMid), m3 = __uint_as_float(kOneLo);
    const float t1 = __fadd_rn(w, m1), r1 = __fsub_rn(w, __fsub_rn(t1, m1));         // places of 2^-22
    const float t2 = __fadd_rn(r1, m2), r2 = __fsub_rn(r1, __fsub_rn(t2, m2));       // 2^-44
    const float t3 = __fadd_rn(r2, m3);                                             // 2^-48
    s.hi += __float_as_uint(t1);
    s.mid += __float_as_uint(t2);
    s.lo += __float_as_uint(t3);
}
// of n additions: a value below 2 is at most 2^23 places of the first word, so 511 of them stay in its 32 bits
constexpr int kStepsMost = 511;
static_assert(4 * kVfAhead <= kStepsMost, "a lane's additions between two sums");
__device__ __forceinline__ u64 steps_sum(const Steps &s, uint32_t n)
{
    const long long mid = (int32_t)(s.mid - n * kOneMid), lo = (int32_t)(s.lo - n * kOneLo);
    return ((u64)(s.hi - n * kOneHi) << 26) + (u64)((mid << 4) + lo);
}
__device__ __forceinline__ u64 steps(float w)
{
    if (!(w < 2.f)) return __float2ull_rn(w * 0x1p48f);
    Steps s{0, 0, 0};
    steps_add(s, w);
    return steps_sum(s, 1);
}

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

// w of the four elements of a chunk, from their probabilities (chosen tokens are not taken out here)
__device__ __forceinline__ void vf_weights(const VfRow &r, const float4 &p4, const float4 &f4, float (&w)[4])
{
    w[0] = prob(p4.x), w[1] = prob(p4.y), w[2] = prob(p4.z), w[3] = prob(p4.w);
    if (r.f) {
        const float f[4] = {prob(f4.x), prob(f4.y), prob(f4.z), prob(f4.w)};
#pragma unroll 1
        for (int j = 0; j < r.refused; ++j) {
            const float z = r.z[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = prob(__fsub_rn(w[e], __fmul_rn(z, f[e])));
        }
    }
}

// The sum of a warp's chunks c0 .. c1, every lane has it.  groups[g]: of the chunks in front of c0 + g stride.
__device__ __forceinline__ u64 vf_sum(const VfRow &r, int c0, int c1, int stride, u64 *groups, int lane)
{
    u64 sum = 0;
#pragma unroll 1
    for (int cb = c0, g = 0; cb < c1; ++g) {
        if (lane == 0) groups[g] = sum;
        u64 mine = 0;
#pragma unroll 1
        for (const int end = min(c1, cb + stride); cb < end; cb += 32 * kVfAhead) {
            const int c = cb + lane;
            float4 p4[kVfAhead], f4[kVfAhead];
#pragma unroll
            for (int i = 0; i < kVfAhead; ++i) {
                const int cc = c + 32 * i;
                p4[i] = cc < end ? vf_load(r.p, cc, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f);
                f4[i] = cc < end && r.f ? vf_load(r.f, cc, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            Steps s{0, 0, 0};
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < kVfAhead; ++i) {
                float w[4];
                vf_weights(r, p4[i], f4[i], w);
                if (fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])) < 2.f) {
                    n += 4;
#pragma unroll
                    for (int e = 0; e < 4; ++e) steps_add(s, w[e]);
                } else {
                    // (no probability)
                    mine += steps(w[0]) + steps(w[1]) + steps(w[2]) + steps(w[3]);
                }
            }
            mine += steps_sum(s, n);
        }
        cb = min(c1, c0 + (g + 1) * stride);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        sum += mine;
    }
    return sum;
}

// A piece of at most 128 chunks, kept in the registers of its warp from one refusal to the next: w is not computed, nor
// the row read, again.
struct VfHeld {
    int64_t row;            // -1: nothing
    int refused;            // taken off so far
    float4 w[kVfAhead], f[kVfAhead];
};
__device__ __forceinline__ u64 vf_sum_held(const VfRow &r, int64_t row, int c0, int c1, VfHeld &h, int lane)
{
    if (h.row != row) {
        h.row = row;
        h.refused = 0;
#pragma unroll
        for (int i = 0; i < kVfAhead; ++i) {
            const int c = c0 + lane + 32 * i;
            const float4 p = c < c1 ? vf_load(r.p, c, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 f = c < c1 && r.f ? vf_load(r.f, c, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f);
            h.w[i] = make_float4(prob(p.x), prob(p.y), prob(p.z), prob(p.w));
            h.f[i] = make_float4(prob(f.x), prob(f.y), prob(f.z), prob(f.w));
        }
    }
    if (r.f) {
#pragma unroll 1
        for (; h.refused < r.refused; ++h.refused) {
            const float z = r.z[h.refused];
#pragma unroll
            for (int i = 0; i < kVfAhead; ++i) {
                h.w[i].x = prob(__fsub_rn(h.w[i].x, __fmul_rn(z, h.f[i].x)));
                h.w[i].y = prob(__fsub_rn(h.w[i].y, __fmul_rn(z, h.f[i].y)));
                h.w[i].z = prob(__fsub_rn(h.w[i].z, __fmul_rn(z, h.f[i].z)));
                h.w[i].w = prob(__fsub_rn(h.w[i].w, __fmul_rn(z, h.f[i].w)));
            }
        }
    }
    u64 sum = 0;
    Steps s{0, 0, 0};
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < kVfAhead; ++i) {
        const float w[4] = {h.w[i].x, h.w[i].y, h.w[i].z, h.w[i].w};
        if (fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])) < 2.f) {
            n += 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) steps_add(s, w[e]);
        } else {
            sum += steps(w[0]) + steps(w[1]) + steps(w[2]) + steps(w[3]);
        }
    }
    sum += steps_sum(s, n);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// The first element of chunks c0 .. c1 at which the running sum, from `run` on, passes `goal`.
__device__ __forceinline__ int vf_find(const VfRow &r, int c0, int c1, u64 run, u64 goal, int lane)
{
#pragma unroll 1
    for (int cb = c0; cb < c1; cb += 32 * kVfAhead) {
        float4 p4[kVfAhead], f4[kVfAhead];
#pragma unroll
        for (int i = 0; i < kVfAhead; ++i) {
            const int c = cb + 32 * i + lane;
            p4[i] = c < c1 ? vf_load(r.p, c, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f);
            f4[i] = c < c1 && r.f ? vf_load(r.f, c, r.lead, r.V) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kVfAhead; ++i) {
            const int c = cb + 32 * i + lane;
            float w[4];
            vf_weights(r, p4[i], f4[i], w);
            if (!r.f) {
#pragma unroll 1
                for (int j = 0; j < r.refused; ++j) {
                    const int d = r.x[j] - (4 * c - r.lead);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (d == e) w[e] = 0.f;
                }
            }
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
    }
    return -1;
}

template <int kVfThreads, int kBlocks, bool HELD>
__global__ void __launch_bounds__(kVfThreads, kBlocks) tree_verify_kernel(const VerifyArgs a)
{
    constexpr int kVfWarps = kVfThreads / 32;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = blockIdx.x / C;
    __shared__ int s_parent[kVfMaxNodes], s_tok[kVfMaxNodes];
    __shared__ float s_p[kVfMaxNodes], s_f[kVfMaxNodes], s_u[kVfMaxNodes];
    __shared__ float s_z[kVfMaxNodes];             // Z of each refusal behind cur (f given)
    __shared__ int s_x[kVfMaxNodes];               // or its token (chosen), each once
    __shared__ float s_xp[kVfMaxNodes];            // and that one's probability
    __shared__ u64 s_sum[2][kVfWarps], s_total[2][kVfMaxCluster];   // sums of this CTA's warps, of the cluster's CTAs
    __shared__ u64 s_groups[kVfWarps][kVfGroups];
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
    cl.barrier_arrive();                           // every CTA of the cluster runs before any writes into it
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

    cl.barrier_wait();
    int round = 0;
    float Z = 1.f;                                 // warp 0: of the weights behind the refusals so far
    VfRow w;
    VfHeld held;
    held.row = -1;
    int c0 = 0, c1 = 0, stride = 1;
    u64 mine = 0, total = 0, before = 0;
    while (true) {
        if (warp == 0) {
            // nodes from `next` on whose parent is cur, in order; stops at one that needs a Z which is yet to be summed
            int cur = s_state[0], refused = s_state[1], next = s_state[2], kept = s_state[3];
            bool pending = false, sum = false;     // pending: the last refusal's Z is not known
            int older = refused;                   // refused tokens that are not among the chunk's lanes
            unsigned gone = 0;                     // lanes whose tokens were refused behind cur
            // 32 nodes at a time, a lane's in its registers
#pragma unroll 1
            for (int b = next & ~31; b < n && !sum; b += 32) {
                const int i = b + lane;
                const bool in = i < n;
                const int par = in ? s_parent[i] : -1, tok = in ? s_tok[i] : -1;
                const float np = in ? s_p[i] : 0.f, nf = in ? s_f[i] : 0.f, nu = in ? s_u[i] : 0.f;
                while (kept < a.max_path) {
                    const unsigned hit = __ballot_sync(0xffffffffu, i >= next && par == cur);
                    if (!hit) break;
                    const int src = __ffs(hit) - 1;
                    next = b + src;
                    sum = pending;
                    if (sum) break;
                    ++next;
                    // w[x] behind the refusals
                    float have = __shfl_sync(0xffffffffu, np, src);
                    const float f = __shfl_sync(0xffffffffu, nf, src), u = __shfl_sync(0xffffffffu, nu, src);
                    const int x = __shfl_sync(0xffffffffu, tok, src);
                    if (a.f) {
#pragma unroll 1
                        for (int j = 0; j < refused; ++j) have = prob(__fsub_rn(have, __fmul_rn(s_z[j], f)));
                    } else {
#pragma unroll 1
                        for (int j = 0; j < older; j += 32)
                            if (__any_sync(0xffffffffu, j + lane < older && s_x[j + lane] == x)) have = 0.f;
                        if (__ballot_sync(0xffffffffu, tok == x) & gone) have = 0.f;
                    }
                    const float share = __fmul_rn(u, a.f ? __fmul_rn(Z, f) : Z);
                    if (share < have) {
                        if (lane == 0 && rank == 0) path[kept] = b + src;
                        ++kept;
                        cur = b + src;
                        refused = older = 0;
                        gone = 0;
                        Z = 1.f;
                    } else if (a.f) {
                        ++refused;                 // s_z[refused] is Z once it is summed
                        pending = true;
                    } else if (have > 0.f) {       // (else it adds nothing, or was refused before)
                        if (lane == 0) {
                            s_x[refused] = x;
                            s_xp[refused] = have;
                        }
                        ++refused;
                        gone |= 1u << src;
                        Z = prob(__fsub_rn(Z, have));
                    }
                }
                older = refused;
                gone = 0;
                __syncwarp();
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
        stride = ((per + kVfGroups - 1) / kVfGroups + 32 * kVfAhead - 1) / (32 * kVfAhead) * (32 * kVfAhead);
        bool plain = false;
        while (true) {
            u64 *sums = s_sum[round & 1], *totals = s_total[round & 1];
            if constexpr (HELD) {
                if (lane == 0) s_groups[warp][0] = 0;
                mine = vf_sum_held(w, plain ? row + ((int64_t)1 << 62) : row, c0, c1, held, lane);
            } else {
                mine = vf_sum(w, c0, c1, stride, s_groups[warp], lane);
            }
            if (lane == 0) sums[warp] = mine;
            __syncthreads();
            if (!w.f && w.refused > 0) {
                // chosen tokens that were refused come off the sums of the pieces that hold them
                for (int j = tid; j < w.refused; j += kVfThreads) {
                    const int g = (s_x[j] + w.lead) / 4 / per - rank * kVfWarps;
                    if (g < 0 || g >= kVfWarps) continue;
                    const u64 off = 0ull - steps(s_xp[j]);
                    atomicAdd(sums + g, off);
                    for (int i = ((s_x[j] + w.lead) / 4 - (g + rank * kVfWarps) * per) / stride + 1; i < kVfGroups; ++i)
                        atomicAdd(s_groups[g] + i, off);
                }
                __syncthreads();
                mine = sums[warp];
            }
            u64 block = 0;
            before = 0;
#pragma unroll
            for (int i = 0; i < kVfWarps; ++i) {
                const u64 x = sums[i];
                if (i < warp) before += x;
                block += x;
            }
            // every CTA's sum goes to all of them
            if (tid < C) *cl.map_shared_rank(totals + rank, tid) = block;
            cl.sync();
            total = 0;
            u64 t[kVfMaxCluster];
#pragma unroll
            for (int i = 0; i < kVfMaxCluster; ++i) t[i] = i < C ? totals[i] : 0;
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
            // its group of the piece, from the running sums in front of them
            const int groups = (c1 - c0 + stride - 1) / stride;
            const int g = __popc(__ballot_sync(0xffffffffu, lane < groups && before + s_groups[warp][lane % kVfGroups] <= goal)) - 1;
            before += s_groups[warp][g];
            const int v = vf_find(w, c0 + g * stride, c1, before, goal, lane);
            if (lane == 0) a.next_token[r] = v;
        }
    }
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
    // the more threads the fewer round trips a piece of a row takes: 512 (two CTAs an SM) where all CTAs are then on the
    // GPU at once, else 256 (four).  Drawn nodes' rows are summed after every refusal: kept in registers where a warp's
    // piece fits (512 chunks of four to a CTA of 16 warps, 128 a warp) and an SM has one CTA
    const int64_t ctas = (int64_t)n_reqs * cs;
    const bool held = draft_probs && ctas <= num_sms() && (vocab + (vocab % 4 ? 3 : 0) + 3) / 4 <= cs * 16 * 32 * kVfAhead;
    const int threads = ctas <= 2 * num_sms() ? 512 : 256;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
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
    auto kern = held ? tree_verify_kernel<512, 1, true>
                     : threads == 512 ? tree_verify_kernel<512, 2, false> : tree_verify_kernel<256, 4, false>;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
