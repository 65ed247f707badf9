#pragma once
// pa_decode_block.cuh -- decode attention on the tcgen05 tensor cores, over an
// e4m3 cache with a power-of-two scale per (block of slots, kv head) and over
// the bf16 cache, optionally keeping every token's attention weight.
//
// What it computes, for request b and query head hq = h G + g:
//     s_j = scale <q[b, hq], K_j>,  K_j = e4m3(k byte) 2^(ek_j - 127)   (or the bf16 row)
//     out[b, hq] = sum_j softmax(s)_j V_j
//     weights[row, j] += sum_hq softmax(s)_{hq, j}                      (WT)
//
// How.  The G query heads are far fewer than the 128 rows a tensor-core tile
// wants, and the cached tokens are many, so tokens (and in the second product
// the head dimension) take the M = 128 side and the heads the N side:
//     S[token, head]  = K[token, :] . Q[head, :]            A = K tile,   B = Q
//     O^T[d, head]    = sum_token V[token, d] P[head, token]  A = V^T tile, B = P
// A tile of 128 tokens then goes from TMA straight into the tensor core: no
// thread reads, converts or scales a K or V byte.  What is left for threads is
// one token (and one d) each: 128 x G scores per 128 x 2D bytes.
//   * kind::f8f6f4 takes e4m3 on both sides, so Q and P are split into e4m3
//     terms in columns of their own.  q 2^-k (k per head, its largest element
//     within 448) = q1 + q2 / 16: a bf16 has 8 significant bits, an e4m3 four,
//     so the two terms hold it exactly down to 2^-22 of the head's largest
//     element.  P = p1 + p2 / 16 + p3 / 256 holds 12 bits, with a range of
//     2^-14 below the tile's largest weight before bits are lost (f16: 11 bits).
//     bf16 cache: Q is one term, exact; P = p1 + p2 in bf16 (16 bits).
//   * a token's K scale multiplies its scores (one thread, one token); its V
//     scale joins its weight's exponent, P'_j = 2^(s_j + ev_j - R + 8), R the
//     tile's maximum of s + ev, so that a range of scales costs no bits of the
//     tokens that matter.  Each tile's O is read from tensor memory and added
//     in fp32 registers with its own 2^(R - r): nothing in tensor memory is
//     ever rescaled.
//   * l sums 2^(s - m) in fp32 with the running maximum m; each thread keeps
//     its own tokens' sum until the item ends.
//
// Work: the requests' 128-token tiles (at least one each), laid end to end, are
// cut into equal ranges of W tiles, as many as there are warpgroups (two on an
// SM) per kv head; unit (range i, head h) is worker i Hkv + h's.  All heads of a
// token are then read at about the same time, so that HBM finishes a page it has
// opened (a row's 128 bytes of one head alone, 1 KB apart: 70 us for 48 requests
// of 500 to 8192 tokens, 32 heads over 8, D = 128; 61 side by side).  A unit has
// at most two (request, head) segments it shares with others, its first and its
// last, so the fp32 partials are two slots per unit whatever the batch is.  The one that finishes a shared segment's
// last piece (a ticket per segment) merges its pieces in order (deterministic);
// a second kernel adds the weights (WT).
//
// Roles: the two warpgroups work apart, each on its own range, ring and
// tensor-memory columns, so one's softmax, item starts and item ends run beside
// the other's products; each issues its own MMAs.  Two loader warps serve each
// warpgroup: one the K tiles and exponents, one the V's.  16 consecutive slots
// move as one TMA box, any other four rows as one gather4 copy (16-byte cp.async
// copies instead: at pages of one slot 80.6 us against 75.0 for the 48 requests,
// 25.6 against 27.5 for one of 32K tokens).  Positions past the end repeat a valid
// row (weight zero), so nothing behind the last token is read.
//
// Bound, and what was measured (e4m3, D = 128, 32 heads over 8, blocks and pages of
// 16; in a graph): HBM, 2 D + 2 / block bytes per token and head: those 48 requests
// 56.4 to 57.7 us from one GPU to another, 5.1 TB/s (the floor is 42.9 us); one of
// 32768 tokens 24.9 to 25.7 (9.9); of 1000 tokens 9.7 to 10.1 (0.3): launch and plan, the first tile's chain of
// table, exponents, rows, the products' chain, then tickets and merge, each one or
// two round trips; its instructions are cold as well (a quarter of the issue slots
// lost wait for them).  Two tiles a warpgroup are too few to hide a tile's chain of
// two products, but issuing the next tile's S before O is read gains nothing (58.7
// us against 58.0): the copies are what is waited for.
#include <math.h>
#include <string.h>

#include "pa_internal.h"
#include "pa_sm100.cuh"

namespace pa {
using namespace sm100;

constexpr int kBlkTile = 128;          // tokens per tile: the MMA's M
constexpr int kBlkThreads = 256 + 128;  // two warpgroups, two loader warps for each
constexpr int kBlkMaxWorkers = 320;     // warpgroups of a launch: two per SM (152 SMs)
constexpr int kBlkMaxStages = 6;        // per warpgroup and operand
constexpr int kBlkMaxBatch = 4096;
constexpr int kBlkMaxHeads = 4096;      // query heads: their log-sum-exps beside the batch's plan in the weights kernel
constexpr int kBlkAhead = 2;            // tiles of a loader's batch
constexpr int kBlkStageBytes = (kBlkAhead * (32 * 20 + 12) + 15) / 16 * 16;
constexpr uint32_t kBlkTmemCols = 256; // per warpgroup 128: S at 0, O at 64
constexpr int kMasked = 255;           // exponent byte of a position without a token

struct BlkArgs {
    CUtensorMap tm_k16, tm_k1, tm_v16, tm_v1;   // 2-D (element, row): boxes of 16 rows, and one row (gather4)
    const __nv_bfloat16 *q;
    const int32_t *req_to_token, *req_pool_indices, *seq_lens;
    const uint8_t *k_exp, *v_exp;               // the layer's [n_blocks, Hkv] (e4m3 cache)
    __nv_bfloat16 *out;
    int32_t *err;
    int32_t *tickets;                           // [workers]: finished pieces of the shared segment that starts there
    float *ml_part;                             // [2 workers][G][2]: maximum (log2 units), sum
    float *o_part;                              // [2 workers][G][D]: relative to that maximum
    float *lse;                                 // [batch, Hq]: log2-sum-exp (WT)
    float *scores;                              // [Hkv][cap_tiles][128][G], log2 units (WT)
    float *weights;                             // [req_rows, max_ctx] (WT)
    int batch, Hq, Hkv, G, size, req_rows, max_ctx, layer_row0, block_shift, cap_tiles, early_meta, total_rows;
    int workers, stages_k, stages_v;            // two workers per CTA; ring stages per worker
    int ranges, spread;                         // ranges per head; ranges that a worker per SM serves
    uint64_t wait_ns;
    float scale_log2;
};

// Sizes of one instance: D the head dimension, E8 an e4m3 cache, GP the heads
// per kv head the columns are laid out for.
template <int D, bool E8, int GP>
struct BlkCfg {
    static constexpr int ES = E8 ? 1 : 2;
    static constexpr int QT = E8 ? 2 : 1;                 // terms of q
    static constexpr int PT = E8 ? 3 : 2;                 // terms of P
    static constexpr int NQ = (QT * GP + 15) / 16 * 16;   // columns of S
    static constexpr int NP = (PT * GP + 15) / 16 * 16;   // columns of O^T
    static constexpr int RB = D * ES;                     // bytes of a row
    static constexpr int AW = RB < 128 ? RB : 128;        // bytes of a swizzled row: 128, or 64
    static constexpr int HALVES = RB / AW;
    static constexpr int HALF = kBlkTile * AW;
    static constexpr int TILE = kBlkTile * RB;
    static constexpr int QB = NQ * RB;                    // one warpgroup's q
    // and P, which also holds O [GP][128] in fp32 when a piece ends
    static constexpr int PB = NP * kBlkTile * ES > GP * 512 ? NP * kBlkTile * ES : GP * 512;
    static constexpr int QSteps = RB / 32, PSteps = kBlkTile * ES / 32;   // a K step is 32 bytes of either type
    // offsets behind the rings
    __host__ __device__ static constexpr int align_k(int x) { return (x + 1023) & ~1023; }
    static constexpr int OffQ = 0;
    static constexpr int OffP = 2 * align_k(QB);
    static constexpr int OffMeta = OffP + 2 * align_k(PB);              // exponent bytes [2][K, V][stages][128]
    static constexpr int OffStage = OffMeta + 4 * kBlkMaxStages * kBlkTile;   // the loaders' batches
    static constexpr int OffBar = OffStage + 4 * kBlkStageBytes;
    static constexpr int kBars = 4 * kBlkMaxStages + 3;   // per warpgroup: K and V full and empty, S, O, drain
    static constexpr int OffRed = OffBar + 2 * kBars * 8; // fp32 per warpgroup: [4][2 GP] maxima, [4][GP] sums, [GP] q factors
    static constexpr int kRed = 13 * GP;
    static constexpr int OffPref = (OffRed + 2 * kRed * 4 + 7) & ~7;
    // after the prefix array [batch + 1]: each request's (length, table row), int2 [batch]
    __host__ __device__ static constexpr int off_req(int batch) { return OffPref + (batch + 2) / 2 * 8; }
    static constexpr size_t fixed(int batch) { return 1024 + (size_t)off_req(batch) + (size_t)batch * 8; }
};
constexpr size_t kBlkSmemLimit = 232448 - 512;   // opt-in maximum minus static shared memory

// smem descriptor with the swizzle of AW-byte rows (128: type 2, 64: type 4)
template <int AW>
__device__ __forceinline__ uint64_t blk_desc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes)
{
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)((lbo_bytes >> 4) & 0x3FFF) << 16 |
           (uint64_t)((sbo_bytes >> 4) & 0x3FFF) << 32 | (uint64_t)1 << 46 | (uint64_t)(AW == 128 ? 2 : 4) << 61;
}
// byte offset of 16-byte chunk c of row r in a swizzled tile of AW-byte rows
template <int AW>
__device__ __forceinline__ uint32_t blk_off(int r, int c)
{
    return AW == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <bool E8>
__device__ __forceinline__ void blk_umma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc)
{
    if constexpr (E8) umma_ss_f8(d_tmem, a_desc, b_desc, idesc, acc);
    else umma_ss(d_tmem, a_desc, b_desc, idesc, acc);
}

__device__ __forceinline__ float blk_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// warp maximum; a NaN is ignored unless all are
__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int blk_tiles(int n) { return n > 0 ? (n + kBlkTile - 1) / kBlkTile : 1; }
__device__ __forceinline__ int blk_len(const BlkArgs &a, int b)
{
    const int n = __ldg(a.seq_lens + b), row = __ldg(a.req_pool_indices + b);
    return (row < 0 || row >= a.req_rows || n < 0) ? 0 : min(n, a.max_ctx);
}

// s_pref[0 .. batch] = first tile of each request within one kv head's run;
// s_req (may be null) = each request's length and table row.  Whole block of
// NT threads; s_w holds one int per warp.
template <int NT>
__device__ __forceinline__ void blk_plan(const BlkArgs &a, int *s_pref, int2 *s_req, int *s_w)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.batch;
    const int per = (B + NT - 1) / NT, lo = min(B, tid * per), hi = min(B, lo + per);
    int run = 0;
#pragma unroll 1
    for (int b = lo; b < hi; ++b) run += blk_tiles(blk_len(a, b));
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_w[warp] = incl;
    __syncthreads();
    int base = 0;
#pragma unroll 1
    for (int w = 0; w < warp; ++w) base += s_w[w];
    int excl = base + incl - run;
#pragma unroll 1
    for (int b = lo; b < hi; ++b) {
        s_pref[b] = excl;
        const int n = blk_len(a, b);
        if (s_req) s_req[b] = make_int2(n, __ldg(a.req_pool_indices + b));
        excl += blk_tiles(n);
    }
    if (tid == NT - 1) s_pref[B] = base + incl;
    __syncthreads();
}

// Length of a head's ranges in tiles.
__device__ __forceinline__ int blk_width(const int *s_pref, int B, int ranges) { return (s_pref[B] + ranges - 1) / ranges; }

// The walk over one unit's pieces of segments.
struct BlkWalk {
    int x, xe, h, b;       // next tile and end of the range, head, request
    int S0, tb;            // the request's first tile and its tiles
    int t0, t1, n, row;    // the piece: tiles [t0, t1) of the request, its tokens and table row
    int live;              // tiles of the piece with tokens: t1 - t0, or 0
};
__device__ __forceinline__ BlkWalk blk_begin(const int *s_pref, int B, int Hkv, int W, int unit)
{
    BlkWalk k;
    const int i = unit / Hkv, total = s_pref[B];
    k.h = unit - i * Hkv;
    k.x = (int)min((long long)i * W, (long long)total);
    k.xe = min(k.x + W, total);
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pref[mid] <= k.x) lo = mid; else hi = mid;
    }
    k.b = lo;
    return k;
}
// the piece at k.x; false past the end
__device__ __forceinline__ bool blk_piece(const int *s_pref, const int2 *s_req, BlkWalk &k)
{
    if (k.x >= k.xe) return false;
    k.S0 = s_pref[k.b];
    k.tb = s_pref[k.b + 1] - k.S0;
    k.t0 = k.x - k.S0;
    k.t1 = min(k.xe - k.S0, k.tb);
    k.n = s_req[k.b].x;
    k.row = s_req[k.b].y;
    k.live = k.n > 0 ? k.t1 - k.t0 : 0;
    return true;
}
__device__ __forceinline__ void blk_next(BlkWalk &k)
{
    k.x = k.S0 + k.t1;
    if (k.t1 == k.tb) ++k.b;
}

// ------------------------------------------------------------------ loader
// K (isv false) or V rows and exponents of a worker's tiles, in order of its
// units (unit, unit + workers, ...), in
// batches of kBlkAhead: while a batch is copied, the next one's table entries
// are on their way to registers and, from its middle on, the exponents that
// hang on them.  (With tens of MB in flight a read takes several microseconds;
// a look-ahead kept in rotating registers, each move of which waits for the
// value, left the copies waiting for their indices: 70 us for 48 ragged requests
// against 57; batches of 4 and 6 tiles took 58.6 and 63.2.)
// A batch that has arrived is put in shared memory, so that the copies are one
// rolled loop: a TMA instruction costs its warp about 100 cycles of issue, a
// tile of 16-slot pages eight of them per operand.
struct BlkStage {
    int4 slot[kBlkAhead][32];       // table entries of positions p0 + 4 lane + e
    uint32_t ex[kBlkAhead][32];     // their exponent bytes
    int h[kBlkAhead], n[kBlkAhead], p0[kBlkAhead];   // kv head, tokens of the request (0: no more tiles), first position
};
static_assert(sizeof(BlkStage) <= kBlkStageBytes, "a batch fits its area");

template <int D, bool E8, int GP>
__device__ __forceinline__ void blk_loader(const BlkArgs &a, const int *s_pref, const int2 *s_req, int W, int unit,
                                           uint32_t ring, int stages, BlkStage *stage, unsigned char *meta, uint32_t full,
                                           uint32_t empty, volatile int *s_abort, bool isv, int lane)
{
    using C = BlkCfg<D, E8, GP>;
    const CUtensorMap *m16 = isv ? &a.tm_v16 : &a.tm_k16, *m1 = isv ? &a.tm_v1 : &a.tm_k1;
    const uint8_t *exps = isv ? a.v_exp : a.k_exp;
    const int units = a.ranges * a.Hkv;
    BlkWalk k;
    bool more = false;
    // to the next unit that has a piece
    auto open = [&]() {
#pragma unroll 1
        for (more = false; !more && unit < units; unit += a.workers) {
            k = blk_begin(s_pref, a.batch, a.Hkv, W, unit);
            more = blk_piece(s_pref, s_req, k);
        }
    };
    open();
    int i = 0;                  // next tile of the piece
    // the batch on its way
    int slot[kBlkAhead][4], ex[kBlkAhead][4], h[kBlkAhead], n[kBlkAhead], p0[kBlkAhead];
    auto fetch = [&]() {
#pragma unroll
        for (int u = 0; u < kBlkAhead; ++u) {
#pragma unroll 1
            while (more && i >= k.live) {
                blk_next(k);
                more = blk_piece(s_pref, s_req, k);
                if (!more) open();
                i = 0;
            }
            n[u] = p0[u] = h[u] = 0;
            int64_t row = 0;
            if (more) {
                row = k.row;
                h[u] = k.h;
                n[u] = k.n;
                p0[u] = (k.t0 + i) * kBlkTile;
                ++i;
            }
            const int32_t *src = a.req_to_token + row * a.max_ctx;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int p = p0[u] + 4 * lane + e;
                slot[u][e] = ld_nc_ordered_s32_if(p < n[u], src + (p < n[u] ? p : 0));
            }
        }
    };
    auto load_exps = [&]() {
#pragma unroll
        for (int u = 0; u < kBlkAhead; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool ok = slot[u][e] >= 0 && slot[u][e] < a.size;
                ex[u][e] = !ok ? kMasked : !E8 ? 0 : __ldcg(exps + (int64_t)(slot[u][e] >> a.block_shift) * a.Hkv + h[u]);
            }
    };
    fetch();
    load_exps();
    int st = 0, seq = 0, errs = 0;      // ring stage and number of the next tile
    uint32_t ph = 0;
    bool go = true;
    while (go) {
#pragma unroll
        for (int u = 0; u < kBlkAhead; ++u) {
            stage->slot[u][lane] = make_int4(slot[u][0], slot[u][1], slot[u][2], slot[u][3]);
            if (lane == 0) {
                stage->h[u] = h[u];
                stage->n[u] = n[u];
                stage->p0[u] = p0[u];
            }
        }
        __syncwarp();
        fetch();
#pragma unroll 1
        for (int u = 0; u < kBlkAhead; ++u) {
            const int tn = stage->n[u];
            if (tn <= 0) {
                go = false;
                break;
            }
            if (u == kBlkAhead / 2) load_exps();
            // the stage's previous tile has been multiplied
            if (seq >= stages &&
                !__all_sync(0xffffffffu, mbar_wait(empty + st * 8, ph ^ 1, s_abort, a.err, PA_DEVERR_TIMEOUT, a.wait_ns))) {
                go = false;
                break;
            }
            const uint32_t dst = ring + st * C::TILE, fb = full + st * 8;
            const int4 raw = stage->slot[u][lane];
            int sl[4] = {raw.x, raw.y, raw.z, raw.w};
            bool ok[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ok[e] = sl[e] >= 0 && sl[e] < a.size;
                if (!ok[e] && stage->p0[u] + 4 * lane + e < tn) errs |= PA_DEVERR_SLOT;
            }
            const int mine = ok[0] ? sl[0] : ok[1] ? sl[1] : ok[2] ? sl[2] : ok[3] ? sl[3] : -1;
            const unsigned has = __ballot_sync(0xffffffffu, mine >= 0);
            const int some = __shfl_sync(0xffffffffu, mine, has ? __ffs(has) - 1 : 0);   // a valid row of the tile
            const int s0 = __shfl_sync(0xffffffffu, sl[0], lane & ~3);
            const bool run = ok[0] && ok[1] && ok[2] && ok[3] && sl[0] == s0 + 4 * (lane & 3) && sl[1] == sl[0] + 1 &&
                             sl[2] == sl[0] + 2 && sl[3] == sl[0] + 3;
            const bool page = ((__ballot_sync(0xffffffffu, run) >> (lane & ~3)) & 0xFu) == 0xFu;
            const bool none = ((has >> (lane & ~3)) & 0xFu) == 0u;      // the lane's 16 positions have no row
            if (has) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sl[e] = a.layer_row0 + (ok[e] ? sl[e] : some);
                const int col = stage->h[u] * D;
                if (page || none) {
                    // a page's rows, or rows out of range, which read as zeros
                    if ((lane & 3) == 0) {
#pragma unroll
                        for (int hh = 0; hh < C::HALVES; ++hh)
                            tma_load_2d(dst + hh * C::HALF + (lane >> 2) * 16 * C::AW, m16, col + hh * (C::AW / C::ES),
                                        none ? a.total_rows : sl[0], fb);
                    }
                } else {
#pragma unroll
                    for (int hh = 0; hh < C::HALVES; ++hh)
                        tma_gather4(dst + hh * C::HALF + lane * 4 * C::AW, m1, col + hh * (C::AW / C::ES), sl[0], sl[1], sl[2],
                                    sl[3], fb);
                }
            } else {
                // no valid row at all: zeros (weight zero times whatever bits lie there could be NaN)
#pragma unroll 1
                for (int o = lane * 16; o < C::TILE; o += 512) st_shared_v4(dst + o, 0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            if (u == 0) {
                // the batch's exponents, behind its first copies: they may still be on their way
#pragma unroll
                for (int w = 0; w < kBlkAhead; ++w)
                    stage->ex[w][lane] = (uint32_t)(ex[w][0] | ex[w][1] << 8 | ex[w][2] << 16 | ex[w][3] << 24);
            }
            reinterpret_cast<uint32_t *>(meta + st * kBlkTile)[lane] = stage->ex[u][lane];
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(fb, has ? C::TILE : 0u);
            ++seq;
            if (++st == stages) {
                st = 0;
                ph ^= 1;
            }
        }
        __syncwarp();
    }
    // the warp leaves only when its copies have landed, whether or not anyone has
    // given up by now: the other warpgroup may do so later, after which nobody
    // waits for these, and the shared memory would go away under them
#pragma unroll 1
    for (int j = max(0, seq - stages); j < seq; ++j) mbar_drain(full + (j % stages) * 8, (j / stages) & 1);
    if (errs) set_error(a.err, errs);
    __syncwarp();
}

// Pieces of request b's segments: ranges i0 .. i1.  A piece that does not start
// its range is the unit's last (slot 1).
struct BlkSpan {
    int i0, i1, first;      // first: piece 0 does not start range i0
};
__device__ __forceinline__ BlkSpan blk_span(const int *s_pref, int W, int b)
{
    BlkSpan s;
    const int S0 = s_pref[b];
    s.i0 = S0 / W;
    s.i1 = (s_pref[b + 1] - 1) / W;
    s.first = S0 > s.i0 * W;
    return s;
}

// Merge of a shared segment by the warpgroup that finished its last piece: all
// partials into `scratch` (the worker's ring, free by now) by asynchronous
// copies, the (m, l) pairs beside them, one round trip for all the pieces that
// fit (38 of a single long request do), then every element summed in the
// pieces' order.
template <int D, int GP, bool WT>
__device__ __forceinline__ void blk_merge(const BlkArgs &a, const BlkSpan &s, int b, int h, int t, int bar_id,
                                          float *scratch, int scratch_bytes)
{
    const int lane = t & 31, warp = t >> 5, G = a.G, np = s.i1 - s.i0 + 1;
    auto slot = [&](int p) { return 2 * ((s.i0 + p) * a.Hkv + h) + (p == 0 ? s.first : 0); };   // piece p's partials
    // [G] sums, [G] log-sum-exps; [np][G] maxima, later weights; [np][G] sums; partials
    float *s_L = scratch, *s_lse = scratch + 16, *s_w = scratch + 32, *s_l = s_w + np * G;
    float *s_o = scratch + (32 + 2 * np * G + 3) / 4 * 4;
    const int chunks = G * D / 4;                          // 16-byte chunks of a piece
    const int cap = (scratch_bytes - (int)((s_o - scratch) * 4)) / (G * D * 4);
    auto copy = [&](int p0, int n) {
#pragma unroll 2
        for (int p = 0; p < n; ++p) {
            const float *src = a.o_part + (int64_t)slot(p0 + p) * G * D;
#pragma unroll 1
            for (int c = t; c < chunks; c += 128) cp_async_16(smem_u32(s_o) + (p * chunks + c) * 16, src + c * 4, 16);
        }
    };
    copy(0, min(np, cap));
#pragma unroll 1
    for (int i = t; i < np * G; i += 128) {
        const int p = i / G;
        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.ml_part + (slot(p) * G + (i - p * G)) * 2));
        s_w[i] = ml.x;
        s_l[i] = ml.y;
    }
    named_bar_sync(bar_id, 128);
#pragma unroll 1
    for (int g = warp; g < G; g += 4) {
        float M = -INFINITY;
#pragma unroll 1
        for (int p = lane; p < np; p += 32) M = fmaxf(M, s_w[p * G + g]);
        M = warp_max(M);
        const float Mz = M == -INFINITY ? 0.f : M;
        float L = 0.f;
#pragma unroll 1
        for (int p = lane; p < np; p += 32) {
            const float w = blk_ex2(s_w[p * G + g] - Mz);
            s_w[p * G + g] = w;
            L += w * s_l[p * G + g];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0) {
            s_L[g] = L;
            s_lse[g] = L != 0.f ? M + log2f(L) : INFINITY;
        }
    }
    constexpr int NJ = (GP * D / 4 + 127) / 128;           // chunks per thread
    float4 acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int p0 = 0; p0 < np; p0 += cap) {
        const int n = min(cap, np - p0);
        if (p0 > 0) {
            named_bar_sync(bar_id, 128);                   // the last batch has been read
            copy(p0, n);
        }
        cp_async_wait_all();
        named_bar_sync(bar_id, 128);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int c = t + j * 128;
            if (c >= chunks) break;
            const float4 *so = reinterpret_cast<const float4 *>(s_o) + c;
            const float *w = s_w + p0 * G + c * 4 / D;
#pragma unroll 2
            for (int p = 0; p < n; ++p) {
                const float4 v = so[p * chunks];
                const float x = w[p * G];
                acc[j].x += x * v.x;
                acc[j].y += x * v.y;
                acc[j].z += x * v.z;
                acc[j].w += x * v.w;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int c = t + j * 128;
        if (c >= chunks) break;
        const int g = c * 4 / D;
        const float L = s_L[g], inv = L != 0.f ? 1.f / L : 0.f;
        const int64_t hq = (int64_t)b * a.Hq + h * G + g;
        const uint2 o = make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv), pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
        *reinterpret_cast<uint2 *>(a.out + hq * D + (c * 4 - g * D)) = o;
        if (WT && c * 4 == g * D) a.lse[hq] = s_lse[g];
    }
    named_bar_sync(bar_id, 128);                           // scratch reuse
}

// ------------------------------------------------------------------ kernel
template <int D, bool E8, int GP, bool WT>
__global__ void __launch_bounds__(kBlkThreads, 1) decode_block_kernel(const __grid_constant__ BlkArgs a)
{
    using C = BlkCfg<D, E8, GP>;
    constexpr int ES = C::ES, AW = C::AW;
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_w[kBlkThreads / 32];
    __shared__ int s_abort_storage;
    __shared__ uint32_t s_tmem;
    __shared__ int s_last[2][2];
    const uint32_t raw = smem_u32(smem_raw), rings = (raw + 1023u) & ~1023u;
    const int ring_bytes = (a.stages_k + a.stages_v) * C::TILE;          // one worker's
    unsigned char *base = smem_raw + (rings - raw) + (size_t)2 * ring_bytes;
    volatile int *s_abort = &s_abort_storage;
    int *s_pref = reinterpret_cast<int *>(base + C::OffPref);
    int2 *s_req = reinterpret_cast<int2 *>(base + C::off_req(a.batch));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // this warp's warpgroup (loaders: the one they serve) and its barriers
    const int wg = warp < 8 ? warp >> 2 : (warp - 8) >> 1;
    const uint32_t all_bars = smem_u32(base + C::OffBar), bars = all_bars + wg * C::kBars * 8;
    const uint32_t kfull = bars, vfull = bars + kBlkMaxStages * 8, kempty = vfull + kBlkMaxStages * 8,
                   vempty = kempty + kBlkMaxStages * 8, sfull = vempty + kBlkMaxStages * 8, ofull = sfull + 8, drain = ofull + 8;
    const uint32_t kring = rings + wg * ring_bytes, vring = kring + a.stages_k * C::TILE;
    unsigned char *kmeta = base + C::OffMeta + wg * 2 * kBlkMaxStages * kBlkTile, *vmeta = kmeta + kBlkMaxStages * kBlkTile;

    if (tid < 2 * C::kBars) mbar_init(all_bars + tid * 8, 1);
    if (tid < 32) fence_mbar_init();
    static_assert(2 * C::kBars <= 64, "the first two warps initialise the barriers");
    if (tid >= 32 && tid < 64) fence_mbar_init();
    if (tid == 0) s_abort_storage = 0;
    if (warp == 4) tmem_alloc(smem_u32(&s_tmem), kBlkTmemCols);
    if (warp >= 8 && lane == 0) {
        prefetch_tmap(warp & 1 ? &a.tm_v16 : &a.tm_k16);
        prefetch_tmap(warp & 1 ? &a.tm_v1 : &a.tm_k1);
    }
    if (!a.early_meta) pdl_wait();
    blk_plan<kBlkThreads>(a, s_pref, s_req, s_w);
    if (a.early_meta) pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0) {
#pragma unroll 1
        for (int b = tid; b < a.batch; b += kBlkThreads) {
            const int row = __ldg(a.req_pool_indices + b), n = __ldg(a.seq_lens + b);
            if (row < 0 || row >= a.req_rows) set_error(a.err, PA_DEVERR_ROW);
            if (n < 0 || n > a.max_ctx) set_error(a.err, PA_DEVERR_LEN);
        }
    }
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int units = a.ranges * a.Hkv, W = blk_width(s_pref, a.batch, a.ranges);
    // few units: one per SM; else the heads of a range side by side on an SM
    const int worker = s_pref[a.batch] <= (long long)a.spread * W ? (int)blockIdx.x + wg * (int)gridDim.x
                                                                  : 2 * (int)blockIdx.x + wg;

    if (warp >= 8) {
        const bool isv = warp & 1;
        blk_loader<D, E8, GP>(a, s_pref, s_req, W, worker, isv ? vring : kring, isv ? a.stages_v : a.stages_k,
                              reinterpret_cast<BlkStage *>(base + C::OffStage + (warp - 8) * kBlkStageBytes), isv ? vmeta : kmeta, isv ? vfull : kfull, isv ? vempty : kempty, s_abort, isv, lane);
    } else {
        const int t = tid & 127, bar_id = 1 + wg;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = tmem + wg * 128, o_col = s_col + 64;
        const uint32_t sQ = smem_u32(base + C::OffQ) + wg * C::align_k(C::QB), sP = smem_u32(base + C::OffP) + wg * C::align_k(C::PB);
        float *s_max = reinterpret_cast<float *>(base + C::OffRed) + wg * C::kRed;    // [4][2 GP]
        float *s_sum = s_max + 8 * GP, *s_fq = s_sum + 4 * GP;                         // [4][GP], [GP]
        constexpr uint32_t kFmt = E8 ? 0u : (1u << 7 | 1u << 10);      // e4m3 : bf16
        constexpr uint32_t kIdS = 1u << 4 | kFmt | (uint32_t)(C::NQ >> 3) << 17 | 8u << 24;
        constexpr uint32_t kIdO = 1u << 4 | kFmt | 1u << 15 | (uint32_t)(C::NP >> 3) << 17 | 8u << 24;   // A is MN-major
        constexpr float kShift = E8 ? 8.f : 0.f;    // P' reaches 2^8, within e4m3's 448
        bool bad = false;
        int done = 0;                               // tiles of this worker
        int stk = 0, stv = 0;                       // ring stages
        uint32_t phk = 0, phv = 0;
        // warp-uniform; after a time-out the warps run through the remaining
        // barriers without issuing or waiting, so none of them is left behind
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (!bad) bad = !__all_sync(0xffffffffu, mbar_wait(bar, parity, s_abort, a.err, PA_DEVERR_TIMEOUT, a.wait_ns));
        };
        int shared_b[2], shared = 0;                // requests of whose segment the unit has a part: at most two
        int ticket[2];
        // this thread's chunks of the piece's query rows, requested while the piece before it ends
        constexpr int CH = D / 8;                   // 8-element chunks of a head row
        constexpr int QR = (GP * CH + 127) / 128;   // chunks per thread
        uint4 qn[QR];
        auto load_q = [&](const BlkWalk &k) {
#pragma unroll
            for (int r = 0; r < QR; ++r) {
                const int g = (t + r * 128) / CH, c = (t + r * 128) % CH;
                qn[r] = make_uint4(0u, 0u, 0u, 0u);
                if (g < a.G) qn[r] = __ldg(reinterpret_cast<const uint4 *>(a.q + ((int64_t)k.b * a.Hq + k.h * a.G + g) * D) + c);
            }
        };
#pragma unroll 1
        for (int unit = worker; unit < units; unit += a.workers) {
        BlkWalk kn = blk_begin(s_pref, a.batch, a.Hkv, W, unit);
        bool more = blk_piece(s_pref, s_req, kn);
        if (more) load_q(kn);
        shared = 0;
        while (more) {
            const BlkWalk k = kn;
            if (a.wait_ns == 0 && !bad) {
                // a wait limit of 0: give up at the first item, as a timed-out wait would
                *s_abort = 1;
                set_error(a.err, PA_DEVERR_TIMEOUT);
                bad = true;
            }
            // ---- q as the B operand, rows (term, head)
#pragma unroll
            for (int r0 = 0; r0 < QR; ++r0) {
                const int g = (t + r0 * 128) / CH, c = (t + r0 * 128) % CH;
                const uint4 w = qn[r0];
                if constexpr (E8) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t u = e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w;
                        x[2 * e] = __uint_as_float(u << 16);
                        x[2 * e + 1] = __uint_as_float(u & 0xFFFF0000u);
                    }
                    float mx = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, isfinite(x[e]) ? fabsf(x[e]) : 0.f);
#pragma unroll
                    for (int o = CH / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const int eq = max(block_exponent(mx), 1);
                    const float inv = __uint_as_float((uint32_t)(254 - eq) << 23);
                    uint32_t b1[2] = {0, 0}, b2[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float y0 = isfinite(x[e]) ? x[e] * inv : NAN, y1 = isfinite(x[e + 1]) ? x[e + 1] * inv : NAN;
                        const uint32_t p = e4m3x2_of(y0, y1);
                        float f0, f1;
                        e4m3x2_floats(p, f0, f1);
                        b1[e >> 2] |= p << (8 * (e & 3));
                        b2[e >> 2] |= e4m3x2_of((y0 - f0) * 16.f, (y1 - f1) * 16.f) << (8 * (e & 3));
                    }
                    if (g < GP) {
                        const uint32_t o1 = blk_off<AW>(g, c >> 1) + (c & 1) * 8, o2 = blk_off<AW>(GP + g, c >> 1) + (c & 1) * 8;
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(sQ + o1), "r"(b1[0]), "r"(b1[1]) : "memory");
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(sQ + o2), "r"(b2[0]), "r"(b2[1]) : "memory");
                        if (c == 0) s_fq[g] = a.scale_log2 * __uint_as_float((uint32_t)eq << 23);
                    }
                } else if (g < GP) {
                    st_shared_v4(sQ + (c >> 3) * (C::NQ * 128) + blk_off<AW>(g, c & 7), w.x, w.y, w.z, w.w);
                    if (c == 0) s_fq[g] = a.scale_log2;
                }
            }
            fence_proxy_async_smem();
            named_bar_sync(bar_id, 128);
            float m[GP], r[GP], l[GP], o[GP];
#pragma unroll
            for (int g = 0; g < GP; ++g) m[g] = r[g] = -INFINITY, l[g] = o[g] = 0.f;

#pragma unroll 1
            for (int i = 0; i < k.live; ++i, ++done) {
                const uint32_t kt = kring + stk * C::TILE, vt = vring + stv * C::TILE;
                // S = K Q^T
                wait(kfull + stk * 8, phk);
                if ((warp & 3) == 0) {
                    tc_fence_after();
                    if (!bad) if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < C::QSteps; ++s) {
                            constexpr int SPH = AW / 32;    // steps per half
                            const uint64_t da = blk_desc<AW>(kt + (s / SPH) * C::HALF + (s % SPH) * 32, 16, 8 * AW);
                            const uint64_t db = blk_desc<AW>(sQ + (s / SPH) * (C::NQ * AW) + (s % SPH) * 32, 16, 8 * AW);
                            blk_umma<E8>(s_col, da, db, kIdS, s > 0);
                        }
                        umma_commit(sfull);
                    }
                    __syncwarp();
                }
                const int ek = kmeta[stk * kBlkTile + t];
                // the V tile has long landed when the weights are there; its exponents are read now
                wait(vfull + stv * 8, phv);
                const int ev = E8 ? vmeta[stv * kBlkTile + t] : 0;
                wait(sfull, done & 1);
                tc_fence_after();
                uint32_t sr[C::NQ];
#pragma unroll
                for (int c = 0; c < C::NQ; c += 16) tmem_ld16(s_col + lane_base + c, *reinterpret_cast<uint32_t(*)[16]>(&sr[c]));
                tmem_wait_ld();
                float x[GP];
                const float fk = E8 ? __uint_as_float((uint32_t)ek << 23) : 1.f;
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    float s = __uint_as_float(sr[g]);
                    if constexpr (E8) s = fmaf(__uint_as_float(sr[GP + g]), 0.0625f, s) * fk;
                    x[g] = ek == kMasked ? -INFINITY : s * s_fq[g];
                }
                if constexpr (WT) {
                    const int tile = s_pref[k.b] + k.t0 + i;
                    if (tile < a.cap_tiles) {
                        float *dst = a.scores + (((int64_t)k.h * a.cap_tiles + tile) * kBlkTile + t) * a.G;
#pragma unroll
                        for (int g = 0; g < GP; ++g)
                            if (g < a.G) dst[g] = x[g];
                    }
                }
                // the tile's maxima of s (for l) and of s + ev (for P')
                float *red = s_max + (warp & 3) * 2 * GP;
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float mx = warp_max(x[g]), rx = E8 ? warp_max(x[g] + (float)ev) : mx;
                    if (lane == 0) {
                        red[g] = mx;
                        red[GP + g] = rx;
                    }
                }
                named_bar_sync(bar_id, 128);
                float bt[GP], at[GP];
                float pp[GP];
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float *w = s_max + g;
                    const float mt = fmaxf(fmaxf(w[0], w[2 * GP]), fmaxf(w[4 * GP], w[6 * GP]));
                    const float rt = E8 ? fmaxf(fmaxf(w[GP], w[3 * GP]), fmaxf(w[5 * GP], w[7 * GP])) : mt;
                    const float mn = fmaxf(m[g], mt), rn = fmaxf(r[g], rt);
                    const float mz = mn == -INFINITY ? 0.f : mn, rz = rn == -INFINITY ? 0.f : rn;
                    const float rtz = rt == -INFINITY ? 0.f : rt;
                    l[g] = l[g] * blk_ex2(m[g] - mz) + blk_ex2(x[g] - mz);
                    // (an empty block's values, ev = 0, are 0, not 2^-127: its tokens weigh in l alone)
                    pp[g] = E8 && ev == 0 ? 0.f : blk_ex2(x[g] + (float)ev - rtz + kShift);
                    at[g] = blk_ex2(r[g] - rz);
                    bt[g] = rt == -INFINITY ? 0.f : blk_ex2(rt - rz);
                    m[g] = mn;
                    r[g] = rn;
                }
                // P' in terms, rows (term, head), this thread's token a column
#pragma unroll
                for (int g = 0; g < GP; g += 2) {
                    float y0 = pp[g], y1 = pp[g + 1];
#pragma unroll
                    for (int j = 0; j < C::PT; ++j) {
                        const int n0 = j * GP + g, n1 = n0 + 1;
                        if constexpr (E8) {
                            const uint32_t p = e4m3x2_of(y0, y1);
                            float f0, f1;
                            e4m3x2_floats(p, f0, f1);
                            y0 = (y0 - f0) * 16.f;
                            y1 = (y1 - f1) * 16.f;
                            st_shared_u8(sP + blk_off<128>(n0, t >> 4) + (t & 15), p);
                            st_shared_u8(sP + blk_off<128>(n1, t >> 4) + (t & 15), p >> 8);
                        } else {
                            const uint32_t p = pack_bf16x2(y0, y1);
                            y0 -= __uint_as_float(p << 16);
                            y1 -= __uint_as_float(p & 0xFFFF0000u);
                            const uint32_t half = sP + (t >> 6) * (C::NP * 128);
                            st_shared_u16(half + blk_off<128>(n0, (t & 63) >> 3) + (t & 7) * 2, p);
                            st_shared_u16(half + blk_off<128>(n1, (t & 63) >> 3) + (t & 7) * 2, p >> 16);
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                named_bar_sync(bar_id, 128);
                // O^T = V^T P^T; K's stage is free: its products are done and every thread has read its exponents
                if ((warp & 3) == 0) {
                    tc_fence_after();
                    if (!bad) if (elect_one()) {
                        mbar_arrive(kempty + stk * 8);
#pragma unroll
                        for (int s = 0; s < C::PSteps; ++s) {
                            // V is [token][d]: 32 / ES tokens per step; the second 128-byte half of a bf16 row is the
                            // upper 64 of M; a row of 64 elements serves both halves of M (leading offset 0)
                            const uint64_t da = blk_desc<AW>(vt + s * (32 / ES) * AW, C::HALVES > 1 ? C::HALF : 0, 8 * AW);
                            const uint64_t db = blk_desc<128>(sP + (s >> 2) * (C::NP * 128) + (s & 3) * 32, 16, 1024);
                            blk_umma<E8>(o_col, da, db, kIdO, s > 0);
                        }
                        umma_commit(ofull);
                        umma_commit(vempty + stv * 8);
                    }
                    __syncwarp();
                }
                if (++stk == a.stages_k) {
                    stk = 0;
                    phk ^= 1;
                }
                if (++stv == a.stages_v) {
                    stv = 0;
                    phv ^= 1;
                }
                wait(ofull, done & 1);
                tc_fence_after();
                uint32_t orr[C::NP];
#pragma unroll
                for (int c = 0; c < C::NP; c += 16) tmem_ld16(o_col + lane_base + c, *reinterpret_cast<uint32_t(*)[16]>(&orr[c]));
                tmem_wait_ld();
                tc_fence_before();
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    float v;
                    if constexpr (E8)
                        v = fmaf(fmaf(__uint_as_float(orr[2 * GP + g]), 0.0625f, __uint_as_float(orr[GP + g])), 0.0625f,
                                 __uint_as_float(orr[g]));
                    else
                        v = __uint_as_float(orr[g]) + __uint_as_float(orr[GP + g]);
                    o[g] = fmaf(o[g], at[g], v * bt[g]);
                }
            }

            // ---- the piece ends
            blk_next(kn);
            more = blk_piece(s_pref, s_req, kn);
            if (more) load_q(kn);
            // O, m and r through the P tile (its products are done), so that the stores below are one rolled loop
            float *so = reinterpret_cast<float *>(base + C::OffP + wg * C::align_k(C::PB)), *smr = s_max;   // [GP][128]; [GP] m, [GP] r
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                float s = l[g];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                if (lane == 0) s_sum[(warp & 3) * GP + g] = s;
                so[g * 128 + t] = o[g];
                if (t == 0) {
                    smr[g] = m[g];
                    smr[GP + g] = r[g];
                }
            }
            named_bar_sync(bar_id, 128);
            const bool whole = k.t0 == 0 && k.t1 == k.tb;
            const int part = unit * 2 + (k.t0 == 0 && k.S0 % W != 0 ? 1 : 0);
#pragma unroll 1
            for (int g = 0; g < a.G && !bad; ++g) {
                const float L = s_sum[g] + s_sum[GP + g] + s_sum[2 * GP + g] + s_sum[3 * GP + g];
                const float mg = smr[g], rg = smr[GP + g];
                // O relative to m: 2^(r - 127 - 8 - m), in two factors where one would be flushed to 0 (r - m is the
                // exponent byte of the largest weight's value or more: down to 2^-134)
                const float mz = mg == -INFINITY ? 0.f : mg, rz = rg == -INFINITY ? 0.f : rg;
                const float d = rz - mz - 135.f;
                const float O = E8 ? so[g * 128 + t] * (d < -64.f ? 0x1p-64f : 1.f) * blk_ex2(d < -64.f ? d + 64.f : d)
                                   : so[g * 128 + t];
                if (whole) {
                    const int64_t hq = (int64_t)k.b * a.Hq + k.h * a.G + g;
                    if (t < D) a.out[hq * D + t] = __float2bfloat16_rn(L != 0.f ? O / L : 0.f);
                    if (WT && t == 0) a.lse[hq] = L != 0.f ? mg + log2f(L) : INFINITY;
                } else {
                    const int at = part * a.G + g;
                    if (t < D) a.o_part[at * D + t] = O;
                    if (t == 0) *reinterpret_cast<float2 *>(a.ml_part + at * 2) = make_float2(mg, L);
                }
            }
            if (!whole) {
                // a ticket for the piece: the barrier orders the partials' stores before thread 0's releasing addition;
                // the answer is looked at (and acquired from) after the unit's last piece
                named_bar_sync(bar_id, 128);
                if (t == 0 && !bad) {
                    const int old = atom_add_release_gpu(a.tickets + k.S0 / W * a.Hkv + k.h, 1);
                    if (shared == 0) ticket[0] = old;
                    else ticket[1] = old;
                }
                if (shared == 0) shared_b[0] = k.b;
                else shared_b[1] = k.b;
                ++shared;
            }
        }
        // shared segments whose last piece was this unit's
#pragma unroll 1
        for (int i = 0; i < shared; ++i) {
            const int sb = i == 0 ? shared_b[0] : shared_b[1];
            const BlkSpan s = blk_span(s_pref, W, sb);
            const int h = unit % a.Hkv;
            if (t == 0) {
                const bool last = !bad && (i == 0 ? ticket[0] : ticket[1]) == s.i1 - s.i0;
                if (last) fence_acq_rel_gpu();      // the other workers' partials are visible to what follows
                s_last[wg][i] = last;
            }
            named_bar_sync(bar_id, 128);
            if (s_last[wg][i]) {
                blk_merge<D, GP, WT>(a, s, sb, h, t, bar_id, reinterpret_cast<float *>(smem_raw + (kring - raw)), ring_bytes);
                if (t == 0) a.tickets[s.i0 * a.Hkv + h] = 0;
            }
        }
        }
        if (__any_sync(0xffffffffu, *s_abort) && (warp & 3) == 0) {
            // aborted: every MMA this lane issued completes before tensor memory is freed
            if (elect_one()) umma_commit(drain);
            __syncwarp();
            mbar_drain(drain, 0);
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, kBlkTmemCols);
    }
}

// ---------------------------------------------------------------- weights
constexpr int kBlkWeightThreads = 128;

// weights[row, j] += sum over the heads of 2^(score - lse), one 128-token tile
// of a request at a time, heads in order.  A kernel of its own, because a score's
// sum is known only when its last piece is; scores pass through L2 (4 Hq bytes per
// token each way).  32 requests of 700 to 8192 tokens take 57.2 us with it, this
// kernel about 7 of them; at 64 registers eight blocks fit an SM.  (In one session at
// 55.7 us: 4 blocks per SM 57.0, the scores loaded behind the sums 61.3.  The look at
// the error word costs 0.5 us.)
static __global__ void __launch_bounds__(kBlkWeightThreads) decode_block_weights_kernel(const __grid_constant__ BlkArgs a)
{
    extern __shared__ int s_pref[];                 // [batch + 1], then float [Hq]
    __shared__ int s_w[kBlkWeightThreads / 32];
    const int tid = threadIdx.x, B = a.batch, G = a.G;
    float *s_lse = reinterpret_cast<float *>(s_pref + B + 1);
    if (!a.early_meta) pdl_wait();
    blk_plan<kBlkWeightThreads>(a, s_pref, nullptr, s_w);
    if (a.early_meta) pdl_wait();
    pdl_launch_dependents();
    // a decode kernel that gave up left scores and sums that belong to nothing: the table outlives the call and
    // the workspace, so nothing is added (the word is on its way while the scores are read)
    const int state = __float_as_int(ld_cg_ordered_if(true, reinterpret_cast<const float *>(a.err)));
    const int tiles = s_pref[B];
#pragma unroll 1
    for (int x = blockIdx.x; x < tiles; x += gridDim.x) {
        int lo = 0, hi = B;
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pref[mid] <= x) lo = mid; else hi = mid;
        }
        const int b = lo, n = blk_len(a, b), row = __ldg(a.req_pool_indices + b);
        if (n <= 0) continue;
        const int j = (x - s_pref[b]) * kBlkTile + tid;
        const bool in = j < n && x < a.cap_tiles;
        const float *sc = a.scores + ((int64_t)x * kBlkTile + tid) * G;
        const int64_t head = (int64_t)a.cap_tiles * kBlkTile * G;
        float *dst = a.weights + (int64_t)row * a.max_ctx + j;
        // four scores a load where G allows it, the first eight loads and the
        // old weight on their way while the sums arrive
        const int quads = G % 4 == 0 ? a.Hq / 4 : 0;
        auto load = [&](int q) {
            const int h = q / (G / 4), g = (q - h * (G / 4)) * 4;
            return __ldcg(reinterpret_cast<const float4 *>(sc + h * head + g));
        };
        float4 v[8];
        float w = 0.f, old = 0.f;
        if (in) {
            old = __ldcg(dst);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < quads) v[q] = load(q);
        }
        // two requests of a row would both add to it: the later one is refused
        // (after one without tokens, a batch's padding, it is not)
        int again = 0;
#pragma unroll 1
        for (int c = tid; c < b; c += kBlkWeightThreads)
            if (__ldg(a.req_pool_indices + c) == row) again |= blk_len(a, c) > 0;
        __syncthreads();   // s_lse is free
#pragma unroll 1
        for (int hq = tid; hq < a.Hq; hq += kBlkWeightThreads) s_lse[hq] = __ldcg(a.lse + (int64_t)b * a.Hq + hq);
        again = __syncthreads_or(again);
        if (again || x >= a.cap_tiles) {
            if (tid == 0) set_error(a.err, again ? PA_DEVERR_ROW : PA_DEVERR_LEN);
            continue;
        }
        if (!in) continue;
        auto add = [&](int q, float4 u) {
            const float *l = s_lse + q * 4;
            w += blk_ex2(u.x - l[0]) + blk_ex2(u.y - l[1]) + (blk_ex2(u.z - l[2]) + blk_ex2(u.w - l[3]));
        };
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < quads) add(q, v[q]);
#pragma unroll 4
        for (int q = 8; q < quads; ++q) add(q, load(q));
        if (quads == 0) {
#pragma unroll 4
            for (int hq = 0; hq < a.Hq; ++hq) {
                const int h = hq / G;
                w += blk_ex2(__ldcg(sc + h * head + hq - h * G) - s_lse[hq]);
            }
        }
        if (!(state & PA_DEVERR_TIMEOUT)) *dst = old + w;
    }
}

template <int D, bool E8, int GP, bool WT>
static pa_status launch_block(BlkArgs a, cudaStream_t st)
{
    using C = BlkCfg<D, E8, GP>;
    // ring stages per worker and operand: as many as fit, K one more than V where half a stage is left
    const int tiles = (int)((kBlkSmemLimit - C::fixed(a.batch)) / C::TILE) / 2;
    a.stages_v = tiles / 2 < kBlkMaxStages ? tiles / 2 : kBlkMaxStages;
    a.stages_k = tiles - a.stages_v < kBlkMaxStages ? tiles - a.stages_v : kBlkMaxStages;
    static_assert((kBlkSmemLimit - C::fixed(kBlkMaxBatch)) / C::TILE >= 4, "a stage per worker and operand fits at the largest batch");
    constexpr int kLeast = (int)((kBlkSmemLimit - C::fixed(kBlkMaxBatch)) / C::TILE) / 2;
    static_assert((kLeast < 2 * kBlkMaxStages ? kLeast : 2 * kBlkMaxStages) * C::TILE >=
                      (36 + 2 * kBlkMaxWorkers * GP + GP * D) * 4, "the merge's scratch holds a piece");
    auto kern = decode_block_kernel<D, E8, GP, WT>;
    const size_t smem = C::fixed(a.batch) + (size_t)2 * (a.stages_k + a.stages_v) * C::TILE;
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem)) return PA_ERR_CUDA;
    const int grid = num_sms() < kBlkMaxWorkers / 2 ? num_sms() : kBlkMaxWorkers / 2;
    a.workers = 2 * grid;
    a.ranges = a.workers / a.Hkv > 1 ? a.workers / a.Hkv : 1;
    a.spread = grid / a.Hkv;
    const size_t wsmem = ((size_t)a.batch + 1) * 4 + (size_t)a.Hq * 4;
    if (WT && !ensure_dynamic_smem(reinterpret_cast<const void *>(decode_block_weights_kernel), wsmem)) return PA_ERR_CUDA;
    if (launch_kernel(kern, dim3(grid), dim3(kBlkThreads), smem, st, a) != cudaSuccess) return PA_ERR_CUDA;
    if constexpr (WT) {
        if (launch_kernel(decode_block_weights_kernel, dim3(8 * grid), dim3(kBlkWeightThreads), wsmem, st, a) != cudaSuccess)
            return PA_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <bool E8, bool WT>
static pa_status dispatch_block(const BlkArgs &a, int D, cudaStream_t st)
{
    if (D == 128) {
        if (a.G <= 4) return launch_block<128, E8, 4, WT>(a, st);
        if (a.G <= 8) return launch_block<128, E8, 8, WT>(a, st);
        return launch_block<128, E8, 16, WT>(a, st);
    }
    if (a.G <= 4) return launch_block<64, E8, 4, WT>(a, st);
    if (a.G <= 8) return launch_block<64, E8, 8, WT>(a, st);
    return launch_block<64, E8, 16, WT>(a, st);
}

}  // namespace pa
