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
// Work: every (kv head, request) is a segment of 128-token tiles (at least
// one), laid end to end head-major; CTA c takes tiles [c W, (c + 1) W).  A CTA
// has at most two segments it shares with others, its first and its last, so
// the fp32 partials are two slots per CTA whatever the batch is.  The CTA that
// finishes a shared segment's last piece (a ticket per segment) merges its
// pieces in CTA order (deterministic); a second kernel adds the weights (WT).
//
// Roles: two warpgroups take the tiles in turn (softmax of one beside the
// products of the other), each issuing its own MMAs; warp 8 loads K tiles and
// K exponents, warp 9 the V's.  16 consecutive slots move as one TMA box, any
// other four rows as one gather4 copy.  Positions past the end repeat a valid
// row (weight zero), so nothing behind the last token is read.
#include <math.h>
#include <string.h>

#include "pa_internal.h"
#include "pa_sm100.cuh"

namespace pa {
using namespace sm100;

constexpr int kBlkTile = 128;          // tokens per tile: the MMA's M
constexpr int kBlkConsumers = 256;     // two warpgroups
constexpr int kBlkLoaders = 2;         // loader warps per operand, taking its tiles in turn
constexpr int kBlkThreads = kBlkConsumers + 64 * kBlkLoaders;
constexpr int kBlkMaxCtas = 160;       // partial slots in the workspace (152 SMs)
constexpr int kBlkMaxStages = 8;
constexpr int kBlkMaxBatch = 4096;
constexpr uint32_t kBlkTmemCols = 256; // per warpgroup 128: S at 0, O at 64
constexpr int kMasked = 255;           // exponent byte of a position without a token

struct BlkArgs {
    CUtensorMap tm_k16, tm_k1, tm_v16, tm_v1;   // 2-D (element, row): boxes of 16 rows, and one row (gather4)
    const __nv_bfloat16 *q;
    const int32_t *req_to_token, *req_pool_indices, *seq_lens;
    const uint8_t *k_exp, *v_exp;               // the layer's [n_blocks, Hkv] (e4m3 cache)
    __nv_bfloat16 *out;
    int32_t *err;
    int32_t *tickets;                           // [CTAs]: finished pieces of the shared segment that starts in that CTA
    float *ml_part;                             // [2 CTAs][G][2]: maximum (log2 units), sum
    float *o_part;                              // [2 CTAs][G][D]: relative to that maximum
    float *lse;                                 // [batch, Hq]: log2-sum-exp (WT)
    float *scores;                              // [Hkv][cap_tiles][128][G], log2 units (WT)
    float *weights;                             // [req_rows, max_ctx] (WT)
    int batch, Hq, Hkv, G, size, req_rows, max_ctx, layer_row0, block_shift, stages, cap_tiles, early_meta, grid;
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
    static constexpr int STAGE = 2 * TILE;
    static constexpr int QB = NQ * RB;
    static constexpr int PB = NP * kBlkTile * ES;         // one warpgroup's P
    static constexpr int QSteps = RB / 32, PSteps = kBlkTile * ES / 32;   // a K step is 32 bytes of either type
    // offsets behind the ring of `stages` tiles
    __host__ __device__ static constexpr int align_k(int x) { return (x + 1023) & ~1023; }
    static constexpr int OffQ = 0;
    static constexpr int OffP = align_k(QB);
    static constexpr int OffMeta = OffP + 2 * align_k(PB);
    static constexpr int OffBar = OffMeta + 2 * kBlkMaxStages * kBlkTile;
    static constexpr int OffRed = OffBar + 256;            // fp32: [2][4][2 GP] maxima, [2][4][GP] sums, [GP] q factors, m, l
    static constexpr int OffPref = (OffRed + (16 * GP + 8 * GP + GP + 4 * GP) * 4 + 7) & ~7;
    // after the prefix array [batch + 1]: each request's (length, table row), int2 [batch]
    __host__ __device__ static constexpr int off_req(int batch) { return OffPref + (batch + 2) / 2 * 8; }
    static constexpr size_t fixed(int batch) { return 1024 + (size_t)off_req(batch) + (size_t)batch * 8; }
    static constexpr size_t bytes(int batch, int stages) { return fixed(batch) + (size_t)stages * STAGE; }
    static_assert(2 * align_k(PB) >= GP * D * 4, "the item-end scratch reuses the P tiles");
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
    for (int w = 0; w < warp; ++w) base += s_w[w];
    int excl = base + incl - run;
    for (int b = lo; b < hi; ++b) {
        s_pref[b] = excl;
        const int n = blk_len(a, b);
        if (s_req) s_req[b] = make_int2(n, __ldg(a.req_pool_indices + b));
        excl += blk_tiles(n);
    }
    if (tid == NT - 1) s_pref[B] = base + incl;
    __syncthreads();
}

// One CTA's walk over its pieces of segments.
struct BlkWalk {
    int x, xe, h, b;       // next tile, end of the CTA's range, segment
    int S0, tb;            // the segment's first tile and its tiles
    int t0, t1, n, row;    // the piece: tiles [t0, t1) of the segment, tokens and table row of the request
    int live;              // tiles of the piece with tokens: t1 - t0, or 0
};
__device__ __forceinline__ BlkWalk blk_begin(const int *s_pref, int B, int Hkv, int W, int cta)
{
    BlkWalk k;
    const int tph = s_pref[B];
    k.x = min((long long)cta * W, (long long)Hkv * tph);
    k.xe = min((long long)k.x + W, (long long)Hkv * tph);
    k.h = k.x / tph;
    const int local = k.x - k.h * tph;
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pref[mid] <= local) lo = mid; else hi = mid;
    }
    k.b = lo;
    return k;
}
// the piece at k.x; false past the end
__device__ __forceinline__ bool blk_piece(const BlkArgs &a, const int *s_pref, const int2 *s_req, BlkWalk &k)
{
    if (k.x >= k.xe) return false;
    k.S0 = k.h * s_pref[a.batch] + s_pref[k.b];
    k.tb = s_pref[k.b + 1] - s_pref[k.b];
    k.t0 = k.x - k.S0;
    k.t1 = min(k.xe - k.S0, k.tb);
    k.n = s_req[k.b].x;
    k.row = s_req[k.b].y;
    k.live = k.n > 0 ? k.t1 - k.t0 : 0;
    return true;
}
__device__ __forceinline__ void blk_next(const BlkArgs &a, BlkWalk &k)
{
    k.x = k.S0 + k.t1;
    if (k.t1 == k.tb && ++k.b == a.batch) {
        k.b = 0;
        ++k.h;
    }
}
__device__ __forceinline__ int blk_width(const int *s_pref, int B, int Hkv, int grid)
{
    const long long T = (long long)Hkv * s_pref[B];
    return (int)((T + grid - 1) / grid);
}

// ------------------------------------------------------------------ loader
// K (isv false) or V rows and exponents of tiles first, first + kBlkLoaders, ...
// of the CTA, in order.  (A TMA instruction costs its warp about 100 cycles of
// issue, a tile of 16-slot pages eight of them: one warp per operand fell
// behind HBM, 1830 cycles a tile against 1460.)
// Table entries and exponents come through registers in batches of kBlkAhead
// tiles: a batch's table entries are requested while the batch before it is
// copied, its exponents (which hang on them) half a batch later, so a tile's
// copies wait for neither round trip.
constexpr int kBlkAhead = 4;

template <int D, bool E8, int GP>
__device__ __forceinline__ void blk_loader(const BlkArgs &a, const int *s_pref, const int2 *s_req, int W, uint32_t ring,
                                           unsigned char *meta, uint32_t full, uint32_t empty, volatile int *s_abort,
                                           bool isv, int first, int lane)
{
    using C = BlkCfg<D, E8, GP>;
    struct Tile {
        int h, n, p0;           // kv head, tokens of the request (0: no more tiles), first position
        int slot[4];            // table entries of positions p0 + 4 lane + e
        int ex[4];              // exponent bytes
    };
    const CUtensorMap *m16 = isv ? &a.tm_v16 : &a.tm_k16, *m1 = isv ? &a.tm_v1 : &a.tm_k1;
    const uint8_t *exps = isv ? a.v_exp : a.k_exp;
    BlkWalk k = blk_begin(s_pref, a.batch, a.Hkv, W, blockIdx.x);
    bool more = blk_piece(a, s_pref, s_req, k);
    int i = first;              // next tile of the piece
    int errs = 0;
    auto fetch = [&](Tile &t) {
        while (more && i >= k.live) {
            i -= k.live;
            blk_next(a, k);
            more = blk_piece(a, s_pref, s_req, k);
        }
        t.n = t.p0 = t.h = 0;
        int64_t row = 0;
        if (more) {
            row = k.row;
            t.h = k.h;
            t.n = k.n;
            t.p0 = (k.t0 + i) * kBlkTile;
            i += kBlkLoaders;
        }
        const int32_t *src = a.req_to_token + row * a.max_ctx;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = t.p0 + 4 * lane + e;
            t.slot[e] = ld_nc_ordered_s32_if(p < t.n, src + (p < t.n ? p : 0));
        }
    };
    auto load_exps = [&](Tile &t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool ok = t.slot[e] >= 0 && t.slot[e] < a.size;
            t.ex[e] = !ok ? kMasked : !E8 ? 0 : __ldcg(exps + (int64_t)(t.slot[e] >> a.block_shift) * a.Hkv + t.h);
        }
    };
    int st = first, seq = first;    // ring stage and number of the next tile (stages >= kBlkLoaders)
    uint32_t ph = 0;
    // copies of one tile; false if the wait for its stage timed out
    auto put = [&](const Tile &c) -> bool {
        // the stage's previous tile has been multiplied
        if (seq >= a.stages &&
            !__all_sync(0xffffffffu, mbar_wait(empty + st * 8, ph ^ 1, s_abort, a.err, PA_DEVERR_TIMEOUT, a.wait_ns)))
            return false;
        const uint32_t dst = ring + st * C::STAGE + (isv ? C::TILE : 0), fb = full + st * 8;
        bool ok[4];
        int sl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sl[e] = c.slot[e];
            ok[e] = sl[e] >= 0 && sl[e] < a.size;
            if (!ok[e] && c.p0 + 4 * lane + e < c.n) errs |= PA_DEVERR_SLOT;
        }
        const int mine = ok[0] ? sl[0] : ok[1] ? sl[1] : ok[2] ? sl[2] : ok[3] ? sl[3] : -1;
        const unsigned has = __ballot_sync(0xffffffffu, mine >= 0);
        const int some = __shfl_sync(0xffffffffu, mine, has ? __ffs(has) - 1 : 0);   // a valid row of the tile
        const int s0 = __shfl_sync(0xffffffffu, sl[0], lane & ~3);
        const bool run = ok[0] && ok[1] && ok[2] && ok[3] && sl[0] == s0 + 4 * (lane & 3) && sl[1] == sl[0] + 1 &&
                         sl[2] == sl[0] + 2 && sl[3] == sl[0] + 3;
        const bool page = ((__ballot_sync(0xffffffffu, run) >> (lane & ~3)) & 0xFu) == 0xFu;
        if (has) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sl[e] = a.layer_row0 + (ok[e] ? sl[e] : some);
            const int col = c.h * D;
            if (page) {
                if ((lane & 3) == 0) {
#pragma unroll
                    for (int hh = 0; hh < C::HALVES; ++hh)
                        tma_load_2d(dst + hh * C::HALF + (lane >> 2) * 16 * C::AW, m16, col + hh * (C::AW / C::ES), sl[0], fb);
                }
            } else {
#pragma unroll
                for (int hh = 0; hh < C::HALVES; ++hh)
                    tma_gather4(dst + hh * C::HALF + lane * 4 * C::AW, m1, col + hh * (C::AW / C::ES), sl[0], sl[1], sl[2],
                                sl[3], fb);
            }
        } else {
            // no valid row at all: zeros (weight zero times whatever bits lie there could be NaN)
            for (int o = lane * 16; o < C::TILE; o += 512) st_shared_v4(dst + o, 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
        }
        reinterpret_cast<uint32_t *>(meta + ((isv ? kBlkMaxStages : 0) + st) * kBlkTile)[lane] =
            (uint32_t)(c.ex[0] | c.ex[1] << 8 | c.ex[2] << 16 | c.ex[3] << 24);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(fb, has ? C::TILE : 0u);
        seq += kBlkLoaders;
        st += kBlkLoaders;
        if (st >= a.stages) {
            st -= a.stages;
            ph ^= 1;
        }
        return true;
    };
    Tile cur[kBlkAhead], nxt[kBlkAhead];
#pragma unroll
    for (int u = 0; u < kBlkAhead; ++u) fetch(cur[u]);
#pragma unroll
    for (int u = 0; u < kBlkAhead; ++u) load_exps(cur[u]);
    bool go = true;
    while (go) {
#pragma unroll
        for (int u = 0; u < kBlkAhead; ++u) fetch(nxt[u]);
#pragma unroll
        for (int u = 0; u < kBlkAhead; ++u) {
            if (u == kBlkAhead / 2) {
#pragma unroll
                for (int w = 0; w < kBlkAhead; ++w) load_exps(nxt[w]);
            }
            if (go) go = cur[u].n > 0 && put(cur[u]);
        }
#pragma unroll
        for (int u = 0; u < kBlkAhead; ++u) cur[u] = nxt[u];
    }
    if (*s_abort) {
        // aborted: the copies already issued land before the shared memory goes away
        for (int j = seq - kBlkLoaders; j >= 0 && j >= seq - kBlkLoaders - a.stages; j -= kBlkLoaders)
            mbar_drain(full + (j % a.stages) * 8, (j / a.stages) & 1);
    }
    if (errs) set_error(a.err, errs);
    __syncwarp();
}

// Pieces of segment (b, h): CTAs c0 .. c1; a piece that does not start its
// CTA's range is that CTA's last (slot 1).
struct BlkSpan {
    int c0, c1, S0;
};
__device__ __forceinline__ BlkSpan blk_span(const int *s_pref, int B, int W, int b, int h)
{
    BlkSpan s;
    s.S0 = h * s_pref[B] + s_pref[b];
    s.c0 = s.S0 / W;
    s.c1 = (s.S0 + s_pref[b + 1] - s_pref[b] - 1) / W;
    return s;
}
__device__ __forceinline__ int blk_slot(const BlkSpan &s, int c, int W) { return 2 * c + (s.S0 > c * W ? 1 : 0); }

// Merge of a shared segment by the CTA that finished its last piece: every
// element summed in CTA order.  All consumer threads; a warp's elements belong
// to one head.  The first pieces' partials and the (m, l) pairs of the first 32
// are all requested before any is used: one round trip, for the 20 pieces that
// a single long request has as for two.
template <int D, int GP, bool WT>
__device__ __forceinline__ void blk_merge(const BlkArgs &a, const BlkSpan &s, int W, int b, int h)
{
    constexpr int EPT = GP * D / kBlkConsumers;      // elements per thread
    constexpr int SB = EPT <= 2 ? 20 : 8;            // pieces requested at once (registers)
    const int tid = threadIdx.x, lane = tid & 31, G = a.G, np = s.c1 - s.c0 + 1;
    auto slot = [&](int p) { return blk_slot(s, s.c0 + p, W); };   // piece p's partials
    float v[EPT][SB], mv[EPT], lv[EPT];
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
        const int e = tid + k * kBlkConsumers, g = e / D;
        const bool in = g < G;
#pragma unroll
        for (int p = 0; p < SB; ++p)
            v[k][p] = ld_cg_ordered_if(in && p < np, a.o_part + ((int64_t)slot(p) * G * D + e));
        mv[k] = ld_cg_ordered_if(in && lane < np, a.ml_part + (slot(lane) * G + g) * 2);
        lv[k] = ld_cg_ordered_if(in && lane < np, a.ml_part + (slot(lane) * G + g) * 2 + 1);
    }
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
        const int e = tid + k * kBlkConsumers, g = e / D;
        if (g >= G) break;
        float M = lane < np ? mv[k] : -INFINITY;
        for (int p = 32 + lane; p < np; p += 32) M = fmaxf(M, __ldcg(a.ml_part + (slot(p) * G + g) * 2));
        M = warp_max(M);
        const float Mz = M == -INFINITY ? 0.f : M;
        float L = 0.f, O = 0.f;
        for (int p0 = 0; p0 < np; p0 += 32) {
            const int p = p0 + lane;
            float w = 0.f, l = 0.f;
            if (p < np) {
                w = blk_ex2((p0 == 0 ? mv[k] : __ldcg(a.ml_part + (slot(p) * G + g) * 2)) - Mz);
                l = w * (p0 == 0 ? lv[k] : __ldcg(a.ml_part + (slot(p) * G + g) * 2 + 1));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            L += l;
            if (p0 == 0) {
#pragma unroll
                for (int q = 0; q < SB; ++q) O += __shfl_sync(0xffffffffu, w, q) * v[k][q];
            }
            for (int q = p0 == 0 ? SB : 0; q < 32 && p0 + q < np; ++q)
                O += __shfl_sync(0xffffffffu, w, q) * __ldcg(a.o_part + ((int64_t)slot(p0 + q) * G * D + e));
        }
        const int64_t hq = (int64_t)b * a.Hq + h * G + g;
        a.out[hq * D + (e - g * D)] = __float2bfloat16_rn(L != 0.f ? O / L : 0.f);
        if (WT && e == g * D) a.lse[hq] = L != 0.f ? M + log2f(L) : INFINITY;
    }
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
    __shared__ int s_last[2];
    const uint32_t raw = smem_u32(smem_raw), ring = (raw + 1023u) & ~1023u;
    unsigned char *base = smem_raw + (ring - raw) + (size_t)a.stages * C::STAGE;
    volatile int *s_abort = &s_abort_storage;
    unsigned char *meta = base + C::OffMeta;
    float *s_max = reinterpret_cast<float *>(base + C::OffRed);     // [2][4][2 GP]
    float *s_sum = s_max + 16 * GP;                                 // [2][4][GP]
    float *s_fq = s_sum + 8 * GP;                                   // [GP]
    float *s_ml = s_fq + GP;                                        // [2][GP][2]
    int *s_pref = reinterpret_cast<int *>(base + C::OffPref);
    const uint32_t bars = smem_u32(base + C::OffBar);
    const uint32_t full = bars, empty = bars + 64, sfull = bars + 128, ofull = bars + 144, drain = bars + 160;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        s_abort_storage = 0;
        for (int i = 0; i < kBlkMaxStages; ++i) {
            mbar_init(full + i * 8, 2);
            mbar_init(empty + i * 8, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull + i * 8, 1);
            mbar_init(ofull + i * 8, 1);
            mbar_init(drain + i * 8, 1);
        }
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(&s_tmem), kBlkTmemCols);
    if (warp >= 8 && lane == 0) {
        prefetch_tmap(warp & 1 ? &a.tm_v16 : &a.tm_k16);
        prefetch_tmap(warp & 1 ? &a.tm_v1 : &a.tm_k1);
    }
    if (!a.early_meta) pdl_wait();
    int2 *s_req = reinterpret_cast<int2 *>(base + C::off_req(a.batch));
    blk_plan<kBlkThreads>(a, s_pref, s_req, s_w);
    if (a.early_meta) pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0) {
        for (int b = tid; b < a.batch; b += kBlkThreads) {
            const int row = __ldg(a.req_pool_indices + b), n = __ldg(a.seq_lens + b);
            if (row < 0 || row >= a.req_rows) set_error(a.err, PA_DEVERR_ROW);
            if (n < 0 || n > a.max_ctx) set_error(a.err, PA_DEVERR_LEN);
        }
    }
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int W = blk_width(s_pref, a.batch, a.Hkv, a.grid);

    if (warp >= 8) {
        blk_loader<D, E8, GP>(a, s_pref, s_req, W, ring, meta, full, empty, s_abort, warp & 1, (warp - 8) >> 1, lane);
    } else {
        const int wg = warp >> 2, t = tid & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = tmem + wg * 128, o_col = s_col + 64;
        const uint32_t sQ = smem_u32(base + C::OffQ), sP = smem_u32(base + C::OffP) + wg * C::align_k(C::PB);
        constexpr uint32_t kFmt = E8 ? 0u : (1u << 7 | 1u << 10);      // e4m3 : bf16
        constexpr uint32_t kIdS = 1u << 4 | kFmt | (uint32_t)(C::NQ >> 3) << 17 | 8u << 24;
        constexpr uint32_t kIdO = 1u << 4 | kFmt | 1u << 15 | (uint32_t)(C::NP >> 3) << 17 | 8u << 24;   // A is MN-major
        constexpr float kShift = E8 ? 8.f : 0.f;    // P' reaches 2^8, within e4m3's 448
        bool bad = false;
        int st = 0, seq = 0, done = 0;              // ring stage, tile of the CTA, tiles of this warpgroup
        uint32_t ph = 0;
        // warp-uniform; after a time-out the warps run through the remaining
        // barriers without issuing or waiting, so none of them is left behind
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (!bad) bad = !__all_sync(0xffffffffu, mbar_wait(bar, parity, s_abort, a.err, PA_DEVERR_TIMEOUT, a.wait_ns));
        };
        int shared_b[2], shared_h[2], shared = 0;   // segments of which this CTA has a piece: at most two
        int ticket[2];
        // this thread's chunk of the piece's query rows, requested while the piece before it ends
        constexpr int CH = D / 8;               // 8-element chunks of a head row
        const int qg = tid / CH, qc = tid % CH;
        auto load_q = [&](const BlkWalk &k) -> uint4 {
            if (qg >= a.G) return make_uint4(0u, 0u, 0u, 0u);
            return __ldg(reinterpret_cast<const uint4 *>(a.q + ((int64_t)k.b * a.Hq + k.h * a.G + qg) * D) + qc);
        };
        BlkWalk k = blk_begin(s_pref, a.batch, a.Hkv, W, blockIdx.x), kn = k;
        uint4 qn = make_uint4(0u, 0u, 0u, 0u);
        bool more = blk_piece(a, s_pref, s_req, kn);
        if (more) qn = load_q(kn);
        while (more) {
            k = kn;
            if (a.wait_ns == 0 && !bad) {
                // a wait limit of 0: give up at the first item, as a timed-out wait would
                *s_abort = 1;
                set_error(a.err, PA_DEVERR_TIMEOUT);
                bad = true;
            }
            // ---- q as the B operand, rows (term, head)
            {
                const int g = qg, c = qc;
                const uint4 w = qn;
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
                fence_proxy_async_smem();
                named_bar_sync(3, kBlkConsumers);
            }
            float m[GP], r[GP], l[GP], o[GP];
#pragma unroll
            for (int g = 0; g < GP; ++g) m[g] = r[g] = -INFINITY, l[g] = o[g] = 0.f;

            for (int i = 0; i < k.live; ++i, ++seq) {
                const int cst = st;
                const uint32_t cph = ph;
                if (++st == a.stages) {
                    st = 0;
                    ph ^= 1;
                }
                if ((seq & 1) != wg) continue;
                const uint32_t kt = ring + cst * C::STAGE, vt = kt + C::TILE;
                wait(full + cst * 8, cph);
                // S = K Q^T
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
                        umma_commit(sfull + wg * 8);
                    }
                    __syncwarp();
                }
                const int ek = meta[cst * kBlkTile + t], ev = E8 ? meta[(kBlkMaxStages + cst) * kBlkTile + t] : 0;
                wait(sfull + wg * 8, done & 1);
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
                float *red = s_max + (wg * 4 + (warp & 3)) * 2 * GP;
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float mx = warp_max(x[g]), rx = E8 ? warp_max(x[g] + (float)ev) : mx;
                    if (lane == 0) {
                        red[g] = mx;
                        red[GP + g] = rx;
                    }
                }
                named_bar_sync(1 + wg, 128);
                float bt[GP], at[GP];
                float pp[GP];
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float *w = s_max + wg * 8 * GP + g;
                    const float mt = fmaxf(fmaxf(w[0], w[2 * GP]), fmaxf(w[4 * GP], w[6 * GP]));
                    const float rt = E8 ? fmaxf(fmaxf(w[GP], w[3 * GP]), fmaxf(w[5 * GP], w[7 * GP])) : mt;
                    const float mn = fmaxf(m[g], mt), rn = fmaxf(r[g], rt);
                    const float mz = mn == -INFINITY ? 0.f : mn, rz = rn == -INFINITY ? 0.f : rn;
                    const float rtz = rt == -INFINITY ? 0.f : rt;
                    l[g] = l[g] * blk_ex2(m[g] - mz) + blk_ex2(x[g] - mz);
                    pp[g] = blk_ex2(x[g] + (float)ev - rtz + kShift);
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
                named_bar_sync(1 + wg, 128);
                // O^T = V^T P^T
                if ((warp & 3) == 0) {
                    tc_fence_after();
                    if (!bad) if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < C::PSteps; ++s) {
                            // V is [token][d]: 32 / ES tokens per step; the second 128-byte half of a bf16 row is the
                            // upper 64 of M; a row of 64 elements serves both halves of M (leading offset 0)
                            const uint64_t da = blk_desc<AW>(vt + s * (32 / ES) * AW, C::HALVES > 1 ? C::HALF : 0, 8 * AW);
                            const uint64_t db = blk_desc<128>(sP + (s >> 2) * (C::NP * 128) + (s & 3) * 32, 16, 1024);
                            blk_umma<E8>(o_col, da, db, kIdO, s > 0);
                        }
                        umma_commit(ofull + wg * 8);
                        umma_commit(empty + cst * 8);
                    }
                    __syncwarp();
                }
                wait(ofull + wg * 8, done & 1);
                ++done;
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

            // ---- the item ends: the warpgroup's sums, then both warpgroups
            blk_next(a, kn);
            more = blk_piece(a, s_pref, s_req, kn);
            if (more) qn = load_q(kn);
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                float s = l[g];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                if (lane == 0) s_sum[(wg * 4 + (warp & 3)) * GP + g] = s;
                // this warpgroup's O relative to its m: 2^(r - 127 - 8 - m)
                const float mz = m[g] == -INFINITY ? 0.f : m[g], rz = r[g] == -INFINITY ? 0.f : r[g];
                o[g] *= blk_ex2(E8 ? rz - mz - 135.f : 0.f);
            }
            float *scratch = reinterpret_cast<float *>(base + C::OffP);      // [GP][D]: warpgroup 1's O
            named_bar_sync(3, kBlkConsumers);   // the P tiles are free
            if (wg == 1 && t < D) {
#pragma unroll
                for (int g = 0; g < GP; ++g) scratch[g * D + t] = o[g];
            }
            if (t == 0) {
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float *w = s_sum + wg * 4 * GP + g;
                    s_ml[(wg * GP + g) * 2] = m[g];
                    s_ml[(wg * GP + g) * 2 + 1] = w[0] + w[GP] + w[2 * GP] + w[3 * GP];
                }
            }
            named_bar_sync(3, kBlkConsumers);
            const bool whole = k.t0 == 0 && k.t1 == k.tb;
            if (wg == 0 && t < D && !bad) {
                const int part = (int)blockIdx.x * 2 + (k.t0 == 0 && k.S0 > (int)blockIdx.x * W ? 1 : 0);
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    if (g >= a.G) break;
                    const float m0 = s_ml[g * 2], l0 = s_ml[g * 2 + 1], m1 = s_ml[(GP + g) * 2], l1 = s_ml[(GP + g) * 2 + 1];
                    const float M = fmaxf(m0, m1), Mz = M == -INFINITY ? 0.f : M;
                    const float w0 = blk_ex2(m0 - Mz), w1 = blk_ex2(m1 - Mz);
                    const float L = w0 * l0 + w1 * l1, O = w0 * o[g] + w1 * scratch[g * D + t];
                    const int64_t hq = (int64_t)k.b * a.Hq + k.h * a.G + g;
                    if (whole) {
                        a.out[hq * D + t] = __float2bfloat16_rn(L != 0.f ? O / L : 0.f);
                        if (WT && t == 0) a.lse[hq] = L != 0.f ? M + log2f(L) : INFINITY;
                    } else {
                        a.o_part[((int64_t)part * a.G + g) * D + t] = O;
                        if (t == 0) {
                            a.ml_part[(part * a.G + g) * 2] = M;
                            a.ml_part[(part * a.G + g) * 2 + 1] = L;
                        }
                    }
                }
            }
            if (!whole) {
                // a ticket for the piece: the barrier orders the partials' stores before thread 0's acquire-release
                // addition; the answer is looked at after the CTA's last piece
                if (wg == 0) {
                    named_bar_sync(1, 128);
                    if (t == 0 && !bad) {
                        const int old = atom_add_acq_rel_gpu(a.tickets + k.S0 / W, 1);
                        if (shared == 0) ticket[0] = old;
                        else ticket[1] = old;
                    }
                }
                if (shared == 0) shared_b[0] = k.b, shared_h[0] = k.h;
                else shared_b[1] = k.b, shared_h[1] = k.h;
                ++shared;
            }
        }
        // shared segments whose last piece was this CTA's
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i >= shared) break;
            const BlkSpan s = blk_span(s_pref, a.batch, W, shared_b[i], shared_h[i]);
            if (tid == 0) s_last[i] = !bad && ticket[i] == s.c1 - s.c0;
            named_bar_sync(3, kBlkConsumers);
            if (s_last[i]) {
                blk_merge<D, GP, WT>(a, s, W, shared_b[i], shared_h[i]);
                if (tid == 0) a.tickets[s.c0] = 0;
            }
        }
        if (__any_sync(0xffffffffu, *s_abort) && (warp & 3) == 0) {
            // aborted: every MMA this lane issued completes before tensor memory is freed
            if (elect_one()) umma_commit(drain + wg * 8);
            __syncwarp();
            mbar_drain(drain + wg * 8, 0);
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kBlkTmemCols);
    }
}

// ---------------------------------------------------------------- weights
constexpr int kBlkWeightThreads = 128;

// weights[row, j] += sum over the heads of 2^(score - lse), one 128-token tile
// of a request at a time, heads in order.
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
    const int tiles = s_pref[B];
    for (int x = blockIdx.x; x < tiles; x += gridDim.x) {
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pref[mid] <= x) lo = mid; else hi = mid;
        }
        const int b = lo, n = blk_len(a, b), row = __ldg(a.req_pool_indices + b);
        // two requests of a row would both add to it: the later one is refused
        int again = 0;
        for (int c = tid; c < b; c += kBlkWeightThreads) again |= __ldg(a.req_pool_indices + c) == row;
        __syncthreads();   // s_lse is free
        for (int hq = tid; hq < a.Hq; hq += kBlkWeightThreads) s_lse[hq] = __ldcg(a.lse + (int64_t)b * a.Hq + hq);
        again = __syncthreads_or(again);
        if (n <= 0) continue;
        if (again || x >= a.cap_tiles) {
            if (tid == 0) set_error(a.err, again ? PA_DEVERR_ROW : PA_DEVERR_LEN);
            continue;
        }
        const int j = (x - s_pref[b]) * kBlkTile + tid;
        if (j < n) {
            float w = 0.f;
            for (int h = 0; h < a.Hkv; ++h) {
                const float *sc = a.scores + (((int64_t)h * a.cap_tiles + x) * kBlkTile + tid) * G;
                for (int g = 0; g < G; ++g) w += blk_ex2(__ldcg(sc + g) - s_lse[h * G + g]);
            }
            a.weights[(int64_t)row * a.max_ctx + j] += w;
        }
    }
}

template <int D, bool E8, int GP, bool WT>
static pa_status launch_block(BlkArgs a, cudaStream_t st)
{
    using C = BlkCfg<D, E8, GP>;
    int stages = (int)((kBlkSmemLimit - C::fixed(a.batch)) / C::STAGE);
    a.stages = stages < kBlkMaxStages ? stages : kBlkMaxStages;
    static_assert(C::bytes(kBlkMaxBatch, 2) <= kBlkSmemLimit, "two stages fit at the largest batch");
    auto kern = decode_block_kernel<D, E8, GP, WT>;
    const size_t smem = C::bytes(a.batch, a.stages);
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem)) return PA_ERR_CUDA;
    a.grid = num_sms() < kBlkMaxCtas ? num_sms() : kBlkMaxCtas;
    if (launch_kernel(kern, dim3(a.grid), dim3(kBlkThreads), smem, st, a) != cudaSuccess) return PA_ERR_CUDA;
    if constexpr (WT) {
        const size_t wsmem = ((size_t)a.batch + 1) * 4 + (size_t)a.Hq * 4;
        if (!ensure_dynamic_smem(reinterpret_cast<const void *>(decode_block_weights_kernel), wsmem)) return PA_ERR_CUDA;
        if (launch_kernel(decode_block_weights_kernel, dim3(4 * a.grid), dim3(kBlkWeightThreads), wsmem, st, a) != cudaSuccess)
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
