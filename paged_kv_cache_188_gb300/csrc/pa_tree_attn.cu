// pa_tree_attn.cu -- attention of drafted tokens (a tree or a chain per request)
// over the paged cache on tcgen05, bf16 or block-scaled e4m3.
//
// For node i of a request (n nodes, the last of its L cached tokens, context c = L
// - n) and query head hq = h G + g:
//     s_j = scale <q_i, K_j>,   out_i = sum_j softmax(s)_j V_j
// over j < c and the nodes whose bits the mask has for it.
//
// How.  All (node, head) pairs of a kv head read the same keys, so they are the
// rows of one product: a tile of M = 128 rows, row = node G + g.  K and V come
// once per 256 rows (a "pair" of tiles), and decode's problem stays: few rows, many
// keys, the keys' bytes are the bound (up to about 256 rows: 128 x 128 x D x 4
// operations take the tensor core half of the time that HBM takes for the
// 128-token tile).  So the work is cut along the keys: the segments (request,
// pair), 128-token tiles laid end to end, are cut into equal ranges, as many as
// there are CTAs per kv head; (range i, head h) is unit i Hkv + h, so that the heads
// of a token are read at about the same time.  A unit shares at most its first
// and its last segment with others: two slots of fp32 partials per unit, merged
// by a second kernel in the pieces' order (deterministic).
//
// A CTA has two streams, X = A and B, each with a warpgroup, a warp that issues its
// products, S columns, O columns and running maximum and sum:
//   more than 128 rows:  A and B are the two tiles of rows, over every token tile;
//   up to 128 rows:      A takes the even token tiles, B the odd ones, of the same
//                        rows, joined when the piece ends.
// The tensor core runs S_A S_B | PV_A S_A | PV_B S_B | ..., in turn (TURN): a step's
// softmax has the time of the other stream's products.
//   S = Q K^T      A = Q, B = K tile as TMA left it, fp32 in tensor memory
//   P over S       bf16 (2^-8 of a weight; the sum is of the unrounded ones), read by
//                  the second product from tensor memory
//   O += P V       fp32 in tensor memory, rescaled only when the running maximum
//                  grows by more than 2^8
// Warps 0-7: softmax, one row a thread; 8 and 9: K and V copies through the page
// table, of which 8 also walks the units' pieces and hands them to every role; 10
// and 11: a stream's products each.  16 consecutive slots are one TMA box.  Any
// other rows are 16-byte asynchronous copies (bf16), handed on when the next tile's
// have been issued: pages of one slot, 32 requests of up to 8192 tokens, 139 us by
// gather4 copies, 104 us so; and the end of a request's last page, 97.7 -> 93.6 us
// over 32 ragged requests.
//
// e4m3 cache.  K stays e4m3 in its product, against q's row as two e4m3 terms that
// share a scale (q within 2^-17 of its row's largest element); a key's scale joins
// the softmax scale where 16 keys share one.  V becomes bf16 with its scale, exactly,
// by the softmax warpgroups while S is on its way (48 requests of 500 to 8192
// tokens, before ranges counted pieces: behind the exponentials 193 us, like this
// 160; to fp16 with a running exponent 209; by warps without nodes' rows 178 to 192).
//
// Hidden rows: a hidden token's weight is 0, but 0 times a NaN or an infinity in
// its V row would reach every node.  Only drafted tokens are ever hidden (context
// is seen by all), so these V rows are looked through in shared memory, one
// that holds such a value becomes zeros, and the rows that do see it add its
// part by hand when the piece ends.
//
// Measured, both kernels in a graph, D = 128, 8 kv heads of 4 query heads: 403 MB of
// cache (32 requests of 500 to 8192 tokens, trees of up to 32 nodes) 90.5 us, 66 % of
// a copy's rate (6.78 TB/s); ncu over the first kernel: 403.4 MB read, tensor pipe
// active 28 %, issue slots 20 %.  One request of 32K tokens 51 us for 136 MB; of 1K
// 12.0 us, which is start, plan, two steps and the merge.  e4m3: 48 requests, 320 MB,
// 142 us; left out in copies that measured nothing else: the widening with the look through
// nodes' V rows 109, that look alone 133, q's split 139 (ncu: tensor pipe 25 %, issue slots 39 %
// of active cycles, DRAM 29 %: the widening and the softmax of a step follow one another).
// What bounds it.  Within a long piece over bf16 pages, HBM: a tile of 64 KB every
// 2700 cycles and SM.  Around it the start (10000 cycles to the first S), and each
// piece's end (5000 to 8000 for the partials, the next piece's Q and first tiles).
// With 256 rows, and over e4m3, a step's chain (S, its read-back of 128 columns,
// exponentials, P, PV), of which two are in flight.  S in two halves of 64 columns
// (2900 cycles a step for 2050), a tile kept from one piece to the next (99.6 us for
// 93.6), one ring for K and V in the order of their use (96.0 for 93.0), and rows
// without nodes skipped (spills: 26 -> 29 us at 96 small requests) lost.
#include <math.h>
#include <string.h>

#include "pa_e4m3_tiles.cuh"
#include "pa_internal.h"
#include "pa_sm100.cuh"

namespace pa {
using namespace sm100;

constexpr int kTreeMaxReqs = 4096;
constexpr int kTrTile = 128;             // tokens of a tile, rows of a stream
constexpr int kTrPair = 256;             // rows of two streams
constexpr int kTrThreads = 384;
constexpr int kTrHalf = 128 * 128;       // 128 rows of 64 bf16, 128-byte swizzle
constexpr int kTrMeta = 8;               // tiles whose valid positions are kept: see tr_copy
constexpr int kTrPieces = 4;             // pieces handed from the walk to the other roles
constexpr int kTrReaders = 1 + 2 + 8;    // V copies, products, softmax warps
constexpr int kTrMaxPieceCost = 6;
constexpr int kTrMaxCtas = 160;
constexpr int kTrMaxUnits = 2 * kTrMaxCtas;   // units that share segments
constexpr uint32_t kTrTmemCols = 512;    // S_A | S_B | O_A | O_B

struct TreeArgs {
    CUtensorMap tm_q;                            // 3-D (element, head, token): boxes of 64 x G x TQ
    CUtensorMap tm_k16, tm_k1, tm_v16, tm_v1;    // 2-D (element, row): boxes of 16 rows, and (e4m3) one row (gather4)
    const __nv_bfloat16 *q;
    const uint8_t *k, *v;                        // the layer's rows
    const uint8_t *k_exp, *v_exp;                // the layer's exponents (e4m3 cache)
    const int32_t *qo_indptr, *req_to_token, *req_pool_indices, *seq_lens, *tree_mask;
    __nv_bfloat16 *out;
    int32_t *err;
    float *ml_part;                              // [2 units][256][2]: maximum (log2 units), sum
    float *o_part;                               // [2 units][D / 4][256][4]: relative to that maximum
    int T, R, Hq, Hkv, G, size, req_rows, max_ctx, mask_words, block_shift, layer_row0, total_rows, early_meta;
    int ranges;                                  // per kv head
    int piece_cost;                              // what a piece's start and end take, in tiles
    uint64_t wait_ns;
    float scale_log2;                            // of the scale's magnitude, not 0
    int negate;                                  // the scale is negative: the products take Q with its sign changed
    int tq;                                      // nodes of a stream's tile of rows: 128 / G
    int inv_g;                                   // 65536 / G + 1: x / G = x inv_g >> 16 for x below 272
};

// ------------------------------------------------------------------- plan
struct alignas(16) TrReq {
    int q0, n, L, row;      // n = 0: nothing to do
};
// A request, and what is wrong with it: `zeros` where its rows become zeros.
__device__ __forceinline__ TrReq tr_request(const TreeArgs &a, int r, int &bits, bool &zeros)
{
    TrReq q;
    q.q0 = __ldg(a.qo_indptr + r);
    const int q1 = __ldg(a.qo_indptr + r + 1);
    q.L = __ldg(a.seq_lens + r);
    q.row = __ldg(a.req_pool_indices + r);
    q.n = q1 - q.q0;
    bits = 0;
    zeros = false;
    if (q1 <= q.q0 || q.q0 < 0 || q1 > a.T) {
        if (q1 != q.q0) bits = PA_DEVERR_LEN;
        q.n = 0;
        return q;
    }
    if (q.row < 0 || q.row >= a.req_rows) bits |= PA_DEVERR_ROW;
    if (q.L < q.n || q.L > a.max_ctx || (a.tree_mask && q.n > 32 * (int64_t)a.mask_words)) bits |= PA_DEVERR_LEN;
    zeros = bits != 0;
    return q;
}
// The largest end of the ranges in front of request r that lie in [0, T].  (A call: only a broken batch makes it, and
// copies of it in each place took 0.1 to 0.5 us more.)
__device__ __noinline__ int tr_front(const int32_t *qo_indptr, int T, int r)
{
    int front = 0;
#pragma unroll 1
    for (int j = 0; j < r; ++j) {
        const int q0 = __ldg(qo_indptr + j), q1 = __ldg(qo_indptr + j + 1);
        if (q0 >= 0 && q0 < q1 && q1 <= T) front = max(front, q1);
    }
    return front;
}
// `down`: the starts decrease somewhere.  Only then can a range begin in front of an earlier one's end; such a request is
// left out, so that no row is two requests' and all segments together are no more than the host allowed for.
__device__ __forceinline__ TrReq tr_request(const TreeArgs &a, int r, bool down, int &bits, bool &zeros)
{
    TrReq q = tr_request(a, r, bits, zeros);
    if (down && q.n > 0 && q.q0 < tr_front(a.qo_indptr, a.T, r)) {
        q.n = 0;
        bits = PA_DEVERR_LEN;
        zeros = false;
    }
    return q;
}
__device__ __forceinline__ TrReq tr_request(const TreeArgs &a, int r, bool down)
{
    int bits;
    bool zeros;
    TrReq q = tr_request(a, r, down, bits, zeros);
    if (zeros) q.n = 0;
    return q;
}
__device__ __forceinline__ int tr_pairs(const TreeArgs &a, int n) { return n <= 2 * a.tq ? 1 : (n + 2 * a.tq - 1) / (2 * a.tq); }
__device__ __forceinline__ int tr_ktiles(int L) { return (L + kTrTile - 1) / kTrTile; }
// The segments laid end to end: a segment is `cost` places that nobody works on and then its tiles, so that a range with
// several segments has fewer tiles (32 ragged requests 93.0 -> 89.6 us, 48 over e4m3 164.5 -> 141).  At most half of a
// range's tiles: 96 requests of up to 4000 tokens, two kv heads, 28.7 us at an eighth, 22.3 at a quarter, 20.3 at half,
// 21.3 at all of them; few long requests take the same time at each.
__device__ __forceinline__ int tr_places(const TreeArgs &a, const TrReq &q, int cost)
{
    return q.n > 0 ? tr_pairs(a, q.n) * (tr_ktiles(q.L) + cost) : 0;
}
// segments and tiles, to be summed together
__device__ __forceinline__ uint64_t tr_load(const TreeArgs &a, const TrReq &q)
{
    const uint32_t pairs = q.n > 0 ? tr_pairs(a, q.n) : 0;
    return (uint64_t)pairs << 32 | (pairs ? pairs * (uint32_t)tr_ktiles(q.L) : 0u);
}
__device__ __forceinline__ int tr_cost(const TreeArgs &a, uint64_t total) { return min(a.piece_cost, (int)((uint32_t)total / (2u * a.ranges))); }
__device__ __forceinline__ int tr_places(uint64_t load, int cost) { return (int)((uint32_t)load + (uint32_t)(load >> 32) * cost); }

struct TrPlan {
    int total, W, cost;     // places in all, of a range, of a segment before its tiles
    int down;               // the starts decrease somewhere
    int start[2][2];        // (request, its first place) where the CTA's units start (a third unit exists only where all
                            // of them are the whole of one kv head)
    TrReq req[2];           // that request
};
// A piece of a unit's range, for every role of the CTA: token tiles [t0, t1) of nodes 2 tq pair .. of a request.
struct alignas(16) TrPiece {
    int q0, n, L, row;
    int t0, t1, h, unit;
    int pair, whole, first, end;    // whole: all of its segment; first: it starts the range; end: no more pieces
};
// Walk over the pieces of the CTA's units (blockIdx, + grid, ...): range i = unit / Hkv is the places [i W, (i + 1) W) of
// the segments laid end to end.  One warp walks and hands the pieces on.
struct TrWalk {
    int unit, u, h;         // unit, its number in the CTA, kv head
    int x, xe, x0, r, S0;   // next place, end, start of the range; request and its first place
    int w0;                 // the lanes hold requests w0 + lane
    TrReq w;
};
__device__ __forceinline__ void tr_unit(const TreeArgs &a, const TrPlan &p, TrWalk &k)
{
    const int i = k.unit / a.Hkv, v = a.ranges > 1 ? k.u : 0;
    k.h = k.unit - i * a.Hkv;
    k.x = k.x0 = (int)min((int64_t)p.total, (int64_t)i * p.W);
    k.xe = min(p.total, k.x + p.W);
    k.r = p.start[v][0];
    k.S0 = p.start[v][1];
    k.w0 = k.r - 32;        // nothing there yet: the first request comes from the plan
}
__device__ __forceinline__ void tr_begin(const TreeArgs &a, const TrPlan &p, TrWalk &k)
{
    k.unit = blockIdx.x;
    k.u = 0;
    k.x = k.xe = 0;
    if (k.unit < a.ranges * a.Hkv) tr_unit(a, p, k);
}
__device__ __forceinline__ bool tr_next(const TreeArgs &a, const TrPlan &p, TrWalk &k, TrPiece &o, int lane)
{
#pragma unroll 1
    while (true) {
#pragma unroll 1
        while (k.x >= k.xe) {
            k.unit += gridDim.x;
            ++k.u;
            if (k.unit >= a.ranges * a.Hkv) return false;
            tr_unit(a, p, k);
        }
        TrReq q;
        int places;
#pragma unroll 1
        while (true) {
            const int v = a.ranges > 1 ? k.u : 0;
            if (k.x == k.x0 && k.r == p.start[v][0] && p.total > 0 && a.ranges > 1) {
                q = p.req[v];
            } else {
                if (k.r - k.w0 >= 32) {
                    k.w0 = k.r;
                    k.w = TrReq{0, 0, 0, 0};
                    if (k.r + lane < a.R) k.w = tr_request(a, k.r + lane, p.down);
                }
                const int i = k.r - k.w0;
                q.q0 = __shfl_sync(0xffffffffu, k.w.q0, i);
                q.n = __shfl_sync(0xffffffffu, k.w.n, i);
                q.L = __shfl_sync(0xffffffffu, k.w.L, i);
                q.row = __shfl_sync(0xffffffffu, k.w.row, i);
            }
            places = tr_places(a, q, p.cost);
            if (k.x < k.S0 + places) break;
            k.S0 += places;
            if (++k.r >= a.R) return false;      // (not reached: x lies below the total)
        }
        const int kt = tr_ktiles(q.L), off = k.x - k.S0, seg = kt + p.cost;
        o.q0 = q.q0, o.n = q.n, o.L = q.L, o.row = q.row;
        o.pair = places == seg ? 0 : off / seg;
        const int at = off - o.pair * seg - p.cost;      // the tile at place x, below 0 in front of them
        const int len = min(k.xe - k.x, kt - at);
        o.t0 = max(at, 0);
        o.t1 = at + len;
        o.h = k.h;
        o.unit = k.unit;
        o.whole = o.t0 == 0 && o.t1 == kt;
        o.first = k.x == k.x0 && at >= 0;
        o.end = 0;
        k.x += len;
        if (o.t1 > o.t0) return true;
    }
}
// the piece has rows for both streams
__device__ __forceinline__ bool tr_two(const TreeArgs &a, const TrPiece &k) { return k.n - 2 * a.tq * k.pair > a.tq; }

// 32 bits of what node i (row `qrow` of the mask) sees, from node s on (s < 0: context, all ones)
__device__ __forceinline__ uint32_t tr_seen(const TreeArgs &a, int64_t qrow, int i, int s)
{
    if (!a.tree_mask) {
        const int ones = i - s + 1;
        return ones <= 0 ? 0u : ones >= 32 ? 0xFFFFFFFFu : (1u << ones) - 1u;
    }
    const int w = s >> 5;
    const int32_t *m = a.tree_mask + qrow * a.mask_words;
    const uint32_t lo = w < 0 ? 0xFFFFFFFFu : w < a.mask_words ? (uint32_t)__ldg(m + w) : 0u;
    const uint32_t hi = w + 1 < 0 ? 0xFFFFFFFFu : w + 1 < a.mask_words ? (uint32_t)__ldg(m + w + 1) : 0u;
    return __funnelshift_r(lo, hi, s & 31);
}

// Shared memory: Q of both streams; (e4m3) V widened to bf16, a buffer per stream; the rings of K and V as they are in
// the cache; barriers; what goes with the tiles.
template <int D, bool E8>
struct TrCfg {
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = HALVES * kTrHalf;        // bf16
    static constexpr int RAW = E8 ? kTrTile * D : TILE;  // as cached
    static constexpr int NK = D == 128 ? 3 : 5, NV = D == 128 ? 2 : 5;   // ring stages
    static constexpr int OffWide = 2 * TILE;
    static constexpr int OffK = OffWide + (E8 ? 2 * TILE : 0);
    static constexpr int OffV = OffK + NK * RAW;
    static constexpr int OffBar = OffV + NV * RAW;
    enum { K_FULL, K_EMPTY = K_FULL + NK, V_FULL = K_EMPTY + NK, V_EMPTY = V_FULL + NV, S_FULL = V_EMPTY + NV,
           P_READY = S_FULL + 2, O_FULL = P_READY + 2, O_FREE = O_FULL + 2, Q_FULL = O_FREE + 2, DRAIN = Q_FULL + 2,
           Q_SPLIT = DRAIN + 2,                          // e4m3: Q is there in its terms
           WIDE_FREE = Q_SPLIT + 2,                      // and the stream's product with V is done
           TURN = WIDE_FREE + 2,                         // whose products are next
           JOINT = TURN + 2,                             // stream A's Q, for stream B
           ITEM_FULL, ITEM_EMPTY = ITEM_FULL + kTrPieces, N_BARS = ITEM_EMPTY + kTrPieces };
    static constexpr int OffMeta = (OffBar + N_BARS * 8 + 15) & ~15;     // uint4 [kTrMeta]: valid positions
    static constexpr int OffML = OffMeta + kTrMeta * 16;                 // float2 [128]: stream B's (m, l)
    static constexpr int OffKS = OffML + 128 * 8;                        // e4m3: float [kTrMeta][128], keys' scales
    static constexpr int OffVE = OffKS + (E8 ? kTrMeta * 512 : 0);       // bytes [kTrMeta][128], values' exponents
    static constexpr int OffGr = OffVE + (E8 ? kTrMeta * 128 : 0);       // int [kTrMeta]: 16 keys share a scale
    static constexpr int OffQS = OffGr + (E8 ? kTrMeta * 4 : 0);         // float [128], rows' scales of a joint piece
    static constexpr int OffEnd = OffQS + (E8 ? 512 : 0);
    static constexpr int Smem = OffEnd + 1024;
    static constexpr uint32_t ColO = 256;
    static constexpr uint32_t kIdS = E8 ? idesc_e4m3_f32(128, 128, 0, 0) : idesc_bf16_f32(128, 128, 0, 0);
    static constexpr uint32_t kIdPV = idesc_bf16_f32(128, D, 0, 1);
    static_assert(N_BARS <= 64, "two warps initialise the barriers");
    static_assert(OffKS % 16 == 0 && OffVE % 16 == 0 && OffQS % 16 == 0);
    static_assert(Smem <= 232448 - 512, "fits with the static shared memory");
    static_assert(kTrMeta >= NK + 3, "a tile's valid positions and scales outlive its ring stage");
};

__device__ __forceinline__ float tr_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a softmax scale that is not 0, as which a hidden key's minus infinity would be a NaN
__device__ __forceinline__ float tr_scale(float x) { return x < 0x1p-126f ? 0x1p-126f : x; }

// mbar_wait without a call, so that nothing is kept in memory for one: whole warp, the same answer in every lane.
__device__ __forceinline__ bool tr_wait(const TreeArgs &a, uint32_t bar, uint32_t parity, volatile int *s_abort)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_ns();
    bool ok = false;
#pragma unroll 1
    while (a.wait_ns != 0) {
        ok = mbar_try_wait(bar, parity);
        if (ok || *s_abort || global_ns() - t0 > a.wait_ns) break;
    }
    if (!ok && !*s_abort) {
        *s_abort = 1;
        set_error(a.err, PA_DEVERR_TIMEOUT);
    }
    return __all_sync(0xffffffffu, ok);
}

// The ring of pieces.  These two wait for nothing but other warps' control flow, and the roles run through every
// piece even when a copy or product has been given up (without waiting or issuing), so that no warp is missed at a
// barrier: the limit is only a last resort.
__device__ __forceinline__ void tr_wait_ring(uint32_t bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity) && global_ns() - t0 < 10000000000ull) {}
    __syncwarp();
}

// ----------------------------------------------------------------- copies
// K (isv false) or V tiles of the CTA's units.  Positions without a row (past the
// end, or a bad slot) are zeros; the K warp also writes which positions are valid:
// a ring of its own, because softmax reads them behind S, when the K stage is
// already free.  (Tile x is copied when S(x - NK) is done, which was issued behind
// softmax of tile x - NK - 1 at the latest.)
template <int D, bool E8>
__device__ __forceinline__ void tr_copy(const TreeArgs &a, const TrPlan &plan, TrPiece *pieces, uint32_t item_full,
                                        uint32_t item_empty, bool isv, uint32_t ring, uint32_t full, uint32_t empty,
                                        unsigned char *sb, volatile int *s_abort, int lane)
{
    using C = TrCfg<D, E8>;
    uint4 *meta = reinterpret_cast<uint4 *>(sb + C::OffMeta);
    const uint8_t *exps = isv ? a.v_exp : a.k_exp;
    const int stages = isv ? C::NV : C::NK;
    const CUtensorMap *m16 = isv ? &a.tm_v16 : &a.tm_k16, *m1 = isv ? &a.tm_v1 : &a.tm_k1;
    int st = 0, seq = 0, errs = 0;
    uint32_t ph = 0;
    bool go = true;
    // bf16: the tile whose 16-byte copies are on their way.  It is handed on when the next one's have been issued, or
    // before this warp waits for anything else
    uint32_t held = 0, held_bytes = 0;
    auto release_held = [&](int later) {
        if (later) cp_async_wait<1>();
        else cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(held, held_bytes);
        held = 0;
    };
    TrWalk w;
    if (!isv) tr_begin(a, plan, w);
#pragma unroll 1
    for (int it = 0;; ++it) {
        TrPiece k;
        const int slot = it % kTrPieces;
        if (isv) {
            tr_wait_ring(item_full + slot * 8, (it / kTrPieces) & 1);
            k = pieces[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(item_empty + slot * 8);
        } else {
            // this warp walks, and hands the pieces on
            k.end = !tr_next(a, plan, w, k, lane);
            if (it >= kTrPieces) tr_wait_ring(item_empty + slot * 8, (it / kTrPieces - 1) & 1);
            if (lane == 0) {
                pieces[slot] = k;
                mbar_arrive(item_full + slot * 8);
            }
        }
        if (k.end) break;
        const int col = k.h * D;
        const int32_t *tab = a.req_to_token + (int64_t)k.row * a.max_ctx;
        // a tile's table entries are requested while the tile before is copied, and (e4m3) its exponents, which hang on
        // them, behind that one's copies
        int nx[4], ex[4] = {0, 0, 0, 0};
        auto fetch = [&](int t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int p = t * kTrTile + 4 * lane + e;
                nx[e] = ld_nc_ordered_s32_if(p < k.L, tab + (p < k.L ? p : 0));
            }
        };
        auto fetch_exps = [&]() {
            if constexpr (E8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool in = nx[e] >= 0 && nx[e] < a.size;
                    ex[e] = in ? __ldcg(exps + (int64_t)(nx[e] >> a.block_shift) * a.Hkv + k.h) : 255;
                }
            }
        };
        fetch(k.t0);
        fetch_exps();
#pragma unroll 1
        for (int t = k.t0; t < k.t1 && go; ++t) {
            int sl[4] = {nx[0], nx[1], nx[2], nx[3]};
            if (t + 1 < k.t1) fetch(t + 1);
            if (!E8 && seq >= stages && held != 0 && !__all_sync(0xffffffffu, mbar_try_wait(empty + st * 8, ph ^ 1)))
                release_held(0);
            if (seq >= stages && !tr_wait(a, empty + st * 8, ph ^ 1, s_abort)) {
                go = false;
                break;
            }
            const uint32_t dst = ring + st * C::RAW, fb = full + st * 8;
            bool ok[4];
            uint32_t nib = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = t * kTrTile + 4 * lane + e < k.L;
                ok[e] = in && sl[e] >= 0 && sl[e] < a.size;
                if (in && !ok[e]) errs |= PA_DEVERR_SLOT;
                nib |= (uint32_t)ok[e] << e;
            }
            const int s0 = __shfl_sync(0xffffffffu, sl[0], lane & ~3);
            const bool run = nib == 15u && sl[0] == s0 + 4 * (lane & 3) && sl[1] == sl[0] + 1 && sl[2] == sl[0] + 2 &&
                             sl[3] == sl[0] + 3;
            const bool page = ((__ballot_sync(0xffffffffu, run) >> (lane & ~3)) & 0xFu) == 0xFu;
            const unsigned has = __ballot_sync(0xffffffffu, nib != 0u);
            const bool none = ((has >> (lane & ~3)) & 0xFu) == 0u;
            int some = 0;              // a valid row of the tile
            if constexpr (E8)
                some = __shfl_sync(0xffffffffu, nib & 1u ? sl[0] : nib & 2u ? sl[1] : nib & 4u ? sl[2] : sl[3],
                                   has ? __ffs(has) - 1 : 0);
            constexpr int HV = E8 ? 1 : C::HALVES, PITCH = E8 ? D : 128;     // boxes of a row, and their bytes
            if (page || none) {
                // a page's rows, or rows out of range, which read as zeros
                if ((lane & 3) == 0) {
#pragma unroll
                    for (int hh = 0; hh < HV; ++hh)
                        tma_load_2d(dst + hh * kTrHalf + (lane >> 2) * 16 * PITCH, m16, col + hh * 64,
                                    none ? a.total_rows : a.layer_row0 + sl[0], fb);
                }
            } else if constexpr (E8) {
                // a position without a row repeats a valid one of the tile: its exponent byte and its bit say so
#pragma unroll
                for (int e = 0; e < 4; ++e) sl[e] = a.layer_row0 + (ok[e] ? sl[e] : some);
                tma_gather4(dst + lane * 4 * PITCH, m1, col, sl[0], sl[1], sl[2], sl[3], fb);
            }
            uint32_t bytes = C::RAW;
            bool copied = false;
            if constexpr (!E8) {
                // rows anywhere, and the ends of pages: 16-byte copies, four lanes on 64 bytes of a row; zeros where there
                // is no row.  (gather4 copies cost 100 cycles of issue each, 64 a tile at D = 128: 32 requests of up to
                // 8192 tokens at pages of one slot took 139 us against 115; at D = 64 there is no difference.)
                const bool gathered = !page && !none;
                copied = __any_sync(0xffffffffu, gathered);
                if (copied) {
                    const uint8_t *rows = isv ? a.v : a.k;
                    bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, !gathered)) * 4u * 128u * C::HALVES;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const int from = __shfl_sync(0xffffffffu, sl[x & 3], (lane & ~3) + (x >> 2));
                        const bool row = __shfl_sync(0xffffffffu, (int)ok[x & 3], (lane & ~3) + (x >> 2));
                        if (!gathered) continue;
                        const int r = (lane >> 2) * 16 + x;
                        const uint8_t *src = rows + ((int64_t)(row ? from : 0) * a.Hkv + k.h) * (2 * D);
#pragma unroll
                        for (int q = 0; q < 2 * C::HALVES; ++q) {
                            const int ch = q * 4 + (lane & 3);
                            cp_async_16(dst + (ch >> 3) * kTrHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4), src + ch * 16, row ? 16 : 0);
                        }
                    }
                }
                cp_async_commit();
            }
            if (!isv) {
                uint32_t w = nib << (4 * (lane & 7));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
                if ((lane & 7) == 0) reinterpret_cast<uint32_t *>(meta + seq % kTrMeta)[lane >> 3] = w;
                __syncwarp();
            }
            if constexpr (E8) {
                const int at = seq % kTrMeta;
                if (isv) {
                    reinterpret_cast<uint32_t *>(sb + C::OffVE + at * 128)[lane] =
                        (uint32_t)((ok[0] ? ex[0] : 255) | (ok[1] ? ex[1] : 255) << 8 | (ok[2] ? ex[2] : 255) << 16 |
                                   (ok[3] ? ex[3] : 255) << 24);
                } else {
                    // do 16 keys share a scale? (those past the end do not matter)
                    const int x0 = __shfl_sync(0xffffffffu, ex[0], lane & ~3);
                    bool one = true;
#pragma unroll
                    for (int e = 0; e < 4; ++e) one = one && (t * kTrTile + 4 * lane + e >= k.L || (ok[e] && ex[e] == x0));
                    const bool grouped = __all_sync(0xffffffffu, one);
                    if (lane == 0) reinterpret_cast<int *>(sb + C::OffGr)[at] = grouped;
                    // (an empty block's scale is 2^-126 in place of 0: a hidden column's minus infinity stays that)
                    auto scale_of = [](int e) { return __uint_as_float((uint32_t)max(e, 1) << 23); };
                    reinterpret_cast<float4 *>(sb + C::OffKS + at * 512)[lane] =
                        make_float4(scale_of(ok[0] ? ex[0] : 0), scale_of(ok[1] ? ex[1] : 0), scale_of(ok[2] ? ex[2] : 0),
                                    scale_of(ok[3] ? ex[3] : 0));
                }
                __syncwarp();
            }
            if constexpr (!E8) {
                if (held != 0) release_held(1);
                if (copied) {
                    held = fb;
                    held_bytes = bytes;
                }
            }
            if (!copied && lane == 0) mbar_arrive_expect_tx(fb, bytes);
            __syncwarp();
            if (t + 1 < k.t1) fetch_exps();
            ++seq;
            if (++st == stages) {
                st = 0;
                ph ^= 1;
            }
        }
        if (!E8 && held != 0) release_held(0);
    }
    // the warp leaves only when its copies have landed, whether or not anyone has given up by now
#pragma unroll 1
    for (int j = max(0, seq - stages); j < seq; ++j) mbar_drain(full + (j % stages) * 8, (j / stages) & 1);
    if (errs && !isv) set_error(a.err, errs);
    __syncwarp();
}

// Does a 16-byte chunk hold a bf16 NaN or infinity?
__device__ __forceinline__ bool tr_wild(const uint4 &v)
{
    constexpr uint32_t M = 0x7F80u;
    auto w = [](uint32_t x) { return (x & M) == M || (x & M << 16) == M << 16; };
    return w(v.x) || w(v.y) || w(v.z) || w(v.w);
}

// Rows lo .. hi of a V tile that hold a NaN or an infinity become zeros; true if there was one.  Whole warp.
template <int D>
__device__ __forceinline__ bool tr_tame(uint32_t tile, int lo, int hi, int lane)
{
    constexpr int CH = D / 8, PER = 32 / CH;        // chunks of a row, rows at a time
    bool any = false;
#pragma unroll 1
    for (int r0 = lo; r0 < hi; r0 += 4 * PER) {
        // every chunk of the rows, in any order
        uint4 v[4];
        uint32_t at[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = r0 + e * PER + lane / CH;
            at[e] = tile + ((lane % CH) >> 3) * kTrHalf + r * 128 + (lane & 7) * 16;
            v[e] = r < hi ? ld_shared_v4(at[e]) : make_uint4(0u, 0u, 0u, 0u);
        }
        const bool bad = tr_wild(v[0]) || tr_wild(v[1]) || tr_wild(v[2]) || tr_wild(v[3]);
        if (!__any_sync(0xffffffffu, bad)) continue;
        any = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned b = __ballot_sync(0xffffffffu, tr_wild(v[e]));
            if ((b >> (lane / CH * CH)) & ((1u << CH) - 1u)) st_shared_v4(at[e], 0u, 0u, 0u, 0u);
        }
    }
    if (any) fence_proxy_async_smem();
    return any;
}

// Element d of a cached row (K, or V: their bytes and exponents) at `at` = (slot, head) D.
template <bool E8>
__device__ __forceinline__ float tr_element(const uint8_t *rows, const uint8_t *exps, int64_t at, int64_t block, int d)
{
    if constexpr (!E8) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(rows)[at + d]);
    const int e = exps[block];
    float x, y;
    e4m3x2_floats(rows[at + d], x, y);
    return e == 0 && x == x ? 0.f : x * __uint_as_float((uint32_t)e << 23);
}

// Rows r0 .. r0 + 31 of an e4m3 tile (rows of D bytes) times their scales as bf16, in the swizzled layout of the second
// product's operand; exponent byte 255 marks a position without a row, which becomes zeros.  Whole warp, D / 16 lanes a
// row; everything is read before anything is converted.
template <int D>
__device__ __forceinline__ void tr_widen(uint32_t src, uint32_t dst, const unsigned char *exps, int r0, int lane)
{
    constexpr int LPR = D / 16, RPP = 32 / LPR, N = 32 / RPP;    // lanes of a row, rows at a time, times
    const int rr = lane / LPR, j = lane % LPR;
    uint4 v[N];
    uint32_t ex[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        v[u] = ld_shared_v4(src + (uint32_t)((r0 + u * RPP + rr) * D + j * 16));
        ex[u] = exps[r0 + u * RPP + rr];
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int r = r0 + u * RPP + rr;
        const bool row = ex[u] != 255u;
        const uint32_t mul = row ? ex[u] * 0x00800080u : 0u;     // 2^(e - 127) as a pair of bf16
        if (!row) v[u] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            // (a row's second half of lanes writes its odd chunk first: eight lanes then hit all banks once)
            const int half = hh ^ (j >= LPR / 2);
            const uint32_t a = half ? v[u].z : v[u].x, b = half ? v[u].w : v[u].y;
            const int c = 2 * j + half;
            st_shared_v4(dst + (uint32_t)((c >> 3) * kTrHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                         mul_bf16x2(e4m3x2_to_bf16x2(a), mul), mul_bf16x2(e4m3x2_to_bf16x2(a >> 16), mul),
                         mul_bf16x2(e4m3x2_to_bf16x2(b), mul), mul_bf16x2(e4m3x2_to_bf16x2(b >> 16), mul));
        }
    }
    __syncwarp();
}

// What tr_tame took out, for one row of the piece (node i, query head hq) and 32 columns from d0 on: the parts of the
// nodes' V rows that hold a NaN or an infinity and that the node sees, weights relative to m2.
template <int D, bool E8>
__device__ __forceinline__ void tr_wild_rows(const TreeArgs &a, const TrPiece &q, int i, int hq, float m2, int d0,
                                             float (&o)[32])
{
    const int c = q.L - q.n;
    const int32_t *tab = a.req_to_token + (int64_t)q.row * a.max_ctx;
    const __nv_bfloat16 *qr = a.q + ((int64_t)(q.q0 + i) * a.Hq + hq) * D;
#pragma unroll 1
    for (int j = max(c, q.t0 * kTrTile); j < min(q.L, q.t1 * kTrTile); ++j) {
        const int slot = __ldg(tab + j);
        if (slot < 0 || slot >= a.size || !(tr_seen(a, q.q0 + i, i, j - c) & 1u)) continue;
        const int64_t at = ((int64_t)slot * a.Hkv + q.h) * D, block = (int64_t)(slot >> a.block_shift) * a.Hkv + q.h;
        bool wild = false;
#pragma unroll 1
        for (int d = 0; d < D; ++d) wild |= !isfinite(tr_element<E8>(a.v, a.v_exp, at, block, d));
        if (!wild) continue;
        float s = 0.f;
#pragma unroll 1
        for (int d = 0; d < D; ++d) s = fmaf(__bfloat162float(qr[d]), tr_element<E8>(a.k, a.k_exp, at, block, d), s);
        const float p = tr_ex2(fmaf(a.negate ? -s : s, a.scale_log2, -m2));
#pragma unroll
        for (int d = 0; d < 32; ++d) o[d] = fmaf(p, tr_element<E8>(a.v, a.v_exp, at, block, d0 + d), o[d]);
    }
}

// ----------------------------------------------------------------- kernel
template <int D, bool E8>
__global__ void __launch_bounds__(kTrThreads, 1) tree_attn_kernel(const __grid_constant__ TreeArgs a)
{
    using C = TrCfg<D, E8>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_w[kTrThreads / 32];
    __shared__ int s_abort_storage;
    __shared__ TrPlan plan;
    __shared__ TrPiece s_piece[kTrPieces];
    __shared__ int s_wild[2][8];               // per stream, at piece % 8: piece + 1 where a V row was taken out (the
                                               // rings keep the streams within 8 pieces of one another)
    __shared__ uint32_t s_tmem;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char *sb = smem_raw + (base - raw);
    volatile int *s_abort = &s_abort_storage;
    uint4 *meta = reinterpret_cast<uint4 *>(sb + C::OffMeta);
    float2 *s_ml = reinterpret_cast<float2 *>(sb + C::OffML);
    auto bar = [&](int i) -> uint32_t { return base + C::OffBar + i * 8; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid < C::N_BARS) {
        const bool softmax = (tid >= C::P_READY && tid < C::O_FULL) || (tid >= C::O_FREE && tid < C::Q_FULL) ||
                             (tid >= C::Q_SPLIT && tid < C::WIDE_FREE);
        const bool kempty = tid >= C::K_EMPTY && tid < C::V_FULL, vempty = tid >= C::V_EMPTY && tid < C::S_FULL;
        mbar_init(bar(tid), softmax ? 128u : kempty ? 2u : vempty ? (E8 ? 8u : 2u)
                                           : tid >= C::ITEM_EMPTY ? (uint32_t)kTrReaders : 1u);
    }
    if (warp < 2) fence_mbar_init();
    if (tid >= 64 && tid < 80) s_wild[(tid >> 3) & 1][tid & 7] = 0;
    if (tid == 0) {
        s_abort_storage = 0;
        plan.start[0][0] = plan.start[0][1] = plan.start[1][0] = plan.start[1][1] = 0;
    }
    if (warp == 10) tmem_alloc(smem_u32(&s_tmem), kTrTmemCols);
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&a.tm_k16);
        if (E8) prefetch_tmap(&a.tm_k1);
    }
    if (warp == 9 && lane == 0) {
        prefetch_tmap(&a.tm_v16);
        if (E8) prefetch_tmap(&a.tm_v1);
    }
    if (!a.early_meta) pdl_wait();

    if (warp == 4 && lane == 0) prefetch_tmap(&a.tm_q);
    // ---- plan: the segments' tiles in all, and where this CTA's units start
    int bits;
    bool zeros, down = false;
    {
        const int per = (a.R + kTrThreads - 1) / kTrThreads, lo = min(a.R, tid * per), hi = min(a.R, lo + per);
        uint64_t run, incl;
        TrReq q;                               // the thread's last request
#pragma unroll 1
        while (true) {                         // (again where the starts turn out to decrease)
            bool less = false;
            run = 0;
            bits = 0;
            zeros = false;
#pragma unroll 1
            for (int r = lo; r < hi; ++r) {
                int b;
                bool z;
                q = tr_request(a, r, down, b, z);
                less |= __ldg(a.qo_indptr + r + 1) < q.q0;
                if (z) q.n = 0;
                run += tr_load(a, q);
                bits |= b;
                zeros |= z;
            }
            incl = run;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) s_w[warp] = incl;
            if (!__syncthreads_or(zeros || (less && !down))) break;
            zeros = __syncthreads_or(zeros);
            if (down || !__syncthreads_or(less)) break;
            down = true;
        }
        uint64_t before = incl - run, all = 0, sums[kTrThreads / 32];
#pragma unroll
        for (int w = 0; w < kTrThreads / 32; ++w) sums[w] = s_w[w];
#pragma unroll
        for (int w = 0; w < kTrThreads / 32; ++w) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
        const int cost = tr_cost(a, all), total = tr_places(all, cost), mine = tr_places(before, cost), len = tr_places(run, cost);
        const int W = (total + a.ranges - 1) / a.ranges;
        if (tid == 0) {
            plan.total = total;
            plan.W = W;
            plan.cost = cost;
            plan.down = down;
        }
        if (a.ranges > 1 && len > 0) {
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                const int x = (int)((blockIdx.x + u * gridDim.x) / a.Hkv) * W;
                if (x < mine || x >= mine + len) continue;
                int S0 = mine, r = lo;
#pragma unroll 1
                for (; r < hi - 1; ++r) {
                    const int t = tr_places(a, tr_request(a, r, down), cost);
                    if (x < S0 + t) break;
                    S0 += t;
                }
                plan.start[u][0] = r;
                plan.start[u][1] = S0;
                plan.req[u] = r == hi - 1 ? q : tr_request(a, r, down);
            }
        }
    }
    if (a.early_meta) pdl_wait();
    pdl_launch_dependents();
    if (bits && blockIdx.x == 0) set_error(a.err, bits);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    if (zeros) {
        // requests that cannot be read: their rows become zeros
#pragma unroll 1
        for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
            int b;
            bool z;
            const TrReq q = tr_request(a, r, down, b, z);
            if (!z) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + (int64_t)q.q0 * a.Hq * D);
            for (int64_t x = tid; x < (int64_t)q.n * a.Hq * D / 8; x += kTrThreads) dst[x] = make_uint4(0u, 0u, 0u, 0u);
        }
    }

    if (warp == 8 || warp == 9) {
        const bool isv = warp == 9;
        tr_copy<D, E8>(a, plan, s_piece, bar(C::ITEM_FULL), bar(C::ITEM_EMPTY), isv, base + (isv ? C::OffV : C::OffK),
                       bar(isv ? C::V_FULL : C::K_FULL), bar(isv ? C::V_EMPTY : C::K_EMPTY), sb, s_abort, lane);
    } else if (warp >= 10) {
        // ======================================================= products
        // A warp per stream, so that one waits for its weights while the other issues; they issue a step's two products in
        // turn, in the order of the steps.  (Interleaved, both streams' products would end at the same time, and their
        // softmaxes, which want the same units, would run at the same time again.)
        const int X = warp - 10;
        const uint32_t sQ = base, sK = base + C::OffK, sV = base + C::OffV;
        const uint32_t id_s = C::kIdS | (!E8 && a.negate ? 1u << 13 : 0u);   // bit 13: A negated
        int seq = 0, piece = 0, px = 0, pq = 0, p2 = 0, pj = 0;   // token tiles, pieces before; this stream's steps, pieces; of
                                                                  // stream B: those with rows of its own, and with A's
        bool bad = false, turn = X == 0;
        int turns = 0;
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (!bad) bad = !tr_wait(a, b, parity, s_abort);
        };
#pragma unroll 1
        for (int it = 0;; ++it) {
            const int slot = it % kTrPieces;
            tr_wait_ring(bar(C::ITEM_FULL + slot), (it / kTrPieces) & 1);
            const TrPiece k = s_piece[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::ITEM_EMPTY + slot));
            if (k.end) break;
            const int nt = k.t1 - k.t0, two = tr_two(a, k);
            const int N = two ? 2 * nt : nt, c = k.L - k.n;
            // a ring stage is free when both streams are through with it, or twice the one that uses it
            auto release = [&](uint32_t b) {
                umma_commit(b);
                if (!two) umma_commit(b);
            };
            auto qk = [&](int st) {
                const uint32_t q = sQ + (two ? X : 0) * C::TILE, kk = sK + st * C::RAW;
                if constexpr (E8) {
                    // both terms of q against the same keys, 32 of D a step; D = 64: the terms share a 128-byte row
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                        constexpr int SPT = D / 32;
                        const int term = s / SPT, o = (s % SPT) * 32;
                        const uint64_t kd = D == 128 ? smem_desc_sw128(kk + o, 16, 1024) : smem_desc_sw64(kk + o, 16, 512);
                        umma_ss_f8(tmem + X * 128, smem_desc_sw128(q + term * (D == 128 ? kTrHalf : 64) + o, 16, 1024), kd,
                                   id_s, s > 0);
                    }
                } else
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    umma_ss(tmem + X * 128, smem_desc_sw128(q + (s >> 2) * kTrHalf + (s & 3) * 32, 16, 1024),
                            smem_desc_sw128(kk + (s >> 2) * kTrHalf + (s & 3) * 32, 16, 1024), id_s, s > 0);
                umma_commit(bar(C::S_FULL + X));
                release(bar(C::K_EMPTY + st));
            };
            const int dt = two ? 1 : 2;        // token tiles from one step of the stream to the next
            if (X < N) {
                const int s = seq + (two ? 0 : X), st = s % C::NK;
                // (stream B hears of A's Q from A's warp: it does not follow every phase of that barrier)
                if (X == 0) {
                    wait(bar(E8 ? C::Q_SPLIT : C::Q_FULL), piece & 1);
                    if (!two && N > 1 && lane == 0) mbar_arrive(bar(C::JOINT));
                } else {
                    wait(two ? bar((E8 ? C::Q_SPLIT : C::Q_FULL) + 1) : bar(C::JOINT), (two ? p2 : pj) & 1);
                    if (two) ++p2;
                    else ++pj;
                }
                wait(bar(C::K_FULL + st), (s / C::NK) & 1);
                tc_fence_after();
                if (!bad) if (elect_one()) qk(st);
                __syncwarp();
            }
#pragma unroll 1
            for (int t = two ? 0 : X; t < nt; t += dt, ++px) {
                const int s = seq + t, st = s % C::NV, sk = (s + dt) % C::NK;
                // (e4m3: the softmax warpgroup has widened V into the stream's buffer when the weights are there)
                const uint32_t vt = E8 ? base + C::OffWide + X * C::TILE : sV + st * C::RAW;
                if constexpr (!E8) wait(bar(C::V_FULL + st), (s / C::NV) & 1);
                // drafted tokens' rows must not hold what a weight of 0 does not cancel
                const int p0 = (k.t0 + t) * kTrTile, lo = max(0, c - p0), hi = min(kTrTile, k.L - p0);
                if (!E8 && lo < hi) {
                    if (X == 0 || !two) {
                        if (!bad && tr_tame<D>(vt, lo, hi, lane)) {
                            if (lane == 0) *(volatile int *)&s_wild[X][piece & 7] = piece + 1;
                            __threadfence_block();
                        }
                        __syncwarp();
                    }
                    if (two) named_bar_sync(2, 64);
                }
                // the piece's first product overwrites O
                if (t < dt && pq++ > 0) wait(bar(C::O_FREE + X), pq & 1);
                wait(bar(C::P_READY + X), px & 1);
                if (!turn) wait(bar(C::TURN + X), turns++ & 1);
                tc_fence_after();
                if (!bad) if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kTrTile / 16; ++kk)
                        umma_ts(tmem + C::ColO + X * D, tmem + X * 128 + kk * 8,
                                smem_desc_sw128(vt + kk * 2048, kTrHalf, 1024), C::kIdPV, kk > 0 || t >= dt);
                    if constexpr (E8) umma_commit(bar(C::WIDE_FREE + X));
                    else release(bar(C::V_EMPTY + st));
                    if (t + dt >= nt) umma_commit(bar(C::O_FULL + X));
                }
                __syncwarp();
                if (t + dt < nt) {
                    // (looked for in its turn only: the tile that was in the stage before may be the other stream's, whose
                    // arrival this warp has not followed, and a wait for a phase passes two phases early as well)
                    wait(bar(C::K_FULL + sk), ((s + dt) / C::NK) & 1);
                    tc_fence_after();
                    if (!bad) if (elect_one()) qk(sk);
                    __syncwarp();
                }
                // the next step, or the next piece's first
                turn = X == 0 && t + 1 >= nt && !two;
                if (!turn && lane == 0) mbar_arrive(bar(C::TURN + 1 - X));
            }
            seq += nt;
            ++piece;
        }
        // one more commit, which arrives once every product issued has completed, before tensor memory is freed
        if (elect_one()) umma_commit(bar(C::DRAIN + X));
        __syncwarp();
        mbar_drain(bar(C::DRAIN + X), 0);
        __syncwarp();
    } else {
        // ======================================== softmax, and the piece's end
        const int X = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + X * 128;
        int piece = 0, sx = 0, ox = 0, kseq = 0, p2 = 0;   // pieces, steps, ends of this stream, token tiles, pairs
        int qloads = 0;
        bool bad = false;
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (!bad) bad = !tr_wait(a, b, parity, s_abort);
        };
        // this stream's rows of Q (rows of nodes past the piece's are another's, or zeros: nobody reads their results)
        auto load_q = [&](const TrPiece &k) {
            if (row == 0 && (X == 0 || tr_two(a, k)) && !bad) {
                mbar_arrive_expect_tx(bar(C::Q_FULL + X), C::HALVES * 128 * a.G * a.tq);
#pragma unroll
                for (int hh = 0; hh < C::HALVES; ++hh)
                    tma_load_3d(base + X * C::TILE + hh * kTrHalf, &a.tm_q, hh * 64, k.h * a.G, k.q0 + (2 * k.pair + X) * a.tq,
                                bar(C::Q_FULL + X));
                ++qloads;
            }
        };
        tr_wait_ring(bar(C::ITEM_FULL), 0);
        if (!s_piece[0].end) load_q(s_piece[0]);
#pragma unroll 1
        while (!s_piece[piece % kTrPieces].end) {
            const TrPiece &k = s_piece[piece % kTrPieces];
            const int nt = k.t1 - k.t0, c = k.L - k.n;
            const bool two = tr_two(a, k);
            const int N = two ? 2 * nt : nt, t00 = k.t0;
            // this thread's row: a node and a head of its own
            const int nd = (row * a.inv_g) >> 16, node = (2 * k.pair + (two ? X : 0)) * a.tq + nd;
            const bool live = nd < a.tq && node < k.n;
            const int64_t qrow = k.q0 + node;
            float sl2 = a.scale_log2;
            if (a.wait_ns == 0 && !bad) {
                // a wait limit of 0: give up at the first piece, as a timed-out wait would
                *s_abort = 1;
                set_error(a.err, PA_DEVERR_TIMEOUT);
                bad = true;
            }
            if constexpr (E8) {
                // this thread's row of q, in place, into its two e4m3 terms; the row's scale joins the softmax scale
                if (X == 0 || two) {
                    wait(bar(C::Q_FULL + X), (X == 0 ? piece : p2) & 1);
                    const uint32_t qt = base + X * C::TILE;
                    float qs = split_q_row<D>(qt, row, a.negate ? -1.f : 1.f);
                    if (!(qs == qs)) {
                        // a NaN or an infinity in the row: its first term becomes NaN, and with it every score.  (As the
                        // softmax scale it would reach what the row does not see as well.)
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c)
                            st_shared_v4(qt + row * 128 + ((c ^ (row & 7)) << 4), 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        qs = 1.f;
                    }
                    if (X == 0) reinterpret_cast<float *>(sb + C::OffQS)[row] = qs;
                    fence_proxy_async_smem();
                    mbar_arrive(bar(C::Q_SPLIT + X));
                    sl2 = tr_scale(sl2 * qs);
                }
                p2 += two;
            }
            float m = -INFINITY, l = 0.f;      // maximum of s (not yet scaled), sum
#pragma unroll 1
            for (int i = X; i < N; i += 2, ++sx) {
                const int t = two ? i >> 1 : i, p0 = (t00 + t) * kTrTile;
                // what of the tile this row sees, before S is there
                uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
                const bool nodes = p0 + kTrTile > c;
                if (nodes) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int s = p0 - c + 32 * w;
                        if (s > -32) seen[w] = live ? tr_seen(a, qrow, node, s) : 0u;
                    }
                }
                if constexpr (E8) {
                    // V in bf16 with its scales, 32 rows a warp, while S is on its way: the stream's product before this
                    // step is done
                    const int s = kseq + t, st = s % C::NV;
                    const uint32_t wide = base + C::OffWide + X * C::TILE;
                    wait(bar(C::V_FULL + st), (s / C::NV) & 1);
                    if (sx > 0) wait(bar(C::WIDE_FREE + X), (sx - 1) & 1);
                    const int r0 = (warp & 3) * 32;
                    tr_widen<D>(base + C::OffV + st * C::RAW, wide, sb + C::OffVE + s % kTrMeta * 128, r0, lane);
                    if (lane == 0) {
                        mbar_arrive(bar(C::V_EMPTY + st));
                        if (!two) mbar_arrive(bar(C::V_EMPTY + st));
                    }
                    const int lo = max(c - p0, r0), hi = min(k.L - p0, r0 + 32);
                    if (lo < hi && tr_tame<D>(wide, lo, hi, lane) && lane == 0)
                        *(volatile int *)&s_wild[X][piece & 7] = piece + 1;
                    fence_proxy_async_smem();
                }
                wait(bar(C::S_FULL + X), sx & 1);
                tc_fence_after();
                const uint4 valid = meta[(kseq + t) % kTrMeta];
                if constexpr (E8) {
                    if (i == 1 && X == 1 && !two) sl2 = tr_scale(sl2 * reinterpret_cast<const float *>(sb + C::OffQS)[row]);
                }
                const bool masked = nodes || (valid.x & valid.y & valid.z & valid.w) != ~0u;
                seen[0] &= valid.x, seen[1] &= valid.y, seen[2] &= valid.z, seen[3] &= valid.w;
                uint32_t r[128];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) tmem_ld32(s_addr + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(&r[ch * 32]));
                tmem_wait_ld();
                // e4m3: a column's key scale joins the softmax scale where 16 columns share one, else S takes it now
                const int at = (kseq + t) % kTrMeta;
                float gs[8];
                if constexpr (E8) {
                    const float *ks = reinterpret_cast<const float *>(sb + C::OffKS + at * 512);
                    if (reinterpret_cast<const int *>(sb + C::OffGr)[at]) {
#pragma unroll
                        for (int g = 0; g < 8; ++g) gs[g] = ks[16 * g];
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float4 f = reinterpret_cast<const float4 *>(ks)[j];
                            r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) * f.x);
                            r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) * f.y);
                            r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) * f.z);
                            r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) * f.w);
                        }
#pragma unroll
                        for (int g = 0; g < 8; ++g) gs[g] = 1.f;
                    }
                }
                if (masked) {
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (!(seen[j >> 5] >> (j & 31) & 1u)) r[j] = __float_as_uint(-INFINITY);
                }
                float mx = -INFINITY;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    auto f = [&](int j) { return __uint_as_float(r[16 * g + j]); };
                    const float a0 = max3(f(0), f(1), f(2)), a1 = max3(f(3), f(4), f(5)), a2 = max3(f(6), f(7), f(8));
                    const float a3 = max3(f(9), f(10), f(11)), a4 = max3(a0, f(12), f(13)), a5 = max3(a1, f(14), f(15));
                    const float top = fmaxf(max3(a2, a3, a4), a5);
                    mx = fmaxf(mx, E8 ? top * gs[g] : top);
                }
                bool rescale = false;
                float m_new = m;
                if (mx > m && (m == -INFINITY || (mx - m) * sl2 > 8.f)) {
                    rescale = m != -INFINITY;
                    m_new = mx;
                }
                const float alpha = rescale ? tr_ex2((m - m_new) * sl2) : 1.f;
                m = m_new;
                const float mb = m == -INFINITY ? 0.f : m * sl2;
                const uint64_t nmb2 = f32x2_pack(-mb, -mb);
                uint64_t sl22 = f32x2_pack(sl2, sl2), sum2 = f32x2_pack(0.f, 0.f);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t pk[32];
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        if (E8 && j % 16 == 0) {
                            const float sg = tr_scale(sl2 * gs[hh * 4 + j / 16]);
                            sl22 = f32x2_pack(sg, sg);
                        }
                        const uint64_t x = fma_f32x2(
                            f32x2_pack(__uint_as_float(r[hh * 64 + j]), __uint_as_float(r[hh * 64 + j + 1])), sl22, nmb2);
                        const float v0 = tr_ex2(f32x2_lo(x)), v1 = tr_ex2(f32x2_hi(x));
                        sum2 = add_f32x2(sum2, f32x2_pack(v0, v1));
                        pk[j / 2] = pack_bf16x2(v0, v1);
                    }
                    tmem_st32(s_addr + hh * 32, pk);
                }
                l = l * alpha + (f32x2_lo(sum2) + f32x2_hi(sum2));
                // O is stable here: S(i) completing implies that the stream's product before it did
                if (i >= 2 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t o[32];
                        tmem_ld32(tmem + lane_base + C::ColO + X * D + ch * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                        tmem_st32(tmem + lane_base + C::ColO + X * D + ch * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(C::P_READY + X));
            }
            kseq += nt;
            // ---- the piece ends
            if (X < N) wait(bar(C::O_FULL + X), ox & 1), ++ox;
            tc_fence_after();
            float m2 = m == -INFINITY ? -INFINITY : m * sl2, fa = 1.f, fb = 0.f;
            const bool join = !two && N > 1;   // stream B's part of the same rows
            // one tile of rows: the warpgroups end it together, with or without steps for stream B, whose roles else got ahead
            // of tiles that they do not follow: a wait for a stage's next tile would pass before this one's has come
            if (join && X == 1) s_ml[row] = make_float2(m2, l);
            if (!two) {
                // (stream A reads B's O below: B's wait for its last product is ordered in front of that)
                tc_fence_before();
                named_bar_sync(1, 256);
                tc_fence_after();
            }
            if (join) {
                if (X == 0) {
                    const float2 b = s_ml[row];
                    const float mm = fmaxf(m2, b.x), mz = mm == -INFINITY ? 0.f : mm;
                    fa = tr_ex2(m2 - mz);
                    fb = tr_ex2(b.x - mz);
                    l = l * fa + b.y * fb;
                    m2 = mm;
                }
            }
            // the next piece's Q comes while this one ends (both streams are through with S)
            tr_wait_ring(bar(C::ITEM_FULL + (piece + 1) % kTrPieces), ((piece + 1) / kTrPieces) & 1);
            if (!s_piece[(piece + 1) % kTrPieces].end) load_q(s_piece[(piece + 1) % kTrPieces]);
            const bool ends = two || X == 0;
            if (ends) {
                const bool wild = *(volatile int *)&s_wild[0][piece & 7] == piece + 1 ||
                                  *(volatile int *)&s_wild[1][piece & 7] == piece + 1;
                const float inv = l != 0.f ? 1.f / l : 0.f;
                const int mine = (two ? X * kTrTile : 0) + row, hq = k.h * a.G + row - nd * a.G;
                const bool whole = k.whole;
                const int64_t slot = 2 * k.unit + (k.first ? 0 : 1), out_row = (qrow * a.Hq + hq) * D;
                float4 *part = reinterpret_cast<float4 *>(a.o_part + slot * kTrPair * D) + mine;   // [D / 4][256]
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t ob[32];
                    float o[32];
                    tmem_ld32(tmem + lane_base + C::ColO + X * D + ch * 32, ob);
                    if (join) {
                        uint32_t oc[32];
                        tmem_ld32(tmem + lane_base + C::ColO + D + ch * 32, oc);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(ob[j]) * fa + __uint_as_float(oc[j]) * fb;
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(ob[j]);
                    }
                    if (wild && live) tr_wild_rows<D, E8>(a, k, node, hq, m2 == -INFINITY ? 0.f : m2, ch * 32, o);
                    if (live && !bad && whole) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            uint32_t p[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) p[e] = l != 0.f ? pack_bf16x2(o[j + 2 * e] * inv, o[j + 2 * e + 1] * inv) : 0u;
                            *reinterpret_cast<uint4 *>(a.out + out_row + ch * 32 + j) = make_uint4(p[0], p[1], p[2], p[3]);
                        }
                    } else if (live && !bad) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            part[(ch * 8 + j / 4) * kTrPair] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    }
                    __syncwarp();
                }
                if (!whole && live && !bad) reinterpret_cast<float2 *>(a.ml_part)[slot * kTrPair + mine] = make_float2(m2, l);
                tc_fence_before();
                mbar_arrive(bar(C::O_FREE + X));
                if (join) mbar_arrive(bar(C::O_FREE + 1));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::ITEM_EMPTY + piece % kTrPieces));
            ++piece;
        }
        // the copies of Q have landed before the shared memory goes
        if (qloads > 0) mbar_drain(bar(C::Q_FULL + X), (qloads - 1) & 1);
    }
    __syncthreads();
    if (warp == 10) {
        tc_fence_after();
        tmem_dealloc(tmem, kTrTmemCols);
    }
}

// ------------------------------------------------------------------ merge
// The rows of segments that several units worked on, pieces in order.  A CTA
// takes a part of a node's heads; a thread has 8 columns of a row, its
// neighbours the other heads of the group, whose partials lie side by side.  PG
// threads share those pieces where there are few nodes (a long request's 19 pieces are
// then one round trip or two).
constexpr int kTrMergeThreads = 256, kTrMergeCols = 8;

template <int D, int PG>
__global__ void __launch_bounds__(kTrMergeThreads, 2) tree_merge_kernel(const __grid_constant__ TreeArgs a)
{
    constexpr int NC = kTrMergeCols / 4, GROUPS = D / kTrMergeCols, U = PG > 1 ? 6 : 4;
    constexpr int EPC = kTrMergeThreads / PG, EPW = 32 / PG;     // elements of a CTA, of a warp
    extern __shared__ int s_pref[];                    // [R + 1] first places, [R] first rows of q, tiles of a segment
    __shared__ uint64_t s_w[kTrMergeThreads / 32];
    __shared__ int s_cost;
    int *s_q0 = s_pref + a.R + 1, *s_kt = s_q0 + a.R;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    {
        const int per = (a.R + kTrMergeThreads - 1) / kTrMergeThreads, lo = min(a.R, tid * per), hi = min(a.R, lo + per);
        uint64_t run, before, all;
        bool down = false;
#pragma unroll 1
        while (true) {                         // (again where the starts turn out to decrease)
            bool less = false;
            run = 0;
#pragma unroll 1
            for (int r = lo; r < hi; ++r) {
                const TrReq q = tr_request(a, r, down);
                less |= __ldg(a.qo_indptr + r + 1) < q.q0;
                s_pref[r] = q.n > 0 ? tr_pairs(a, q.n) : 0;
                // a node's request is found by bisection over the starts: where they decrease, a request that is left out
                // gets the end of those in front of it in place of its own start
                s_q0[r] = down && q.n == 0 ? tr_front(a.qo_indptr, a.T, r) : q.q0;
                s_kt[r] = q.n > 0 ? tr_ktiles(q.L) : 0;
                run += tr_load(a, q);
            }
            uint64_t incl = run;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            // (bit 63, which no sum reaches: a start below the one before.  With the warps' sums it costs no barrier more)
            less = __any_sync(0xffffffffu, less && !down);
            if (lane == 31) s_w[warp] = incl | (uint64_t)less << 63;
            __syncthreads();
            uint64_t flags = 0;
            before = incl - run;
            all = 0;
#pragma unroll
            for (int w = 0; w < kTrMergeThreads / 32; ++w) {
                const uint64_t x = s_w[w];
                if (w < warp) before += x;
                all += x;
                flags |= x;
            }
            if (!(flags >> 63)) break;
            down = true;
            __syncthreads();
        }
        const int c = tr_cost(a, all);
        int at = tr_places(before, c);
#pragma unroll 1
        for (int r = lo; r < hi; ++r) {
            const int places = s_pref[r] * (s_kt[r] + c);
            s_pref[r] = at;
            at += places;
        }
        if (tid == kTrMergeThreads - 1) {
            s_pref[a.R] = tr_places(all, c);
            s_cost = c;
        }
    }
    __syncthreads();
    const int total = s_pref[a.R], W = (total + a.ranges - 1) / a.ranges, cost = s_cost;
    const int per_row = a.Hq * GROUPS, parts = (per_row + EPC - 1) / EPC, sub = lane / EPW;
    bool waited = false;
#pragma unroll 1
    for (int64_t item = blockIdx.x; item < (int64_t)a.T * parts; item += gridDim.x) {
        const int t = (int)(item / parts), e = (int)(item - (int64_t)t * parts) * EPC + warp * EPW + lane % EPW;
        // the last request that starts at or in front of the node
        int lo = 0, hi = a.R;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_q0[mid] <= t) lo = mid; else hi = mid;
        }
        const int S0 = s_pref[lo], places = s_pref[lo + 1] - S0, node = t - s_q0[lo], tile = node / a.tq;
        const int pair = tile >> 1, kt = s_kt[lo], S = S0 + pair * (kt + cost) + cost;      // place of its first tile
        // (past the request's nodes; or its segment lies in one range and was never shared)
        if (places == 0 || node < 0 || (pair + 1) * (kt + cost) > places || S / W == (S + kt - 1) / W) continue;
        if (node >= __ldg(a.qo_indptr + lo + 1) - s_q0[lo]) continue;
        if (!waited) {
            pdl_wait();
            waited = true;
        }
        const bool in = e < per_row;
        const int hc = (in ? e : 0) / a.G, g = (in ? e : 0) - hc * a.G, h = hc / GROUPS, cg = hc - h * GROUPS;
        const int i0 = S / W, i1 = (S + kt - 1) / W, row = (tile & 1) * kTrTile + (node - tile * a.tq) * a.G + g;   // of the pair's 256
        auto slot = [&](int i) { return (int64_t)(2 * (i * a.Hkv + h) + (i == i0 && S > i0 * W ? 1 : 0)); };
        float M = -INFINITY, L = 0.f, o[kTrMergeCols];
#pragma unroll
        for (int x = 0; x < kTrMergeCols; ++x) o[x] = 0.f;
#pragma unroll 1
        for (int i = i0 + sub; i <= i1; i += PG * U) {
            float2 ml[U];
            float4 v[U][NC];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int x = 0; x < NC; ++x) v[u][x] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i + u * PG > i1) continue;
                const int64_t s = slot(i + u * PG);
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(a.ml_part) + s * kTrPair + row);
                const float4 *src = reinterpret_cast<const float4 *>(a.o_part + s * kTrPair * D) + cg * NC * kTrPair + row;
#pragma unroll
                for (int x = 0; x < NC; ++x) v[u][x] = __ldcg(src + x * kTrPair);
            }
            float mn = M;
#pragma unroll
            for (int u = 0; u < U; ++u) mn = fmaxf(mn, ml[u].x);
            const float mz = mn == -INFINITY ? 0.f : mn, f0 = tr_ex2(M - mz);
            L *= f0;
#pragma unroll
            for (int x = 0; x < kTrMergeCols; ++x) o[x] *= f0;
            M = mn;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u * PG > i1) continue;
                const float w = tr_ex2(ml[u].x - mz);
                L = fmaf(w, ml[u].y, L);
#pragma unroll
                for (int x = 0; x < NC; ++x) {
                    o[4 * x] = fmaf(w, v[u][x].x, o[4 * x]);
                    o[4 * x + 1] = fmaf(w, v[u][x].y, o[4 * x + 1]);
                    o[4 * x + 2] = fmaf(w, v[u][x].z, o[4 * x + 2]);
                    o[4 * x + 3] = fmaf(w, v[u][x].w, o[4 * x + 3]);
                }
            }
        }
        if constexpr (PG > 1) {
            // the threads' parts, in their order
            float mn = M;
#pragma unroll
            for (int d = EPW; d < 32; d <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
            const float f0 = tr_ex2(M - (mn == -INFINITY ? 0.f : mn));
            L *= f0;
#pragma unroll
            for (int x = 0; x < kTrMergeCols; ++x) o[x] *= f0;
#pragma unroll
            for (int d = EPW; d < 32; d <<= 1) {
                L += __shfl_xor_sync(0xffffffffu, L, d);
#pragma unroll
                for (int x = 0; x < kTrMergeCols; ++x) o[x] += __shfl_xor_sync(0xffffffffu, o[x], d);
            }
        }
        if (!in || sub != 0) continue;
        const float inv = L != 0.f ? 1.f / L : 0.f;
        uint32_t y[kTrMergeCols / 2];
#pragma unroll
        for (int x = 0; x < kTrMergeCols / 2; ++x) y[x] = L != 0.f ? pack_bf16x2(o[2 * x] * inv, o[2 * x + 1] * inv) : 0u;
        *reinterpret_cast<uint4 *>(a.out + ((int64_t)t * a.Hq + h * a.G + g) * D + cg * kTrMergeCols) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    if (!waited) pdl_wait();
    pdl_launch_dependents();
}

// --------------------------------------------------------------- host side
// Workspace: header, then two slots of partials per unit that shares segments.
struct TrWs {
    size_t ml_off, o_off, total;
};
static TrWs tr_ws(int D)
{
    TrWs w;
    w.ml_off = kWorkspaceHeader;
    w.o_off = align_up(w.ml_off + (size_t)2 * kTrMaxUnits * kTrPair * 8, 256);
    w.total = w.o_off + (size_t)2 * kTrMaxUnits * kTrPair * D * 4;
    return w;
}

// Ranges per kv head: a unit per CTA, or two where that leaves fewer CTAs without one.
static int tr_ranges(int grid, int Hkv)
{
    const int r1 = grid / Hkv, r2 = 2 * grid / Hkv;
    if (r1 < 1) return 1;
    return r2 * Hkv > 2 * r1 * Hkv + grid / 16 ? r2 : r1;
}

template <int D, bool E8>
static pa_status tr_launch(const TreeArgs &a, cudaStream_t st)
{
    auto kern = tree_attn_kernel<D, E8>;
    constexpr int smem = TrCfg<D, E8>::Smem;
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem)) return PA_ERR_CUDA;
    const int grid = num_sms() < kTrMaxCtas ? num_sms() : kTrMaxCtas;
    TreeArgs b = a;
    b.ranges = tr_ranges(grid, a.Hkv);
    if (launch_kernel(kern, dim3(grid), dim3(kTrThreads), smem, st, b) != cudaSuccess) return PA_ERR_CUDA;
    if (b.ranges > 1) {
        // behind this call's own kernel, whose end it waits for: overlapped whatever the mode
        const int64_t elems = (int64_t)a.Hq * (D / kTrMergeCols);
        auto parts = [&](int pg) { return (elems * pg + kTrMergeThreads - 1) / kTrMergeThreads * a.T; };
        const bool few = parts(1) <= grid;
        auto merge = few ? tree_merge_kernel<D, 4> : tree_merge_kernel<D, 1>;
        const int64_t want = parts(few ? 4 : 1);
        const size_t msmem = ((size_t)3 * a.R + 1) * 4;
        if (!ensure_dynamic_smem(reinterpret_cast<const void *>(merge), msmem)) return PA_ERR_CUDA;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(want < 4 * grid ? want : 4 * grid));
        cfg.blockDim = dim3(kTrMergeThreads);
        cfg.dynamicSmemBytes = msmem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, merge, b) != cudaSuccess) return PA_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_tree_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim)
{
    if (n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || n_q_heads % n_kv_heads != 0) return 0;
    return tr_ws(head_dim).total;
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
    // places of all segments (2 x 128 / G nodes over 128 cached tokens) in 32 bits
    if (((int64_t)n_tokens / (2 * (kTrTile / G)) + n_reqs) * (((int64_t)max_ctx + 127) / 128 + kTrMaxPieceCost) >= (int64_t)1 << 30) return PA_ERR_SHAPE;
    if (!workspace) return PA_ERR_NULL;
    if (!aligned256(workspace)) return PA_ERR_ALIGN;
    if (workspace_bytes < pa_tree_workspace_bytes(n_q_heads, s.n_kv_heads, s.head_dim)) return PA_ERR_WORKSPACE;
    if (n_tokens == 0 || n_reqs == 0) return PA_OK;
    if (!q || !k_buf || !v_buf || !qo_indptr || !req_to_token || !req_pool_indices || !seq_lens || !out) return PA_ERR_NULL;
    if (e4m3 && (!k_exp || !v_exp)) return PA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_buf) || !aligned16(v_buf) || !aligned16(out) || !aligned4(qo_indptr) ||
        !aligned4(req_to_token) || !aligned4(req_pool_indices) || !aligned4(seq_lens) || !aligned4(tree_mask))
        return PA_ERR_ALIGN;
    TreeArgs a;
    memset(&a, 0, sizeof a);
    // rows as the tensor core takes them, but an e4m3 cache's V, which is widened, as they are
    const cuuint64_t inner = (cuuint64_t)s.n_kv_heads * s.head_dim, rows = (cuuint64_t)s.n_layers * s.size;
    const cuuint32_t box = e4m3 ? s.head_dim : 64, box16[2] = {box, 16}, box1[2] = {box, 1};
    const int sw = e4m3 ? s.head_dim : 128;
    const cuuint64_t dims[2] = {inner, rows}, strides[1] = {inner};
    if (!encode_tmap_rows(&a.tm_k16, k_buf, !e4m3, inner, rows, box, 16, sw)) return PA_ERR_CUDA;
    if (e4m3 ? !encode_tmap_rows(&a.tm_k1, k_buf, false, inner, rows, box, 1, sw) ||
                   !encode_tmap_u8(&a.tm_v16, v_buf, 2, dims, strides, box16) || !encode_tmap_u8(&a.tm_v1, v_buf, 2, dims, strides, box1)
             : !encode_tmap_rows(&a.tm_v16, v_buf, true, inner, rows, box, 16, sw))
        return PA_ERR_CUDA;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)s.head_dim, (cuuint64_t)n_q_heads, (cuuint64_t)n_tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)s.head_dim * 2, (cuuint64_t)n_q_heads * s.head_dim * 2};
        const cuuint32_t qbox[3] = {64, (cuuint32_t)G, (cuuint32_t)(kTrTile / G)};
        if (!encode_tmap_bf16(&a.tm_q, q, 3, dims, strides, qbox)) return PA_ERR_CUDA;
    }
    const TrWs ws = tr_ws(s.head_dim);
    unsigned char *wp = static_cast<unsigned char *>(workspace);
    a.ml_part = reinterpret_cast<float *>(wp + ws.ml_off);
    a.o_part = reinterpret_cast<float *>(wp + ws.o_off);
    a.layer_row0 = layer_id * s.size;
    a.total_rows = s.n_layers * s.size;
    a.early_meta = early_metadata();
    a.wait_ns = wait_limit_ns();
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
    a.inv_g = 65536 / G + 1;
    // (6 in place of 4: 48 ragged requests over e4m3 146 -> 141 us, 32 over bf16 in pages of one slot 97.8 -> 100)
    a.piece_cost = e4m3 ? kTrMaxPieceCost : 4;
    a.tq = kTrTile / G;
    a.size = s.size;
    a.req_rows = req_rows;
    a.max_ctx = max_ctx;
    a.scale_log2 = (float)(fabs((double)scale) * 1.4426950408889634);
    a.negate = scale < 0.f;
    // a scale of 0 as one that no score survives: a hidden key's minus infinity stays what it is
    if (a.scale_log2 < 0x1p-126f) a.scale_log2 = 0x1p-126f;
    if (e4m3) return s.head_dim == 64 ? tr_launch<64, true>(a, st) : tr_launch<128, true>(a, st);
    return s.head_dim == 64 ? tr_launch<64, false>(a, st) : tr_launch<128, false>(a, st);
}
