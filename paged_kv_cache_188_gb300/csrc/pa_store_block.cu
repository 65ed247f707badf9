// pa_store_block.cu -- storing into an e4m3 cache with a power-of-two scale
// per (block of slots, kv head), and marking blocks empty.
//
// For the rows x of one call that fall into a block, and one kv head:
//     e  = max(e_old, need), need = the smallest e with amax |x| <= 448 2^(e - 127)
//     byte = e4m3(x 2^(127 - e))                                  (nearest even)
//     the block's other rows, if e > e_old > 0: byte' = e4m3(e4m3(byte) 2^(e_old - e))
// Scales are powers of two, so a row keeps its exact ratio to the scale it is
// rounded at: e4m3 is a floating format, and a finer scale would buy at most
// one bit of range, no precision; raising a scale rounds only what falls among
// the subnormals.
//
// How: the tokens of a call that share a block stand next to each other (the
// caller's contract, as packed prompts and one-token appends do), so a run of
// them is found by comparing neighbours and one group of lanes does a whole
// (run, head): maximum, earlier rows, new rows, exponent.  No atomics, no
// second pass over the tokens, the same bytes on every run.  D / 16 lanes hold
// a row, 16 values each.  Blocks of at least as many rows as a warp holds at once
// (32 / (D/16)) take a warp per run; smaller ones a row's lanes per run.
// Bound: HBM, 2 D bytes read and D written per row and head: 8000 prompt tokens
// into fresh pages, 8 heads of 128, blocks of 16, take 13.8 us with the reset
// before it (the bytes alone 7.2 us); 64 appends into partly filled blocks 2.2 us.
// Larger blocks are latency: one warp does a whole run, and finds the end of one of
// more than 32 rows a row at a time: the 8000 tokens take 14.1 us in blocks of 32,
// 22.7 of 64 and 41.2 of 128 (24.1 us in blocks of 1: an exponent per row and head).
#include <cuda_runtime.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

struct StoreBlockArgs {
    uint8_t *k_buf, *v_buf;            // the layer's rows [size, Hkv, D]
    const __nv_bfloat16 *k_new, *v_new;
    const int32_t *loc;
    uint8_t *k_exp, *v_exp;            // the layer's [n_blocks, Hkv]
    int32_t *err;
    int n_tokens, size, Hkv, block, shift, chunk;
    int64_t units;                     // (chunk of tokens, head, K or V)
};

__device__ __forceinline__ void bf16x8_floats(uint4 w, float *x)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
// magnitudes of eight bf16 values joined to m: two 16-bit integer maxima a word
__device__ __forceinline__ uint32_t join8(uint32_t m, uint4 w)
{
    const uint32_t a = __vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), b = __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu);
    return __vmaxu2(m, __vmaxu2(a, b));
}
// the same without infinities and NaN
__device__ __noinline__ uint32_t join8_finite(uint32_t m, uint4 w)
{
    const uint32_t u[4] = {w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu, w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu};
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = u[i] & 0xFFFFu, hi = u[i] >> 16;
        m = max(m & 0xFFFFu, lo < 0x7F80u ? lo : 0u) | max(m >> 16, hi < 0x7F80u ? hi : 0u) << 16;
    }
    return m;
}
__device__ __forceinline__ uint2 quant8(uint4 w, float inv)
{
    float x[8];
    bf16x8_floats(w, x);
    return make_uint2(e4m3x2_of(x[0] * inv, x[1] * inv) | e4m3x2_of(x[2] * inv, x[3] * inv) << 16,
                      e4m3x2_of(x[4] * inv, x[5] * inv) | e4m3x2_of(x[6] * inv, x[7] * inv) << 16);
}
__device__ __forceinline__ uint32_t requant4(uint32_t w, float f)
{
    float a, b, c, d;
    e4m3x2_floats(w, a, b);
    e4m3x2_floats(w >> 16, c, d);
    return e4m3x2_of(a * f, b * f) | e4m3x2_of(c * f, d * f) << 16;
}

// GW lanes per (run, head): 32, or a row's D / 16.  A unit is a chunk of tokens
// of one head; it does the runs that begin in its chunk.
template <int D, int GW>
__global__ void __launch_bounds__(256, 4) kv_store_block_kernel(const StoreBlockArgs a)
{
    constexpr int LPR = D / 16, RPP = GW / LPR;     // lanes per row, rows per pass
    constexpr int KEEP = 16 / RPP < 2 ? 16 / RPP : 2;   // passes whose rows stay in registers
    const int lane = threadIdx.x & 31, gl = lane % GW;
    const unsigned mask = GW == 32 ? 0xffffffffu : ((1u << GW) - 1u) << (lane - gl);
    const int rr = gl / LPR, c = gl % LPR;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row_elems = (int64_t)a.Hkv * D;
    for (int64_t u = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / GW; u < a.units;
         u += (int64_t)gridDim.x * blockDim.x / GW) {
        const bool isv = u & 1;
        const int64_t uh = u >> 1, ch = uh / a.Hkv;
        const int h = (int)(uh - ch * a.Hkv);
        const __nv_bfloat16 *src = (isv ? a.v_new : a.k_new) + (int64_t)h * D + c * 16;
        uint8_t *buf = (isv ? a.v_buf : a.k_buf) + (int64_t)h * D + c * 16;
        uint8_t *exp = isv ? a.v_exp : a.k_exp;
        const int c0 = (int)(ch * a.chunk), c1 = min(a.n_tokens, c0 + a.chunk);
        auto block_of = [&](int s) -> int { return s < 0 || s >= a.size ? -1 : s >> a.shift; };
        int before = c0 > 0 ? block_of(__ldg(a.loc + c0 - 1)) : -1;
        for (int t0 = c0; t0 < c1;) {
            // lane i of the group: token t0 + i; the tokens that share t0's block
            const int sl = t0 + gl < a.n_tokens ? __ldg(a.loc + t0 + gl) : -1;
            const int mine = block_of(sl), blk = __shfl_sync(mask, mine, 0, GW);
            const unsigned same = __ballot_sync(mask, mine == blk && t0 + gl < a.n_tokens) >> (lane - gl);
            int len = GW == 32 && same == 0xffffffffu ? 32 : __ffs(~same) - 1;
            if (GW < 32 && len > GW) len = GW;
            if (blk < 0 || blk == before) {
                // out of range, or the rest of a run that began before this chunk
                if (blk < 0 && gl == 0 && h == 0 && !isv) set_error(a.err, PA_DEVERR_SLOT);
                before = blk;
                t0 += len;
                continue;
            }
            before = blk;
            if (len == GW) {
                while (t0 + len < a.n_tokens && len < a.block && block_of(__ldg(a.loc + t0 + len)) == blk) ++len;
            }
            len = min(len, a.block);
            const int64_t ei = (int64_t)blk * a.Hkv + h;
            const int e_old = exp[ei];
            // the run's first KEEP * RPP rows stay in registers, requested together (8 rows at D = 128 and 16 at 64 where
            // a warp takes a run, 2 where a row's lanes do); the others are read again after the maximum.  Four passes
            // instead of two, for 16 rows at D = 128, were slower: 14.6 us against 13.8 for the 8000 tokens below
            uint4 keep[KEEP][2];
#pragma unroll
            for (int q = 0; q < KEEP; ++q) {
                const int i = q * RPP + rr;
                keep[q][0] = keep[q][1] = make_uint4(0u, 0u, 0u, 0u);
                if (i < len) {
                    const uint4 *p = reinterpret_cast<const uint4 *>(src + (int64_t)(t0 + i) * row_elems);
                    keep[q][0] = __ldg(p);
                    keep[q][1] = __ldg(p + 1);
                }
            }
            // the run's largest magnitude, as bf16 bits: in nearly every run all are finite
            auto largest = [&](auto join) {
                uint32_t m = 0;
#pragma unroll
                for (int q = 0; q < KEEP; ++q) m = join(join(m, keep[q][0]), keep[q][1]);
                for (int i = KEEP * RPP + rr; i < len; i += RPP) {
                    const uint4 *p = reinterpret_cast<const uint4 *>(src + (int64_t)(t0 + i) * row_elems);
                    const uint4 w0 = __ldg(p), w1 = __ldg(p + 1);
                    m = join(join(m, w0), w1);
                }
                return __reduce_max_sync(mask, max(m & 0xFFFFu, m >> 16));
            };
            uint32_t mb = largest([](uint32_t m, uint4 w) { return join8(m, w); });
            if (mb >= 0x7F80u) mb = largest([](uint32_t m, uint4 w) { return join8_finite(m, w); });
            const float mx = __uint_as_float(mb << 16);
            const int e = max(e_old, block_exponent(mx));
            if (e > e_old && e_old > 0) {
                // earlier rows of the block, rounded again to the larger scale; in: the run's rows, a bit each
                uint32_t in[4] = {0u, 0u, 0u, 0u};
                for (int i = gl; i < len; i += GW) {
                    const int off = __ldg(a.loc + t0 + i) & (a.block - 1);
                    in[0] |= off < 32 ? 1u << off : 0u;
                    in[1] |= off >= 32 && off < 64 ? 1u << (off - 32) : 0u;
                    in[2] |= off >= 64 && off < 96 ? 1u << (off - 64) : 0u;
                    in[3] |= off >= 96 ? 1u << (off - 96) : 0u;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) in[w] = __reduce_or_sync(mask, in[w]);
                const float f = __uint_as_float((uint32_t)max(127 + e_old - e, 0) << 23);
                const int s_lo = blk << a.shift, rows = min(a.size - s_lo, a.block);
#pragma unroll 4
                for (int r = rr; r < rows; r += RPP) {
                    if ((r < 32 ? in[0] : r < 64 ? in[1] : r < 96 ? in[2] : in[3]) >> (r & 31) & 1u) continue;
                    uint4 *p = reinterpret_cast<uint4 *>(buf + (int64_t)(s_lo + r) * row_elems);
                    const uint4 w = *p;
                    *p = make_uint4(requant4(w.x, f), requant4(w.y, f), requant4(w.z, f), requant4(w.w, f));
                }
            }
            const float inv = __uint_as_float(e < 254 ? (uint32_t)(254 - e) << 23 : 1u << 22);   // 2^(127 - e)
            auto put = [&](int i, uint4 w0, uint4 w1, int slot) {
                const uint2 lo = quant8(w0, inv), hi = quant8(w1, inv);
                *reinterpret_cast<uint4 *>(buf + (int64_t)slot * row_elems) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            };
#pragma unroll
            for (int q = 0; q < KEEP; ++q) {
                const int i = q * RPP + rr, slot = __shfl_sync(mask, sl, i < GW ? i : 0, GW);
                if (i < len) put(i, keep[q][0], keep[q][1], i < GW ? slot : __ldg(a.loc + t0 + i));
            }
            for (int i = KEEP * RPP + rr; i < len; i += RPP) {
                const uint4 *p = reinterpret_cast<const uint4 *>(src + (int64_t)(t0 + i) * row_elems);
                put(i, __ldg(p), __ldg(p + 1), __ldg(a.loc + t0 + i));
            }
            if (gl == 0 && e != e_old) exp[ei] = (uint8_t)e;
            __syncwarp(mask);
            t0 += len;
        }
    }
}

__global__ void __launch_bounds__(256) kv_reset_block_kernel(uint8_t *k_exp, uint8_t *v_exp, int n_layers, int n_blocks,
                                                             int Hkv, const int32_t *blocks, int64_t total, int n,
                                                             int32_t *err)
{
    pdl_wait();
    pdl_launch_dependents();
    // element (layer, listed block, head), heads innermost
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t lb = i / Hkv, layer = lb / n;
        const int h = (int)(i - lb * Hkv), b = __ldg(blocks + (lb - layer * n));
        if (b < 0 || b >= n_blocks) {
            if (h == 0 && layer == 0) set_error(err, PA_DEVERR_SLOT);
            continue;
        }
        const int64_t at = (layer * n_blocks + b) * Hkv + h;
        k_exp[at] = 0;
        v_exp[at] = 0;
    }
}

template <int D>
static pa_status launch_store_block(StoreBlockArgs a, cudaStream_t st)
{
    const bool small = a.block < 32 / (D / 16);
    const int gw = small ? D / 16 : 32;
    // one token per unit while that is at most about one wave of warps (a run's
    // other tokens then cost a warp that sees it and leaves: 64 appends take 16
    // runs one after the other else, 15.6 us), then up to a block: a prompt's
    // tokens are mostly not the first of their run
    const int64_t wave = (int64_t)num_sms() * 48 * (32 / gw);
    a.chunk = 1;
    while (a.chunk < a.block && ((int64_t)a.n_tokens + a.chunk - 1) / a.chunk * a.Hkv * 2 > wave) a.chunk *= 2;
    a.units = ((int64_t)a.n_tokens + a.chunk - 1) / a.chunk * a.Hkv * 2;
    int64_t g = (a.units * gw + 255) / 256;
    const int64_t cap = (int64_t)num_sms() * 32;
    if (g > cap) g = cap;
    const cudaError_t rc = small ? launch_kernel(kv_store_block_kernel<D, D / 16>, dim3((unsigned)g), dim3(256), 0, st, a)
                                 : launch_kernel(kv_store_block_kernel<D, 32>, dim3((unsigned)g), dim3(256), 0, st, a);
    if (rc != cudaSuccess) return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_kv_store_fp8_block(void *k_buf, void *v_buf, pa_kv_shape s, int layer_id, const void *k_new,
                                           const void *v_new, const int32_t *loc, int n_tokens, uint8_t *k_exp,
                                           uint8_t *v_exp, int block, int32_t *error_word, cudaStream_t st)
{
    if (n_tokens < 0 || s.n_layers <= 0 || s.size <= 0 || s.n_kv_heads <= 0 || s.head_dim <= 0) return PA_ERR_SHAPE;
    if (layer_id < 0 || layer_id >= s.n_layers || !block_ok(block)) return PA_ERR_SHAPE;
    if (s.head_dim != 64 && s.head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (n_tokens == 0) return PA_OK;
    if (!k_buf || !v_buf || !k_new || !v_new || !loc || !k_exp || !v_exp) return PA_ERR_NULL;
    if (!aligned16(k_buf) || !aligned16(v_buf) || !aligned16(k_new) || !aligned16(v_new) || !aligned4(loc) ||
        (error_word && !aligned4(error_word)))
        return PA_ERR_ALIGN;
    StoreBlockArgs a{};
    const int64_t rows = (int64_t)layer_id * s.size * s.n_kv_heads * s.head_dim;
    const int64_t exps = block_layer_offset(layer_id, s.size, s.n_kv_heads, block);
    a.k_buf = static_cast<uint8_t *>(k_buf) + rows;
    a.v_buf = static_cast<uint8_t *>(v_buf) + rows;
    a.k_new = static_cast<const __nv_bfloat16 *>(k_new);
    a.v_new = static_cast<const __nv_bfloat16 *>(v_new);
    a.loc = loc;
    a.k_exp = k_exp + exps;
    a.v_exp = v_exp + exps;
    a.err = error_word;
    a.n_tokens = n_tokens;
    a.size = s.size;
    a.Hkv = s.n_kv_heads;
    a.block = block;
    while ((1 << a.shift) < block) ++a.shift;
    return s.head_dim == 128 ? launch_store_block<128>(a, st) : launch_store_block<64>(a, st);
}

extern "C" pa_status pa_kv_reset_fp8_block(uint8_t *k_exp, uint8_t *v_exp, int n_layers, int n_blocks, int n_kv_heads,
                                           const int32_t *blocks, int n, int32_t *error_word, cudaStream_t st)
{
    if (n_layers <= 0 || n_blocks <= 0 || n_kv_heads <= 0 || n < 0) return PA_ERR_SHAPE;
    if (n == 0) return PA_OK;
    if (!k_exp || !v_exp || !blocks) return PA_ERR_NULL;
    if (!aligned4(blocks) || (error_word && !aligned4(error_word))) return PA_ERR_ALIGN;
    const int64_t total = (int64_t)n_layers * n * n_kv_heads;
    int64_t g = (total + 255) / 256;
    const int64_t cap = (int64_t)num_sms() * 16;
    if (g > cap) g = cap;
    if (launch_kernel(kv_reset_block_kernel, dim3((unsigned)g), dim3(256), 0, st, k_exp, v_exp, n_layers, n_blocks,
                      n_kv_heads, blocks, total, n, error_word) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
