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
// Bound: HBM, 2 D bytes read and D written per row and head.
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
    int n_tokens, size, Hkv, block, shift, early_meta;
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
// largest finite magnitude of eight bf16 values
__device__ __forceinline__ float amax8(uint4 w)
{
    float x[8], m = 0.f;
    bf16x8_floats(w, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
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

// GW lanes per (run, head): 32, or a row's D / 16.
template <int D, int GW>
__global__ void __launch_bounds__(256) kv_store_block_kernel(const StoreBlockArgs a)
{
    constexpr int LPR = D / 16, RPP = GW / LPR;     // lanes per row, rows per pass
    constexpr int KEEP = 4;                         // passes whose rows stay in registers
    if (!a.early_meta) pdl_wait();
    const int lane = threadIdx.x & 31, gl = lane % GW;
    const unsigned mask = GW == 32 ? 0xffffffffu : ((1u << GW) - 1u) << (lane - gl);
    const int rr = gl / LPR, c = gl % LPR;
    const int chunk = a.block > RPP ? a.block : RPP;   // tokens per unit
    if (a.early_meta) pdl_wait();
    pdl_launch_dependents();
    for (int64_t u = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / GW; u < a.units;
         u += (int64_t)gridDim.x * blockDim.x / GW) {
        const bool isv = u & 1;
        const int64_t uh = u >> 1;
        const int h = (int)(uh % a.Hkv);
        const int64_t ch = uh / a.Hkv;
        const __nv_bfloat16 *src = (isv ? a.v_new : a.k_new) + (int64_t)h * D + c * 16;
        uint8_t *buf = (isv ? a.v_buf : a.k_buf) + (int64_t)h * D + c * 16;
        uint8_t *exp = isv ? a.v_exp : a.k_exp;
        const int64_t row_elems = (int64_t)a.Hkv * D;
        const int c0 = (int)(ch * chunk), c1 = min(a.n_tokens, c0 + chunk);
        auto block_of = [&](int t) -> int {
            const int s = __ldg(a.loc + t);
            return s < 0 || s >= a.size ? -1 : s >> a.shift;
        };
        int before = c0 > 0 ? block_of(c0 - 1) : -1;
        for (int t0 = c0; t0 < c1;) {
            const int blk = block_of(t0);
            if (blk < 0 || blk == before) {
                if (blk < 0 && gl == 0 && h == 0 && !isv) set_error(a.err, PA_DEVERR_SLOT);
                before = blk;
                ++t0;
                continue;
            }
            before = blk;
            // the run [t0, t1): at most `block` neighbours in this block
            int t1 = t0 + 1;
            while (t1 < a.n_tokens && t1 - t0 < a.block && block_of(t1) == blk) ++t1;
            const int64_t ei = (int64_t)blk * a.Hkv + h;
            const int e_old = exp[ei];
            uint4 keep[KEEP][2];
            float mx = 0.f;
            for (int p = 0, t = t0 + rr; t - rr < t1; ++p, t += RPP) {
                uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
                if (t < t1) {
                    const uint4 *s = reinterpret_cast<const uint4 *>(src + (int64_t)t * row_elems);
                    w0 = __ldg(s);
                    w1 = __ldg(s + 1);
                }
#pragma unroll
                for (int q = 0; q < KEEP; ++q)
                    if (p == q) keep[q][0] = w0, keep[q][1] = w1;
                mx = fmaxf(mx, fmaxf(amax8(w0), amax8(w1)));
            }
#pragma unroll
            for (int o = GW / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(mask, mx, o, GW));
            const int e = max(e_old, block_exponent(mx));
            if (e > e_old && e_old > 0) {
                // earlier rows of the block, rounded again to the larger scale
                const float f = __uint_as_float((uint32_t)max(127 + e_old - e, 0) << 23);
                const int s_lo = blk << a.shift, s_hi = min(a.size, s_lo + a.block);
                for (int s = s_lo + rr; s - rr < s_hi; s += RPP) {
                    bool mine = s < s_hi;
                    for (int t = t0; t < t1; ++t) mine = mine && __ldg(a.loc + t) != s;
                    if (!mine) continue;
                    uint4 *p = reinterpret_cast<uint4 *>(buf + (int64_t)s * row_elems);
                    const uint4 w = *p;
                    *p = make_uint4(requant4(w.x, f), requant4(w.y, f), requant4(w.z, f), requant4(w.w, f));
                }
            }
            const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
            for (int p = 0, t = t0 + rr; t - rr < t1; ++p, t += RPP) {
                if (t >= t1) break;
                uint4 w0, w1;
                if (p < KEEP) {
#pragma unroll
                    for (int q = 0; q < KEEP; ++q)
                        if (p == q) w0 = keep[q][0], w1 = keep[q][1];
                } else {
                    const uint4 *s = reinterpret_cast<const uint4 *>(src + (int64_t)t * row_elems);
                    w0 = __ldg(s);
                    w1 = __ldg(s + 1);
                }
                const uint2 lo = quant8(w0, inv), hi = quant8(w1, inv);
                *reinterpret_cast<uint4 *>(buf + (int64_t)__ldg(a.loc + t) * row_elems) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
            if (gl == 0 && e != e_old) exp[ei] = (uint8_t)e;
            __syncwarp(mask);
            t0 = t1 < c1 ? t1 : c1;
        }
    }
}

__global__ void __launch_bounds__(256) kv_reset_block_kernel(uint8_t *k_exp, uint8_t *v_exp, int n_layers, int n_blocks,
                                                             int Hkv, const int32_t *blocks, int64_t total, int n,
                                                             int32_t *err, int early_meta)
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
    constexpr int RPP = 32 / (D / 16);
    const bool small = a.block < RPP;
    const int chunk = small ? a.block : (a.block > RPP ? a.block : RPP), gw = small ? D / 16 : 32;
    a.units = (((int64_t)a.n_tokens + chunk - 1) / chunk) * a.Hkv * 2;
    int64_t g = (a.units * gw + 255) / 256;
    const int64_t cap = (int64_t)num_sms() * 16;
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
    const int64_t exps = (int64_t)layer_id * ((s.size + block - 1) / block) * s.n_kv_heads;
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
    a.early_meta = early_metadata();
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
                      n_kv_heads, blocks, total, n, error_word, (int)early_metadata()) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
