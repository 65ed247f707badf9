// pa_e4m3_tiles.cuh -- tiles of an e4m3 cache in shared memory as the tensor
// core's operands: rows widened to bf16, and a row of q split into e4m3 terms.
#pragma once

#include "pa_sm100.cuh"

namespace pa {
using namespace sm100;

constexpr int kTileRows = 128;
constexpr int kTileHalf = 128 * 128;    // one 128-row x 128-byte swizzled half tile: 64 columns in bf16

// Widen one e4m3 tile (128 rows of D bytes at a 128-byte pitch at `src`) to bf16 in the
// 128-byte-swizzled K/V stage layout at `dst` (16-byte chunk c of row r at
// (c / 8) halves + r * 128 + ((c % 8) ^ (r % 8)) * 16).  D / 16 lanes share a
// row, each widening one 16-byte chunk into two; every row's bytes are read
// (and the warp synchronised) before any of its bf16 chunks is written, so
// the in-place D = 128 layout is safe.  Exact: e4m3 values are bf16 numbers,
// and so are their products with a block-scaled row's power of two, down to
// bf16's subnormal step of 2^-133 (at e = 1 and 2 an e4m3 subnormal is finer) (BLK:
// exps[r] is row r's exponent byte e, and e << 7 the bf16 number 2^(e - 127);
// 255 marks a position without a row, which becomes zeros).
template <int D, bool BLK = false>
__device__ __forceinline__ void widen_e4m3_tile(uint32_t src, uint32_t dst, int lane, const unsigned char *exps = nullptr,
                                                int row_lo = 0, int row_hi = kTileRows)
{
    constexpr int PITCH = BLK ? D : 128;   // bytes between rows as loaded
    constexpr int LPR = D / 16;     // lanes per row
    constexpr int RPP = 32 / LPR;   // rows per pass of the warp
    constexpr int U = 4;            // passes whose loads are in flight together
    const int rr = lane / LPR, j = lane % LPR;
#pragma unroll 1
    for (int r0 = row_lo; r0 < row_hi; r0 += RPP * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_shared_v4(src + (uint32_t)((r0 + u * RPP + rr) * PITCH + j * 16));
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * RPP + rr;
            const uint32_t ex = BLK ? exps[r] : 0u, sc = ex * 0x00800080u;
            if (BLK && ex == 255u) v[u] = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t mul = BLK && ex == 255u ? 0u : sc;
            auto wide = [&](uint32_t two) -> uint32_t {
                const uint32_t w = e4m3x2_to_bf16x2(two);
                return BLK ? mul_bf16x2(w, mul) : w;
            };
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                // (BLK) the lanes of a row's second half write their odd chunk
                // first: a row's eight lanes then hit all banks once
                const int half = BLK ? hh ^ (j >= LPR / 2) : hh;
                const uint32_t a = half ? v[u].z : v[u].x, b = half ? v[u].w : v[u].y;
                const int c = 2 * j + half;   // bf16 chunk: d = 8 c .. 8 c + 7
                st_shared_v4(dst + (uint32_t)((c >> 3) * kTileHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                             wide(a), wide(a >> 16), wide(b), wide(b >> 16));
            }
        }
        __syncwarp();
    }
}

// Row `row` of a q tile (bf16, 128-byte swizzle) into two e4m3 terms in its
// place: q 2^-k = q1 + q2, k such that the row's largest element is within 448.
// D = 128: q1 in the first half tile's row, q2 in the second's; D = 64: q1 and q2
// side by side in the row.  Every element of at least 2^-9 of the largest is
// exact (a bf16 has 8 significant bits, an e4m3 four), smaller ones are off by
// less than 2^-17 of it: the largest is above 224 2^k, and below 2^-2 2^k the second
// term's step of 2^-9 2^k leaves half of it out.  A row's bytes belong to one thread.
// The terms are those of sg q; returns 2^k.
template <int D>
__device__ __forceinline__ float split_q_row(uint32_t tile, int row, float sg)
{
    constexpr int NC = D / 8;       // 16-byte chunks of the bf16 row
    auto at = [&](int c) { return tile + (uint32_t)((c >> 3) * kTileHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)); };
    uint4 w[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) w[c] = ld_shared_v4(at(c));
    // largest magnitude, as bits (two bf16 per word: NaN and infinity are the largest)
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
        top = __vmaxu2(__vmaxu2(top, __vmaxu2(w[c].x & 0x7FFF7FFFu, w[c].y & 0x7FFF7FFFu)),
                       __vmaxu2(w[c].z & 0x7FFF7FFFu, w[c].w & 0x7FFF7FFFu));
    top = max(top & 0xFFFFu, top >> 16);
    const float mx = __uint_as_float(top << 16);
    // a row with a NaN or an infinity has no softmax: its scale is NaN
    if (top >= 0x7F80u) return NAN;
    auto val = [&](int c, int e) -> float {     // element 8 c + e
        const uint32_t u = e < 2 ? w[c].x : e < 4 ? w[c].y : e < 6 ? w[c].z : w[c].w;
        return __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
    };
    const int k = mx > 0.f ? block_exponent(mx) : 127;
    const float inv = sg * __uint_as_float((uint32_t)(254 - k) << 23);
#pragma unroll
    for (int c = 0; c < NC; c += 2) {
        uint32_t b1[4], b2[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {       // four elements
            b1[g] = b2[g] = 0;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float y0 = val(c + (g >> 1), (g & 1) * 4 + e) * inv;
                const float y1 = val(c + (g >> 1), (g & 1) * 4 + e + 1) * inv;
                const uint32_t q1 = e4m3x2_of(y0, y1);
                float f0, f1;
                e4m3x2_floats(q1, f0, f1);
                b1[g] |= q1 << (8 * e);
                b2[g] |= e4m3x2_of(y0 - f0, y1 - f1) << (8 * e);
            }
        }
        st_shared_v4(at(c / 2), b1[0], b1[1], b1[2], b1[3]);
        st_shared_v4(at(c / 2 + (D == 128 ? 8 : 4)), b2[0], b2[1], b2[2], b2[3]);
    }
    return __uint_as_float((uint32_t)k << 23);
}

}  // namespace pa
