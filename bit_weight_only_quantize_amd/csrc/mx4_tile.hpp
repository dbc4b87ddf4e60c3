// A 16 x 16 tile of a product with microscaled 4-bit weights, in one wavefront.
#pragma once

#include "mx4.hpp"

namespace w4 {

// acc[r] += sum_k X[4g + r][k] W[c][k] for lane 16g + c, whose pointers are those of row
// c of X and of W. Sixteen bytes of codes are one group, so lane 16g + c takes group 4s +
// g of step s, word j of them in matrix instruction j, and the same k of its row of X.
template <bool X4>
__device__ __forceinline__ void mx4_tile_product(const uint16_t* x, const uint8_t* xc, const uint8_t* xs,
                                                 const uint8_t* wc, const uint8_t* ws, int K, f32x4_t& acc) {
    const int g = (threadIdx.x & 63) >> 4, groups = K / kMxGroup;
    for (int s = 0; s < groups; s += 4) {
        const bool in = s + g < groups;  // past the end: zeros on both sides
        const int at = in ? s + g : 0;
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(wc + 16 * at);
        const float sw = mx4_scale(ws[at]);
        u32x4_t xw;
        float sx = 0.f;
        if constexpr (X4) {
            xw = *reinterpret_cast<const u32x4_t*>(xc + 16 * at);
            sx = mx4_scale(xs[at]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bf16x8_t a, b = mx4_to_bf16(w[j], sw);
            if constexpr (X4) a = mx4_to_bf16(xw[j], sx);
            else a = *reinterpret_cast<const bf16x8_t*>(x + 32 * at + 8 * j);
            if (!in) a = b = bf16x8_t{};
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
        }
    }
}

}  // namespace w4
