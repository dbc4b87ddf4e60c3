// The microscaled 4-bit format (W4_MX4_G32): E2M1 codes in groups of 32 along a
// row, one E8M0 scale byte each. Views, conversions and the launchers of its
// operators.
//
// A code's value is (-1)^s * {0, .5, 1, 1.5, 2, 3, 4, 6}, the scale byte b stands
// for 2^(b - 127), 255 for NaN. A product value times scale has two significant
// bits, so it is exact in bf16 (and in fp32) wherever it is not below the type's
// smallest number: v_cvt_scalef32_pk_bf16_fp4 turns two codes and the scale into
// two bf16 values in one instruction, and the 4-bit matrix instructions take codes
// and scale bytes as they are stored.
#pragma once

#include "common.hpp"
#include "mx4_plan.hpp"

namespace w4 {

struct Mx4Mat {  // [N][K / 2] codes, [N][K / 32] scale bytes, of one matrix or of a stack of them
    const uint8_t* codes;
    const uint8_t* scale;
    int64_t N, K;
};

// 2^(b - 127) as fp32; b = 255 gives infinity, which the conversions below take as NaN
__device__ __forceinline__ float mx4_scale(uint32_t b) {
    return __uint_as_float(max(b << 23, 1u << 22));
}

// Eight codes of one group -> eight bf16 values
__device__ __forceinline__ bf16x8_t mx4_to_bf16(uint32_t w, float scale) {
    uint32_t o[4];
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    return __builtin_bit_cast(bf16x8_t, u32x4_t{o[0], o[1], o[2], o[3]});
}

__device__ __forceinline__ uint16_t to_bf16(float v) {  // nearest even, NaN stays NaN
    const bf16x2_t p = {(__bf16)v, (__bf16)0.f};
    return (uint16_t)__builtin_bit_cast(uint32_t, p);
}

enum : int { kActGeluTanh = 0, kActSilu = 1 };
__device__ __forceinline__ float gated(float g, float u, int act) {
    // silu through exp2: -g log2(e) past 128 gives infinity and the quotient 0
    return (act == kActSilu ? g / (1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g)) : gelu_tanh(g)) * u;
}

// A row of values kept to 16 bits, as two bf16 pieces: each value's nearest bf16 number and that of the rest. Group g of
// 32 values lies at 64 g, its first pieces, then its second ones, so that a product over a row's 2 K pieces is
// one over K values with every group of W taken twice.
__device__ __forceinline__ void store_pieces(uint16_t* row, int64_t k, float v) {
    const uint16_t hi = to_bf16(v);
    const float f = __uint_as_float((uint32_t)hi << 16);
    uint16_t* p = row + k + (k & ~(int64_t)(kMxGroup - 1));
    p[0] = hi;
    p[kMxGroup] = fabsf(f) < INFINITY ? to_bf16(v - f) : (uint16_t)0;
}

// A launch holds under 2^32 threads.
inline bool launchable(int64_t blocks, int threads) { return blocks <= 0xffffffffLL / threads; }

// More LDS than the default 64 KiB for a kernel with static arrays of up to 16 KiB and `bytes` of dynamic LDS, up to
// `most` of them (kMostLds beside such arrays); asked for once on each device.
template <typename F>
inline hipError_t allow_lds(F* kern, int bytes, int most, uint64_t* asked) {
    if (bytes <= (48 << 10)) return hipSuccess;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (__atomic_load_n(asked, __ATOMIC_RELAXED) & bit)) return hipSuccess;
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == hipSuccess && dev < 64) __atomic_fetch_or(asked, bit, __ATOMIC_RELAXED);
    return e;
}

// ---- rows <-> codes (mx4_rows.hip)
hipError_t launch_mx4_quantize(const void* x, bool bf16, int64_t row_stride, int64_t rows, int64_t K,
                               uint8_t* codes, uint8_t* scale, hipStream_t st);
hipError_t launch_mx4_read(const Mx4Mat& q, void* out, bool bf16, int64_t row_stride, hipStream_t st);

// ---- products (mx4_gemm.hip): Y [M][N] = X [M][K] W [N][K]^T
struct Mx4X {           // the left side: bf16 rows, or rows in the same 4 bits
    const uint16_t* x;  // null: codes and scale
    int64_t row_stride;
    const uint8_t* codes;
    const uint8_t* scale;
};
size_t mx4_gemm_workspace(int64_t M, int64_t N, int64_t K, bool x4);
hipError_t launch_mx4_gemm(const Mx4Mat& W, const Mx4X& X, int64_t M, void* Y, bool y_bf16,
                           int64_t y_stride, void* work, hipStream_t st);

// ---- selection of experts (select.hip)
struct SelectArgs {
    const void* logits;
    int64_t row_stride;
    const float* bias;  // or null
    int32_t* ids;
    float* weights;
    int64_t M;
    int E, k, sigmoid, groups, top_groups, best, renormalize;
    float scale;
    int size, share;  // of the launcher: experts a group, log2 of lanes a group
};
hipError_t launch_moe_select(SelectArgs a, bool bf16, hipStream_t st);

// ---- experts' products (mx4_moe.hip)
struct Mx4Moe {
    Mx4Mat gate, up, down;  // stacks
    int E, k, act;
    int64_t M, D, F;
    const uint16_t* x;
    int64_t x_stride;
    const int32_t* ids;
    const float* weights;
    uint16_t* y;
    int64_t y_stride;
};
size_t mx4_moe_workspace(int64_t M, int k, int64_t E, int64_t D, int64_t F);
hipError_t launch_mx4_moe(const Mx4Moe& a, void* work, hipStream_t st);

}  // namespace w4
