// Rows of fp32 or bf16 values into the microscaled 4-bit format and back.
//
// Per group of 32 consecutive values: a = max |v|, X = 2^(floor(log2 a) - 2) (the
// largest E2M1 exponent is 2, so the largest value lands in [4, 8)), code =
// E2M1(v / X), nearest with ties to the even code, magnitudes over 6 to 6. floor(log2
// a) is a's exponent field; a division by a power of two is exact, so the codes are
// exactly those of the definition. Groups whose scale would lie under 2^-127 take
// 2^-127; a group with an infinity or a NaN takes the scale byte 255 (NaN) and codes 0.
//
// Eight values a thread, four neighbouring lanes a group, one conversion instruction for two values. Bound by
// memory: 11008 x 4096 fp32 to codes and back to bf16 59 us, 5.0 TB/s (a large copy runs at 5.1); 48 x 2048 takes 2.3 us
// each way, less than its launches' host time.
#include "mx4.hpp"

namespace w4 {

constexpr int kRowsThreads = 256;

template <bool BF16>
__device__ __forceinline__ void load8(const void* x, int64_t at, float (&v)[8]) {
    if constexpr (BF16) {
        const u32x4_t r = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    } else {
        const f32x4_t* p = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(x) + at);
        const f32x4_t a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
}

// Lanes 4j .. 4j + 3 hold a group, eight values each.
template <bool BF16>
__global__ __launch_bounds__(kRowsThreads) void mx4_quantize_kernel(const void* __restrict__ x,
                                                                    int64_t row_stride, int64_t rows,
                                                                    int64_t K, uint8_t* __restrict__ codes,
                                                                    uint8_t* __restrict__ scale) {
    const int64_t per_row = K / 8, n = rows * per_row;
    // (a group's four lanes stay together: n and the grid are multiples of 4)
    for (int64_t i = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kRowsThreads) {
        const int64_t r = i / per_row, c = i - r * per_row;
        float v[8];
        load8<BF16>(x, r * row_stride + 8 * c, v);
        // magnitudes as integers: an infinity or a NaN is the largest of its group
        uint32_t a = 0;
    #pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xF, 0xF, false));  // lane ^ 1
        a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xF, 0xF, false));  // lane ^ 2
        const int e = (int)(a >> 23);
        const bool bad = e == 255;
        const int b = bad ? 255 : max(e - 2, 0);
        const float X = mx4_scale(b);
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], X, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], X, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], X, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], X, 3);
        reinterpret_cast<uint32_t*>(codes)[i] = bad ? 0u : w;
        if ((i & 3) == 0) scale[i >> 2] = (uint8_t)b;
    }
}

template <bool BF16>
__global__ __launch_bounds__(kRowsThreads) void mx4_read_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scale,
                                                                int64_t rows, int64_t K, void* __restrict__ out,
                                                                int64_t row_stride) {
    const int64_t per_row = K / 8, n = rows * per_row;
    for (int64_t i = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kRowsThreads) {
        const int64_t r = i / per_row, c = i - r * per_row;
        const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[i];
        const float X = mx4_scale(scale[i >> 2]);
        if constexpr (BF16) {
            *reinterpret_cast<bf16x8_t*>(static_cast<uint16_t*>(out) + r * row_stride + 8 * c) = mx4_to_bf16(w, X);
        } else {
            const u32x4_t b = __builtin_bit_cast(u32x4_t, mx4_to_bf16(w, X));  // exact in bf16
            f32x4_t* p = reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + r * row_stride + 8 * c);
            f32x4_t lo, hi;
    #pragma unroll
            for (int j = 0; j < 2; ++j) {
                lo[2 * j] = __uint_as_float(b[j] << 16);
                lo[2 * j + 1] = __uint_as_float(b[j] & 0xFFFF0000u);
                hi[2 * j] = __uint_as_float(b[2 + j] << 16);
                hi[2 * j + 1] = __uint_as_float(b[2 + j] & 0xFFFF0000u);
            }
            p[0] = lo;
            p[1] = hi;
        }
    }
}

static int64_t row_blocks(int64_t n) {  // a launch holds under 2^32 threads
    const int64_t b = (n + kRowsThreads - 1) / kRowsThreads;
    return b < (1 << 23) ? b : 1 << 23;
}

hipError_t launch_mx4_quantize(const void* x, bool bf16, int64_t row_stride, int64_t rows, int64_t K,
                               uint8_t* codes, uint8_t* scale, hipStream_t st) {
    const int64_t blocks = row_blocks(rows * (K / 8));
    auto kern = bf16 ? mx4_quantize_kernel<true> : mx4_quantize_kernel<false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kRowsThreads), 0, st, x, row_stride, rows, K, codes,
                       scale);
    return hipGetLastError();
}

hipError_t launch_mx4_read(const Mx4Mat& q, void* out, bool bf16, int64_t row_stride, hipStream_t st) {
    const int64_t blocks = row_blocks(q.N * (q.K / 8));
    auto kern = bf16 ? mx4_read_kernel<true> : mx4_read_kernel<false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kRowsThreads), 0, st, q.codes, q.scale, q.N, q.K, out,
                       row_stride);
    return hipGetLastError();
}

}  // namespace w4
