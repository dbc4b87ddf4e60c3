// Products with microscaled 4-bit weights: Y = X W^T.
#include "mx4_tile.hpp"

namespace w4 {

// One wavefront a tile of 16 rows of X and 16 rows of W.
template <bool X4>
__global__ __launch_bounds__(64) void mx4_gemm_kernel(Mx4Mat W, Mx4X X, int64_t M, void* __restrict__ Y,
                                                      bool y_bf16, int64_t y_stride, int tiles_n) {
    const int lane = threadIdx.x, g = lane >> 4, c = lane & 15;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * 16, n0 = (int64_t)(blockIdx.x % tiles_n) * 16;
    const int64_t m = min(m0 + c, M - 1), n = min(n0 + c, W.N - 1);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    mx4_tile_product<X4>(X4 ? nullptr : X.x + m * X.row_stride, X.codes + m * (W.K / 2),
                         X.scale + m * (W.K / 32), W.codes + n * (W.K / 2), W.scale + n * (W.K / 32), (int)W.K,
                         acc);
    if (n0 + c >= W.N) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t row = m0 + 4 * g + r;
        if (row >= M) break;
        const int64_t at = row * y_stride + n0 + c;
        if (y_bf16) static_cast<uint16_t*>(Y)[at] = to_bf16(acc[r]);
        else static_cast<float*>(Y)[at] = acc[r];
    }
}

size_t mx4_gemm_workspace(int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_mx4_gemm(const Mx4Mat& W, const Mx4X& X, int64_t M, void* Y, bool y_bf16,
                           int64_t y_stride, void*, hipStream_t st) {
    const int64_t tm = (M + 15) / 16, tn = (W.N + 15) / 16;
    auto kern = X.x ? mx4_gemm_kernel<false> : mx4_gemm_kernel<true>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(tm * tn)), dim3(64), 0, st, W, X, M, Y, y_bf16, y_stride, (int)tn);
    return hipGetLastError();
}

}  // namespace w4
