// Products with microscaled 4-bit weights: Y = X W^T.
#include "mx4_block.hpp"
#include "mx4_block_x4.hpp"
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

// ---- many rows: blocks (mx4_block.hpp), K in `parts` pieces where there are few
struct BlockArgs {
    Mx4Mat W;
    Mx4X X;
    int64_t M;
    void* Y;
    int64_t y_stride;
    int y_bf16, tiles_n, tiles, parts;
    float* part;  // parts > 1: fp32 sums of each piece, [tile][piece][wavefront][32 x 32 tile][quarter][lane][4]
};

// The 16 sums of a 32 x 32 tile that a lane holds: D[i][j] is in lane j + 32 ((i / 4) % 2), register
// 4 (i / 8) + i % 4. Single bf16 values, 32 lanes a row (pairs of columns by exchange with the
// neighbouring lane, two rows at a time, took 180 us instead of 167 for 2048 x 11008).
__device__ __forceinline__ void store_tile(const BlockArgs& a, const f32x16_t& v, int64_t m, int64_t n) {
    if (n >= a.W.N) return;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int64_t row = m + 8 * (r >> 2) + (r & 3);
        if (row >= a.M) continue;
        if (a.y_bf16) static_cast<uint16_t*>(a.Y)[row * a.y_stride + n] = to_bf16(v[r]);
        else static_cast<float*>(a.Y)[row * a.y_stride + n] = v[r];
    }
}

// Consecutive tiles go to one XCD (workgroups are dealt to the eight in turn) and run along W
// first: they share their rows of X.
template <bool X4, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx4_block_kernel(BlockArgs a) {
    extern __shared__ __align__(16) uint8_t lds[];
    constexpr int NI = BM / WM / 32, NJ = BN / WN / 32, NW = WM * WN;
    const int units = a.tiles * a.parts, per = (units + 7) / 8;
    const int unit = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
    if ((int)(blockIdx.x / 8) >= per || unit >= units) return;
    const int tile = unit / a.parts, z = unit % a.parts;
    const int64_t m0 = (int64_t)(tile / a.tiles_n) * BM, n0 = (int64_t)(tile % a.tiles_n) * BN;
    const int K = (int)a.W.K, steps = (K + (X4 ? kBlockK4 : kBlockK) - 1) / (X4 ? kBlockK4 : kBlockK);
    const int t0 = (int)((int64_t)steps * z / a.parts), t1 = (int)((int64_t)steps * (z + 1) / a.parts);
    f32x16_t acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16_t{};
    const auto wcol = [&](int c) {
        const int64_t n = min(n0 + c, a.W.N - 1);
        return Mx4Mat{a.W.codes + n * (K / 2), a.W.scale + n * (K / 32), 0, 0};
    };
    if constexpr (X4) {
        const auto xrow = [&](int r) {
            const int64_t m = min(m0 + r, a.M - 1);
            return Mx4Mat{a.X.codes + m * (K / 2), a.X.scale + m * (K / 32), 0, 0};
        };
        mx4_block_product_x4<BM, BN, WM, WN>(lds, xrow, wcol, K, t0, t1, acc);
    } else {
        const auto xrow = [&](int r) { return a.X.x + min(m0 + r, a.M - 1) * a.X.row_stride; };
        mx4_block_product<BM, BN, WM, WN>(lds, xrow, wcol, K, t0, t1, acc);
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (a.parts > 1) {
        f32x4_t* p = reinterpret_cast<f32x4_t*>(a.part) + ((int64_t)unit * NW + wave) * (NI * NJ * 256) + lane;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16_t& v = acc[i][j];
                    p[((i * NJ + j) * 4 + q) * 64] = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                }
        return;
    }
    const int64_t m = m0 + (wave / WN) * (BM / WM) + 4 * (lane >> 5), n = n0 + (wave % WN) * (BN / WN) + (lane & 31);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) store_tile(a, acc[i][j], m + 32 * i, n + 32 * j);
}

// Adds up the pieces of one 32 x 32 tile of every wavefront, in their order.
template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void mx4_block_sum_kernel(BlockArgs a) {
    constexpr int NI = BM / WM / 32, NJ = BN / WN / 32, NW = WM * WN;
    const int tile = blockIdx.x / (NI * NJ), b = blockIdx.x % (NI * NJ);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(a.part) +
                       ((int64_t)tile * a.parts * NW + wave) * (NI * NJ * 256) + b * 256 + lane;
    f32x16_t v = {};
    for (int z = 0; z < a.parts; ++z)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4_t u = p[(int64_t)z * NW * (NI * NJ * 256) + q * 64];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * q + r] += u[r];
        }
    const int64_t m0 = (int64_t)(tile / a.tiles_n) * BM, n0 = (int64_t)(tile % a.tiles_n) * BN;
    store_tile(a, v, m0 + (wave / WN) * (BM / WM) + 32 * (b / NJ) + 4 * (lane >> 5),
               n0 + (wave % WN) * (BN / WN) + 32 * (b % NJ) + (lane & 31));
}

template <bool X4, int BM, int BN, int WM, int WN>
static hipError_t launch_block(BlockArgs a, hipStream_t st) {
    const int64_t tm = (a.M + BM - 1) / BM, tn = (a.W.N + BN - 1) / BN;
    if (tm * tn * a.parts > 0x7fffffff - 8) return hipErrorInvalidValue;
    a.tiles_n = (int)tn;
    a.tiles = (int)(tm * tn);
    const int lds = kStages * (X4 ? mx4_stage_bytes_x4<BM, BN>() : mx4_stage_bytes<BM, BN>());
    auto kern = mx4_block_kernel<X4, BM, BN, WM, WN>;
    (void)hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.tiles * a.parts + 7) / 8 * 8)), dim3(64 * WM * WN), lds, st, a);
    if (a.parts > 1)
        hipLaunchKernelGGL((mx4_block_sum_kernel<BM, BN, WM, WN>), dim3((unsigned)(a.tiles * (BM / WM / 32) * (BN / WN / 32))),
                           dim3(64 * WM * WN), 0, st, a);
    return hipGetLastError();
}

// Which block, and in how many pieces of K: the least estimated time. A workgroup's time is its
// steps times the step's measured time with all slots taken (us; 4096 x 12288 rows, K = 4096: 330 us
// with 256 x 256, 361, 400, 385, 395 and 512 with the others, in this order), plus its start and end;
// rounds of workgroups follow one another. Pieces cost a launch and their sums' way through
// memory (2048 x 11008 in 344 blocks of 256 x 256 on 256 slots takes 192 us, in 464 of 256 x 192 171).
struct BlockShape {
    int bm, bn, slots;  // slots: workgroups that the GPU holds at once
    double step, head;
};
static const BlockShape kShapes[] = {
    {256, 256, 256, 1.60, 6}, {256, 192, 256, 1.33, 6}, {256, 128, 256, 1.02, 5}, {128, 256, 256, 0.98, 5},
    {128, 128, 512, 1.00, 5}, {64, 128, 768, 0.97, 5},
};
// 4 bits on both sides: steps of 128 k (4096 x 12288 rows, K = 16384: 560 us with 256 x 192, then 651,
// 731, 716 and 1093). 256 x 256 needs more registers than there are and takes 632.
static const BlockShape kShapesX4[] = {
    {0, 0, 0, 0, 0}, {256, 192, 256, 1.09, 6}, {256, 128, 256, 0.85, 5}, {128, 256, 256, 0.95, 4},
    {128, 128, 512, 0.93, 3}, {64, 128, 768, 1.07, 2},
};
struct BlockPlan {
    int shape, parts;
};
static size_t part_bytes(const BlockShape& s, int64_t M, int64_t N) {
    return (size_t)((M + s.bm - 1) / s.bm * s.bm) * ((N + s.bn - 1) / s.bn * s.bn) * 4;
}
static BlockPlan block_plan(int64_t M, int64_t N, int64_t K, bool x4, bool can_split) {
    const BlockShape* shapes = x4 ? kShapesX4 : kShapes;
    BlockPlan best = {0, 1};
    double least = 1e30;
    const int64_t steps = x4 ? (K + kBlockK4 - 1) / kBlockK4 : (K + kBlockK - 1) / kBlockK;
    for (int i = x4 ? 1 : 0; i < 6; ++i) {
        const BlockShape& s = shapes[i];
        const int64_t tiles = ((M + s.bm - 1) / s.bm) * ((N + s.bn - 1) / s.bn);
        for (int p = 1; p <= 16 && 4 * p <= steps + 3; ++p) {
            if (p > 1 && (!can_split || tiles * p > s.slots)) break;
            const double rounds = (double)((tiles * p + s.slots - 1) / s.slots);
            // workgroups that have a CU to themselves take two thirds of the time of two, half that of three
            const double alone = s.slots > 256 && tiles * p <= 256 ? 0.6 : 1.0;
            double t = rounds * ((double)((steps + p - 1) / p) * s.step * alone + s.head);
            if (p > 1) t += 4 + 2.0 * p * part_bytes(s, M, N) / 5e6;
            if (t < least) {
                least = t;
                best = {i, p};
            }
        }
    }
    return best;
}

static constexpr int64_t kFewRows = 16;

size_t mx4_gemm_workspace(int64_t M, int64_t N, int64_t K, bool x4) {
    if (M <= kFewRows) return 0;
    const BlockPlan p = block_plan(M, N, K, x4, true);
    return p.parts > 1 ? p.parts * part_bytes(kShapes[p.shape], M, N) : 0;
}

template <bool X4>
static hipError_t launch_blocks(int shape, const BlockArgs& a, hipStream_t st) {
    if constexpr (!X4)
        if (shape == 0) return launch_block<X4, 256, 256, 2, 4>(a, st);
    switch (shape) {
        case 1: return launch_block<X4, 256, 192, 4, 2>(a, st);
        case 2: return launch_block<X4, 256, 128, 4, 2>(a, st);
        case 3: return launch_block<X4, 128, 256, 2, 4>(a, st);
        case 4: return launch_block<X4, 128, 128, 2, 2>(a, st);
        default: return launch_block<X4, 64, 128, 1, 4>(a, st);
    }
}

hipError_t launch_mx4_gemm(const Mx4Mat& W, const Mx4X& X, int64_t M, void* Y, bool y_bf16,
                           int64_t y_stride, void* work, hipStream_t st) {
    if (M > kFewRows) {
        const BlockPlan p = block_plan(M, W.N, W.K, !X.x, work != nullptr);
        const BlockArgs a = {W, X, M, Y, y_stride, y_bf16, 0, 0, p.parts, (float*)work};
        return X.x ? launch_blocks<false>(p.shape, a, st) : launch_blocks<true>(p.shape, a, st);
    }
    const int64_t tm = (M + 15) / 16, tn = (W.N + 15) / 16;
    auto kern = X.x ? mx4_gemm_kernel<false> : mx4_gemm_kernel<true>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(tm * tn)), dim3(64), 0, st, W, X, M, Y, y_bf16, y_stride, (int)tn);
    return hipGetLastError();
}

}  // namespace w4
