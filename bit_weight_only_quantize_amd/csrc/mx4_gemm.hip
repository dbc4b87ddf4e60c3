// Products with microscaled 4-bit weights: Y = X W^T.
#include "mx4_block.hpp"
#include "mx4_few.hpp"
#include "mx4_gemv.hpp"

namespace w4 {

// ---- one row of bf16 (mx4_gemv.hpp): a row of W a wavefront, two loads in flight, 16 wavefronts. 4096 -> 11008
// takes 7.5 us, 11008 -> 4096 7.6; two or four rows or four loads a wavefront, or four or eight wavefronts, 7.4 to 9.3.
constexpr int kGemvWaves = 16;
__global__ __launch_bounds__(64 * kGemvWaves) void mx4_gemv_kernel(Mx4Mat W, const uint16_t* x, void* __restrict__ Y, int y_bf16) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = (int)W.K, V = gemv_vectors(K);
    const int64_t n = (int64_t)blockIdx.x * kGemvWaves + wave, at = min(n, W.N - 1);
    GemvStream<1, 2> f;
    f.groups = K / kMxGroup;
    f.wc[0] = W.codes + at * (K / 2);
    f.ws[0] = W.scale + at * (K / 32);
    float acc[1] = {0.f};
    f.load(0);
    gemv_stage(lds, x, K);
    __syncthreads();
    f.finish(lds, V, acc);
    if (lane == 0 && n < W.N) {
        if (y_bf16) static_cast<uint16_t*>(Y)[n] = to_bf16(acc[0]);
        else static_cast<float*>(Y)[n] = acc[0];
    }
}

static constexpr int64_t kGemvMaxK = 65536;  // x in LDS: 128 KiB
static constexpr int64_t kGemvMaxN = 0xffffffffLL / (64 * kGemvWaves) * kGemvWaves;  // under 2^32 threads

static hipError_t launch_gemv1(const Mx4Mat& W, const uint16_t* x, void* Y, bool y_bf16, hipStream_t st) {
    const int lds = gemv_lds_bytes((int)W.K);
    static uint64_t asked;
    if (const hipError_t e = allow_lds(mx4_gemv_kernel, lds, kMostLds, &asked)) return e;
    hipLaunchKernelGGL(mx4_gemv_kernel, dim3((unsigned)((W.N + kGemvWaves - 1) / kGemvWaves)), dim3(64 * kGemvWaves), lds, st,
                       W, x, Y, y_bf16);
    return hipGetLastError();
}

// ---- up to 16 rows of bf16 (mx4_few.hpp): one workgroup of 16 wavefronts a CU owns consecutive
// tiles of 16 rows of W, `side` of them at a time with 16 / side wavefronts on each one's steps
// (their sums meet in LDS, in a fixed order), over X staged `chunk` steps at a time. One step of codes in
// flight a wavefront: 12.8 us for 13 rows, 5120 -> 13824 (with loads of half lines, at 13.7 then: 14.8 with up to four tiles side by
// side, 15.5 and 15.9 with two and three steps in flight). 80 us (5.1 TB/s) for 2 rows, 5120 -> 152064.
constexpr int kFewWaves = 16;

__global__ __launch_bounds__(64 * kFewWaves) void mx4_few_kernel(Mx4Mat W, Mx4X X, int M, void* __restrict__ Y,
                                                                 int y_bf16, int64_t y_stride, int tiles, int side,
                                                                 int chunk) {
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ f32x4_t sums[kFewWaves][64];
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = (int)W.K, steps = few_steps(K), by = kFewWaves / side;
    const int mine = wave / by, ks = wave % by;
    const int first = (int)((int64_t)tiles * blockIdx.x / gridDim.x);
    const int last = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
    const uint8_t* x = lds + min(c, M - 1) * few_row_bytes(chunk) + 64 * g;
    FewStream<1> f;
    f.groups = K / kMxGroup;
    bool staged = false;
    for (int t0 = first; t0 < last; t0 += side) {
        const bool live = mine < side && t0 + mine < last;
        f.tile(0, [&](int r) {
            const int64_t n = min((int64_t)(t0 + mine) * 16 + r, W.N - 1);
            return Mx4Mat{W.codes + n * (K / 2), W.scale + n * (K / 32), 0, 0};
        });
        FewSums acc[1];
        acc[0].clear();
        for (int s0 = 0; s0 < steps; s0 += chunk) {
            const int end = min(s0 + chunk, steps);
            if (live) f.load(min(s0 + ks, end - 1));
            if (!staged || chunk < steps) {
                __syncthreads();  // the chunk before has been read
                few_stage(lds, [&](int r) { return X.x + r * X.row_stride; }, M, K, s0, chunk);
                __syncthreads();
                staged = true;
            }
            if (live) f.run(x, s0 + ks, by, end, s0, acc);
        }
        __syncthreads();  // the tiles before have been written
        sums[wave][lane] = acc[0].rows();
        __syncthreads();
        if (wave < side && t0 + wave < last) {
            f32x4_t v = sums[wave * by][lane];
            for (int k = 1; k < by; ++k) v += sums[wave * by + k][lane];
            const int64_t col = (int64_t)(t0 + wave) * 16 + few_row(c);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * g + r < M && col < W.N) {
                    const int64_t at = (4 * g + r) * y_stride + col;
                    if (y_bf16) static_cast<uint16_t*>(Y)[at] = to_bf16(v[r]);
                    else static_cast<float*>(Y)[at] = v[r];
                }
        }
    }
}

static hipError_t launch_few(const Mx4Mat& W, const Mx4X& X, int64_t M, void* Y, bool y_bf16, int64_t y_stride,
                             hipStream_t st) {
    const int tiles = (int)((W.N + 15) / 16), steps = few_steps(W.K);
    int chunk = steps;  // all of X in LDS, or as even pieces as there must be
    const int room = kMostLds;
    if (few_row_bytes(steps) * M > room) {
        const int most = (int)((room / M - 16) / (2 * kFewK));
        const int n = (steps + most - 1) / most;
        chunk = (steps + n - 1) / n;
    }
    const int grid = tiles < 256 ? tiles : 256, per = (tiles + grid - 1) / grid;
    const int side = per < 8 ? per : 8, lds = few_row_bytes(chunk) * (int)M;
    auto kern = mx4_few_kernel;
    static uint64_t asked;
    if (const hipError_t e = allow_lds(kern, lds, kMostLds, &asked)) return e;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * kFewWaves), lds, st, W, X, (int)M, Y, y_bf16, y_stride, tiles, side,
                       chunk);
    return hipGetLastError();
}

// ---- up to 16 rows of 4 bits: a workgroup of four wavefronts owns 32 rows of W, each every fourth step
__global__ __launch_bounds__(256) void mx4_few_x4_kernel(Mx4Mat W, Mx4X X, int M, void* __restrict__ Y, int y_bf16,
                                                         int64_t y_stride) {
    constexpr int RT = 2, KS = 4, U = 2;
    __shared__ f32x4_t sums[KS][RT][64];
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
    const int m = min(c, M - 1), groups = (int)W.K / kMxGroup;
    const uint8_t *xc = X.codes + m * (W.K / 2), *xs = X.scale + m * (W.K / 32);
    const uint8_t *wc[RT][2], *ws[RT][2];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t n = min(n0 + 16 * t + 8 * h + c / 2, W.N - 1);
            wc[t][h] = W.codes + n * (W.K / 2);
            ws[t][h] = W.scale + n * (W.K / 32);
        }
    FewSums acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t].clear();
    for (int s = wave; 8 * s < groups; s += U * KS) {
        u32x4_t w[U][RT][2], xv[U][2];  // all loads of U steps first
        uint32_t sw[U][RT][2], sx[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k0 = 8 * (s + u * KS), at = min(k0 + 4 * (lane & 1) + g, groups - 1);
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w[u][t][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(wc[t][h] + 16 * at));
                    sw[u][t][h] = ws[t][h][at];
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // past the end: the last group again, against zeros of X
                const int k = k0 + 4 * i + g, ax = min(k, groups - 1);
                xv[u][i] = *reinterpret_cast<const u32x4_t*>(xc + 16 * ax);
                sx[u][i] = xs[ax];
                if (k >= groups) {
                    xv[u][i] = u32x4_t{0, 0, 0, 0};
                    sx[u][i] = 0;
                }
            }
        }
        const auto wide = [](const u32x4_t& v) { return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; };
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        acc[t].v[h][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wide(xv[u][i]), wide(w[u][t][h]), acc[t].v[h][i], 4, 4, 0, (int)sx[u][i], 0, (int)sw[u][t][h]);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) sums[wave][t][lane] = acc[t].rows();
    __syncthreads();
    if (wave >= RT) return;
    f32x4_t v = sums[0][wave][lane];
#pragma unroll
    for (int k = 1; k < KS; ++k) v += sums[k][wave][lane];
    const int64_t n = n0 + 16 * wave + few_row(c);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * g + r < M && n < W.N) {
            const int64_t at = (4 * g + r) * y_stride + n;
            if (y_bf16) static_cast<uint16_t*>(Y)[at] = to_bf16(v[r]);
            else static_cast<float*>(Y)[at] = v[r];
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
    if (!launchable((tm * tn * a.parts + 7) / 8 * 8, 64 * WM * WN)) return hipErrorInvalidValue;
    a.tiles_n = (int)tn;
    a.tiles = (int)(tm * tn);
    const int lds = kStages * (X4 ? mx4_stage_bytes_x4<BM, BN>() : mx4_stage_bytes<BM, BN>());
    auto kern = mx4_block_kernel<X4, BM, BN, WM, WN>;
    static uint64_t asked;
    if (const hipError_t e = allow_lds(kern, lds, lds, &asked)) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.tiles * a.parts + 7) / 8 * 8)), dim3(64 * WM * WN), lds, st, a);
    if (a.parts > 1)
        hipLaunchKernelGGL((mx4_block_sum_kernel<BM, BN, WM, WN>), dim3((unsigned)(a.tiles * (BM / WM / 32) * (BN / WN / 32))),
                           dim3(64 * WM * WN), 0, st, a);
    return hipGetLastError();
}

size_t mx4_gemm_workspace(int64_t M, int64_t N, int64_t K, bool x4) {
    if (M <= kFewRows) return 0;
    const BlockPlan p = block_plan(M, N, K, x4, true);
    return p.parts > 1 ? p.parts * part_bytes((x4 ? kShapesX4 : kShapes)[p.shape], M, N) : 0;
}

template <bool X4>
static hipError_t launch_blocks(int shape, const BlockArgs& a, hipStream_t st) {
    if constexpr (X4) {
        if (shape == 2) return launch_block<X4, 256, 128, 4, 2>(a, st);
    } else {
        if (shape == 0) return launch_block<X4, 256, 256, 2, 4>(a, st);
        if (shape == 3) return launch_block<X4, 128, 256, 2, 4>(a, st);
    }
    switch (shape) {
        case 1: return launch_block<X4, 256, 192, 4, 2>(a, st);
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
    if (X.x && M == 1 && W.K <= kGemvMaxK && W.N <= kGemvMaxN) return launch_gemv1(W, X.x, Y, y_bf16, st);
    if (X.x) return launch_few(W, X, M, Y, y_bf16, y_stride, st);
    hipLaunchKernelGGL(mx4_few_x4_kernel, dim3((unsigned)((W.N + 31) / 32)), dim3(256), 0, st, W, X, (int)M, Y, y_bf16,
                       y_stride);
    return hipGetLastError();
}

}  // namespace w4
