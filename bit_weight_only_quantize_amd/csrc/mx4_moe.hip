// The gated FFN of each token's chosen experts, with microscaled 4-bit weights:
//   y[m] = sum_j weights[m][j] W_down[e] h,  h = act(W_gate[e] x[m]) * (W_up[e] x[m]),  e = ids[m][j].
//
// h is kept to 16 bits, two bf16 pieces a value, which the down product multiplies one after the other: with a single
// piece its rounding was most of what results were off by (2.4e-3 of 64 bits in norm, 1.7e-3 with two, which is the
// rounding of y). The second piece took 4096 tokens from 520 us to 604 (645 with every operand of W unpacked for each piece), 61
// tokens from 112 to 116, one token nothing.
// Pair p = m k + j. Three ways, by the number of pairs and of pairs an expert gets:
//   * few pairs (kDirectPairs): each pair's gate and up rows by the one-row kernel, then a token's
//     y in one pass over its experts' down rows. Two launches, no sorting.
//   * otherwise the pairs are sorted by expert (mx4_sort_kernel) into tiles of rows of one expert, so
//     that an expert's weights are read once for a tile; the gate/up product writes h in sorted order,
//     the down product each pair's part of y in fp32 (parts in bf16 took 16-bit results from 2.4e-3 off to
//     2.9e-3), and the last launch adds up a token's k parts in their order. Tiles of 8 or 16 rows stream
//     the weights (mx4_few.hpp), tiles of 64 or 128 are blocks on the matrix cores (mx4_block.hpp).
// A pair's place among its expert's is not fixed (it comes from an integer atomic), but its
// results do not depend on it.
#include "mx4_few.hpp"
#include "mx4_gemv.hpp"

namespace w4 {

struct Mx4MoeWork {  // byte offsets
    size_t tiles, pairs, place, h, part, total;
    int64_t slots;
};
static Mx4MoeWork moe_layout(int64_t M, int k, int64_t E, int64_t D, int64_t F) {
    const int64_t P = M * k;
    const MoeWay way = moe_way(M, k, E, D, F);
    Mx4MoeWork L;
    const auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    L.slots = way.direct ? 0 : (E + P / way.rows + 7) / 8 * 8;
    L.tiles = 0;
    L.pairs = up((size_t)L.slots * 16);
    L.place = L.pairs + (way.direct ? 0 : up((size_t)P * 4));
    L.h = L.place + (way.direct ? 0 : up((size_t)P * 4));
    L.part = L.h + up((size_t)P * F * 4);
    L.total = L.part + (size_t)P * D * 4;
    return L;
}
size_t mx4_moe_workspace(int64_t M, int k, int64_t E, int64_t D, int64_t F) {
    return moe_layout(M, k, E, D, F).total;
}

// ---------------------------------------------------------------- few pairs
constexpr int kDirectWaves = 8;

// Pieces of h of pair blockIdx.y: a gate and an up row a wavefront
__global__ __launch_bounds__(64 * kDirectWaves) void mx4_gate_up_one_kernel(Mx4Moe a, uint16_t* __restrict__ h) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int p = blockIdx.y, e = a.ids[p], D = (int)a.D;
    if (e < 0 || e >= a.E) return;
    const int64_t f = (int64_t)blockIdx.x * kDirectWaves + wave, row = (int64_t)e * a.F + min(f, a.F - 1);
    GemvStream<2, 1> s;
    s.groups = D / kMxGroup;
    s.wc[0] = a.gate.codes + row * (D / 2);
    s.ws[0] = a.gate.scale + row * (D / 32);
    s.wc[1] = a.up.codes + row * (D / 2);
    s.ws[1] = a.up.scale + row * (D / 32);
    float acc[2] = {0.f, 0.f};
    s.load(0);
    gemv_stage(lds, a.x + (p / a.k) * a.x_stride, D);
    __syncthreads();
    s.finish(lds, gemv_vectors(D), acc);
    if (lane == 0 && f < a.F) store_pieces(h + 2 * p * a.F, f, gated(acc[0], acc[1], a.act));
}

// y[m][d] of token blockIdx.y, a wavefront a d: the rows d of the token's k experts as one row of k F
// values, against the token's k rows of h, each vector's product times its expert's weight
__global__ __launch_bounds__(64 * kDirectWaves) void mx4_down_one_kernel(Mx4Moe a, const uint16_t* h) {
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ int ids[32];
    __shared__ float wts[32];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m = blockIdx.y;
    const int F = (int)a.F, G = F / kMxGroup, all = a.k * G, V = gemv_vectors(a.k * F);
    const int64_t d = (int64_t)blockIdx.x * kDirectWaves + wave, row = min(d, a.D - 1);
    if ((int)threadIdx.x < a.k) {
        const int e = a.ids[m * a.k + threadIdx.x];
        const bool in = e >= 0 && e < a.E;
        ids[threadIdx.x] = in ? e : -1;
        wts[threadIdx.x] = in ? a.weights[m * a.k + threadIdx.x] : 0.f;
    }
    // h of a slot without an expert was never written: its vectors are left out below
    gemv_stage<2>(lds, h + 2 * m * a.k * F, a.k * F);
    __syncthreads();
    float acc = 0.f;
    constexpr int U = 4;
    for (int v0 = 0; v0 < V; v0 += 64 * U) {
        u32x4_t w[U];
        uint32_t sc[U];
        float wt[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = min(v0 + 64 * u + lane, all - 1), j = v / G, g = v - j * G, e = ids[j];
            in[u] = v0 + 64 * u + lane < all && e >= 0;
            const int64_t at = (int64_t)max(e, 0) * a.D + row;
            w[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(a.down.codes + at * (F / 2) + 16 * g));
            sc[u] = a.down.scale[at * (F / 32) + g];
            wt[u] = wts[j];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v0 + 64 * u >= V) break;
            const float f = mx4_scale(sc[u]);
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4_t b = __builtin_bit_cast(u32x4_t, mx4_to_bf16(w[u][j], f));
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(lds + (j + 4 * s) * (16 * V) + (v0 + 64 * u + lane) * 16);
#pragma unroll
                    for (int q = 0; q < 4; ++q) dot = dot2_bf16(b[q], x[q], dot);
                }
            }
            if (in[u]) acc = fmaf(wt[u], dot, acc);
        }
    }
    acc = group_sum<64>(acc);
    if (lane == 0 && d < a.D) a.y[m * a.y_stride + d] = to_bf16(acc);
}

// ---------------------------------------------------------------- sorting
// Workgroup e: how many pairs lower experts have (o) and how many this one (c), its pairs at sorted places
// o .. o + c - 1, and its tiles {expert, first place, pairs} at slots from o / rows + e on: one more than
// its whole tiles at most, so the slots of different experts never meet; unused ones are {-1}.
// place[p]: the pair's place, -1 for an id outside [0, E).
constexpr int kSortThreads = 1024;
__global__ __launch_bounds__(kSortThreads) void mx4_sort_kernel(const int32_t* __restrict__ ids, int P, int E, int rows,
                                                                int slots, int4* __restrict__ tiles,
                                                                int32_t* __restrict__ pairs, int32_t* __restrict__ place) {
    __shared__ int low[kSortThreads / 64], same[kSortThreads / 64], next;
    const int e = blockIdx.x, t = threadIdx.x;
    const auto four = [&](int p) {  // ids p .. p + 3; behind the last, one that is no expert's and has no place
        if (p + 4 <= P) return *reinterpret_cast<const int4*>(ids + p);
        int4 v = {INT32_MIN, INT32_MIN, INT32_MIN, INT32_MIN};
        if (p < P) v.x = ids[p];
        if (p + 1 < P) v.y = ids[p + 1];
        if (p + 2 < P) v.z = ids[p + 2];
        return v;
    };
    int lo = 0, eq = 0;
    for (int p = 4 * t; p < P; p += 4 * kSortThreads) {
        const int4 v = four(p);
        lo += (v.x >= 0 && v.x < e) + (v.y >= 0 && v.y < e) + (v.z >= 0 && v.z < e) + (v.w >= 0 && v.w < e);
        eq += (v.x == e) + (v.y == e) + (v.z == e) + (v.w == e);
    }
    for (int o = 32; o >= 1; o >>= 1) {
        lo += __shfl_xor(lo, o, 64);
        eq += __shfl_xor(eq, o, 64);
    }
    if ((t & 63) == 0) {
        low[t >> 6] = lo;
        same[t >> 6] = eq;
    }
    if (t == 0) next = 0;
    __syncthreads();
    int off = 0, cnt = 0;
#pragma unroll
    for (int i = 0; i < kSortThreads / 64; ++i) {
        off += low[i];
        cnt += same[i];
    }
    const int base = off / rows + e, end = e + 1 < E ? (off + cnt) / rows + e + 1 : slots;
    for (int i = base + t; i < end; i += kSortThreads) {
        const int first = (i - base) * rows;
        tiles[i] = first < cnt ? make_int4(e, off + first, min(rows, cnt - first), 0) : make_int4(-1, 0, 0, 0);
    }
    if (cnt == 0 && e > 0) return;  // whole workgroup
    const auto put = [&](int p, int v) {
        if (v == e) {
            const int at = off + atomicAdd(&next, 1);
            pairs[at] = p;
            place[p] = at;
        } else if (e == 0 && p < P && (v < 0 || v >= E)) {
            place[p] = -1;
        }
    };
    for (int p = 4 * t; p < P; p += 4 * kSortThreads) {
        const int4 v = four(p);
        put(p, v.x);
        put(p + 1, v.y);
        put(p + 2, v.z);
        put(p + 3, v.w);
    }
}

// The tile and the column block of workgroup b: tiles are dealt to the eight XCDs in turn, and a tile's nb
// column blocks, which share its rows, follow one another on its XCD.
__device__ __forceinline__ int4 moe_tile(const int4* tiles, int nb, int& block) {
    const int b = blockIdx.x, i = b / 8;
    block = i % nb;
    const int4 t = tiles[i / nb * 8 + b % 8];
    return make_int4(__builtin_amdgcn_readfirstlane(t.x), __builtin_amdgcn_readfirstlane(t.y),
                     __builtin_amdgcn_readfirstlane(t.z), 0);
}

// ---------------------------------------------------------------- tiles of up to 16 rows
// Wavefront w takes 16 gate rows and the same 16 up rows (or 16 down rows) and all of K. 61 tokens over 128
// experts of 768 x 2048, top 8: gate/up 73 us (209 MB; 2, 6 or 8 wavefronts 75 to 81), down 29 (105 MB; 25 with one piece of h).
template <bool GU, int NW>
__global__ __launch_bounds__(64 * NW) void mx4_moe_few_kernel(Mx4Moe a, const int4* __restrict__ tiles,
                                                              const int32_t* __restrict__ pairs, uint16_t* h,
                                                              float* __restrict__ part, int nb) {
    extern __shared__ __align__(16) uint8_t lds[];
    constexpr int RT = GU ? 2 : 1;
    int block;
    const int4 t = moe_tile(tiles, nb, block);
    if (t.x < 0) return;
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t N = GU ? a.F : a.D, n0 = ((int64_t)block * NW + wave) * 16;
    constexpr int P = GU ? 1 : 2;  // pieces of a value of x or h
    const int K = (int)(GU ? a.D : a.F), steps = few_steps(K);
    FewStream<RT> f;
    f.groups = K / kMxGroup;
#pragma unroll
    for (int i = 0; i < RT; ++i)
        f.tile(i, [&](int r) {
            const Mx4Mat& w = !GU ? a.down : i ? a.up : a.gate;
            const int64_t row = (int64_t)t.x * N + min(n0 + r, N - 1);
            return Mx4Mat{w.codes + row * (K / 2), w.scale + row * (K / 32), 0, 0};
        });
    FewSums acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i].clear();
    f.load(0);
    few_stage(lds, [&](int r) { return GU ? a.x + (pairs[t.y + r] / a.k) * a.x_stride : h + (int64_t)(t.y + r) * (P * K); }, t.z,
              P * K, 0, P * steps);
    __syncthreads();
    if (n0 >= N) return;
    f.template run<P>(lds + min(c, t.z - 1) * few_row_bytes(P * steps) + 64 * P * g, 0, 1, steps, 0, acc);
    const int64_t n = n0 + few_row(c);
    if (n >= N) return;
    const f32x4_t v = acc[0].rows(), u = acc[RT - 1].rows();
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * g + r < t.z) {
            const int64_t row = t.y + 4 * g + r;
            if constexpr (GU) store_pieces(h + row * 2 * N, n, gated(v[r], u[r], a.act));
            else part[row * N + n] = v[r];
        }
}

// ---------------------------------------------------------------- blocks
// A wavefront's columns are pairs of 32 gate and the same 32 up rows, so that it holds both sums of an h.
template <bool GU, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx4_moe_block_kernel(Mx4Moe a, const int4* __restrict__ tiles,
                                                                        const int32_t* __restrict__ pairs, uint16_t* h,
                                                                        float* __restrict__ part, int nb) {
    extern __shared__ __align__(16) uint8_t lds[];
    constexpr int NI = BM / WM / 32, NJ = BN / WN / 32, COLS = GU ? BN / 2 : BN;
    static_assert(NJ == 2, "a gate and an up tile");
    int block;
    const int4 t = moe_tile(tiles, nb, block);
    if (t.x < 0) return;
    const int64_t N = GU ? a.F : a.D, n0 = (int64_t)block * COLS;
    const int K = (int)(GU ? a.D : a.F);
    f32x16_t acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16_t{};
    const auto xrow = [&](int r) -> const uint16_t* {
        const int p = t.y + min(r, t.z - 1);
        return GU ? a.x + (pairs[p] / a.k) * a.x_stride : h + (int64_t)p * (2 * K);
    };
    const auto wcol = [&](int c) {
        const Mx4Mat& w = !GU ? a.down : (c / 32) & 1 ? a.up : a.gate;
        const int64_t n = (int64_t)t.x * N + min(n0 + (GU ? c / 64 * 32 + c % 32 : c), N - 1);
        return Mx4Mat{w.codes + n * (K / 2), w.scale + n * (K / 32), 0, 0};
    };
    mx4_block_product<BM, BN, WM, WN, !GU>(lds, xrow, wcol, K, 0, GU ? (K + kBlockK - 1) / kBlockK : K / kMxGroup, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = (wave / WN) * (BM / WM) + 4 * (lane >> 5);
    const int64_t n = n0 + (wave % WN) * (GU ? 32 : 64) + (lane & 31);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int m = row + 32 * i + 8 * (r >> 2) + (r & 3);
            if (m >= t.z) continue;
            const int64_t at = (int64_t)(t.y + m) * N + n;
            if constexpr (GU) {
                if (n < N) store_pieces(h + (int64_t)(t.y + m) * 2 * N, n, gated(acc[i][0][r], acc[i][1][r], a.act));
            } else {
                if (n < N) part[at] = acc[i][0][r];
                if (n + 32 < N) part[at + 32] = acc[i][1][r];
            }
        }
}

// ---------------------------------------------------------------- a token's parts
constexpr int64_t kCombineMost = 1 << 23;  // tokens of a launch, 256 threads each
__global__ __launch_bounds__(256) void mx4_combine_kernel(Mx4Moe a, const int32_t* __restrict__ place,
                                                          const float* __restrict__ part) {
    const int64_t m = blockIdx.x;
    for (int64_t d = 8 * threadIdx.x; d < a.D; d += 8 * 256) {
        float y[8] = {};
        for (int j = 0; j < a.k; ++j) {
            const int p = place[m * a.k + j];
            if (p < 0) continue;
            const float w = a.weights[m * a.k + j];
            const f32x4_t* v = reinterpret_cast<const f32x4_t*>(part + (int64_t)p * a.D + d);
            const f32x4_t lo = v[0], hi = v[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = fmaf(w, lo[i], y[i]);
                y[4 + i] = fmaf(w, hi[i], y[4 + i]);
            }
        }
        uint16_t* out = a.y + m * a.y_stride + d;
        if ((a.y_stride & 7) == 0) {
            bf16x8_t o;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = (__bf16)y[i];
            *reinterpret_cast<bf16x8_t*>(out) = o;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = to_bf16(y[i]);
        }
    }
}

template <bool GU, int BM, int BN, int WM, int WN>
static hipError_t launch_moe_block(const Mx4Moe& a, int64_t slots, const int4* tiles, const int32_t* pairs, uint16_t* h,
                                   float* part, hipStream_t st) {
    const int64_t N = GU ? a.F : a.D;
    const int lds = kStages * mx4_stage_bytes<BM, BN, !GU>(), cols = GU ? BN / 2 : BN, nb = (int)((N + cols - 1) / cols);
    auto kern = mx4_moe_block_kernel<GU, BM, BN, WM, WN>;
    static uint64_t asked;
    if (const hipError_t e = allow_lds(kern, lds, lds, &asked)) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)(slots * nb)), dim3(64 * WM * WN), lds, st, a, tiles, pairs, h, part, nb);
    return hipGetLastError();
}

hipError_t launch_mx4_moe(const Mx4Moe& a, void* work, hipStream_t st) {
    const Mx4MoeWork L = moe_layout(a.M, a.k, a.E, a.D, a.F);
    const MoeWay way = moe_way(a.M, a.k, a.E, a.D, a.F);
    // columns of a workgroup of the gate/up and of the down product, and threads, as launched below
    const int gu_cols = way.rows == 64 ? 128 : 64, down_cols = 2 * gu_cols, down_threads = way.rows <= 16 ? 512 : 256;
    if (!launchable(L.slots * ((a.F + gu_cols - 1) / gu_cols), 256) ||
        !launchable(L.slots * ((a.D + down_cols - 1) / down_cols), down_threads))
        return hipErrorInvalidValue;  // before the first launch
    uint8_t* base = (uint8_t*)work;
    int4* tiles = (int4*)(base + L.tiles);
    int32_t* pairs = (int32_t*)(base + L.pairs);
    int32_t* place = (int32_t*)(base + L.place);
    uint16_t* h = (uint16_t*)(base + L.h);
    float* part = (float*)(base + L.part);
    if (way.direct) {
        const dim3 gu((unsigned)((a.F + kDirectWaves - 1) / kDirectWaves), (unsigned)(a.M * a.k));
        const dim3 gd((unsigned)((a.D + kDirectWaves - 1) / kDirectWaves), (unsigned)a.M);
        const int lg = gemv_lds_bytes((int)a.D), ld = 2 * gemv_lds_bytes((int)(a.k * a.F));
        static uint64_t asked_gu, asked_down;
        if (const hipError_t e = allow_lds(mx4_gate_up_one_kernel, lg, kMostLds, &asked_gu)) return e;
        if (const hipError_t e = allow_lds(mx4_down_one_kernel, ld, kMostLds, &asked_down)) return e;
        hipLaunchKernelGGL(mx4_gate_up_one_kernel, gu, dim3(64 * kDirectWaves), lg, st, a, h);
        hipLaunchKernelGGL(mx4_down_one_kernel, gd, dim3(64 * kDirectWaves), ld, st, a, h);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(mx4_sort_kernel, dim3((unsigned)a.E), dim3(kSortThreads), 0, st, a.ids, (int)(a.M * a.k), a.E, way.rows,
                       (int)L.slots, tiles, pairs, place);
    if (way.rows <= 16) {
        constexpr int GW = 4, DW = 8;
        const int nf = (int)((a.F + 16 * GW - 1) / (16 * GW)), nd = (int)((a.D + 16 * DW - 1) / (16 * DW));
        const int lg = way.rows * few_row_bytes(few_steps(a.D)), ld = way.rows * few_row_bytes(2 * few_steps(a.F));
        auto gu = mx4_moe_few_kernel<true, GW>;
        auto down = mx4_moe_few_kernel<false, DW>;
        static uint64_t asked_gu, asked_down;
        if (const hipError_t e = allow_lds(gu, lg, kMostLds, &asked_gu)) return e;
        if (const hipError_t e = allow_lds(down, ld, kMostLds, &asked_down)) return e;
        hipLaunchKernelGGL(gu, dim3((unsigned)(L.slots * nf)), dim3(64 * GW), lg, st, a, tiles, pairs, h, part, nf);
        hipLaunchKernelGGL(down, dim3((unsigned)(L.slots * nd)), dim3(64 * DW), ld, st, a, tiles, pairs, h, part, nd);
    } else {
        const auto blocks = [&](auto gu, auto down) {
            const hipError_t e = gu(a, L.slots, tiles, pairs, h, part, st);
            return e == hipSuccess ? down(a, L.slots, tiles, pairs, h, part, st) : e;
        };
        const hipError_t e = way.rows == 64
                                 ? blocks(launch_moe_block<true, 64, 256, 1, 4>, launch_moe_block<false, 64, 256, 1, 4>)
                                 : blocks(launch_moe_block<true, 128, 128, 2, 2>, launch_moe_block<false, 128, 128, 2, 2>);
        if (e != hipSuccess) return e;
    }
    for (int64_t m = 0; m < a.M; m += kCombineMost) {
        Mx4Moe b = a;
        b.weights += m * a.k;
        b.y += m * a.y_stride;
        hipLaunchKernelGGL(mx4_combine_kernel, dim3((unsigned)(a.M - m < kCombineMost ? a.M - m : kCombineMost)), dim3(256),
                           0, st, b, place + m * a.k, part);
    }
    return hipGetLastError();
}

}  // namespace w4
