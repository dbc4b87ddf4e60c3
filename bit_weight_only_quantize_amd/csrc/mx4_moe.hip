// The gated FFN of each token's chosen experts, with microscaled 4-bit weights:
//   y[m] = sum_j weights[m][j] W_down[e] h,  h = bf16(act(W_gate[e] x[m]) * (W_up[e] x[m])),  e = ids[m][j].
//
// Pair p = m k + j. The pairs are sorted by expert (mx4_sort_kernel), so that an
// expert's weights are read once for all of its tokens; the gate/up product writes h in
// sorted order, the down product each pair's partial row, and the last launch adds up a
// token's k rows in a fixed order. A pair's place among its expert's is not fixed (it comes
// from integer atomics), but its results do not depend on it.
#include "mx4_tile.hpp"

namespace w4 {

constexpr int kMoeTile = 16;  // pairs of one tile

struct Mx4MoeWork {  // byte offsets
    size_t tiles, pairs, h, part, total;
    int64_t slots;
};
static Mx4MoeWork moe_layout(int64_t M, int k, int64_t E, int64_t D, int64_t F) {
    const int64_t P = M * k;
    Mx4MoeWork L;
    const auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    L.slots = (E < P ? E : P) + P / kMoeTile;
    L.tiles = 0;
    L.pairs = up((size_t)L.slots * 16);
    L.h = L.pairs + up((size_t)P * 4);
    L.part = L.h + up((size_t)P * F * 2);
    L.total = L.part + up((size_t)P * D * 4);
    return L;
}
size_t mx4_moe_workspace(int64_t M, int k, int64_t E, int64_t D, int64_t F) {
    return moe_layout(M, k, E, D, F).total;
}

// One workgroup: counts, offsets, tiles {expert, first sorted pair, pairs} (-1 past the
// last) and the sorted pairs. Ids outside [0, E) are no expert's.
__global__ __launch_bounds__(1024) void mx4_sort_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                        int64_t slots, int4* __restrict__ tiles,
                                                        int32_t* __restrict__ pairs) {
    __shared__ int cnt[1024], off[1024], tile[1024];
    __shared__ int used;
    const int t = threadIdx.x;
    cnt[t] = 0;
    __syncthreads();
    for (int64_t p = t; p < P; p += 1024) {
        const int e = ids[p];
        if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    if (t < 64) {  // exclusive sums of counts and tiles, 16 experts a lane
        int c = 0, n = 0;
        for (int i = 0; i < 16; ++i) {
            c += cnt[16 * t + i];
            n += (cnt[16 * t + i] + kMoeTile - 1) / kMoeTile;
        }
        int ic = c, in = n;
        for (int d = 1; d < 64; d <<= 1) {
            const int oc = __shfl_up(ic, d), on = __shfl_up(in, d);
            if (t >= d) { ic += oc; in += on; }
        }
        int o = ic - c, a = in - n;
        for (int i = 0; i < 16; ++i) {
            const int v = cnt[16 * t + i];
            off[16 * t + i] = o;
            tile[16 * t + i] = a;
            o += v;
            a += (v + kMoeTile - 1) / kMoeTile;
        }
        if (t == 63) used = in;
    }
    __syncthreads();
    if (t < E)
        for (int i = 0; i * kMoeTile < cnt[t]; ++i)
            tiles[tile[t] + i] = make_int4(t, off[t] + i * kMoeTile, min(kMoeTile, cnt[t] - i * kMoeTile), 0);
    for (int64_t s = used + t; s < slots; s += 1024) tiles[s] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    for (int64_t p = t; p < P; p += 1024) {
        const int e = ids[p];
        if (e >= 0 && e < E) pairs[atomicAdd(&off[e], 1)] = (int)p;
    }
}

__global__ __launch_bounds__(64) void mx4_gate_up_kernel(Mx4Moe a, const int4* __restrict__ tiles,
                                                         const int32_t* __restrict__ pairs,
                                                         uint16_t* __restrict__ h, int tiles_f) {
    const int lane = threadIdx.x, g = lane >> 4, c = lane & 15;
    const int4 t = tiles[blockIdx.x / tiles_f];
    if (t.x < 0) return;
    const int64_t f0 = (int64_t)(blockIdx.x % tiles_f) * 16, f = min(f0 + c, a.F - 1);
    const int64_t row = (int64_t)t.x * a.F + f;
    const uint16_t* x = a.x + (int64_t)(pairs[t.y + min(c, t.z - 1)] / a.k) * a.x_stride;
    f32x4_t ag = {0.f, 0.f, 0.f, 0.f}, au = {0.f, 0.f, 0.f, 0.f};
    mx4_tile_product<false>(x, nullptr, nullptr, a.gate.codes + row * (a.D / 2), a.gate.scale + row * (a.D / 32),
                            (int)a.D, ag);
    mx4_tile_product<false>(x, nullptr, nullptr, a.up.codes + row * (a.D / 2), a.up.scale + row * (a.D / 32),
                            (int)a.D, au);
    if (f0 + c >= a.F) return;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * g + r < t.z) h[(int64_t)(t.y + 4 * g + r) * a.F + f] = to_bf16(gated(ag[r], au[r], a.act));
}

__global__ __launch_bounds__(64) void mx4_down_kernel(Mx4Moe a, const int4* __restrict__ tiles,
                                                      const int32_t* __restrict__ pairs,
                                                      const uint16_t* __restrict__ h, float* __restrict__ part,
                                                      int tiles_d) {
    const int lane = threadIdx.x, g = lane >> 4, c = lane & 15;
    const int4 t = tiles[blockIdx.x / tiles_d];
    if (t.x < 0) return;
    const int64_t d0 = (int64_t)(blockIdx.x % tiles_d) * 16, d = min(d0 + c, a.D - 1);
    const int64_t row = (int64_t)t.x * a.D + d;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    mx4_tile_product<false>(h + (int64_t)(t.y + min(c, t.z - 1)) * a.F, nullptr, nullptr,
                            a.down.codes + row * (a.F / 2), a.down.scale + row * (a.F / 32), (int)a.F, acc);
    if (d0 + c >= a.D) return;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * g + r < t.z) part[(int64_t)pairs[t.y + 4 * g + r] * a.D + d] = acc[r];
}

__global__ __launch_bounds__(256) void mx4_combine_kernel(Mx4Moe a, const float* __restrict__ part) {
    const int64_t m = blockIdx.x;
    for (int64_t d = threadIdx.x; d < a.D; d += 256) {
        float y = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const int e = a.ids[m * a.k + j];
            if (e >= 0 && e < a.E) y = fmaf(a.weights[m * a.k + j], part[(m * a.k + j) * a.D + d], y);
        }
        a.y[m * a.y_stride + d] = to_bf16(y);
    }
}

hipError_t launch_mx4_moe(const Mx4Moe& a, void* work, hipStream_t st) {
    const Mx4MoeWork L = moe_layout(a.M, a.k, a.E, a.D, a.F);
    uint8_t* base = (uint8_t*)work;
    int4* tiles = (int4*)(base + L.tiles);
    int32_t* pairs = (int32_t*)(base + L.pairs);
    uint16_t* h = (uint16_t*)(base + L.h);
    float* part = (float*)(base + L.part);
    const int tf = (int)((a.F + 15) / 16), td = (int)((a.D + 15) / 16);
    hipLaunchKernelGGL(mx4_sort_kernel, dim3(1), dim3(1024), 0, st, a.ids, a.M * a.k, a.E, L.slots, tiles, pairs);
    hipLaunchKernelGGL(mx4_gate_up_kernel, dim3((unsigned)(L.slots * tf)), dim3(64), 0, st, a, tiles, pairs, h, tf);
    hipLaunchKernelGGL(mx4_down_kernel, dim3((unsigned)(L.slots * td)), dim3(64), 0, st, a, tiles, pairs, h, part,
                       td);
    hipLaunchKernelGGL(mx4_combine_kernel, dim3((unsigned)a.M), dim3(256), 0, st, a, part);
    return hipGetLastError();
}

}  // namespace w4
