// One row of X times microscaled 4-bit rows of W, in the vector units.
//
// With a single row the matrix cores would take sixteen rows of W side by side, 64 bytes of
// each; here a wavefront reads whole rows, 1 KiB of consecutive codes a load (4096 -> 11008: 7.5 us
// against 12). Lane l takes vectors l, l + 64, ... of 16 code bytes, which are one group each, so the
// scale bytes of a load are consecutive too; one instruction converts two weights to bf16
// (exactly, scale included) and one v_dot2_f32_bf16 multiplies them with two of x.
// x waits in LDS in four planes: 16 bytes (eight values) j of vector v at plane j, place v, so that lanes read
// consecutive 16 bytes. Zeros behind K.
#pragma once

#include "mx4.hpp"

namespace w4 {

__host__ __device__ inline int gemv_vectors(int K) { return (K / kMxGroup + 63) / 64 * 64; }
__host__ __device__ inline int gemv_lds_bytes(int K) { return 64 * gemv_vectors(K); }  // a piece

// By all threads of the workgroup. P = 2 pieces of x (store_pieces): eight planes, the second pieces' behind the first ones'.
template <int P = 1>
__device__ __forceinline__ void gemv_stage(uint8_t* lds, const uint16_t* x, int K) {
    const int V = gemv_vectors(K);
    for (int i = threadIdx.x; i < 4 * P * V; i += blockDim.x) {
        u32x4_t v = {0, 0, 0, 0};
        if (8 * i < P * K) v = *reinterpret_cast<const u32x4_t*>(x + 8 * i);
        *reinterpret_cast<u32x4_t*>(lds + i % (4 * P) * (16 * V) + i / (4 * P) * 16) = v;
    }
}

template <int R, int U>
struct GemvStream {
    u32x4_t w[U][R];
    uint32_t sc[U][R];
    const uint8_t *wc[R], *ws[R];  // wave-uniform rows
    int groups;
    __device__ __forceinline__ void load(int v0) {  // vectors v0 + lane, + 64, ...; past the end the last one (x is 0 there)
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = min(v0 + 64 * u + lane, groups - 1);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                w[u][r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(wc[r] + 16 * v));
                sc[u][r] = ws[r][v];
            }
        }
    }
    __device__ __forceinline__ void add(const uint8_t* lds, int V, int v0, float (&acc)[R]) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v0 + 64 * u >= V) break;
            u32x4_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const u32x4_t*>(lds + j * (16 * V) + (v0 + 64 * u + lane) * 16);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float f = mx4_scale(sc[u][r]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x4_t b = __builtin_bit_cast(u32x4_t, mx4_to_bf16(w[u][r][j], f));
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[r] = dot2_bf16(b[q], x[j][q], acc[r]);
                }
            }
        }
    }
    // The rows' whole products, load(0) having been called, in every lane
    __device__ __forceinline__ void finish(const uint8_t* lds, int V, float (&acc)[R]) {
        for (int v0 = 0; v0 < V; v0 += 64 * U) {
            add(lds, V, v0, acc);
            if (v0 + 64 * U < V) load(v0 + 64 * U);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = group_sum<64>(acc[r]);
    }
};

}  // namespace w4
