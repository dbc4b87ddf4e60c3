// Products with microscaled 4-bit weights for few rows (one tile of 16): the weights are
// streamed from memory to registers once, so the work is laid out for loads in flight.
//
// Sixteen code bytes are one group of 32 k: lane 16g + c loads those of group 4s + g of row c of W
// in step s of 128 k, converts them (exact, one instruction for two weights) and multiplies word j
// of them with the same k of row c of X in matrix instruction j of v_mfma_f32_16x16x32_bf16, so
// weights go from memory to the matrix cores with no exchange between lanes.
//   * X waits in LDS, zeros behind K: operands of X are four times the codes they meet, and
//     as lane loads from the caches they were what bounded the kernel (13 rows, 5120 -> 13824: 25 us against 18.5). Rows are 16 bytes off a multiple of 256, so that
//     sixteen rows' operands lie in different banks.
//   * A wavefront keeps DEPTH steps of codes in flight and starts them before X is staged.
//   * Rows of X in 4 bits need no conversion and no LDS: one v_mfma_scale_f32_16x16x128_f8f6f4 a
//     step on the codes of both sides as stored.
#pragma once

#include "mx4_block_x4.hpp"

namespace w4 {

// bytes of one row of X of `steps` steps in LDS
__host__ __device__ inline int few_row_bytes(int steps) { return 256 * steps + 16; }

// Stages k [128 s0, 128 (s0 + steps)) of `rows` rows, by all threads of the workgroup. row(r): the row's values.
template <typename Row>
__device__ __forceinline__ void few_stage(uint8_t* lds, Row row, int rows, int K, int s0, int steps) {
    const int per = 16 * steps, stride = few_row_bytes(steps);
    for (int v = threadIdx.x; v < rows * per; v += blockDim.x) {
        const int r = v / per, i = v - r * per, k = 128 * s0 + 8 * i;
        u32x4_t x = {0, 0, 0, 0};
        if (k < K) x = *reinterpret_cast<const u32x4_t*>(row(r) + k);
        *reinterpret_cast<u32x4_t*>(lds + r * stride + 16 * i) = x;
    }
}

// The wavefront's steps s = first, first + by, ... < end, over X staged from step s0 on: acc[t][r] +=
// X[4g + r] . W_t[c]. wc[t], ws[t]: row c's codes and scales.
template <int RT, int DEPTH>
struct FewStream {
    u32x4_t w[DEPTH][RT];
    uint32_t sc[DEPTH][RT];
    const uint8_t *wc[RT], *ws[RT];
    int groups;
    __device__ __forceinline__ void load(int u, int s) {  // past the end: the last group (against zeros of X)
        const int at = min(4 * s + (int)((threadIdx.x & 63) >> 4), groups - 1);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            w[u][t] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(wc[t] + 16 * at));
            sc[u][t] = ws[t][at];
        }
    }
    __device__ __forceinline__ void start(int first, int by, int end) {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            load(u, min(first + u * by, end - 1));
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __device__ __forceinline__ void run(const uint8_t* x, int first, int by, int end, int s0, f32x4_t (&acc)[RT]) {
        for (int s = first; s < end; s += DEPTH * by) {
#pragma unroll
            for (int u = 0; u < DEPTH; ++u) {
                const int at = s + u * by;
                if (at >= end) break;
                const uint8_t* p = x + 256 * (at - s0);
                bf16x8_t a[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) a[j] = *reinterpret_cast<const bf16x8_t*>(p + 16 * j);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const float f = mx4_scale(sc[u][t]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], mx4_to_bf16(w[u][t][j], f), acc[t], 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                load(u, min(at + DEPTH * by, end - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
};

}  // namespace w4
