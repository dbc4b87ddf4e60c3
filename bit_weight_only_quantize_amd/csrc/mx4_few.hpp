// Products with microscaled 4-bit weights for few rows (one tile of 16): the weights are
// streamed from memory to registers once, so the work is laid out for loads in flight.
//
// Sixteen code bytes are one group of 32 k. A load takes 128 consecutive bytes (eight groups, a whole
// cache line) of eight rows of W: lane 16g + c group 4 (c % 2) + g of row c / 2. (64 bytes of 16 rows, the
// plain layout of a matrix operand, reach 3.2 TB/s instead of 4.3 on a long stream.) Column c of a
// 16-column operand is then half c % 2 of row c / 2, and meets both halves of X in two products, of which
// the even columns of one and the odd ones of the other are kept; neighbouring lanes add theirs up
// at the end. Codes become bf16 exactly, one instruction for two weights, and go to
// v_mfma_f32_16x16x32_bf16 word by word, with no exchange between lanes before.
//   * X waits in LDS, zeros behind K: as lane loads from the caches its operands, four times the codes they
//     meet, were what bounded the kernel. Rows are 16 bytes off a multiple of 256, so that sixteen
//     rows' operands lie in different banks.
//   * A wavefront starts its first step of codes before X is staged, and the next one once a step is used up: with
//     16 or more wavefronts a CU more loads in flight made every kernel here slower.
#pragma once

#include "mx4_block_x4.hpp"

namespace w4 {

// Stages steps s0 .. s0 + steps - 1 of `rows` rows, by all threads of the workgroup. row(r): the row's values.
template <typename Row>
__device__ __forceinline__ void few_stage(uint8_t* lds, Row row, int rows, int K, int s0, int steps) {
    const int per = kFewK / 8 * steps, stride = few_row_bytes(steps);
    for (int v = threadIdx.x; v < rows * per; v += blockDim.x) {
        const int r = v / per, i = v - r * per, k = kFewK * s0 + 8 * i;
        u32x4_t x = {0, 0, 0, 0};
        if (k < K) x = *reinterpret_cast<const u32x4_t*>(row(r) + k);
        *reinterpret_cast<u32x4_t*>(lds + r * stride + 16 * i) = x;
    }
}

// Row of a 16-row tile whose result lane 16g + c holds after few_rows, and the row of its loads h = 0, 1
__device__ __forceinline__ int few_row(int c) { return (c >> 1) + 8 * (c & 1); }

struct FewSums {
    f32x4_t v[2][2];  // [rows 0..7 or 8..15][half of X]
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) v[h][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // X rows 4g .. 4g + 3 times row few_row(c) of the tile, in lane 16g + c
    __device__ __forceinline__ f32x4_t rows() const {
        const bool odd = threadIdx.x & 1;
        f32x4_t r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float own = odd ? v[h][1][i] : v[h][0][i];
                s[h] = own + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(own), 0xB1, 0xF, 0xF, false));
            }
            r[i] = odd ? s[1] : s[0];
        }
        return r;
    }
};

// The wavefront's steps s = first, first + by, ... < end over RT tiles of W, with X staged from step s0 on.
template <int RT>
struct FewStream {
    u32x4_t w[RT][2];
    uint32_t sc[RT][2];
    const uint8_t *wc[RT][2], *ws[RT][2];
    int groups;
    // row(r): {codes, scales} of row r of tile t
    template <typename Row>
    __device__ __forceinline__ void tile(int t, Row row) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const Mx4Mat m = row(8 * h + (int)(threadIdx.x & 15) / 2);
            wc[t][h] = m.codes;
            ws[t][h] = m.scale;
        }
    }
    __device__ __forceinline__ void load(int s) {  // past the end: the last group (against zeros of X)
        const int lane = threadIdx.x & 63, at = min(8 * s + 4 * (lane & 1) + (lane >> 4), groups - 1);
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[t][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(wc[t][h] + 16 * at));
                sc[t][h] = ws[t][h][at];
            }
    }
    // load(first) has been called. x: this lane's row of X in LDS, at byte 64 g; for P = 2 pieces of X (store_pieces), staged
    // as steps of twice as many values, at 128 g
    template <int P = 1>
    __device__ __forceinline__ void run(const uint8_t* x, int first, int by, int end, int s0, FewSums (&acc)[RT]) {
        for (int s = first; s < end; s += by) {
            const uint8_t* p = x + 2 * kFewK * P * (s - s0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf16x8_t a[P][2];  // [piece][half of the step]
#pragma unroll
                for (int q = 0; q < P; ++q)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        a[q][i] = *reinterpret_cast<const bf16x8_t*>(p + kFewK * P * i + 2 * kMxGroup * q + 16 * j);
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bf16x8_t b = mx4_to_bf16(w[t][h][j], mx4_scale(sc[t][h]));
#pragma unroll
                        for (int q = 0; q < P; ++q)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                acc[t].v[h][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q][i], b, acc[t].v[h][i], 0, 0, 0);
                    }
            }
            __builtin_amdgcn_sched_barrier(0);
            load(min(s + by, end - 1));
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

}  // namespace w4
