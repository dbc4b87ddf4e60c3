// What the microscaled operators choose by sizes: a block and pieces of K for a product of many rows, a way
// and the rows of a tile for the experts. Host code without dependencies.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace w4 {

constexpr int kMxGroup = 32;
constexpr int kMostLds = 144 << 10;  // dynamic LDS of a workgroup, beside 16 KiB of static arrays

constexpr int64_t kFewRows = 16;  // up to these rows a product streams the weights
constexpr int kFewK = 256;        // k of a step, there
constexpr int kBlockK = 64, kBlockK4 = 128;  // k of a step of blocks; with 4 bits on both sides

// bytes of one row of X of `steps` steps in LDS, for few rows
constexpr int few_row_bytes(int steps) { return 2 * kFewK * steps + 16; }
constexpr int few_steps(int64_t K) { return (int)((K + kFewK - 1) / kFewK); }

// ---- products
// Which block, and in how many pieces of K: the least estimated time. A workgroup's time is its
// steps times the step's measured time with all slots taken (us; 4096 x 12288 rows, K = 4096: 330 us
// with 256 x 256, 361, 385, 395 and 512 with the others, in this order; 256 x 128 takes 400 and
// never wins), plus its start and end;
// rounds of workgroups follow one another. Pieces cost a launch and their sums' way through
// memory (2048 x 11008 in 344 blocks of 256 x 256 on 256 slots takes 192 us, in 464 of 256 x 192 171).
struct BlockShape {
    int bm, bn, slots;  // slots: workgroups that the GPU holds at once
    double step, head;
};
static constexpr BlockShape kShapes[] = {
    {256, 256, 256, 1.60, 6}, {256, 192, 256, 1.33, 6}, {0, 0, 0, 0, 0}, {128, 256, 256, 0.98, 5},
    {128, 128, 512, 1.00, 5}, {64, 128, 768, 0.97, 5},
};
// 4 bits on both sides: steps of 128 k (4096 x 12288 rows, K = 16384: 560 us with 256 x 192, then 651,
// 716 and 1093). 128 x 256 takes 731, 256 x 256 needs more registers than there are and takes 632.
static constexpr BlockShape kShapesX4[] = {
    {0, 0, 0, 0, 0}, {256, 192, 256, 1.09, 6}, {256, 128, 256, 0.85, 5}, {0, 0, 0, 0, 0},
    {128, 128, 512, 0.93, 3}, {64, 128, 768, 1.07, 2},
};
struct BlockPlan {
    int shape, parts;
};
inline size_t part_bytes(const BlockShape& s, int64_t M, int64_t N) {
    return (size_t)((M + s.bm - 1) / s.bm * s.bm) * ((N + s.bn - 1) / s.bn * s.bn) * 4;
}
inline BlockPlan block_plan(int64_t M, int64_t N, int64_t K, bool x4, bool can_split) {
    const BlockShape* shapes = x4 ? kShapesX4 : kShapes;
    BlockPlan best = {0, 1};
    double least = 1e30;
    const int64_t steps = x4 ? (K + kBlockK4 - 1) / kBlockK4 : (K + kBlockK - 1) / kBlockK;
    for (int i = 0; i < 6; ++i) {
        const BlockShape& s = shapes[i];
        if (!s.slots) continue;  // never the best for these operands
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

// ---- experts
struct MoeWay {
    bool direct;
    int rows;  // of a tile
};

constexpr int64_t kDirectPairs = 16;

// Rows of a tile: half a tile an expert is wasted, and the weights are read once a tile. Blocks of 64 x 256
// against 128 x 128, whose steps cost less for their size and which waste more (us a call, F x D):
//   pairs an expert     256           384           512
//   128 x (768 x 2048)  597 and 650   845 and 889   1087 and 1151
//   60 x (1408 x 2048)  515 and 516   726 and 736   917 and 922
//   8 x (1408 x 4096)   152 and 165   214 and 196   269 and 251
//   32 x (1408 x 4096)  534 and 522   735 and 718   927 and 912
//   8 x (8192 x 4096)                 1153 and 988  1462 and 1237
// The larger blocks win with long sums, by up to 15%, and lose up to 6% with short ones; with 256 pairs and less they lose in more
// of these than they win.
inline MoeWay moe_way(int64_t M, int k, int64_t E, int64_t D, int64_t F) {
    const int64_t P = M * k;
    if (P <= kDirectPairs && k * F <= (32 << 10) && D <= (64 << 10)) return {true, 0};
    // rows that fit in LDS, of x and of pieces of h. (h a part at a time instead: 50 tokens, 8 experts of 4096 x 2048, top 2, 94 us
    // against 98 in blocks, but 16 tokens over 8192 x 4096 247 against 199.)
    const int steps = few_steps(D) > 2 * few_steps(F) ? few_steps(D) : 2 * few_steps(F);
    const int64_t each = P / E, room = kMostLds / few_row_bytes(steps);
    if (each <= 6 && room >= 8) return {false, 8};
    if (each <= 16 && room >= 16) return {false, 16};
    return {false, each <= 320 ? 64 : 128};
}

}  // namespace w4
