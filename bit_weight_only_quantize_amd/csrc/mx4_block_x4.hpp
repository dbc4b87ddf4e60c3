// Blocks of a product with microscaled 4-bit values on both sides, for many rows.
//
// The scheme of mx4_block.hpp with v_mfma_scale_f32_32x32x64_f8f6f4, which takes 16 bytes
// of codes a lane and side, as they are stored, and a scale byte for them: no unpacking at all,
// four times the bf16 rate. A step is 128 k, 64 code bytes of every row of X and of W.
//   * Slice s of lane half h takes group 2h + s of the step, so a lane's two scale bytes of a
//     step lie side by side. Sixteen scale bytes of a row (four steps) come in one load and
//     are packed to the lane's eight, which the instruction addresses by byte.
//   * A row's four 16-byte chunks are XOR-swizzled by row / 4: sixteen lanes read 256
//     bytes a clock, four rows.
#pragma once

#include "mx4_block.hpp"

namespace w4 {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

template <int BM, int BN>
constexpr int mx4_stage_bytes_x4() { return (BM + BN) * kBlockK4 / 2; }

// As mx4_block_product, with row(r) / wcol(c) giving {codes, scales} of a row of X / of W.
template <int BM, int BN, int WM, int WN, typename XRow, typename WCol>
__device__ __forceinline__ void mx4_block_product_x4(uint8_t* lds, XRow xrow, WCol wcol, int K, int t0, int t1,
                                                     f32x16_t (&acc)[BM / WM / 32][BN / WN / 32]) {
    constexpr int NW = WM * WN, NI = BM / WM / 32, NJ = BN / WN / 32, NR = NI + NJ;
    constexpr int XT = BM / 16, CT = BN / 16;  // direct loads of a step, 16 rows each
    constexpr int XL = (XT + NW - 1) / NW, CL = (CT + NW - 1) / NW;
    constexpr int X_BYTES = BM * kBlockK4 / 2, STAGE = mx4_stage_bytes_x4<BM, BN>();
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN, half = lane >> 5, l32 = lane & 31;
    const int groups = K / kMxGroup;

    // a load covers 16 rows, four lanes each; a lane fetches the chunk that the swizzle puts at its
    // place. (Wavefronts past the last load repeat it.)
    const int chunk = (lane & 3) ^ ((lane >> 4) & 3);
    const uint8_t* xsrc[XL];
    const uint8_t* csrc[CL];
#pragma unroll
    for (int i = 0; i < XL; ++i) xsrc[i] = xrow(16 * min(XL * wave + i, XT - 1) + (lane >> 2)).codes + 16 * chunk;
#pragma unroll
    for (int i = 0; i < CL; ++i) csrc[i] = wcol(16 * min(CL * wave + i, CT - 1) + (lane >> 2)).codes + 16 * chunk;
    const uint8_t* ssrc[NR];  // scale bytes of the rows of this lane's operands: X's, then W's
#pragma unroll
    for (int i = 0; i < NI; ++i) ssrc[i] = xrow(wm * (BM / WM) + 32 * i + l32).scale;
#pragma unroll
    for (int j = 0; j < NJ; ++j) ssrc[NI + j] = wcol(wn * (BN / WN) + 32 * j + l32).scale;

    // Scale bytes of the four steps from t on; 0 past the end of a row
    struct S16 { uint64_t lo, hi; };
    S16 sb[NR];
    auto load_scales = [&](int t) {
        if (groups >= 16) {
            const int g = min(4 * t, groups - 16);
#pragma unroll
            for (int i = 0; i < NR; ++i) __builtin_memcpy(&sb[i], ssrc[i] + g, 16);
        } else {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                uint64_t v[2] = {0, 0};
                for (int k = 4 * t; k < groups; ++k) v[(k - 4 * t) >> 3] |= (uint64_t)ssrc[i][k] << (8 * ((k - 4 * t) & 7));
                sb[i] = S16{v[0], v[1]};
            }
        }
    };
    uint32_t sc[NR][2];  // the lane's bytes: step i of the round, slice s in byte 2 (i % 2) + s of word i / 2
    auto take_scales = [&](int t) {
        const int over = groups >= 16 ? 8 * min(4 * t - min(4 * t, groups - 16), 16) : 0;  // bits read before step t
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            uint64_t lo = sb[i].lo, hi = sb[i].hi;
            if (over) {
                lo = over >= 64 ? (over >= 128 ? 0 : hi >> (over - 64)) : (lo >> over) | (hi << (64 - over));
                hi = over >= 64 ? 0 : hi >> over;
            }
            const uint32_t sel = half ? 0x07060302u : 0x05040100u;
            sc[i][0] = __builtin_amdgcn_perm((uint32_t)(lo >> 32), (uint32_t)lo, sel);
            sc[i][1] = __builtin_amdgcn_perm((uint32_t)(hi >> 32), (uint32_t)hi, sel);
        }
    };
    auto issue = [&](int t, int stage) {
        t = min(t, t1 - 1);  // past the end: a step again, into a stage nobody reads
        uint8_t* st = lds + stage * STAGE;
        if (4 * t + 4 <= groups) {
#pragma unroll
            for (int i = 0; i < XL; ++i)
                __builtin_amdgcn_global_load_lds((gbl_void*)(xsrc[i] + 64 * t),
                                                 (lds_void*)(st + min(XL * wave + i, XT - 1) * 1024), 16, 0, 0);
#pragma unroll
            for (int i = 0; i < CL; ++i)
                __builtin_amdgcn_global_load_lds((gbl_void*)(csrc[i] + 64 * t),
                                                 (lds_void*)(st + X_BYTES + min(CL * wave + i, CT - 1) * 1024), 16, 0, 0);
        } else {  // part of a step: zero codes behind the ends of rows
            const bool in = 4 * t + chunk < groups;
#pragma unroll
            for (int i = 0; i < XL; ++i)
                __builtin_amdgcn_global_load_lds((gbl_void*)(in ? xsrc[i] + 64 * t : (const uint8_t*)kMx4Zeros),
                                                 (lds_void*)(st + min(XL * wave + i, XT - 1) * 1024), 16, 0, 0);
#pragma unroll
            for (int i = 0; i < CL; ++i)
                __builtin_amdgcn_global_load_lds((gbl_void*)(in ? csrc[i] + 64 * t : (const uint8_t*)kMx4Zeros),
                                                 (lds_void*)(st + X_BYTES + min(CL * wave + i, CT - 1) * 1024), 16, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    int aoff[2], boff[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int at = l32 * 64 + (((2 * half + s) ^ ((l32 >> 2) & 3)) << 4);
        aoff[s] = wm * (BM / WM) * 64 + at;
        boff[s] = X_BYTES + wn * (BN / WN) * 64 + at;
    }
    u32x4_t a[2][NI], b[2][NJ];
    auto load = [&](int stage, int s) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[s][j] = *reinterpret_cast<const u32x4_t*>(lds + stage * STAGE + boff[s] + 2048 * j);
#pragma unroll
        for (int i = 0; i < NI; ++i) a[s][i] = *reinterpret_cast<const u32x4_t*>(lds + stage * STAGE + aoff[s] + 2048 * i);
    };
    auto wide = [](const u32x4_t& v) { return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; };
    auto products = [&](auto step, auto slice) {
        constexpr int I = decltype(step)::v, s = decltype(slice)::v, B = 2 * (I & 1) + s;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(a[s][i]), wide(b[s][j]), acc[i][j], 4, 4, B,
                                                                            (int)sc[i][I / 2], B, (int)sc[NI + j][I / 2]);
#pragma unroll
        for (int r = 0; r < NI * NJ; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            if (r < NR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int S = kStages, NB = XL + CL;
    static_assert(S == 4, "a round of scales is four steps");
    // as in mx4_block_product, the wait and the barrier before the second slice
    auto step = [&](int r, auto at) {
        constexpr int cur = decltype(at)::v;
        load(cur, 1);
        products(at, Const<0>());
        loads_done_barrier<(S - 3) * NB>();
        if (cur == 0) load_scales(r + S);
        issue(r + cur + S - 1, (cur + S - 1) % S);
        load((cur + 1) % S, 0);
        products(at, Const<1>());
        if (cur == S - 1) take_scales(r + S);
    };
    load_scales(t0);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(t0 + i, i);
    loads_done_barrier<(S - 2) * NB>();
    take_scales(t0);
    load(0, 0);
    __builtin_amdgcn_sched_barrier(0);
    int t = t0;
    for (; t + S <= t1; t += S) {
        step(t, Const<0>());
        step(t, Const<1>());
        step(t, Const<2>());
        step(t, Const<3>());
    }
    if (t < t1) step(t, Const<0>());
    if (t + 1 < t1) step(t, Const<1>());
    if (t + 2 < t1) step(t, Const<2>());
    __builtin_amdgcn_s_waitcnt(7 << 4);  // no direct load may be in flight when the workgroup ends
}

}  // namespace w4
