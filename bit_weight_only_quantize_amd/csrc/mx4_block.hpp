// Blocks of a product with microscaled 4-bit weights and bf16 rows, for many rows.
//
// A workgroup of WM x WN wavefronts owns BM rows of X and BN rows ("columns") of W, a
// wavefront BM / WM by BN / WN of them in tiles of v_mfma_f32_32x32x16_bf16. Per step of
// 64 k the rows' 128 bytes and the columns' 32 code bytes arrive in LDS by direct
// global -> LDS loads in a ring of four stages, three steps ahead; a wavefront's codes
// become its B operands in registers, one conversion instruction per two weights (exact).
//   * Bound by the matrix cores and what feeds them: with the largest block (256 x 256,
//     eight wavefronts, 160 KiB of LDS) a step without any load takes 83% of its time.
//     4096 x 8192, K = 4096: 216 us, 1271 TFLOP/s (the library's bf16 product of the same
//     sizes 178 us on that machine); 2048 x 11008: 168 us (198).
//   * Weights are 4 bits wide in LDS, so operand reads of W cost a quarter of X's, and
//     several wavefronts converting the same columns costs less than sharing bf16 tiles:
//     one conversion per matrix instruction hides under it wherever two wavefronts share a SIMD.
//   * One barrier a step, in its middle, after a wait that leaves the last batch of loads in
//     flight; the next step's first operands are read and unpacked under this step's last
//     matrix instructions. (Two stages and two workgroups a CU: 306 us; three stages 322.)
//   * Scale bytes go to registers, eight at a time (one at a time 250 us: a lane load of
//     single bytes from as many rows touches as many lines as all other loads together).
//   * Inside a step slice kk of lane half h takes the k of code word 4h + kk, so the 16 code
//     bytes a lane reads are one group of 32 and have one scale.
//   * X's 16-byte chunks are XOR-swizzled by row / 2 through the chunk each lane of a direct
//     load fetches: sixteen lanes read 256 bytes a clock, so two rows of 128 bytes fill the
//     banks and every second row needs another place (by row, reads took twice the clocks).
#pragma once

#include "mx4.hpp"

namespace w4 {

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void gbl_void;

template <int V>
struct Const {
    static constexpr int v = V;
};

// Waits until at most this wavefront's last N loads are in flight, then the barrier: after it the
// direct loads before those are in LDS, every wavefront's. The empty asm keeps memory operations
// on their side of it.
template <int N>
__device__ __forceinline__ void loads_done_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ const __align__(16) uint16_t kMx4Zeros[8] = {};

constexpr int kStages = 4;
template <int BM, int BN, bool PIECES = false>
constexpr int mx4_stage_bytes() { return BM * kBlockK * 2 + BN * kBlockK / (PIECES ? 4 : 2); }

// The k loop. xrow(r): row r (0 .. BM - 1) of the block, any valid row where it has none; wcol(c):
// the same for W as {codes, scales} of column c. Steps t0 .. t1 - 1. acc: of the wavefront's tiles. PIECES: X holds
// pieces (store_pieces), so a step is one group of W, and an operand of W meets both pieces: slice kk of lane half h takes
// piece kk % 2 of the k of code word 2h + kk / 2.
template <int BM, int BN, int WM, int WN, bool PIECES = false, typename XRow, typename WCol>
__device__ __forceinline__ void mx4_block_product(uint8_t* lds, XRow xrow, WCol wcol, int K, int t0, int t1,
                                                  f32x16_t (&acc)[BM / WM / 32][BN / WN / 32]) {
    constexpr int NW = WM * WN, NI = BM / WM / 32, NJ = BN / WN / 32;
    constexpr int PER = PIECES ? 1 : 2;  // groups of a step
    constexpr int XL = BM / 8 / NW, CC = 64 / PER, CL = BN / CC;  // direct loads of a step: X per wavefront, codes in all
    static_assert(BM % (8 * NW) == 0 && BN % CC == 0 && (CL % NW == 0 || CL < NW), "loads per wavefront");
    constexpr int X_BYTES = BM * kBlockK * 2, STAGE = mx4_stage_bytes<BM, BN, PIECES>();
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN, half = lane >> 5, l32 = lane & 31;

    // load q of a step covers rows 8q .. 8q + 7, eight lanes each; a lane fetches the chunk that the
    // swizzle puts at its place
    auto chunk = [&](int i) { return ((lane & 7) ^ ((4 * (XL * wave + i) + (lane >> 4)) & 7)) * 8; };
    const uint16_t* xsrc[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) xsrc[i] = xrow(8 * (XL * wave + i) + (lane >> 3)) + chunk(i);
    constexpr int CW = CL >= NW ? CL / NW : 1;
    const uint8_t* csrc[CW];
#pragma unroll
    for (int i = 0; i < CW; ++i) csrc[i] = wcol(CC * (min(wave, CL - 1) * CW + i) + lane % CC).codes;
    const uint8_t* ssrc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) ssrc[j] = wcol(wn * (BN / WN) + 32 * j + l32).scale;
    const int groups = K / kMxGroup, own = PIECES ? 0 : half;

    // A column's scale bytes for the kStages steps from t on, in 8 bytes (a lane load of single
    // bytes touches 32 lines a step, as many as all else); past the end of a row, its last ones.
    uint64_t sb[NJ];
    auto load_scales = [&](int t) {
        if (groups >= 2 * kStages) {
            const int g = min(PER * t, groups - 2 * kStages);
#pragma unroll
            for (int j = 0; j < NJ; ++j) __builtin_memcpy(&sb[j], ssrc[j] + g, 8);
        } else {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                sb[j] = 0;
                for (int i = 0; i < groups; ++i) sb[j] |= (uint64_t)ssrc[j][i] << (8 * i);
            }
        }
    };
    auto scale_of = [&](uint64_t v, int t, int i) {  // step t + i of the bytes loaded for step t
        const int g = groups >= 2 * kStages ? min(PER * t, groups - 2 * kStages) : 0;
        return mx4_scale((uint32_t)(v >> (8 * (min(PER * (t + i) + own, groups - 1) - g))) & 255u);
    };
    auto issue = [&](int t, int stage) {
        t = min(t, t1 - 1);  // past the end: a step again, into a stage nobody reads
        uint8_t* st = lds + stage * STAGE;
        const int g = min(PER * t + own, groups - 1);
        if (PIECES || 2 * t + 1 < groups) {
#pragma unroll
            for (int i = 0; i < XL; ++i)
                __builtin_amdgcn_global_load_lds((gbl_void*)(xsrc[i] + kBlockK * t),
                                                 (lds_void*)(st + (XL * wave + i) * 1024), 16, 0, 0);
        } else {  // half a step: zeros of X behind its end (the codes there are any, the last group's)
#pragma unroll
            for (int i = 0; i < XL; ++i)
                __builtin_amdgcn_global_load_lds((gbl_void*)(chunk(i) < 32 ? xsrc[i] + kBlockK * t : kMx4Zeros),
                                                 (lds_void*)(st + (XL * wave + i) * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < CW; ++i)  // (wavefronts past the last columns fetch those again)
            __builtin_amdgcn_global_load_lds((gbl_void*)(csrc[i] + 16 * g),
                                             (lds_void*)(st + X_BYTES + (min(wave, CL - 1) * CW + i) * 1024), 16, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    int aoff[4];  // of this lane's chunk of slice kk in row l32 of a tile
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) aoff[kk] = (wm * (BM / WM) + l32) * 128 + (((PIECES ? 4 * (kk & 1) + 2 * half + (kk >> 1) : 4 * half + kk) ^ ((l32 >> 1) & 7)) << 4);
    bf16x8_t a[2][NI], b[2][NJ];
    typedef unsigned Codes __attribute__((ext_vector_type(4 / (3 - PER))));  // of a lane and column in a step
    Codes cw[NJ];
    float sw[NJ];
    auto load_a = [&](int stage, int kk) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            a[kk & 1][i] = *reinterpret_cast<const bf16x8_t*>(lds + stage * STAGE + aoff[kk] + 4096 * i);
    };
    auto load_codes = [&](int stage) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint8_t* p = lds + stage * STAGE + X_BYTES;
            if constexpr (PIECES) cw[j] = *reinterpret_cast<const Codes*>(p + (wn * NJ + j) * 512 + l32 * 16 + half * 8);
            else cw[j] = *reinterpret_cast<const Codes*>(p + (wn * NJ + j) * 1024 + lane * 16);
        }
    };
    auto unpack = [&](int kk) {
        if (PIECES && (kk & 1)) return;  // both pieces' slices share it
        const int w = PIECES ? kk >> 1 : kk;
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[w & 1][j] = mx4_to_bf16(cw[j][w], sw[j]);
    };
    auto products = [&](int kk, int reads) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[kk & 1][i], b[(PIECES ? kk >> 1 : kk) & 1][j], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int r = 0; r < NI * NJ; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);  // a matrix instruction
            if (r < reads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
            __builtin_amdgcn_sched_group_barrier(0x2, (4 * NJ + NI * NJ - 1) / (NI * NJ), 0);  // conversions
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int S = kStages, NB = XL + CW;  // direct loads of a step's batch
    uint64_t sc[NJ];  // scale bytes of the present round of S steps; sb: of the next
    // Step t = r + cur of round r. The wait in its middle leaves the last batch in flight, so a batch
    // has two steps to arrive; the barrier after it also frees the stage of step t - 1.
    auto step = [&](int r, int cur) {
        load_a(cur, 1);
        unpack(1);
        products(0, NI);
        load_a(cur, 2);
        unpack(2);
        products(1, NI);
        loads_done_barrier<(S - 3) * NB>();
        if (cur == 0) load_scales(r + S);
        issue(r + cur + S - 1, (cur + S - 1) % S);
        load_a(cur, 3);
        unpack(3);
        products(2, NI);
        load_codes((cur + 1) % S);
        load_a((cur + 1) % S, 0);
        if (cur == S - 1) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) sc[j] = sb[j];
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) sw[j] = cur == S - 1 ? scale_of(sc[j], r + S, 0) : scale_of(sc[j], r, cur + 1);
        unpack(0);
        products(3, NI + NJ);
    };
    load_scales(t0);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(t0 + i, i);
    loads_done_barrier<(S - 2) * NB>();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        sc[j] = sb[j];
        sw[j] = scale_of(sc[j], t0, 0);
    }
    load_codes(0);
    load_a(0, 0);
    unpack(0);
    __builtin_amdgcn_sched_barrier(0);
    int t = t0;
    for (; t + S <= t1; t += S) {
#pragma unroll
        for (int i = 0; i < S; ++i) step(t, i);
    }
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        if (t + i < t1) step(t, i);
    __builtin_amdgcn_s_waitcnt(7 << 4);  // no direct load may be in flight when the workgroup ends
}

}  // namespace w4
