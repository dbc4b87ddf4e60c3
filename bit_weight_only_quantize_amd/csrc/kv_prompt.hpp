// Attention over the batched INT4 KV cache for many rows a sequence (prompts):
// the same products and softmax as kv_decode.hpp, with the keys' operands made
// once for a workgroup.
//
// A workgroup of eight wavefronts takes 128 NC (row, query head) columns of one
// (sequence, kv head), 16 NC a wavefront, and walks over the keys in stages of
// four tiles (two with D = 256). Per stage each wavefront turns its share of the codes
// into operands in LDS (one of two buffers, filled a stage ahead) and then takes
// every tile for its own columns: unpacking costs an eighth of what it does in
// kv_split_kernel. The causal edge makes the last columns the longest: they go first.
//
// A tile takes each wavefront about 3400 clocks, two wavefronts a SIMD; the matrix
// cores work 30% of the time and the vector unit 60%, with a wavefront's phases waiting
// on one another. 8192 rows of 32 heads of 128: 730 us, 753 TFLOP/s over the causal pairs,
// where a library's bf16 product of 8192^3 runs at 1205; with fp32 rows, in two pieces, 1000
// (13 to 16 of its vector registers are spilled; no other kernel here spills vector registers).
#pragma once

#include "kv_decode.hpp"

namespace w4 {

template <int D> struct KvStage {
    static constexpr int KW = D / 32, NO = D / 16;
    static constexpr int TILES = D == 256 ? 2 : 4;  // two stages fit the 160 KB of a CU
    f16x8_t k[TILES][2][KW][64];  // [tile][half][k-step][lane]
    f16x8_t v[TILES][NO][64];     // [tile][operand][lane]
    float ks[TILES][32], vs[TILES][32];
    int n[TILES][2];              // keys there, of each half
};

// What one wavefront brings of a stage, on its way through registers: the keys of
// a tile with its scales, or its values (D = 256: of a half, or one word of each
// of the lane's pieces). A lane's loads are as wide as its operands allow: how many
// there are bounds the filling, not their bytes.
template <int D> struct KvBring {
    static constexpr int KW = D / 32, VB = D / 2, WPT = 8 / KvStage<D>::TILES;  // wavefronts a tile
    static constexpr int HALVES = 4 / WPT;  // halves of a keys' wavefront
    static constexpr int VN = D == 64 ? 4 : 8;
    uint32_t raw[8];  // keys: [half][word], values: [key]
    float scale;      // of key lane % 16: lanes 0-15, 16-31, ... hold (keys', values') x (halves)
    int n[HALVES];

    static __device__ __forceinline__ bool of_keys(int s) { return s < WPT / 2; }

    __device__ __forceinline__ void load(const KvPages& c, const KvHalf (&half)[2], int s, int lane) {
        const int l16 = lane & 15, g = lane >> 4;
        if (of_keys(s)) {
            KvHalf mine[HALVES];
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const int64_t v0 = half[0].vec, v1 = half[1].vec;
                const int n0 = half[0].n, n1 = half[1].n;
                mine[h].vec = (HALVES == 2 ? h : s) ? v1 : v0;
                mine[h].n = (HALVES == 2 ? h : s) ? n1 : n0;
                n[h] = mine[h].n;
                const rsrc_t r = make_rsrc(c.codes[0] + mine[h].vec * VB, mine[h].n * VB);
                const int off = l16 * VB + g * (VB / 4);
                if constexpr (KW == 2) {
                    const u32v2_t x = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
                    raw[2 * h] = x[0], raw[2 * h + 1] = x[1];
                } else {
#pragma unroll
                    for (int q = 0; q < KW / 4; ++q) {
                        const u32v4_t x = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * q, 0, 0);
#pragma unroll
                        for (int j = 0; j < 4; ++j) raw[h * KW + 4 * q + j] = x[j];
                    }
                }
            }
            // one load for all the scales; keys that are not there: 0
            const bool second = HALVES == 2 && (g & 1), values = HALVES == 2 ? g >= 2 : g & 1;
            const int64_t v0 = mine[0].vec, v1 = mine[HALVES - 1].vec;
            const int n0 = n[0], n1 = n[HALVES - 1];
            const bool there = l16 < (second ? n1 : n0);
            const float *p0 = c.scales[0], *p1 = c.scales[1];
            const float* p = (values ? p1 : p0) + (there ? (second ? v1 : v0) + l16 : 0);
            scale = there ? *p : 0.f;
        } else {
            const int word = WPT == 4 ? s - 2 : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const rsrc_t r = make_rsrc(c.codes[1] + half[h].vec * VB, half[h].n * VB);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = 4 * g * VB + l16 * (VB / 16) + 4 * word + k * VB;
                    if constexpr (D == 64)
                        raw[4 * h + k] = __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
                    else
                        raw[4 * h + k] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
                }
            }
        }
    }

    __device__ __forceinline__ void store(KvStage<D>& st, int tile, int s, int lane) const {
        if (of_keys(s)) {
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const int a = HALVES == 2 ? h : s;
#pragma unroll
                for (int j = 0; j < KW; ++j) st.k[tile][a][j][lane] = nibbles_a<true>(raw[h * KW + j]);
                if (lane == 0) st.n[tile][a] = n[h];
            }
            const int l16 = lane & 15, g = lane >> 4;
            if (g < 2 * HALVES) {
                const bool values = HALVES == 2 ? g >= 2 : g & 1;
                (values ? st.vs : st.ks)[tile][16 * (HALVES == 2 ? g & 1 : s) + l16] = scale;
            }
        } else {
            const int word = WPT == 4 ? s - 2 : 0;
            f16x8_t f[VN];
            nibble_columns(raw, f);
#pragma unroll
            for (int q = 0; q < VN; ++q) st.v[tile][word * VN + q][lane] = f[q];
        }
    }
};

template <int D, int NC, int PIECES, typename TQ, typename TO>
__global__ __launch_bounds__(512, 2) void kv_prompt_kernel(KvPages c, KvAttn a, int column_tiles, int splits) {
    constexpr int KW = D / 32, NO = D / 16, CW = 16 * NC, CB = 8 * CW;
    __shared__ KvStage<D> stage[2];
    const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The last columns see the most keys: they go first, those of all heads side by side.
    // (Workgroups go to the 8 XCDs in turn, so with 8 n heads an XCD keeps to its own.)
    const int pairs = c.B * c.Hkv, turn = blockIdx.x / pairs, pair = blockIdx.x - turn * pairs;
    const int split = blockIdx.y, b = pair / c.Hkv, head = pair - b * c.Hkv;
    const KvSeq s = kv_seq(c, b);
    const int columns = s.n * a.group;  // rows * Hq fits 31 bits
    const int pos0 = s.len - s.n;
    const KvTable table(c, b);
    constexpr int TILES = KvStage<D>::TILES, WPT = KvBring<D>::WPT;
    const int tw = wave / WPT, sw = wave % WPT;
    for (int64_t ct = column_tiles - 1 - turn; ct * CB < columns; ct += column_tiles) {
        const int col0 = (int)ct * CB, col1 = min(col0 + CB, columns) - 1;
        const KvWalk walk = kv_walk(pos0 + col0 / a.group, pos0 + col1 / a.group, a.window, a.sinks);
        // count < 2^26 and splits <= 64: 32 bits hold the products
        const int j0 = (int)((unsigned)walk.count * (unsigned)split / (unsigned)splits);
        const int j1 = (int)((unsigned)walk.count * (unsigned)(split + 1) / (unsigned)splits);

        const int tiles = j1 - j0;  // tile i of this part is j0 + i of the walk

        KvBring<D> bring;
        KvHalf half[2];
        int entry[2];
        auto entries = [&](int i) {  // of this wavefront's tile of the stage that starts at i
            const int t0 = walk.tile(j0 + min(i + tw, tiles)) * 32;
            entry[0] = table.entry(t0);
            entry[1] = table.entry(t0 + 16);
        };
        auto fetch = [&](int i) {
            const int t0 = walk.tile(j0 + min(i + tw, tiles)) * 32;
            half[0] = kv_half(c, b, head, t0, entry[0]);
            half[1] = kv_half(c, b, head, t0 + 16, entry[1]);
            if (i + tw >= tiles) half[0].n = half[1].n = 0;  // past the end: reads nothing
            bring.load(c, half, sw, lane);
            entries(i + TILES);
        };
        entries(0);
        fetch(0);

        // this wavefront's columns
        const int w0 = col0 + wave * CW;
        const bool any = w0 < columns;
        const int p_lo = any ? pos0 + w0 / a.group : -1;
        const int p_hi = any ? pos0 + min(w0 + CW - 1, columns - 1) / a.group : -1;
        const int low_any = a.window > 0 ? max(p_lo, 0) - a.window : -1;
        f16x8_t q[NC][PIECES][KW];
        float qc[NC];
        int pos[NC], low[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int col = w0 + 16 * n + l16, row = col / a.group;
            const bool live = col < columns;
            const TQ* p = live ? static_cast<const TQ*>(a.q) + (int64_t)(s.first + row) * a.q_row +
                                     (int64_t)(head * a.group + col - row * a.group) * a.q_head
                               : nullptr;
            load_query<D, PIECES>(p, g, a.scale, q[n], qc[n]);
            pos[n] = live ? pos0 + row : -1;
            low[n] = a.window > 0 ? max(pos[n], 0) - a.window : -1;
        }
        KvSoftmax<NC, PIECES, NO> sm;
        sm.start();
        bring.store(stage[0], tw, sw, lane);

        // Filling the next stage falls between different tiles for the two wavefronts of a
        // SIMD (w and w + 4), beside the other's work.
        int buf = 0;
        for (int i0 = 0; i0 < tiles; i0 += TILES, buf ^= 1) {
            __syncthreads();  // this stage is whole, and nobody reads the other buffer
            fetch(i0 + TILES);
            const KvStage<D>& st = stage[buf];
            const int count = min(TILES, tiles - i0);
            // no key of its tiles is missing (pages that are not there, the end of the pool)
            const bool pages = __builtin_amdgcn_ballot_w64(lane < 2 * count && (&st.n[0][0])[lane] != 16) == 0;
#pragma unroll 1
            for (int ti = 0; ti < TILES; ++ti) {
                if (ti >= count) continue;
                const int t0 = walk.tile(j0 + i0 + ti) * 32;
                const bool whole = pages && t0 + 31 <= p_lo && (a.window == 0 || t0 > max(p_hi, 0) - a.window || t0 + 31 < a.sinks);
                // nothing of it for these columns
                if (!whole && (t0 > p_hi || (a.window > 0 && t0 + 31 <= low_any && t0 >= a.sinks))) continue;
                // all of a product's operands are asked for before its first use: left to
                // itself the compiler waits for each in turn
                constexpr int NV = NO < 8 ? NO : 8;
                f16x8_t kf[KW][2], vf[NV];
#pragma unroll
                for (int w = 0; w < KW; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) kf[w][h] = st.k[ti][h][w][lane];
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);  // products before the other wavefront's softmax: 735 -> 729 us
                f32v4_t z[NC][2];
#pragma unroll
                for (int n = 0; n < NC; ++n) z[n][0] = z[n][1] = f32v4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < KW; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < NC; ++n)
#pragma unroll
                            for (int p = 0; p < PIECES; ++p) z[n][h] = mfma16(kf[w][h], q[n][p][w], z[n][h]);
                f32v4_t ks[2], vs[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ks[h] = *reinterpret_cast<const f32v4_t*>(&st.ks[ti][16 * h + 4 * g]);
                    vs[h] = *reinterpret_cast<const f32v4_t*>(&st.vs[ti][16 * h + 4 * g]);
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) vf[k] = st.v[ti][k][lane];
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                if (whole) {
                    sm.scale(z, ks);
                } else {
                    const int n0 = __builtin_amdgcn_readfirstlane(st.n[ti][0]);
                    const int n1 = __builtin_amdgcn_readfirstlane(st.n[ti][1]);
                    sm.scale_masked(z, ks, vs, t0, g, n0, n1, p_hi, low_any, a.sinks, pos, low);
                }
                f16x8_t pf[NC][PIECES];
                sm.weights(z, vs, qc, pf);
#pragma unroll
                for (int k0 = 0; k0 < NO; k0 += NV) {
                    if (k0) {
#pragma unroll
                        for (int k = 0; k < NV; ++k) vf[k] = st.v[ti][k0 + k][lane];
                        __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                    for (int k = 0; k < NV; ++k)
#pragma unroll
                        for (int n = 0; n < NC; ++n)
#pragma unroll
                            for (int p = 0; p < PIECES; ++p) sm.o[n][k0 + k] = mfma16(vf[k], pf[n][p], sm.o[n][k0 + k]);
                }
            }
            bring.store(stage[buf ^ 1], tw, sw, lane);
        }
        __syncthreads();  // the buffers are free for the next columns

        sm.total();
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int col = w0 + 16 * n + l16;
            if (col >= columns) continue;
            const int row = s.first + col / a.group, h = head * a.group + col % a.group;
            const float top = sm.reference(n, qc[n]);
            const float f = sm.l[n] == 0.f ? 0.f : 1.f / sm.l[n], inv = 1.f / sm.rv[n];
            if (splits > 1) {
                float* w = static_cast<float*>(a.work) +
                           (((int64_t)row * a.Hq + h) * splits + split) * kv_partial_floats(D);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < NO; i += 4)
                        *reinterpret_cast<f32v4_t*>(w + (4 * g + r) * NO + i) =
                            f32v4_t{sm.o[n][i][r], sm.o[n][i + 1][r], sm.o[n][i + 2][r], sm.o[n][i + 3][r]} * f * inv;
                if (g == 0) *reinterpret_cast<f32v4_t*>(w + D) = f32v4_t{top, sm.l[n], 0.f, 0.f};
                continue;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float y[NO];
#pragma unroll
                for (int i = 0; i < NO; ++i) y[i] = sm.o[n][i][r] * f * inv;
                store_run<NO>(static_cast<TO*>(a.out) + row * a.out_row + h * a.out_head + (4 * g + r) * NO, y);
            }
            if (a.lse && g == 0)
                a.lse[(int64_t)row * a.Hq + h] = kv_lse(top, sm.l[n]);
        }
    }
}

// ---------------------------------------------------------------- host side
template <int D, int NC, int PIECES, typename TQ, typename TO>
hipError_t launch_kv_prompt_as(const KvPages& c, const KvAttn& a, const KvPlan& p, hipStream_t st) {
    const dim3 grid((unsigned)((int64_t)p.column_tiles * c.B * c.Hkv), (unsigned)p.splits);
    hipLaunchKernelGGL((kv_prompt_kernel<D, NC, PIECES, TQ, TO>), grid, dim3(512), 0, st, c, a, p.column_tiles,
                       p.splits);
    hipError_t e = hipGetLastError();
    return e != hipSuccess || p.splits == 1 ? e : launch_kv_join<D, TO>(c, a, p.splits, st);
}

}  // namespace w4
