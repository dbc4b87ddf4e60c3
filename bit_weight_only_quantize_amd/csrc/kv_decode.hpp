// Attention over the batched INT4 KV cache with the keys split: the kernel for
// few rows a sequence (single tokens above all).
//
//   z_t = scale * s_k[t] * sum_i q[i] c_k[t][i]   over the visible t
//   out = sum_t exp(z_t) s_v[t] c_v[t] / sum_t exp(z_t)
// in one pass over the keys, with the softmax's maximum and sum kept running.
//
// A workgroup takes one (sequence, kv head), up to 16 NC of its (row, query
// head) columns and one part of its tiles of 32 keys; its four wavefronts take
// the tiles in turn, straight from memory to registers (kv_tile.hpp), and meet
// through LDS at the end. Parts of a sequence meet in kv_join_kernel.
//
// 16 columns cost what one does (the matrix cores' least width), so a kv head's query
// heads share one pass over its codes: 136 bytes a key of 128 + 128 values. Long contexts
// are bound by memory: two of up to 131072 positions, 5 query heads a kv head, 44 us for
// 260 MB (5.9 TB/s, some of it from the last-level cache), a ragged batch of 48 of up to
// 8192 48 us for 196 MB; the join 4. A tile takes one of a SIMD's three wavefronts some 3500 clocks: 900 the
// values' unpacking and product, 760 the weights, 770 finding and asking for the next
// keys, 170 waiting for them. Short ones are bound by the chain before the first product
// (arguments, lengths, page table, codes: some 4500 clocks, and as many for
// queries and the end): 6.2 us for 129 positions, 15 for 8193 in 22 parts a head.
#pragma once

#include <type_traits>

#include "kv_tile.hpp"

namespace w4 {

// How one call is laid out; host values only, so that the workspace's size is
// known before the call.
struct KvPlan {
    int column_tiles;  // of the sequence with the most rows
    bool prompt;       // kv_prompt_kernel, else kv_split_kernel
    int nc;            // 16-column tiles of a wavefront
    int splits;        // parts of a sequence's keys
};
constexpr int kMaxSplits = 64;
KvPlan kv_plan(const KvPages& c, int D, int group, int pieces, int64_t max_rows, int64_t max_len, int64_t window,
               int64_t sinks);

// Partial results of a part: out[D] over its own keys, then the exponent's reference
// (base 2) and the sum. Results are divided by their sums before anything is added to
// them: sums of weights times values could pass the end of fp32 where their mean does not.
__host__ __device__ constexpr int kv_partial_floats(int D) { return D + 4; }
inline size_t kv_partial_bytes(int64_t vectors, int splits, int D) {
    return (size_t)vectors * splits * kv_partial_floats(D) * sizeof(float);
}

template <int D, int NC, int PIECES, typename TQ, typename TO>
__global__ __launch_bounds__(256, (NC == 1 && D <= 128) ? 3 : 2) void kv_split_kernel(KvPages c, KvAttn a, int column_tiles, int splits) {
    constexpr int KW = D / 32, VN = D == 64 ? 4 : 8, VW = KvValues<D>::VW;
    constexpr int LD = D + 4;  // floats a column in LDS
    // exact key codes where results are fp32; for bf16 ones they would cost 14% of a long
    // context's time (53 -> 60 us, two sequences of 131072 positions)
    constexpr bool EXACT = PIECES == 2;
    constexpr bool HOLD = PIECES * KW * NC <= 4;  // queries in registers, else read from LDS for every tile
    union Lds {
        KvQueries<D, NC, PIECES> q;
        float part[4][16][LD];  // after the last tile
    };
    __shared__ __align__(16) char lds_raw[sizeof(Lds)];
    Lds& lds = *reinterpret_cast<Lds*>(lds_raw);
    __shared__ float q_zero[16 * NC], q_c[16 * NC];
    __shared__ float stat[4][NC * 16][2];  // per wavefront and column: reference, sum
    const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroups go to the 8 XCDs in turn: heads side by side, then parts, spread every
    // sequence over all of them, however the lengths differ.
    const int split = blockIdx.x / c.Hkv, head = blockIdx.x - split * c.Hkv;
    const int item = blockIdx.y + blockIdx.z * gridDim.y;  // (sequence, column tile)
    if (item >= c.B * column_tiles) return;
    const int b = item / column_tiles;
    const KvSeq s = kv_seq(c, b);
    const int columns = s.n * a.group;  // rows * Hq fits 31 bits
    const int pos0 = s.len - s.n;
    const KvTable table(c, b);
    for (int ct = item - b * column_tiles; (int64_t)ct * 16 * NC < columns; ct += column_tiles) {
        const int col0 = ct * 16 * NC, col1 = min(col0 + 16 * NC, columns) - 1;
        const int p_lo = pos0 + col0 / a.group, p_hi = pos0 + col1 / a.group;
        const int low_any = a.window > 0 ? max(p_lo, 0) - a.window : -1;
        const KvWalk walk = kv_walk(p_lo, p_hi, a.window, a.sinks);
        // count < 2^26 and splits <= 64: 32 bits hold the products
        const int j1 = (int)((unsigned)walk.count * (unsigned)(split + 1) / (unsigned)splits);
        int j = (int)((unsigned)walk.count * (unsigned)split / (unsigned)splits) + wave;

        KvRawQueries<D, NC> raw;
        raw.load([&](int i) -> const TQ* {
            const int col = col0 + i, row = col / a.group;
            return col < columns ? static_cast<const TQ*>(a.q) + (int64_t)(s.first + row) * a.q_row +
                                       (int64_t)(head * a.group + col - row * a.group) * a.q_head
                                 : nullptr;
        });
        // One tile's registers: the next tile's keys are loaded once the scores are
        // formed, its values once the second product is, its page table entries a
        // step before. The other wavefronts of the SIMD cover the rest.
        KvKeys<D> keys;
        KvValues<D> vals;
        KvHalf half[2];
        int entry[2];
        auto entries = [&](int jj) {
            const int t0 = walk.tile(min(jj, j1)) * 32;
            entry[0] = table.entry(t0);
            entry[1] = table.entry(t0 + 16);
        };
        auto locate = [&](int jj) {
            const int t0 = walk.tile(min(jj, j1)) * 32;
            half[0] = kv_half(c, b, head, t0, entry[0]);
            half[1] = kv_half(c, b, head, t0 + 16, entry[1]);
            if (jj >= j1) half[0].n = half[1].n = 0;  // past the end: reads nothing
        };
        entries(j);
        locate(j);
        keys.load(c, half, lane);
        vals.load(c, half, lane);
        entries(j + 4);

        raw.template finish<EXACT, PIECES>(lds.q, q_zero, q_c, a.scale);
        __syncthreads();
        f16x8_t q[HOLD ? PIECES : 1][HOLD ? NC : 1][HOLD ? KW : 1];
        if constexpr (HOLD) {
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int n = 0; n < NC; ++n)
#pragma unroll
                    for (int w = 0; w < KW; ++w) q[p][n][w] = lds.q.frag[p][n][w][lane];
        }
        int pos[NC], low[NC];
        float qz[NC], qc[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int col = col0 + 16 * n + l16;
            pos[n] = col < columns ? pos0 + col / a.group : -1;
            low[n] = a.window > 0 ? max(pos[n], 0) - a.window : -1;
            qz[n] = q_zero[16 * n + l16];
            qc[n] = q_c[16 * n + l16];
        }
        KvSoftmax<NC, PIECES, VW * VN> sm;
        sm.start();

        for (; j < j1; j += 4) {
            const int t0 = walk.tile(j) * 32;
            int at = lane;  // opaque, so that queries read from LDS stay there
            if constexpr (!HOLD) asm volatile("" : "+v"(at));
            // scores
            f32v4_t z[NC][2];
#pragma unroll
            for (int n = 0; n < NC; ++n) z[n][0] = z[n][1] = f32v4_t{qz[n], qz[n], qz[n], qz[n]};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    const f16x8_t k = nibbles_a<EXACT>(keys.w[h][w]);
#pragma unroll
                    for (int n = 0; n < NC; ++n)
#pragma unroll
                        for (int p = 0; p < PIECES; ++p)
                            z[n][h] = mfma16(k, HOLD ? q[HOLD ? p : 0][HOLD ? n : 0][HOLD ? w : 0] : lds.q.frag[p][n][w][at], z[n][h]);
                }
            // masks where the tile needs them: the rows' ends, the window's, the pages'
            const bool whole = half[0].n == 16 && half[1].n == 16;
            const bool seen = whole && t0 + 31 <= p_lo &&
                              (a.window == 0 || t0 > max(p_hi, 0) - a.window || t0 + 31 < a.sinks);
            if (seen)
                sm.scale(z, keys.scale);
            else
                sm.scale_masked(z, keys.scale, vals.scale, t0, g, half[0].n, half[1].n, p_hi, low_any, a.sinks, pos, low);
            locate(j + 4);
            keys.load(c, half, lane);
            entries(j + 8);
            f16x8_t pf[NC][PIECES];
            sm.weights(z, vals.scale, qc, pf);
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                uint32_t words[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) words[i] = vals.w[i][w];
                f16x8_t vf[VN];
                nibble_columns(words, vf);
#pragma unroll
                for (int i = 0; i < VN; ++i)
#pragma unroll
                    for (int n = 0; n < NC; ++n)
#pragma unroll
                        for (int p = 0; p < PIECES; ++p)
                            sm.o[n][w * VN + i] = mfma16(vf[i], pf[n][p], sm.o[n][w * VN + i]);
            }
            vals.load(c, half, lane);
        }

        // the wavefronts' references and sums
        sm.total();
#pragma unroll
        for (int n = 0; n < NC; ++n)
            if (g == 0) {
                stat[wave][16 * n + l16][0] = sm.reference(n, qc[n]);
                stat[wave][16 * n + l16][1] = sm.l[n];
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) top = fmaxf(top, stat[w][16 * n + l16][0]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float mw = stat[w][16 * n + l16][0];
                sum += mw == -INFINITY ? 0.f : stat[w][16 * n + l16][1] * __builtin_amdgcn_exp2f(mw - top);
            }
            // this wavefront's share of the columns, d consecutive per lane
            // (its own reference as stored: an fma of the product with -top would not give 0)
            const float own = stat[wave][16 * n + l16][0];
            const float f = own == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(own - top) / sum, inv = 1.f / sm.rv[n];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < VW * VN; i += 4)
                    *reinterpret_cast<f32v4_t*>(&lds.part[wave][l16][(4 * g + r) * (VW * VN) + i]) =
                        f32v4_t{sm.o[n][i][r], sm.o[n][i + 1][r], sm.o[n][i + 2][r], sm.o[n][i + 3][r]} * f * inv;
            __syncthreads();
            // 16 threads a column add the four and store
            const int cl = threadIdx.x >> 4, col = col0 + 16 * n + cl;
            constexpr int E = D / 16;
            const int e0 = (threadIdx.x & 15) * E;
            float y[E];
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const f32v4_t v = (*reinterpret_cast<const f32v4_t*>(&lds.part[0][cl][e0 + i]) +
                                   *reinterpret_cast<const f32v4_t*>(&lds.part[1][cl][e0 + i])) +
                                  (*reinterpret_cast<const f32v4_t*>(&lds.part[2][cl][e0 + i]) +
                                   *reinterpret_cast<const f32v4_t*>(&lds.part[3][cl][e0 + i]));
#pragma unroll
                for (int u = 0; u < 4; ++u) y[i + u] = v[u];
            }
            // top and sum of column l16 are those of column cl on the threads that store it
            const float ctop = __shfl(top, cl), csum = __shfl(sum, cl);
            if (col < columns) {
                const int row = s.first + col / a.group, h = head * a.group + col % a.group;
                if (splits > 1) {
                    float* w = static_cast<float*>(a.work) +
                               ((int64_t)row * a.Hq + h) * splits * kv_partial_floats(D) + (int64_t)split * kv_partial_floats(D);
#pragma unroll
                    for (int i = 0; i < E; i += 4)
                        *reinterpret_cast<f32v4_t*>(w + e0 + i) = f32v4_t{y[i], y[i + 1], y[i + 2], y[i + 3]};
                    if (e0 == 0) *reinterpret_cast<f32v4_t*>(w + D) = f32v4_t{ctop, csum, 0.f, 0.f};
                } else {
                    store_run<E>(static_cast<TO*>(a.out) + row * a.out_row + h * a.out_head + e0, y);
                    if (a.lse && e0 == 0)
                        a.lse[(int64_t)row * a.Hq + h] = kv_lse(ctop, csum);
                }
            }
            __syncthreads();
        }
    }
}

// The parts of a (row, query head) meet: one wavefront each. Lane i holds part
// i's reference and sum (kMaxSplits = 64 parts at most); D / 4 lanes share a
// part's values, so 256 / D parts are read side by side, and kAhead loads a
// lane are in flight before the references are known.
template <int D, typename TO>
__global__ __launch_bounds__(256) void kv_join_kernel(KvPages c, KvAttn a, int splits) {
    constexpr int PF = kv_partial_floats(D), LANES = D / 4, SIDE = 64 / LANES, kAhead = 8;
    const int lane = threadIdx.x & 63;
    const int64_t vectors = (int64_t)c.rows * a.Hq;
    // whole wavefronts
    for (int64_t v = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); v < vectors; v += (int64_t)gridDim.x * 4) {
        const int row = (int)(v / a.Hq), h = (int)(v - (int64_t)row * a.Hq);
        const float* w = static_cast<const float*>(a.work) + v * splits * PF;
        const int mine = min(lane, splits - 1), side = lane / LANES, e0 = 4 * (lane % LANES);
        const f32v2_t ms = *reinterpret_cast<const f32v2_t*>(w + (int64_t)mine * PF + D);
        f32v4_t x[kAhead];
        auto load = [&](int base) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                x[k] = *reinterpret_cast<const f32v4_t*>(w + (int64_t)min(base + SIDE * k + side, splits - 1) * PF + e0);
        };
        load(0);
        // rows of no sequence have no parts
        if (c.starts && (row < c.starts[0] || row >= c.starts[c.B])) continue;
        const float m = lane < splits ? ms[0] : -INFINITY;
        const float top = wave_max(m);
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
        const float sum = group_sum<64>(f * ms[1]), share = sum == 0.f ? 0.f : f * ms[1] / sum;
        f32v4_t y = {0.f, 0.f, 0.f, 0.f};
        for (int base = 0; base < splits; base += SIDE * kAhead) {
            if (base) load(base);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = base + SIDE * k + side;
                const float fi = __shfl(share, min(i, 63));
                y += x[k] * (i < splits ? fi : 0.f);
            }
        }
#pragma unroll
        for (int o = LANES; o < 64; o <<= 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] += __shfl_xor(y[e], o);
        if (side == 0) {
            const float r[4] = {y[0], y[1], y[2], y[3]};
            store_run<4>(static_cast<TO*>(a.out) + row * a.out_row + h * a.out_head + e0, r);
        }
        if (a.lse && lane == 0) a.lse[v] = kv_lse(top, sum);
    }
}

// ---------------------------------------------------------------- host side
template <int D, typename TO>
hipError_t launch_kv_join(const KvPages& c, const KvAttn& a, int splits, hipStream_t st) {
    const int64_t blocks = ((int64_t)c.rows * a.Hq + 3) / 4;  // a launch holds 2^32 - 1 threads: more loop
    hipLaunchKernelGGL((kv_join_kernel<D, TO>), dim3((unsigned)(blocks < (1 << 22) ? blocks : 1 << 22)), dim3(256), 0,
                       st, c, a, splits);
    return hipGetLastError();
}

template <int D, int NC, int PIECES, typename TQ, typename TO>
hipError_t launch_kv_split_as(const KvPages& c, const KvAttn& a, const KvPlan& p, hipStream_t st) {
    const int items = c.B * p.column_tiles, y = items < 32768 ? items : 32768;  // < 2^23
    const dim3 grid((unsigned)(c.Hkv * p.splits), (unsigned)y, (unsigned)((items + y - 1) / y));
    hipLaunchKernelGGL((kv_split_kernel<D, NC, PIECES, TQ, TO>), grid, dim3(256), 0, st, c, a, p.column_tiles,
                       p.splits);
    hipError_t e = hipGetLastError();
    return e != hipSuccess || p.splits == 1 ? e : launch_kv_join<D, TO>(c, a, p.splits, st);
}

}  // namespace w4
