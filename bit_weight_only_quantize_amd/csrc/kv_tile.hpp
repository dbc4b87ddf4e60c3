// Tiles of the INT4 KV cache in matrix-core form, shared by the attention kernels.
//
// v_mfma_f32_16x16x32_f16 takes A [16][32] and B [32][16]: lane l holds row (A)
// or column (B) l % 16 and the 8 k-slots of group g = l / 16; the result has
// column l % 16 and rows 4 g .. 4 g + 3 on lane l.
//
// A tile is 32 keys in two halves of 16 (a page never ends inside a half).
// Scores are formed transposed, S^T = K Q^T, so that a lane holds the scores of
// ONE query column for the keys 16 a + 4 g + r (half a, r = 0 .. 3) - which are
// exactly the k-slots 4 a + r of group g that the second product, O^T = V^T
// P^T, wants of P on that lane: the weights go from one product to the next
// in registers.
//
// Codes to 16-bit floats: a nibble u in bits 0-3 of a 16-bit half is the
// subnormal u * 2^-24, in bits 4-7 it is u * 2^-20, and the matrix cores take
// subnormals as they are, so one AND makes two operands. The factors are powers
// of two and go into the other operand or the result; the offset of 8 is a
// term that does not depend on the code.
#pragma once

#include "kv_attention.hpp"

namespace w4 {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32v4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32v4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32v2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32v4_t mfma16(const f16x8_t a, const f16x8_t b, const f32v4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The word's eight nibbles as one A operand, unsigned subnormals; slot order
// (elements) 0 4 1 5 2 6 3 7, the odd elements 16 times the even ones' factor.
__device__ __forceinline__ f16x8_t nibbles_a(uint32_t w) {
    const uint32_t h = w >> 8;
    const u32v4_t f = {w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u};
    return __builtin_bit_cast(f16x8_t, f);
}
__device__ constexpr int nibble_slot(int i) { return (i >> 1) + 4 * (i & 1); }  // slot -> element

// 16 head vectors (one half) of a cache array as a buffer whose reads past its
// end return zero without touching memory: `bytes` is what may be read.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}

// Where the keys of one half live: uniform over the wavefront.
struct KvHalf {
    int64_t vec;  // head vector of its first key in the pool
    int n;        // keys of it that may be read (0: no page)
};
typedef const int __attribute__((address_space(4)))* const_int_ptr;  // scalar loads

__device__ __forceinline__ KvHalf kv_half(const KvPages& c, int b, int h, int t) {
    KvHalf r;
    int page = b, off = t;
    bool good = t < c.capacity;
    if (c.table) {
        const int slot = good ? t >> c.page_shift : 0;
        page = ((const_int_ptr)c.table)[b * c.table_stride + slot];
        off = t & (c.page_size - 1);
        good = good && (unsigned)page < (unsigned)c.num_pages;
    }
    r.vec = good ? ((int64_t)page * c.Hkv + h) * c.page_size + off : 0;
    r.n = good ? min(16, c.page_size - off) : 0;
    return r;
}

// Raw contents of one tile on one wavefront.
//   k[a][j]: word j of the lane's quarter of key 16 a + l % 16 (D / 32 words)
//   v[i]: of key 16 a + 4 g + r (i = 4 a + r), the l % 16-th sixteenth of the
//         vector: 4, 8 or 16 nibbles
//   sk, sv[a]: the scales of keys 16 a + 4 g .. + 3
template <int D> struct KvTile {
    static constexpr int KW = D / 32;
    static constexpr int VW = D == 256 ? 2 : 1;
    uint32_t k[2][KW];
    uint32_t v[8][VW];
    f32v4_t sk[2], sv[2];

    __device__ __forceinline__ void load(const KvPages& c, const KvHalf* half, int lane) {
        const int l16 = lane & 15, g = lane >> 4;
        constexpr int VB = D / 2;  // bytes of a vector
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const rsrc_t rs = make_rsrc(c.scales[0] + half[a].vec, half[a].n * 4);
            const rsrc_t rk = make_rsrc(c.codes[0] + half[a].vec * VB, half[a].n * VB);
            sk[a] = __builtin_bit_cast(f32v4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * g, 0, 0));
            if constexpr (D == 64) {
                const u32v2_t w = __builtin_amdgcn_raw_buffer_load_b64(rk, l16 * VB + 8 * g, 0, 0);
                k[a][0] = w[0], k[a][1] = w[1];
            } else {
#pragma unroll
                for (int q = 0; q < KW / 4; ++q) {
                    const u32v4_t w = __builtin_amdgcn_raw_buffer_load_b128(rk, l16 * VB + g * (VB / 4) + 16 * q, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) k[a][4 * q + j] = w[j];
                }
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const rsrc_t rs = make_rsrc(c.scales[1] + half[a].vec, half[a].n * 4);
            const rsrc_t rv = make_rsrc(c.codes[1] + half[a].vec * VB, half[a].n * VB);
            sv[a] = __builtin_bit_cast(f32v4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * g, 0, 0));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int off = (4 * g + r) * VB + l16 * (VB / 16);
                if constexpr (D == 64) {
                    v[4 * a + r][0] = __builtin_amdgcn_raw_buffer_load_b16(rv, off, 0, 0);
                } else if constexpr (D == 128) {
                    v[4 * a + r][0] = __builtin_amdgcn_raw_buffer_load_b32(rv, off, 0, 0);
                } else {
                    const u32v2_t w = __builtin_amdgcn_raw_buffer_load_b64(rv, off, 0, 0);
                    v[4 * a + r][0] = w[0], v[4 * a + r][1] = w[1];
                }
            }
        }
    }
};

// The A operands of O^T = V^T P^T: operand n of word m holds, for the lane's
// vector element 8 m + n (of its sixteenth), the 8 keys in k-slot order. The
// words of two keys meet by halves, so that a 32-bit AND cuts both keys' nibble
// of one element: 1024 + u as a 16-bit float, less 1032, and from bits 4-7
// 1024 + 16 u, times 1/16 and less 72: the codes -8 .. 7, exact. (Unsigned ones
// and a term -8 sum P would be cheaper, but where the heaviest keys' code is 0
// the result is the difference of two large sums.)
template <int N>
__device__ __forceinline__ void nibble_columns(const uint32_t (&w)[8], f16x8_t (&out)[N]) {
    u32v4_t f[N];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x05040100u);
        const uint32_t hi = N == 8 ? __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07060302u) : 0u;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t x = (n < 4 ? lo : hi) >> (n & 2 ? 8 : 0);
            f16x2_t y;
            if (n & 1) {
                y = __builtin_bit_cast(f16x2_t, (x & 0x00F000F0u) | 0x64006400u);
                y = __builtin_elementwise_fma(y, f16x2_t{(_Float16)0.0625f, (_Float16)0.0625f},
                                              f16x2_t{(_Float16)-72.f, (_Float16)-72.f});
            } else {
                y = __builtin_bit_cast(f16x2_t, (x & 0x000F000Fu) | 0x64006400u);
                y = y - f16x2_t{(_Float16)1032.f, (_Float16)1032.f};
            }
            f[n][i] = __builtin_bit_cast(uint32_t, y);
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) out[n] = __builtin_bit_cast(f16x8_t, f[n]);
}

// One column's query on the lane: its quarter of the vector (group g: elements
// g D / 4 ...), scaled by a power of two to 2^14 .. 2^15 at the row's largest
// element, as B operands of S^T = K Q^T for the operands of nibbles_a (odd
// elements 1/16). PIECES = 2: x = hi + lo, 11 bits each. `zero` is the
// accumulator's start, -8 sum x, that turns unsigned codes into signed ones;
// `c` turns score * key scale into the exponent of 2.
template <int D, int PIECES> struct KvQuery {
    f16x8_t f[PIECES][D / 32];
    float zero, c;

    template <typename T>
    __device__ __forceinline__ void load(const T* q, bool live, float scale) {
        float x[D / 4];
        if (live) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) load8(q + 8 * j, x + 8 * j);
        } else {
#pragma unroll
            for (int j = 0; j < D / 4; ++j) x[j] = 0.f;
        }
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < D / 4; ++j) m = fmaxf(m, fabsf(x[j]));
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const bool some = m > 0.f && scale != 0.f;
        const int e = some ? 14 - ilogbf(m) : 0;
        const float sign = some ? copysignf(1.f, scale) : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int el = nibble_slot(i);
                float y = sign * ldexpf(x[8 * j + el], (el & 1) ? e - 4 : e);
#pragma unroll
                for (int p = 0; p < PIECES; ++p) {
                    const _Float16 h = (_Float16)y;
                    f[p][j][i] = h;
                    sum += (el & 1) ? 16.f * (float)h : (float)h;
                    y -= (float)h;
                }
            }
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        zero = -8.f * 0x1p-24f * sum;
        // finite and positive for any finite scale and query
        c = some ? fminf(fmaxf(ldexpf(fabsf(scale) * 1.4426950408889634f, 24 - e), 0x1p-120f), 0x1p120f) : 1.f;
    }
};

// The keys a tile of columns walks over: the sinks' tiles, then the window's.
struct KvWalk {
    int sink_tiles, first, count;  // tile j is j < sink_tiles ? j : j - sink_tiles + first
    __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : j - sink_tiles + first; }
};
// For rows at positions p_lo .. p_hi.
__device__ __forceinline__ KvWalk kv_walk(int p_lo, int p_hi, int window, int sinks) {
    KvWalk w;
    const int lo = window > 0 ? max(0, max(p_lo, 0) - window + 1) : 0;
    w.first = lo >> 5;
    w.sink_tiles = min((int)(((int64_t)min(sinks, lo) + 31) >> 5), w.first);
    w.count = p_hi < 0 ? 0 : w.sink_tiles + (p_hi >> 5) + 1 - w.first;
    return w;
}

}  // namespace w4
