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
// Codes to 16-bit floats: exact codes -8 .. 7 in two instructions a pair
// (signed_pair). Or, for the keys under bf16 queries, in one: a nibble u in bits
// 0-3 of a 16-bit half is the subnormal u * 2^-24, in bits 4-7 it is u * 2^-20, and
// the matrix cores take subnormals as they are. The factors are powers of two and
// go into the other operand or the result; the offset of 8 is a term that does not
// depend on the code.
#pragma once

#include "kv_attention.hpp"

namespace w4 {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32v2_t __attribute__((ext_vector_type(2)));
typedef float f32v4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32v4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32v2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32v4_t mfma16(const f16x8_t a, const f16x8_t b, const f32v4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// One nibble of each 16-bit half, as the code -8 .. 7 in a 16-bit float: bits 0-3
// as 1024 + u less 1032, bits 4-7 (odd) as 1024 + 16 u times 1/16 less 72; exact.
__device__ __forceinline__ uint32_t signed_pair(uint32_t x, bool odd) {
    f16x2_t y;
    if (odd) {
        y = __builtin_bit_cast(f16x2_t, (x & 0x00F000F0u) | 0x64006400u);
        y = __builtin_elementwise_fma(y, f16x2_t{(_Float16)0.0625f, (_Float16)0.0625f},
                                      f16x2_t{(_Float16)-72.f, (_Float16)-72.f});
    } else {
        y = __builtin_bit_cast(f16x2_t, (x & 0x000F000Fu) | 0x64006400u);
        y = y - f16x2_t{(_Float16)1032.f, (_Float16)1032.f};
    }
    return __builtin_bit_cast(uint32_t, y);
}

// The word's eight nibbles as one A operand of the scores; slot order (elements)
// 0 4 1 5 2 6 3 7. EXACT: codes -8 .. 7. Otherwise unsigned subnormals, the odd
// elements 16 times the even ones' factor: half the instructions, but scores are then
// the difference of sum q u and 8 sum q and lose three bits in it (fp32 results
// were 2 to 7e-6 off in norm, 3 to 8e-7 with exact codes; bf16 ones do not show it).
template <bool EXACT> __device__ __forceinline__ f16x8_t nibbles_a(uint32_t w) {
    const uint32_t h = w >> 8;
    if constexpr (EXACT) {
        const u32v4_t f = {signed_pair(w, false), signed_pair(w, true), signed_pair(h, false), signed_pair(h, true)};
        return __builtin_bit_cast(f16x8_t, f);
    } else {
        const u32v4_t f = {w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u};
        return __builtin_bit_cast(f16x8_t, f);
    }
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

// The page table as one uniform walks it: entries are loaded well before they
// are used, without a branch (no table: any word is loaded, and not looked at).
struct KvTable {
    const_int_ptr row;
    int shift, last;  // of the positions
    __device__ __forceinline__ KvTable(const KvPages& c, int b) {
        row = (const_int_ptr)(c.table ? c.table + b * c.table_stride : c.lens);
        shift = c.table ? c.page_shift : 31;
        last = c.capacity - 1;
    }
    __device__ __forceinline__ int entry(int t) const { return row[min(t, last) >> shift]; }
};
__device__ __forceinline__ KvHalf kv_half(const KvPages& c, int b, int h, int t, int entry) {
    const int page = c.table ? entry : b;
    const int off = c.table ? t & (c.page_size - 1) : t;
    const bool good = t < c.capacity && (unsigned)page < (unsigned)c.num_pages;
    KvHalf r;
    r.vec = good ? ((int64_t)page * c.Hkv + h) * c.page_size + off : 0;
    r.n = good ? min(16, c.page_size - off) : 0;
    return r;
}

// Raw contents of one tile on one wavefront.
//   keys: word j of the lane's quarter of key 16 a + l % 16 (D / 32 words)
//   values: of key 16 a + 4 g + r (i = 4 a + r), the l % 16-th sixteenth of the
//           vector: 4, 8 or 16 nibbles
//   scale[a]: the scales of keys 16 a + 4 g .. + 3
template <int D> struct KvKeys {
    static constexpr int KW = D / 32, VB = D / 2;  // words a lane, bytes of a vector
    uint32_t w[2][KW];
    f32v4_t scale[2];

    __device__ __forceinline__ void load(const KvPages& c, const KvHalf* half, int lane) {
        const int l16 = lane & 15, g = lane >> 4;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const rsrc_t rk = make_rsrc(c.codes[0] + half[a].vec * VB, half[a].n * VB);
            if constexpr (D == 64) {
                const u32v2_t x = __builtin_amdgcn_raw_buffer_load_b64(rk, l16 * VB + 8 * g, 0, 0);
                w[a][0] = x[0], w[a][1] = x[1];
            } else {
#pragma unroll
                for (int q = 0; q < KW / 4; ++q) {
                    const u32v4_t x = __builtin_amdgcn_raw_buffer_load_b128(rk, l16 * VB + g * (VB / 4) + 16 * q, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[a][4 * q + j] = x[j];
                }
            }
            const rsrc_t rs = make_rsrc(c.scales[0] + half[a].vec, half[a].n * 4);
            scale[a] = __builtin_bit_cast(f32v4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * g, 0, 0));
        }
    }
};

template <int D> struct KvValues {
    static constexpr int VW = D == 256 ? 2 : 1, VB = D / 2;
    uint32_t w[8][VW];
    f32v4_t scale[2];

    __device__ __forceinline__ void load(const KvPages& c, const KvHalf* half, int lane) {
        const int l16 = lane & 15, g = lane >> 4;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const rsrc_t rs = make_rsrc(c.scales[1] + half[a].vec, half[a].n * 4);
            scale[a] = __builtin_bit_cast(f32v4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * g, 0, 0));
            const rsrc_t rv = make_rsrc(c.codes[1] + half[a].vec * VB, half[a].n * VB);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int off = 4 * g * VB + l16 * (VB / 16);
                if constexpr (D == 64) {
                    w[4 * a + r][0] = __builtin_amdgcn_raw_buffer_load_b16(rv, off + r * VB, 0, 0);
                } else if constexpr (D == 128) {
                    w[4 * a + r][0] = __builtin_amdgcn_raw_buffer_load_b32(rv, off + r * VB, 0, 0);
                } else {
                    const u32v2_t x = __builtin_amdgcn_raw_buffer_load_b64(rv, off + r * VB, 0, 0);
                    w[4 * a + r][0] = x[0], w[4 * a + r][1] = x[1];
                }
            }
        }
    }
};

// The A operands of O^T = V^T P^T: operand n of word m holds, for the lane's
// vector element 8 m + n (of its sixteenth), the 8 keys in k-slot order. The
// words of two keys meet by halves, so that a 32-bit AND cuts both keys' nibble
// of one element. Exact codes: unsigned subnormals and a term -8 sum P would be
// cheaper, but where the heaviest keys' code is 0 the result is the difference of
// two large sums.
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
            f[n][i] = signed_pair(x, n & 1);
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) out[n] = __builtin_bit_cast(f16x8_t, f[n]);
}

// Queries as B operands of S^T = K Q^T for the operands of nibbles_a<EXACT>. A
// column's vector is scaled by a power of two to 2^14 .. 2^15 at its largest element
// (odd elements to 1/16 of that for unsigned codes). PIECES = 1, for bf16 queries: exact;
// PIECES = 2: x = hi + lo, 11 bits each. Eight elements 8 u and up are one lane's operand of one k-step: lane group g = u / (D / 32), step
// u % (D / 32).
//   zero: the accumulator's start: -8 sum x turns unsigned codes into signed ones
//   c:    turns score * key scale into the exponent of 2
template <bool EXACT> struct KvScaling {
    int e;
    float sign;
    __device__ __forceinline__ KvScaling(float largest, float scale) {
        const bool some = largest > 0.f && scale != 0.f;
        e = some ? 14 - ilogbf(largest) : 0;
        sign = some ? copysignf(1.f, scale) : 0.f;
    }
    static __device__ __forceinline__ float zero(float sum) { return EXACT ? 0.f : -8.f * 0x1p-24f * sum; }
    // Finite and positive for any finite scale and query. Down to the least subnormal: scores times key
    // scales reach 2^123, and what c loses under 2^-126 is less than 2^-26 of the exponent even so.
    __device__ __forceinline__ float c(float scale) const {
        if (sign == 0.f) return 1.f;
        return fminf(fmaxf(ldexpf(fabsf(scale), (EXACT ? 0 : 24) - e) * 1.4426950408889634f, 0x1p-149f), 0x1p120f);
    }
    // one operand (and its share of sum x) from eight elements
    template <int PIECES>
    __device__ __forceinline__ float pieces(const float* x, f16x8_t (&f)[PIECES]) const {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int el = nibble_slot(i);
            const bool small = !EXACT && (el & 1);
            float y = sign * ldexpf(x[el], small ? e - 4 : e);
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                f[p][i] = (_Float16)y;
                const float r = (float)f[p][i];
                sum += small ? 16.f * r : r;
                y -= r;
            }
        }
        return sum;
    }
};

// By the whole workgroup in LDS: 16 threads a column, 16 NC columns by 256
// threads; row(col) gives the column's vector or null. In two steps, so that the
// loads are on their way while the first tile is found.
template <int D, int NC, int PIECES> struct KvQueries {
    f16x8_t frag[PIECES][NC][D / 32][64];  // [..][k-step][lane]
};
template <int D, int NC> struct KvRawQueries {
    static constexpr int UNITS = D / 8, PER = (UNITS + 15) / 16;
    float x[NC][PER][8];

    template <typename F> __device__ __forceinline__ void load(F row) {
        const int part = threadIdx.x & 15, col = threadIdx.x >> 4;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const auto* q = row(16 * n + col);
#pragma unroll
            for (int k = 0; k < PER; ++k) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[n][k][i] = 0.f;
                if (q && part + 16 * k < UNITS) load8(q + 8 * (part + 16 * k), x[n][k]);
            }
        }
    }

    template <bool EXACT, int PIECES>
    __device__ __forceinline__ void finish(KvQueries<D, NC, PIECES>& out, float* zero, float* cs, float scale) const {
        constexpr int KW = D / 32;
        const int part = threadIdx.x & 15, col = threadIdx.x >> 4;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < PER; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[n][k][i]));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
            const KvScaling<EXACT> sc(m, scale);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int u = part + 16 * k;
                f16x8_t f[PIECES];
                sum += sc.template pieces<PIECES>(x[n][k], f);
                if (u < UNITS) {
#pragma unroll
                    for (int p = 0; p < PIECES; ++p) out.frag[p][n][u % KW][16 * (u / KW) + col] = f[p];
                }
            }
            if constexpr (!EXACT) {
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor(sum, o);
            }
            if (part == 0) {
                zero[16 * n + col] = sc.zero(sum);
                cs[16 * n + col] = sc.c(scale);
            }
        }
    }
};

// By the wavefront in registers, for exact codes: a column's four lanes take a
// quarter each; q is the column's vector or null.
template <int D, int PIECES, typename T>
__device__ __forceinline__ void load_query(const T* q, int g, float scale, f16x8_t (&frag)[PIECES][D / 32], float& c) {
    constexpr bool EXACT = true;
    float x[D / 4], m = 0.f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
    if (q) {
#pragma unroll
        for (int w = 0; w < D / 32; ++w) load8(q + g * (D / 4) + 8 * w, x + 8 * w);
    }
#pragma unroll
    for (int i = 0; i < D / 4; ++i) m = fmaxf(m, fabsf(x[i]));
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const KvScaling<EXACT> sc(m, scale);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        f16x8_t f[PIECES];
        sc.template pieces<PIECES>(x + 8 * w, f);
#pragma unroll
        for (int p = 0; p < PIECES; ++p) frag[p][w] = f[p];
    }
    c = sc.c(scale);
}

// ---------------------------------------------------------------- the running softmax
// With x the score times the key's scale (one fma with the reference mx) weights
// are 2^((x - mx) c): exactly 1 at the reference, however large x c is. mx
// follows the maximum lazily, once a weight would pass 2^kLift, so that most
// tiles scale nothing.
constexpr float kLift = 4.f;
// Weights times value scales, y = p s_v, enter the second product as 16-bit floats, times
// a power of two of the column's own, rv. It is set where the reference moves, or where a y
// would reach 2^15, so that the largest y so far stands at 2^kBoost: what the format's
// least step drops is 2^-33 of the largest y of the column. Values that a column does not
// see, or gives no weight, do not move it: a row's result depends on nothing but what it sees.
constexpr int kBoost = 8;
constexpr float kTop = 15.f;  // log2 of what y rv stays below

// p times a value scale, 0 where p is 0: a hidden key's scale may be infinite or NaN. (The
// instruction v_mul_legacy_f32 by the intrinsic's name: in inline assembly the compiler would not keep it
// a cycle away from the exponential before it.)
__device__ float kv_weigh(float p, float scale) __asm("llvm.amdgcn.fmul.legacy");

// The largest of a column's four lanes (l, l ^ 16, l ^ 32, l ^ 48), on each of them.
__device__ __forceinline__ float column_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// One wavefront's NC column tiles; NO operands of 16 output elements each.
template <int NC, int PIECES, int NO> struct KvSoftmax {
    float mx[NC], thr[NC], l[NC];  // thr -inf: nothing seen so far; l: this lane's keys only
    float rv[NC];                  // 2^-119 .. 2^126: it and its inverse are normal
    f32v4_t o[NC][NO];

    __device__ __forceinline__ void start() {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            thr[n] = -INFINITY;
            mx[n] = l[n] = 0.f;
            rv[n] = 0x1p126f;
#pragma unroll
            for (int i = 0; i < NO; ++i) o[n][i] = f32v4_t{0.f, 0.f, 0.f, 0.f};
        }
    }

    // z: scores in, relative to mx out
    __device__ __forceinline__ void scale(f32v4_t (&z)[NC][2], const f32v4_t (&ks)[2]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int n = 0; n < NC; ++n) z[n][h][r] = fmaf(z[n][h][r], ks[h][r], -mx[n]);
    }
    // The same where rows end or pages are missing: keys t0 .. t0 + 31, of which n0 and n1
    // of the halves are there, columns at pos that see t <= pos and t > low or t < sinks.
    // Scales of keys that no column sees may be stale, any bits: they become 0.
    __device__ __forceinline__ void scale_masked(f32v4_t (&z)[NC][2], f32v4_t (&ks)[2], f32v4_t (&vs)[2], int t0, int g,
                                                 int n0, int n1, int p_hi, int low_any, int sinks,
                                                 const int (&pos)[NC], const int (&low)[NC]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int idx = 4 * g + r, t = t0 + 16 * h + idx;
                const bool there = idx < (h ? n1 : n0) && t <= p_hi && (t > low_any || t < sinks);
                ks[h][r] = there ? ks[h][r] : 0.f;
                vs[h][r] = there ? vs[h][r] : 0.f;
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    const bool see = there && t <= pos[n] && (t > low[n] || t < sinks);
                    z[n][h][r] = see ? fmaf(z[n][h][r], ks[h][r], -mx[n]) : -INFINITY;
                }
                __builtin_amdgcn_sched_barrier(0);  // few masks at a time: scalar registers
            }
    }

    // Weights of a tile, as operands of the second product.
    __device__ __forceinline__ void weights(f32v4_t (&z)[NC][2], const f32v4_t (&vs)[2], const float (&c)[NC],
                                            f16x8_t (&pf)[NC][PIECES]) {
        float top[NC], big = fabsf(vs[0][0]);
        bool move = false;
#pragma unroll
        for (int i = 1; i < 8; ++i) big = fmaxf(big, fabsf(vs[i >> 2][i & 3]));
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            top[n] = z[n][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top[n] = fmaxf(top[n], z[n][i >> 2][i & 3]);
            // weights are at most 2^kLift where the reference stays
            move = move | (top[n] > thr[n]) | (big * rv[n] >= 0x1p11f);
        }
        if (__builtin_amdgcn_ballot_w64(move) != 0) {  // rarely, but where values of little weight are large
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                // the largest weight times the largest scale of the lane's keys bounds their y
                const bool far = fmaf(top[n], c[n], __builtin_amdgcn_logf(big * rv[n])) >= kTop;
                if (__builtin_amdgcn_ballot_w64(top[n] > thr[n] | far) == 0) continue;
                // decisions are alike on the column's four lanes, and do not depend on other columns
                const float t = column_max(top[n]);
                float f = 1.f, fv = 1.f;
                const bool moved = t > thr[n];
                if (moved) {
                    const float to = mx[n] + t, by = to - mx[n];
                    f = thr[n] > -INFINITY ? __builtin_amdgcn_exp2f(-by * c[n]) : 0.f;
                    mx[n] = to;
                    thr[n] = kLift / c[n];
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[n][i >> 2][i & 3] -= by;
                }
                float y = 0.f, cn = c[n];
                asm("" : "+v"(cn));  // other exponentials than those below, which would wait in registers
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y = fmaxf(y, kv_weigh(__builtin_amdgcn_exp2f(z[n][i >> 2][i & 3] * cn), fabsf(vs[i >> 2][i & 3])));
                y = column_max(y);
                if (moved || y * rv[n] >= 0x1p15f) {
                    // the largest so far: 2^kBoost / rv when rv was set, less what the reference moved
                    const float inv = __uint_as_float((254u << 23) - __float_as_uint(rv[n]));  // 1 / rv
                    const int e = min(max(ilogbf(fmaxf((0x1p8f * inv) * f, y)), -118), 127);
                    const float r = ldexpf(1.f, kBoost - e);
                    fv = fminf(r * inv, 0x1p127f);  // a power of two
                    rv[n] = r;
                }
                l[n] *= f;
                f *= fv;
#pragma unroll
                for (int i = 0; i < NO; ++i) o[n][i] *= f;
            }
        }
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float y[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float p = __builtin_amdgcn_exp2f(z[n][(i + u) >> 2][(i + u) & 3] * c[n]);
                    l[n] += p;
                    y[u] = kv_weigh(p, vs[(i + u) >> 2][(i + u) & 3]) * rv[n];
                    // one fp32 value for both pieces: a product fused into one of the conversions
                    // would round another way and lose the second piece
                    if constexpr (PIECES == 2) asm("" : "+v"(y[u]));
                }
#pragma unroll
                for (int p = 0; p < PIECES; ++p) {
                    const f16x2_t v = {(_Float16)y[0], (_Float16)y[1]};  // to nearest
                    pf[n][p][i] = v[0];
                    pf[n][p][i + 1] = v[1];
                    y[0] -= (float)v[0];
                    y[1] -= (float)v[1];
                }
            }
    }

    // The exponent of 2 that a column's weights are relative to; -inf: nothing seen, NaN: no score but NaN.
    // (After total: a NaN score does not move the reference, and shows in the sum.)
    __device__ __forceinline__ float reference(int n, float c) const {
        return thr[n] > -INFINITY ? mx[n] * c : l[n] == 0.f ? -INFINITY : l[n];
    }

    // the whole sum of a column, on its four lanes
    __device__ __forceinline__ void total() {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            l[n] += __shfl_xor(l[n], 16);
            l[n] += __shfl_xor(l[n], 32);
        }
    }
};

// log sum exp from the reference (an exponent of 2) and the sum relative to it; a sum of 0: nothing
// seen. NaN stays NaN.
__device__ __forceinline__ float kv_lse(float top, float sum) {
    return sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

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
