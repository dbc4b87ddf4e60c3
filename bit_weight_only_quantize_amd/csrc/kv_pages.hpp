// The batched INT4 KV cache as the kernels see it: a pool of pages (codes
// [page][Hkv][page_size][D / 2], scales [page][Hkv][page_size]) and, per
// sequence, its length, its rows of the call and its pages. The arrays' contents
// come from the caller's device memory and are bounded here, once per use.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace w4 {

struct KvPages {  // passed to kernels by value
    uint8_t* codes[2];  // keys, values
    float* scales[2];
    int Hkv;
    int page_size;   // positions per page
    int page_shift;  // log2(page_size) with a table
    int num_pages;
    const int* lens;
    const int* starts;
    const int* table;
    int64_t table_stride;
    int capacity;  // positions a sequence can hold
    int B, rows;
    int even_rows;  // rows per sequence where starts is null
};

struct KvSeq {
    int first;  // its first row in the packed tensors
    int n;      // its rows
    int len;    // positions it holds
};

__device__ __forceinline__ KvSeq kv_seq(const KvPages& c, int b) {
    KvSeq s;
    if (c.starts) {
        s.first = min(max(c.starts[b], 0), c.rows);
        s.n = max(min(max(c.starts[b + 1], 0), c.rows) - s.first, 0);
    } else {
        s.first = b * c.even_rows;
        s.n = c.even_rows;
    }
    s.len = min(max(c.lens[b], 0), c.capacity);
    return s;
}

// Index of position t (0 <= t < capacity) of sequence b and kv head h among
// the pool's head vectors, or -1 where the table names no page of the pool.
__device__ __forceinline__ int64_t kv_vector(const KvPages& c, int b, int h, int t) {
    int page = b, off = t;
    if (c.table) {
        page = c.table[b * c.table_stride + (t >> c.page_shift)];
        off = t & (c.page_size - 1);
        if ((unsigned)page >= (unsigned)c.num_pages) return -1;
    }
    return ((int64_t)page * c.Hkv + h) * c.page_size + off;
}

// 8 consecutive values of a row tensor as floats, and back (bf16 rounded to
// nearest even, the row tensors' output type).
__device__ __forceinline__ void load8(const float* p, float* v) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __bf16* p, float* v) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// E consecutive results of a row tensor, E * sizeof(T) bytes aligned.
template <int E> __device__ __forceinline__ void store_run(float* p, const float* v) {
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int i = 0; i < E; i += 4)
            reinterpret_cast<float4*>(p)[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = v[i];
    }
}
// Two values to bf16, to nearest even by v_cvt_pk_bf16_f32: a NaN stays one whatever its mantissa
// (rounding by an integer addition would carry a mantissa of ones into the exponent and sign).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef float f2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
    const f2_t f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, b2_t));
}
template <int E> __device__ __forceinline__ void store_run(__bf16* p, const float* v) {
    uint32_t w[(E + 1) / 2];
#pragma unroll
    for (int i = 0; i < (E + 1) / 2; ++i) w[i] = bf16_pair(v[2 * i], 2 * i + 1 < E ? v[2 * i + 1] : 0.f);
    if constexpr (E % 8 == 0) {
#pragma unroll
        for (int i = 0; i < E / 2; i += 4)
            reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (E == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (E == 2) {
        *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
}

}  // namespace w4
