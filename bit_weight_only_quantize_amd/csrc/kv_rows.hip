// Rows in and out of the batched INT4 KV cache: w4_kv_write and w4_kv_read.
//
// Codec (Shimmy article, §3.2), per head vector x of D values:
//   s = max|x| / 7.5 (fp32),  c_i = clamp(round(x_i / s), -8, 7) (halves away
//   from zero, fp32 quotient),  nibble c_i + 8;  s = 0: every nibble 8.
// Read back: (nibble - 8) * s, one fp32 rounding, then the row type's.
//
// Both are bound by memory: a bf16 vector of 128 is 256 bytes on one side and
// 68 on the other. Eight values a lane, so D / 8 lanes share a vector: 16 bytes
// of bf16 (or two times 16 of fp32) on the row side, one 32-bit word of codes on
// the cache side. Consecutive lane groups take consecutive rows of one head,
// whose codes and scales are neighbours in the cache; a row tensor's vectors are
// 128 bytes or more by themselves.
#include "common.hpp"
#include "kv_pages.hpp"
#include "kv_attention.hpp"

namespace w4 {

struct KvRowsArg {  // the row tensors of keys and values; null: not wanted
    void* data[2];
    int64_t row_stride[2], head_stride[2];
};

// Which head vector a group of lanes handles: grid (sequence, chunk, K or V).
struct KvSpot {
    int64_t vec;  // in the cache, -1: none
    int row, head;
    bool live;
};
__device__ __forceinline__ KvSpot kv_spot(const KvPages& c, const KvSeq& s, int b, int64_t v) {
    KvSpot p;
    p.live = v < (int64_t)s.n * c.Hkv;
    const int h = p.live ? (int)(v / s.n) : 0;
    const int i = p.live ? (int)(v - (int64_t)h * s.n) : 0;
    const int t = s.len - s.n + i;
    p.row = s.first + i;
    p.head = h;
    p.vec = p.live && t >= 0 ? kv_vector(c, b, h, t) : -1;
    return p;
}

template <int LANES>  // max over aligned groups of 8, 16 or 32 lanes
__device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    return m;
}

template <int D, typename T>
__global__ __launch_bounds__(256) void kv_write_kernel(KvPages c, KvRowsArg a, int chunks) {
    constexpr int LANES = D / 8, VECS = 256 / LANES;
    const int kv = blockIdx.y;
    if (!a.data[kv]) return;
    const int b = blockIdx.x / chunks, chunk = blockIdx.x - b * chunks;
    const KvSeq s = kv_seq(c, b);
    const int l = threadIdx.x % LANES;
    for (int64_t v = (int64_t)chunk * VECS + threadIdx.x / LANES; v < (int64_t)s.n * c.Hkv;
         v += (int64_t)chunks * VECS) {
        const KvSpot p = kv_spot(c, s, b, v);
        const T* x = static_cast<const T*>(a.data[kv]) + p.row * a.row_stride[kv] + p.head * a.head_stride[kv];
        float e[8];
        load8(x + 8 * l, e);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(e[i]));
        m = lanes_max<LANES>(m);
        const float sc = m / 7.5f;
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = sc > 0.f ? fminf(fmaxf(roundf(e[i] / sc), -8.f), 7.f) : 0.f;
            w |= (uint32_t)((int)q + 8) << (4 * i);
        }
        if (p.vec >= 0) {
            reinterpret_cast<uint32_t*>(c.codes[kv] + p.vec * (D / 2))[l] = w;
            if (l == 0) c.scales[kv][p.vec] = sc;
        }
    }
}

template <int D, typename T>
__global__ __launch_bounds__(256) void kv_read_kernel(KvPages c, KvRowsArg a, int chunks) {
    constexpr int LANES = D / 8, VECS = 256 / LANES;
    const int kv = blockIdx.y;
    if (!a.data[kv]) return;
    const int b = blockIdx.x / chunks, chunk = blockIdx.x - b * chunks;
    const KvSeq s = kv_seq(c, b);
    const int l = threadIdx.x % LANES;
    for (int64_t v = (int64_t)chunk * VECS + threadIdx.x / LANES; v < (int64_t)s.n * c.Hkv;
         v += (int64_t)chunks * VECS) {
        const KvSpot p = kv_spot(c, s, b, v);
        uint32_t w = 0x88888888u;  // no position: zeros
        float sc = 0.f;
        if (p.vec >= 0) {
            w = reinterpret_cast<const uint32_t*>(c.codes[kv] + p.vec * (D / 2))[l];
            sc = c.scales[kv][p.vec];
        }
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = (float)((int)((w >> (4 * i)) & 15u) - 8) * sc;
        store_run<8>(static_cast<T*>(a.data[kv]) + p.row * a.row_stride[kv] + p.head * a.head_stride[kv] + 8 * l, e);
    }
}

// ---------------------------------------------------------------- host side
namespace {
template <int D, typename T>
hipError_t launch_rows(bool write, const KvPages& c, const KvRowsArg& a, int max_rows, hipStream_t st) {
    constexpr int VECS = 256 / (D / 8);
    // one vector a lane group; sequences with more rows than max_rows loop
    int64_t chunks = ((int64_t)max_rows * c.Hkv + VECS - 1) / VECS;
    chunks = chunks < 1 ? 1 : chunks;
    const int64_t most = 0x3fffffffLL / c.B;
    chunks = chunks > most ? most : chunks;
    const dim3 grid((unsigned)(c.B * chunks), 2);
    if (write)
        hipLaunchKernelGGL((kv_write_kernel<D, T>), grid, dim3(256), 0, st, c, a, (int)chunks);
    else
        hipLaunchKernelGGL((kv_read_kernel<D, T>), grid, dim3(256), 0, st, c, a, (int)chunks);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_kv_rows(bool write, int D, bool bf16, const KvPages& c, void* const* data,
                          const int64_t* row_stride, const int64_t* head_stride, int max_rows,
                          hipStream_t st) {
    KvRowsArg a;
    for (int i = 0; i < 2; ++i) {
        a.data[i] = data[i];
        a.row_stride[i] = row_stride[i];
        a.head_stride[i] = head_stride[i];
    }
    switch (D * 2 + (bf16 ? 1 : 0)) {
        case 128: return launch_rows<64, float>(write, c, a, max_rows, st);
        case 129: return launch_rows<64, __bf16>(write, c, a, max_rows, st);
        case 256: return launch_rows<128, float>(write, c, a, max_rows, st);
        case 257: return launch_rows<128, __bf16>(write, c, a, max_rows, st);
        case 512: return launch_rows<256, float>(write, c, a, max_rows, st);
        case 513: return launch_rows<256, __bf16>(write, c, a, max_rows, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace w4
