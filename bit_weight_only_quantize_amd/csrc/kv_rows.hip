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
// the cache side. A workgroup's lane groups take 2^rb consecutive rows of one head
// (whose codes and scales are neighbours in the cache) and walk over heads: the
// rows' vectors of all heads, neighbours in a [row][head] tensor, are touched
// within a short time.
#include "common.hpp"
#include "kv_attention.hpp"

namespace w4 {

struct KvRowsArg {  // the row tensors of keys and values; null: not wanted
    void* data[2];
    int64_t row_stride[2], head_stride[2];
};

// How a launch is laid out over (sequence, chunk of 2^rb rows, chunk of heads).
struct KvRowsGrid {
    int row_chunks, head_chunks;  // in the grid; longer sequences loop
    int rb;                       // log2 of the rows side by side
    int heads;                    // heads of a chunk
};

template <int LANES>  // over aligned groups of 8, 16 or 32 lanes
__device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    return m;
}

// One lane's eight codes as a word, from its values and its vector's scale.
// The codec rounds the correctly rounded fp32 quotient |x| / s. Dividing costs some
// twenty instructions a value, and the kernel would be bound by them; instead
// |x| * rcp(s) + 0.5, good to 2e-6, names the nearest border h = k - 0.5 between two codes,
// and which side of it the rounded quotient falls on is decided exactly: fl(|x| / s) >= h
// exactly when |x| / s >= h - d, d half a step below h (h's last bit is 0, so the middle rounds up to
// it), that is when |x| - h s, one fma and exact near 0, is at least -d s. d is 2^-24 of
// the power of two at or under the float before h. Scales under 2^-60, whose products
// with d would leave the format, are raised by 2^64 with their values (exact).
// 20209 rows of 8 + 8 bf16 heads of 128: 28 us (3.7 TB/s of what it has to move), with
// true divisions 43.
__device__ __forceinline__ uint32_t kv_codes(float (&e)[8], float s) {
    if (__builtin_amdgcn_ballot_w64(s < 0x1p-60f) != 0) {
        const float f = s < 0x1p-60f ? 0x1p64f : 1.f;
        s *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] *= f;
    }
    const float r = __builtin_amdgcn_rcpf(s), ds = s * -0x1p-24f;
    float half[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float k = rintf(fabsf(e[i] * r) + 0.5f), h = k - 0.5f;
        const float d = __uint_as_float((__float_as_uint(h) - 1u) & 0x7F800000u) * ds;
        const float q = fmaf(-h, s, fabsf(e[i])) >= d ? k : k - 1.f;
        half[i >> 2] = fmaf(__builtin_amdgcn_fmed3f(copysignf(q, e[i]), -8.f, 7.f), (float)(1 << (4 * (i & 3))),
                            half[i >> 2]);
    }
    // sums of q 16^i, i < 4: exact, and 8 in every nibble makes them unsigned
    const uint32_t w = (uint32_t)((int)half[0] + 0x8888) | ((uint32_t)((int)half[1] + 0x8888) << 16);
    return s > 0.f ? w : 0x88888888u;
}

// Lane groups of a workgroup: which row and head, and where in the cache.
template <int D, bool WRITE, typename T>
__global__ __launch_bounds__(256) void kv_rows_kernel(KvPages c, KvRowsArg a, KvRowsGrid grid) {
    constexpr int LANES = D / 8, VECS = 256 / LANES, AHEAD = 4;
    const int kv = blockIdx.y;
    if (!a.data[kv]) return;
    int x = blockIdx.x;
    const int hc = x % grid.head_chunks;
    x /= grid.head_chunks;
    const int b = x / grid.row_chunks, rc = x - b * grid.row_chunks;
    const KvSeq s = kv_seq(c, b);
    const int l = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int step = VECS >> grid.rb;  // heads side by side
    const int h1 = min((hc + 1) * grid.heads, c.Hkv);
    T* const data = static_cast<T*>(a.data[kv]) + 8 * l;
    for (int64_t r0 = (int64_t)rc << grid.rb; r0 < s.n; r0 += (int64_t)grid.row_chunks << grid.rb) {
        const int i = (int)r0 + (slot & ((1 << grid.rb) - 1));
        if (i >= s.n) continue;  // whole lane groups
        const int t = s.len - s.n + i;
        const int64_t first = t >= 0 ? kv_vector(c, b, 0, t) : -1;  // head h: + h * page_size
        T* const row = data + (int64_t)(s.first + i) * a.row_stride[kv];
        const int h0 = hc * grid.heads + (slot >> grid.rb);
        for (int h = h0; h < h1; h += AHEAD * step) {
            if constexpr (WRITE) {
                float e[AHEAD][8];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k)
                    load8(row + (int64_t)min(h + k * step, h1 - 1) * a.head_stride[kv], e[k]);
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    if (h + k * step >= h1) break;
                    float m = fabsf(e[k][0]);  // fmaxf passes over NaN: a vector of nothing else has a NaN scale
#pragma unroll
                    for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(e[k][j]));
                    m = lanes_max<LANES>(m);
                    const float sc = m / 7.5f;
                    const uint32_t w = kv_codes(e[k], sc);
                    if (first >= 0) {
                        const int64_t vec = first + (int64_t)(h + k * step) * c.page_size;
                        reinterpret_cast<uint32_t*>(c.codes[kv] + vec * (D / 2))[l] = w;
                        if (l == 0) c.scales[kv][vec] = sc;
                    }
                }
            } else {
                uint32_t w[AHEAD];
                float sc[AHEAD];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    // no position: any vector is read, and not looked at
                    const int64_t vec = first >= 0 ? first + (int64_t)min(h + k * step, h1 - 1) * c.page_size : 0;
                    w[k] = reinterpret_cast<const uint32_t*>(c.codes[kv] + vec * (D / 2))[l];
                    sc[k] = c.scales[kv][vec];
                }
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    if (h + k * step >= h1) break;
                    float e[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        e[j] = first >= 0 ? (float)((int)((w[k] >> (4 * j)) & 15u) - 8) * sc[k] : 0.f;
                    store_run<8>(row + (int64_t)(h + k * step) * a.head_stride[kv], e);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- host side
namespace {
template <int D, typename T>
hipError_t launch_rows(bool write, const KvPages& c, const KvRowsArg& a, int64_t max_rows, hipStream_t st) {
    constexpr int VECS = 256 / (D / 8);
    KvRowsGrid g;
    g.rb = 0;
    while ((1 << g.rb) < VECS && (1 << g.rb) < max_rows) ++g.rb;
    const int step = VECS >> g.rb;
    const int64_t most = (1 << 22) / c.B;
    const int64_t rows = (max_rows + (1 << g.rb) - 1) >> g.rb;
    g.row_chunks = (int)(rows < 1 ? 1 : rows < most ? rows : most);
    // heads of a workgroup: as few as fill the chip with 8 workgroups a CU, up to eight steps
    const int64_t steps = (c.Hkv + step - 1) / step;
    int64_t per = (int64_t)c.B * g.row_chunks * steps / (256 * 8);
    per = per < 1 ? 1 : per > 8 ? 8 : per;
    const int64_t chunks = (steps + per - 1) / per;
    g.heads = (int)((steps + chunks - 1) / chunks) * step;  // alike, but for the last
    g.head_chunks = (c.Hkv + g.heads - 1) / g.heads;
    const int64_t x = (int64_t)c.B * g.row_chunks * g.head_chunks;
    if (x > 0x7fffffLL) {  // more heads a workgroup instead
        g.heads = c.Hkv;
        g.head_chunks = 1;
    }
    const dim3 grid((unsigned)((int64_t)c.B * g.row_chunks * g.head_chunks), 2);
    if (write)
        hipLaunchKernelGGL((kv_rows_kernel<D, true, T>), grid, dim3(256), 0, st, c, a, g);
    else
        hipLaunchKernelGGL((kv_rows_kernel<D, false, T>), grid, dim3(256), 0, st, c, a, g);
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
