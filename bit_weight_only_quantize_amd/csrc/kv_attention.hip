// Attention over the batched INT4 KV cache (w4_kv_attention).
//
// Row at position p of a sequence, query head h, kv head g = h / (Hq / Hkv):
//   z_t = scale * s_k[t] * sum_i q[i] c_k[t][i]   over the visible t
//   out = sum_t exp(z_t) s_v[t] c_v[t] / sum_t exp(z_t)
// in one pass over the keys with a running maximum m and sum l of the softmax:
// a larger maximum scales what was summed before by exp(m_old - m_new).
#include "common.hpp"
#include "kv_attention.hpp"

namespace w4 {

// One wavefront per (row, query head): 64 keys at a time, one a lane, for the
// scores; then D / 64 output elements a lane over the same 64 values.
template <int D, typename TQ, typename TO>
__global__ __launch_bounds__(64) void kv_attention_kernel(KvPages c, KvAttn a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x;
    const int h = blockIdx.x % a.Hq, g = h / a.group;
    const int64_t item = blockIdx.x / a.Hq;
    const int b = (int)(item / a.max_rows);
    const KvSeq s = kv_seq(c, b);
    for (int i = (int)(item % a.max_rows); i < s.n; i += a.max_rows) {
        const int p = s.len - s.n + i;
        const TQ* q = static_cast<const TQ*>(a.q) + (int64_t)(s.first + i) * a.q_row + h * a.q_head;
        float m = -INFINITY, l = 0.f, o[E] = {};
        const int near = a.window > 0 ? max(0, p - a.window + 1) : 0;
        for (int t0 = 0; t0 <= p; t0 += 64) {
            if (t0 >= a.sinks && t0 + 63 < near) continue;
            const int t = t0 + lane;
            const bool see = t <= p && (t >= near || t < a.sinks);
            const int64_t vec = see ? kv_vector(c, b, g, t) : -1;
            float z = -INFINITY, sv = 0.f;
            if (vec >= 0) {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(c.codes[0] + vec * (D / 2));
                float d = 0.f;
                for (int j = 0; j < D / 8; ++j) {
                    const uint32_t u = w[j];
                    float e[8];
                    load8(q + 8 * j, e);
#pragma unroll
                    for (int k = 0; k < 8; ++k) d = fmaf(e[k], (float)((int)((u >> (4 * k)) & 15u) - 8), d);
                }
                z = d * c.scales[0][vec] * a.scale;
                sv = c.scales[1][vec];
            }
            const float top = fmaxf(m, wave_max(z));
            if (top == -INFINITY) continue;  // nothing visible so far
            const float f = m == -INFINITY ? 0.f : expf(m - top);
            const float e = vec >= 0 ? expf(z - top) : 0.f;
            const float pv = vec >= 0 ? e * sv : 0.f;
            m = top;
            l = l * f + e;
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] *= f;
            for (int j = 0; j < 64; ++j) {
                const int64_t vj = __shfl(vec, j);
                if (vj < 0) continue;
                const float pj = __shfl(pv, j);
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const int i2 = lane * E + k;
                    const uint8_t byte = c.codes[1][vj * (D / 2) + i2 / 2];
                    o[k] = fmaf(pj, (float)((int)((byte >> (4 * (i2 & 1))) & 15u) - 8), o[k]);
                }
            }
        }
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
        TO* out = static_cast<TO*>(a.out) + (int64_t)(s.first + i) * a.out_row + h * a.out_head;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const float r = l > 0.f ? o[k] / l : 0.f;
            if constexpr (sizeof(TO) == 2)
                reinterpret_cast<uint16_t*>(out)[lane * E + k] = (uint16_t)f32_to_bf16_rne(r);
            else
                out[lane * E + k] = r;
        }
        if (a.lse && lane == 0) a.lse[(int64_t)(s.first + i) * a.Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
    }
}

namespace {
template <int D, typename TQ>
hipError_t launch(const KvPages& c, const KvAttn& a, bool out_bf16, hipStream_t st) {
    const dim3 grid((unsigned)((int64_t)c.B * a.max_rows * a.Hq));
    if (out_bf16)
        hipLaunchKernelGGL((kv_attention_kernel<D, TQ, __bf16>), grid, dim3(64), 0, st, c, a);
    else
        hipLaunchKernelGGL((kv_attention_kernel<D, TQ, float>), grid, dim3(64), 0, st, c, a);
    return hipGetLastError();
}
}  // namespace

size_t kv_attention_workspace(const KvPages&, int, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_kv_attention(int D, bool q_bf16, bool out_bf16, const KvPages& c, const KvAttn& a,
                               hipStream_t st) {
    switch (D * 2 + (q_bf16 ? 1 : 0)) {
        case 128: return launch<64, float>(c, a, out_bf16, st);
        case 129: return launch<64, __bf16>(c, a, out_bf16, st);
        case 256: return launch<128, float>(c, a, out_bf16, st);
        case 257: return launch<128, __bf16>(c, a, out_bf16, st);
        case 512: return launch<256, float>(c, a, out_bf16, st);
        case 513: return launch<256, __bf16>(c, a, out_bf16, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace w4
