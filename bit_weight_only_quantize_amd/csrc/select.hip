// Selection of experts from router logits.
//
// Scores s = softmax(l) or sigmoid(l), choice values c = s + bias. Scores lie close
// together (two of 256 experts' values are within a unit in the last place of fp32 about once in
// ten thousand tokens), so choices are made in 64 bits; without a bias they are made on the
// logits themselves, whose order the scores have.
#include "mx4.hpp"
#include "topk.hpp"

namespace w4 {

// A double as an unsigned integer of the same order; 0 and 1 stay free below
// every value: 0 an expert that cannot be chosen, 1 a masked one (logit -infinity,
// or NaN).
__device__ __forceinline__ uint64_t order_key(double v) {
    const int64_t b = __double_as_longlong(v + 0.0);  // -0 counts as 0
    return b < 0 ? ~(uint64_t)b : (uint64_t)b | (1ull << 63);
}

__device__ __forceinline__ uint32_t wave_max_u(uint32_t v) {
    return (uint32_t)wave_reduce_i((int)v, [](int a, int b) { return (uint32_t)a > (uint32_t)b ? a : b; });
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
    const uint32_t hi = wave_max_u((uint32_t)(v >> 32));
    const uint32_t lo = wave_max_u((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ double wave_sum_d(double v) {
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// One wavefront a token; lane holds the experts lane + 64 j.
template <int EPL, bool BF16>
__global__ __launch_bounds__(64) void moe_select_kernel(SelectArgs a) {
    const int lane = threadIdx.x;
    const int64_t m = blockIdx.x;
    __shared__ double gval[1024];
    float l[EPL];
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + 64 * j;
        const int64_t at = m * a.row_stride + min(e, a.E - 1);
        const float v = BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.logits)[at])
                             : static_cast<const float*>(a.logits)[at];
        l[j] = e < a.E ? v : -INFINITY;
        nan |= e < a.E && v != v;
        mx = fmaxf(mx, l[j]);
    }
    mx = wave_max_dpp(mx);
    nan = __any(nan);
    double p[EPL];
    double sum = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        p[j] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[j])) : exp((double)l[j] - (double)mx);
        if (mx == -INFINITY) p[j] = 0;
        sum += lane + 64 * j < a.E ? p[j] : 0.0;
    }
    if (!a.sigmoid) {
        sum = wave_sum_d(sum);
#pragma unroll
        for (int j = 0; j < EPL; ++j) p[j] = sum > 0 ? p[j] / sum : p[j];
    }
    uint64_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + 64 * j;
        const bool masked = !(l[j] > -INFINITY);
        const double c = a.bias && e < a.E ? p[j] + (double)a.bias[e] : a.bias ? 0.0 : (double)l[j];
        key[j] = e >= a.E ? 0 : masked || c != c ? 1 : order_key(c);
    }
    if (a.groups > 1) {
        const int size = a.E / a.groups;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 64 * j;
            if (e < a.E) gval[e] = !(l[j] > -INFINITY) ? -INFINITY : p[j] + (a.bias ? (double)a.bias[e] : 0.0);
        }
        __syncthreads();
        double v = 0;
        if (lane < a.groups) {
            double b0 = -INFINITY, b1 = -INFINITY;
            for (int i = 0; i < size; ++i) {
                const double x = gval[lane * size + i];
                if (x > b0) { b1 = b0; b0 = x; }
                else if (x > b1) b1 = x;
            }
            v = a.best == 2 ? b0 + b1 : b0;
        }
        uint64_t gk = lane < a.groups ? (v > -INFINITY ? order_key(v) : 1) : 0;
        uint64_t kept = 0;
        for (int r = 0; r < a.top_groups; ++r) {
            const uint64_t best = wave_max_u64(gk);
            const int g = wave_min_dpp(gk == best ? lane : 0x7FFFFFFF);
            kept |= 1ull << g;
            if (lane == g) gk = 0;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 64 * j;
            if (e < a.E && !((kept >> (e / size)) & 1)) key[j] = 0;
        }
    }
    // k rounds of the largest key, the lowest expert of equal ones
    int id = 0;
    double w = 0, total = 0;
    for (int r = 0; r < a.k; ++r) {
        uint64_t b = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) b = key[j] > b ? key[j] : b;
        const uint64_t best = wave_max_u64(b);
        int e = 0x7FFFFFFF;
#pragma unroll
        for (int j = EPL - 1; j >= 0; --j) e = key[j] == best ? lane + 64 * j : e;
        e = wave_min_dpp(e);
        double pe = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (e == lane + 64 * j) {
                pe = p[j];
                key[j] = 0;
            }
        pe = __shfl(pe, e & 63, 64);
        total += pe;
        if (lane == r) {
            id = e;
            w = pe;
        }
    }
    if (lane < a.k) {
        if (a.renormalize) w = total > 0 ? w / total : 0.0;
        a.ids[m * a.k + lane] = id;
        a.weights[m * a.k + lane] = nan ? NAN : (float)(w * (double)a.scale);
    }
}

hipError_t launch_moe_select(const SelectArgs& a, bool bf16, hipStream_t st) {
    const dim3 grid((unsigned)a.M), block(64);
#define W4_SELECT(EPL)                                                                                   \
    if (a.E <= 64 * EPL) {                                                                               \
        if (bf16) hipLaunchKernelGGL((moe_select_kernel<EPL, true>), grid, block, 0, st, a);             \
        else hipLaunchKernelGGL((moe_select_kernel<EPL, false>), grid, block, 0, st, a);                 \
        return hipGetLastError();                                                                        \
    }
    W4_SELECT(2)
    W4_SELECT(4)
    W4_SELECT(16)
#undef W4_SELECT
    return hipErrorInvalidValue;
}

}  // namespace w4
