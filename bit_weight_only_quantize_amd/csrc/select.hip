// Selection of experts from router logits.
//
// Scores s = softmax(l) or sigmoid(l), choice values c = s + bias. Values lie close together (two of
// 256 experts' are within a unit in the last place of fp32 of each other about once in ten
// thousand tokens), and choices are those of 64-bit arithmetic. A wavefront takes a token:
//   * Without a bias the choice is made on the logits, exactly; group values of one expert too.
//   * Otherwise values are computed in fp32, with a bound on their errors, and every
//     decision (each chosen expert against the next, kept groups against the best other one) has to
//     have a margin beyond it. A token without (ties, mostly) is done again in 64 bits.
// Sorting is k rounds of a wave-wide maximum over 32-bit keys; a lane holds consecutive experts, so the
// first lane with the maximum has the lowest index. Bound by its dependent steps and instruction issue (920 vector
// instructions a token): 8192 tokens, 256 experts in
// 8 groups, top 8, sigmoid with bias: 18 to 20 us (27 with everything in 64 bits; 1.7 for the bytes). Finding the k-th key bit by
// bit with ballots instead of the rounds, and ranking what it leaves, took 26.
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
__device__ __forceinline__ uint32_t order_key(float v) {
    const int32_t b = __float_as_int(v + 0.f);
    return b < 0 ? ~(uint32_t)b : (uint32_t)b | (1u << 31);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); }

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

// LDS written by this wavefront's lanes, before others of them read it
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <bool BF16>
__device__ __forceinline__ float logit(const SelectArgs& a, int64_t m, int e) {
    const int64_t at = m * a.row_stride + e;
    return BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
}

// A token with everything in 64 bits; lane holds the experts lane + 64 j. values: [64 EPL] in LDS. NaN logits
// count as masked, so that they stay out of the softmax's sum.
template <int EPL, bool BF16>
__device__ void select_exact(const SelectArgs& a, int64_t m, double* values) {
    const int lane = threadIdx.x & 63;
    float l[EPL];
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + 64 * j;
        const float v = logit<BF16>(a, m, min(e, a.E - 1));
        l[j] = e < a.E && v == v ? v : -INFINITY;
        mx = fmaxf(mx, l[j]);
    }
    mx = wave_max_dpp(mx);
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
        const int size = a.size;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 64 * j;
            if (e < a.E) values[e] = !(l[j] > -INFINITY) ? -INFINITY : p[j] + (a.bias ? (double)a.bias[e] : 0.0);
        }
        wave_lds_sync();
        // 1 << share lanes scan a group, then merge their two largest; the first of them speaks for it
        const int share = 1 << a.share, group = lane >> a.share;
        double b0 = -INFINITY, b1 = -INFINITY;
        if (group < a.groups)
            for (int i = lane & (share - 1); i < size; i += share) {
                const double x = values[group * size + i];
                if (x > b0) { b1 = b0; b0 = x; }
                else if (x > b1) b1 = x;
            }
        for (int o = 1; o < share; o *= 2) {
            const double o0 = __shfl_xor(b0, o, 64), o1 = __shfl_xor(b1, o, 64);
            b1 = o0 > b0 ? (b0 > o1 ? b0 : o1) : (b1 > o0 ? b1 : o0);
            b0 = o0 > b0 ? o0 : b0;
        }
        const double v = a.best == 2 ? b0 + b1 : b0;
        uint64_t gk = (lane & (share - 1)) == 0 && group < a.groups ? (v > -INFINITY ? order_key(v) : 1) : 0;
        uint64_t kept = 0;
        for (int r = 0; r < a.top_groups; ++r) {
            const uint64_t best = wave_max_u64(gk);
            const int at = wave_min_dpp(gk == best ? lane : 0x7FFFFFFF);
            kept |= 1ull << (at >> a.share);
            if (lane == at) gk = 0;
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
        a.weights[m * a.k + lane] = (float)(w * (double)a.scale);
    }
}

// Errors of the fp32 values, in units u = 2^-23. y = (l - max) log2 e is off by 1.2 u |y|, so the power by
// 2^y (0.8 |y| + 1) u of its own, at most 1.1 u. Their sum S >= 1 is off by up to (0.8 |y| + 1) u of each summand (5 and 1 u of
// S at the worst, most of 1024 logits some 8 binades below the largest) and 22 additions (11 u), its reciprocal by half a
// unit: a factor 1 + d common to all scores, |d| < 18 u. Two scores' difference is then off by d times itself, at most 18 u / S, and by
// their own errors, 2 (1.1 + 0.5 for the product) u / S: 22 u / S, under the 2 kSoftmaxOff / S = 32 u / S that a decision
// between two asks for. Sums of two scores: 36 + 7 u / S, under 4 kSoftmaxOff. A sigmoid s has s (1 - s) times the power's
// relative error, and units for the sum and the reciprocal: within 2^-21. c's rounding: 2^-24 |c|.
constexpr float kSoftmaxOff = 0x1p-19f, kSigmoidOff = 0x1p-21f;  // (the first divided by S)

constexpr int kSelectWaves = 4;

template <int EPL, bool BF16>
__global__ __launch_bounds__(64 * kSelectWaves) void moe_select_kernel(SelectArgs a) {
    __shared__ double all[kSelectWaves][64 * EPL];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    double* values = all[wave];
    const int64_t m = (int64_t)blockIdx.x * kSelectWaves + wave;
    if (m >= a.M) return;  // wavefronts share nothing
    float l[EPL], c[EPL];
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane * EPL + j;
        const float v = logit<BF16>(a, m, min(e, a.E - 1));
        l[j] = e < a.E ? v : -INFINITY;
        nan |= e < a.E && v != v;
        mx = fmaxf(mx, l[j]);
    }
    if (__any(nan)) {  // NaN experts are masked, and every weight is NaN
        select_exact<EPL, BF16>(a, m, values);
        if (lane < a.k) a.weights[m * a.k + lane] = NAN;
        return;
    }
    const bool grouped = a.groups > 1, by_logit = !a.bias;
    const bool need_sum = !a.sigmoid, need_scores = a.bias || (grouped && a.best == 2);
    float inv = 1.f, off = kSigmoidOff;
    if (need_sum) {
        mx = wave_max_dpp(mx);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            c[j] = __builtin_amdgcn_exp2f(1.4426950408889634f * (l[j] - mx));  // -infinity gives 0
            sum += c[j];
        }
        sum = wave_sum_dpp(sum);
        inv = mx > -INFINITY ? 1.f / sum : 0.f;
        off = kSoftmaxOff * inv;
    }
    if (need_scores) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float s = a.sigmoid ? __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * l[j])) : c[j] * inv;
            const int e = lane * EPL + j;
            c[j] = !(l[j] > -INFINITY) ? -INFINITY : a.bias && e < a.E ? s + a.bias[e] : s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) c[j] = l[j];
    }
    bool close = false;  // some decision is within the errors; an infinite or NaN c compares so too
    uint64_t kept = ~0ull;
    const int size = a.size;
    const float per = 1.f / (float)size;  // (e + .5) per: its integer part is e / size, as e < 1024
    if (grouped) {
        // `share` lanes (a power of two) scan a group, then merge their two largest
        float* vals = reinterpret_cast<float*>(values);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane * EPL + j;
            if (e < a.E) vals[e] = c[j];
        }
        wave_lds_sync();
        const int share = 1 << a.share;
        const int g = lane >> a.share;
        float b0 = -INFINITY, b1 = -INFINITY, big = 0.f;
        if (g < a.groups)
            for (int i = lane & (share - 1); i < size; i += share) {
                const float x = vals[g * size + i];
                b1 = fmaxf(b1, fminf(b0, x));
                b0 = fmaxf(b0, x);
            }
        for (int o = 1; o < share; o *= 2) {
            const float o0 = __shfl_xor(b0, o, 64), o1 = __shfl_xor(b1, o, 64);
            b1 = fmaxf(fmaxf(b1, o1), fminf(b0, o0));
            b0 = fmaxf(b0, o0);
        }
        const float v = a.best == 2 ? b0 + b1 : b0;
        if (need_scores) {
            big = b0 > -INFINITY ? fabsf(b0) : 0.f;
            if (a.best == 2 && b1 > -INFINITY) big = fmaxf(big, fabsf(b1));
            big = wave_max_dpp(big);
            close |= v != v;
        }
        // (lane & (share - 1)) == 0 speaks for group g
        uint32_t gk = (lane & (share - 1)) == 0 && g < a.groups ? (v > -INFINITY ? order_key(v) : 1u) : 0u;
        uint32_t last = 0;
        kept = 0;
        for (int r = 0; r < a.top_groups; ++r) {
            last = wave_max_u(gk);
            const int at = __ffsll((unsigned long long)__ballot(gk == last)) - 1;
            kept |= 1ull << (at >> a.share);
            if (lane == at) gk = 0;
        }
        const uint32_t next = wave_max_u(gk);
        if (next > 1 && last > 1) {
            const float p = key_value(last), q = key_value(next);
            if (need_scores) close |= !(p - q > 4.f * off + 0x1p-21f * big);
            // logits of the best experts order their scores; but where scores saturate in 64 bits, or
            // logits differ by next to nothing, equal scores of different logits are a tie
            else close |= p != q && (p - q < 0x1p-30f || q < (a.sigmoid ? -600.f : mx - 600.f) || (a.sigmoid && q > 16.f));
        }
    }
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane * EPL + j;
        const float v = by_logit ? l[j] : c[j];
        const bool can = e < a.E && (!grouped || ((kept >> (int)(((float)e + 0.5f) * per)) & 1));
        if (!by_logit) close |= v != v;
        key[j] = !can ? 0u : l[j] > -INFINITY ? order_key(v) : 1u;
    }
    int id = 0;
    uint32_t prev = 0;
    for (int r = 0; r <= a.k; ++r) {
        uint32_t b = key[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j) b = max(b, key[j]);
        const uint32_t best = wave_max_u(b);
        if (!by_logit && r > 0 && prev > 1 && best > 1) {
            const float p = key_value(prev), q = key_value(best);
            close |= !(p - q > 2.f * off + 0x1p-22f * fmaxf(fabsf(p), fabsf(q)));
        }
        prev = best;
        if (r == a.k) break;
        const int at = __ffsll((unsigned long long)__ballot(b == best)) - 1;
        int j = 0;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i) j = key[i] == best ? i : j;
        j = __builtin_amdgcn_readlane(j, at);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane == at && i == j) key[i] = 0;
        if (lane == r) id = at * EPL + j;
    }
    if (__any(close)) {
        select_exact<EPL, BF16>(a, m, values);
        return;
    }
    // the chosen experts' scores in 64 bits, each by its lane
    double w = 0, total = 0;
    if (lane < a.k) {
        const float x = logit<BF16>(a, m, id);
        if (x > -INFINITY) w = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)mx) * (double)inv;
    }
    if (a.renormalize) {
        total = w;
        for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor(total, o, 64);  // k <= 32 lanes
        w = total > 0 ? w / total : 0.0;
    }
    if (lane < a.k) {
        a.ids[m * a.k + lane] = id;
        a.weights[m * a.k + lane] = (float)(w * (double)a.scale);
    }
}

hipError_t launch_moe_select(SelectArgs a, bool bf16, hipStream_t st) {
    a.size = a.E / a.groups;
    a.share = 0;
    while (2 * (a.groups << a.share) <= 64) ++a.share;
    constexpr int64_t kMost = 1 << 25;  // tokens of a launch, 64 threads each
    if (a.M > kMost) {
        SelectArgs b = a;
        b.M = kMost;
        if (const hipError_t e = launch_moe_select(b, bf16, st)) return e;
        b.M = a.M - kMost;
        b.logits = static_cast<const char*>(a.logits) + kMost * a.row_stride * (bf16 ? 2 : 4);
        b.ids += kMost * a.k;
        b.weights += kMost * a.k;
        return launch_moe_select(b, bf16, st);
    }
    const dim3 grid((unsigned)((a.M + kSelectWaves - 1) / kSelectWaves)), block(64 * kSelectWaves);
#define W4_SELECT(EPL)                                                                                   \
    if (a.E <= 64 * EPL) {                                                                               \
        if (bf16) hipLaunchKernelGGL((moe_select_kernel<EPL, true>), grid, block, 0, st, a);             \
        else hipLaunchKernelGGL((moe_select_kernel<EPL, false>), grid, block, 0, st, a);                 \
        return hipGetLastError();                                                                        \
    }
    W4_SELECT(1)
    W4_SELECT(2)
    W4_SELECT(4)
    W4_SELECT(16)
#undef W4_SELECT
    return hipErrorInvalidValue;
}

}  // namespace w4
