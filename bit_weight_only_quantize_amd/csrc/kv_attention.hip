// Attention over the batched INT4 KV cache (w4_kv_attention): the launch.
#include "common.hpp"
#include "kv_prompt.hpp"

namespace w4 {

namespace {
template <int D, int PIECES, typename TQ, typename TO>
hipError_t launch_as(const KvPages& c, const KvAttn& a, hipStream_t st) {
    const KvPlan p = kv_plan(c, D, a.group, PIECES, a.max_rows, a.max_len, a.window, a.sinks);
    if (p.prompt) return launch_kv_prompt_as<D, D == 256 ? 1 : 2, PIECES, TQ, TO>(c, a, p, st);
    if constexpr (D < 256)
        if (p.nc == 2) return launch_kv_split_as<D, 2, PIECES, TQ, TO>(c, a, p, st);
    return launch_kv_split_as<D, 1, PIECES, TQ, TO>(c, a, p, st);
}

// fp32 on either side takes its operands in two 16-bit pieces
template <int D> hipError_t launch(const KvPages& c, const KvAttn& a, bool q_bf16, bool out_bf16, hipStream_t st) {
    if (q_bf16) return out_bf16 ? launch_as<D, 1, __bf16, __bf16>(c, a, st) : launch_as<D, 2, __bf16, float>(c, a, st);
    return out_bf16 ? launch_as<D, 2, float, __bf16>(c, a, st) : launch_as<D, 2, float, float>(c, a, st);
}
}  // namespace

// Two kernels and the parts of the keys, by an estimate of the time in clocks: rounds of
// workgroups over the 256 CUs, each as long as a wavefront's share of the tiles of keys
// (and no shorter than the longest workgroup) plus what a workgroup costs besides, two
// tiles' time, in kv_prompt_kernel 14 (its first stage and last barriers serve few tiles);
// parts cost two more for the launch that joins them. A tile takes a wavefront about 4850
// clocks in kv_split_kernel (5900 with D = 256; 6000 in two pieces) and 3500 (4600) in
// kv_prompt_kernel, for the same columns. Measured, 8 kv heads, bf16, us:
//   split kernel, a batch of 48 of up to 8192 positions: 79 whole, 51 in two parts (one
//   round), 55 in eight, 69 in sixteen; two of up to 131072: 50 in 48 parts, 67 in 16.
//   split against prompt kernel, each in the parts that the estimate gives it (G = 4; the last with
//   G = 1, 32 kv heads, 16 with D = 256):
//                  512 rows   2048 rows   64 behind 16384   512 behind 16384   8192 rows
//     bf16  D 128   18 / 37    98 / 121       47 / 54           244 / 211       969 / 728
//           D 256   26 / 41   180 / 128       82 / 80           492 / 393      1031 / 800
//     fp32  D 128   21 / 43   126 / 146       60 / 67           358 / 285      1365 / 1000
//           D 256   34 / 46   248 / 174      117 / 97           742 / 517      1541 / 1040
// The estimate takes the faster one of each pair, but for fp32, D = 256, 64 behind 16384.
// It takes `rows` for every sequence's where the caller gives no max_rows: 64 single tokens with
// starts, up to 8192 positions, take 73 us with the bounds and 388 without. One kernel serves
// all sequences of a call: 47 such tokens beside 1024 rows behind 7168 take 1003, apart 62 and 199.
namespace {
struct KvGuess {
    int64_t clocks;
    int splits;
};
KvGuess kv_guess(int64_t blocks, int64_t fit, int64_t tiles, int64_t mean_tiles, int share, int besides, int clocks) {
    KvGuess best{0, 1};
    int64_t cap = (tiles + share - 1) / share;
    cap = cap < kMaxSplits ? cap : kMaxSplits;
    for (int64_t s = 1; s <= cap && (s == 1 || blocks * s <= 8 * fit); ++s) {
        const int64_t longest = (tiles + share * s - 1) / (share * s) + besides;
        const int64_t mean = (mean_tiles + share * s - 1) / (share * s) + besides;
        const int64_t rounds = (blocks * s + fit - 1) / fit;
        const int64_t t = (rounds * mean > longest ? rounds * mean : longest) + (s > 1 ? 2 : 0);
        if (s == 1 || t * clocks < best.clocks) best = {t * clocks, (int)s};
    }
    return best;
}
}  // namespace

KvPlan kv_plan(const KvPages& c, int D, int group, int pieces, int64_t max_rows, int64_t max_len, int64_t window,
               int64_t sinks) {
    const int64_t columns = max_rows * group, pairs = (int64_t)c.B * c.Hkv;
    KvPlan plan[2];
    KvGuess guess[2];
    for (int prompt = 0; prompt < 2; ++prompt) {
        KvPlan& p = plan[prompt];
        p.prompt = prompt;
        p.nc = (prompt || columns > 16) && D < 256 ? 2 : 1;
        const int per = 16 * p.nc * (prompt ? 8 : 1);  // columns of a workgroup
        const int64_t tiles = (columns + per - 1) / per, most = (1 << 22) / (c.B * (prompt ? (int64_t)c.Hkv : 1));
        p.column_tiles = (int)(tiles < most ? tiles : most);  // longer sequences loop
        // keys that a workgroup's columns walk over, at most and in the mean
        const int64_t rows = per / group + 2 < max_rows ? per / group + 2 : max_rows;
        int64_t keys = max_len, mean = max_len - (max_rows < max_len ? max_rows : max_len) / 2;
        if (window > 0 && window + rows < max_len) {
            const int64_t rest = max_len - window - rows;
            keys = window + rows + (sinks < rest ? sinks : rest) + 64;
            mean = keys < mean ? keys : mean;
        }
        const int fit = 256 * (prompt ? 1 : p.nc == 1 && D < 256 ? 3 : 2);
        const int clocks = prompt ? (pieces == 1 ? 3500 : 4600) : pieces == 2 ? 6000 : D == 256 ? 5900 : 4850;
        guess[prompt] = kv_guess(p.column_tiles * pairs, fit, (keys + 31) / 32, (mean + 31) / 32, prompt ? 1 : 4,
                                 prompt ? 14 : 2, clocks);
        p.splits = guess[prompt].splits;
    }
    // (the prompt kernel's grid has sequences and heads in one dimension)
    return plan[columns > 64 && pairs <= 1 << 20 && guess[1].clocks < guess[0].clocks];
}

size_t kv_attention_workspace(const KvPages& c, int D, int64_t Hq, int64_t max_rows, int64_t max_len,
                              int64_t window, int64_t sinks) {
    int splits = 1;  // whatever the types will be
    for (int pieces = 1; pieces <= 2; ++pieces) {
        const KvPlan p = kv_plan(c, D, (int)(Hq / c.Hkv), pieces, max_rows, max_len, window, sinks);
        splits = p.splits > splits ? p.splits : splits;
    }
    return splits > 1 ? kv_partial_bytes((int64_t)c.rows * Hq, splits, D) : 0;
}

hipError_t launch_kv_attention(int D, bool q_bf16, bool out_bf16, const KvPages& c, const KvAttn& a,
                               hipStream_t st) {
    switch (D) {
        case 64: return launch<64>(c, a, q_bf16, out_bf16, st);
        case 128: return launch<128>(c, a, q_bf16, out_bf16, st);
        case 256: return launch<256>(c, a, q_bf16, out_bf16, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace w4
