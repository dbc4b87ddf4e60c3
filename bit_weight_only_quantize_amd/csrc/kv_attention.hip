// Attention over the batched INT4 KV cache (w4_kv_attention): the launch.
#include "common.hpp"
#include "kv_decode.hpp"

namespace w4 {

namespace {
template <int D, int PIECES>
hipError_t launch(const KvPages& c, const KvAttn& a, bool q_bf16, bool out_bf16, hipStream_t st) {
    return launch_kv_split<D, PIECES>(c, a, q_bf16, out_bf16, st);
}
}  // namespace

KvPlan kv_plan(const KvPages& c, int D, int group, int64_t max_rows, int64_t max_len, int64_t window,
               int64_t sinks) {
    KvPlan p;
    const int64_t columns = max_rows * group;
    p.nc = columns > 16 && D < 256 ? 2 : 1;
    const int64_t tiles = (columns + 16 * p.nc - 1) / (16 * p.nc);
    const int64_t most = 0x7fffffLL / c.B;  // longer sequences loop
    p.column_tiles = (int)(tiles < most ? tiles : most);
    // the keys that a tile of columns walks over, in tiles of 32
    int64_t keys = max_len;
    const int64_t rows = 16 * p.nc / group + 2 < max_rows ? 16 * p.nc / group + 2 : max_rows;
    if (window > 0 && window + rows < max_len) {
        const int64_t rest = max_len - window - rows;
        keys = window + rows + (sinks < rest ? sinks : rest) + 64;
    }
    const int64_t key_tiles = (keys + 31) / 32;
    // Parts of the keys: rounds of workgroups over the chip (3 a CU fit its registers, 2 of
    // the wider kernels), each as long as a wavefront's share of the tiles and what a
    // workgroup costs besides, about two tiles' time, as does the launch that joins them. Measured with 8 kv heads: a batch of 48
    // of up to 8192 positions (384 workgroups a part) 77 us whole, 50 in two parts (one round),
    // 58 in three, 62 in eight; two sequences of 131072 (16) 52 us in 48 parts, 67 in 16.
    const int64_t blocks = (int64_t)p.column_tiles * c.B * c.Hkv;
    const int64_t fit = 256 * (p.nc == 1 && D < 256 ? 3 : 2);
    const int64_t cap = key_tiles < 4 * kMaxSplits ? (key_tiles + 3) / 4 : kMaxSplits;
    int64_t best = 0;
    p.splits = 1;
    for (int64_t s = 1; s <= cap && (s == 1 || blocks * s <= 8 * fit); ++s) {
        const int64_t cost = (blocks * s + fit - 1) / fit * ((key_tiles + 4 * s - 1) / (4 * s) + 2) + (s > 1 ? 2 : 0);
        if (s == 1 || cost < best) best = cost, p.splits = (int)s;
    }
    return p;
}

size_t kv_attention_workspace(const KvPages& c, int D, int64_t Hq, int64_t max_rows, int64_t max_len,
                              int64_t window, int64_t sinks) {
    const KvPlan p = kv_plan(c, D, (int)(Hq / c.Hkv), max_rows, max_len, window, sinks);
    return p.splits > 1 ? kv_partial_bytes((int64_t)c.rows * Hq, p.splits, D) : 0;
}

hipError_t launch_kv_attention(int D, bool q_bf16, bool out_bf16, const KvPages& c, const KvAttn& a,
                               hipStream_t st) {
    // fp32 on either side takes its operands in two 16-bit pieces
    const bool one = q_bf16 && out_bf16;
    switch (D) {
        case 64: return one ? launch<64, 1>(c, a, true, true, st) : launch<64, 2>(c, a, q_bf16, out_bf16, st);
        case 128: return one ? launch<128, 1>(c, a, true, true, st) : launch<128, 2>(c, a, q_bf16, out_bf16, st);
        case 256: return one ? launch<256, 1>(c, a, true, true, st) : launch<256, 2>(c, a, q_bf16, out_bf16, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace w4
