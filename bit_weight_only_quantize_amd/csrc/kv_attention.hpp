// What the host and the attention kernels over the batched INT4 KV cache share.
#pragma once

#include "kv_pages.hpp"

namespace w4 {

struct KvAttn {  // passed to kernels by value
    const void* q;
    void* out;
    float* lse;  // or null
    void* work;
    int64_t q_row, q_head, out_row, out_head;  // strides in elements
    int Hq, group;                             // query heads, and per kv head
    int window, sinks;                         // window 0: none
    int max_rows, max_len;                     // shape the launch only
    float scale;
};

// Device bytes the launch for these sizes takes in KvAttn::work.
size_t kv_attention_workspace(const KvPages& c, int D, int64_t Hq, int64_t max_rows, int64_t max_len,
                              int64_t window, int64_t sinks);
hipError_t launch_kv_attention(int D, bool q_bf16, bool out_bf16, const KvPages& c, const KvAttn& a,
                               hipStream_t st);
hipError_t launch_kv_rows(bool write, int D, bool bf16, const KvPages& c, void* const* data,
                          const int64_t* row_stride, const int64_t* head_stride, int max_rows,
                          hipStream_t st);

}  // namespace w4
