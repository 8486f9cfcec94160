// q4q_attn_internal.h -- host-side declarations shared by the attention translation units.
#pragma once

#include "q4q_mx_internal.h"

namespace q4q {

unsigned int rope_take_device_status();
unsigned int kv_take_device_status();
unsigned int attn_take_device_status();

// The shape rules of a cache (q4q_kv.cu): its page size as a power of two.
q4q_status kv_check(int64_t n_pages, int page_tokens, int n_kv_heads, int64_t head_dim, int& page_log);

// One call of q4q_kv_attn.
struct AttnArgs {
    const void* q;
    int64_t q_stride;
    const uint8_t* cache;
    const int32_t *pages, *kv_len, *first;
    int64_t n_q, n_pages, max_pages, window;
    int n_seqs, heads, kv_heads, shared;       // shared: query heads of a key-value head
    uint32_t shared_m, shared_s;               // division by it (MxDivisor), from 2 on
    int type, page_log, causal, align;         // align: of every row of q and dst, 32, 16 or 1
    float scale_log2;                          // scale * log2(e)
    void* dst;
    float* lse;
    uint64_t limit_ns;
    int fault;                                 // test support: the first CTA leaves out its first hand-off
};

// The kernels of each head size (q4q_attn_d*.cu).
#define Q4Q_ATTN_DIM(D)                                                                                                  \
    q4q_status attn_run_##D(const AttnArgs& a, bool wide, void* workspace, cudaStream_t stream, const DeviceInfo& info); \
    size_t attn_workspace_##D(const DeviceInfo& info);                                                                   \
    unsigned int attn_take_device_status_##D();
Q4Q_ATTN_DIM(64)
Q4Q_ATTN_DIM(96)
Q4Q_ATTN_DIM(128)
Q4Q_ATTN_DIM(256)
#undef Q4Q_ATTN_DIM

// Prompts on the tcgen05 tensor cores (q4q_attn_tc.cu): bf16 and fp16, heads of 64, 96 and 128 values.
q4q_status attn_tc_run(const AttnArgs& a, int64_t head_dim, void* workspace, cudaStream_t stream, const DeviceInfo& info);
size_t attn_tc_workspace(int64_t head_dim, const DeviceInfo& info);
unsigned int attn_tc_take_device_status();

}  // namespace q4q
