// q4q_attn.cu -- host side of the attention over the paged 4-bit cache: argument checks and the choice
// of the kernel (q4q_attn_kernel.cuh).
#include <algorithm>
#include <initializer_list>

#include "q4q_attn.cuh"
#include "q4q_attn_internal.h"

namespace q4q {
namespace {

constexpr int64_t STEP_TOKENS = 2 * KV_GROUP;      // of the warp-level kernel

// The tcgen05 kernel may take bf16 and fp16 rows where a sequence has 64 of them or more for a key-value head, on average, and
// does where its longer start pays: from 256 rows, a CTA's tiles, or from 6 2^20 pairs of a row of queries and a key of the tables,
// which bound the keys.  us, warp-level MMAs / tcgen05, 8 key-value heads of 128, rows a head: bf16, 64 rows over 8192 keys (4.2 M pairs)
// 28 / 33, 128 over 8192 40 / 34, 256 over 8192 64 / 37, 16 x 64 over 2048 82 / 64, 2 x 128 over 300 21 / 37, 8 x 400 over 100 73 / 53;
// fp16, 64 over 1023 19.6 / 27.5, 128 over 8192 71 / 35, 2048 over 8192 920 / 101.
// One kernel takes the whole call, by what the host knows.  A batch of unlike sequences is slower than its parts in calls of their own: a
// prompt of 2048 bf16 tokens beside 63 single ones over 8192 keys 827 us (tcgen05), apart 275 + 139; one of 512 beside them 593
// (warp-level), apart 100 + 138.  A page table wider than the sequences counts as if they were that long.
bool may_use_tensor_cores(int type, int64_t head_dim, int64_t n_q, int shared, int64_t n_seqs) {
    return type != Q4Q_TYPE_F32 && head_dim <= 128 && n_q * shared >= n_seqs * 64;
}
// Not with tables of more than 2^24 keys: its loaders wait through a piece, 2.4 us for 128 keys, and a wait is bounded by a second.
constexpr int64_t TC_MOST_KEYS = 1ll << 24;
bool on_tensor_cores(const AttnArgs& a, int64_t head_dim) {
    return may_use_tensor_cores(a.type, head_dim, a.n_q, a.shared, a.n_seqs) && (a.max_pages << a.page_log) <= TC_MOST_KEYS &&
           (a.n_q * a.shared >= a.n_seqs * 256ll || (double)a.n_q * a.heads * (double)(a.max_pages << a.page_log) >= 6.0 * (1 << 20));
}

size_t workspace_bytes(int type, int64_t head_dim, int64_t n_q, int shared, int64_t n_seqs, const DeviceInfo& info) {
    const size_t most = may_use_tensor_cores(type, head_dim, n_q, shared, n_seqs) ? attn_tc_workspace(head_dim, info) : 0;
    switch (head_dim) {
        case 64: return std::max(most, attn_workspace_64(info));
        case 96: return std::max(most, attn_workspace_96(info));
        case 128: return std::max(most, attn_workspace_128(info));
        default: return attn_workspace_256(info);
    }
}

q4q_status check(AttnArgs& a, const void* q, int64_t q_stride, int type, int64_t n_q, int n_q_heads, int n_kv_heads, int64_t head_dim,
                 const void* cache, int64_t n_pages, int page_tokens, const int32_t* pages, int64_t max_pages, const int32_t* kv_len,
                 const int32_t* first, int64_t n_seqs, float scale, int causal, int64_t window, void* dst, float* lse, void* workspace,
                 size_t workspace_bytes_given, bool& empty, DeviceInfo& info) {
    q4q_status st = kv_check(n_pages, page_tokens, n_kv_heads, head_dim, a.page_log);
    if (st != Q4Q_OK) return st;
    if (n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % n_kv_heads || n_q < 0 || n_q >= (1 << 24) || n_seqs < 0 || n_seqs >= (1 << 20) ||
        max_pages < 0 || max_pages >= (1ll << 30) / page_tokens || window < 0)
        return Q4Q_ERR_SHAPE;
    if (q_stride < n_q_heads * head_dim || q_stride >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (!first && n_seqs > n_q) return Q4Q_ERR_SHAPE;
    if (n_q * (n_q_heads / n_kv_heads) >= (1ll << 30)) return Q4Q_ERR_SHAPE;
    if (!mx_type_ok(type) || !(scale == scale)) return Q4Q_ERR_ARG;
    empty = n_q == 0 || n_seqs == 0;
    if (empty) return Q4Q_OK;
    if (!q || !dst || !kv_len || !workspace || (max_pages > 0 && !pages) || (n_pages > 0 && !cache)) return Q4Q_ERR_NULL;
    const size_t size = mx_type_bytes(type);
    if (!aligned(q, size) || !aligned(dst, size) || !aligned(cache, 16) || !aligned(workspace, 256) || !aligned(pages, 4) || !aligned(kv_len, 4) ||
        !aligned(first, 4) || !aligned(lse, 4))
        return Q4Q_ERR_ALIGN;
    // other CTAs read a row's queries after its result is written
    const uintptr_t q0 = (uintptr_t)q, d0 = (uintptr_t)dst;
    if (q0 < d0 + (uintptr_t)(n_q * n_q_heads * head_dim) * size && d0 < q0 + (uintptr_t)((n_q - 1) * q_stride + n_q_heads * head_dim) * size) return Q4Q_ERR_ARG;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    if (workspace_bytes_given < workspace_bytes(type, head_dim, n_q, n_q_heads / n_kv_heads, n_seqs, info)) return Q4Q_ERR_WORKSPACE;
    a.q = q;
    a.q_stride = q_stride;
    a.cache = static_cast<const uint8_t*>(cache);
    a.pages = pages;
    a.kv_len = kv_len;
    a.first = first;
    a.n_q = n_q;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.window = std::min<int64_t>(window, 1ll << 31);      // which is past every key
    a.n_seqs = (int)n_seqs;
    a.heads = n_q_heads;
    a.kv_heads = n_kv_heads;
    a.shared = n_q_heads / n_kv_heads;
    if (a.shared > 1) {
        const MxDivisor d = mx_divisor((uint32_t)a.shared);
        a.shared_m = d.m;
        a.shared_s = d.s;
    }
    a.type = type;
    a.causal = causal != 0;
    a.align = aligned(q, 32) && aligned(dst, 32) && q_stride * size % 32 == 0 ? 32 : aligned(q, 16) && aligned(dst, 16) && q_stride * size % 16 == 0 ? 16 : 1;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    a.dst = dst;
    a.lse = lse;
    a.limit_ns = WAIT_LIMIT_NS;
    a.fault = 0;
    return Q4Q_OK;
}

// Two groups of columns where a key-value head has more rows than one group holds (8, or 4 that are split in two
// fp16), by the average of the rows a sequence: a chunk is then unpacked once for twice the rows, by half as many CTAs an
// SM.  With few steps (by the table's keys, 24 for each of the 2 CTAs an SM that one group has) the single groups' shorter end of
// a piece counts more.  us, one group / two, 8 key-value heads of 128, rows a head: fp32, 8 rows over 1023 keys 14.7 / 18.1, 4095
// 17.0 / 19.5, 16383 20.7 / 19.2, 64 rows over 1023 20.0 / 21.7, 8191 51 / 45; 64 sequences of up to 8192 keys, bf16 4 rows
// (one group by the rule) 98 / 163.  A batch whose sequences have 4 or 8 rows, between 4 and 8 on average, would be better off with one
// (fp32, 142 / 199): the host sees the average alone.
bool wide(const AttnArgs& a, const DeviceInfo& info) {
    const int64_t one = a.type == Q4Q_TYPE_BF16 ? 8 : 4, rows = a.n_q * a.shared;
    const double steps = (double)((rows + one - 1) / one) * a.kv_heads * (double)(((a.max_pages << a.page_log) + STEP_TOKENS - 1) / STEP_TOKENS);
    return rows > a.n_seqs * one && steps >= 24.0 * 2 * info.sm_count;
}

q4q_status dispatch(const AttnArgs& a, int64_t head_dim, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    const bool two = wide(a, info);
    switch (head_dim) {
        case 64: return attn_run_64(a, two, workspace, stream, info);
        case 96: return attn_run_96(a, two, workspace, stream, info);
        case 128: return attn_run_128(a, two, workspace, stream, info);
        default: return attn_run_256(a, two, workspace, stream, info);
    }
}

}  // namespace

unsigned int attn_take_device_status() {
    unsigned int first = 0;
    for (unsigned int w : {attn_take_device_status_64(), attn_take_device_status_96(), attn_take_device_status_128(), attn_take_device_status_256(),
                           attn_tc_take_device_status()})
        if (!first) first = w;
    return first;
}

}  // namespace q4q

using namespace q4q;

extern "C" q4q_status q4q_kv_attn_workspace_size(int64_t n_q, int n_q_heads, int n_kv_heads, int64_t head_dim, int64_t n_seqs, int type, size_t* bytes) {
    if (!bytes) return Q4Q_ERR_NULL;
    if (!kv_dim_ok(head_dim) || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads || n_q_heads > 1024 || n_q < 0 || n_q >= (1 << 24) || n_seqs < 0 ||
        n_seqs >= (1 << 20))
        return Q4Q_ERR_SHAPE;
    if (!mx_type_ok(type)) return Q4Q_ERR_ARG;
    DeviceInfo info;
    const q4q_status st = current_device_info(&info);
    if (st != Q4Q_OK) return st;
    // what the same rows need as one sequence: fewer sequences may take the form with the larger workspace
    *bytes = workspace_bytes(type, head_dim, n_q, n_q_heads / n_kv_heads, std::min<int64_t>(n_seqs, 1), info);
    return Q4Q_OK;
}

extern "C" q4q_status q4q_kv_attn(const void* q, int64_t q_stride, int type, int64_t n_q, int n_q_heads, int n_kv_heads, int64_t head_dim,
                                  const void* cache, int64_t n_pages, int page_tokens, const int32_t* pages, int64_t max_pages,
                                  const int32_t* kv_len, const int32_t* first, int64_t n_seqs, float scale, int causal, int64_t window,
                                  void* dst, float* lse, void* workspace, size_t workspace_bytes, q4q_stream_t stream) {
    AttnArgs a{};
    DeviceInfo info;
    bool empty;
    const q4q_status st = check(a, q, q_stride, type, n_q, n_q_heads, n_kv_heads, head_dim, cache, n_pages, page_tokens, pages, max_pages, kv_len,
                                first, n_seqs, scale, causal, window, dst, lse, workspace, workspace_bytes, empty, info);
    if (st != Q4Q_OK || empty) return st;
    if (on_tensor_cores(a, head_dim)) return attn_tc_run(a, head_dim, workspace, (cudaStream_t)stream, info);
    return dispatch(a, head_dim, workspace, (cudaStream_t)stream, info);
}

extern "C" q4q_status q4q_debug_kv_attn_timeout(const void* q, int64_t q_stride, int type, int64_t n_q, int n_q_heads, int n_kv_heads,
                                                int64_t head_dim, const void* cache, int64_t n_pages, int page_tokens, const int32_t* pages,
                                                int64_t max_pages, const int32_t* kv_len, const int32_t* first, int64_t n_seqs, float scale,
                                                void* dst, void* workspace, size_t workspace_bytes_given, int path, uint64_t limit_ns,
                                                q4q_stream_t stream) {
    if (limit_ns < 1 || limit_ns > WAIT_LIMIT_NS || path < 0 || path > 1) return Q4Q_ERR_ARG;
    AttnArgs a{};
    DeviceInfo info;
    bool empty;
    const q4q_status st = check(a, q, q_stride, type, n_q, n_q_heads, n_kv_heads, head_dim, cache, n_pages, page_tokens, pages, max_pages, kv_len,
                                first, n_seqs, scale, 1, 0, dst, nullptr, workspace, workspace_bytes_given, empty, info);
    if (st != Q4Q_OK || empty) return st;
    a.limit_ns = limit_ns;
    a.fault = 1;
    if (path == 0) return dispatch(a, head_dim, workspace, (cudaStream_t)stream, info);
    if (type == Q4Q_TYPE_F32 || head_dim > 128) return Q4Q_ERR_SHAPE;
    if (workspace_bytes_given < attn_tc_workspace(head_dim, info)) return Q4Q_ERR_WORKSPACE;
    return attn_tc_run(a, head_dim, workspace, (cudaStream_t)stream, info);
}
