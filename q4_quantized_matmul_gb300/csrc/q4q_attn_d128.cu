// q4q_attn_d128.cu -- attention over the paged 4-bit cache for heads of 128 values.
#include "q4q_attn_kernel.cuh"

namespace q4q {

q4q_status attn_run_128(const AttnArgs& a, bool wide, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    return attn_run<4>(a, wide, workspace, stream, info);
}
size_t attn_workspace_128(const DeviceInfo& info) { return attn_workspace<4>(info); }
unsigned int attn_take_device_status_128() { return attn_take_status_word(); }

}  // namespace q4q
