// q4q_attn_d64.cu -- attention over the paged 4-bit cache for heads of 64 values.
#include "q4q_attn_kernel.cuh"

namespace q4q {

q4q_status attn_run_64(const AttnArgs& a, bool wide, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    return attn_run<2>(a, wide, workspace, stream, info);
}
size_t attn_workspace_64(const DeviceInfo& info) { return attn_workspace<2>(info); }
unsigned int attn_take_device_status_64() { return attn_take_status_word(); }

}  // namespace q4q
