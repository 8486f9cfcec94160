// q4q_attn_d96.cu -- attention over the paged 4-bit cache for heads of 96 values.
#include "q4q_attn_kernel.cuh"

namespace q4q {

q4q_status attn_run_96(const AttnArgs& a, bool wide, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    return attn_run<3>(a, wide, workspace, stream, info);
}
size_t attn_workspace_96(const DeviceInfo& info) { return attn_workspace<3>(info); }
unsigned int attn_take_device_status_96() { return attn_take_status_word(); }

}  // namespace q4q
