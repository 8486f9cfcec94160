// q4q_attn_d256.cu -- attention over the paged 4-bit cache for heads of 256 values.
#include "q4q_attn_kernel.cuh"

namespace q4q {

q4q_status attn_run_256(const AttnArgs& a, bool wide, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    return attn_run<8>(a, wide, workspace, stream, info);
}
size_t attn_workspace_256(const DeviceInfo& info) { return attn_workspace<8>(info); }
unsigned int attn_take_device_status_256() { return attn_take_status_word(); }

}  // namespace q4q
