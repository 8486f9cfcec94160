// q4q_mx_internal.h -- host-side declarations shared by the MXFP4 translation units.
#pragma once

#include "q4q_internal.h"

namespace q4q {

inline bool mx_type_ok(int t) { return t == Q4Q_TYPE_F32 || t == Q4Q_TYPE_F16 || t == Q4Q_TYPE_BF16; }
inline size_t mx_type_bytes(int t) { return t == Q4Q_TYPE_F32 ? 4 : 2; }
inline bool mx_acts_ok(int a) { return a == Q4Q_ACTS_MXFP4 || a == Q4Q_ACTS_MXFP8; }

// The activation side of a product.
struct MxActs {
    const void* src;
    int type, acts;
    int64_t n_src;           // rows of src
    int64_t n_rows;          // rows of the product
    int64_t K;
    const int32_t* first;    // experts' first rows (device), null: dense
    const int32_t* slot;     // slot of each sorted row (device), null: src is sorted already
    int n_experts, top_k;
};

unsigned int mxfp4_take_device_status();
unsigned int mxmm_take_device_status();

// The tensor map of MXFP4 weights: boxes of 128 rows and stage_atoms atoms of 128 bytes of
// shared memory a row (q4q_mxmm.cu).
bool mx_encode_weight_map(CUtensorMap* map, const void* src0, int64_t ne00, int64_t ne01, int n_mats, bool e4m3, int stage_atoms);

// Encode the activations of a product into `codes` and `scales` (token tiles of bn rows, at
// most max_groups of them) and zero the call's abort word (q4q_mxfp4.cu).
q4q_status mx_encode_acts(const MxActs& m, unsigned int* abort_word, uint8_t* codes, uint8_t* scales, int bn,
                          int64_t max_groups, bool pdl, cudaStream_t stream, const DeviceInfo& info);

}  // namespace q4q
