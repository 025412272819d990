// Arguments and selection of the gated delta rule's single-token kernel; reads of single values.
#pragma once

#include "kernels.h"

namespace ret {

struct DeltaStepArgs {
    const void *q, *k, *v;  // [B, Hk, dk], [B, H, dv]
    const void *g, *beta;   // [B, H]
    float* state;           // [B, H, dk, dv], updated in place
    void* o;                // [B, H, dv]
    int B, H, Hk, dv, out_bf16, gate_bf16;
    float scale;
};
typedef void (*delta_step_kernel_t)(DeltaStepArgs);
// d_k in {16, 32, 64, 128, 256}, d_v a multiple of 16; grid (B*H, ceil(d_v / 64)), max(64, 2 d_k) threads.
delta_step_kernel_t delta_step_kernel_get(bool bf16_in, int dk);

// The i-th value of an array in either type, as fp32.
__device__ __forceinline__ float gate_at(const void* p, long long i, int bf16) {
    return bf16 ? bf16_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}

}  // namespace ret
