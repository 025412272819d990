// Arguments and selection of the selective scan's single-token kernel.
#pragma once

#include "scan.h"

namespace ret {

struct ScanStepArgs {
    const void *u, *dt, *z, *b, *c;  // u, dt [B, D]; z rows of ldz; b, c rows of ldb, ldc with [G, S] in each
    const float *A, *skip, *bias;
    float* state;                    // [B, D, S], updated in place
    void* y;                         // [B, D]
    long long ldz, ldb, ldc;
    int B, D, G, blocks, softplus, bc_vec;  // blocks: workgroups a sequence, of 1024 / S channels
};
typedef void (*scan_step_kernel_t)(ScanStepArgs);
scan_step_kernel_t scan_step_kernel_get(bool bf16_in, bool bf16_out, int S);

}  // namespace ret
