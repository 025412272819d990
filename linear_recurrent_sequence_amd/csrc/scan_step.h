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
    int B, D, G, blocks, seqs, softplus, bc_vec;  // blocks: workgroups of 1024 / S channels; seqs: sequences a workgroup
};
// Sequences a workgroup takes, while so many workgroups are left: 128 sequences of 8192 channels and 16 states 26.2 us with
// four, 26.4 with two, 31.4 with one.
constexpr int kScanStepSeqs = 4, kScanStepWgs = 4096;
typedef void (*scan_step_kernel_t)(ScanStepArgs);
scan_step_kernel_t scan_step_kernel_get(bool bf16_in, bool bf16_out, int S);

}  // namespace ret
