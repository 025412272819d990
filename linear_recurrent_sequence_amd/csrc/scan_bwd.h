// Gradients of the selective scan: arguments and kernels.
#pragma once

#include "rows.h"
#include "scan.h"

namespace ret {

struct ScanBwdArgs {
    ScanArgs f;                                // the forward's; segments are chunks: nseg of them, seg_tokens = CH
    const void* dy;                            // [B, N, D]
    const float* dstate_out;                   // [B, D, S] or null
    float* dstate_in;                          // or null
    float* seg_g;                              // [B][nseg][D][S]: gradients of the states leaving the chunks
    float* part_bc;                            // [parts][B N][2][S]: sums over a workgroup's channels of dB, dC
    float* part_a;                             // [B nseg][D (S + 2)]: dA, dskip, dbias
    void *du, *ddt, *dz, *db, *dc;             // dz or null
    int parts_g;                               // parts a group of channels, each every parts_g-th block of 16
    PartSumArgs cols;                          // dA, dskip and dbias from part_a
    int deal_parts;                            // of grad's workgroups to the XCDs
    unsigned bc_blocks;                        // workgroups of sums for dB and dC, before those for cols
};
typedef void (*scan_bwd_kernel_t)(ScanBwdArgs);
struct ScanBwdKernels {
    scan_bwd_kernel_t local, local_split, join, grad, sums;
    int chunk, waves;
};
bool scan_bwd_kernels_get(bool bf16_in, bool bf16_out, int S, ScanBwdKernels* o);

}  // namespace ret
