// Vectors of W consecutive values of an fp32 or bf16 array (the dtype is a run-time flag, uniform over the launch),
// and the reduction of per-workgroup column sums, for the row-wise normalization kernels.
#pragma once

#include "kernels.h"

namespace ret {

// W consecutive values at element offset i. W = 8: 16-byte vectors, for arrays whose rows are all 16-byte aligned;
// W = 1: any offset.
template <int W>
__device__ __forceinline__ void row_load(const void* p, long long i, bool bf16, float* f) {
    if constexpr (W == 8) {
        if (bf16) {
            const u32x4_t u = *reinterpret_cast<const u32x4_t*>((const uint16_t*)p + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[2 * e] = __uint_as_float(u[e] << 16);
                f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const f32x4_t x = *reinterpret_cast<const f32x4_t*>((const float*)p + i + e);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[e + j] = x[j];
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) f[e] = bf16 ? bf16_to_f32(((const uint16_t*)p)[i + e]) : ((const float*)p)[i + e];
    }
}

template <int W>
__device__ __forceinline__ void row_store(void* p, long long i, bool bf16, const float* f) {
    if constexpr (W == 8) {
        if (bf16) {
            *reinterpret_cast<u32x4_t*>((uint16_t*)p + i) =
                u32x4_t{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7])};
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<f32x4_t*>((float*)p + i + e) = f32x4_t{f[e], f[e + 1], f[e + 2], f[e + 3]};
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            if (bf16) ((uint16_t*)p)[i + e] = f32_to_bf16(f[e]);
            else ((float*)p)[i + e] = f[e];
        }
    }
}

// Column sums left by `parts` workgroups, partial [parts][2][cols] fp32, added up in a fixed order: sums over the
// first half into out0, over the second into out1 (either may be null).
struct ColSumArgs {
    const float* partial;
    float *out0, *out1;
    int parts, cols;
};
typedef void (*colsum_kernel_t)(ColSumArgs);
colsum_kernel_t colsum_kernel_get();
constexpr int kColSumCols = 64, kColSumThreads = 1024;  // columns (of the 2 * cols) and threads per workgroup

// Layer norm of rows of D values, with an optional residual added first, and its gradients.
struct LnArgs {
    const void *x, *res;        // [rows][D], one dtype
    void *sum, *y;              // sum: x + res rounded to x's dtype (or null)
    const float *weight, *bias; // [D] or null
    float *mean, *rstd;         // [rows] or null
    long long rows;
    int D, x_bf16, y_bf16;
    float eps;
};
struct LnBwdArgs {
    const void *dy, *x, *dsum;  // dsum (or null): added to dx, in dx's dtype
    const float *weight, *mean, *rstd;
    void* dx;
    float* partial;             // [gridDim.x][2][D] column sums of dy xh and dy, or null
    long long rows;
    int D, x_bf16, dy_bf16, dx_bf16;
};
typedef void (*ln_kernel_t)(LnArgs);
typedef void (*ln_bwd_kernel_t)(LnBwdArgs);
struct LnKernels {
    ln_kernel_t fwd;
    ln_bwd_kernel_t bwd;
    int fwd_rows, fwd_threads;  // rows in flight and threads per workgroup
    int bwd_rows;               // the same of the gradients (kLnBwdThreads threads)
};
constexpr int kLnBwdThreads = 1024;
constexpr int kLnMaxD = 16384;
bool ln_kernels_get(int D, LnKernels* out);

// Gradients of the multi-scale retention epilogue.
struct EpiBwdArgs {
    const void *dy, *o, *gate;
    const float *weight, *bias;
    void *dout, *dgate;
    float* partial;  // [gridDim.y][2][H * dv], or null
    long long rows;
    int H, dy_bf16, o_bf16, gate_bf16, do_bf16, dgate_bf16;
    float eps;
};
typedef void (*epi_bwd_kernel_t)(EpiBwdArgs);
constexpr int kEpiBwdCols = 512;     // columns (of H * dv) per workgroup
constexpr int kEpiBwdWaves = 16;     // waves per workgroup, each its own rows
epi_bwd_kernel_t epi_bwd_kernel_get(int dv);

}  // namespace ret
