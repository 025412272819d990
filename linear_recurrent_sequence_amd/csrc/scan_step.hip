// One token of the selective scan with the state updated in place: S / 4 lanes a channel, four states each, so that a wave's
// accesses of the state are contiguous. The state is read and written once, which is all the traffic that
// counts: 128 sequences of 8192 channels and 16 states 26.2 us, 5.5 TB/s.
#include "scan_step.h"

namespace ret {

namespace {

// A lane takes its states of a channel for `seqs` sequences (at most kScanStepSeqs), so that A is read once for all of them.
template <class E, class O, int S>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanStepArgs a) {
    constexpr int L = S / 4, e = sizeof(typename E::st);
    const int b0 = blockIdx.x / a.blocks * a.seqs, lane = threadIdx.x % L;
    const long long d = (long long)(blockIdx.x % a.blocks) * (256 / L) + threadIdx.x / L;
    if (d >= a.D) return;  // the lanes of a channel together
    const int g = (int)(d / (a.D / a.G)), off = (g * S + 4 * lane) * e;
    f32x4_t h[kScanStepSeqs];
    typename Raw<E>::one u[kScanStepSeqs], dt[kScanStepSeqs], z[kScanStepSeqs];
    typename Raw<E>::four B[kScanStepSeqs], C[kScanStepSeqs];
#pragma unroll
    for (int i = 0; i < kScanStepSeqs; ++i) {
        const int b = b0 + i;
        if (i >= a.seqs || b >= a.B) break;
        const long long row = (long long)b * a.D + d;
        h[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(a.state + row * S + 4 * lane));
        u[i] = Raw<E>::get((const char*)a.u + row * e, 0);
        dt[i] = Raw<E>::get((const char*)a.dt + row * e, 0);
        if (a.z) z[i] = Raw<E>::get((const char*)a.z + (b * a.ldz + d) * e, 0);
        B[i] = Raw<E>::get4((const char*)a.b + b * a.ldb * e, off, a.bc_vec);
        C[i] = Raw<E>::get4((const char*)a.c + b * a.ldc * e, off, a.bc_vec);
    }
    f32x4_t A = *reinterpret_cast<const f32x4_t*>(a.A + d * S + 4 * lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] = decay_rate(A[j]);
    const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
#pragma unroll
    for (int i = 0; i < kScanStepSeqs; ++i) {
        const int b = b0 + i;
        if (i >= a.seqs || b >= a.B) break;
        const long long row = (long long)b * a.D + d;
        float step = Raw<E>::value(dt[i]) + bias, slope;
        if (a.softplus) softplus(step, &step, &slope);
        const float ui = Raw<E>::value(u[i]), du = step * ui;
        const f32x4_t Bv = Raw<E>::values(B[i]), Cv = Raw<E>::values(C[i]);
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[i][j] = fmaf(__builtin_amdgcn_exp2f(step * A[j]), h[i][j], du * Bv[j]);
            y = fmaf(Cv[j], h[i][j], y);
        }
        __builtin_nontemporal_store(h[i], reinterpret_cast<f32x4_t*>(a.state + row * S + 4 * lane));
        y = lanes_sum<L>(y);
        y = fmaf(skip, ui, y);
        if (a.z) y *= swish_hw(Raw<E>::value(z[i]));
        if (lane == 0) store_out((typename O::st*)a.y + row, y);
    }
}

template <class E, class O>
scan_step_kernel_t pick(int S) {
    switch (S) {
        case 8: return scan_step_kernel<E, O, 8>;
        case 16: return scan_step_kernel<E, O, 16>;
        case 32: return scan_step_kernel<E, O, 32>;
        case 64: return scan_step_kernel<E, O, 64>;
        default: return nullptr;
    }
}

}  // namespace

scan_step_kernel_t scan_step_kernel_get(bool bf16_in, bool bf16_out, int S) {
    if (!bf16_in) return pick<F32, F32>(S);
    return bf16_out ? pick<BF16, BF16>(S) : pick<BF16, F32>(S);
}

}  // namespace ret
