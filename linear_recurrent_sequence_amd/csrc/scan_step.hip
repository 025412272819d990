// One token of the selective scan with the state updated in place: S / 4 lanes a channel, four states each, so that a wave's
// accesses of the state are contiguous. The state is read and written once, which is all the traffic that counts.
#include "scan_step.h"

namespace ret {

namespace {

template <class E, class O, int S>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanStepArgs a) {
    constexpr int L = S / 4;
    const int b = blockIdx.x / a.blocks, lane = threadIdx.x % L;
    const long long d = (long long)(blockIdx.x % a.blocks) * (256 / L) + threadIdx.x / L;
    if (d >= a.D) return;  // the lanes of a channel together
    const int g = (int)(d / (a.D / a.G));
    const long long row = (long long)b * a.D + d;
    float* sp = a.state + row * S + 4 * lane;
    f32x4_t h = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(sp));
    const f32x4_t A = *reinterpret_cast<const f32x4_t*>(a.A + d * S + 4 * lane);
    float B[4], C[4];
    load4<E>(a.b, b * a.ldb + g * S + 4 * lane, a.bc_vec, B);
    load4<E>(a.c, b * a.ldc + g * S + 4 * lane, a.bc_vec, C);
    const float u = at<E>(a.u, row);
    float dt = at<E>(a.dt, row) + (a.bias ? a.bias[d] : 0.f), slope;
    if (a.softplus) softplus(dt, &dt, &slope);
    float y = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = fmaf(__builtin_amdgcn_exp2f(dt * decay_rate(A[e])), h[e], dt * u * B[e]);
        y = fmaf(C[e], h[e], y);
    }
    __builtin_nontemporal_store(h, reinterpret_cast<f32x4_t*>(sp));
    y = lanes_sum<L>(y);
    if (lane != 0) return;
    if (a.skip) y = fmaf(a.skip[d], u, y);
    if (a.z) y *= swish_hw(at<E>(a.z, b * a.ldz + d));
    store_out((typename O::st*)a.y + row, y);
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
