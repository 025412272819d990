// One token of the gated delta rule with the state updated in place. With S read once,
//     x = S^T k,  z = S^T q,  u = beta (v - alpha x),  S <- alpha S + k u^T,  o = scale (alpha z + (q.k) u),
// so both sums over the state come from the same read and one exchange between the waves; the state is read and written
// once, which is all the traffic there is. Measured: 128 sequences of 16 heads of 128 x 256, 99 us (5.4 TB/s); one sequence
// of 8 heads of 64 x 64, 3.5 us.
#include "delta_step.h"

#include "kernels.h"

namespace ret {

namespace {

// 64 columns per workgroup, 4 per lane; lane group rg of wave w holds rows RPT (4 w + rg) ..: a wave's load of one row
// index is four runs of 256 bytes.
template <class E, int DK>
__global__ __launch_bounds__(DK >= 32 ? DK * 2 : 64) void delta_step_kernel(DeltaStepArgs a) {
    typedef typename E::st st;
    constexpr int NW = DK >= 32 ? DK / 32 : 1, RPT = DK / (4 * NW);
    __shared__ float part[NW][16][9];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), cg = lane & 15, rg = lane >> 4;
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H;
    const int c0 = blockIdx.y * 64 + 4 * cg, r0 = RPT * (4 * w + rg);
    const bool in = c0 < a.dv;
    const int cc = in ? c0 : 0;
    const long long qrow = ((long long)b * a.Hk + h / (a.H / a.Hk)) * DK + r0;
    float* sp = a.state + ((long long)bh * DK + r0) * a.dv + cc;
    f32x4_t s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(sp + (long long)i * a.dv));
    float q[RPT], k[RPT], v[4];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        q[i] = gate_at(a.q, qrow + i, sizeof(st) == 2);
        k[i] = gate_at(a.k, qrow + i, sizeof(st) == 2);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = gate_at(a.v, (long long)bh * a.dv + cc + j, sizeof(st) == 2);
    const float alpha = expf(gate_at(a.g, bh, a.gate_bf16)), beta = gate_at(a.beta, bh, a.gate_bf16);
    f32x4_t x = {0.f, 0.f, 0.f, 0.f}, z = {0.f, 0.f, 0.f, 0.f};
    float qk = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        x += s[i] * k[i];
        z += s[i] * q[i];
        qk += q[i] * k[i];
    }
#pragma unroll
    for (int m = 16; m < 64; m *= 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] += __shfl_xor(x[j], m);
            z[j] += __shfl_xor(z[j], m);
        }
        qk += __shfl_xor(qk, m);
    }
    if constexpr (NW > 1) {
        if (rg == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                part[w][cg][j] = x[j];
                part[w][cg][4 + j] = z[j];
            }
            part[w][cg][8] = qk;
        }
        __syncthreads();
        x = z = f32x4_t{0.f, 0.f, 0.f, 0.f};
        qk = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] += part[i][cg][j];
                z[j] += part[i][cg][4 + j];
            }
            qk += part[i][cg][8];
        }
    }
    if (!in) return;
    f32x4_t u;
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = beta * (v[j] - alpha * x[j]);
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        __builtin_nontemporal_store(alpha * s[i] + k[i] * u, reinterpret_cast<f32x4_t*>(sp + (long long)i * a.dv));
    if (w == 0 && rg == 0) {
        const f32x4_t o = a.scale * (alpha * z + qk * u);
        const long long e = (long long)bh * a.dv + c0;
        if (a.out_bf16) store4((uint16_t*)a.o + e, o);
        else store4((float*)a.o + e, o);
    }
}

template <class E>
delta_step_kernel_t pick(int dk) {
    switch (dk) {
        case 16: return delta_step_kernel<E, 16>;
        case 32: return delta_step_kernel<E, 32>;
        case 64: return delta_step_kernel<E, 64>;
        case 128: return delta_step_kernel<E, 128>;
        case 256: return delta_step_kernel<E, 256>;
        default: return nullptr;
    }
}

}  // namespace

delta_step_kernel_t delta_step_kernel_get(bool bf16_in, int dk) { return bf16_in ? pick<BF16>(dk) : pick<F32>(dk); }

}  // namespace ret
