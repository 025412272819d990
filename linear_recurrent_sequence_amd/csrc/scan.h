// Selective scan: arguments and the device code that its kernels share.
//
// Per batch b, channel d and state s, group g = d / (D / G):
//     dt_t = softplus(delta_t + bias),  a_t = exp(dt_t A),  h_t = a_t h_{t-1} + dt_t u_t B_t[g],
//     y_t = (sum_s C_t[g] h_t + D u_t) silu(z_t)
//
// Layout of every sequence kernel: a wave holds 16 channels, four neighbouring lanes a channel, each with SL = S / 4 of its
// states, and T = 256 / S tokens at a time, so that the T SL decays a_t of a lane are 64 registers whatever S is. The values
// per token and channel (u, delta, z, y) lie one in a lane: lane q of a channel's four holds tokens 4 i + q, and sums over
// the states leave each token's in that lane. B and C of a wave's tokens are staged in its own part of the LDS, in fp32.
#pragma once

#include "kernels.h"

namespace ret {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kScanCh = 16;  // channels of a wave

template <int S>
struct ScanShape {
    static constexpr int SL = S / 4;            // states a lane
    static constexpr int T = 256 / S;           // tokens of a wave's block
    static constexpr int TL = T / 4;            // of which a lane holds the scalars
    static constexpr int NW = S <= 16 ? 8 : 4;  // waves of a workgroup, neighbouring blocks of tokens
    static constexpr int CH = NW * T;           // tokens of a workgroup's chunk
    static constexpr int THREADS = 64 * NW;
};

struct ScanArgs {
    const void *u, *dt, *z, *b, *c;      // u, dt [B, N, D]; z rows of ldz; b, c rows of ldb, ldc with [G, S] in each
    const float *A, *skip, *bias;        // [D, S]; [D] or null
    const int32_t* lengths;              // [B] or null
    const float* state_in;               // [B, D, S] or null
    float* state_out;                    // [B, D, S] or null
    void* y;                             // [B, N, D]
    float *seg_h, *seg_dt;               // [B][nseg][D][S], [B][nseg][D]
    long long ldz, ldb, ldc;
    int B, N, D, G, nseg, seg_tokens, cblocks, softplus, bc_vec;
};

// One value of either type as fp32.
template <class E>
__device__ __forceinline__ float at(const void* p, long long i) {
    if constexpr (sizeof(typename E::st) == 2) return bf16_to_f32(((const uint16_t*)p)[i]);
    else return ((const float*)p)[i];
}

__device__ __forceinline__ int scan_length(const int32_t* lengths, int b, int N) {
    if (!lengths) return N;
    const int n = lengths[b];
    return n < 0 ? 0 : n > N ? N : n;
}

// Workgroup number -> position, so that the workgroups of neighbouring positions run on one XCD (they are dealt to the 8 in
// turn): n is a multiple of 8.
__device__ __forceinline__ long long xcd_order(long long id, long long n) { return (id & 7) * (n >> 3) + (id >> 3); }

// log(1 + exp(x)) and its derivative. exp(-|x|) by the hardware 2^x with the rounding of |x| log2(e) made up for;
// log(1 + e) = 2 atanh(e / (2 + e)) by its series, whose ninth term is below 2e-9 of the sum at e = 1.
__device__ __forceinline__ void softplus(float x, float* value, float* slope) {
    const float m = fabsf(x), t = m * kLog2e;
    const float rest = fmaf(m, kLog2e, -t) + m * 1.925963033e-8f;  // log2(e) - kLog2e
    float e = __builtin_amdgcn_exp2f(-t);
    e = fmaf(e, -kLn2 * rest, e);
    if (m > 87.f) e = 0.f;
    const float r = e * __builtin_amdgcn_rcpf(2.f + e), w = r * r;
    float p = fmaf(w, 1.f / 15.f, 1.f / 13.f);
    p = fmaf(w, p, 1.f / 11.f);
    p = fmaf(w, p, 1.f / 9.f);
    p = fmaf(w, p, 1.f / 7.f);
    p = fmaf(w, p, 1.f / 5.f);
    p = fmaf(w, p, 1.f / 3.f);
    p = fmaf(w, p, 1.f);
    *value = (x > 0.f ? x : 0.f) + 2.f * r * p;
    if (x != x) *value = x;
    const float s = __builtin_amdgcn_rcpf(1.f + e);
    *slope = x > 0.f ? s : e * s;
}

__device__ __forceinline__ float sigmoid_of(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// A in units of log2(e), so that a_t = 2^(dt_t A). An infinite A (a state without memory) becomes the largest number: steps of
// length 0 then still leave the state.
__device__ __forceinline__ float decay_rate(float A) {
    const float r = A * kLog2e;
    return r < -3.4e38f ? -3.4e38f : r > 3.4e38f ? 3.4e38f : r;
}

// The value that lane K of every four holds.
template <int K>
__device__ __forceinline__ float quad_of(float v) {
    return dpp_mov<K * 0x55>(v);
}
__device__ __forceinline__ float quad_of(float v, int k) {  // k a constant after unrolling
    return k == 0 ? quad_of<0>(v) : k == 1 ? quad_of<1>(v) : k == 2 ? quad_of<2>(v) : quad_of<3>(v);
}
// Lane q of every four gets the sum of the four's v[q].
__device__ __forceinline__ float quad_sums(float v0, float v1, float v2, float v3, int q) {
    const bool odd = q & 1, high = q & 2;
    const float a = (odd ? v1 : v0) + dpp_mov<0xb1>(odd ? v0 : v1);
    const float b = (odd ? v3 : v2) + dpp_mov<0xb1>(odd ? v2 : v3);
    return (high ? b : a) + dpp_mov<0x4e>(high ? a : b);
}

// Four neighbouring values.
template <class E>
__device__ __forceinline__ void load4(const void* p, long long i, bool vec, float* f) {
    typedef typename E::st st;
    if (vec) {
        if constexpr (sizeof(st) == 2) {
            const uint2 w = *reinterpret_cast<const uint2*>((const uint16_t*)p + i);
            f[0] = __uint_as_float(w.x << 16);
            f[1] = __uint_as_float(w.x & 0xffff0000u);
            f[2] = __uint_as_float(w.y << 16);
            f[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
            const f32x4_t w = *reinterpret_cast<const f32x4_t*>((const float*)p + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = w[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = at<E>(p, i + e);
    }
}

// Reads u and dt of the lane's tokens (any in-range row where a token is past the end).
template <class E, int S>
__device__ __forceinline__ void load_scalars(const void* p, long long row0, long long ld, int N, int t0, int q, int d,
                                             float (&f)[ScanShape<S>::TL]) {
#pragma unroll
    for (int i = 0; i < ScanShape<S>::TL; ++i) {
        const int t = t0 + 4 * i + q;
        f[i] = at<E>(p, (row0 + (t < N ? t : N - 1)) * ld + d);
    }
}
// The lane's part of B or C: 4 neighbouring values of the wave's [T][S], zero from token n on.
template <class E, int S>
__device__ __forceinline__ void load_bc(const void* p, long long row0, long long ld, int N, int n, int t0, int g, int lane,
                                        bool vec, float (&f)[4]) {
    const int t = t0 + 4 * lane / S;
    load4<E>(p, (row0 + (t < N ? t : N - 1)) * ld + g * S + 4 * lane % S, vec, f);
    if (t >= n)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = 0.f;
}

// Keeps a wave's LDS accesses on either side of it in order: they are carried out in the order they are issued.
__device__ __forceinline__ void lds_order() { __asm__ volatile("" ::: "memory"); }

// A wave's block: dt and dt u of the lane's tokens (0 from token n on: such a token changes nothing), B and C to LDS.
template <class E, int S>
struct ScanBlock {
    typedef ScanShape<S> P;
    float u[P::TL], dt[P::TL], z[P::TL], b[4], c[4];
    __device__ __forceinline__ void load(const ScanArgs& a, long long row0, int n, int t0, int q, int lane, int d, int g,
                                         bool out) {
        load_scalars<E, S>(a.u, row0, a.D, a.N, t0, q, d, u);
        load_scalars<E, S>(a.dt, row0, a.D, a.N, t0, q, d, dt);
        if (out && a.z) load_scalars<E, S>(a.z, row0, a.ldz, a.N, t0, q, d, z);
        load_bc<E, S>(a.b, row0, a.ldb, a.N, n, t0, g, lane, a.bc_vec, b);
        if (out) load_bc<E, S>(a.c, row0, a.ldc, a.N, n, t0, g, lane, a.bc_vec, c);
    }
    // dt becomes the length of the step, du its product with u
    __device__ __forceinline__ void steps(const ScanArgs& a, float bias, int n, int t0, int q, float (&du)[P::TL]) {
#pragma unroll
        for (int i = 0; i < P::TL; ++i) {
            float v = dt[i] + bias, s;
            if (a.softplus) softplus(v, &v, &s);
            const bool live = t0 + 4 * i + q < n;
            dt[i] = live ? v : 0.f;
            u[i] = live ? u[i] : 0.f;
            du[i] = dt[i] * u[i];
        }
    }
};

template <int SL>
__device__ __forceinline__ void lds_vec(const float* p, float (&f)[SL]) {
    if constexpr (SL == 2) {
        const f32x2_t w = *reinterpret_cast<const f32x2_t*>(p);
        f[0] = w[0];
        f[1] = w[1];
    } else {
#pragma unroll
        for (int j = 0; j < SL; j += 4) {
            const f32x4_t w = *reinterpret_cast<const f32x4_t*>(p + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[j + e] = w[e];
        }
    }
}
// Values of a lane in an exchange buffer: [SL / 4][64][4] (SL = 2: [64][2]), so that a wave's accesses are contiguous.
template <int SL>
__device__ __forceinline__ void ex_put(float* p, int lane, const float (&f)[SL]) {
    if constexpr (SL == 2) *reinterpret_cast<f32x2_t*>(p + 2 * lane) = f32x2_t{f[0], f[1]};
    else
#pragma unroll
        for (int j = 0; j < SL; j += 4)
            *reinterpret_cast<f32x4_t*>(p + 64 * j + 4 * lane) = f32x4_t{f[j], f[j + 1], f[j + 2], f[j + 3]};
}
template <int SL>
__device__ __forceinline__ void ex_get(const float* p, int lane, float (&f)[SL]) {
    if constexpr (SL == 2) {
        lds_vec<2>(p + 2 * lane, f);
    } else {
#pragma unroll
        for (int j = 0; j < SL; j += 4) {
            const f32x4_t w = *reinterpret_cast<const f32x4_t*>(p + 64 * j + 4 * lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[j + e] = w[e];
        }
    }
}

template <int SL>
__device__ __forceinline__ void state_get(const float* p, float (&f)[SL]) {  // 4-byte aligned or better
#pragma unroll
    for (int j = 0; j < SL; ++j) f[j] = p[j];
}

struct ScanPos {
    int cb, seg, b;
};
__device__ __forceinline__ bool scan_pos(const ScanArgs& a, ScanPos* p) {
    const long long id = xcd_order(blockIdx.x, gridDim.x);
    p->cb = (int)(id % a.cblocks);
    const long long rest = id / a.cblocks;
    p->seg = (int)(rest % a.nseg);
    p->b = (int)(rest / a.nseg);
    return p->b < a.B;
}

typedef void (*scan_kernel_t)(ScanArgs);
struct ScanKernels {
    scan_kernel_t local, join, full;
    int chunk, threads;  // tokens of a workgroup's chunk and threads of local and full
};
bool scan_kernels_get(bool bf16_in, bool bf16_out, int S, ScanKernels* o);

}  // namespace ret
