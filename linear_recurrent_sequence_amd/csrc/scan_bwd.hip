// Gradients of the selective scan. With dp = dy silu(z) the gradient before the gate and g_t that of the state h_t,
//     g_t = C_t dp_t + a_{t+1} g_{t+1},  e_t = g_t a_t (it goes on to h_{t-1}),  k_t = e_t h_{t-1} (= dL/da_t a_t)
//     du = dt sum_s g B + skip dp,  d(dt) = sum_s A k + u sum_s g B,  dA = sum_t dt k,
//     dB = sum_d g dt u,  dC = sum_d dp h,  dskip = sum_t dp u,  dz = dy y silu'(z).
//
// Sequences are cut into the chunks of a workgroup (NW blocks of T tokens). local finds what each chunk does to a state
// entering it and to a gradient leaving it (both from zero, one exp2 a state); join carries the states forward and the
// gradients back over the chunks; grad does the chunks, all independent: decays once, kept in 64 registers a lane, the
// waves' blocks joined through LDS both ways, the states kept in 64 more, then the tokens in reverse.
//
// dB and dC are sums over all channels. A wave adds its 16 channels up by halving exchanges, 8 values at a time (16
// instructions for 8 values where separate sums would take 32), keeps one register for each of its 16 groups of 8 over the
// `run` blocks of channels that its workgroup does one after another, and leaves them as partial sums for sum_bc. Every sum
// has one order.
#include "scan_bwd.h"

namespace ret {

namespace {

// Sums of 8 values over the lanes of equal q (lane & 3): after the exchanges the lanes of equal bits 3..5 hold value
// 4 bit5 + 2 bit4 + bit3, the two of them that differ in bit 2 each a half of the sum.
__device__ __forceinline__ float halving_sums(const float (&v)[8], int lane) {
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[4 + i]), false, false);
        r[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    float t[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(r[i]), __float_as_uint(r[2 + i]), false, false);
        t[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    const bool high = lane & 8;
    return (high ? t[1] : t[0]) + dpp_mov<0x128>(high ? t[0] : t[1]);  // row_ror:8
}

// What both kernels do with a block: steps and gradients before the gate.
template <class E, int S>
struct GradBlock {
    typedef ScanShape<S> P;
    float u[P::TL], dt[P::TL], z[P::TL], dy[P::TL];
    __device__ __forceinline__ void load(const ScanBwdArgs& a, long long row0, int t0, int q, int d) {
        load_scalars<E, S>(a.f.u, row0, a.f.D, a.f.N, t0, q, d, u);
        load_scalars<E, S>(a.f.dt, row0, a.f.D, a.f.N, t0, q, d, dt);
        load_scalars<E, S>(a.dy, row0, a.f.D, a.f.N, t0, q, d, dy);
        if (a.f.z) load_scalars<E, S>(a.f.z, row0, a.f.ldz, a.f.N, t0, q, d, z);
    }
};

template <class E, int S>
__global__ __launch_bounds__(ScanShape<S>::THREADS) void scan_local_bwd_kernel(ScanBwdArgs a) {
    typedef ScanShape<S> P;
    constexpr int SL = P::SL, T = P::T, TL = P::TL;
    __shared__ float bc[P::NW][2][T * S];
    __shared__ float ex[P::NW][3][64 * SL];
    __shared__ float sums[P::NW][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane & 3;
    ScanPos at;
    if (!scan_pos(a.f, &at)) return;
    const int d = at.cb * kScanCh + (lane >> 2), D = a.f.D, dc = d < D ? d : D - 1;
    const int g = __builtin_amdgcn_readfirstlane(dc / (D / a.f.G));
    const int n = scan_length(a.f.lengths, at.b, a.f.N), c0 = at.seg * P::CH, t0 = c0 + w * T;
    const long long row0 = (long long)at.b * a.f.N, seg = ((long long)at.b * a.f.nseg + at.seg) * D + d;
    if (c0 >= n) {  // nothing in it: neither a state nor a gradient changes
        if (w == 0 && d < D) {
#pragma unroll
            for (int j = 0; j < SL; ++j) a.f.seg_h[seg * S + q * SL + j] = a.seg_g[seg * S + q * SL + j] = 0.f;
            if (q == 0) a.f.seg_dt[seg] = 0.f;
        }
        return;
    }
    GradBlock<E, S> x;
    x.load(a, row0, t0, q, dc);
    float *Bs = bc[w][0], *Cs = bc[w][1], v[4];
    load_bc<E, S>(a.f.b, row0, a.f.ldb, a.f.N, n, t0, g, lane, a.f.bc_vec, v);
    *reinterpret_cast<f32x4_t*>(Bs + 4 * lane) = f32x4_t{v[0], v[1], v[2], v[3]};
    load_bc<E, S>(a.f.c, row0, a.f.ldc, a.f.N, n, t0, g, lane, a.f.bc_vec, v);
    *reinterpret_cast<f32x4_t*>(Cs + 4 * lane) = f32x4_t{v[0], v[1], v[2], v[3]};
    const float bias = a.f.bias ? a.f.bias[dc] : 0.f;
    float A2[SL], h[SL], G[SL], total = 0.f, du[TL];
#pragma unroll
    for (int j = 0; j < SL; ++j) {
        A2[j] = decay_rate(a.f.A[(long long)dc * S + q * SL + j]);
        h[j] = G[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < TL; ++i) {
        const bool live = t0 + 4 * i + q < n;
        float s, step = x.dt[i] + bias;
        if (a.f.softplus) softplus(step, &step, &s);
        total += x.dt[i] = live ? step : 0.f;
        du[i] = live ? x.dt[i] * x.u[i] : 0.f;
        x.dy[i] = live ? a.f.z ? x.dy[i] * swish_hw(x.z[i]) : x.dy[i] : 0.f;
    }
    lds_order();
    float al[T][SL];
#pragma unroll
    for (int k = 0; k < T; ++k) {
        float B[SL];
        lds_vec<SL>(Bs + k * S + q * SL, B);
        const float dk = quad_of(x.dt[k / 4], k % 4), uk = quad_of(du[k / 4], k % 4);
#pragma unroll
        for (int j = 0; j < SL; ++j) {
            al[k][j] = __builtin_amdgcn_exp2f(dk * A2[j]);
            h[j] = fmaf(al[k][j], h[j], uk * B[j]);
        }
    }
#pragma unroll
    for (int k = T - 1; k >= 0; --k) {
        float C[SL];
        lds_vec<SL>(Cs + k * S + q * SL, C);
        const float yk = quad_of(x.dy[k / 4], k % 4);
#pragma unroll
        for (int j = 0; j < SL; ++j) G[j] = fmaf(C[j], yk, G[j]) * al[k][j];
    }
    total = lanes_sum<4>(total);
    float p[SL];
#pragma unroll
    for (int j = 0; j < SL; ++j) p[j] = __builtin_amdgcn_exp2f(total * A2[j]);
    ex_put<SL>(ex[w][0], lane, h);
    ex_put<SL>(ex[w][1], lane, p);
    ex_put<SL>(ex[w][2], lane, G);
    sums[w][lane] = total;
    __syncthreads();
    if (w > 1 || d >= D) return;
    if (w == 0) {
#pragma unroll
        for (int v = 1; v < P::NW; ++v) {
            float hv[SL], pv[SL];
            ex_get<SL>(ex[v][0], lane, hv);
            ex_get<SL>(ex[v][1], lane, pv);
#pragma unroll
            for (int j = 0; j < SL; ++j) h[j] = fmaf(pv[j], h[j], hv[j]);
            total += sums[v][lane];
        }
#pragma unroll
        for (int j = 0; j < SL; ++j) a.f.seg_h[seg * S + q * SL + j] = h[j];
        if (q == 0) a.f.seg_dt[seg] = total;
    } else {
        ex_get<SL>(ex[P::NW - 1][2], lane, G);
#pragma unroll
        for (int v = P::NW - 2; v >= 0; --v) {
            float gv[SL], pv[SL];
            ex_get<SL>(ex[v][2], lane, gv);
            ex_get<SL>(ex[v][1], lane, pv);
#pragma unroll
            for (int j = 0; j < SL; ++j) G[j] = fmaf(pv[j], G[j], gv[j]);
        }
#pragma unroll
        for (int j = 0; j < SL; ++j) a.seg_g[seg * S + q * SL + j] = G[j];
    }
}

// Chunks' states and gradients from zero -> the states entering and the gradients leaving the chunks, in place.
template <int S>
__global__ __launch_bounds__(256) void scan_join_bwd_kernel(ScanBwdArgs a) {
    const long long per = (long long)a.f.D * S, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const int b = blockIdx.y, d = (int)(i / S), K = a.f.nseg;
    const float A2 = decay_rate(a.f.A[i]);
    float* hp = a.f.seg_h + (long long)b * K * per + i;
    float* gp = a.seg_g + (long long)b * K * per + i;
    const float* sp = a.f.seg_dt + (long long)b * K * a.f.D + d;
    constexpr int U = 8;
    if (blockIdx.z == 0) {
        float h = a.f.state_in ? a.f.state_in[b * per + i] : 0.f;
        for (int k = 0; k < K; k += U) {
            float x[U], p[U];
#pragma unroll
            for (int e = 0; e < U; ++e) {
                const int s = k + e < K ? k + e : K - 1;
                x[e] = hp[s * per];
                p[e] = sp[(long long)s * a.f.D];
            }
#pragma unroll
            for (int e = 0; e < U; ++e) {
                if (k + e >= K) break;
                hp[(k + e) * per] = h;
                h = fmaf(__builtin_amdgcn_exp2f(p[e] * A2), h, x[e]);
            }
        }
    } else {
        float g = a.dstate_out ? a.dstate_out[b * per + i] : 0.f;
        for (int k = K - 1; k >= 0; k -= U) {
            float x[U], p[U];
#pragma unroll
            for (int e = 0; e < U; ++e) {
                const int s = k - e > 0 ? k - e : 0;
                x[e] = gp[s * per];
                p[e] = sp[(long long)s * a.f.D];
            }
#pragma unroll
            for (int e = 0; e < U; ++e) {
                if (k - e < 0) break;
                gp[(k - e) * per] = g;
                g = fmaf(__builtin_amdgcn_exp2f(p[e] * A2), g, x[e]);
            }
        }
        if (a.dstate_in) a.dstate_in[b * per + i] = g;
    }
}

// blockIdx.x -> (part, chunk, b) with neighbouring parts on one XCD; a part is `run` blocks of channels of one group.
template <class E, class O, int S>
__global__ __launch_bounds__(ScanShape<S>::THREADS) void scan_grad_kernel(ScanBwdArgs a) {
    typedef ScanShape<S> P;
    typedef typename O::st ost;
    constexpr int SL = P::SL, T = P::T, TL = P::TL, NW = P::NW;
    __shared__ float bc[NW][2][T * S];
    __shared__ float ex[NW][3][64 * SL];
    __shared__ float red[NW][64 * SL];
    __shared__ float red2[NW][2][kScanCh];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane & 3;
    const int parts = a.parts_g * a.f.G, D = a.f.D, N = a.f.N;
    const long long id = xcd_order(blockIdx.x, gridDim.x);
    const int part = (int)(id % parts), chunk = (int)(id / parts % a.f.nseg), b = (int)(id / parts / a.f.nseg);
    if (b >= a.f.B) return;
    const int g = part / a.parts_g, blocks_g = (D / a.f.G + kScanCh - 1) / kScanCh;
    const int cb0 = g * blocks_g + part % a.parts_g * a.run;
    const int cb1 = cb0 + a.run < (g + 1) * blocks_g ? cb0 + a.run : (g + 1) * blocks_g;
    const int n = scan_length(a.f.lengths, b, N), c0 = chunk * P::CH, t0 = c0 + w * T;
    const long long row0 = (long long)b * N;
    float* out_bc = a.part_bc + ((long long)part * a.f.B * N + row0) * 2 * S;
    float* out_a = a.part_a + ((long long)b * a.f.nseg + chunk) * D * (S + 2);
    ost *du_p = (ost*)a.du, *ddt_p = (ost*)a.ddt, *dz_p = (ost*)a.dz;
    if (c0 >= n) {  // padding: zeros
        const int rows = N - c0 < P::CH ? N - c0 : P::CH;
        const int d0 = cb0 * kScanCh, cols = (cb1 * kScanCh < D ? cb1 * kScanCh : D) - d0;
        for (int i = threadIdx.x; i < rows * cols; i += P::THREADS) {
            const long long o = (row0 + c0 + i / cols) * D + d0 + i % cols;
            store_out(du_p + o, 0.f);
            store_out(ddt_p + o, 0.f);
            if (dz_p) store_out(dz_p + o, 0.f);
        }
        for (int i = threadIdx.x; i < rows * 2 * S; i += P::THREADS) out_bc[(long long)c0 * 2 * S + i] = 0.f;
        for (int i = threadIdx.x; i < cols * S; i += P::THREADS) out_a[(long long)d0 * S + i] = 0.f;
        for (int i = threadIdx.x; i < cols; i += P::THREADS)
            out_a[(long long)D * S + d0 + i] = out_a[(long long)D * (S + 1) + d0 + i] = 0.f;
        return;
    }
    float *Bs = bc[w][0], *Cs = bc[w][1];
    {
        float v[4];
        load_bc<E, S>(a.f.b, row0, a.f.ldb, N, n, t0, g, lane, a.f.bc_vec, v);
        *reinterpret_cast<f32x4_t*>(Bs + 4 * lane) = f32x4_t{v[0], v[1], v[2], v[3]};
        load_bc<E, S>(a.f.c, row0, a.f.ldc, N, n, t0, g, lane, a.f.bc_vec, v);
        *reinterpret_cast<f32x4_t*>(Cs + 4 * lane) = f32x4_t{v[0], v[1], v[2], v[3]};
    }
    lds_order();
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    GradBlock<E, S> x;
    {
        const int d = cb0 * kScanCh + (lane >> 2);
        x.load(a, row0, t0, q, d < D ? d : D - 1);
    }
    for (int cb = cb0; cb < cb1; ++cb) {
        const int d = cb * kScanCh + (lane >> 2), dc = d < D ? d : D - 1;
        const bool own = d < D;
        const long long seg = (((long long)b * a.f.nseg + chunk) * D + dc) * S + q * SL;
        float A2[SL], hin[SL], gin[SL];
        state_get<SL>(a.f.seg_h + seg, hin);
        state_get<SL>(a.seg_g + seg, gin);
#pragma unroll
        for (int j = 0; j < SL; ++j) A2[j] = decay_rate(a.f.A[(long long)dc * S + q * SL + j]);
        const float bias = a.f.bias ? a.f.bias[dc] : 0.f, skip = a.f.skip ? a.f.skip[dc] : 0.f;
        float u[TL], dt[TL], du[TL], slope[TL], dp[TL], dzf[TL], total = 0.f;  // dzf: dy silu'(z)
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            const bool live = own && t0 + 4 * i + q < n;
            float step = x.dt[i] + bias;
            slope[i] = 1.f;
            if (a.f.softplus) softplus(step, &step, &slope[i]);
            if (!live) slope[i] = 0.f;
            total += dt[i] = live ? step : 0.f;
            u[i] = live ? x.u[i] : 0.f;
            du[i] = dt[i] * u[i];
            dp[i] = live ? x.dy[i] : 0.f;
            dzf[i] = 0.f;
            if (a.f.z && live) {
                const float s = sigmoid_of(x.z[i]);
                dzf[i] = dp[i] * (s * (1.f + x.z[i] * (1.f - s)));
                dp[i] *= x.z[i] * s;
            }
        }
        if (cb + 1 < cb1) {
            const int e = d + kScanCh;
            x.load(a, row0, t0, q, e < D ? e : D - 1);
        }
        float al[T][SL], h[SL], G[SL];
#pragma unroll
        for (int j = 0; j < SL; ++j) h[j] = G[j] = 0.f;
#pragma unroll
        for (int k = 0; k < T; ++k) {
            float B[SL];
            lds_vec<SL>(Bs + k * S + q * SL, B);
            const float dk = quad_of(dt[k / 4], k % 4), uk = quad_of(du[k / 4], k % 4);
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                al[k][j] = __builtin_amdgcn_exp2f(dk * A2[j]);
                h[j] = fmaf(al[k][j], h[j], uk * B[j]);
            }
        }
#pragma unroll
        for (int k = T - 1; k >= 0; --k) {
            float C[SL];
            lds_vec<SL>(Cs + k * S + q * SL, C);
            const float yk = quad_of(dp[k / 4], k % 4);
#pragma unroll
            for (int j = 0; j < SL; ++j) G[j] = fmaf(C[j], yk, G[j]) * al[k][j];
        }
        total = lanes_sum<4>(total);
        float p[SL];
#pragma unroll
        for (int j = 0; j < SL; ++j) p[j] = __builtin_amdgcn_exp2f(total * A2[j]);
        ex_put<SL>(ex[w][0], lane, h);
        ex_put<SL>(ex[w][1], lane, p);
        ex_put<SL>(ex[w][2], lane, G);
        __syncthreads();
        for (int v = 0; v < w; ++v) {
            float hv[SL], pv[SL];
            ex_get<SL>(ex[v][0], lane, hv);
            ex_get<SL>(ex[v][1], lane, pv);
#pragma unroll
            for (int j = 0; j < SL; ++j) hin[j] = fmaf(pv[j], hin[j], hv[j]);
        }
        for (int v = NW - 1; v > w; --v) {
            float gv[SL], pv[SL];
            ex_get<SL>(ex[v][2], lane, gv);
            ex_get<SL>(ex[v][1], lane, pv);
#pragma unroll
            for (int j = 0; j < SL; ++j) gin[j] = fmaf(pv[j], gin[j], gv[j]);
        }
        float hh[T][SL], yp[T];
#pragma unroll
        for (int k = 0; k < T; ++k) {
            float B[SL], C[SL];
            lds_vec<SL>(Bs + k * S + q * SL, B);
            lds_vec<SL>(Cs + k * S + q * SL, C);
            const float uk = quad_of(du[k / 4], k % 4);
            yp[k] = 0.f;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                hh[k][j] = fmaf(al[k][j], k ? hh[k ? k - 1 : 0][j] : hin[j], uk * B[j]);
                yp[k] = fmaf(C[j], hh[k][j], yp[k]);
            }
        }
        if (dz_p)
#pragma unroll
            for (int i = 0; i < TL; ++i) {
                float y = quad_sums(yp[4 * i], yp[4 * i + 1], yp[4 * i + 2], yp[4 * i + 3], q);
                y = fmaf(skip, u[i], y);
                const int t = t0 + 4 * i + q;
                if (t < N && own) store_out(dz_p + (row0 + t) * D + d, dzf[i] * y);
            }
        float dA[SL], s1[4], s2[4], v[8], dskip = 0.f, dbias = 0.f;
#pragma unroll
        for (int j = 0; j < SL; ++j) dA[j] = 0.f;
#pragma unroll
        for (int k = T - 1; k >= 0; --k) {
            float B[SL], C[SL];
            lds_vec<SL>(Bs + k * S + q * SL, B);
            lds_vec<SL>(Cs + k * S + q * SL, C);
            const float dk = quad_of(dt[k / 4], k % 4), uk = quad_of(du[k / 4], k % 4), yk = quad_of(dp[k / 4], k % 4);
            s1[k % 4] = s2[k % 4] = 0.f;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                gin[j] = fmaf(C[j], yk, gin[j]);
                const int at = SL == 2 ? 2 * (k & 1) + j : j & 3;
                v[at] = uk * gin[j];
                v[4 + at] = yk * hh[k][j];
                s1[k % 4] = fmaf(gin[j], B[j], s1[k % 4]);
                gin[j] *= al[k][j];
                const float along = gin[j] * (k ? hh[k ? k - 1 : 0][j] : hin[j]);
                s2[k % 4] = fmaf(A2[j], along, s2[k % 4]);
                dA[j] = fmaf(dk, along, dA[j]);
                if constexpr (SL >= 4)
                    if (j % 4 == 3) acc[k * (SL / 4) + j / 4] += halving_sums(v, lane);
            }
            if constexpr (SL == 2)
                if (k % 2 == 0) acc[k / 2] += halving_sums(v, lane);
            if (k % 4 == 0) {
                const int i = k / 4, t = t0 + 4 * i + q;
                const float gb = quad_sums(s1[0], s1[1], s1[2], s1[3], q), ak = quad_sums(s2[0], s2[1], s2[2], s2[3], q);
                const float ddt = fmaf(kLn2, ak, u[i] * gb) * slope[i];
                dskip = fmaf(dp[i], u[i], dskip);
                dbias += ddt;
                if (t < N && own) {
                    store_out(du_p + (row0 + t) * D + d, t < n ? fmaf(skip, dp[i], dt[i] * gb) : 0.f);
                    store_out(ddt_p + (row0 + t) * D + d, t < n ? ddt : 0.f);
                }
            }
        }
        dskip = lanes_sum<4>(dskip);
        dbias = lanes_sum<4>(dbias);
        ex_put<SL>(red[w], lane, dA);
        if (q == 0) {
            red2[w][0][lane >> 2] = dskip;
            red2[w][1][lane >> 2] = dbias;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * SL; i += P::THREADS) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < NW; ++v) s += red[v][i];
            const int l = SL == 2 ? i / 2 : i % 256 / 4, j = SL == 2 ? i % 2 : i / 256 * 4 + i % 4;
            const int e = cb * kScanCh + (l >> 2);
            if (e < D) out_a[(long long)e * S + (l & 3) * SL + j] = s;
        }
        if (threadIdx.x < 2 * kScanCh) {
            const int which = threadIdx.x / kScanCh, c = threadIdx.x % kScanCh, e = cb * kScanCh + c;
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < NW; ++v) s += red2[v][which][c];
            if (e < D) out_a[(long long)D * (S + which) + e] = s;
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        acc[i] += dpp_mov<0x12c>(acc[i]);  // row_ror:12, the value of lane + 4: whole where bit 2 is clear
        const int hi = lane >> 5, mid = lane >> 4 & 1, lo = lane >> 3 & 1;
        const int k = SL == 2 ? 2 * i + mid : i / (SL / 4 ? SL / 4 : 1);
        const int s = SL == 2 ? 2 * q + lo : q * SL + i % (SL / 4 ? SL / 4 : 1) * 4 + 2 * mid + lo;
        if (!(lane & 4) && t0 + k < N) out_bc[(long long)(t0 + k) * 2 * S + hi * S + s] = t0 + k < n ? acc[i] : 0.f;
    }
}

// dB and dC from the parts of their group.
template <class O, int S>
__global__ __launch_bounds__(256) void scan_sum_bc_kernel(ScanBwdArgs a) {
    const long long rows = (long long)a.f.B * a.f.N, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * 2 * S) return;
    const int g = blockIdx.y, which = (int)(i / S % 2), s = (int)(i % S);
    const float* p = a.part_bc + (long long)g * a.parts_g * rows * 2 * S + i;
    float t = 0.f;
    for (int k = 0; k < a.parts_g; k += 8) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = p[(k + e < a.parts_g ? k + e : k) * rows * 2 * S];
#pragma unroll
        for (int e = 0; e < 8; ++e) t += k + e < a.parts_g ? x[e] : 0.f;
    }
    typename O::st* out = (typename O::st*)(which ? a.dc : a.db);
    store_out(out + (i / (2 * S) * a.f.G + g) * S + s, t);
}

template <class E, class O, int S>
bool pick(ScanBwdKernels* o) {
    *o = {scan_local_bwd_kernel<E, S>, scan_join_bwd_kernel<S>, scan_grad_kernel<E, O, S>, scan_sum_bc_kernel<O, S>,
          ScanShape<S>::CH, ScanShape<S>::THREADS};
    return true;
}
template <class E, class O>
bool of_states(int S, ScanBwdKernels* o) {
    switch (S) {
        case 8: return pick<E, O, 8>(o);
        case 16: return pick<E, O, 16>(o);
        case 32: return pick<E, O, 32>(o);
        case 64: return pick<E, O, 64>(o);
        default: return false;
    }
}

}  // namespace

bool scan_bwd_kernels_get(bool bf16_in, bool bf16_out, int S, ScanBwdKernels* o) {
    if (!bf16_in) return of_states<F32, F32>(S, o);
    return bf16_out ? of_states<BF16, BF16>(S, o) : of_states<BF16, F32>(S, o);
}

}  // namespace ret
