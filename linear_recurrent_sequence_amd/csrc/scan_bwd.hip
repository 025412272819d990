// Gradients of the selective scan. With dp = dy silu(z) the gradient before the gate and g_t that of the state h_t,
//     g_t = C_t dp_t + a_{t+1} g_{t+1},  e_t = g_t a_t (it goes on to h_{t-1}),  k_t = e_t h_{t-1} (= dL/da_t a_t)
//     du = dt sum_s g B + skip dp,  d(dt) = sum_s A k + u sum_s g B,  dA = sum_t dt k,
//     dB = sum_d g dt u,  dC = sum_d dp h,  dskip = sum_t dp u,  dz = dy y silu'(z).
//
// Sequences are cut into the chunks of a workgroup (NW blocks of T tokens). local finds what each chunk does to a state
// entering it and to a gradient leaving it (both from zero); join carries the states forward and the gradients back over the
// chunks; grad does the chunks, all independent: decays once, kept in 64 registers a lane, the waves' blocks joined through
// LDS both ways, the states kept in 64 more, then the tokens in reverse.
//
// dB and dC are sums over all channels. A wave adds its 16 channels up by halving exchanges, 8 values at a time (16
// instructions for 8 values where separate sums would take 32), keeps one register for each of its groups of 8 over the
// blocks of channels that its workgroup does one after another, and leaves them as partial sums for the sums' kernel. Every sum
// has one order. Through LDS instead (each wave's products laid down and read back transposed, one add a value) grad took
// 656 us where this took 635.
//
// Bound by the vector units: grad has 28 instructions per token, channel and state of a wave's 16 x 4, which are 440 us of the
// 598 that 2 x 2048 tokens of 8192 channels and 16 states take (two waves a SIMD, whose registers are full; waves of 8 tokens
// with room for four joined twice as often and took as long); local has 11 and takes 155, join 14, the sums 12: together 778.
// The tensors' bytes alone are 92. At 8 states 436 + 124 + 7 + 7 us.
//
// At 32 and 64 states a chunk is 32 and 16 tokens instead of 128, so that the states, gradients and sums at its edges are 4 and
// 8 times as many a token, and grad takes 264 and 346 registers, which leaves one wave a SIMD: grad 1558 and 3324 us, local 278
// and 614, join 93 and 444, the sums 30 and 108.
#include "scan_bwd.h"

namespace ret {

namespace {

// A sum is added to here, not when it is wanted: until then its terms, one a token, would take registers.
__device__ __forceinline__ void sum_now(float& s) { __asm__ volatile("" : "+v"(s)); }

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

// A wave's block of 16 channels, loaded ahead.
template <class E, int S>
struct GradBlock {
    typedef ScanShape<S> P;
    typedef Raw<E> R;
    typename R::one u[P::TL], dt[P::TL], z[P::TL], dy[P::TL];
    float A[P::SL], bias;
    __device__ __forceinline__ void load(const ScanBwdArgs& a, const ScanRows& r, int q, int d) {
        load_scalars<E, P>(r, a.f.u, a.f.D, q, d, u);
        load_scalars<E, P>(r, a.f.dt, a.f.D, q, d, dt);
        load_scalars<E, P>(r, a.dy, a.f.D, q, d, dy);
        if (a.f.z) load_scalars<E, P>(r, a.f.z, a.f.ldz, q, d, z);
        state_get<P::SL>(a.f.A + (long long)d * S + q * P::SL, A);
        bias = a.f.bias ? a.f.bias[d] : 0.f;
    }
};

// The decays of a wave's block, and what it leaves of a state from zero (h) and of a gradient behind it from zero (G).
template <int S>
__device__ __forceinline__ void grad_local(const float* Bs, const float* Cs, int q, const float (&A2)[S / 4],
                                           const float (&dt)[ScanShape<S>::TL], const float (&du)[ScanShape<S>::TL],
                                           const float (&dp)[ScanShape<S>::TL], float (&al)[ScanShape<S>::T][S / 4],
                                           float (&h)[S / 4], float (&G)[S / 4]) {
    constexpr int SL = S / 4, T = ScanShape<S>::T, GT = SL >= 16 ? 1 : 16 / SL;
    float v[2][GT][SL];
#pragma unroll
    for (int j = 0; j < SL; ++j) h[j] = G[j] = 0.f;
    lds_group<S, GT>(Bs, 0, q, v[0]);
#pragma unroll
    for (int k = 0; k < T; ++k) {
        if (k % GT == 0) {
            if (k + GT < T) lds_group<S, GT>(Bs, k + GT, q, v[(k / GT + 1) & 1]);
            else lds_group<S, GT>(Cs, T - GT, q, v[(k / GT + 1) & 1]);
        }
        const float(&B)[SL] = v[k / GT & 1][k % GT];
        const float dk = quad_of(dt[k / 4], k % 4), uk = quad_of(du[k / 4], k % 4);
#pragma unroll
        for (int j = 0; j < SL; ++j) {
            al[k][j] = __builtin_amdgcn_exp2f(dk * A2[j]);
            h[j] = fmaf(al[k][j], h[j], uk * B[j]);
        }
        if (k % GT == GT - 1) lds_order();
    }
#pragma unroll
    for (int k = T - 1; k >= 0; --k) {
        // group k / GT in reverse, the buffer after the last of the ones above
        const int g = (T / GT + (T - 1 - k) / GT) & 1;
        if (k % GT == GT - 1 && k >= GT) lds_group<S, GT>(Cs, k + 1 - 2 * GT, q, v[g ^ 1]);
        const float(&C)[SL] = v[g][k % GT];
        const float yk = quad_of(dp[k / 4], k % 4);
#pragma unroll
        for (int j = 0; j < SL; ++j) G[j] = fmaf(C[j], yk, G[j]) * al[k][j];
        if (k % GT == 0) lds_order();
    }
}

// Workgroup -> part, chunk and sequence with neighbouring parts on one XCD. A part is every parts_g-th block of 16 channels of
// a group, so that the workgroups that run at the same time share the 128-byte lines of the rows in their L2: taken as runs of
// neighbouring blocks, a line was gone before the next of its four blocks asked for it (3 times the reads from HBM).
struct GradPos {
    int part, chunk, b, g, cb0, cb1, step;
};
__device__ __forceinline__ bool grad_pos(const ScanBwdArgs& a, GradPos* p) {
    const int parts = a.parts_g * a.f.G, blocks_g = (a.f.D / a.f.G + kScanCh - 1) / kScanCh;
    const long long rest = scan_order(parts, a.deal_parts, &p->part);
    const int segs = deal_segs(a.deal_parts, a.f.nseg);
    p->chunk = (int)(rest % segs);
    p->b = (int)(rest / segs);
    p->g = p->part / a.parts_g;
    p->step = a.parts_g;
    p->cb0 = p->g * blocks_g + p->part % a.parts_g;
    p->cb1 = (p->g + 1) * blocks_g;
    return p->b < a.f.B && p->chunk < a.f.nseg;
}

// What each chunk leaves of a state from zero (h) and of a gradient behind it from zero (G), in one walk along the tokens: with
// P the product of the decays so far, h = a h + du B and G += P C dp. A wave walks a chunk on its own; where that leaves the
// card idle (SPLIT) a workgroup's waves walk a block of it each and join them.
template <class E, int S, bool SPLIT>
__global__ __launch_bounds__(ScanShape<S>::THREADS) void scan_local_bwd_kernel(ScanBwdArgs a) {
    typedef ScanShape<S> P;
    constexpr int SL = P::SL, T = P::T, TL = P::TL, NW = P::NW;
    __shared__ float bc[NW][2][T * S];
    __shared__ float ex[SPLIT ? NW : 1][3][SPLIT ? 64 * SL : 1];
    __shared__ float sums[SPLIT ? NW : 1][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane & 3, D = a.f.D;
    ScanPos at;
    if (!scan_pos(a.f, &at)) return;
    if (!SPLIT) {
        at.cb = at.cb * NW + w;
        if (at.cb * kScanCh >= D) return;
    }
    const int d = at.cb * kScanCh + (lane >> 2), dc = d < D ? d : D - 1;
    const int g = __builtin_amdgcn_readfirstlane(dc / (D / a.f.G));
    const int n = length_of(a.f.lengths, at.b, a.f.N), c0 = at.seg * P::CH, first = SPLIT ? c0 + w * T : c0;
    const int c1 = n - first < (SPLIT ? T : P::CH) ? n : first + (SPLIT ? T : P::CH);
    const long long row0 = (long long)at.b * a.f.N, seg = ((long long)at.b * a.f.nseg + at.seg) * D + d;
    const float bias = a.f.bias ? a.f.bias[dc] : 0.f;
    float A2[SL], h[SL], G[SL], p[SL], total = 0.f;
    state_get<SL>(a.f.A + (long long)dc * S + q * SL, A2);
#pragma unroll
    for (int j = 0; j < SL; ++j) {
        A2[j] = decay_rate(A2[j]);
        h[j] = G[j] = 0.f;
        p[j] = 1.f;
    }
    float *Bs = bc[w][0], *Cs = bc[w][1];
    ScanBlock<E, S> x;
    typename Raw<E>::one dy[TL];
    auto load = [&](int t0) {
        x.load(a.f, row0, t0, q, lane, dc, g, true);
        load_scalars<E, P>(ScanRows(row0, t0, a.f.N), a.dy, D, q, dc, dy);
    };
    if (first < c1) load(first);
    for (int t0 = first; t0 < c1; t0 += T) {
        float dt[TL], du[TL], u[TL], dp[TL];
        x.steps(a.f, bias, n, t0, q, dt, u, du);
        put_bc<E, P>(Bs, x.b, n, t0, lane);
        put_bc<E, P>(Cs, x.c, n, t0, lane);
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            dp[i] = Raw<E>::value(dy[i]);
            if (a.f.z) dp[i] *= swish_hw(Raw<E>::value(x.z[i]));
            if (t0 + 4 * i + q >= n) dp[i] = 0.f;
            total += dt[i];
        }
        if (t0 + T < c1) load(t0 + T);
        lds_order();
#pragma unroll
        for (int k = 0; k < T; ++k) {
            float B[SL], C[SL];
            lds_vec<SL>(Bs + k * S + q * SL, B);
            lds_vec<SL>(Cs + k * S + q * SL, C);
            const float dk = quad_of(dt[k / 4], k % 4), uk = quad_of(du[k / 4], k % 4), yk = quad_of(dp[k / 4], k % 4);
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                const float al = __builtin_amdgcn_exp2f(dk * A2[j]);
                h[j] = fmaf(al, h[j], uk * B[j]);
                p[j] *= al;
                G[j] = fmaf(p[j], C[j] * yk, G[j]);
            }
        }
        lds_order();
    }
    total = lanes_sum<4>(total);
    if (!SPLIT) {
        if (d >= D) return;
        state_put<SL>(a.f.seg_h + seg * S + q * SL, h);
        state_put<SL>(a.seg_g + seg * S + q * SL, G);
        if (q == 0) a.f.seg_dt[seg] = total;
        return;
    }
    ex_put<SL>(ex[w][0], lane, h);
    ex_put<SL>(ex[w][1], lane, p);
    ex_put<SL>(ex[w][2], lane, G);
    sums[w][lane] = total;
    __syncthreads();
    if (w > 1 || d >= D) return;
    // two waves join the waves' parts, the states forward and the gradients back
#pragma unroll
    for (int j = 0; j < SL; ++j) h[j] = 0.f;
    total = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
        const int o = w ? NW - 1 - v : v;
        float hv[SL], pv[SL];
        ex_get<SL>(ex[o][w ? 2 : 0], lane, hv);
        ex_get<SL>(ex[o][1], lane, pv);
#pragma unroll
        for (int j = 0; j < SL; ++j) h[j] = fmaf(pv[j], h[j], hv[j]);
        total += sums[v][lane];
    }
    state_put<SL>((w ? a.seg_g : a.f.seg_h) + seg * S + q * SL, h);
    if (w == 0 && q == 0) a.f.seg_dt[seg] = total;
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

template <class E, class O, int S>
__global__ __launch_bounds__(ScanShape<S>::THREADS) void scan_grad_kernel(ScanBwdArgs a) {
    typedef ScanShape<S> P;
    typedef Raw<E> R;
    typedef typename O::st ost;
    constexpr int SL = P::SL, T = P::T, TL = P::TL, NW = P::NW;
    __shared__ float bc[NW][2][T * S];
    __shared__ float ex[NW][3][64 * SL];
    __shared__ float red[NW][64 * SL];
    __shared__ float red2[NW][2][kScanCh];
    constexpr int NA = T * SL / 4;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane & 3;
    const int D = a.f.D, N = a.f.N;
    GradPos pos;
    if (!grad_pos(a, &pos)) return;
    const int part = pos.part, chunk = pos.chunk, b = pos.b, g = pos.g, cb0 = pos.cb0, cb1 = pos.cb1;
    const int n = length_of(a.f.lengths, b, N), c0 = chunk * P::CH, t0 = c0 + w * T;
    const int live = n - t0;  // tokens of the wave's block before n
    const long long row0 = (long long)b * N;
    float* out_bc = a.part_bc + ((long long)part * a.f.B * N + row0) * 2 * S;
    float* out_a = a.part_a + ((long long)b * a.f.nseg + chunk) * D * (S + 2);
    ost *du_p = (ost*)a.du, *ddt_p = (ost*)a.ddt, *dz_p = (ost*)a.dz;
    if (c0 >= n) {  // padding: zeros
        const int rows = N - c0 < P::CH ? N - c0 : P::CH;
        for (int cb = cb0; cb < cb1; cb += pos.step) {
            const int d0 = cb * kScanCh, cols = D - d0 < kScanCh ? D - d0 : kScanCh;
            for (int i = threadIdx.x; i < rows * kScanCh; i += P::THREADS) {
                if (i % kScanCh >= cols) continue;
                const long long o = (row0 + c0 + i / kScanCh) * D + d0 + i % kScanCh;
                store_out(du_p + o, 0.f);
                store_out(ddt_p + o, 0.f);
                if (dz_p) store_out(dz_p + o, 0.f);
            }
            for (int i = threadIdx.x; i < cols * S; i += P::THREADS) out_a[(long long)d0 * S + i] = 0.f;
            if ((int)threadIdx.x < cols)
                out_a[(long long)D * S + d0 + threadIdx.x] = out_a[(long long)D * (S + 1) + d0 + threadIdx.x] = 0.f;
        }
        for (int i = threadIdx.x; i < rows * 2 * S; i += P::THREADS) out_bc[(long long)c0 * 2 * S + i] = 0.f;
        return;
    }
    float *Bs = bc[w][0], *Cs = bc[w][1];
    {
        const ScanRows rows(row0, t0, N);
        put_bc<E, P>(Bs, load_bc<E, P>(rows, a.f.b, a.f.ldb, g, lane, a.f.bc_vec), n, t0, lane);
        put_bc<E, P>(Cs, load_bc<E, P>(rows, a.f.c, a.f.ldc, g, lane, a.f.bc_vec), n, t0, lane);
    }
    lds_order();
    constexpr int GT = SL >= 4 ? 1 : 2;  // tokens of B and C read at a time
    char *du_row = (char*)(du_p + (row0 + t0) * D), *ddt_row = (char*)(ddt_p + (row0 + t0) * D);
    char* dz_row = (char*)(dz_p + (row0 + t0) * D);
    float acc[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) acc[i] = 0.f;
    const ScanRows rows(row0, t0, N);
    const float* seg_h = a.f.seg_h + ((long long)b * a.f.nseg + chunk) * D * S;
    const float* seg_g = a.seg_g + ((long long)b * a.f.nseg + chunk) * D * S;
    GradBlock<E, S> x;
    {
        const int d = cb0 * kScanCh + (lane >> 2);
        x.load(a, rows, q, d < D ? d : D - 1);
    }
    for (int cb = cb0; cb < cb1; cb += pos.step) {
        const int d = cb * kScanCh + (lane >> 2), dc = d < D ? d : D - 1;
        const bool own = d < D;
        const float skip = a.f.skip && own ? a.f.skip[d] : 0.f;
        float A2[SL], hin[SL], gin[SL];
#pragma unroll
        for (int j = 0; j < SL; ++j) A2[j] = decay_rate(x.A[j]);
        state_get<SL>(seg_h + (long long)dc * S + q * SL, hin);
        state_get<SL>(seg_g + (long long)dc * S + q * SL, gin);
        float u[TL], dt[TL], du[TL], slope[TL], dp[TL], dzf[TL], total = 0.f;  // dzf: dy silu'(z)
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            u[i] = R::value(x.u[i]);
            dt[i] = R::value(x.dt[i]) + x.bias;
            dp[i] = R::value(x.dy[i]);
            slope[i] = 1.f;
            dzf[i] = 0.f;
        }
        if (a.f.softplus)
#pragma unroll
            for (int i = 0; i < TL; ++i) softplus(dt[i], &dt[i], &slope[i]);
        if (a.f.z)
#pragma unroll
            for (int i = 0; i < TL; ++i) {
                const float z = R::value(x.z[i]), s = sigmoid_hw(z);
                dzf[i] = dp[i] * (s * (1.f + z * (1.f - s)));
                dp[i] *= z * s;
            }
        if (t0 + T > n || (cb + 1) * kScanCh > D)
#pragma unroll
            for (int i = 0; i < TL; ++i)
                if (!own || t0 + 4 * i + q >= n) dt[i] = u[i] = dp[i] = dzf[i] = slope[i] = 0.f;
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            total += dt[i];
            du[i] = dt[i] * u[i];
        }
        float al[T][SL], h[SL], G[SL];
        grad_local<S>(Bs, Cs, q, A2, dt, du, dp, al, h, G);
        total = lanes_sum<4>(total);
        float p[SL];
#pragma unroll
        for (int j = 0; j < SL; ++j) p[j] = __builtin_amdgcn_exp2f(total * A2[j]);
        ex_put<SL>(ex[w][0], lane, h);
        ex_put<SL>(ex[w][1], lane, p);
        ex_put<SL>(ex[w][2], lane, G);
        __syncthreads();
        // half of the waves' parts in registers at a time
#pragma unroll
        for (int v0 = 0; v0 < NW; v0 += NW / 2) {
            float hv[NW / 2][SL], pv[NW / 2][SL];
#pragma unroll
            for (int e = 0; e < NW / 2; ++e) {
                if (v0 + e == NW - 1) continue;
                ex_get<SL>(ex[v0 + e][0], lane, hv[e]);
                ex_get<SL>(ex[v0 + e][1], lane, pv[e]);
            }
#pragma unroll
            for (int e = 0; e < NW / 2; ++e)
                if (v0 + e < NW - 1 && v0 + e < w)
#pragma unroll
                    for (int j = 0; j < SL; ++j) hin[j] = fmaf(pv[e][j], hin[j], hv[e][j]);
        }
#pragma unroll
        for (int v0 = NW / 2; v0 >= 0; v0 -= NW / 2) {
            float gv[NW / 2][SL], pv[NW / 2][SL];
#pragma unroll
            for (int e = 0; e < NW / 2; ++e) {
                if (v0 + e == 0) continue;
                ex_get<SL>(ex[v0 + e][2], lane, gv[e]);
                ex_get<SL>(ex[v0 + e][1], lane, pv[e]);
            }
#pragma unroll
            for (int e = NW / 2 - 1; e >= 0; --e)
                if (v0 + e > 0 && v0 + e > w)
#pragma unroll
                    for (int j = 0; j < SL; ++j) gin[j] = fmaf(pv[e][j], gin[j], gv[e][j]);
        }
        lds_order();
        float hh[T][SL], yp[4], b2[2][GT][SL], c2[2][GT][SL];
        lds_group<S, GT>(Bs, 0, q, b2[0]);
        lds_group<S, GT>(Cs, 0, q, c2[0]);
#pragma unroll
        for (int k = 0; k < T; ++k) {
            const int gk = k / GT & 1;
            if (k % GT == 0 && k + GT < T) {
                lds_group<S, GT>(Bs, k + GT, q, b2[gk ^ 1]);
                lds_group<S, GT>(Cs, k + GT, q, c2[gk ^ 1]);
            }
            if (k == 1)  // the gradient entering from behind: its parts have come by now
#pragma unroll
                for (int j = 0; j < SL; ++j) sum_now(gin[j]);
            const float uk = quad_of(du[k / 4], k % 4);
            yp[k % 4] = 0.f;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                hh[k][j] = fmaf(al[k][j], k ? hh[k ? k - 1 : 0][j] : hin[j], uk * b2[gk][k % GT][j]);
                yp[k % 4] = fmaf(c2[gk][k % GT][j], hh[k][j], yp[k % 4]);
            }
            if (k % 4 == 3) {
                float dz = fmaf(skip, u[k / 4], quad_sums(yp[0], yp[1], yp[2], yp[3], q)) * dzf[k / 4];
                if (k - 3 + q >= live) dz = 0.f;
                if (dz_p && own && t0 + k - 3 + q < N)
                    store_out((ost*)(dz_row + (__umul24(k - 3 + q, (uint32_t)D * (uint32_t)sizeof(ost)) +
                                               d * (uint32_t)sizeof(ost))), dz);
            }
            if (k % GT == GT - 1) lds_order();
        }
        float dA[SL], s1[4], s2[4], v[8], dskip = 0.f, dbias = 0.f;
        // Tokens from n on have steps of 0, but the last state and its gradient pass over them: what is not finite, or
        // overflows with A, would come into dA. So the last state's one product, in dC of token n - 1, is added here, and the
        // states from there on become 0.
        if (live < T) {
            float yk = 0.f;
#pragma unroll
            for (int k = 0; k < T; ++k)
                if (k == live - 1) yk = quad_of(dp[k / 4], k % 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                const float dc = yk * hh[T - 1][j];
                if constexpr (SL == 2) v[4 + j] = live & 1 ? dc : 0.f, v[6 + j] = live & 1 ? 0.f : dc;
                else v[4 + j % 4] = dc;
                if (SL == 2 ? j == 0 : j % 4 != 3) continue;
                const float sum = halving_sums(v, lane);
#pragma unroll
                for (int k = 0; k < T; ++k)
                    if (k == live - 1) acc[SL == 2 ? k / 2 : k * (SL / 4) + j / 4] += sum;
            }
#pragma unroll
            for (int j = 0; j < SL; ++j) {
#pragma unroll
                for (int k = 0; k < T; ++k)
                    if (k >= live - 1) hh[k][j] = 0.f;
                if (live <= 0) hin[j] = gin[j] = 0.f;
            }
        }
        // in reverse, from the group that the loop above read last
        constexpr int last = (T / GT - 1) & 1;
#pragma unroll
        for (int j = 0; j < SL; ++j) dA[j] = 0.f;
#pragma unroll
        for (int k = T - 1; k >= 0; --k) {
            const int gk = (last + (T - 1 - k) / GT) & 1;
            if (k % GT == GT - 1 && k >= GT) {
                lds_group<S, GT>(Bs, k + 1 - 2 * GT, q, b2[gk ^ 1]);
                lds_group<S, GT>(Cs, k + 1 - 2 * GT, q, c2[gk ^ 1]);
            }
            const float(&B)[SL] = b2[gk][k % GT];
            const float(&C)[SL] = c2[gk][k % GT];
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
                    if (j % 4 == 3) sum_now(acc[k * (SL / 4) + j / 4] += halving_sums(v, lane));
            }
            if constexpr (SL == 2)
                if (k % 2 == 0) sum_now(acc[k / 2] += halving_sums(v, lane));
#pragma unroll
            for (int j = 0; j < SL; ++j) sum_now(dA[j]);
            if (k % 4 == 0) {
                const int i = k / 4;
                const float gb = quad_sums(s1[0], s1[1], s1[2], s1[3], q);
                float ak = quad_sums(s2[0], s2[1], s2[2], s2[3], q);
                if (slope[i] == 0.f) ak = 0.f;  // a step below fp32's range: A times what stays may be outside of it
                float x1 = fmaf(skip, dp[i], dt[i] * gb), x2 = fmaf(kLn2, ak, u[i] * gb) * slope[i];
                if (k + q >= live) x1 = x2 = 0.f;
                dskip = fmaf(dp[i], u[i], dskip);
                dbias += x2;
                sum_now(dskip);
                sum_now(dbias);
                if (own && t0 + k + q < N) {
                    const uint32_t o = __umul24(k + q, (uint32_t)D * (uint32_t)sizeof(ost)) + d * (uint32_t)sizeof(ost);
                    store_out((ost*)(du_row + o), x1);
                    store_out((ost*)(ddt_row + o), x2);
                }
            }
            if (k % GT == 0) lds_order();
            if (k == T / 2 && cb + pos.step < cb1) {  // half of the decays and states are done with: room for the next channels
                const int e = d + pos.step * kScanCh;
                int ql = q;  // the rows' offsets, made anew: kept from turn to turn they would take registers
                __asm__ volatile("" : "+v"(ql));
                x.load(a, rows, ql, e < D ? e : D - 1);
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
    for (int i = 0; i < NA; ++i) {
        const float sum = acc[i] + dpp_mov<0x12c>(acc[i]);  // row_ror:12, the value of lane + 4: whole where bit 2 is clear
        const int hi = lane >> 5, mid = lane >> 4 & 1, lo = lane >> 3 & 1;
        const int k = SL == 2 ? 2 * i + mid : i / (SL / 4 ? SL / 4 : 1);
        const int s = SL == 2 ? 2 * q + lo : q * SL + i % (SL / 4 ? SL / 4 : 1) * 4 + 2 * mid + lo;
        if (!(lane & 4) && t0 + k < N) out_bc[(long long)(t0 + k) * 2 * S + hi * S + s] = t0 + k < n ? sum : 0.f;
    }
}

// dB and dC from the parts of their group, and the sums of part_a.
template <class O, int S>
__global__ __launch_bounds__(kColSumThreads) void scan_sums_kernel(ScanBwdArgs a) {
    if (blockIdx.x >= a.bc_blocks) return part_sums(a.cols, blockIdx.x - a.bc_blocks);
    const long long rows = (long long)a.f.B * a.f.N, per = rows * 2 * S;
    const long long id = (long long)blockIdx.x * kColSumThreads + threadIdx.x, i = id % per;
    const int g = (int)(id / per), which = (int)(i / S % 2), s = (int)(i % S);
    if (g >= a.f.G) return;
    const float* p = a.part_bc + (long long)g * a.parts_g * per + i;
    float t = 0.f;
    for (int k = 0; k < a.parts_g; k += 8) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = p[(k + e < a.parts_g ? k + e : k) * per];
#pragma unroll
        for (int e = 0; e < 8; ++e) t += k + e < a.parts_g ? x[e] : 0.f;
    }
    typename O::st* out = (typename O::st*)(which ? a.dc : a.db);
    store_out(out + (i / (2 * S) * a.f.G + g) * S + s, t);
}

template <class E, class O, int S>
bool pick(ScanBwdKernels* o) {
    *o = {scan_local_bwd_kernel<E, S, false>, scan_local_bwd_kernel<E, S, true>, scan_join_bwd_kernel<S>,
          scan_grad_kernel<E, O, S>, scan_sums_kernel<O, S>,
          ScanShape<S>::CH, ScanShape<S>::NW};
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
