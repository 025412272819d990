// Selective scan over sequences, forward. Bound by the vector units: per token, channel and state one exp2 (about twice the time
// of the other instructions) and four products or sums where the states are reached in one pass, 24 cycles of a SIMD for 64 of
// them; the tensors' bytes take half of that time at 16 states.
//
// walk: a wave takes 16 channels along the tokens with their states in registers; one pass, for as many waves as there are
// blocks of channels. 4 x 2741 tokens of 8192 channels (16 states, bf16, gated): 469 us, 2 waves a SIMD, 186 cycles a token
// and wave where 148 are left when 5 share the SIMD (as many as its 87 registers let): B and C of a token come from LDS right
// before they are used, and few waves leave that time open. fp32: 510 us.
//
// chunks: a workgroup walks the chunks of its sequence, NW waves a chunk, each its own T tokens. A wave computes its decays
// once, keeps them in 64 registers a lane, and from them the state its tokens leave if they start from zero; the waves exchange
// these with the products of their decays, each forms the state entering its tokens, and goes over them again with the
// decays it kept (three products a state more, where a second exp2 would cost the time of four). A token takes 30 ns where a
// walking wave takes 122, but three times the instructions: for few blocks of channels. 64 tokens of 128 channels 7.6 us.
//
// Few, long sequences are cut into segments: local, a walk, leaves each segment's state from zero; join carries the states
// over the segments by their decays, exp(A sum dt); then the walk starts from them. 65536 tokens of 1024 channels: 189 + 15 +
// 279 us, of which the cycles above, in two passes, are 320.
#include "scan.h"

namespace ret {

namespace {

// A wave on its own: 16 channels of a segment, token by token. LOCAL: the states that the segment leaves if it starts from
// zero, and the sum of its steps; else the outputs, from the state entering it.
template <class E, class O, int S, bool LOCAL>
__global__ __launch_bounds__(256) void scan_walk_kernel(ScanArgs a) {
    typedef ScanShape<S> P;
    constexpr int SL = P::SL, T = P::T, TL = P::TL;
    __shared__ float bc[4][2][T * S];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane & 3;
    ScanPos at;
    if (!scan_pos(a, &at) || (LOCAL && at.seg == a.nseg - 1)) return;  // nothing follows the last segment
    at.cb = 4 * at.cb + w;
    if (at.cb * kScanCh >= a.D) return;
    const int d = at.cb * kScanCh + (lane >> 2), dc = d < a.D ? d : a.D - 1;
    const int g = __builtin_amdgcn_readfirstlane(dc / (a.D / a.G));  // one for the whole wave
    const int n = length_of(a.lengths, at.b, a.N);
    const int s0 = at.seg * a.seg_tokens, s1 = a.N - s0 < a.seg_tokens ? a.N : s0 + a.seg_tokens, e1 = s1 < n ? s1 : n;
    const long long row0 = (long long)at.b * a.N;
    const float bias = a.bias ? a.bias[dc] : 0.f, skip = !LOCAL && a.skip ? a.skip[dc] : 0.f;
    float A2[SL], h[SL], total = 0.f;
    const long long st = ((long long)at.b * a.D + dc) * S + q * SL;
#pragma unroll
    for (int j = 0; j < SL; ++j) {
        A2[j] = decay_rate(a.A[(long long)dc * S + q * SL + j]);
        h[j] = 0.f;
    }
    const long long seg = ((long long)at.b * a.nseg + at.seg) * a.D + dc;
    if (!LOCAL) {
        if (a.nseg > 1) state_get<SL>(a.seg_h + seg * S + q * SL, h);
        else if (a.state_in) state_get<SL>(a.state_in + st, h);
    }
    float *Bs = bc[w][0], *Cs = bc[w][1];
    typename O::st* y = (typename O::st*)a.y;
    ScanBlock<E, S> x;
    if (s0 < e1) x.load(a, row0, s0, q, lane, dc, g, !LOCAL);
    for (int t0 = s0; t0 < e1; t0 += T) {
        float du[TL], dt[TL], u[TL], z[TL];
        x.steps(a, bias, n, t0, q, dt, u, du);
        put_bc<E, P>(Bs, x.b, n, t0, lane);
        if (!LOCAL) put_bc<E, P>(Cs, x.c, n, t0, lane);
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            if (LOCAL) total += dt[i];
            else z[i] = a.z ? swish_hw(Raw<E>::value(x.z[i])) : 1.f;
        }
        if (t0 + T < e1) x.load(a, row0, t0 + T, q, lane, dc, g, !LOCAL);
        lds_order();
        float o[TL];
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            float yp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float B[SL], C[SL];
                lds_vec<SL>(Bs + (4 * i + k) * S + q * SL, B);
                if (!LOCAL) lds_vec<SL>(Cs + (4 * i + k) * S + q * SL, C);
                const float dk = quad_of(dt[i], k), uk = quad_of(du[i], k);
                yp[k] = 0.f;
#pragma unroll
                for (int j = 0; j < SL; ++j) {
                    h[j] = fmaf(__builtin_amdgcn_exp2f(dk * A2[j]), h[j], uk * B[j]);
                    if (!LOCAL) yp[k] = fmaf(C[j], h[j], yp[k]);
                }
            }
            if (!LOCAL) o[i] = fmaf(skip, u[i], quad_sums(yp[0], yp[1], yp[2], yp[3], q)) * z[i];
        }
        lds_order();
        if (LOCAL) continue;
        if (d < a.D) store_scalars<O, P>(a.y, row0 + t0, a.D, e1 - t0, q, d, o);
    }
    if (LOCAL) {
        total = lanes_sum<4>(total);
        if (d >= a.D) return;
#pragma unroll
        for (int j = 0; j < SL; ++j) a.seg_h[seg * S + q * SL + j] = h[j];
        if (q == 0) a.seg_dt[seg] = total;
        return;
    }
    // tokens past the sequence's length: zeros
    for (int t = (e1 > s0 ? e1 : s0) + (lane >> 4); t < s1; t += 4) {
        const int dz = at.cb * kScanCh + (lane & 15);
        if (dz < a.D) store_out(y + (row0 + t) * a.D + dz, 0.f);
    }
    if (a.state_out && at.seg == a.nseg - 1 && d < a.D)
#pragma unroll
        for (int j = 0; j < SL; ++j) a.state_out[st + j] = h[j];
}

// Segments' states from zero -> the states entering them, in place.
template <int S>
__global__ __launch_bounds__(256) void scan_join_kernel(ScanArgs a) {
    const long long per = (long long)a.D * S, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const int b = blockIdx.y, d = (int)(i / S);
    const float A2 = decay_rate(a.A[i]);
    float h = a.state_in ? a.state_in[b * per + i] : 0.f;
    float* hp = a.seg_h + (long long)b * a.nseg * per + i;
    const float* sp = a.seg_dt + (long long)b * a.nseg * a.D + d;
    constexpr int U = 8;
    for (int k = 0; k < a.nseg; k += U) {
        float x[U], p[U];
#pragma unroll
        for (int e = 0; e < U; ++e) {
            const int s = k + e < a.nseg - 1 ? k + e : 0;
            x[e] = hp[s * per];
            p[e] = sp[(long long)s * a.D];
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
            if (k + e >= a.nseg) break;
            hp[(k + e) * per] = h;
            h = fmaf(__builtin_amdgcn_exp2f(p[e] * A2), h, x[e]);
        }
    }
}

// A workgroup on 16 channels of a segment, NW blocks of T tokens at a time.
template <class E, class O, int S>
__global__ __launch_bounds__(ScanShape<S>::THREADS) void scan_chunks_kernel(ScanArgs a) {
    typedef ScanShape<S> P;
    constexpr int SL = P::SL, T = P::T, TL = P::TL;
    __shared__ float bc[P::NW][2][T * S];
    __shared__ float ex[2][P::NW][2][64 * SL];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane & 3;
    ScanPos at;
    if (!scan_pos(a, &at)) return;
    const int d = at.cb * kScanCh + (lane >> 2), dc = d < a.D ? d : a.D - 1;
    const int g = __builtin_amdgcn_readfirstlane(dc / (a.D / a.G));
    const int n = length_of(a.lengths, at.b, a.N);
    const int s0 = at.seg * a.seg_tokens, s1 = a.N - s0 < a.seg_tokens ? a.N : s0 + a.seg_tokens;
    const long long row0 = (long long)at.b * a.N;
    const float bias = a.bias ? a.bias[dc] : 0.f, skip = a.skip ? a.skip[dc] : 0.f;
    float A2[SL], run[SL];
    const long long st = ((long long)at.b * a.D + dc) * S + q * SL;
#pragma unroll
    for (int j = 0; j < SL; ++j) {
        A2[j] = decay_rate(a.A[(long long)dc * S + q * SL + j]);
        run[j] = 0.f;
    }
    if (a.nseg > 1) state_get<SL>(a.seg_h + (((long long)at.b * a.nseg + at.seg) * a.D + dc) * S + q * SL, run);
    else if (a.state_in) state_get<SL>(a.state_in + st, run);
    float *Bs = bc[w][0], *Cs = bc[w][1];
    typename O::st* y = (typename O::st*)a.y;
    const int live1 = s1 < n ? s1 : n;
    ScanBlock<E, S> x;
    if (s0 < live1) x.load(a, row0, s0 + w * T, q, lane, dc, g, true);
    int parity = 0;
    for (int c0 = s0; c0 < live1; c0 += P::CH, parity ^= 1) {
        const int t0 = c0 + w * T;
        float du[TL], dt[TL], u[TL], z[TL], total = 0.f;
        x.steps(a, bias, n, t0, q, dt, u, du);
        put_bc<E, P>(Bs, x.b, n, t0, lane);
        put_bc<E, P>(Cs, x.c, n, t0, lane);
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            z[i] = a.z ? swish_hw(Raw<E>::value(x.z[i])) : 1.f;
            total += dt[i];
        }
        if (c0 + P::CH < live1) x.load(a, row0, t0 + P::CH, q, lane, dc, g, true);
        lds_order();
        float al[T][SL], h[SL];
#pragma unroll
        for (int j = 0; j < SL; ++j) h[j] = 0.f;
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
        total = lanes_sum<4>(total);
        float p[SL];
#pragma unroll
        for (int j = 0; j < SL; ++j) p[j] = __builtin_amdgcn_exp2f(total * A2[j]);
        ex_put<SL>(ex[parity][w][0], lane, h);
        ex_put<SL>(ex[parity][w][1], lane, p);
        __syncthreads();
#pragma unroll
        for (int v = 0; v < P::NW; ++v) {
            if (v == w)
#pragma unroll
                for (int j = 0; j < SL; ++j) h[j] = run[j];
            float hv[SL], pv[SL];
            ex_get<SL>(ex[parity][v][0], lane, hv);
            ex_get<SL>(ex[parity][v][1], lane, pv);
#pragma unroll
            for (int j = 0; j < SL; ++j) run[j] = fmaf(pv[j], run[j], hv[j]);
        }
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            float yp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float B[SL], C[SL];
                lds_vec<SL>(Bs + (4 * i + k) * S + q * SL, B);
                lds_vec<SL>(Cs + (4 * i + k) * S + q * SL, C);
                const float uk = quad_of(du[i], k);
                yp[k] = 0.f;
#pragma unroll
                for (int j = 0; j < SL; ++j) {
                    h[j] = fmaf(al[4 * i + k][j], h[j], uk * B[j]);
                    yp[k] = fmaf(C[j], h[j], yp[k]);
                }
            }
            z[i] *= fmaf(skip, u[i], quad_sums(yp[0], yp[1], yp[2], yp[3], q));
        }
        if (d < a.D) store_scalars<O, P>(a.y, row0 + t0, a.D, live1 - t0, q, d, z);
        lds_order();
    }
    // tokens past the sequence's length: zeros
    for (int t = (live1 > s0 ? live1 : s0) + (int)(threadIdx.x / kScanCh); t < s1; t += P::THREADS / kScanCh) {
        const int dz = at.cb * kScanCh + (int)(threadIdx.x % kScanCh);
        if (dz < a.D) store_out(y + (row0 + t) * a.D + dz, 0.f);
    }
    if (w == 0 && a.state_out && at.seg == a.nseg - 1 && d < a.D)
#pragma unroll
        for (int j = 0; j < SL; ++j) a.state_out[st + j] = run[j];
}

template <class E, class O, int S>
bool pick(ScanKernels* o) {
    typedef ScanShape<S> P;
    *o = {scan_walk_kernel<E, O, S, true>, scan_join_kernel<S>, scan_walk_kernel<E, O, S, false>, scan_chunks_kernel<E, O, S>,
          P::T, P::CH, P::THREADS};
    return true;
}
template <class E, class O>
bool of_states(int S, ScanKernels* o) {
    switch (S) {
        case 8: return pick<E, O, 8>(o);
        case 16: return pick<E, O, 16>(o);
        case 32: return pick<E, O, 32>(o);
        case 64: return pick<E, O, 64>(o);
        default: return false;
    }
}

}  // namespace

bool scan_kernels_get(bool bf16_in, bool bf16_out, int S, ScanKernels* o) {
    if (!bf16_in) return of_states<F32, F32>(S, o);
    return bf16_out ? of_states<BF16, BF16>(S, o) : of_states<BF16, F32>(S, o);
}

}  // namespace ret
