// The gated delta rule over a sequence: the per-chunk matrices, the chain over chunks, and the chain over segments.
#include "delta.h"

namespace ret {

namespace {

typedef double f64;

// ---------------------------------------------------------------------------------------------------
// delta_prep: T = (I + A)^-1 and P of one chunk, for the H / Hk value heads that share a key head (the products K K^T
// and Q K^T are made once for them). One workgroup per (chunk, b, key head); wave w owns rows 16w .. 16w+15.
//
// The decays are exp2 of differences of the running sum of g, kept in fp64 and scaled to base 2: a difference of two
// fp32 sums would lose the small decays that stand behind a large one. g below -200 counts as -200 (exp is 0 in fp32),
// so that g = -inf, which clears the state, leaves no inf - inf.
//
// The unit triangular inverse goes by 16 x 16 blocks: the four diagonal ones by forward substitution, a column per lane,
// then twice the block rule [[X, 0], [A, Y]]^-1 = [[X', 0], [-Y' A X', Y']] with fp32 MFMA.
// ---------------------------------------------------------------------------------------------------
constexpr int kTriLD = 68;  // row pitch of the fp32 matrices in LDS

// acc += X[r0.., c0..16] Y[16 rows at y0, columns n0..] of fp32 LDS matrices; fragments in accumulator order
__device__ __forceinline__ f32x4_t tri_a(const float* X, int r0, int c0, int lane) {
    return *reinterpret_cast<const f32x4_t*>(X + (r0 + (lane & 15)) * kTriLD + c0 + 4 * (lane >> 4));
}
__device__ __forceinline__ f32x4_t tri_b(const float* X, int r0, int c0, int lane) {
    const float* p = X + (r0 + 4 * (lane >> 4)) * kTriLD + c0 + (lane & 15);
    return f32x4_t{p[0], p[kTriLD], p[2 * kTriLD], p[3 * kTriLD]};
}
__device__ __forceinline__ void tri_store(float* X, int r0, int c0, int lane, f32x4_t v) {
    float* p = X + (r0 + 4 * (lane >> 4)) * kTriLD + c0 + (lane & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i * kTriLD] = v[i];
}

// Writes a 64 x 64 fp32 LDS matrix (or its transpose) as operand fragments, two row tiles' worth of work per wave pair.
template <class E, bool TR>
__device__ __forceinline__ void write_mat(char* m, const float* X, int w, int lane) {
    typedef DOps<E> D;
    constexpr int NS = kDeltaC / D::KS;
    const int r = 16 * w + (lane & 15), g4 = 4 * (lane >> 4);
    auto take = [&](int c) {
        if constexpr (!TR) return *reinterpret_cast<const f32x4_t*>(X + r * kTriLD + c);
        else return f32x4_t{X[c * kTriLD + r], X[(c + 1) * kTriLD + r], X[(c + 2) * kTriLD + r], X[(c + 3) * kTriLD + r]};
    };
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        if constexpr (D::TPS == 2) D::mat_store(m, w * NS + s, lane, take(32 * s + g4), take(32 * s + 16 + g4));
        else D::mat_store(m, w * NS + s, lane, take(16 * s + g4));
    }
}

// sT <- (I + sA)^-1 for a strictly lower triangular sA, by the workgroup's four waves. Ends with a barrier.
__device__ __forceinline__ void tri_inverse(const float* sA, float* sT, int w, int lane) {
    const int n16 = lane & 15, g = lane >> 4;
    // diagonal block w: column n16 of its inverse (the four lane groups hold the same)
    {
        float x[16];
        const float* Ad = sA + (16 * w) * kTriLD + 16 * w;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == n16 ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; ++m) s -= Ad[i * kTriLD + m] * x[m];
            x[i] = s;
        }
        if (g == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sT[(16 * w + i) * kTriLD + 16 * w + n16] = x[i];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)  // the blocks above the diagonal
            if (j > w) tri_store(sT, 16 * w, 16 * j, lane, f32x4_t{0.f, 0.f, 0.f, 0.f});
    }
    __syncthreads();
    // 32 x 32 blocks: rows 16 .. 31 (wave 0) and 48 .. 63 (wave 1)
    if (w < 2) {
        const int r0 = 32 * w + 16, c0 = 32 * w;
        f32x4_t m = {0.f, 0.f, 0.f, 0.f}, t = {0.f, 0.f, 0.f, 0.f};
        DOps<F32>::mma_ab(m, tri_a(sA, r0, c0, lane), tri_b(sT, c0, c0, lane));
        DOps<F32>::mma_ab(t, tri_a(sT, r0, r0, lane), m);
        tri_store(sT, r0, c0, lane, -t);
    }
    __syncthreads();
    // the 64 x 64 one: wave w makes the tile at rows 32 + 16 (w / 2), columns 16 (w % 2)
    {
        const int rt = w / 2, ct = w % 2;
        f32x4_t m[2], t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; ++j)
                DOps<F32>::mma_ab(m[i], tri_a(sA, 32 + 16 * i, 16 * j, lane), tri_b(sT, 16 * j, 16 * ct, lane));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) DOps<F32>::mma_ab(t, tri_a(sT, 32 + 16 * rt, 32 + 16 * i, lane), m[i]);
        tri_store(sT, 32 + 16 * rt, 16 * ct, lane, -t);
    }
    __syncthreads();
}

template <class E, int DK, bool BWD>
__global__ __launch_bounds__(kThreads) void delta_prep_kernel(DeltaArgs a) {
    typedef typename E::st st;
    typedef DRows<E, DK> Rows;
    typedef typename Rows::Tile Tile;
    typedef DOps<E> D;
    __shared__ __align__(16) st sk[kDeltaC * Tile::LD];
    __shared__ __align__(16) st sq[kDeltaC * Tile::LD];
    __shared__ __align__(16) float sA[kDeltaC * kTriLD];
    __shared__ __align__(16) float sT[kDeltaC * kTriLD];
    __shared__ f64 sG[kDeltaC];
    __shared__ float sB[kDeltaC];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n16 = lane & 15, g = lane >> 4;
    const int c = blockIdx.x, b = blockIdx.y / a.Hk, hk = blockIdx.y % a.Hk, rep = a.H / a.Hk;
    const int t0 = c * kDeltaC, live = min(kDeltaC, delta_len(a, b) - t0);
    if (live <= 0) return;  // no one reads this chunk
    {
        Rows rk, rq;
        const long long base = (((long long)b * a.N + t0) * a.Hk + hk) * DK;
        rk.load((const st*)a.k + base, a.Hk * DK, live, tid);
        rq.load((const st*)a.q + base, a.Hk * DK, live, tid);
        rk.store(sk, tid);
        rq.store(sq, tid);
    }
    __syncthreads();
    // K K^T and Q K^T, row tile w, column tiles 0 .. w (the ones past it stay zero)
    f32x4_t kk[4], qk[4], av[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto dot = [&](f32x4_t& acc, const typename D::Fa& x, const typename D::Fa& y) {
        if constexpr (D::TPS == 2) D::mfma1(acc, x, y);
        else D::mma_ab(acc, x, y);
    };
#pragma unroll
    for (int s = 0; s < DK / D::KS; ++s) {
        const typename D::Fa fk = Tile::rows(sk, 16 * w, s * D::KS, lane), fq = Tile::rows(sq, 16 * w, s * D::KS, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > w) continue;
            const typename D::Fa fb = Tile::rows(sk, 16 * j, s * D::KS, lane);
            dot(kk[j], fk, fb);
            dot(qk[j], fq, fb);
        }
    }
    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        const long long unit = ((long long)b * a.H + h) * a.nchunks + c;
        if (w == 0) {
            const bool in = lane < live;
            const long long i = ((long long)b * a.N + t0 + (in ? lane : 0)) * a.H + h;
            const float gv = gate_at(a.g, i, a.gate_bf16);
            f64 G = in ? (f64)(gv < -200.f ? -200.f : gv) * 1.4426950408889634 : 0.0;
#pragma unroll
            for (int m = 1; m < 64; m *= 2) {
                const f64 up = __shfl_up(G, m);
                if (lane >= m) G += up;
            }
            const float be = in ? gate_at(a.beta, i, a.gate_bf16) : 0.f;
            sG[lane] = G;
            sB[lane] = be;
            float* f = a.fac + unit * kDeltaFac;
            const float tail = __builtin_amdgcn_exp2f((float)(__shfl(G, 63) - G));
            f[lane] = __builtin_amdgcn_exp2f((float)G);
            f[64 + lane] = tail * be;
            f[128 + lane] = tail;
            f[192 + lane] = be;
            reinterpret_cast<f64*>(f + 256)[lane] = G;
        }
        __syncthreads();
        char* mats = a.mats + unit * a.nmats * kDeltaMatBytes;
        // A into sA; P into sT until it is written out (the gradients take P without beta)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4_t pv;
            const int col = 16 * j + n16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * w + 4 * g + i;
                const float d = col <= row ? __builtin_amdgcn_exp2f((float)(sG[row] - sG[col])) : 0.f;
                av[j][i] = col < row ? d * kk[j][i] : 0.f;
                pv[i] = col <= row ? a.scale * (BWD ? 1.f : sB[col]) * d * qk[j][i] : 0.f;
            }
            tri_store(sA, 16 * w, 16 * j, lane, av[j] * sB[col]);
            tri_store(sT, 16 * w, 16 * j, lane, pv);
        }
        __syncthreads();
        if constexpr (BWD) write_mat<E, true>(mats + 2 * kDeltaMatBytes, sT, w, lane);
        else write_mat<E, false>(mats + kDeltaMatBytes, sT, w, lane);
        __syncthreads();
        tri_inverse(sA, sT, w, lane);
        write_mat<E, false>(mats, sT, w, lane);
        if constexpr (BWD) {
            // Tr = (I + Ar)^-1 with beta along the rows: the gradients' solve
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4_t x = av[j];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] *= sB[16 * w + 4 * g + i];
                tri_store(sA, 16 * w, 16 * j, lane, x);
            }
            __syncthreads();
            tri_inverse(sA, sT, w, lane);
            write_mat<E, true>(mats + kDeltaMatBytes, sT, w, lane);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------------
// delta_chain: one segment of one head, 64 NC columns per workgroup (16 NC per wave), the state in accumulators.
// LOCAL: the segment's end state from zero (columns of V; segment 0 starts from state_in) or its transition (columns of
// the identity, V = 0), into segE / segM. Otherwise the outputs, and after the last segment the final state.
// ---------------------------------------------------------------------------------------------------
enum { kFull = 0, kLocal = 1, kStates = 2 };
template <class E, int DK, int NC, int MODE>
__global__ __launch_bounds__(kThreads) void delta_chain_kernel(DeltaArgs a) {
    typedef typename E::st st;
    typedef DOps<E> D;
    typedef DRows<E, DK> Rows;
    typedef typename Rows::Tile Tile;
    constexpr bool LOCAL = MODE == kLocal, FULL = MODE == kFull;
    constexpr int DT = DK / 16, NS = kDeltaC / D::KS;
    __shared__ __align__(16) st sk[kDeltaC * Tile::LD];
    __shared__ __align__(16) st sq[FULL ? kDeltaC * Tile::LD : 16];
    __shared__ __align__(16) float sf[128];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n16 = lane & 15, g4 = 4 * (lane >> 4);
    const int bh = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg, b = bh / a.H, h = bh % a.H;
    const int nE = (a.dv + 64 * NC - 1) / (64 * NC);  // workgroups over d_v; a local pass has those of d_k behind them
    const bool trans = LOCAL && (int)blockIdx.y >= nE;
    const int width = trans ? DK : a.dv;
    const int col0 = ((int)blockIdx.y - (trans ? nE : 0)) * 64 * NC + w * 16 * NC;
    const int hk = h / (a.H / a.Hk), len = delta_len(a, b);
    const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nchunks);
    const bool active = col0 < width;
    // segment 0's end state is known, and no one asks for the last one's
    if (LOCAL && (trans ? seg == 0 : seg == a.nseg - 1)) return;

    f32x4_t S[NC][DT];
    const float* sin = nullptr;
    if (!LOCAL) sin = a.nseg > 1 ? a.segE + ((long long)bh * a.nseg + seg) * DK * a.dv : nullptr;
    if (!LOCAL && a.nseg == 1) sin = a.state_in ? a.state_in + (long long)bh * DK * a.dv : nullptr;
    if (LOCAL && seg == 0 && !trans && a.state_in) sin = a.state_in + (long long)bh * DK * a.dv;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int col = col0 + 16 * n + n16;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * t + g4 + i;
                float x = trans && row == col ? 1.f : 0.f;
                if (sin && col0 + 16 * n < width) x = sin[(long long)row * a.dv + col];
                S[n][t][i] = x;
            }
    }

    Rows rk, rq;
    float ff = 0.f;
    const st* kp = (const st*)a.k + (((long long)b * a.N) * a.Hk + hk) * DK;
    const st* qp = (const st*)a.q + (((long long)b * a.N) * a.Hk + hk) * DK;
    auto fetch = [&](int c) {
        const int live = min(kDeltaC, len - c * kDeltaC);
        const long long base = (long long)c * kDeltaC * a.Hk * DK;
        rk.load(kp + base, a.Hk * DK, live, tid);
        if constexpr (FULL) rq.load(qp + base, a.Hk * DK, live, tid);
        if (tid < 128) ff = a.fac[((long long)bh * a.nchunks + c) * kDeltaFac + tid];
    };
    const int cend = min(c1, (len + kDeltaC - 1) / kDeltaC);  // chunks with live tokens
    if (c0 < cend) fetch(c0);
    for (int c = c0; c < cend; ++c) {
        __syncthreads();
        rk.store(sk, tid);
        if constexpr (FULL) rq.store(sq, tid);
        if (tid < 128) sf[tid] = ff;
        __syncthreads();
        if (c + 1 < cend) fetch(c + 1);
        if (!active) continue;
        const int live = min(kDeltaC, len - c * kDeltaC);
        const char* mats = a.mats + ((long long)bh * a.nchunks + c) * a.nmats * kDeltaMatBytes;
        // V in accumulator order: lane's column, tokens 16 m + 4 g + i
        float v[NC][4][4];
        if (!trans) {
            const int stride = a.H * a.dv;
            const st* vp = (const st*)a.v + (((long long)b * a.N + c * kDeltaC) * a.H + h) * a.dv;
            const rsrc_t r = bytes_rsrc(vp, ((live - 1) * stride + a.dv) * (int)sizeof(st));
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int off = col0 + 16 * n < width ? (g4 * stride + col0 + 16 * n + n16) * (int)sizeof(st)
                                                              : 0x40000000;
                        const int so = (16 * m + i) * stride * (int)sizeof(st);
                        if constexpr (sizeof(st) == 2)
                            v[n][m][i] = bf16_to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, so, 0));
                        else v[n][m][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, so, 0));
                    }
        }
        // Y = K S, and (Q S)^T beside it
        f32x4_t y[NC][4], o[NC][4];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m) y[n][m] = o[n][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < DK / D::KS; ++s) {
            typename D::Fb fs[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) fs[n] = D::step(S[n], s);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const typename D::Fa fk = Tile::rows(sk, 16 * m, s * D::KS, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) D::mma_ab(y[n][m], fk, fs[n]);
                if constexpr (FULL) {
                    const typename D::Fa fq = Tile::rows(sq, 16 * m, s * D::KS, lane);
#pragma unroll
                    for (int n = 0; n < NC; ++n) D::mma_ba(o[n][m], fq, fs[n]);
                }
            }
        }
        if constexpr (MODE == kStates) {
            st* sp = (st*)a.s0t + ((long long)bh * a.nchunks + c) * a.dv * DK;
#pragma unroll
            for (int n = 0; n < NC; ++n)
                if (col0 + 16 * n < width)
#pragma unroll
                    for (int t = 0; t < DT; ++t) store4(sp + (long long)(col0 + 16 * n + n16) * DK + 16 * t + g4, S[n][t]);
        }
        // R = V - exp(G) Y
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4_t ga = *reinterpret_cast<const f32x4_t*>(sf + 16 * m + g4);
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[n][m][i] = (trans ? 0.f : v[n][m][i]) - ga[i] * y[n][m][i];
        }
        // E = T R
        f32x4_t u[NC][4];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m) u[n][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            typename D::Fb fr[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) fr[n] = D::step(y[n], s);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (s * D::KS > 16 * m + 15) continue;  // above the diagonal
                const typename D::Fm ft = D::mat_frag(mats, m * NS + s, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) D::mma_mb(u[n][m], ft, fr[n]);
            }
        }
        if constexpr (MODE == kStates) {
            st* ep = (st*)a.et + ((long long)bh * a.nchunks + c) * a.dv * kDeltaC;
#pragma unroll
            for (int n = 0; n < NC; ++n)
                if (col0 + 16 * n < width)
#pragma unroll
                    for (int m = 0; m < 4; ++m) store4(ep + (col0 + 16 * n + n16) * kDeltaC + 16 * m + g4, u[n][m]);
        }
        if constexpr (FULL) {
            // O^T = scale exp(G) (Q S)^T + E^T P^T: a lane holds 4 columns of token 16 m + n16
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float f = a.scale * sf[16 * m + n16];
#pragma unroll
                for (int n = 0; n < NC; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][m][i] *= f;
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                typename D::Fb fu[NC];
#pragma unroll
                for (int n = 0; n < NC; ++n) fu[n] = D::step(u[n], s);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (s * D::KS > 16 * m + 15) continue;
                    const typename D::Fm fp = D::mat_frag(mats + kDeltaMatBytes, m * NS + s, lane);
#pragma unroll
                    for (int n = 0; n < NC; ++n) D::mma_bm(o[n][m], fp, fu[n]);
                }
            }
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                if (col0 + 16 * n >= width) continue;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int t = c * kDeltaC + 16 * m + n16;
                    if (t >= a.N) continue;
                    const f32x4_t x = t < len ? o[n][m] : f32x4_t{0.f, 0.f, 0.f, 0.f};
                    const long long e = (((long long)b * a.N + t) * a.H + h) * a.dv + col0 + 16 * n + g4;
                    if (a.out_bf16) store4((uint16_t*)a.o + e, x);
                    else store4((float*)a.o + e, x);
                }
            }
        }
        // S = exp(G_C) S + K^T (exp(G_C - G) beta E)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4_t ta = *reinterpret_cast<const f32x4_t*>(sf + 64 + 16 * m + g4);
#pragma unroll
            for (int n = 0; n < NC; ++n) u[n][m] *= ta;
        }
        const float end = sf[63];  // exp(G_C)
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int t = 0; t < DT; ++t) S[n][t] *= end;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            typename D::Fb fu[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) fu[n] = D::step(u[n], s);
#pragma unroll
            for (int t = 0; t < DT; ++t) {
                const typename D::Fa fk = Tile::cols(sk, s * D::KS, 16 * t, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) D::mma_ab(S[n][t], fk, fu[n]);
            }
        }
    }
    if (!active) return;
    // outputs of padding chunks are zero
    if constexpr (FULL) {
        for (int c = max(c0, cend); c < c1; ++c)
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                if (col0 + 16 * n >= width) continue;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int t = c * kDeltaC + 16 * m + n16;
                    if (t >= a.N) continue;
                    const long long e = (((long long)b * a.N + t) * a.H + h) * a.dv + col0 + 16 * n + g4;
                    if (a.out_bf16) store4((uint16_t*)a.o + e, f32x4_t{0.f, 0.f, 0.f, 0.f});
                    else store4((float*)a.o + e, f32x4_t{0.f, 0.f, 0.f, 0.f});
                }
            }
    }
    if constexpr (MODE == kStates) return;
    float* out = nullptr;
    if (LOCAL) out = (trans ? a.segM : a.segE) + ((long long)bh * a.nseg + seg) * DK * width;
    else if (seg == a.nseg - 1 && a.state_out) out = a.state_out + (long long)bh * DK * a.dv;
    if (!out) return;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        if (col0 + 16 * n >= width) continue;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[(long long)(16 * t + g4 + i) * width + col0 + 16 * n + n16] = S[n][t][i];
    }
}

// ---------------------------------------------------------------------------------------------------
// delta_scan: the states entering the segments. In: segE[s] = segment s's end state from zero (segment 0: its true end
// state), segM[s] its transition. Out: segE[s] = the state entering segment s, S_{s+1} = M_s S_s + E_s. One workgroup per
// (b, h, 16 columns); REV: the gradients' chain, D_{s-1} = M_s^T D_s + F_s over segF from the right. The waves share the rows of M, S goes round through LDS. BF16
// input: M and S split in two bf16 parts like the chain's operands.
// ---------------------------------------------------------------------------------------------------
template <class E, int DK, bool REV>
__global__ __launch_bounds__(kThreads) void delta_scan_kernel(DeltaArgs a) {
    typedef DOps<E> D;
    constexpr int NT = DK / 16, TW = NT >= 4 ? NT / 4 : 1, LD = 20;
    __shared__ __align__(16) float sS[DK * LD];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n16 = lane & 15, g4 = 4 * (lane >> 4);
    const int bh = blockIdx.x, col = blockIdx.y * 16 + n16;
    const bool mine = w * TW < NT;
    const long long sz = (long long)DK * a.dv;
    float* X = (REV ? a.segF : a.segE) + (long long)bh * a.nseg * sz;
    const float* M = a.segM + (long long)bh * a.nseg * DK * DK;
    const float* from = REV ? a.dstate_out : a.state_in;
    const float* sin = from ? from + bh * sz : nullptr;
    const int len = delta_len(a, bh / a.H);
    f32x4_t S[TW];
    auto tile = [&](int k) {  // 16 rows of the entering state as accumulators hold them
        f32x4_t x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = sS[(16 * k + g4 + i) * LD + n16];
        return x;
    };
    for (int j = 0; j < a.nseg; ++j) {
        const int s = REV ? a.nseg - 1 - j : j;
        if (mine) {
            f32x4_t e[TW];
#pragma unroll
            for (int t = 0; t < TW; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long at = (long long)(16 * (w * TW + t) + g4 + i) * a.dv + col;
                    if (j < a.nseg - 1) e[t][i] = X[s * sz + at];
                    X[s * sz + at] = j == 0 ? (sin ? sin[at] : 0.f) : S[t][i];
                }
            if (j == a.nseg - 1) break;
            if (j > 0 && s * a.seg_chunks * kDeltaC >= len) {  // no live token: the state passes as it is
#pragma unroll
                for (int t = 0; t < TW; ++t) e[t] = S[t];
            } else if (j > 0) {
                const float* Ms = M + (long long)s * DK * DK;
#pragma unroll
                for (int k = 0; k < DK / D::KS; ++k) {
                    f32x4_t x[D::TPS];
#pragma unroll
                    for (int p = 0; p < D::TPS; ++p) x[p] = tile(D::TPS * k + p);
                    const typename D::Fb fs = D::step(x, 0);
#pragma unroll
                    for (int t = 0; t < TW; ++t) {
                        f32x4_t y[D::TPS];
                        if constexpr (REV) {  // rows of the transpose
                            const float* m = Ms + (D::KS * k + g4) * DK + 16 * (w * TW + t) + n16;
#pragma unroll
                            for (int p = 0; p < D::TPS; ++p)
#pragma unroll
                                for (int i = 0; i < 4; ++i) y[p][i] = m[(16 * p + i) * DK];
                        } else {
                            const float* m = Ms + (16 * (w * TW + t) + n16) * DK + D::KS * k + g4;
#pragma unroll
                            for (int p = 0; p < D::TPS; ++p) y[p] = *reinterpret_cast<const f32x4_t*>(m + 16 * p);
                        }
                        D::mma_mb(e[t], D::step(y, 0), fs);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < TW; ++t) S[t] = e[t];
        } else if (j == a.nseg - 1) {
            break;
        }
        __syncthreads();
        if (mine)
#pragma unroll
            for (int t = 0; t < TW; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) sS[(16 * (w * TW + t) + g4 + i) * LD + n16] = S[t][i];
        __syncthreads();
    }
}

template <class E, int DK, int NC>
void pick_cols(DeltaKernels* o) {
    *o = {};
    o->prep = delta_prep_kernel<E, DK, false>;
    o->bprep = delta_prep_kernel<E, DK, true>;
    o->local = delta_chain_kernel<E, DK, NC, kLocal>;
    o->full = delta_chain_kernel<E, DK, NC, kFull>;
    o->states = delta_chain_kernel<E, DK, NC, kStates>;
    o->scan = delta_scan_kernel<E, DK, false>;
    o->rscan = delta_scan_kernel<E, DK, true>;
    o->cols = 64 * NC;
}
// Two column tiles per wave halve the operand reads per product; one where d_v would leave waves idle.
template <class E, int DK>
void pick(int dv, DeltaKernels* o) {
    if (dv > 64) pick_cols<E, DK, 2>(o);
    else pick_cols<E, DK, 1>(o);
}

}  // namespace

bool delta_kernels_get(bool bf16_in, int dk, int dv, DeltaKernels* o) {
    if (dv <= 0 || dv % 16) return false;
    if (bf16_in) {
        switch (dk) {
            case 32: pick<BF16, 32>(dv, o); break;
            case 64: pick<BF16, 64>(dv, o); break;
            case 128: pick<BF16, 128>(dv, o); break;
            case 256: pick<BF16, 256>(dv, o); break;
            default: return false;
        }
        delta_bwd_kernels_get(true, dk, dv, o);
        return true;
    }
    switch (dk) {
        case 16: pick<F32, 16>(dv, o); break;
        case 32: pick<F32, 32>(dv, o); break;
        case 64: pick<F32, 64>(dv, o); break;
        case 128: pick<F32, 128>(dv, o); break;
        default: return false;
    }
    delta_bwd_kernels_get(false, dk, dv, o);
    return true;
}

}  // namespace ret
