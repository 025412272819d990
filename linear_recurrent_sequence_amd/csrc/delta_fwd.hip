// The gated delta rule over a sequence: the per-chunk matrices, the chain over chunks, and the chain over segments.
#include "delta.h"

#include <type_traits>

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

// Writes a lower triangular 64 x 64 fp32 LDS matrix (or its transpose) as operand fragments, a row tile per wave, this
// lane's row (16 w + lane % 16) times `scale`.
template <class E, bool TR>
__device__ __forceinline__ void write_mat(char* m, const float* X, int w, int lane, bool lo, float scale = 1.f) {
    typedef DOps<E> D;
    typedef TriFrags<D::KS> F;
    const int r = 16 * w + (lane & 15), g4 = 4 * (lane >> 4);
    auto take = [&](int c) {
        if constexpr (!TR) return *reinterpret_cast<const f32x4_t*>(X + r * kTriLD + c);
        else return f32x4_t{X[c * kTriLD + r], X[(c + 1) * kTriLD + r], X[(c + 2) * kTriLD + r], X[(c + 3) * kTriLD + r]};
    };
#pragma unroll
    for (int s = 0; s < F::NS; ++s) {
        if (TR ? !F::upper(w, s) : !F::lower(w, s)) continue;
        const int f = F::at(w, s, TR);
        if constexpr (D::TPS == 2) D::mat_store(m, f, lane, scale * take(32 * s + g4), scale * take(32 * s + 16 + g4), lo);
        else D::mat_store(m, f, lane, scale * take(16 * s + g4));
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
    typedef DRows<E, DK, kThreads> Rows;
    typedef typename Rows::Tile Tile;
    typedef DOps<E> D;
    __shared__ __align__(16) st sk[kDeltaC * Tile::LD];
    __shared__ __align__(16) st sq[kDeltaC * Tile::LD];
    __shared__ __align__(16) float sA[kDeltaC * kTriLD];
    __shared__ __align__(16) float sT[kDeltaC * kTriLD];
    __shared__ f64 sG[kDeltaC];
    __shared__ float sB[kDeltaC], sF[kDeltaC];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15, g = lane >> 4;
    const int c = blockIdx.x, b = blockIdx.y / a.Hk, hk = blockIdx.y % a.Hk, rep = a.H / a.Hk;
    const int t0 = c * kDeltaC, live = min(kDeltaC, delta_len(a, b) - t0);
    if (live <= 0) return;  // no one reads this chunk
    {
        Rows rk, rq;
        const long long base = (((long long)b * a.N + t0) * a.Hk + hk) * DK;
        rk.load((const st*)a.k + base, a.Hk * DK, live, DK, tid);
        rq.load((const st*)a.q + base, a.Hk * DK, live, DK, tid);
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
            f[64 + lane] = sF[lane] = tail * be;
            f[128 + lane] = tail;
            f[192 + lane] = be;
            reinterpret_cast<f64*>(f + 256)[lane] = G;
        }
        __syncthreads();
        char* mats = a.mats + unit * a.nmats * kDeltaMatBytes;
        f32x4_t pv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = 16 * j + n16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * w + 4 * g + i;
                const float d = col <= row ? __builtin_amdgcn_exp2f((float)(sG[row] - sG[col])) : 0.f;
                av[j][i] = col < row ? d * kk[j][i] : 0.f;
                pv[j][i] = col <= row ? a.scale * d * qk[j][i] : 0.f;
            }
            tri_store(sA, 16 * w, 16 * j, lane, av[j] * sB[col]);
            if constexpr (BWD) tri_store(sT, 16 * w, 16 * j, lane, pv[j]);  // until it is written out
        }
        __syncthreads();
        if constexpr (BWD) {
            write_mat<E, true>(mats + 2 * kDeltaMatBytes, sT, w, lane, true);
            __syncthreads();
        }
        tri_inverse(sA, sT, w, lane);
        if constexpr (BWD) {
            write_mat<E, false>(mats, sT, w, lane, true);
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
            write_mat<E, true>(mats + kDeltaMatBytes, sT, w, lane, true);
        } else {
            // P T: row tile w through sA (its own rows only), and T with its rows scaled
#pragma unroll
            for (int j = 0; j < 4; ++j) tri_store(sA, 16 * w, 16 * j, lane, pv[j] * sB[16 * j + n16]);
            __syncthreads();
            f32x4_t pt[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pt[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = j; i < 4; ++i)
                    if (i <= w) DOps<F32>::mma_ab(pt[j], tri_a(sA, 16 * w, 16 * i, lane), tri_b(sT, 16 * i, 16 * j, lane));
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) tri_store(sA, 16 * w, 16 * j, lane, pt[j]);
            __syncthreads();
            write_mat<E, false>(mats + kDeltaMatBytes, sA, w, lane, a.p_lo);
            write_mat<E, false>(mats, sT, w, lane, true, sF[16 * w + n16]);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------------
// delta_chain: one segment of one head, 64 NC columns per workgroup (16 NC per wave), the state in accumulators.
// LOCAL: the segment's end state from zero (columns of V; segment 0 starts from state_in) or its transition (columns of
// the identity, V = 0), into segE / segM. Otherwise the outputs, and after the last segment the final state.
// ---------------------------------------------------------------------------------------------------
// A step's order keeps registers few and every latency behind work: the next chunk's rows are requested first; Y and R;
// then K and V of the next chunk go to LDS (K has two buffers; a wave stages the columns of V it owns, so no one else
// reads them); Q S; a barrier frees Q's buffer; O; E; the state. Fragments of one reduction
// step are read while the products of the step before run.
// kFull: outputs (bf16 from bf16 input, else fp32); kFullF32: BF16 input, F32 output; kLocal / kLocalRaw: end state or
// transition, with Ts / with T; kStates: with T, the states entering the chunks and E, for the gradients.
enum { kFull = 0, kFullF32 = 1, kLocal = 2, kLocalRaw = 3, kStates = 4 };
// Waves per SIMD that the LDS leaves room for (at most 2: the state and the fragments in flight take half the registers).
template <class E, int DK, int NC, int NW, int MODE>
constexpr int chain_waves() {
    typedef DOps<E> D;
    const int rows = kDeltaC * (int)sizeof(typename E::st);
    const int lds = rows * ((MODE <= kFullF32 ? 3 : 2) * D::template Tile<DK>::LD + D::template Tile<16 * NC * NW>::LD) + 1024;
    if (NW == 8) return 2 * lds <= 160 * 1024 ? 4 : 2;
    return (2 * lds <= 160 * 1024 && (sizeof(typename E::st) == 2 || DK * NC <= 64)) ? 2 : 1;
}
template <class E, int DK, int NC, int NW, int MODE>
__global__ __launch_bounds__(64 * NW, (chain_waves<E, DK, NC, NW, MODE>())) void delta_chain_kernel(DeltaArgs a) {
    typedef typename E::st st;
    typedef DOps<E> D;
    constexpr int NT = 64 * NW, COLS = 16 * NC * NW;
    typedef DRows<E, DK, NT> Rows;
    typedef DRows<E, 16 * NC, 64, typename D::template Tile<COLS>> VRows;  // a wave's own columns
    typedef typename Rows::Tile Tile;
    typedef typename VRows::Tile VTile;
    typedef TriFrags<D::KS> F;
    constexpr bool LOCAL = MODE == kLocal || MODE == kLocalRaw, FULL = MODE == kFull || MODE == kFullF32;
    constexpr bool RAW = MODE == kLocalRaw || MODE == kStates;
    constexpr bool HI = MODE == kFull && sizeof(st) == 2;  // outputs in bf16: the high parts of S and P T suffice, whose
                                                           // rounding is like the output's own
    typedef typename std::conditional<HI, uint16_t, float>::type out_t;
    constexpr int DT = DK / 16, NS = F::NS, KN = DK / D::KS;
    constexpr int MB = NC == 2 ? 2 : 4, MG = 4 / MB;  // token tiles whose fragments are read together: 8 products' worth
    __shared__ __align__(16) st sk[2][kDeltaC * Tile::LD];
    __shared__ __align__(16) st sq[FULL ? kDeltaC * Tile::LD : 16];
    __shared__ __align__(16) st sv[kDeltaC * VTile::LD];
    __shared__ __align__(16) float sf[2][128];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15, g4 = 4 * (lane >> 4);
    const int nE = (a.dv + COLS - 1) / COLS;  // workgroups over d_v; a local pass has those of d_k behind them
    const DeltaBlock blk = delta_block(a, nE + (LOCAL ? (DK + COLS - 1) / COLS : 0));
    if (blk.bh >= a.B * a.H) return;
    const int bh = blk.bh, seg = blk.seg, b = bh / a.H, h = bh % a.H;
    const bool trans = LOCAL && blk.cb >= nE;
    const int width = trans ? DK : a.dv;
    const int col0 = (blk.cb - (trans ? nE : 0)) * COLS + w * 16 * NC;
    const int hk = h / (a.H / a.Hk), len = delta_len(a, b);
    const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nchunks);
    const bool active = col0 < width;
    // segment 0's end state is known, and no one asks for the last one's
    if (LOCAL && (trans ? seg == 0 : seg == a.nseg - 1)) return;
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};

    f32x4_t S[NC][DT];
    const float* sin = nullptr;
    if (!LOCAL) sin = a.nseg > 1 ? a.segE + ((long long)bh * a.nseg + seg) * DK * a.dv : nullptr;
    if (!LOCAL && a.nseg == 1) sin = a.state_in ? a.state_in + (long long)bh * DK * a.dv : nullptr;
    if (LOCAL && seg == 0 && !trans && a.state_in) sin = a.state_in + (long long)bh * DK * a.dv;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int col = col0 + 16 * n + n16;
        const bool in = sin && col0 + 16 * n < width;
        const float* p = in ? sin + (long long)g4 * a.dv + col : nullptr;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[n][t][i] = trans && 16 * t + g4 + i == col ? 1.f : 0.f;
        if (in)
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[n][t][i] = p[(long long)(16 * t + i) * a.dv];
    }

    Rows rk, rq;
    VRows rv;
    float ff = 0.f;
    const st* kp = (const st*)a.k + (((long long)b * a.N) * a.Hk + hk) * DK;
    const st* qp = (const st*)a.q + (((long long)b * a.N) * a.Hk + hk) * DK;
    const st* vp = (const st*)a.v + (((long long)b * a.N) * a.H + h) * a.dv + col0;
    auto fetch = [&](int c) {
        const int live = min(kDeltaC, len - c * kDeltaC);
        const long long base = (long long)c * kDeltaC * a.Hk * DK;
        rk.load(kp + base, a.Hk * DK, live, DK, tid);
        rv.load(vp + (long long)c * kDeltaC * a.H * a.dv, a.H * a.dv, !trans && active ? live : 0, a.dv - col0, lane);
        if constexpr (FULL) rq.load(qp + base, a.Hk * DK, live, DK, tid);
        ff = a.fac[((long long)bh * a.nchunks + c) * kDeltaFac + (tid & 127)];
    };
    auto stage = [&](int p) {
        rk.store(sk[p], tid);
        if (!trans && active) rv.store(sv, lane, 16 * NC * w);
        if (tid < 128) sf[p][tid] = ff;
    };
    const int cend = min(c1, (len + kDeltaC - 1) / kDeltaC);  // chunks with live tokens
    if (c0 < cend) {
        fetch(c0);
        stage(0);
        if constexpr (FULL) rq.store(sq, tid);
    }
    for (int c = c0, p = 0; c < cend; ++c, p ^= 1) {
        __syncthreads();
        const bool more = c + 1 < cend;
        // (the last chunk again at the end: a conditional request would make its registers wait where the branches join)
        fetch(more ? c + 1 : c);
        const char* mats = a.mats + ((long long)bh * a.nchunks + c) * a.nmats * kDeltaMatBytes;
        const st* K = sk[p];
        f32x4_t y[NC][4];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m) y[n][m] = zero;
        if (active) {
            if constexpr (MODE == kStates) {
                st* sp = (st*)a.s0t + ((long long)bh * a.nchunks + c) * a.dv * DK;
#pragma unroll
                for (int n = 0; n < NC; ++n)
                    if (col0 + 16 * n < width)
#pragma unroll
                        for (int t = 0; t < DT; ++t)
                            store4(sp + (long long)(col0 + 16 * n + n16) * DK + 16 * t + g4, S[n][t]);
            }
            // Y = K S
            typename D::Fa fk[2][MB];
            typename D::Fb fs[2][NC];
#pragma unroll
            for (int m = 0; m < MB; ++m) fk[0][m] = Tile::rows(K, 16 * m, 0, lane);
#pragma unroll
            for (int n = 0; n < NC; ++n) fs[0][n] = D::step(S[n], 0);
#pragma unroll
            for (int i = 0; i < KN * MG; ++i) {
                const int s = i / MG, m0 = i % MG * MB, s1 = (i + 1) / MG, m1 = (i + 1) % MG * MB;
                if (i + 1 < KN * MG)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        fk[(i + 1) & 1][m] = Tile::rows(K, 16 * (m1 + m), s1 * D::KS, lane);
                keep_order();
                D::template products<MB, NC>(y, m0, fk[i & 1], fs[s & 1]);
                if (m1 == 0 && s1 < KN)
#pragma unroll
                    for (int n = 0; n < NC; ++n) fs[s1 & 1][n] = D::step(S[n], s1);
                keep_order();
            }
            // R = V - exp(G) Y
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f32x4_t ga = *reinterpret_cast<const f32x4_t*>(sf[p] + 16 * m + g4);
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    const f32x4_t v = trans ? zero : VTile::acc(sv, m, 16 * NC * w + 16 * n, lane);
                    y[n][m] = v - ga * y[n][m];
                }
            }
        }
        keep_order();
        if (more) stage(p ^ 1);
        keep_order();
        typename D::Fm ft[F::COUNT];
        if constexpr (!FULL)
#pragma unroll
            for (int f = 0; f < F::COUNT; ++f) ft[f] = D::mat_frag(mats, f, lane);
        typename D::Fb fr[NC][NS];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int s = 0; s < NS; ++s) fr[n][s] = D::step(y[n], s);
        if constexpr (FULL) {
            // O^T = scale exp(G) (Q S)^T + R^T (P T)^T: a lane holds 4 columns of token 16 m + n16
            f32x4_t o[NC][4];
            if (active) {
#pragma unroll
                for (int n = 0; n < NC; ++n)
#pragma unroll
                    for (int m = 0; m < 4; ++m) o[n][m] = zero;
                typename D::Fa fq[2][MB];
                typename D::Fb fs[NC];
                typename D::Fx fx[2][NC];
#pragma unroll
                for (int m = 0; m < MB; ++m) fq[0][m] = Tile::rows(sq, 16 * m, 0, lane);
                if constexpr (HI)
#pragma unroll
                    for (int n = 0; n < NC; ++n) fx[0][n] = D::step_exact(S[n], 0);
#pragma unroll
                for (int i = 0; i < KN * MG; ++i) {
                    const int s = i / MG, m0 = i % MG * MB, s1 = (i + 1) / MG, m1 = (i + 1) % MG * MB;
                    if (i + 1 < KN * MG)
#pragma unroll
                        for (int m = 0; m < MB; ++m)
                            fq[(i + 1) & 1][m] = Tile::rows(sq, 16 * (m1 + m), s1 * D::KS, lane);
                    keep_order();
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        if constexpr (!HI)
                            if (m0 == 0) fs[n] = D::step(S[n], s);
#pragma unroll
                        for (int m = 0; m < MB; ++m) {
                            if constexpr (HI) D::mma_aa(o[n][m0 + m], fx[s & 1][n], fq[i & 1][m]);
                            else D::mma_ba(o[n][m0 + m], fq[i & 1][m], fs[n]);
                        }
                        if constexpr (HI)
                            if (m1 == 0 && s1 < KN) fx[s1 & 1][n] = D::step_exact(S[n], s1);
                    }
                    keep_order();
                }
            }
            keep_order();
            typename D::Fa fp[F::COUNT];
#pragma unroll
            for (int f = 0; f < F::COUNT; ++f) fp[f] = D::mat_frag_hi(mats + kDeltaMatBytes, f, lane);
#pragma unroll
            for (int f = 0; f < F::COUNT; ++f) ft[f] = D::mat_frag(mats, f, lane);
            if (more) {
                __syncthreads();
                rq.store(sq, tid);
            }
            if (active) {
                const int live = min(kDeltaC, len - c * kDeltaC);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float f = a.scale * sf[p][16 * m + n16];
#pragma unroll
                    for (int n = 0; n < NC; ++n) o[n][m] *= f;
                }
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        if (F::lower(m, s)) {
#pragma unroll
                            for (int n = 0; n < NC; ++n) D::mma_ba(o[n][m], fp[F::at(m, s, false)], fr[n][s]);
                            if constexpr (MODE == kFullF32) {
                                const typename D::Fm fl = D::mat_frag(mats + kDeltaMatBytes, F::at(m, s, false), lane);
#pragma unroll
                                for (int n = 0; n < NC; ++n) D::mma_lo(o[n][m], fl, fr[n][s]);
                            }
                        }
                if (live < kDeltaC)  // padding
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int n = 0; n < NC; ++n)
                            if (16 * m + n16 >= live) o[n][m] = zero;
                DOut out;
                out.init(a.o, ((long long)b * a.N + c * kDeltaC) * a.H + h, min(kDeltaC, a.N - c * kDeltaC), a.H, a.dv,
                         sizeof(out_t), col0 + g4, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n)
                    if (col0 + 16 * n < width)
#pragma unroll
                        for (int m = 0; m < 4; ++m) out.put((out_t*)nullptr, m, n, o[n][m]);
            }
        }
        keep_order();
        if (!active) continue;
        // E' = exp(G_C - G) beta T R
        f32x4_t u[NC][4];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m) u[n][m] = zero;
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int m = 0; m < 4; ++m)
                if (F::lower(m, s)) {
#pragma unroll
                    for (int n = 0; n < NC; ++n) D::mma_mb(u[n][m], ft[F::at(m, s, false)], fr[n][s]);
                }
        keep_order();
        if constexpr (MODE == kStates) {
            st* ep = (st*)a.et + ((long long)bh * a.nchunks + c) * a.dv * kDeltaC;
#pragma unroll
            for (int n = 0; n < NC; ++n)
                if (col0 + 16 * n < width)
#pragma unroll
                    for (int m = 0; m < 4; ++m) store4(ep + (col0 + 16 * n + n16) * kDeltaC + 16 * m + g4, u[n][m]);
        }
        if constexpr (RAW)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f32x4_t ta = *reinterpret_cast<const f32x4_t*>(sf[p] + 64 + 16 * m + g4);
#pragma unroll
                for (int n = 0; n < NC; ++n) u[n][m] *= ta;
            }
        // S = exp(G_C) S + K^T E'
        const float end = sf[p][63];
        typename D::Fb fu[NC][NS];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int s = 0; s < NS; ++s) fu[n][s] = D::step(u[n], s);
        constexpr int TB = DT < MB ? DT : MB;  // tiles whose fragments are read together
        typename D::Fa fc[2][TB];
#pragma unroll
        for (int t = 0; t < TB; ++t) fc[0][t] = Tile::cols(K, 0, 16 * t, lane);
#pragma unroll
        for (int i = 0; i < NS * DT / TB; ++i) {
            const int s = i % NS, t0 = i / NS * TB, s1 = (i + 1) % NS, t1 = (i + 1) / NS * TB;
            if (i + 1 < NS * DT / TB)
#pragma unroll
                for (int t = 0; t < TB; ++t) fc[(i + 1) & 1][t] = Tile::cols(K, s1 * D::KS, 16 * (t1 + t), lane);
            keep_order();
            if (s == 0)
#pragma unroll
                for (int n = 0; n < NC; ++n)
#pragma unroll
                    for (int t = 0; t < TB; ++t) S[n][t0 + t] *= end;
            D::template products<TB, NC>(S, t0, fc[i & 1], fu, s);
            keep_order();
        }
    }
    if (!active) return;
    // outputs of padding chunks are zero
    if constexpr (FULL) {
        for (int c = max(c0, cend); c < c1; ++c) {
            DOut out;
            out.init(a.o, ((long long)b * a.N + c * kDeltaC) * a.H + h, min(kDeltaC, a.N - c * kDeltaC), a.H, a.dv,
                     sizeof(out_t), col0 + g4, lane);
#pragma unroll
            for (int n = 0; n < NC; ++n)
                if (col0 + 16 * n < width)
#pragma unroll
                    for (int m = 0; m < 4; ++m) out.put((out_t*)nullptr, m, n, zero);
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
        float* p = out + (long long)g4 * width + col0 + 16 * n + n16;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) p[(long long)(16 * t + i) * width] = S[n][t][i];
    }
}

// ---------------------------------------------------------------------------------------------------
// delta_scan: the states entering the segments. In: segE[s] = segment s's end state from zero (segment 0: its true end
// state), segM[s] its transition. Out: segE[s] = the state entering segment s, S_{s+1} = M_s S_s + E_s. One workgroup per
// (b, h, 16 columns); REV: the gradients' chain, D_{s-1} = M_s^T D_s + F_s over segF from the right. The waves share the rows of M, S goes round through LDS. BF16
// input: M and S split in two bf16 parts like the chain's operands.
// ---------------------------------------------------------------------------------------------------
// waves of a scan workgroup: 16 rows of the state each, 32 at d_k = 256 (the rows of M in flight take the registers)
template <int DK>
constexpr int scan_waves() { return DK / 16 <= 8 ? DK / 16 : 8; }
template <class E, int DK, bool REV>
__global__ __launch_bounds__(64 * scan_waves<DK>()) void delta_scan_kernel(DeltaArgs a) {
    typedef DOps<E> D;
    constexpr int NS = DK / D::KS, TPS = D::TPS, RT = DK / 16 / scan_waves<DK>(), CT = kScanCols / 16, LD = kScanCols + 4;
    __shared__ __align__(16) float sS[2][DK * LD];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15;
    const int g4 = 4 * (lane >> 4), bh = blockIdx.x, c0 = blockIdx.y * kScanCols;
    const long long sz = (long long)DK * a.dv;
    float* X = (REV ? a.segF : a.segE) + (long long)bh * a.nseg * sz + (long long)(16 * RT * w + g4) * a.dv + c0 + n16;
    // this lane's part of the rows of M (REV: of its transpose) that wave w multiplies
    const float* M = a.segM + (long long)bh * a.nseg * DK * DK +
                     (REV ? g4 * DK + 16 * RT * w + n16 : (16 * RT * w + n16) * DK + g4);
    const float* from = REV ? a.dstate_out : a.state_in;
    const float* sin = from ? from + bh * sz + (long long)(16 * RT * w + g4) * a.dv + c0 + n16 : nullptr;
    const int len = delta_len(a, bh / a.H);
    f32x4_t S[RT][CT], e[RT][CT], m[RT][NS][TPS];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[r][t][i] = sin && c0 + 16 * t < a.dv ? sin[(long long)(16 * r + i) * a.dv + 16 * t] : 0.f;
    auto fetch = [&](int j) {  // the j-th segment on the way: its end state from zero and its transition
        const int s = REV ? a.nseg - 1 - j : j;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < CT; ++t)
                if (c0 + 16 * t < a.dv)
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[r][t][i] = X[s * sz + (long long)(16 * r + i) * a.dv + 16 * t];
        if (j == 0) return;
        const float* p = M + (long long)s * DK * DK;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int k = 0; k < NS; ++k)
#pragma unroll
                for (int t = 0; t < TPS; ++t) {
                    if constexpr (REV) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) m[r][k][t][i] = p[(D::KS * k + 16 * t + i) * DK + 16 * r];
                    } else {
                        m[r][k][t] = *reinterpret_cast<const f32x4_t*>(p + 16 * r * DK + D::KS * k + 16 * t);
                    }
                }
    };
    fetch(0);
    for (int j = 0;; ++j) {
        const int s = REV ? a.nseg - 1 - j : j;
        float* x = sS[j & 1];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[(16 * (RT * w + r) + g4 + i) * LD + 16 * t + n16] = S[r][t][i];
                    if (c0 + 16 * t < a.dv) X[s * sz + (long long)(16 * r + i) * a.dv + 16 * t] = S[r][t][i];
                }
        if (j == a.nseg - 1) return;
        __syncthreads();
        if (j == 0) {  // from the state entering the first segment
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < CT; ++t) S[r][t] = e[r][t];
        } else if (s * a.seg_chunks * kDeltaC < len) {  // else no live token: the state passes as it is
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < CT; ++t) S[r][t] = e[r][t];
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                typename D::Fb fm[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) fm[r] = D::step(m[r][k], 0);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    f32x4_t y[TPS];
#pragma unroll
                    for (int p = 0; p < TPS; ++p)
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[p][i] = x[(D::KS * k + 16 * p + g4 + i) * LD + 16 * t + n16];
                    const typename D::Fb fy = D::step(y, 0);
#pragma unroll
                    for (int r = 0; r < RT; ++r) D::mma_mb(S[r][t], fm[r], fy);
                }
            }
        }
        if (j + 1 < a.nseg - 1) fetch(j + 1);
    }
}

template <class E, int DK, int NC, int NW>
void pick_cols(DeltaKernels* o) {
    *o = {};
    o->prep = delta_prep_kernel<E, DK, false>;
    o->bprep = delta_prep_kernel<E, DK, true>;
    o->local = delta_chain_kernel<E, DK, NC, NW, kLocal>;
    o->blocal = delta_chain_kernel<E, DK, NC, NW, kLocalRaw>;
    o->full = delta_chain_kernel<E, DK, NC, NW, kFull>;
    o->full_f32 = delta_chain_kernel<E, DK, NC, NW, sizeof(typename E::st) == 2 ? kFullF32 : kFull>;
    o->states = delta_chain_kernel<E, DK, NC, NW, kStates>;
    o->scan = delta_scan_kernel<E, DK, false>;
    o->rscan = delta_scan_kernel<E, DK, true>;
    o->scan_threads = 64 * scan_waves<DK>();
    o->cols = 16 * NC * NW;
    o->threads = 64 * NW;
}
// Two column tiles per wave halve the operand reads per product; one where d_v would leave waves idle, and where a row of
// K takes 512 bytes: the state of two tiles would take the registers of a second wave on the SIMD, so eight waves share
// the rows instead.
template <class E, int DK>
void pick(int dv, DeltaKernels* o) {
    constexpr bool WIDE = DK * sizeof(typename E::st) >= 256;
    if (dv <= 64 || DK <= 128) pick_cols<E, DK, 1, 4>(o);
    else if constexpr (WIDE) pick_cols<E, DK, 1, 8>(o);
    else pick_cols<E, DK, 2, 4>(o);
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
