// Gradients of the gated delta rule. In the chunk form of delta.h, with the gradient dS_C of the state leaving a chunk,
// Tr = (I + Ar)^-1, Ar_ij = beta_i exp(G_i - G_j) (k_i.k_j) (j < i), Pr_ij = scale exp(G_i - G_j) (q_i.k_j) (j <= i) and
// D_ij = exp(G_i - G_j):
//     W = Pr^T dO + exp(G_C - G) K dS_C,  dU = Tr^T W   (gradients of the writes u = beta e),  dV = beta dU,
//     dS_0 = exp(G_C) dS_C + Q^T (scale exp(G) dO) - K^T (exp(G) beta dU)
// is a second chain, from the last chunk to the first, whose products stay within a wave like the forward's. What is left
// is local to a chunk, given S_0, dS_C, E and dU (stored by the two chains):
//     X_ij = scale D_ij beta_j (dO_i.E_j) (j <= i),   Z_ij = -D_ij beta_i beta_j (dU_i.E_j) (j < i),
//     dQ = scale exp(G) dO S_0^T + X K,
//     dK = Kr + Kw,  Kr = -exp(G) beta dU S_0^T + Z K  (k as it reads),
//                    Kw = exp(G_C - G) beta E dS_C^T + X^T Q + Z^T K  (k as it writes),
//     dbeta_i = dU_i.E_i,
//     dG_i = q_i.dq_i + k_i.Kr_i - k_i.Kw_i,  dG_C gets <S_C, dS_C> more,  dg_t = sum of dG_i over i >= t in the chunk:
// exp(G_i) stands with every q_i and reading k_i, exp(-G_i) with every writing k_i, exp(G_C) with S_C. Solving for E with
// beta along the columns and for dU with beta along the rows leaves no division by beta, which may be zero.
#include "delta.h"

namespace ret {

namespace {

typedef double f64;

// ---------------------------------------------------------------------------------------------------
// The chain from the right: one segment of one head, 16 columns per wave, dS in accumulators. LOCAL: the gradient of the
// state entering the segment from a zero one leaving it (the last segment: from dstate_out), into segF. Otherwise dS_C of
// each chunk and dU, as blocks (TWO: in two parts), and dV; the first segment leaves dstate_in. Built as the forward's chain: requests a chunk
// ahead between the products of K dS, K in two buffers, Q's product before the second barrier. 10 us a step at d_k = 256,
// 7 at 128, by the same measure as the forward's; 8192 tokens, 16 heads, d_k = 256, d_v = 512: 242 us local, 336 us full.
// ---------------------------------------------------------------------------------------------------
template <class E, int DK, int NW, bool LOCAL, bool TWO>
__global__ __launch_bounds__(64 * NW) void delta_rchain_kernel(DeltaArgs a) {
    typedef typename E::st st;
    typedef DOps<E> D;
    constexpr int NT = 64 * NW, COLS = 16 * NW;
    typedef DRows<E, DK, NT, typename D::template STile<DK>> Rows;
    typedef DRows<E, 16, 64, typename D::template Tile<COLS>> ORows;  // a wave's own columns of dO
    typedef typename Rows::Tile Tile;
    typedef typename ORows::Tile OTile;
    typedef TriFrags<D::KS> F;
    constexpr int DT = DK / 16, NS = F::NS, KN = DK / D::KS, TB = DT < 4 ? DT : 4;
    __shared__ __align__(16) st sk[2][kDeltaC * Tile::LD];
    __shared__ __align__(16) st sq[kDeltaC * Tile::LD];
    __shared__ __align__(16) st so[kDeltaC * OTile::LD];
    __shared__ __align__(16) char sm[F::BYTES], sp[F::BYTES];  // Tr^T, Pr^T
    __shared__ __align__(16) float sf[2][256];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15;
    const int g4 = 4 * (lane >> 4);
    const DeltaBlock blk = delta_block(a, (a.dv + COLS - 1) / COLS);
    if (blk.seg >= a.nseg) return;
    const int bh = blk.bh, seg = blk.seg, b = bh / a.H, h = bh % a.H;
    const int mine = 16 * w, col0 = blk.cb * COLS + mine;  // the wave's columns: in the tile, of d_v
    const int hk = h / (a.H / a.Hk), len = delta_len(a, b);
    const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nchunks);
    const bool active = col0 < a.dv;  // (a wave without columns computes on zeros)
    if (LOCAL && seg == 0) return;  // no one is left of it
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};

    f32x4_t S[DT];
    const float* sin = nullptr;
    if (LOCAL ? seg == a.nseg - 1 : a.nseg == 1)
        sin = a.dstate_out ? a.dstate_out + (long long)bh * DK * a.dv : nullptr;
    else if (!LOCAL) sin = a.segF + ((long long)bh * a.nseg + seg) * DK * a.dv;
#pragma unroll
    for (int t = 0; t < DT; ++t) S[t] = zero;
    if (sin && active) {
        const float* p = sin + col0 + n16;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[t][i] = p[(long long)(D::srow(t, g4) + i) * a.dv];
    }
    Rows rk, rq;
    ORows ro;
    DMat<F::BYTES, NT> rm, rp;
    float ff = 0.f;
    const float* fp;
    const st* kp = (const st*)a.k + (((long long)b * a.N) * a.Hk + hk) * DK;
    const st* qp = (const st*)a.q + (((long long)b * a.N) * a.Hk + hk) * DK;
    const st* op = (const st*)a.dout + (((long long)b * a.N) * a.H + h) * a.dv + col0;
    auto from = [&](int c) {  // the places of chunk c's operands
        const int live = min(kDeltaC, len - c * kDeltaC);
        const long long base = (long long)c * kDeltaC * a.Hk * DK;
        const char* mats = a.mats + ((long long)bh * a.nchunks + c) * a.nmats * kDeltaMatBytes;
        rk.from(kp + base, a.Hk * DK, live, DK, tid);
        rq.from(qp + base, a.Hk * DK, live, DK, tid);
        ro.from(op + (long long)c * kDeltaC * a.H * a.dv, a.H * a.dv, active ? live : 0, a.dv - col0, lane);
        rm.from(mats + kDeltaMatBytes, tid);
        rp.from(mats + 2 * kDeltaMatBytes, tid);
        fp = a.fac + ((long long)bh * a.nchunks + c) * kDeltaFac + (tid & 255);
    };
    constexpr int NK = Rows::NP, NO = ORows::NP, NM = DMat<F::BYTES, NT>::NP, NL = 2 * NK + NO + 2 * NM + 1;
    auto request = [&](int i) {
        if (i < NK) rk.get(i);
        else if (i < NK + NM) rp.get(i - NK);
        else if (i < NK + 2 * NM) rm.get(i - NK - NM);
        else if (i < NK + 2 * NM + 1) ff = *fp;
        else if (i < NL - NK) ro.get(i - NK - 2 * NM - 1);
        else rq.get(i - (NL - NK));
    };
    auto stage = [&](int p) {
        rk.store(sk[p], tid);
        rq.store(sq, tid);
        ro.store(so, lane, mine);
        if (tid < 256) sf[p][tid] = ff;
    };
    // Rows of dV of chunk c, 16 bytes a lane, from the wave's own columns of the tile that held dO (zero: zeros); rows past
    // the live ones are zero. 32-bit outputs go from the registers.
    auto store_rows = [&](int c, bool blank) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = (lane + 64 * i) / 2, cc = lane % 2 * 8, t = c * kDeltaC + row;
            if (t >= a.N) continue;
            u32x4_t x = {0, 0, 0, 0};
            if (!blank && t < len) x = *reinterpret_cast<const u32x4_t*>(so + OTile::off(row, mine + cc));
            *reinterpret_cast<u32x4_t*>((uint16_t*)a.dv_ + (((long long)b * a.N + t) * a.H + h) * a.dv + col0 + cc) = x;
        }
    };
    auto store_f32 = [&](int c, int m, const f32x4_t& x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = c * kDeltaC + 16 * m + g4 + i;
            if (t >= a.N) continue;
            ((float*)a.dv_)[(((long long)b * a.N + t) * a.H + h) * a.dv + col0 + n16] = t < len ? x[i] : 0.f;
        }
    };
    const int cend = min(c1, (len + kDeltaC - 1) / kDeltaC);  // chunks with live tokens
    if constexpr (!LOCAL) {
        if (active)
            for (int c = max(c0, cend); c < c1; ++c) {  // dV of padding chunks is zero
                if (a.out_bf16) store_rows(c, true);
                else
#pragma unroll
                    for (int m = 0; m < 4; ++m) store_f32(c, m, zero);
            }
    }
    if (c0 < cend) {
        from(cend - 1);
#pragma unroll
        for (int i = 0; i < NL; ++i) request(i);
        stage(0);
    }
    for (int c = cend - 1, p = 0; c >= c0; --c, p ^= 1) {
        __syncthreads();
        rm.store(sm);  // everyone is past the last chunk's products with them
        rp.store(sp);
        from(max(c - 1, c0));
        const long long unit = (long long)bh * a.nchunks + c;
        const st* K = sk[p];
        if constexpr (!LOCAL) {
            st* out = (st*)a.ds1t + (unit * a.dv + col0) * DK;
            if (active)
#pragma unroll
                for (int t = 0; t < DT / D::TPS; ++t) {
                    D::blk_store(out, t, lane, &S[D::TPS * t]);
                    if constexpr (TWO) D::blk_store_lo(out + a.state_lo, t, lane, &S[D::TPS * t]);
                }
        }
        // W = exp(G_C - G) K dS + Pr^T dO
        f32x4_t x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = zero;
        {
            typename D::Fa fk[2][4];
            typename D::Fb fs[2];
#pragma unroll
            for (int m = 0; m < 4; ++m) fk[0][m] = Tile::rows(K, 16 * m, 0, lane);
            fs[0] = D::step(S, 0);
#pragma unroll
            for (int s = 0; s < KN; ++s) {
                if (s + 1 < KN)
#pragma unroll
                    for (int m = 0; m < 4; ++m) fk[(s + 1) & 1][m] = Tile::rows(K, 16 * m, s + 1, lane);
#pragma unroll
                for (int i = NL * s / KN; i < NL * (s + 1) / KN; ++i) request(i);
                keep_order();
                D::template products<4>(x, 0, fk[s & 1], fs[s & 1]);
                if (s + 1 < KN) fs[(s + 1) & 1] = D::step(S, s + 1);
                keep_order();
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] *= *reinterpret_cast<const f32x4_t*>(sf[p] + 128 + 16 * m + g4);
        // S += X^T F, tile by tile, the first time scaled
        auto update = [&](const st* X, const typename D::Fb (&f)[NS], bool scaled, float end) {
            typename D::Fa fc[2][TB];
#pragma unroll
            for (int t = 0; t < TB; ++t) fc[0][t] = Tile::cols(X, 0, t, lane);
#pragma unroll
            for (int i = 0; i < NS * DT / TB; ++i) {
                const int s = i % NS, t0 = i / NS * TB, s1 = (i + 1) % NS, t1 = (i + 1) / NS * TB;
                if (i + 1 < NS * DT / TB)
#pragma unroll
                    for (int t = 0; t < TB; ++t) fc[(i + 1) & 1][t] = Tile::cols(X, s1 * D::KS, t1 + t, lane);
                keep_order();
                if (scaled && s == 0)
#pragma unroll
                    for (int t = 0; t < TB; ++t) S[t0 + t] *= end;
                D::template products<TB>(S, t0, fc[i & 1], f[s]);
                keep_order();
            }
        };
        typename D::Fx fd[NS];  // dO as it came
        {                       // dS = exp(G_C) dS + Q^T (scale exp(G) dO) ..
            f32x4_t y[4];
            typename D::Fb f[NS];
#pragma unroll
            for (int m = 0; m < 4; ++m) y[m] = OTile::acc(so, m, mine, lane);
#pragma unroll
            for (int s = 0; s < NS; ++s) fd[s] = D::step_exact(y, s);
#pragma unroll
            for (int m = 0; m < 4; ++m) y[m] *= a.scale * *reinterpret_cast<const f32x4_t*>(sf[p] + 16 * m + g4);
#pragma unroll
            for (int s = 0; s < NS; ++s) f[s] = D::step(y, s);
            update(sq, f, true, sf[p][63]);
        }
        __syncthreads();  // the matrices are there, and everyone is done with Q
        {
            typename D::Fm fm[F::COUNT];
#pragma unroll
            for (int f = 0; f < F::COUNT; ++f) fm[f] = D::mat_frag(sp, f, lane);
#pragma unroll
            for (int s = 0; s < NS; ++s) tri<E, true, false>(x, fm, fd[s], s);
        }
        // dU = Tr^T W
        f32x4_t u[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) u[m] = zero;
        {
            typename D::Fm fm[F::COUNT];
#pragma unroll
            for (int f = 0; f < F::COUNT; ++f) fm[f] = D::mat_frag(sm, f, lane);
            typename D::Fb fw[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) fw[s] = D::step(x, s);
#pragma unroll
            for (int s = 0; s < NS; ++s) tri<E, true, false>(u, fm, fw[s], s);
        }
        if constexpr (!LOCAL) {
            if (active) {
                st* out = (st*)a.dut + (unit * a.dv + col0) * kDeltaC;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    D::blk_store(out, s, lane, &u[D::TPS * s]);
                    if constexpr (TWO) D::blk_store_lo(out + a.rows_lo, s, lane, &u[D::TPS * s]);
                }
                const bool rows = sizeof(st) == 2 && a.out_bf16;
                wave_fence();  // the last reads of dO come before
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const f32x4_t y = *reinterpret_cast<const f32x4_t*>(sf[p] + 192 + 16 * m + g4) * u[m];
                    if constexpr (sizeof(st) == 2) {
                        if (rows) {  // over dO, in the wave's own columns
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int col = mine + n16;
                                so[OTile::off(16 * m + g4 + i, col & ~3) + (col & 3)] = f32_to_bf16(y[i]);
                            }
                        }
                    }
                    if (!rows) store_f32(c, m, y);
                }
                if (rows) {
                    wave_fence();  // the rows are read in another order
                    store_rows(c, false);
                    wave_fence();
                }
            }
        }
        // .. - K^T (exp(G) beta dU)
#pragma unroll
        for (int m = 0; m < 4; ++m)
            u[m] *= -(*reinterpret_cast<const f32x4_t*>(sf[p] + 16 * m + g4) *
                      *reinterpret_cast<const f32x4_t*>(sf[p] + 192 + 16 * m + g4));
        typename D::Fb fu[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) fu[s] = D::step(u, s);
        update(K, fu, false, 0.f);
        stage(p ^ 1);
    }
    if (!active) return;
    float* out = nullptr;
    if (LOCAL) out = a.segF + ((long long)bh * a.nseg + seg) * DK * a.dv;
    else if (seg == 0 && a.dstate_in) out = a.dstate_in + (long long)bh * DK * a.dv;
    if (!out) return;
    out += col0 + n16;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(long long)(D::srow(t, g4) + i) * a.dv] = S[t][i];
}

// R rows of W elements to an LDS tile by NT threads: rows at or past `rows` and columns at or past `cols` are zero.
template <class E, int R, int W, int NT>
struct GRows {
    typedef typename E::st st;
    static constexpr int EPS = 16 / sizeof(st), SPR = W / EPS, NP = (R * SPR + NT - 1) / NT;
    typedef typename DOps<E>::template Tile<W> Tile;
    u32x4_t x[NP];
    __device__ __forceinline__ void load(const st* p, int stride, int rows, int cols, int tid) {
        const int bytes = rows > 0 ? ((rows - 1) * stride + cols) * (int)sizeof(st) : 0;
        const rsrc_t r = bytes_rsrc(p, bytes);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int s = tid + i * NT, row = s / SPR, c = s % SPR * EPS;
            x[i] = buf_load16(r, row < rows && c < cols ? (row * stride + c) * (int)sizeof(st) : 0x40000000, 0);
        }
    }
    __device__ __forceinline__ void store(st* lds, int tid) const {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int s = tid + i * NT;
            if (R * SPR % NT == 0 || s < R * SPR)
                *reinterpret_cast<u32x4_t*>(lds + Tile::off(s / SPR, s % SPR * EPS)) = x[i];
        }
    }
};

// Blocks of 16 columns x R rows of an array stored by blk_store, VB columns of them, to an LDS tile [VB][R] by NT threads;
// columns at or past `cols` are zero.
// STATE: rows in the state's order.
template <class E, int R, int VB, int NT, bool STATE>
struct GBlocks {
    typedef typename E::st st;
    typedef DOps<E> D;
    static constexpr int PER = R / (16 * D::TPS), N = VB / 16 * PER * 64, NP = (N + NT - 1) / NT;
    typedef typename D::template Tile<R> Tile;
    u32x4_t x[NP];
    __device__ __forceinline__ void load(const st* p, int cols, int tid) {
        const rsrc_t r = bytes_rsrc(p, cols * R * (int)sizeof(st));
#pragma unroll
        for (int i = 0; i < NP; ++i) x[i] = buf_load16(r, 16 * (tid + i * NT), 0);
    }
    __device__ __forceinline__ void store(st* lds, int tid) const {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int s = tid + i * NT, blk = s / 64, lane = s % 64;
            const int row = blk / PER * 16 + (lane & 15), c0 = blk % PER * 16 * D::TPS;
            if (N % NT != 0 && s >= N) continue;
            if constexpr (STATE) D::template blk_lds_s<Tile>(lds, row, c0, 4 * (lane >> 4), x[i]);
            else D::template blk_lds<Tile>(lds, row, c0, 4 * (lane >> 4), x[i]);
        }
    }
};

// Blocks of E and of dU in two parts: segments of four arrays in one order (E's high and low, dU's high and low part), so that
// every thread moves the same number of them.
template <class E, int R, int VB, int NT>
struct GQuad {
    typedef typename E::st st;
    typedef DOps<E> D;
    static constexpr int PER = R / (16 * D::TPS), SEGS = VB / 16 * PER * 64, NP = 4 * SEGS / NT;
    static_assert(4 * SEGS % NT == 0 && SEGS % 64 == 0, "whole waves per array");
    typedef typename D::template Tile<R> Tile;
    u32x4_t x[NP];
    __device__ static __forceinline__ int array(int w, int i) { return (64 * w + i * NT) / SEGS; }
    __device__ __forceinline__ void load(const st* e, const st* u, long long lo, int cols, int lane, int w) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int k = array(w, i), s = 64 * w + i * NT - k * SEGS + lane;
            const st* p = (k & 2 ? u : e) + (k & 1 ? lo : 0);
            x[i] = buf_load16(bytes_rsrc(p, cols * R * (int)sizeof(st)), 16 * s, 0);
        }
    }
    __device__ __forceinline__ void store(st* lds, int lane, int w) const {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int k = array(w, i), blk = w + i * NT / 64 - k * SEGS / 64;
            const int row = blk / PER * 16 + (lane & 15), c0 = blk % PER * 16 * D::TPS;
            D::template blk_lds<Tile>(lds + k * VB * Tile::LD, row, c0, 4 * (lane >> 4), x[i]);
        }
    }
};

// sum of the products of two operand fragments
__device__ __forceinline__ float frag_dot(bf16x8_t a, bf16x8_t b) {
    const u32x4_t x = __builtin_bit_cast(u32x4_t, a), y = __builtin_bit_cast(u32x4_t, b);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s += __uint_as_float(x[i] << 16) * __uint_as_float(y[i] << 16);
        s += __uint_as_float(x[i] & 0xffff0000u) * __uint_as_float(y[i] & 0xffff0000u);
    }
    return s;
}
__device__ __forceinline__ float frag_dot(f32x4_t a, f32x4_t b) {
    return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}
__device__ __forceinline__ void unpack8(bf16x8_t a, float* f) {
    const u32x4_t x = __builtin_bit_cast(u32x4_t, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(x[i] << 16);
        f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float frag_dot(const DOps<BF16>::Fb& a, const DOps<BF16>::Fb& b) {
    float ah[8], al[8], bh[8], bl[8], s = 0.f;
    unpack8(a.hi, ah);
    unpack8(a.lo, al);
    unpack8(b.hi, bh);
    unpack8(b.lo, bl);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (ah[i] + al[i]) * (bh[i] + bl[i]);
    return s;
}

// What the chains stored and the matrices X and Z as operands: one part in the input's type, or (TWO) two bf16 parts, the
// low one `lo` elements behind the high one. mma adds a product, of operands in two parts all but that of the low ones.
template <class E, bool TWO>
struct GOps {
    typedef typename E::st st;
    typedef DOps<E> D;
    typedef typename D::Fa F;
    template <class Tile>
    __device__ static __forceinline__ F rows(const st* X, int, int r0, int k0, int lane) {
        return Tile::rows(X, r0, k0, lane);
    }
    template <class Tile>
    __device__ static __forceinline__ F cols(const st* X, int, int k0, int n0, int lane) {
        return Tile::cols(X, k0, n0, lane);
    }
    __device__ static __forceinline__ void mma(f32x4_t& acc, const F& a, const F& b) { D::mma_aa(acc, a, b); }
    __device__ static __forceinline__ void store(st* p, int, f32x4_t x) { store4(p, x); }
};
template <>
struct GOps<BF16, true> {
    typedef uint16_t st;
    typedef DOps<BF16> D;
    typedef D::Fb F;
    template <class Tile>
    __device__ static __forceinline__ F rows(const st* X, int lo, int r0, int k0, int lane) {
        return {Tile::rows(X, r0, k0, lane), Tile::rows(X + lo, r0, k0, lane)};
    }
    template <class Tile>
    __device__ static __forceinline__ F cols(const st* X, int lo, int k0, int n0, int lane) {
        return {Tile::cols(X, k0, n0, lane), Tile::cols(X + lo, k0, n0, lane)};
    }
    __device__ static __forceinline__ void mma(f32x4_t& acc, const F& a, const F& b) {
        D::mfma1(acc, a.lo, b.hi);
        D::mfma1(acc, a.hi, b.lo);
        D::mfma1(acc, a.hi, b.hi);
    }
    __device__ static __forceinline__ void mma(f32x4_t& acc, const F& a, bf16x8_t b) {
        D::mfma1(acc, a.lo, b);
        D::mfma1(acc, a.hi, b);
    }
    __device__ static __forceinline__ void mma(f32x4_t& acc, bf16x8_t a, const F& b) {
        D::mfma1(acc, a, b.lo);
        D::mfma1(acc, a, b.hi);
    }
    __device__ static __forceinline__ void store(st* p, int lo, f32x4_t x) {
        const uint2 u = make_uint2(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]));
        const f32x4_t h = {__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u)};
        *reinterpret_cast<uint2*>(p) = u;
        store4(p + lo, x - h);
    }
};

__device__ __forceinline__ f32x4_t lds4(const uint16_t* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return f32x4_t{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                   __uint_as_float(u.y & 0xffff0000u)};
}
__device__ __forceinline__ f32x4_t lds4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }
__device__ __forceinline__ float dot4(f32x4_t a, f32x4_t b) {
    return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}

// ---------------------------------------------------------------------------------------------------
// delta_grad: dq, dk, dg, dbeta of one chunk and key head (GROUP: the value heads that share it one after another, their
// dq and dk added up in registers: no atomics, one order). Wave w owns tokens 16 (w % 4) .. + 15 and 64 columns of d_k
// (all of a shorter one). Every product has its accumulator rows along d_k (or j) and columns along tokens: per-token
// factors are one value per lane and a lane holds 4 consecutive values of its token's row. d_v is walked in blocks of 32.
// Bound by HBM: 830 KB a chunk at d_k = 256, d_v = 512, 1.7 GB in 470 us, 3.6 TB/s (one workgroup of 16 waves per CU;
// with 8 waves, whose sums spilled, 100 us more); 199 us for 4 x 4096 tokens of 16 heads at d_k = d_v = 128 (at the copy
// rate 141). The sums of grouped heads spill 66 registers at d_k = 256 (8 key heads for the 16: 549 us) and 9 at 128 in fp32
// (8192 tokens of 8 heads: 142 us, and 148 ungrouped). X and Z go on in the input's type, like what the chains stored, so
// that a term of dq, dk, dbeta and dg of bf16 input carries two to four roundings of up to 2^-8 each: 0.003 in the 2-norm
// with the output's own 0.0017. dg is a difference of such sums, 0.003 as a rule and up to 0.008 where they nearly cancel.
// TWO (gates or outputs in fp32, whose type holds more): all of these in two bf16 parts, twice the bytes of the chains'
// arrays; dO, which then does not fit the LDS, is read as fragments. 720 us at d_k = 256 (8 waves with twice the registers:
// 16 would spill 87 of theirs), 350 at 128, 67 for 8 x 2048 tokens of 8 heads of 64 (42 in one part). Grouped heads spill
// 114 registers at d_k = 256 and 17 at 64: 908 us for 8 key heads of the 16, 76 for 2 of the 8. X's diagonal stands with q in dq
// and with k in Kw, so that it cancels in dg: in one part exactly (24-bit products), in two it is left to the end.
// ---------------------------------------------------------------------------------------------------
template <class E, int DK, int NW, bool GROUP, bool TWO>
__global__ __launch_bounds__(64 * NW, (NW == 4 && DK * sizeof(typename E::st) <= 128 ? 2 : 1))
void delta_grad_kernel(DeltaArgs a) {
    typedef typename E::st st;
    typedef DOps<E> D;
    typedef GOps<E, TWO> G;
    constexpr int NT = 64 * NW, HF = NW / 4, DH = DK / HF, DT = DH / 16, NS = kDeltaC / D::KS, VB = 32, P = TWO ? 2 : 1;
    typedef typename D::template Tile<DK> TK;
    typedef typename D::template Tile<VB> TO;
    typedef typename D::template Tile<kDeltaC> TC;
    // one part of: S_0 or dS_C, dO, E or dU, X or Z
    constexpr int kS = VB * TK::LD, kO = TWO ? 0 : kDeltaC * TO::LD, kE = VB * TC::LD, kX = kDeltaC * TC::LD;
    constexpr int kStage = 2 * P * (kS + kE) + kO, kXZ = 2 * P * kX;
    __shared__ __align__(16) st sk[kDeltaC * TK::LD];
    __shared__ __align__(16) st sq[kDeltaC * TK::LD];
    __shared__ __align__(16) st buf[kStage > kXZ ? kStage : kXZ];
    __shared__ f64 sG[kDeltaC];
    __shared__ float sF[256], sDg[HF][kDeltaC], sDb[kDeltaC], sR[2][NW], sXd[TWO ? kDeltaC : 1];
    st *sS = buf, *sD = sS + P * kS, *sO = sD + P * kS, *sE = sO + kO, *sU = sE + P * kE;
    st *sX = buf, *sZ = buf + P * kX;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15;
    const int g4 = 4 * (lane >> 4), tw = w & 3, hf = w >> 2, dk0 = hf * DH, i = 16 * tw + n16;  // this lane's token
    const int c = blockIdx.x, b = blockIdx.y / a.Hk, hk = blockIdx.y % a.Hk;
    const int rep = GROUP ? a.H / a.Hk : 1;
    const int t0 = c * kDeltaC, len = delta_len(a, b), live = min(kDeltaC, len - t0);
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    constexpr int kM2 = HF == 1 ? 1 : 0;  // M: E^T dO in the waves of the first columns, E^T dU in those of the last
    f32x4_t tq[GROUP ? DT : 1], tk[GROUP ? DT : 1], Dq[DT], Dr[DT], Du[DT], M[1 + kM2][4];
    if (GROUP)
#pragma unroll
        for (int t = 0; t < DT; ++t) tq[t] = tk[t] = zero;
    if (live > 0) {
        GRows<E, kDeltaC, DK, NT> rk, rq;
        const long long base = (((long long)b * a.N + t0) * a.Hk + hk) * DK;
        rk.load((const st*)a.k + base, a.Hk * DK, live, DK, tid);
        rq.load((const st*)a.q + base, a.Hk * DK, live, DK, tid);
        rk.store(sk, tid);
        rq.store(sq, tid);
    }
    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        if (live <= 0) {  // padding: zero gradients
            if (tid < kDeltaC && t0 + tid < a.N) {
                const long long e = ((long long)b * a.N + t0 + tid) * a.H + h;
                if (a.gate_bf16) ((uint16_t*)a.dg)[e] = ((uint16_t*)a.dbeta)[e] = 0;
                else ((float*)a.dg)[e] = ((float*)a.dbeta)[e] = 0.f;
            }
            continue;
        }
        const long long unit = ((long long)b * a.H + h) * a.nchunks + c;
#pragma unroll
        for (int t = 0; t < DT; ++t) Dq[t] = Dr[t] = Du[t] = zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) M[0][j] = M[kM2][j] = zero;
        float dot = 0.f;
        GBlocks<E, DK, VB, NT, true> rs[P], rd[P];
        GRows<E, kDeltaC, VB, NT> ro;
        GBlocks<E, kDeltaC, VB, NT, false> re, ru;
        GQuad<E, kDeltaC, VB, TWO ? NT : 64> reu;
        u32x4_t xo;  // this lane's part of dO's rows as a fragment
        const st* sp = (const st*)a.s0t + unit * a.dv * DK;
        const st* dp = (const st*)a.ds1t + unit * a.dv * DK;
        const st* ep = (const st*)a.et + unit * a.dv * kDeltaC;
        const st* up = (const st*)a.dut + unit * a.dv * kDeltaC;
        const st* op = (const st*)a.dout + (((long long)b * a.N + t0) * a.H + h) * a.dv;
        auto fetch = [&](int v0) {
            const int nv = min(VB, a.dv - v0);
#pragma unroll
            for (int p = 0; p < P; ++p) rs[p].load(sp + p * a.state_lo + (long long)v0 * DK, nv, tid);
#pragma unroll
            for (int p = 0; p < P; ++p) rd[p].load(dp + p * a.state_lo + (long long)v0 * DK, nv, tid);
            if constexpr (TWO) {
                const rsrc_t r = bytes_rsrc(op + v0, ((live - 1) * a.H * a.dv + nv) * (int)sizeof(st));
                const int at = i < live ? (i * a.H * a.dv + g4) * (int)sizeof(st) : 0x40000000;
                const u32x2_t x = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
                const u32x2_t y = __builtin_amdgcn_raw_buffer_load_b64(r, nv > 16 ? at + 16 * (int)sizeof(st) : 0x40000000, 0, 0);
                xo = u32x4_t{x[0], x[1], y[0], y[1]};
                reu.load(ep + v0 * kDeltaC, up + v0 * kDeltaC, a.rows_lo, nv, lane, w);
            } else {
                ro.load(op + v0, a.H * a.dv, live, nv, tid);
                re.load(ep + v0 * kDeltaC, nv, tid);
                ru.load(up + v0 * kDeltaC, nv, tid);
            }
        };
        fetch(0);
        const float* f = a.fac + unit * kDeltaFac;
        __syncthreads();  // the last head's readers are done
        if (tid < 256) sF[tid] = f[tid];
        if (tid < kDeltaC) sG[tid] = reinterpret_cast<const f64*>(f + 256)[tid];
        for (int v0 = 0; v0 < a.dv; v0 += VB) {
            __syncthreads();
#pragma unroll
            for (int p = 0; p < P; ++p) rs[p].store(sS + p * kS, tid);
#pragma unroll
            for (int p = 0; p < P; ++p) rd[p].store(sD + p * kS, tid);
            u32x4_t xo0;
            if constexpr (TWO) {
                xo0 = xo;
                reu.store(sE, lane, w);
            } else {
                ro.store(sO, tid);
                re.store(sE, tid);
                ru.store(sU, tid);
            }
            __syncthreads();
            fetch(min(v0 + VB, (a.dv - 1) / VB * VB));  // unconditional: see the forward chain
#pragma unroll
            for (int s = 0; s < VB / D::KS; ++s) {
                typename D::Fa fo;
                if constexpr (TWO) fo = __builtin_bit_cast(typename D::Fa, xo0);
                else fo = TO::rows(sO, 16 * tw, s * D::KS, lane);
                const typename G::F fu = G::template cols<TC>(sU, kE, s * D::KS, 16 * tw, lane);
                const typename G::F fe = G::template cols<TC>(sE, kE, s * D::KS, 16 * tw, lane);
#pragma unroll
                for (int t = 0; t < DT; ++t) {
                    const typename G::F fs = G::template cols<TK>(sS, kS, s * D::KS, dk0 + 16 * t, lane);
                    const typename G::F fd = G::template cols<TK>(sD, kS, s * D::KS, dk0 + 16 * t, lane);
                    G::mma(Dq[t], fs, fo);
                    G::mma(Dr[t], fs, fu);
                    G::mma(Du[t], fd, fe);
                    if ((t & 3) == tw) dot += frag_dot(fs, fd);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j > tw) continue;
                    const typename G::F fj = G::template cols<TC>(sE, kE, s * D::KS, 16 * j, lane);
                    if (hf == 0) G::mma(M[0][j], fj, fo);
                    if (hf == HF - 1) G::mma(M[kM2][j], fj, fu);
                }
            }
        }
        __syncthreads();
        const float ga = sF[i], tb = sF[64 + i], be = sF[192 + i], end = sF[63];
        float csum = 0.f;
#pragma unroll
        for (int t = 0; t < DT; ++t) {
            Dq[t] *= a.scale * ga;
            Dr[t] *= -(ga * be);
            Du[t] *= tb;
            csum += dot4(Du[t], lds4(sk + TK::off(i, dk0 + 16 * t + g4)));
        }
        // X and Z: this lane's row i, columns 16 j + g4 ..
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4_t x = zero, z = zero;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int jj = 16 * j + g4 + e;
                if (jj > i) continue;
                const float d = __builtin_amdgcn_exp2f((float)(sG[i] - sG[jj])) * sF[192 + jj];
                x[e] = a.scale * d * M[0][j][e];
                if constexpr (TWO) {
                    if (jj == i) {
                        if (hf == 0) sXd[i] = x[e];
                        x[e] = 0.f;
                    }
                }
                if (jj < i) z[e] = -d * be * M[kM2][j][e];
                else if (hf == HF - 1) sDb[i] = M[kM2][j][e];
            }
            if (hf == 0) G::store(sX + TC::off(i, 16 * j + g4), kX, x);
            if (hf == HF - 1) G::store(sZ + TC::off(i, 16 * j + g4), kX, z);
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const bool lower = s * D::KS <= 16 * tw + 15, upper = (s + 1) * D::KS > 16 * tw;
            const typename G::F fx = G::template rows<TC>(sX, kX, 16 * tw, s * D::KS, lane);
            const typename G::F fz = G::template rows<TC>(sZ, kX, 16 * tw, s * D::KS, lane);
            const typename G::F gx = G::template cols<TC>(sX, kX, s * D::KS, 16 * tw, lane);
            const typename G::F gz = G::template cols<TC>(sZ, kX, s * D::KS, 16 * tw, lane);
#pragma unroll
            for (int t = 0; t < DT; ++t) {
                const typename D::Fa fk = TK::cols(sk, s * D::KS, dk0 + 16 * t, lane);
                if (lower) {
                    G::mma(Dq[t], fk, fx);
                    G::mma(Dr[t], fk, fz);
                }
                if (upper) {
                    G::mma(Du[t], TK::cols(sq, s * D::KS, dk0 + 16 * t, lane), gx);
                    G::mma(Du[t], fk, gz);
                }
            }
        }
        float dg = 0.f;
#pragma unroll
        for (int t = 0; t < DT; ++t) {
            const f32x4_t kv = lds4(sk + TK::off(i, dk0 + 16 * t + g4)), qv = lds4(sq + TK::off(i, dk0 + 16 * t + g4));
            dg += dot4(qv, Dq[t]) + dot4(kv, Dr[t] - Du[t]);
            Dr[t] += Du[t];
            if constexpr (TWO) {
                Dq[t] += sXd[i] * kv;
                Dr[t] += sXd[i] * qv;
            }
            if constexpr (GROUP) {
                tq[t] += Dq[t];
                tk[t] += Dr[t];
            }
        }
        dg += __shfl_xor(dg, 16);
        dg += __shfl_xor(dg, 32);
        if (lane < 16) sDg[hf][i] = dg;
        dot = lanes_sum<64>(dot);
        csum = lanes_sum<64>(csum);
        if (lane == 0) {
            sR[0][w] = dot;
            sR[1][w] = csum;
        }
        __syncthreads();
        if (w == 0) {
            f64 x = 0.0;
#pragma unroll
            for (int j = 0; j < HF; ++j) x += sDg[j][lane];
            if (lane == 63)
#pragma unroll
                for (int j = 0; j < NW; ++j) x += (f64)end * sR[0][j] + sR[1][j];
#pragma unroll
            for (int m = 1; m < 64; m *= 2) {
                const f64 down = __shfl_down(x, m);
                if (lane + m < 64) x += down;
            }
            if (t0 + lane < a.N) {
                const long long e = ((long long)b * a.N + t0 + lane) * a.H + h;
                const float y = lane < live ? (float)x : 0.f, z = lane < live ? sDb[lane] : 0.f;
                if (a.gate_bf16) {
                    ((uint16_t*)a.dg)[e] = f32_to_bf16(y);
                    ((uint16_t*)a.dbeta)[e] = f32_to_bf16(z);
                } else {
                    ((float*)a.dg)[e] = y;
                    ((float*)a.dbeta)[e] = z;
                }
            }
        }
    }
    const int t = t0 + i;
    if (t >= a.N) return;
#pragma unroll
    for (int j = 0; j < DT; ++j) {
        const long long e = (((long long)b * a.N + t) * a.Hk + hk) * DK + dk0 + 16 * j + g4;
        f32x4_t x = GROUP ? tq[GROUP ? j : 0] : Dq[j], y = GROUP ? tk[GROUP ? j : 0] : Dr[j];
        if (t >= len) x = y = zero;
        if (a.out_bf16) {
            store4((uint16_t*)a.dq + e, x);
            store4((uint16_t*)a.dk_ + e, y);
        } else {
            store4((float*)a.dq + e, x);
            store4((float*)a.dk_ + e, y);
        }
    }
}

template <class E, int DK>
void pick(int dv, DeltaKernels* o) {
    constexpr int NW = DK > 64 ? DK / 16 : 4;
    constexpr bool B16 = sizeof(typename E::st) == 2;
    if (dv <= 64) {  // as the forward's
        o->rlocal = delta_rchain_kernel<E, DK, 4, true, false>;
        o->rfull = delta_rchain_kernel<E, DK, 4, false, false>;
        if constexpr (B16) o->rfull2 = delta_rchain_kernel<E, DK, 4, false, true>;
    } else {
        o->rlocal = delta_rchain_kernel<E, DK, 8, true, false>;
        o->rfull = delta_rchain_kernel<E, DK, 8, false, false>;
        if constexpr (B16) o->rfull2 = delta_rchain_kernel<E, DK, 8, false, true>;
    }
    o->grad = delta_grad_kernel<E, DK, NW, false, false>;
    o->grad_group = delta_grad_kernel<E, DK, NW, true, false>;
    if constexpr (B16) {
        constexpr int NW2 = NW < 8 ? NW : 8;
        o->grad2 = delta_grad_kernel<E, DK, NW2, false, true>;
        o->grad_group2 = delta_grad_kernel<E, DK, NW2, true, true>;
        o->grad2_threads = 64 * NW2;
    }
    o->grad_threads = 64 * NW;
}

}  // namespace

void delta_bwd_kernels_get(bool bf16_in, int dk, int dv, DeltaKernels* o) {
    if (bf16_in) {
        switch (dk) {
            case 32: return pick<BF16, 32>(dv, o);
            case 64: return pick<BF16, 64>(dv, o);
            case 128: return pick<BF16, 128>(dv, o);
            case 256: return pick<BF16, 256>(dv, o);
        }
    } else {
        switch (dk) {
            case 16: return pick<F32, 16>(dv, o);
            case 32: return pick<F32, 32>(dv, o);
            case 64: return pick<F32, 64>(dv, o);
            case 128: return pick<F32, 128>(dv, o);
        }
    }
}

}  // namespace ret
