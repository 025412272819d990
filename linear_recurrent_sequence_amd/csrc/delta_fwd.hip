// The gated delta rule over a sequence: the per-chunk matrices, the chain over chunks, and the chain over segments.
#include "delta.h"

#include <type_traits>

namespace ret {

namespace {

typedef double f64;

// ---------------------------------------------------------------------------------------------------
// delta_prep: T = (I + A)^-1 and P of one chunk, for the H / Hk value heads that share a key head (the products K K^T
// and Q K^T are made once for them). One workgroup per (chunk, b, key head), or per value head while that many fit the
// card at once (24 workgroups of 3 heads: 20.5 us, as 72: 9.7); wave w owns rows 16w .. 16w+15.
//
// The decays are exp2 of differences of the running sum of g, kept in fp64 and scaled to base 2: a difference of two
// fp32 sums would lose the small decays that stand behind a large one. g below -200 counts as -200 (exp is 0 in fp32),
// so that g = -inf, which clears the state, leaves no inf - inf.
//
// The unit triangular inverse goes by 16 x 16 blocks: the four diagonal ones by forward substitution, a column per lane,
// then twice the block rule [[X, 0], [A, Y]]^-1 = [[X', 0], [-Y' A X', Y']] with fp32 MFMA.
//
// A workgroup's steps wait for each other (gates, inverse, products: eight barriers), so what counts is how many share a
// CU: the fp32 matrices lie where the rows were. 8192 chunks at d_k = 128: 114 us, 33 KB read and 26 KB written each,
// 4.2 TB/s; the copy rate would give 95.
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
__device__ __forceinline__ void write_mat(char* m, const float* X, int w, int lane, float scale = 1.f) {
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
        if constexpr (D::TPS == 2) D::mat_store(m, f, lane, scale * take(32 * s + g4), scale * take(32 * s + 16 + g4));
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

// acc = row tile w of X Y for lower triangular fp32 LDS matrices
__device__ __forceinline__ void tri_product(f32x4_t (&acc)[4], const float* X, const float* Y, int w, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i > w) continue;
        const f32x4_t x = tri_a(X, 16 * w, 16 * i, lane);
#pragma unroll
        for (int j = 0; j <= i; ++j) DOps<F32>::mma_ab(acc[j], x, tri_b(Y, 16 * i, 16 * j, lane));
    }
}

// As many workgroups on a CU as the LDS takes (their steps wait for each other): 2, 3 or 4.
template <class E, int DK, bool BWD>
__global__ __launch_bounds__(kThreads, (DK * sizeof(typename E::st) > 256 ? 2 : BWD ? 3 : 4))
void delta_prep_kernel(DeltaArgs a) {
    typedef typename E::st st;
    typedef DRows<E, DK, kThreads> Rows;
    typedef typename Rows::Tile Tile;
    typedef DOps<E> D;
    // the rows, then (their products are in registers) the matrices
    constexpr int kRows = 2 * kDeltaC * Tile::LD * (int)sizeof(st), kTri = 2 * kDeltaC * kTriLD * 4;
    __shared__ __align__(16) char pool[kRows > kTri ? kRows : kTri];
    st *sk = reinterpret_cast<st*>(pool), *sq = sk + kDeltaC * Tile::LD;
    float *sA = reinterpret_cast<float*>(pool), *sT = sA + kDeltaC * kTriLD;
    __shared__ f64 sG[kDeltaC];
    __shared__ float sB[kDeltaC], sF[kDeltaC];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15, g = lane >> 4;
    const int c = blockIdx.x, b = blockIdx.y / a.Hk, hk = blockIdx.y % a.Hk, rep = a.H / a.Hk;
    const int t0 = c * kDeltaC, live = min(kDeltaC, delta_len(a, b) - t0);
    if (live <= 0) return;  // no one reads this chunk
    float gv, bv;  // gates of the next head, asked for a head ahead
    auto gates = [&](int h) {
        const long long i = ((long long)b * a.N + t0 + min(lane, live - 1)) * a.H + h;
        gv = gate_at(a.g, i, a.gate_bf16);
        bv = gate_at(a.beta, i, a.gate_bf16);
    };
    const int r0 = blockIdx.z * (rep / gridDim.z), r1 = r0 + rep / gridDim.z;
    gates(hk * rep + r0);
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
    for (int r = r0; r < r1; ++r) {
        const int h = hk * rep + r;
        const long long unit = ((long long)b * a.H + h) * a.nchunks + c;
        if (w == 0) {
            const bool in = lane < live;
            f64 G = in ? (f64)(gv < -200.f ? -200.f : gv) * 1.4426950408889634 : 0.0;
#pragma unroll
            for (int m = 1; m < 64; m *= 2) {
                const f64 up = __shfl_up(G, m);
                if (lane >= m) G += up;
            }
            const float be = in ? bv : 0.f;
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
        gates(min(h + 1, hk * rep + r1 - 1));
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
            write_mat<E, true>(mats + 2 * kDeltaMatBytes, sT, w, lane);
            __syncthreads();
        }
        tri_inverse(sA, sT, w, lane);
        if constexpr (BWD) {
            write_mat<E, false>(mats, sT, w, lane);
            // Tr = (I + Ar)^-1 with beta along the rows, the gradients' solve: with A = L diag(beta) and Ar = diag(beta) L,
            // Tr = I - diag(beta) T L
#pragma unroll
            for (int j = 0; j < 4; ++j) tri_store(sA, 16 * w, 16 * j, lane, av[j]);
            __syncthreads();
            tri_product(av, sT, sA, w, lane);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4_t x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * w + 4 * g + i;
                    x[i] = (row == 16 * j + n16 ? 1.f : 0.f) - sB[row] * av[j][i];
                }
                tri_store(sT, 16 * w, 16 * j, lane, x);
            }
            __syncthreads();
            write_mat<E, true>(mats + kDeltaMatBytes, sT, w, lane);
        } else {
            // P T: row tile w through sA (its own rows only), and T with its rows scaled
#pragma unroll
            for (int j = 0; j < 4; ++j) tri_store(sA, 16 * w, 16 * j, lane, pv[j] * sB[16 * j + n16]);
            __syncthreads();
            tri_product(pv, sA, sT, w, lane);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) tri_store(sA, 16 * w, 16 * j, lane, pv[j]);
            __syncthreads();
            write_mat<E, false>(mats + kDeltaMatBytes, sA, w, lane);
            write_mat<E, false>(mats, sT, w, lane, sF[16 * w + n16]);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------------
// delta_chain: one segment of one head, 16 columns per wave, the state in accumulators. Columns are independent: what the
// waves of a workgroup share are the rows of K and Q and the matrices, which go through LDS once for all of them.
//   kFull: outputs of the input's type; kFullF32: BF16 input, F32 output. After the last segment the state.
//   kLocal / kLocalRaw (with Ts / with T): the segment's end state from zero (columns of V; segment 0 starts from state_in)
//     into segE, or its transition (columns of the identity, V = 0) into segM.
//   kStates (with T): the states entering the chunks and E, for the gradients; kStates2: both in two parts.
// A step: Y = K S and Q S, between their products the requests for everything the next chunk needs, into registers; R; O
// from Q S and P T; E; the state; then the registers go to LDS. K has two buffers, so that nothing but the first barrier
// of a chunk stands between its steps; the second one (after Q S) frees Q's and makes the matrices visible. A wave
// stages the columns of V it owns. Requests are never conditional: where two branches join, their registers would be
// waited for.
// Fragments of the next reduction step are read ahead of a step's products.
//
// At d_k = 256 with 8 waves a step of the full pass takes 6.4 us, 14300 cycles: K S and Q S 5050, R and P T R 1800, T R and
// the store 1300, the state 2700, barriers and staging 3500. MFMA issue is 6000, 1 MB of fragments out of LDS 8000. Rows
// read 8 bytes at a time cost 2300 more. Eight waves rather than four halve the staging per column; more workgroups per CU
// (128 registers) cost more in spills than they hid (local pass at d_k = 128 200 -> 222 us). Full pass, one workgroup per
// CU: 86 us for 16 chunks at d_k = 128, 284 us for 43 at 256; local pass 167 us for 32 at 256; states 221 for 32 at 256,
// of which 670 MB of states and E at the copy rate are 131.
// ---------------------------------------------------------------------------------------------------
enum { kFull = 0, kFullF32 = 1, kLocal = 2, kLocalRaw = 3, kStates = 4, kStates2 = 5 };
template <class E, int DK, int NW, int MODE>
__global__ __launch_bounds__(64 * NW) void delta_chain_kernel(DeltaArgs a) {
    typedef typename E::st st;
    typedef DOps<E> D;
    constexpr int NT = 64 * NW, COLS = 16 * NW;
    typedef DRows<E, DK, NT, typename D::template STile<DK>> Rows;
    typedef DRows<E, 16, 64, typename D::template Tile<COLS>> VRows;  // a wave's own columns
    typedef typename Rows::Tile Tile;
    typedef typename VRows::Tile VTile;
    typedef TriFrags<D::KS> F;
    constexpr bool LOCAL = MODE == kLocal || MODE == kLocalRaw, FULL = MODE == kFull || MODE == kFullF32;
    constexpr bool STATES = MODE == kStates || MODE == kStates2, RAW = MODE == kLocalRaw || STATES;
    constexpr bool OUT16 = MODE == kFull && sizeof(st) == 2;
    typedef typename std::conditional<OUT16, uint16_t, float>::type out_t;
    constexpr int DT = DK / 16, NS = F::NS, KN = DK / D::KS, TB = DT < 4 ? DT : 4;
    constexpr int PB = FULL ? F::BYTES : 16;
    __shared__ __align__(16) st sk[2][kDeltaC * Tile::LD];
    __shared__ __align__(16) st sq[FULL ? kDeltaC * Tile::LD : 16];
    __shared__ __align__(16) st sv[kDeltaC * VTile::LD];
    __shared__ __align__(16) char sm[F::BYTES];  // Ts (or T)
    __shared__ __align__(16) char sp[PB];        // P T
    __shared__ __align__(16) float sf[2][128];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15;
    const int g4 = 4 * (lane >> 4);
    const int nE = (a.dv + COLS - 1) / COLS;  // workgroups over d_v; a local pass has those of d_k behind them
    const DeltaBlock blk = delta_block(a, nE + (LOCAL ? (DK + COLS - 1) / COLS : 0));
    if (blk.seg >= a.nseg) return;
    const int bh = blk.bh, seg = blk.seg, b = bh / a.H, h = bh % a.H;
    const bool trans = LOCAL && blk.cb >= nE;
    const int width = trans ? DK : a.dv;
    const int col0 = (blk.cb - (trans ? nE : 0)) * COLS + 16 * w;
    const int hk = h / (a.H / a.Hk), len = delta_len(a, b);
    const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nchunks);
    const bool active = col0 < width;  // (a wave without columns computes on zeros)
    // no one asks for the last segment's end state, nor (segment 0's being the true one) for either end's transition
    if (LOCAL && (seg == a.nseg - 1 || (trans && seg == 0))) return;
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};

    f32x4_t S[DT];
    const float* sin = nullptr;
    if (!LOCAL) sin = a.nseg > 1 ? a.segE + ((long long)bh * a.nseg + seg) * DK * a.dv : nullptr;
    if (!LOCAL && a.nseg == 1) sin = a.state_in ? a.state_in + (long long)bh * DK * a.dv : nullptr;
    if (LOCAL && seg == 0 && !trans && a.state_in) sin = a.state_in + (long long)bh * DK * a.dv;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[t][i] = trans && D::srow(t, g4) + i == col0 + n16 ? 1.f : 0.f;
    if (sin && active) {
        const float* p = sin + col0 + n16;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[t][i] = p[(long long)(D::srow(t, g4) + i) * a.dv];
    }

    Rows rk, rq;
    VRows rv;
    DMat<F::BYTES, NT> rm;
    DMat<PB, NT> rp;
    float ff = 0.f;
    const float* fp;
    const st* kp = (const st*)a.k + (((long long)b * a.N) * a.Hk + hk) * DK;
    const st* qp = (const st*)a.q + (((long long)b * a.N) * a.Hk + hk) * DK;
    const st* vp = (const st*)a.v + (((long long)b * a.N) * a.H + h) * a.dv + col0;
    auto from = [&](int c) {  // the places of chunk c's operands
        const int live = min(kDeltaC, len - c * kDeltaC);
        const long long base = (long long)c * kDeltaC * a.Hk * DK;
        const char* mats = a.mats + ((long long)bh * a.nchunks + c) * a.nmats * kDeltaMatBytes;
        rk.from(kp + base, a.Hk * DK, live, DK, tid);
        rv.from(vp + (long long)c * kDeltaC * a.H * a.dv, a.H * a.dv, !trans && active ? live : 0, a.dv - col0, lane);
        if constexpr (FULL) rq.from(qp + base, a.Hk * DK, live, DK, tid);
        rm.from(mats, tid);
        if constexpr (FULL) rp.from(mats + kDeltaMatBytes, tid);
        fp = a.fac + ((long long)bh * a.nchunks + c) * kDeltaFac + (tid & 127);
    };
    constexpr int NK = Rows::NP, NV = VRows::NP, NM = DMat<F::BYTES, NT>::NP, NP = FULL ? DMat<PB, NT>::NP : 0;
    constexpr int NQ = FULL ? Rows::NP : 0, NL = NK + NV + NM + NP + NQ + 1;
    auto request = [&](int i) {
        if (i < NK) rk.get(i);
        else if (i < NK + NV) rv.get(i - NK);
        else if (i < NK + NV + NM) rm.get(i - NK - NV);
        else if (i < NK + NV + NM + 1) ff = *fp;
        else if (i < NK + NV + NM + 1 + NP) rp.get(i - NK - NV - NM - 1);
        else rq.get(i - NK - NV - NM - 1 - NP);
    };
    auto stage = [&](int p) {
        rk.store(sk[p], tid);
        rv.store(sv, lane, 16 * w);
        if (tid < 128) sf[p][tid] = ff;
        if constexpr (FULL) rq.store(sq, tid);
    };
    const int cend = min(c1, (len + kDeltaC - 1) / kDeltaC);  // chunks with live tokens
    if (c0 < cend) {
        from(c0);
#pragma unroll
        for (int i = 0; i < NL; ++i) request(i);
        stage(0);
    }
    for (int c = c0, p = 0; c < cend; ++c, p ^= 1) {
        __syncthreads();
        rm.store(sm);  // everyone is past the last chunk's products with them
        if constexpr (FULL) rp.store(sp);
        from(min(c + 1, cend - 1));
        const st* K = sk[p];
        if constexpr (STATES) {
            st* out = (st*)a.s0t + (((long long)bh * a.nchunks + c) * a.dv + col0) * DK;
            if (active)
#pragma unroll
                for (int t = 0; t < DT / D::TPS; ++t) {
                    D::blk_store(out, t, lane, &S[D::TPS * t]);
                    if constexpr (MODE == kStates2) D::blk_store_lo(out + a.state_lo, t, lane, &S[D::TPS * t]);
                }
        }
        // Y = K S and O^T = (Q S)^T: there a lane holds 4 columns of token 16 m + n16
        f32x4_t y[4], o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) y[m] = o[m] = zero;
        {
            typename D::Fa fk[2][4], fq[4];
            typename D::Fb fs[2];
#pragma unroll
            for (int m = 0; m < 4; ++m) fk[0][m] = Tile::rows(K, 16 * m, 0, lane);
            fs[0] = D::step(S, 0);
#pragma unroll
            for (int s = 0; s < KN; ++s) {
                if constexpr (FULL)
#pragma unroll
                    for (int m = 0; m < 4; ++m) fq[m] = Tile::rows(sq, 16 * m, s, lane);
                if (s + 1 < KN)
#pragma unroll
                    for (int m = 0; m < 4; ++m) fk[(s + 1) & 1][m] = Tile::rows(K, 16 * m, s + 1, lane);
#pragma unroll
                for (int i = NL * s / KN; i < NL * (s + 1) / KN; ++i) request(i);
                keep_order();
                D::template products<4>(y, 0, fk[s & 1], fs[s & 1]);
                if constexpr (FULL) {
                    keep_order();
#pragma unroll
                    for (int p = 0; p < 4; ++p)
#pragma unroll
                        for (int m = 0; m < 4; ++m) D::part_t(o[m], fq[m], fs[s & 1], p);
                }
                if (s + 1 < KN) fs[(s + 1) & 1] = D::step(S, s + 1);
                keep_order();
            }
        }
        // R = V - exp(G) Y
#pragma unroll
        for (int m = 0; m < 4; ++m)
            y[m] = VTile::acc(sv, m, 16 * w, lane) - *reinterpret_cast<const f32x4_t*>(sf[p] + 16 * m + g4) * y[m];
        typename D::Fb fr[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) fr[s] = D::step(y, s);
        __syncthreads();  // the matrices are there, and everyone is done with Q
        if constexpr (FULL) {
            typename D::Fm fpt[F::COUNT];
#pragma unroll
            for (int f = 0; f < F::COUNT; ++f) fpt[f] = D::mat_frag(sp, f, lane);
#pragma unroll
            for (int m = 0; m < 4; ++m) o[m] *= a.scale * sf[p][16 * m + n16];
            keep_order();
#pragma unroll
            for (int s = 0; s < NS; ++s) tri<E, false, true>(o, fpt, fr[s], s);
        }
        // E' = exp(G_C - G) beta T R
        f32x4_t u[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) u[m] = zero;
        typename D::Fm ft[F::COUNT];
#pragma unroll
        for (int f = 0; f < F::COUNT; ++f) ft[f] = D::mat_frag(sm, f, lane);
        if constexpr (FULL) {
            const int live = min(kDeltaC, len - c * kDeltaC);
            if (live < kDeltaC)  // padding
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (16 * m + n16 >= live) o[m] = zero;
            DOut out;
            out.init(a.o, ((long long)b * a.N + c * kDeltaC) * a.H + h, min(kDeltaC, a.N - c * kDeltaC), a.H, a.dv,
                     sizeof(out_t), col0 + g4, lane);
            if (active)
#pragma unroll
                for (int m = 0; m < 4; ++m) out.put((out_t*)nullptr, m, o[m]);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) tri<E, false, false>(u, ft, fr[s], s);
        keep_order();
        if constexpr (STATES) {
            st* out = (st*)a.et + (((long long)bh * a.nchunks + c) * a.dv + col0) * kDeltaC;
            if (active)
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    D::blk_store(out, s, lane, &u[D::TPS * s]);
                    if constexpr (MODE == kStates2) D::blk_store_lo(out + a.rows_lo, s, lane, &u[D::TPS * s]);
                }
        }
        if constexpr (RAW)
#pragma unroll
            for (int m = 0; m < 4; ++m) u[m] *= *reinterpret_cast<const f32x4_t*>(sf[p] + 64 + 16 * m + g4);
        // S = exp(G_C) S + K^T E'
        const float end = sf[p][63];
        typename D::Fb fu[NS];
        typename D::Fa fc[2][TB];
#pragma unroll
        for (int t = 0; t < TB; ++t) fc[0][t] = Tile::cols(K, 0, t, lane);
#pragma unroll
        for (int s = 0; s < NS; ++s) fu[s] = D::step(u, s);
#pragma unroll
        for (int i = 0; i < NS * DT / TB; ++i) {
            const int s = i % NS, t0 = i / NS * TB, s1 = (i + 1) % NS, t1 = (i + 1) / NS * TB;
            if (i + 1 < NS * DT / TB)
#pragma unroll
                for (int t = 0; t < TB; ++t) fc[(i + 1) & 1][t] = Tile::cols(K, s1 * D::KS, t1 + t, lane);
            keep_order();
            if (s == 0)
#pragma unroll
                for (int t = 0; t < TB; ++t) S[t0 + t] *= end;
            D::template products<TB>(S, t0, fc[i & 1], fu[s]);
            keep_order();
        }
        stage(p ^ 1);
    }
    if (!active) return;
    // outputs of padding chunks are zero
    if constexpr (FULL) {
        for (int c = max(c0, cend); c < c1; ++c) {
            DOut out;
            out.init(a.o, ((long long)b * a.N + c * kDeltaC) * a.H + h, min(kDeltaC, a.N - c * kDeltaC), a.H, a.dv,
                     sizeof(out_t), col0 + g4, lane);
#pragma unroll
            for (int m = 0; m < 4; ++m) out.put((out_t*)nullptr, m, zero);
        }
    }
    if constexpr (STATES) return;
    float* out = nullptr;
    if (LOCAL) out = (trans ? a.segM : a.segE) + ((long long)bh * a.nseg + seg) * DK * width;
    else if (seg == a.nseg - 1 && a.state_out) out = a.state_out + (long long)bh * DK * a.dv;
    if (!out) return;
    out += col0 + n16;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(long long)(D::srow(t, g4) + i) * width] = S[t][i];
}

// ---------------------------------------------------------------------------------------------------
// delta_scan: the states entering the segments. In: segE[s] = segment s's end state from zero (segment 0: its true end
// state), segM[s] its transition. Out: segE[s] = the state entering segment s, S_{s+1} = M_s S_s + E_s. One workgroup per
// (b, h, 32 columns); REV: the gradients' chain, D_{s-1} = M_s^T D_s + F_s over segF from the right. The waves share the
// rows of M; S goes round through LDS, transposed, so that it is written and read 16 bytes at a time. Each part of M is
// requested for the next segment as soon as its products have it (64 KB transitions 2.8 -> 2.3 us a segment). What is left
// is what a CU draws, 80 KB a segment at d_k = d_v = 128: two segments in flight, or S split once in LDS, change nothing.
// BF16 input: M and S split in two bf16 parts like the chain's operands.
// ---------------------------------------------------------------------------------------------------
// waves of a scan workgroup: 16 rows of the state each, 32 at d_k = 256 (the rows of M in flight take the registers)
template <int DK>
constexpr int scan_waves() { return DK / 16 <= 8 ? DK / 16 : 8; }
template <class E, int DK, bool REV>
__global__ __launch_bounds__(64 * scan_waves<DK>()) void delta_scan_kernel(DeltaArgs a) {
    typedef DOps<E> D;
    constexpr int NS = DK / D::KS, TPS = D::TPS, RT = DK / 16 / scan_waves<DK>(), CT = kScanCols / 16, LD = DK + 4;
    __shared__ __align__(16) float sS[2][kScanCols * LD];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15;
    const int g4 = 4 * (lane >> 4), bh = blockIdx.x, c0 = blockIdx.y * kScanCols;
    const long long sz = (long long)DK * a.dv;
    float* X = (REV ? a.segF : a.segE) + (long long)bh * a.nseg * sz;
    // this lane's places in a segment's state, by column tile: through a buffer resource, which drops the columns past d_v
    int at[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t)
        at[t] = c0 + 16 * t < a.dv ? ((16 * RT * w + g4) * a.dv + c0 + 16 * t + n16) * 4 : 0x40000000;
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
    auto seg = [&](int j) { return REV ? a.nseg - 1 - j : j; };  // the j-th segment on the way
    auto fetch_e = [&](int s) {                                  // its end state from zero
        const rsrc_t x = bytes_rsrc(X + s * sz, (int)sz * 4);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    e[r][t][i] = __uint_as_float(
                        __builtin_amdgcn_raw_buffer_load_b32(x, at[t], (16 * r + i) * a.dv * 4, 0));
    };
    auto fetch_m = [&](int s, int k) {  // part k of its transition
        const float* p = M + (long long)s * DK * DK;
#pragma unroll
        for (int r = 0; r < RT; ++r)
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
    fetch_e(seg(0));
    for (int j = 0;; ++j) {
        const int s = seg(j), next = seg(min(j + 1, a.nseg - 2));  // (the last one's are not needed)
        float* x = sS[j & 1];
        const rsrc_t out = bytes_rsrc(X + s * sz, (int)sz * 4);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                *reinterpret_cast<f32x4_t*>(x + (16 * t + n16) * LD + 16 * (RT * w + r) + g4) = S[r][t];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[r][t][i]), out, at[t],
                                                          (16 * r + i) * a.dv * 4, 0);
            }
        if (j == a.nseg - 1) return;
        __syncthreads();
        // from the state entering the first segment on; one without live tokens passes the state as it is
        const bool live = j == 0 || s * a.seg_chunks * kDeltaC < len;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < CT; ++t)
                if (live) S[r][t] = e[r][t];
        fetch_e(next);
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            if (j > 0 && live) {
                typename D::Fb fm[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) fm[r] = D::step(m[r][k], 0);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    f32x4_t y[TPS];
#pragma unroll
                    for (int p = 0; p < TPS; ++p)
                        y[p] = *reinterpret_cast<const f32x4_t*>(x + (16 * t + n16) * LD + D::KS * k + 16 * p + g4);
                    const typename D::Fb fy = D::step(y, 0);
#pragma unroll
                    for (int r = 0; r < RT; ++r) D::mma_mb(S[r][t], fm[r], fy);
                }
            }
            fetch_m(next, k);
        }
    }
}

template <class E, int DK, int NW>
void pick_waves(DeltaKernels* o) {
    *o = {};
    o->prep = delta_prep_kernel<E, DK, false>;
    o->bprep = delta_prep_kernel<E, DK, true>;
    o->local = delta_chain_kernel<E, DK, NW, kLocal>;
    o->blocal = delta_chain_kernel<E, DK, NW, kLocalRaw>;
    o->full = delta_chain_kernel<E, DK, NW, kFull>;
    o->full_f32 = delta_chain_kernel<E, DK, NW, sizeof(typename E::st) == 2 ? kFullF32 : kFull>;
    o->states = delta_chain_kernel<E, DK, NW, kStates>;
    if constexpr (sizeof(typename E::st) == 2) o->states2 = delta_chain_kernel<E, DK, NW, kStates2>;
    o->scan = delta_scan_kernel<E, DK, false>;
    o->rscan = delta_scan_kernel<E, DK, true>;
    o->scan_threads = 64 * scan_waves<DK>();
    o->cols = 16 * NW;
    o->threads = 64 * NW;
}
// Eight waves share the rows of K and Q; four where d_v would leave the others without columns.
template <class E, int DK>
void pick(int dv, DeltaKernels* o) {
    if (dv <= 64) pick_waves<E, DK, 4>(o);
    else pick_waves<E, DK, 8>(o);
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
