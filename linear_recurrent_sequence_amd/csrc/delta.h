// The gated delta rule (gfx950). Per batch b and value head h, with state S (d_k x d_v), decay alpha_t = exp(g_t) and
// write strength beta_t,
//     S'_t = alpha_t S_{t-1},  u_t = beta_t (v_t - S'_t^T k_t),  S_t = S'_t + k_t u_t^T,  o_t = scale S_t^T q_t.
// Over a chunk of C = 64 tokens with G_i = g_1 + .. + g_i and entering state S_0, write u_i = beta_i e_i. With
//     A_ij = exp(G_i - G_j) (k_i.k_j) beta_j (j < i),   T = (I + A)^-1,   P_ij = scale exp(G_i - G_j) (q_i.k_j) beta_j (j <= i)
// the e solve (I + A) E = R, so that everything is products of matrices:
//     Y = K S_0,  R = V - exp(G) Y,  E = T R,
//     O = scale exp(G) Q S_0 + P E,         S_C = exp(G_C) S_0 + K^T diag(exp(G_C - G) beta) E.
// T and P do not depend on the state: one kernel makes them for every chunk at once (delta_prep); the forward takes
// Ts = diag(exp(G_C - G) beta) T and P T, so that one operand, R, gives both outputs and the state's update. The rest is a
// chain over chunks with the state in MFMA accumulators. Columns of S are independent of each other, so each wave owns 16
// and no product of the chain leaves its wave: an accumulator tile (column in the lane, rows 4g .. 4g+3 of lane group g)
// is the other operand of the next product once the reduction index is taken in that order.
//
// Where B H d_v / 128 chains leave CUs idle, a sequence is cut into segments: a local pass gives each segment's end state
// from zero and its transition (the chain run on the columns of the identity), a scan over the segments the states that
// enter them, and the full pass starts all of them at once. The gradients do the same from the right with the transposed
// transitions. A chain step costs 3 to 10 us whatever the number of workgroups, and one or two of
// them fit a CU: the cut aims at one per CU, two where rows are short (two rounds of workgroups instead: 65536 tokens of 8
// heads 708 us, one 577 then).
//
// Precision. Products run on bf16 MFMA for bf16 inputs. What the kernels compute themselves (S, R, E, T, P) is split in
// two bf16 parts, x = hi + lo + e with |lo| <= 2^-8 |x| and |e| <= 2^-17 |x|, and multiplied as hi.hi + hi.lo + lo.hi (two
// products where the other side is an input, which is exact). A term of two split operands is off by 2^-15 of itself at
// worst: 2^-17 for each split and 2^-16 for the lo.lo left out; sums of them, whose errors are independent, come to 4e-6 to
// 6e-6 of outputs and states in the 2-norm, over any number of chunks (fp32 inputs: 2e-7 to 5e-7), where a single rounding of
// E and S would leave up to 2^-8 of each term. What leaves a chain for the gradients' per-chunk kernel (S_0, dS_C, E, dU) goes
// by the types of the gradients that come of it. All in bf16: rounded once, for the traffic's sake (at d_k = 256, d_v = 512
// S_0 and dS_C are 512 KB of a chunk's 830, and that kernel is bound by them); it costs dq, dk and dbeta an error of 0.002 to
// 0.003 in the 2-norm where their own rounding is 0.0017, dg up to 0.008. Outputs or gates in fp32: in two bf16 parts, errors
// below 1e-5, dg's 2e-5; 8192 tokens of 16 heads, 256 x 512, 1920 us for 1450, 4 x 4096 tokens, 128 x 128, 878 for 650. dv
// and the gradient of the state do not pass that way. F32 inputs run on the fp32 MFMA.
#pragma once

#include "chunk_bf16.h"
#include "delta_step.h"

namespace ret {

constexpr int kDeltaC = 64;    // tokens per chunk
constexpr int kScanCols = 32;  // columns of the state per workgroup of the segment scan

// Factors of a chunk (rows of 64): exp(G_i), exp(G_C - G_i) beta_i, exp(G_C - G_i), beta_i, then G_i log2(e) in fp64.
constexpr int kDeltaFac = 6 * kDeltaC;
// One triangular 64 x 64 matrix as operand fragments (two bf16 parts, or fp32), those with entries only: bytes reserved.
constexpr int kDeltaMatBytes = 12288;

struct DeltaArgs {
    const void *q, *k, *v;       // [B, N, Hk, dk], [B, N, H, dv]
    const void *g, *beta;        // [B, N, H]
    const int* lengths;          // [B] or null (N)
    const float* state_in;       // [B, H, dk, dv] or null (zeros)
    float* state_out;            // [B, H, dk, dv] or null
    void* o;                     // [B, N, H, dv]
    // workspace
    char* mats;                  // [B*H][nchunks][nmats][kDeltaMatBytes]: Ts, P T (gradients: T, Tr^T, Pr^T)
    float* fac;                  // [B*H][nchunks][kDeltaFac] per-token factors
    float* segE;                 // [B*H][nseg][dk][dv]: end states from zero, then the states entering the segments
    float* segM;                 // [B*H][nseg][dk][dk]: transitions
    // gradients
    float* segF;                 // [B*H][nseg][dk][dv]: state gradients of the segments, from their right ends
    // in the input type, as blocks of 16 columns (of d_v) x 16 TPS rows: [B*H][nchunks][dv/16][rows/(16 TPS)][1 KB]
    void *s0t, *ds1t;            // states entering and their gradients leaving the chunks (rows: d_k)
    void *et, *dut;              // E and dU (rows: the chunk's tokens)
    long long state_lo, rows_lo; // elements from a state's, or E's or dU's, high part to its low one, where there are two
    const void* dout;            // [B, N, H, dv]
    const float* dstate_out;     // [B, H, dk, dv] or null (zeros)
    float* dstate_in;            // or null
    void *dq, *dk_, *dv_, *dg, *dbeta;
    int B, N, H, Hk, dk, dv;
    int nchunks, nmats;
    int nseg, seg_chunks;        // segments per sequence and chunks per segment
    int out_bf16, gate_bf16;
    float scale;
};
typedef void (*delta_kernel_t)(DeltaArgs);
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Which segment and column block a workgroup has. Workgroups go round the 8 XCDs by their index; the column blocks of a
// segment read the same q, k and matrices, so they get indices 8 apart: one XCD, one L2, one after the other. Heads go
// before segments: an XCD gets its share of every segment, of which the first and the last are short in a local pass.
struct DeltaBlock {
    int bh, seg, cb;
};
__device__ __forceinline__ DeltaBlock delta_block(const DeltaArgs& a, int ncb) {
    const int i = blockIdx.x / 8, unit = i / ncb * 8 + blockIdx.x % 8;
    return {unit % (a.B * a.H), unit / (a.B * a.H), i % ncb};
}
// Live tokens of sequence b.
__device__ __forceinline__ int delta_len(const DeltaArgs& a, int b) {
    if (!a.lengths) return a.N;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.N ? a.N : n;
}

// Between LDS accesses of one wave whose lanes read what other lanes wrote: the accesses before are complete, and the
// compiler moves none across.
__device__ __forceinline__ void wave_fence() { __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The scheduler moves nothing across: keeps the reads of the next step's fragments ahead of this step's products.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// Fragments of a lower triangular 64 x 64 matrix by (row tile m, step s of KS columns), row after row, and those of the
// transpose of one.
template <int KS>
struct TriFrags {
    static constexpr int NS = kDeltaC / KS, COUNT = NS == 2 ? 6 : 10;
    static constexpr int BYTES = COUNT * (NS == 2 ? 2048 : 1024);  // bf16: two parts
    __host__ __device__ static constexpr bool lower(int m, int s) { return s * KS <= 16 * m + 15; }
    __host__ __device__ static constexpr bool upper(int m, int s) { return (s + 1) * KS > 16 * m; }
    __host__ __device__ static constexpr int at(int m, int s, bool up) {
        int n = 0;
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < NS; ++j) {
                if (i == m && j == s) return n;
                if (up ? upper(i, j) : lower(i, j)) ++n;
            }
        return n;
    }
};

// ---------------------------------------------------------------------------------------------------
// Operands. KS: reduction length of one step; TPS: accumulator tiles (16 rows) that make one step. In a step lane group g
// holds indices 4g..4g+3 of each tile. Fa: rows of an input matrix in LDS (exact). Fb: an operand made from accumulators.
// Fm: a 64 x 64 matrix fragment from the workspace. part(acc, a, b, p) adds the p-th product of a.b with accumulator rows
// along a's rows; part_t swaps the sides (accumulator rows along b's columns), so a lane holds 4 consecutive columns of
// one token.
// ---------------------------------------------------------------------------------------------------
template <class E>
struct DOps;

template <>
struct DOps<BF16> {
    typedef uint16_t st;
    static constexpr int KS = 32, TPS = 2;
    typedef bf16x8_t Fa;
    struct Fb {
        bf16x8_t hi, lo;
    };
    typedef Fb Fm;
    __device__ static __forceinline__ Fb split(f32x4_t a, f32x4_t b) {
        Fb f;
        f.hi = acc_pair(a, b);
        const u32x4_t u = __builtin_bit_cast(u32x4_t, f.hi);
        const f32x4_t ha = {__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u),
                            __uint_as_float(u[1] << 16), __uint_as_float(u[1] & 0xffff0000u)};
        const f32x4_t hb = {__uint_as_float(u[2] << 16), __uint_as_float(u[2] & 0xffff0000u),
                            __uint_as_float(u[3] << 16), __uint_as_float(u[3] & 0xffff0000u)};
        f.lo = acc_pair(a - ha, b - hb);
        return f;
    }
    // step s of a column of accumulator tiles
    template <int NT>
    __device__ static __forceinline__ Fb step(const f32x4_t (&x)[NT], int s) {
        return split(x[2 * s], x[2 * s + 1]);
    }
    __device__ static __forceinline__ void mfma1(f32x4_t& acc, bf16x8_t a, bf16x8_t b) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
    }
    // x[m0 + m] += a[m] b, the low parts first: no product right behind one of the same tile
    template <int MB, int NT>
    __device__ static __forceinline__ void products(f32x4_t (&x)[NT], int m0, const Fa (&a)[MB], const Fb& b) {
#pragma unroll
        for (int m = 0; m < MB; ++m) mfma1(x[m0 + m], a[m], b.lo);
#pragma unroll
        for (int m = 0; m < MB; ++m) mfma1(x[m0 + m], a[m], b.hi);
    }
    // The products of an operand pair, one by one (see tri): an input's rows (Fa), or a matrix (Fm), times b; _t: the
    // sides swapped, accumulator rows along b's columns
    __device__ static __forceinline__ void part(f32x4_t& acc, const Fa& a, const Fb& b, int p) {
        if (p < 2) mfma1(acc, a, p == 0 ? b.lo : b.hi);
    }
    __device__ static __forceinline__ void part_t(f32x4_t& acc, const Fa& a, const Fb& b, int p) {
        if (p < 2) mfma1(acc, p == 0 ? b.lo : b.hi, a);
    }
    __device__ static __forceinline__ void part(f32x4_t& acc, const Fm& a, const Fb& b, int p) {
        if (p < 3) mfma1(acc, p == 1 ? a.lo : a.hi, p == 0 ? b.lo : b.hi);
    }
    __device__ static __forceinline__ void part_t(f32x4_t& acc, const Fm& a, const Fb& b, int p) {
        if (p < 3) mfma1(acc, p == 0 ? b.lo : b.hi, p == 1 ? a.lo : a.hi);
    }
    // a matrix times an exact operand
    __device__ static __forceinline__ void part(f32x4_t& acc, const Fm& a, const bf16x8_t& b, int p) {
        if (p < 2) mfma1(acc, p == 0 ? a.lo : a.hi, b);
    }
    __device__ static __forceinline__ void mma_mb(f32x4_t& acc, const Fm& a, const Fb& b) {
#pragma unroll
        for (int p = 0; p < 3; ++p) part(acc, a, b, p);
    }
    // both sides exact
    __device__ static __forceinline__ void mma_aa(f32x4_t& acc, Fa a, Fa b) { mfma1(acc, a, b); }
    // accumulator-ordered values that are exact in bf16
    typedef bf16x8_t Fx;
    template <int NT>
    __device__ static __forceinline__ Fx step_exact(const f32x4_t (&x)[NT], int s) {
        return acc_pair(x[2 * s], x[2 * s + 1]);
    }
    // fragment f of a workspace matrix
    __device__ static __forceinline__ Fm mat_frag(const char* m, int f, int lane) {
        const u32x4_t* p = reinterpret_cast<const u32x4_t*>(m) + f * 128 + lane;
        return {__builtin_bit_cast(bf16x8_t, p[0]), __builtin_bit_cast(bf16x8_t, p[64])};
    }
    // writes the fragment of x: a: the step's first 4 values of this lane, b: its last 4
    __device__ static __forceinline__ void mat_store(char* m, int f, int lane, f32x4_t a, f32x4_t b) {
        const Fb x = split(a, b);
        u32x4_t* p = reinterpret_cast<u32x4_t*>(m) + f * 128 + lane;
        p[0] = __builtin_bit_cast(u32x4_t, x.hi);
        p[64] = __builtin_bit_cast(u32x4_t, x.lo);
    }
    // A block of 16 TPS rows x 16 columns in accumulators, 16 bytes a lane and 1 KB together (block i of p), and the way
    // of a lane's part to row n16 of an LDS tile (the block transposed: its rows become columns c0 ..)
    __device__ static __forceinline__ void blk_store(st* p, int i, int lane, const f32x4_t* x) {
        *reinterpret_cast<bf16x8_t*>(p + (i * 64 + lane) * 8) = acc_pair(x[0], x[1]);
    }
    // the low part of the same block
    __device__ static __forceinline__ void blk_store_lo(st* p, int i, int lane, const f32x4_t* x) {
        *reinterpret_cast<bf16x8_t*>(p + (i * 64 + lane) * 8) = split(x[0], x[1]).lo;
    }
    template <class Tile>
    __device__ static __forceinline__ void blk_lds(st* lds, int row, int c0, int g4, u32x4_t x) {
        *reinterpret_cast<uint2*>(lds + Tile::off(row, c0 + g4)) = make_uint2(x[0], x[1]);
        *reinterpret_cast<uint2*>(lds + Tile::off(row, c0 + 16 + g4)) = make_uint2(x[2], x[3]);
    }
    // The rows of the state that lane group g holds of tile t: a step's two tiles together are 8 consecutive ones, so that
    // rows of K and Q are read 16 bytes at a time (reads of 8 run at half the LDS's rate)
    __device__ static __forceinline__ int srow(int t, int g4) { return 32 * (t / 2) + 4 * (t % 2) + 2 * g4; }
    template <class T>
    __device__ static __forceinline__ void blk_lds_s(st* lds, int row, int c0, int g4, u32x4_t x) {
        *reinterpret_cast<u32x4_t*>(lds + T::off(row, c0 + 2 * g4)) = x;
    }
    // LDS tile [tokens][W] for the chains: rows(s): step s in the state's order; cols(t): the columns of the state's tile t.
    // Rows 16 banks apart, their 16-byte pieces swapped by row / 4: 8 rows' pieces, and the 4 rows x 4 pieces of a
    // transposing read, lie in different banks.
    template <int W>
    struct STile {
        static constexpr int LD = W + 32;
        __device__ static __forceinline__ int off(int r, int c) { return r * LD + (c ^ (((r >> 2) & 3) << 3)); }
        __device__ static __forceinline__ Fa rows(const st* X, int r0, int s, int lane) {
            return __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(
                                                    X + r0 * LD + 32 * s + off(lane & 15, 8 * (lane >> 4))));
        }
        __device__ static __forceinline__ Fa cols(const st* X, int k0, int t, int lane) {
            typedef __attribute__((address_space(3))) bf16x4_t lds_bf16x4_t;
            st* p = const_cast<st*>(X) + k0 * LD + 32 * (t / 2) + 4 * (t % 2) +
                    off(4 * (lane >> 4) + ((lane >> 2) & 3), 8 * (lane & 3));
            const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t*)p));
            const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t*)(p + 16 * LD)));
            return __builtin_bit_cast(bf16x8_t, make_uint4(lo.x, lo.y, hi.x, hi.y));
        }
    };
    // LDS tile [rows][W], read by rows and transposed
    template <int W>
    struct Tile {
        static constexpr int LD = Swz<W>::LD;
        __device__ static __forceinline__ int off(int r, int c) { return Swz<W>::off(r, c); }
        __device__ static __forceinline__ Fa rows(const st* X, int r0, int k0, int lane) {
            return frag_ps<W>(X, r0, k0, Swz<W>::lane_p(lane));
        }
        __device__ static __forceinline__ Fa cols(const st* X, int k0, int n0, int lane) {
            return frag_trps<W>(X, k0, n0, Swz<W>::lane_trp(lane));
        }
        // rows 16m .. 16m+15, columns n0 .. n0+15 in accumulator order
        __device__ static __forceinline__ f32x4_t acc(const st* X, int m, int n0, int lane) {
            typedef __attribute__((address_space(3))) bf16x4_t lds_bf16x4_t;
            st* p = const_cast<st*>(X) + 16 * m * LD + n0 + Swz<W>::lane_trp(lane);
            const uint2 u = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t*)p));
            return f32x4_t{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u)};
        }
    };
};

template <>
struct DOps<F32> {
    typedef float st;
    static constexpr int KS = 16, TPS = 1;
    typedef f32x4_t Fa;
    typedef f32x4_t Fb;
    typedef f32x4_t Fm;
    template <int NT>
    __device__ static __forceinline__ Fb step(const f32x4_t (&x)[NT], int s) {
        return x[s];
    }
    __device__ static __forceinline__ void mma_ab(f32x4_t& acc, const Fa& a, const Fb& b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], acc, 0, 0, 0);
    }
    template <int MB, int NT>
    __device__ static __forceinline__ void products(f32x4_t (&x)[NT], int m0, const Fa (&a)[MB], const Fb& b) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < MB; ++m)
                x[m0 + m] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[m][i], b[i], x[m0 + m], 0, 0, 0);
    }
    __device__ static __forceinline__ void part(f32x4_t& acc, const Fa& a, const Fb& b, int p) {
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[p], b[p], acc, 0, 0, 0);
    }
    __device__ static __forceinline__ void part_t(f32x4_t& acc, const Fa& a, const Fb& b, int p) { part(acc, b, a, p); }
    __device__ static __forceinline__ void mma_mb(f32x4_t& acc, const Fm& a, const Fb& b) { mma_ab(acc, a, b); }
    __device__ static __forceinline__ void mma_aa(f32x4_t& acc, const Fa& a, const Fa& b) { mma_ab(acc, a, b); }
    __device__ static __forceinline__ void blk_store(st* p, int i, int lane, const f32x4_t* x) {
        *reinterpret_cast<f32x4_t*>(p + (i * 64 + lane) * 4) = x[0];
    }
    template <class Tile>
    __device__ static __forceinline__ void blk_lds(st* lds, int row, int c0, int g4, u32x4_t x) {
        *reinterpret_cast<u32x4_t*>(lds + Tile::off(row, c0 + g4)) = x;
    }
    typedef f32x4_t Fx;
    template <int NT>
    __device__ static __forceinline__ Fx step_exact(const f32x4_t (&x)[NT], int s) {
        return x[s];
    }
    __device__ static __forceinline__ Fm mat_frag(const char* m, int f, int lane) {
        return reinterpret_cast<const f32x4_t*>(m)[f * 64 + lane];
    }
    __device__ static __forceinline__ void mat_store(char* m, int f, int lane, f32x4_t a) {
        reinterpret_cast<f32x4_t*>(m)[f * 64 + lane] = a;
    }
    template <int W>
    struct Tile {
        static constexpr int LD = W + 4;
        __device__ static __forceinline__ int off(int r, int c) { return r * LD + c; }
        __device__ static __forceinline__ Fa rows(const st* X, int r0, int k0, int lane) {
            return *reinterpret_cast<const f32x4_t*>(X + (r0 + (lane & 15)) * LD + k0 + 4 * (lane >> 4));
        }
        __device__ static __forceinline__ Fa cols(const st* X, int k0, int n0, int lane) {
            const st* p = X + (k0 + 4 * (lane >> 4)) * LD + n0 + (lane & 15);
            return f32x4_t{p[0], p[LD], p[2 * LD], p[3 * LD]};
        }
        __device__ static __forceinline__ f32x4_t acc(const st* X, int m, int n0, int lane) {
            return cols(X, 16 * m, n0, lane);
        }
    };
    __device__ static __forceinline__ int srow(int t, int g4) { return 16 * t + g4; }
    template <class T>
    __device__ static __forceinline__ void blk_lds_s(st* lds, int row, int c0, int g4, u32x4_t x) {
        blk_lds<T>(lds, row, c0, g4, x);
    }
    template <int W>
    struct STile {
        typedef Tile<W> T;
        static constexpr int LD = T::LD;
        __device__ static __forceinline__ int off(int r, int c) { return T::off(r, c); }
        __device__ static __forceinline__ Fa rows(const st* X, int r0, int s, int lane) { return T::rows(X, r0, 16 * s, lane); }
        __device__ static __forceinline__ Fa cols(const st* X, int k0, int t, int lane) { return T::cols(X, k0, 16 * t, lane); }
    };
};

// Products of the four row tiles with step s of b; tri: of a triangular matrix (f: its fragments; UP: a transpose's), the
// tiles with entries in that step. SWAP: accumulator rows along b's columns. The parts of a pair go round the tiles, so
// that no product stands right behind one into the same accumulators.
template <class E, bool UP, bool SWAP, class A, class B, int N>
__device__ __forceinline__ void tri(f32x4_t (&x)[4], const A (&f)[N], const B& b, int s) {
    typedef DOps<E> D;
    typedef TriFrags<D::KS> F;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (UP ? F::upper(m, s) : F::lower(m, s)) {
                if constexpr (SWAP) D::part_t(x[m], f[F::at(m, s, UP)], b, p);
                else D::part(x[m], f[F::at(m, s, UP)], b, p);
            }
}

// 64 rows of W elements of one head moved as 16-byte segments by NT threads: rows past the live ones read as zeros (the
// buffer resource ends with the last live row), and so do columns past `cols`. Tile column `at` receives column 0. The
// requests (get) go out one by one, so that a kernel can spread them over its products.
template <class E, int W, int NT, class T = typename DOps<E>::template Tile<W>>
struct DRows {
    typedef typename E::st st;
    static constexpr int EPS = 16 / sizeof(st), SPR = W / EPS, RP = NT / SPR, NP = (kDeltaC + RP - 1) / RP;
    typedef T Tile;
    u32x4_t x[NP];
    rsrc_t r;
    int off, step;
    // p: the head's row of the chunk's first token; stride: elements between tokens; live: rows to read (may be <= 0)
    __device__ __forceinline__ void from(const st* p, int stride, int live, int cols, int tid) {
        r = bytes_rsrc(p, live > 0 ? ((live - 1) * stride + cols) * (int)sizeof(st) : 0);
        const int row = tid / SPR, c = tid % SPR * EPS;
        off = c < cols ? (row * stride + c) * (int)sizeof(st) : 0x40000000;
        step = RP * stride * (int)sizeof(st);
    }
    __device__ __forceinline__ void get(int i) { x[i] = buf_load16(r, off, i * step); }
    __device__ __forceinline__ void load(const st* p, int stride, int live, int cols, int tid) {
        from(p, stride, live, cols, tid);
#pragma unroll
        for (int i = 0; i < NP; ++i) get(i);
    }
    __device__ __forceinline__ void store(st* lds, int tid, int at = 0) const {
        const int row = tid / SPR, c = at + tid % SPR * EPS;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (NP * RP == kDeltaC || row + i * RP < kDeltaC)
                *reinterpret_cast<u32x4_t*>(lds + Tile::off(row + i * RP, c)) = x[i];
    }
};

// `BYTES` bytes of a workspace matrix (a multiple of 16) moved to LDS by NT threads, as they are.
template <int BYTES, int NT>
struct DMat {
    static constexpr int N = BYTES / 16, NP = (N + NT - 1) / NT;
    u32x4_t x[NP];
    const u32x4_t* p;
    int tid;
    __device__ __forceinline__ void from(const char* m, int t) {
        p = reinterpret_cast<const u32x4_t*>(m);
        tid = t;
    }
    __device__ __forceinline__ void get(int i) { x[i] = p[tid + i * NT < N ? tid + i * NT : N - 1]; }
    __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (N % NT == 0 || tid + i * NT < N) reinterpret_cast<u32x4_t*>(lds)[tid + i * NT] = x[i];
    }
};

// A chunk's outputs, 4 consecutive columns of one token per lane (tile m: token 16 m + lane % 16), through a buffer
// resource that ends with the sequence's last row: rows past it are dropped.
struct DOut {
    rsrc_t r;
    int off, stride;  // bytes: this lane's place, and one token
    __device__ __forceinline__ void init(void* base, long long row0, int rows, int H, int dv, int esz, int col, int lane) {
        stride = H * dv * esz;
        r = bytes_rsrc((char*)base + row0 * dv * esz, (rows - 1) * stride + dv * esz);
        off = (lane & 15) * stride + col * esz;
    }
    __device__ __forceinline__ void put(uint16_t*, int m, f32x4_t x) const {
        __builtin_amdgcn_raw_buffer_store_b64(
            __builtin_bit_cast(u32x2_t, make_uint2(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]))), r, off,
            16 * m * stride, 0);
    }
    __device__ __forceinline__ void put(float*, int m, f32x4_t x) const {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, x), r, off, 16 * m * stride, 0);
    }
};

// ---- kernel selection ----
struct DeltaKernels {
    delta_kernel_t prep, local, full, full_f32, scan;  // full_f32: F32 output
    delta_kernel_t bprep, blocal, states, rlocal, rscan, rfull, grad, grad_group;  // gradients (grad_group: H > Hk)
    delta_kernel_t states2, rfull2, grad2, grad_group2;  // the same with what the chains store in two parts (BF16 input)
    int cols, threads; // columns of d_v (or of a transition) and threads per workgroup of the chains
    int grad_threads, grad2_threads, scan_threads;
};
// d_k in {32, 64, 128, 256} for bf16 and {16, 32, 64, 128} for fp32; false otherwise.
bool delta_kernels_get(bool bf16_in, int dk, int dv, DeltaKernels* out);
// The gradients' own kernels (rlocal, rfull, grad, their two-part forms and the threads) of a supported shape.
void delta_bwd_kernels_get(bool bf16_in, int dk, int dv, DeltaKernels* out);

}  // namespace ret
