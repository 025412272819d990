// Selective scan: arguments and the device code that its kernels share.
//
// Per batch b, channel d and state s, group g = d / (D / G):
//     dt_t = softplus(delta_t + bias),  a_t = exp(dt_t A),  h_t = a_t h_{t-1} + dt_t u_t B_t[g],
//     y_t = (sum_s C_t[g] h_t + D u_t) silu(z_t)
//
// Layout of every sequence kernel: a wave holds 16 channels, four neighbouring lanes a channel, each with SL = S / 4 of its
// states, and T tokens at a time: 256 / S of them, at most 16, so that the T SL decays a_t of a lane are at most 64 registers.
// The values per token and channel (u, delta, z, y) lie one in a lane: lane q of a channel's four holds tokens 4 i + q, and
// sums over the states leave each token's in that lane. B and C of a wave's tokens are staged in its own part of the LDS, in
// fp32.
#pragma once

#include "kernels.h"

namespace ret {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kScanCh = 16;  // channels of a wave

template <int S_, int T_, int NW_>
struct ScanTile {
    static constexpr int S = S_;
    static constexpr int SL = S / 4;   // states a lane
    static constexpr int T = T_;       // tokens of a wave's block
    static constexpr int TL = T / 4;   // of which a lane holds the scalars
    static constexpr int NW = NW_;     // waves of a workgroup, neighbouring blocks of tokens
    static constexpr int CH = NW * T;  // tokens of a workgroup's chunk
    static constexpr int THREADS = 64 * NW;
    static_assert(T % 4 == 0 && T * S <= 256, "a wave stages its block's B and C four values a lane");
};
template <int S>
struct ScanShape : ScanTile<S, S < 16 ? 16 : 256 / S, S <= 16 ? 8 : 4> {};

struct ScanArgs {
    const void *u, *dt, *z, *b, *c;      // u, dt [B, N, D]; z rows of ldz; b, c rows of ldb, ldc with [G, S] in each
    const float *A, *skip, *bias;        // [D, S]; [D] or null
    const int32_t* lengths;              // [B] or null
    const float* state_in;               // [B, D, S] or null
    float* state_out;                    // [B, D, S] or null
    void* y;                             // [B, N, D]
    float *seg_h, *seg_dt;               // [B][nseg][D][S], [B][nseg][D]
    long long ldz, ldb, ldc;
    int B, N, D, G, nseg, seg_tokens;
    int cblocks;                         // blocks of a workgroup's channels
    int softplus, bc_vec;                // bc_vec: b and c may be read four values at a time
    int deal;                            // of workgroups to the XCDs: ScanDeal
};

// Workgroup number -> position, so that the workgroups of neighbouring positions run on one XCD (they are dealt to the 8 in
// turn): n is a multiple of 8.
__device__ __forceinline__ long long xcd_order(long long id, long long n) { return (id & 7) * (n >> 3) + (id >> 3); }

// log(1 + exp(x)) and its derivative. e = exp(-|x|) on the hardware 2^x: its argument's rounding makes it |x| units of 2^-24.
// log(1 + e) = 2 atanh(r), r = e / (2 + e) <= 1/3: a polynomial of degree 4 in r^2 for atanh(r) / r, fitted for the least
// largest error on [0, 1/9], which is 4e-9. A NaN comes through e; minus infinity gives 0.
__device__ __forceinline__ void softplus(float x, float* value, float* slope) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(x));
    const float r = e * __builtin_amdgcn_rcpf(2.f + e), w = r * r;
    float p = fmaf(w, 0.14095773673944728f, 0.13978833207656793f);
    p = fmaf(w, p, 0.2001255710881801f);
    p = fmaf(w, p, 0.33333155074914933f);
    p = fmaf(w, p, 1.f);
    *value = fmaf(2.f * r, p, x > 0.f ? x : 0.f);
    const float s = __builtin_amdgcn_rcpf(1.f + e);
    *slope = x > 0.f ? s : e * s;
}

// A in units of log2(e), so that a_t = 2^(dt_t A). An infinite A (a state without memory) becomes the largest number: steps of
// length 0 then still leave the state.
__device__ __forceinline__ float decay_rate(float A) {
    const float r = A * kLog2e;
    return r < -3.4e38f ? -3.4e38f : r > 3.4e38f ? 3.4e38f : r;
}

// The value that lane K of every four holds. In the form that the compiler can make a part of the instruction that uses it.
template <int K>
__device__ __forceinline__ float quad_of(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), K * 0x55, 0xf, 0xf, true));
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

// Values as they lie in memory, so that a load is not waited for before its values are used. off: bytes.
template <class E>
struct Raw;
template <>
struct Raw<BF16> {
    typedef uint32_t one;  // a bf16 value in the low half
    typedef uint2 four;
    static __device__ __forceinline__ one get(const char* p, uint32_t off) { return *(const uint16_t*)(p + off); }
    static __device__ __forceinline__ float value(one r) { return __uint_as_float(r << 16); }
    static __device__ __forceinline__ four get4(const char* p, uint32_t off, bool vec) {
        const uint16_t* q = (const uint16_t*)(p + off);
        if (vec) return *reinterpret_cast<const uint2*>(q);
        return make_uint2(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16);
    }
    static __device__ __forceinline__ f32x4_t values(four w) {
        return f32x4_t{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u)};
    }
};
template <>
struct Raw<F32> {
    typedef float one;
    typedef f32x4_t four;
    static __device__ __forceinline__ one get(const char* p, uint32_t off) { return *(const float*)(p + off); }
    static __device__ __forceinline__ float value(one r) { return r; }
    static __device__ __forceinline__ four get4(const char* p, uint32_t off, bool vec) {
        const float* q = (const float*)(p + off);
        if (vec) return *reinterpret_cast<const f32x4_t*>(q);
        return f32x4_t{q[0], q[1], q[2], q[3]};
    }
    static __device__ __forceinline__ f32x4_t values(four w) { return w; }
};

// Where a wave's block of tokens lies in an array of rows: one address for the wave and 24-bit products for its lanes, so that
// rows of at most kScanMaxLd elements have 32-bit offsets. Tokens past the end are read as the last one; whoever uses them
// leaves those from n on out.
constexpr int64_t kScanMaxLd = (1 << 22) - 1;
struct ScanRows {
    long long row;  // of the block's first token
    int last;       // the last token of the block that there is
    __device__ __forceinline__ ScanRows(long long row0, int t0, int N) {
        const int t = t0 < N ? t0 : N - 1;
        row = row0 + t;
        last = N - 1 - t;
    }
    template <class E>
    __device__ __forceinline__ const char* base(const void* p, long long ld) const {
        return (const char*)p + row * ld * (int)sizeof(typename E::st);
    }
    template <class E>
    __device__ __forceinline__ uint32_t off(int k, long long ld, int col) const {
        const uint32_t e = sizeof(typename E::st);
        return __umul24(k < last ? k : last, (uint32_t)ld * e) + col * e;
    }
};
// The lane's tokens 4 i + q of channel d.
template <class E, class P>
__device__ __forceinline__ void load_scalars(const ScanRows& r, const void* p, long long ld, int q, int d,
                                             typename Raw<E>::one (&f)[P::TL]) {
    const char* base = r.base<E>(p, ld);
#pragma unroll
    for (int i = 0; i < P::TL; ++i) f[i] = Raw<E>::get(base, r.off<E>(4 * i + q, ld, d));
}
// Outputs of the lane's tokens 4 i + q of channel d, those before `end` tokens of the block.
template <class O, class P>
__device__ __forceinline__ void store_scalars(void* p, long long row, long long D, int end, int q, int d,
                                              const float (&f)[P::TL]) {
    typedef typename O::st st;
    char* base = (char*)p + row * D * (int)sizeof(st);
#pragma unroll
    for (int i = 0; i < P::TL; ++i)
        if (4 * i + q < end)
            store_out((st*)(base + (__umul24(4 * i + q, (uint32_t)D * (uint32_t)sizeof(st)) + d * (uint32_t)sizeof(st))), f[i]);
}
// The lane's four values of the block's [T][S] of b or c ...
template <class E, class P>
__device__ __forceinline__ typename Raw<E>::four load_bc(const ScanRows& r, const void* p, long long ld, int g, int lane,
                                                         bool vec) {
    return Raw<E>::get4(r.base<E>(p, ld), r.off<E>(4 * lane / P::S, ld, g * P::S + 4 * lane % P::S), vec);
}
// ... to LDS in fp32, zeros from token n on.
template <class E, class P>
__device__ __forceinline__ void put_bc(float* lds, typename Raw<E>::four r, int n, int t0, int lane) {
    const f32x4_t v = Raw<E>::values(r);
    if (4 * lane < P::T * P::S)
        *reinterpret_cast<f32x4_t*>(lds + 4 * lane) = t0 + 4 * lane / P::S < n ? v : f32x4_t{0.f, 0.f, 0.f, 0.f};
}

// Keeps a wave's LDS accesses on either side of it in order: they are carried out in the order they are issued.
__device__ __forceinline__ void lds_order() { __asm__ volatile("" ::: "memory"); }

// A wave's block of tokens: loaded one block ahead, then steps().
template <class E, int S>
struct ScanBlock {
    typedef ScanShape<S> P;
    typedef Raw<E> R;
    typename R::one u[P::TL], dt[P::TL], z[P::TL];
    typename R::four b, c;
    __device__ __forceinline__ void load(const ScanArgs& a, long long row0, int t0, int q, int lane, int d, int g, bool out) {
        const ScanRows r(row0, t0, a.N);
        load_scalars<E, P>(r, a.u, a.D, q, d, u);
        load_scalars<E, P>(r, a.dt, a.D, q, d, dt);
        if (out && a.z) load_scalars<E, P>(r, a.z, a.ldz, q, d, z);
        b = load_bc<E, P>(r, a.b, a.ldb, g, lane, a.bc_vec);
        if (out) c = load_bc<E, P>(r, a.c, a.ldc, g, lane, a.bc_vec);
    }
    // The lane's step lengths, and their products with u; 0 from token n on: such a token changes nothing.
    __device__ __forceinline__ void steps(const ScanArgs& a, float bias, int n, int t0, int q, float (&step)[P::TL],
                                          float (&us)[P::TL], float (&du)[P::TL]) const {
        float s;
#pragma unroll
        for (int i = 0; i < P::TL; ++i) {
            us[i] = R::value(u[i]);
            step[i] = R::value(dt[i]) + bias;
        }
        if (a.softplus)
#pragma unroll
            for (int i = 0; i < P::TL; ++i) softplus(step[i], &step[i], &s);
        if (t0 + P::T > n)
#pragma unroll
            for (int i = 0; i < P::TL; ++i)
                if (t0 + 4 * i + q >= n) step[i] = us[i] = 0.f;
#pragma unroll
        for (int i = 0; i < P::TL; ++i) du[i] = step[i] * us[i];
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
// GT tokens of a wave's [T][S] in LDS from token k: the lane's states. Read one group ahead of its use, with an lds_order()
// after each group: the compiler would otherwise ask for all of a block at once and run out of registers.
template <int S, int GT>
__device__ __forceinline__ void lds_group(const float* p, int k, int q, float (&f)[GT][S / 4]) {
#pragma unroll
    for (int e = 0; e < GT; ++e) lds_vec<S / 4>(p + (k + e) * S + q * (S / 4), f[e]);
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

template <int SL>
__device__ __forceinline__ void state_put(float* p, const float (&f)[SL]) {
#pragma unroll
    for (int j = 0; j < SL; ++j) p[j] = f[j];
}

struct ScanPos {
    int cb, seg, b;
};
// Workgroup -> unit of `units` (blocks of channels, or several) and number of its segment and sequence, by the XCDs:
enum ScanDeal {
    kDealRanges,  // a range of all, the units of a segment first
    kDealUnits,   // a range of the units (a multiple of 8) with all their segments and sequences
    kDealSegs,    // every eighth segment with all its units; an odd number a sequence, so that they begin on different XCDs
};
__host__ __device__ __forceinline__ int deal_segs(int deal, int nseg) { return deal == kDealSegs ? nseg | 1 : nseg; }
__device__ __forceinline__ long long scan_order(int units, int deal, int* unit) {
    const long long id = blockIdx.x, j = id >> 3;
    if (deal == kDealUnits) {
        const int u8 = units >> 3;
        *unit = (int)(id & 7) * u8 + (int)(j % u8);
        return j / u8;
    }
    if (deal == kDealSegs) {
        *unit = (int)(j % units);
        return j / units * 8 + (id & 7);
    }
    const long long o = xcd_order(id, gridDim.x);
    *unit = (int)(o % units);
    return o / units;
}
__device__ __forceinline__ bool scan_pos(const ScanArgs& a, ScanPos* p) {
    const long long rest = scan_order(a.cblocks, a.deal, &p->cb);
    const int segs = deal_segs(a.deal, a.nseg);
    p->seg = (int)(rest % segs);
    p->b = (int)(rest / segs);
    return p->b < a.B && p->seg < a.nseg;
}

typedef void (*scan_kernel_t)(ScanArgs);
struct ScanKernels {
    scan_kernel_t local, join, walk, chunks;  // local and walk: 4 waves a workgroup, each its own block of 16 channels
    int block, chunk, threads;                // tokens of a wave's block; tokens of a chunk and threads of chunks
};
constexpr int kWalkWaves = 4;
bool scan_kernels_get(bool bf16_in, bool bf16_out, int S, ScanKernels* o);

}  // namespace ret
