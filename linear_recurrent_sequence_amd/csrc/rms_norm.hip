// Root-mean-square norm over rows of D values, forward and gradients.
//
//   forward:  s = x + residual (rounded to x's dtype), xh = s rstd, rstd = 1 / sqrt(mean(s^2) + eps), y = w xh
//             in 8 bits: scale = max |y| / 448 over the row or a group of its columns, y8 = e4m3(y / scale)
//   gradient: a = w dy, dx = rstd (a - xh mean(a xh)) + dsum, dw = sum_rows dy xh
//
// A row is held in the registers of L lanes (4 to 16 values each), as in layer_norm.hip, so that each tensor is read once;
// the maxima of |y| come from the same registers. The weight's gradient leaves one partial row per workgroup, added up in a
// fixed order by a second kernel. Bound by HBM: 8192 x 4096 bf16 with residual, in bf16 and in 8 bits with a scale for 128
// columns, 62.5 us (4.8 TB/s, a large copy reaches 5.1), in fp32 112; its gradients 56 us with the sums' 5, in fp32 109; 128
// rows 5.2 us, of which a launch is most. Rows of 4098 columns, value by value: 244 and 222 us.
#include "host.h"
#include "rows.h"

namespace ret {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite
// Mean squares below are formed again of larger values: a square of less than 2^-126 is rounded by up to 2^-150, which is 2^-30
// of this.
constexpr float kMinSquare = 0x1p-120f;

struct RmsArgs {
    const void *x, *res;  // [rows][D], one dtype
    void *sum, *y;        // each or null
    uint8_t* y8;          // [rows][D] e4m3, or null
    float* scales;        // [rows][groups]
    const float* weight;  // [D] or null
    float* rstd;          // [rows] or null
    long long rows;
    int D, group, ngroups, x_bf16, y_bf16;  // group: columns of a scale, 0 for the whole row
    float eps;
};
struct RmsBwdArgs {
    const void *dy, *x, *dsum;
    const float *weight, *rstd;
    void* dx;
    float* partial;  // [gridDim.x][D], or null
    long long rows;
    int D, x_bf16, dy_bf16, dx_bf16;
};

// The larger of two magnitudes as bits: NaN is above infinity, so it stays.
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
    return umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, false));
}
// Maximum over L <= 64 consecutive lanes (a power of 2), left in every one of them; n: lanes of it, n <= L at run time.
template <int L>
__device__ __forceinline__ uint32_t lanes_umax(uint32_t v, int n = L) {
    if (L >= 2 && n >= 2) v = dpp_umax<0xb1>(v);
    if (L >= 4 && n >= 4) v = dpp_umax<0x4e>(v);
    if (L >= 8 && n >= 8) v = dpp_umax<0x141>(v);
    if (L >= 16 && n >= 16) v = dpp_umax<0x140>(v);
#pragma unroll
    for (int m = 16; m < L; m *= 2)
        if (n > m) v = umax(v, (uint32_t)__shfl_xor((int)v, m));
    return v;
}

// f: what a value is multiplied by for the one of y; m: the largest of the values.
__device__ __forceinline__ float scale_of_max(uint32_t m, float f) {
    const float s = __uint_as_float(m) * f / kE4m3Max;
    return s < kMinScale ? kMinScale : s;  // NaN stays
}

// W values (hi + lo) f / scale in e4m3, rounded to nearest even, where scale is m f / 448: 448 (hi + lo) / m, the quotient in two
// parts, so that f has no part in it and only the rounding of m decides which way a value next to a border between two of the
// format's goes. With y and scale as they are rounded one of 500000 values fell on the other side in every second call; the
// time is the same, HBM bounds it.
template <int W>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* hi, const float* lo, float scale, uint32_t m, float f) {
    const float top = __uint_as_float(m);
    const bool plain = !(scale > kMinScale && scale <= 3.4e38f && top > 1e-30f);  // no quotient by m
    const float inv = 1.f / (plain ? scale : top), inv448 = kE4m3Max * inv;
    float q[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
        const float t = hi[e] * inv;
        q[e] = fmaf(kE4m3Max, t, (fmaf(-t, top, hi[e]) + lo[e]) * inv448);
    }
    if (plain)
#pragma unroll
        for (int e = 0; e < W; ++e) q[e] = hi[e] * f * inv;
    if constexpr (W == 8) {
        uint2 u = make_uint2(0, 0);
        u.x = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], u.x, false);
        u.x = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], u.x, true);
        u.y = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], u.y, false);
        u.y = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], u.y, true);
        *reinterpret_cast<uint2*>(p) = u;
    } else {
        *p = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[0], 0.f, 0, false);
    }
}

// W consecutive columns per vector, K vectors per lane, L lanes per row. Q: with an output in 8 bits.
template <int W, int L, int K, int THREADS, bool Q>
__global__ __launch_bounds__(THREADS) void rms_norm_kernel(RmsArgs a) {
    constexpr int NW = THREADS / 64, G = THREADS / L;
    // groups of 32 columns and more, of rows that move value by value: their maxima meet in LDS
    constexpr int NG = Q && W == 1 ? L * K / 32 : 1;
    __shared__ float red[2 * NW];
    __shared__ uint32_t top[Q ? NW : 1];
    __shared__ uint32_t gtop[NG * G];
    RowSum<L, THREADS> sum{red, 0};
    const int lane = threadIdx.x % L, grp = threadIdx.x / L;
    const long long wg = (long long)blockIdx.y * gridDim.x + blockIdx.x;
    if (wg * G >= a.rows) return;  // the rest of the grid's last row
    const long long row = wg * G + grp;
    const bool live = row < a.rows;
    const long long base = (live ? row : a.rows - 1) * a.D;  // idle groups read the last row
    float x[K][W], s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * W;
        if (c < a.D) {
            row_load<W>(a.x, base + c, a.x_bf16, x[k]);
            if (a.res) {
                float r[W];
                row_load<W>(a.res, base + c, a.x_bf16, r);
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    x[k][e] += r[e];
                    if (a.x_bf16) x[k][e] = bf16_to_f32(f32_to_bf16(x[k][e]));
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) x[k][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < W; ++e) s2 += x[k][e] * x[k][e];
    }
    if constexpr (NG > 1)
        for (int i = threadIdx.x; i < NG * G; i += THREADS) gtop[i] = 0;  // before the barriers below
    static_assert(L <= 64 || L == THREADS, "a row's barriers are the workgroup's");
    const float inv = 1.f / (float)a.D, ms = sum(s2) * inv + a.eps;
    float rstd;
    if (ms >= kMinSquare && ms <= 3.4e38f) {
        rstd = 1.f / sqrtf(ms);
    } else {  // one for the whole row: the squares leave fp32's range, those of the row times 2^-72 or 2^100 do not
        const float f = ms > 1.f ? 0x1p-72f : 0x1p100f;
        s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < W; ++e) s2 += x[k][e] * f * (x[k][e] * f);
        rstd = f / sqrtf(sum(s2) * inv + a.eps * f * f);
    }
    if (live && lane == 0 && a.rstd) a.rstd[row] = rstd;
    // 8 bits: y = w s p2 f with p2 the power of two in rstd, so that only the product with w rounds; lo is what it loses
    const bool normal = rstd > kMinScale && rstd < 3e38f;
    const float p2 = normal ? __uint_as_float(__float_as_uint(rstd) & 0x7f800000u) : rstd;
    const float f = normal ? __uint_as_float((__float_as_uint(rstd) & 0x007fffffu) | 0x3f800000u) : 1.f;
    uint32_t m = 0, mk[K];
    float lo[Q ? K : 1][W];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * W;
        mk[k] = 0;
        if (c >= a.D) continue;
        if (live && a.sum) row_store<W>(a.sum, base + c, a.x_bf16, x[k]);
        float w[W], y[W];
        if (a.weight) row_load<W>(a.weight, c, false, w);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const float v = x[k][e], xh = v * rstd;
            y[e] = a.weight ? xh * w[e] : xh;
            if constexpr (Q) {
                const float u = v * p2;
                x[k][e] = a.weight ? u * w[e] : u;
                lo[k][e] = a.weight ? fmaf(u, w[e], -x[k][e]) : 0.f;
                mk[k] = umax(mk[k], __float_as_uint(x[k][e]) & 0x7fffffffu);
            }
        }
        m = umax(m, mk[k]);
        if (live && a.y) row_store<W>(a.y, base + c, a.y_bf16, y);
    }
    if constexpr (!Q) return;
    if (a.group == 0) {
        if constexpr (L <= 64) {
            m = lanes_umax<L>(m);
        } else {
            m = lanes_umax<64>(m);
            const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            if ((threadIdx.x & 63) == 0) top[w] = m;
            __syncthreads();
            constexpr int GW = L / 64;
#pragma unroll
            for (int i = 0; i < GW; ++i) m = umax(m, top[w / GW * GW + i]);
        }
        const float scale = scale_of_max(m, f);
        if (!live) return;
        if (lane == 0) a.scales[row] = scale;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + lane) * W;
            if (c < a.D) store_e4m3<W>(a.y8 + base + c, x[k], lo[Q ? k : 0], scale, m, f);
        }
        return;
    }
    if constexpr (W == 8) {
        // group / 8 lanes (4, 8 or 16) hold a group's columns
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + lane) * W;
            const uint32_t g = lanes_umax<16>(mk[k], a.group / 8);
            const float scale = scale_of_max(g, f);
            if (!live || c >= a.D) continue;
            if (c % a.group == 0) a.scales[row * a.ngroups + c / a.group] = scale;
            store_e4m3<W>(a.y8 + base + c, x[k], lo[Q ? k : 0], scale, g, f);
        }
    } else {
        if constexpr (L <= 64) __syncthreads();  // gtop is zero (rows of more lanes have had a barrier in their sums)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = k * L + lane;
            if (c < a.D) atomicMax(&gtop[grp * NG + c / a.group], mk[k]);
        }
        __syncthreads();
        if (!live) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = k * L + lane;
            if (c >= a.D) continue;
            const uint32_t g = gtop[grp * NG + c / a.group];
            const float scale = scale_of_max(g, f);
            if (c % a.group == 0) a.scales[row * a.ngroups + c / a.group] = scale;
            store_e4m3<W>(a.y8 + base + c, x[k], lo[Q ? k : 0], scale, g, f);
        }
    }
}

constexpr int kRmsBwdThreads = 1024;

// 128 registers a lane, of which the rows of 16 values a lane one by one (D above 8192, not a multiple of 8) spill 22.
template <int W, int L, int K>
__global__ __launch_bounds__(kRmsBwdThreads) void rms_norm_bwd_kernel(RmsBwdArgs a) {
    constexpr int T = kRmsBwdThreads, G = T / L;  // row groups
    __shared__ float red[2 * (T / 64)];
    __shared__ float cols[G > 1 ? T * W : 1];
    RowSum<L, T> sum{red, 0};
    const int lane = threadIdx.x % L, grp = threadIdx.x / L;
    float dw[K][W], w[K][W];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) dw[k][e] = 0.f, w[k][e] = 1.f;
        if (a.weight && c < a.D) row_load<W>(a.weight, c, false, w[k]);
    }
    const float inv = 1.f / (float)a.D;
    // every group of the workgroup takes part in every round (the sums' barriers)
    for (long long r0 = (long long)blockIdx.x * G; r0 < a.rows; r0 += (long long)gridDim.x * G) {
        const bool live = r0 + grp < a.rows;
        const long long row = live ? r0 + grp : a.rows - 1;
        const long long base = row * a.D;
        const float rstd = a.rstd[row];
        float xh[K][W], g[K][W], s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + lane) * W;
            if (c < a.D) {
                row_load<W>(a.x, base + c, a.x_bf16, xh[k]);
                row_load<W>(a.dy, base + c, a.dy_bf16, g[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool in = (k * L + lane) * W < a.D;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                xh[k][e] = in ? xh[k][e] * rstd : 0.f;
                const float dy = in ? g[k][e] : 0.f;
                if (live) dw[k][e] += dy * xh[k][e];
                g[k][e] = dy * w[k][e];
                s += g[k][e] * xh[k][e];
            }
        }
        s = sum(s) * inv;
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + lane) * W;
            if (c >= a.D) continue;
            float d[W];
#pragma unroll
            for (int e = 0; e < W; ++e) d[e] = 0.f;
            if (a.dsum) row_load<W>(a.dsum, base + c, a.dx_bf16, d);
#pragma unroll
            for (int e = 0; e < W; ++e) d[e] += rstd * (g[k][e] - xh[k][e] * s);
            row_store<W>(a.dx, base + c, a.dx_bf16, d);
        }
    }
    if (!a.partial) return;
    float* out = a.partial + (long long)blockIdx.x * a.D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * W;
        if constexpr (G == 1) {
            if (c < a.D)
#pragma unroll
                for (int e = 0; e < W; ++e) out[c + e] = dw[k][e];
        } else {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < W; ++e) cols[threadIdx.x * W + e] = dw[k][e];
            __syncthreads();
            for (int j = threadIdx.x; j < L * W; j += T) {
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < G; ++i) t += cols[i * L * W + j];
                if (k * L * W + j < a.D) out[k * L * W + j] = t;
            }
        }
    }
}

__global__ __launch_bounds__(kColSumThreads) void part_sum_kernel(PartSumArgs a) { part_sums(a, blockIdx.x); }

typedef void (*rms_kernel_t)(RmsArgs);
typedef void (*rms_bwd_kernel_t)(RmsBwdArgs);
struct RmsKernels {
    rms_kernel_t fwd, fwd8;
    rms_bwd_kernel_t bwd;
    int fwd_rows, fwd_threads, bwd_rows;
};

template <int W, int L, int K>
bool rms_pick(RmsKernels* o) {
    constexpr int T = L > 256 ? L : 256;
    *o = {rms_norm_kernel<W, L, K, T, false>, rms_norm_kernel<W, L, K, T, true>, rms_norm_bwd_kernel<W, L, K>, T / L, T,
          kRmsBwdThreads / L};
    return true;
}

constexpr int kRmsMaxD = 16384;

// The narrowest row group that holds D values (see ln_kernels_get); value by value at most 8 a lane where D allows.
bool rms_kernels_get(int D, RmsKernels* o) {
    if (D <= 0 || D > kRmsMaxD) return false;
    if (D % 8 == 0) {
        if (D <= 128) return rms_pick<8, 16, 1>(o);
        if (D <= 512) return rms_pick<8, 64, 1>(o);
        if (D <= 1024) return rms_pick<8, 64, 2>(o);
        if (D <= 2048) return rms_pick<8, 256, 1>(o);
        if (D <= 4096) return rms_pick<8, 256, 2>(o);
        if (D <= 8192) return rms_pick<8, 1024, 1>(o);
        return rms_pick<8, 1024, 2>(o);
    }
    if (D <= 256) return rms_pick<1, 64, 4>(o);
    if (D <= 512) return rms_pick<1, 64, 8>(o);
    if (D <= 2048) return rms_pick<1, 256, 8>(o);
    if (D <= 8192) return rms_pick<1, 1024, 8>(o);
    return rms_pick<1, 1024, 16>(o);
}

// Workgroups of the gradients' main kernel: one per CU at most, so that the partial sums stay small beside the rows.
int rms_bwd_grid(int64_t rows, const RmsKernels& k) {
    const int64_t g = (rows + k.bwd_rows - 1) / k.bwd_rows;
    return (int)(g < 256 ? g : 256);
}

constexpr int64_t kRmsGridX = 1 << 20;  // workgroups of the forward along x at most (of up to 1024 threads)

bool good_dt(ret_dtype_t t) { return t == RET_F32 || t == RET_BF16; }
size_t esize(ret_dtype_t t) { return t == RET_BF16 ? 2 : 4; }

}  // namespace

part_sum_kernel_t part_sum_kernel_get() { return part_sum_kernel; }

}  // namespace ret

using namespace ret;

extern "C" {

ret_status_t ret_rms_norm_fwd(const void* x, const void* residual, const float* weight, void* y, void* sum_out,
                              float* rstd, void* y8, float* scales, int group, int64_t rows, int D, ret_dtype_t x_dt,
                              ret_dtype_t y_dt, float eps, void* stream, const ret_options_t* opts) {
    if (rows != 0 && !x) return fail(RET_ERR_INVALID_ARG, "null x pointer");
    if (rows != 0 && !y && !y8) return fail(RET_ERR_INVALID_ARG, "neither y nor y8 is wanted");
    if (rows != 0 && (y8 == nullptr) != (scales == nullptr))
        return fail(RET_ERR_INVALID_ARG, "y8 and scales go together");
    if (rows < 0 || D <= 0) return fail(RET_ERR_INVALID_ARG, "bad sizes (rows=%lld D=%d)", (long long)rows, D);
    if (!good_dt(x_dt) || !good_dt(y_dt)) return fail(RET_ERR_INVALID_ARG, "bad dtype %d/%d", (int)x_dt, (int)y_dt);
    if (!(eps >= 0.f) || eps > 3e38f) return fail(RET_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", eps);
    if (group != 0 && group != 32 && group != 64 && group != 128)
        return fail(RET_ERR_INVALID_ARG, "group=%d must be 0, 32, 64 or 128", group);
    RmsKernels k;
    if (!rms_kernels_get(D, &k)) return fail(RET_ERR_UNSUPPORTED, "rms norm: D=%d exceeds %d", D, kRmsMaxD);
    if (rows > (int64_t)1 << 40) return fail(RET_ERR_UNSUPPORTED, "rms norm: %lld rows", (long long)rows);
    if (rows == 0) return RET_OK;
    const int ng = group ? (D + group - 1) / group : 1;
    const size_t n = (size_t)rows * D, nx = n * esize(x_dt);
    // outputs may take an input's place; workgroups write while others still read
    const Buf w[] = {{"y", y, n * esize(y_dt), 3u}, {"sum_out", sum_out, nx, 3u}, {"rstd", rstd, (size_t)rows * 4, 0, 4},
                     {"y8", y8, n}, {"scales", scales, (size_t)rows * ng * 4, 0, 4}};
    const Buf r[] = {{"x", x, nx}, {"residual", residual, nx}, {"weight", weight, (size_t)D * 4}};
    const ret_status_t apart = check_apart(w, r);
    if (apart != RET_OK) return apart;
    const int64_t wgs = (rows + k.fwd_rows - 1) / k.fwd_rows;
    // a launch of 2^32 work-items along one axis runs short without an error: the grid goes on along y
    const int64_t gx = wgs < kRmsGridX ? wgs : kRmsGridX, gy = (wgs + gx - 1) / gx;
    if (gy > 65535) return fail(RET_ERR_UNSUPPORTED, "rms norm: %lld rows", (long long)rows);
    RmsArgs A = {x, residual, sum_out, y, (uint8_t*)y8, scales, weight, rstd, rows, D, group, ng, x_dt == RET_BF16,
                 y_dt == RET_BF16, eps};
    hipStream_t s = (hipStream_t)stream;
    const Opts op = resolve(opts);
    LaunchTimer tm("ret_rms_norm", s, op);
    hipLaunchKernelGGL(y8 ? k.fwd8 : k.fwd, dim3((unsigned)gx, (unsigned)gy), dim3(k.fwd_threads), 0, s, A);
    tm.done();
    return launch_status("ret_rms_norm");
}

size_t ret_rms_norm_bwd_workspace_bytes(int64_t rows, int D) {
    RmsKernels k;
    if (rows < 0 || !rms_kernels_get(D, &k)) return 0;
    const size_t n = (size_t)rms_bwd_grid(rows, k) * D * sizeof(float);
    return n ? n : 16;
}

ret_status_t ret_rms_norm_bwd(const void* dy, const void* x, const float* weight, const float* rstd, const void* dsum,
                              void* dx, float* dweight, int64_t rows, int D, ret_dtype_t x_dt, ret_dtype_t dy_dt,
                              ret_dtype_t dx_dt, void* workspace, size_t workspace_bytes, void* stream,
                              const ret_options_t* opts) {
    if (rows != 0 && (!dy || !x || !rstd || !dx)) return fail(RET_ERR_INVALID_ARG, "null dy/x/rstd/dx pointer");
    if (rows < 0 || D <= 0) return fail(RET_ERR_INVALID_ARG, "bad sizes (rows=%lld D=%d)", (long long)rows, D);
    if (!good_dt(x_dt) || !good_dt(dy_dt) || !good_dt(dx_dt))
        return fail(RET_ERR_INVALID_ARG, "bad dtype %d/%d/%d", (int)x_dt, (int)dy_dt, (int)dx_dt);
    RmsKernels k;
    if (!rms_kernels_get(D, &k)) return fail(RET_ERR_UNSUPPORTED, "rms norm: D=%d exceeds %d", D, kRmsMaxD);
    if (rows > (int64_t)1 << 40) return fail(RET_ERR_UNSUPPORTED, "rms norm: %lld rows", (long long)rows);
    if (dweight && (!workspace || workspace_bytes < ret_rms_norm_bwd_workspace_bytes(rows, D)))
        return fail(RET_ERR_WORKSPACE, "rms norm gradients: workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : 0, ret_rms_norm_bwd_workspace_bytes(rows, D));
    const size_t n = (size_t)rows * D, nd = (size_t)D * 4;
    const Buf w[] = {{"dx", dx, n * esize(dx_dt), 1u << 0 | 1u << 1 | 1u << 2}, {"dweight", dweight, nd},
                     {"the workspace", workspace, dweight ? workspace_bytes : 0}};
    const Buf r[] = {{"dy", dy, n * esize(dy_dt)}, {"x", x, n * esize(x_dt)}, {"dsum", dsum, n * esize(dx_dt)},
                     {"weight", weight, nd}, {"rstd", rstd, (size_t)rows * 4, 0, 4}};
    const ret_status_t apart = check_apart(w, r);
    if (apart != RET_OK) return apart;
    hipStream_t s = (hipStream_t)stream;
    const Opts op = resolve(opts);
    const int grid = rms_bwd_grid(rows, k);
    if (grid > 0) {
        RmsBwdArgs A = {dy, x, dsum, weight, rstd, dx, dweight ? (float*)workspace : nullptr, rows, D, x_dt == RET_BF16,
                        dy_dt == RET_BF16, dx_dt == RET_BF16};
        LaunchTimer tm("ret_rms_norm_bwd", s, op);
        hipLaunchKernelGGL(k.bwd, dim3(grid), dim3(kRmsBwdThreads), 0, s, A);
        tm.done();
        const ret_status_t st = launch_status("ret_rms_norm_bwd");
        if (st != RET_OK) return st;
    }
    if (!dweight) return RET_OK;
    PartSumArgs P = {(const float*)workspace, dweight, nullptr, nullptr, D, D, 0, grid};
    LaunchTimer tm("ret_column_sums", s, op);
    hipLaunchKernelGGL(part_sum_kernel, dim3((D + kColSumCols - 1) / kColSumCols), dim3(kColSumThreads), 0, s, P);
    tm.done();
    return launch_status("ret_column_sums");
}

}  // extern "C"
