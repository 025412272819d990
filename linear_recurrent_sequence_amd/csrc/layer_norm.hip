// Layer norm over rows of D values, forward and gradients.
//
//   forward:  s = x + residual (rounded to x's dtype), xh = (s - mean s) rstd, y = w xh + b
//   gradient: a = w dy, dx = rstd (a - mean a - xh mean(a xh)) + dsum, dw = sum_rows dy xh, db = sum_rows dy
//
// A row is held in the registers of L lanes (4 to 16 values each, so that D up to 16384 needs no second read): both
// kernels read each tensor once. Rows whose length is a multiple of 8 move as 16-byte vectors and are bound by HBM, others
// value by value. Statistics are fp32: mean first, then the squared differences from it, both from registers.
// L <= 64 reduces within a wave (no barrier); wider rows add their waves' sums through LDS. Measured: forward, 128 rows of
// 4096 in bf16 with the residual 5.1 us (launch and one round trip), 8192 of them 57 (4.7 TB/s), 16384 rows of 1001 in fp32
// 35 us (3.7 TB/s), in bf16 30 (2.2); gradients, 8192 rows of 4096 in bf16 58 us and 5 for the column sums (4.3 TB/s
// over both). Gradients of rows of more than 256 values whose number is no multiple of 8 are bound by their 16 values a lane,
// of which the compiler spills 46 to 76 registers, and by 2- and 4-byte accesses: 16384 rows of 1001 93 us in fp32 (2.1
// TB/s) and 137 in bf16 (0.7), 8192 of 4097 in bf16 260; 4 values a lane do not spill (65536 rows of 250 in fp32, 49 us).
//
// The weight's gradients are sums over rows. A workgroup walks the rows with a stride of the grid, keeps the sums of its
// own columns in registers, adds up its row groups through LDS at the end and leaves one partial row of sums; a second
// kernel adds those in a fixed order, so the same call gives the same bits.
#include "host.h"
#include "rows.h"

namespace ret {

namespace {

// Sum over the L lanes of a row group, left in every one of them. red: 2 slots of THREADS / 64 floats, used in turn so
// that one barrier per sum is enough (a slot is written again only after the other slot's barrier).
template <int L, int THREADS>
struct RowSum {
    float* red;
    int slot;
    __device__ __forceinline__ float operator()(float v) {
        if constexpr (L <= 64) {
            return lanes_sum<L>(v);
        } else {
            constexpr int NW = THREADS / 64, GW = L / 64;
            v = lanes_sum<64>(v);
            const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            float* r = red + slot * NW;
            slot ^= 1;
            if ((threadIdx.x & 63) == 0) r[w] = v;
            __syncthreads();
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < GW; ++i) s += r[w / GW * GW + i];
            return s;
        }
    }
};

// W consecutive columns per vector, K vectors per lane, L lanes per row.
template <int W, int L, int K, int THREADS>
__global__ __launch_bounds__(THREADS) void layer_norm_kernel(LnArgs a) {
    __shared__ float red[2 * (THREADS / 64)];
    RowSum<L, THREADS> sum{red, 0};
    const int lane = threadIdx.x % L;
    const long long wg = (long long)blockIdx.y * gridDim.x + blockIdx.x;
    if (wg * (THREADS / L) >= a.rows) return;  // the rest of the grid's last row
    const long long row = wg * (THREADS / L) + threadIdx.x / L;
    const bool live = row < a.rows;
    const long long base = (live ? row : a.rows - 1) * a.D;  // idle groups read the last row
    float x[K][W], s = 0.f;
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
        for (int e = 0; e < W; ++e) s += x[k][e];
    }
    const float inv = 1.f / (float)a.D;
    const float mean = sum(s) * inv;
    float s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if ((k * L + lane) * W < a.D)
#pragma unroll
            for (int e = 0; e < W; ++e) s2 += (x[k][e] - mean) * (x[k][e] - mean);
    const float rstd = 1.f / sqrtf(sum(s2) * inv + a.eps);
    if (!live) return;
    if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * W;
        if (c >= a.D) continue;
        if (a.sum) row_store<W>(a.sum, base + c, a.x_bf16, x[k]);
        float w[W], b[W];
        if (a.weight) row_load<W>(a.weight, c, false, w);
        if (a.bias) row_load<W>(a.bias, c, false, b);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            x[k][e] = (x[k][e] - mean) * rstd;
            if (a.weight) x[k][e] *= w[e];
            if (a.bias) x[k][e] += b[e];
        }
        row_store<W>(a.y, base + c, a.y_bf16, x[k]);
    }
}

template <int W, int L, int K>
__global__ __launch_bounds__(kLnBwdThreads) void layer_norm_bwd_kernel(LnBwdArgs a) {
    constexpr int T = kLnBwdThreads, G = T / L;  // row groups
    __shared__ float red[2 * (T / 64)];
    __shared__ float cols[G > 1 ? T * W : 1];
    RowSum<L, T> sum{red, 0};
    const int lane = threadIdx.x % L, grp = threadIdx.x / L;
    float dw[K][W], db[K][W], w[K][W];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) dw[k][e] = db[k][e] = 0.f, w[k][e] = 1.f;
        if (a.weight && c < a.D) row_load<W>(a.weight, c, false, w[k]);
    }
    const float inv = 1.f / (float)a.D;
    // every group of the workgroup takes part in every round (the sums' barriers)
    for (long long r0 = (long long)blockIdx.x * G; r0 < a.rows; r0 += (long long)gridDim.x * G) {
        const bool live = r0 + grp < a.rows;
        const long long row = live ? r0 + grp : a.rows - 1;
        const long long base = row * a.D;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float xh[K][W], g[K][W], s1 = 0.f, s2 = 0.f;
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
                xh[k][e] = in ? (xh[k][e] - mean) * rstd : 0.f;
                const float dy = in ? g[k][e] : 0.f;
                if (live) {
                    dw[k][e] += dy * xh[k][e];
                    db[k][e] += dy;
                }
                g[k][e] = dy * w[k][e];
                s1 += g[k][e];
                s2 += g[k][e] * xh[k][e];
            }
        }
        s1 = sum(s1) * inv;
        s2 = sum(s2) * inv;
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
            for (int e = 0; e < W; ++e) d[e] += rstd * (g[k][e] - s1 - xh[k][e] * s2);
            row_store<W>(a.dx, base + c, a.dx_bf16, d);
        }
    }
    if (!a.partial) return;
    float* out = a.partial + (long long)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + lane) * W;
            if constexpr (G == 1) {
                if (c < a.D)
#pragma unroll
                    for (int e = 0; e < W; ++e) out[which * a.D + c + e] = which ? db[k][e] : dw[k][e];
            } else {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < W; ++e) cols[threadIdx.x * W + e] = which ? db[k][e] : dw[k][e];
                __syncthreads();
                for (int j = threadIdx.x; j < L * W; j += T) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < G; ++i) s += cols[i * L * W + j];
                    if (k * L * W + j < a.D) out[which * a.D + k * L * W + j] = s;
                }
            }
        }
    }
}

// Sums of `parts` partial rows: 64 columns per workgroup, the rows dealt to its 16 waves, 8 loads of a wave in flight.
__global__ __launch_bounds__(kColSumThreads) void colsum_kernel(ColSumArgs a) {
    constexpr int NW = kColSumThreads / 64, U = 8;
    __shared__ float part[kColSumThreads];
    const int c = blockIdx.x * kColSumCols + (threadIdx.x & 63), w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool in = c < 2 * a.cols;
    const float* p = a.partial + (in ? c : 0);
    float s = 0.f;
    for (int r = w; r < a.parts; r += NW * U) {
        float x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int q = r + i * NW;
            x[i] = p[(long long)(q < a.parts ? q : r) * 2 * a.cols];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) s += r + i * NW < a.parts ? x[i] : 0.f;
    }
    part[threadIdx.x] = s;
    __syncthreads();
    if (w != 0 || !in) return;
#pragma unroll
    for (int i = 1; i < NW; ++i) s += part[threadIdx.x + 64 * i];
    if (c < a.cols) {
        if (a.out0) a.out0[c] = s;
    } else if (a.out1) {
        a.out1[c - a.cols] = s;
    }
}

template <int W, int L, int K>
bool ln_pick(LnKernels* o) {
    constexpr int T = L > 256 ? L : 256;
    *o = {layer_norm_kernel<W, L, K, T>, layer_norm_bwd_kernel<W, L, K>, T / L, T, kLnBwdThreads / L};
    return true;
}

}  // namespace

colsum_kernel_t colsum_kernel_get() { return colsum_kernel; }

// The narrowest row group that holds D values, 8 or 16 per lane: few lanes per row where rows are short, so that a wave
// holds several rows; many where they are long, so that a row's values stay in registers.
bool ln_kernels_get(int D, LnKernels* o) {
    if (D <= 0 || D > kLnMaxD) return false;
    if (D % 8 == 0) {
        if (D <= 128) return ln_pick<8, 16, 1>(o);
        if (D <= 512) return ln_pick<8, 64, 1>(o);
        if (D <= 1024) return ln_pick<8, 64, 2>(o);
        if (D <= 2048) return ln_pick<8, 256, 1>(o);
        if (D <= 4096) return ln_pick<8, 256, 2>(o);
        if (D <= 8192) return ln_pick<8, 1024, 1>(o);
        return ln_pick<8, 1024, 2>(o);
    }
    if (D <= 256) return ln_pick<1, 64, 4>(o);
    if (D <= 1024) return ln_pick<1, 64, 16>(o);
    if (D <= 4096) return ln_pick<1, 256, 16>(o);
    return ln_pick<1, 1024, 16>(o);
}

namespace {

// Workgroups of the gradients' main kernel: one per CU at most, so that the partial sums stay small beside the rows.
int ln_bwd_grid(int64_t rows, const LnKernels& k) {
    const int64_t g = (rows + k.bwd_rows - 1) / k.bwd_rows;
    return (int)(g < 256 ? g : 256);
}

constexpr int64_t kLnGridX = 1 << 20;  // workgroups of the forward along x at most (of up to 1024 threads)

bool good_dt(ret_dtype_t t) { return t == RET_F32 || t == RET_BF16; }
size_t esize(ret_dtype_t t) { return t == RET_BF16 ? 2 : 4; }

}  // namespace

}  // namespace ret

using namespace ret;

extern "C" {

ret_status_t ret_layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias, void* y,
                                void* sum_out, float* mean, float* rstd, int64_t rows, int D, ret_dtype_t x_dt,
                                ret_dtype_t y_dt, float eps, void* stream, const ret_options_t* opts) {
    if (rows != 0 && (!x || !y)) return fail(RET_ERR_INVALID_ARG, "null x/y pointer");
    if (rows < 0 || D <= 0) return fail(RET_ERR_INVALID_ARG, "bad sizes (rows=%lld D=%d)", (long long)rows, D);
    if (!good_dt(x_dt) || !good_dt(y_dt)) return fail(RET_ERR_INVALID_ARG, "bad dtype %d/%d", (int)x_dt, (int)y_dt);
    if (!(eps >= 0.f) || eps > 3e38f) return fail(RET_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", eps);
    LnKernels k;
    if (!ln_kernels_get(D, &k)) return fail(RET_ERR_UNSUPPORTED, "layer norm: D=%d exceeds %d", D, kLnMaxD);
    if (rows > (int64_t)1 << 40) return fail(RET_ERR_UNSUPPORTED, "layer norm: %lld rows", (long long)rows);
    if (rows == 0) return RET_OK;
    const size_t nx = (size_t)rows * D * esize(x_dt), nr = (size_t)rows * 4, nd = (size_t)D * 4;
    // outputs may take an input's place; workgroups write while others still read
    const Buf w[] = {{"y", y, (size_t)rows * D * esize(y_dt), 3u}, {"sum_out", sum_out, nx, 3u}, {"mean", mean, nr, 0, 4},
                     {"rstd", rstd, nr, 0, 4}};
    const Buf r[] = {{"x", x, nx}, {"residual", residual, nx}, {"weight", weight, nd}, {"bias", bias, nd}};
    const ret_status_t apart = check_apart(w, r);
    if (apart != RET_OK) return apart;
    const int64_t wgs = (rows + k.fwd_rows - 1) / k.fwd_rows;
    // a launch of 2^32 work-items along one axis runs short without an error: the grid goes on along y
    const int64_t gx = wgs < kLnGridX ? wgs : kLnGridX, gy = (wgs + gx - 1) / gx;
    if (gy > 65535) return fail(RET_ERR_UNSUPPORTED, "layer norm: %lld rows", (long long)rows);
    LnArgs A = {x, residual, sum_out, y, weight, bias, mean, rstd, rows, D, x_dt == RET_BF16, y_dt == RET_BF16, eps};
    hipStream_t s = (hipStream_t)stream;
    const Opts op = resolve(opts);
    LaunchTimer tm("ret_layer_norm", s, op);
    hipLaunchKernelGGL(k.fwd, dim3((unsigned)gx, (unsigned)gy), dim3(k.fwd_threads), 0, s, A);
    tm.done();
    return launch_status("ret_layer_norm");
}

size_t ret_layer_norm_bwd_workspace_bytes(int64_t rows, int D) {
    LnKernels k;
    if (rows < 0 || !ln_kernels_get(D, &k)) return 0;
    const size_t n = (size_t)ln_bwd_grid(rows, k) * 2 * D * sizeof(float);
    return n ? n : 16;
}

ret_status_t ret_layer_norm_bwd(const void* dy, const void* x, const float* weight, const float* mean,
                                const float* rstd, const void* dsum, void* dx, float* dweight, float* dbias,
                                int64_t rows, int D, ret_dtype_t x_dt, ret_dtype_t dy_dt, ret_dtype_t dx_dt,
                                void* workspace, size_t workspace_bytes, void* stream, const ret_options_t* opts) {
    if (rows != 0 && (!dy || !x || !mean || !rstd || !dx))
        return fail(RET_ERR_INVALID_ARG, "null dy/x/mean/rstd/dx pointer");
    if (rows < 0 || D <= 0) return fail(RET_ERR_INVALID_ARG, "bad sizes (rows=%lld D=%d)", (long long)rows, D);
    if (!good_dt(x_dt) || !good_dt(dy_dt) || !good_dt(dx_dt))
        return fail(RET_ERR_INVALID_ARG, "bad dtype %d/%d/%d", (int)x_dt, (int)dy_dt, (int)dx_dt);
    LnKernels k;
    if (!ln_kernels_get(D, &k)) return fail(RET_ERR_UNSUPPORTED, "layer norm: D=%d exceeds %d", D, kLnMaxD);
    if (rows > (int64_t)1 << 40) return fail(RET_ERR_UNSUPPORTED, "layer norm: %lld rows", (long long)rows);
    const bool cols = dweight || dbias;
    if (cols && (!workspace || workspace_bytes < ret_layer_norm_bwd_workspace_bytes(rows, D)))
        return fail(RET_ERR_WORKSPACE, "layer norm gradients: workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : 0, ret_layer_norm_bwd_workspace_bytes(rows, D));
    // workgroups write their partial sums and rows of dx while others still read
    const size_t n = (size_t)rows * D, nr = (size_t)rows * 4, nd = (size_t)D * 4;
    const Buf w[] = {{"dx", dx, n * esize(dx_dt), 1u << 0 | 1u << 1 | 1u << 2}, {"dweight", dweight, nd},
                     {"dbias", dbias, nd}, {"the workspace", workspace, cols ? workspace_bytes : 0}};
    const Buf r[] = {{"dy", dy, n * esize(dy_dt)}, {"x", x, n * esize(x_dt)}, {"dsum", dsum, n * esize(dx_dt)},
                     {"weight", weight, nd}, {"mean", mean, nr, 0, 4}, {"rstd", rstd, nr, 0, 4}};
    const ret_status_t apart = check_apart(w, r);
    if (apart != RET_OK) return apart;
    hipStream_t s = (hipStream_t)stream;
    const Opts op = resolve(opts);
    const int grid = ln_bwd_grid(rows, k);
    if (grid > 0) {
        LnBwdArgs A = {dy, x, dsum, weight, mean, rstd, dx, cols ? (float*)workspace : nullptr, rows, D,
                       x_dt == RET_BF16, dy_dt == RET_BF16, dx_dt == RET_BF16};
        LaunchTimer tm("ret_layer_norm_bwd", s, op);
        hipLaunchKernelGGL(k.bwd, dim3(grid), dim3(kLnBwdThreads), 0, s, A);
        tm.done();
        const ret_status_t st = launch_status("ret_layer_norm_bwd");
        if (st != RET_OK) return st;
    }
    if (!cols) return RET_OK;
    ColSumArgs C = {(const float*)workspace, dweight, dbias, grid, D};
    LaunchTimer tm("ret_column_sums", s, op);
    hipLaunchKernelGGL(colsum_kernel, dim3((2 * D + kColSumCols - 1) / kColSumCols), dim3(kColSumThreads), 0, s, C);
    tm.done();
    return launch_status("ret_column_sums");
}

}  // extern "C"
