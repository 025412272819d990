// Gradients of the multi-scale retention epilogue y = swish(gate) (.) n, n = w xh + b, xh the standardized head row:
//   dn = dy swish(gate),  dgate = dy n swish'(gate),  swish'(x) = s + x s (1 - s) with s = sigmoid(x)
//   do = rstd (a - mean a - xh mean(a xh)), a = w dn (means over the d_v values of a head),
//   dw = sum_rows dn xh,  db = sum_rows dn  per channel of the concatenated heads.
// Mean and variance are computed again from o: reading two statistics per row instead would save nothing, since o is
// read anyway. Every tensor is read or written once; the kernel is bound by HBM.
//
// A wave owns 512 of the H d_v channels (8 per lane, so a head is a run of d_v / 8 lanes and its sums are shuffles) and
// walks rows; the 16 waves of a workgroup own the same channels and different rows. Each lane keeps the weight and bias
// sums of its channels in registers; they are added up through LDS at the end and left as one partial row per
// workgroup, which the column-sum kernel of the layer norm adds in a fixed order. Measured in bf16 with a gate: 8192 rows
// of 16 heads of 512, 128 us and 5 for the column sums (5.0 TB/s), 16384 rows of 8 heads of 64, 20 and 4 (84 MB, part of
// it from the last-level cache).
#include "host.h"
#include "rows.h"

namespace ret {

namespace {

template <int DV>
__global__ __launch_bounds__(64 * kEpiBwdWaves) void epilogue_bwd_kernel(EpiBwdArgs a) {
    constexpr int LPG = DV / 8;
    __shared__ float cols[kEpiBwdWaves * kEpiBwdCols];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int C = a.H * DV, c = blockIdx.x * kEpiBwdCols + lane * 8;
    const bool in = c < C;  // whole heads: C and the first column of a workgroup are multiples of a head's run
    const int cc = in ? c : 0;
    float wt[8], bs[8], dw[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) wt[e] = 1.f, bs[e] = dw[e] = db[e] = 0.f;
    if (a.weight) row_load<8>(a.weight, cc, false, wt);
    if (a.bias) row_load<8>(a.bias, cc, false, bs);
    const long long step = (long long)gridDim.y * kEpiBwdWaves;
    for (long long row = (long long)blockIdx.y * kEpiBwdWaves + w; row < a.rows; row += step) {
        const long long i = row * C + cc;
        float x[8], dy[8], g[8];
        row_load<8>(a.o, i, a.o_bf16, x);
        row_load<8>(a.dy, i, a.dy_bf16, dy);
        if (a.gate) row_load<8>(a.gate, i, a.gate_bf16, g);
        float s = 0.f, s2 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[e];
        const float mean = lanes_sum<LPG>(s) * (1.f / DV);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] -= mean;
            s2 += x[e] * x[e];
        }
        const float rstd = __builtin_amdgcn_rsqf(lanes_sum<LPG>(s2) * (1.f / DV) + a.eps);
        float dg[8], m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] *= rstd;
            float dn = dy[e];
            if (a.gate) {
                const float sg = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g[e]));
                dg[e] = dn * (x[e] * wt[e] + bs[e]) * (sg + g[e] * sg * (1.f - sg));
                dn *= g[e] * sg;
            }
            dw[e] += dn * x[e];
            db[e] += dn;
            dy[e] = dn * wt[e];
            m1 += dy[e];
            m2 += dy[e] * x[e];
        }
        m1 = lanes_sum<LPG>(m1) * (1.f / DV);
        m2 = lanes_sum<LPG>(m2) * (1.f / DV);
#pragma unroll
        for (int e = 0; e < 8; ++e) dy[e] = rstd * (dy[e] - m1 - x[e] * m2);
        if (!in) continue;
        row_store<8>(a.dout, i, a.do_bf16, dy);
        if (a.dgate) row_store<8>(a.dgate, i, a.dgate_bf16, dg);
    }
    if (!a.partial) return;
    float* out = a.partial + (long long)blockIdx.y * 2 * C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) cols[w * kEpiBwdCols + lane * 8 + e] = which ? db[e] : dw[e];
        __syncthreads();
        const int j = threadIdx.x, col = blockIdx.x * kEpiBwdCols + j;
        if (j < kEpiBwdCols && col < C) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kEpiBwdWaves; ++i) s += cols[i * kEpiBwdCols + j];
            out[which * C + col] = s;
        }
    }
}

// Workgroups along the rows: about two per CU over all column blocks.
int epi_bwd_strips(int64_t rows, int C) {
    const int blocks = (C + kEpiBwdCols - 1) / kEpiBwdCols;
    const int64_t most = (rows + kEpiBwdWaves - 1) / kEpiBwdWaves;
    const int64_t want = (512 + blocks - 1) / blocks;
    return (int)(want < most ? want : most);
}

size_t esize(ret_dtype_t t) { return t == RET_BF16 ? 2 : 4; }

// H d_v below this: the column sums take 32 work-items a channel, and a launch fewer than 2^32.
constexpr int64_t kEpiBwdMaxC = 1 << 27;

}  // namespace

epi_bwd_kernel_t epi_bwd_kernel_get(int dv) {
    switch (dv) {
        case 16: return epilogue_bwd_kernel<16>;
        case 32: return epilogue_bwd_kernel<32>;
        case 64: return epilogue_bwd_kernel<64>;
        case 128: return epilogue_bwd_kernel<128>;
        case 256: return epilogue_bwd_kernel<256>;
        case 512: return epilogue_bwd_kernel<512>;
        default: return nullptr;
    }
}

}  // namespace ret

using namespace ret;

extern "C" {

size_t ret_msr_epilogue_bwd_workspace_bytes(int64_t rows, int H, int dv) {
    if (rows < 0 || H <= 0 || !epi_bwd_kernel_get(dv) || (int64_t)H * dv >= kEpiBwdMaxC) return 0;
    const size_t n = (size_t)epi_bwd_strips(rows, H * dv) * 2 * H * dv * sizeof(float);
    return n ? n : 16;
}

ret_status_t ret_msr_epilogue_bwd(const void* dy, const void* o, const void* gate, const float* gn_weight,
                                  const float* gn_bias, void* dout, void* dgate, float* dweight, float* dbias,
                                  int64_t rows, int H, int dv, ret_dtype_t dy_dt, ret_dtype_t o_dt,
                                  ret_dtype_t gate_dt, ret_dtype_t do_dt, ret_dtype_t dgate_dt, float eps,
                                  void* workspace, size_t workspace_bytes, void* stream, const ret_options_t* opts) {
    if (rows != 0 && (!dy || !o || !dout)) return fail(RET_ERR_INVALID_ARG, "null dy/o/do pointer");
    if (rows != 0 && dgate && !gate) return fail(RET_ERR_INVALID_ARG, "dgate without a gate");
    if (rows < 0 || H <= 0 || dv <= 0)
        return fail(RET_ERR_INVALID_ARG, "bad sizes (rows=%lld H=%d dv=%d)", (long long)rows, H, dv);
    for (ret_dtype_t t : {dy_dt, o_dt, gate_dt, do_dt, dgate_dt})
        if (t != RET_F32 && t != RET_BF16) return fail(RET_ERR_INVALID_ARG, "bad dtype %d", (int)t);
    if (!(eps >= 0.f) || eps > 3e38f) return fail(RET_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", eps);
    const epi_bwd_kernel_t fn = epi_bwd_kernel_get(dv);
    if (!fn) return fail(RET_ERR_UNSUPPORTED, "epilogue gradients: d_v=%d not in {16,32,64,128,256,512}", dv);
    if ((int64_t)H * dv >= kEpiBwdMaxC || rows > (int64_t)1 << 40)
        return fail(RET_ERR_UNSUPPORTED, "epilogue gradients: rows=%lld H=%d too large", (long long)rows, H);
    const bool cols = dweight || dbias;
    const size_t need = ret_msr_epilogue_bwd_workspace_bytes(rows, H, dv);
    if (cols && (!workspace || workspace_bytes < need))
        return fail(RET_ERR_WORKSPACE, "epilogue gradients: workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : 0, need);
    const int C = H * dv;
    const size_t n = (size_t)rows * C, nd = 4 * (size_t)C;
    // each output may take the place of one tensor input; workgroups write while others still read
    const Buf w[] = {{"do", dout, n * esize(do_dt), 7u}, {"dgate", dgate, n * esize(dgate_dt), 7u}, {"dweight", dweight, nd},
                     {"dbias", dbias, nd}, {"the workspace", workspace, cols ? workspace_bytes : 0}};
    const Buf r[] = {{"dy", dy, n * esize(dy_dt)}, {"o", o, n * esize(o_dt)}, {"gate", gate, n * esize(gate_dt)},
                     {"gn_weight", gn_weight, nd}, {"gn_bias", gn_bias, nd}};
    const ret_status_t apart = check_apart(w, r);
    if (apart != RET_OK) return apart;
    hipStream_t s = (hipStream_t)stream;
    const Opts op = resolve(opts);
    const int strips = epi_bwd_strips(rows, C);
    if (strips > 0) {
        EpiBwdArgs A = {dy, o, gate, gn_weight, gn_bias, dout, dgate, cols ? (float*)workspace : nullptr, rows, H,
                        dy_dt == RET_BF16, o_dt == RET_BF16, gate_dt == RET_BF16, do_dt == RET_BF16,
                        dgate_dt == RET_BF16, eps};
        LaunchTimer tm("ret_msr_epilogue_bwd", s, op);
        hipLaunchKernelGGL(fn, dim3((C + kEpiBwdCols - 1) / kEpiBwdCols, strips), dim3(64 * kEpiBwdWaves), 0, s, A);
        tm.done();
        const ret_status_t st = launch_status("ret_msr_epilogue_bwd");
        if (st != RET_OK) return st;
    }
    if (!cols) return RET_OK;
    ColSumArgs R = {(const float*)workspace, dweight, dbias, strips, C};
    LaunchTimer tm("ret_column_sums", s, op);
    hipLaunchKernelGGL(colsum_kernel_get(), dim3((unsigned)((2LL * C + kColSumCols - 1) / kColSumCols)), dim3(kColSumThreads), 0, s, R);
    tm.done();
    return launch_status("ret_column_sums");
}

}  // extern "C"
