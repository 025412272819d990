// Entry points of the gated delta rule: argument checks, segment plan, workspace layout, launches.
#include "delta.h"
#include "host.h"

#include <math.h>
#include <string.h>

namespace ret {

namespace {

size_t esize(ret_dtype_t t) { return t == RET_BF16 ? 2 : 4; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct Shape {
    int B, N, H, Hk, dk, dv;
};

// B H at most: a sequence's kernels have up to B H workgroups along the grid's y, a step's along x (that many are tested).
constexpr int kSeqMaxBH = 65535, kStepMaxBH = 1 << 17;

// Sizes, dtypes and head counts of any of the calls; N = 1 for a step.
ret_status_t check_shape(const Shape& s, ret_dtype_t in_dt, ret_dtype_t out_dt, ret_dtype_t gate_dt, int max_bh) {
    if (s.B <= 0 || s.N <= 0 || s.H <= 0 || s.Hk <= 0 || s.dk <= 0 || s.dv <= 0)
        return fail(RET_ERR_INVALID_ARG, "sizes must be positive (B=%d N=%d H=%d Hk=%d dk=%d dv=%d)", s.B, s.N, s.H,
                    s.Hk, s.dk, s.dv);
    for (ret_dtype_t t : {in_dt, out_dt, gate_dt})
        if (t != RET_F32 && t != RET_BF16) return fail(RET_ERR_INVALID_ARG, "bad dtype %d", (int)t);
    if (in_dt == RET_F32 && (out_dt != RET_F32 || gate_dt != RET_F32))
        return fail(RET_ERR_INVALID_ARG, "F32 input requires F32 output and gates");
    if (s.H % s.Hk) return fail(RET_ERR_INVALID_ARG, "H=%d is not a multiple of Hk=%d", s.H, s.Hk);
    if ((long long)s.B * s.H > max_bh)
        return fail(RET_ERR_UNSUPPORTED, "B*H=%lld exceeds %d", (long long)s.B * s.H, max_bh);
    // a chunk of one head is addressed with 32-bit byte offsets
    const long long w = (long long)s.H * (s.dk > s.dv ? s.dk : s.dv);
    if (w * kDeltaC * 4 >= 1LL << 30)
        return fail(RET_ERR_UNSUPPORTED, "H*max(d_k,d_v)=%lld too large", w);
    if ((long long)s.dk * s.dv * 4 >= 1LL << 30)  // and so is a head's state
        return fail(RET_ERR_UNSUPPORTED, "d_k*d_v=%lld too large", (long long)s.dk * s.dv);
    return RET_OK;
}

float scale_of(float scale, int dk) { return scale == 0.f ? (float)(1.0 / sqrt((double)dk)) : scale; }

// Segments per sequence, by default
//   - one workgroup of the full pass per CU, two where rows are short, rounded down: more go in a second round (129 heads of
//     1024 tokens, 128 x 128: one segment 98 us, two 165; gradients 291 and 412);
//   - at least 4 chunks a segment. Segments of 2, 3, 4 and 6 chunks take, for 4 heads of 2048 tokens, 169, 137, 120 and 123 us
//     at d_k = 256 and 68, 62, 62 and 69 at 128; for 4 x 1024 tokens of 8 heads at 128, 70, -, 60 and 69. Where few heads leave
//     the card idle 2 would be better (1024 tokens of 8 heads of 64: 31 us, 35 at 4 chunks; fp32, 4 heads of 128: 94 and 131),
//     and so would one segment be than two for 8 to 11 chunks of bf16 (512 tokens of 8 heads of 64: 29 us and 32).
struct Plan {
    int nchunks, nseg, seg_chunks;
    size_t mats, fac, segE, segM, segF, s0t, ds1t, et, dut, bytes;  // byte offsets of the parts, and their end
    size_t state, rows;                                             // bytes of one part of s0t or ds1t, of et or dut
};
// parts: 0 for the forward; for the gradients, in how many the chains store what the per-chunk kernel reads.
Plan make_plan(const Shape& s, const DeltaKernels& k, ret_dtype_t in_dt, int parts, const Opts& op) {
    const bool bwd = parts > 0;
    const int nmats = bwd ? 3 : 2;
    Plan p;
    p.nchunks = s.N / kDeltaC + (s.N % kDeltaC != 0);
    const long long units = (long long)s.B * s.H * ((s.dv + k.cols - 1) / k.cols);
    int n = 1;
    if (op.segments > 0) n = op.segments;
    else n = (int)((s.dk * esize(in_dt) >= 256 ? 256 : 512) / units);
    if (op.segments <= 0 && n > p.nchunks / 4) n = p.nchunks / 4;
    if (n > p.nchunks) n = p.nchunks;
    if (n < 1) n = 1;
    p.seg_chunks = (p.nchunks + n - 1) / n;
    p.nseg = (p.nchunks + p.seg_chunks - 1) / p.seg_chunks;
    const size_t bh = (size_t)s.B * s.H;
    p.mats = 0;
    p.fac = p.mats + bh * p.nchunks * nmats * kDeltaMatBytes;
    p.segE = p.fac + round256(bh * p.nchunks * kDeltaFac * sizeof(float));
    p.segM = p.segE + (p.nseg > 1 ? round256(bh * p.nseg * s.dk * s.dv * sizeof(float)) : 0);
    p.segF = p.segM + (p.nseg > 1 ? round256(bh * p.nseg * s.dk * s.dk * sizeof(float)) : 0);
    p.s0t = p.ds1t = p.et = p.dut = p.bytes = p.segF;
    p.state = round256(bh * p.nchunks * s.dk * s.dv * esize(in_dt));
    p.rows = round256(bh * p.nchunks * kDeltaC * s.dv * esize(in_dt));
    if (bwd) {
        p.s0t = p.segF + (p.nseg > 1 ? round256(bh * p.nseg * s.dk * s.dv * sizeof(float)) : 0);
        p.ds1t = p.s0t + parts * p.state;
        p.et = p.ds1t + parts * p.state;
        p.dut = p.et + parts * p.rows;
        p.bytes = p.dut + parts * p.rows;
    }
    return p;
}
// delta_prep: the value heads of a key head share a workgroup unless the card takes one for each at once. 8 value heads of
// 2 key heads at d_k = 128, shared and one each: 512 of them 32 and 18 us, 2048 38 and 34, 4096 51 and 60; at d_k = 256 32
// and 18, 41 and 55, 74 and 100.
dim3 prep_grid(const Plan& p, const Shape& s) {
    return dim3(p.nchunks, s.B * s.Hk, (long long)p.nchunks * s.B * s.H <= 512 ? s.H / s.Hk : 1);
}

void fill(DeltaArgs& A, const Shape& s, const Plan& p, bool bwd, void* workspace, ret_dtype_t out_dt,
          ret_dtype_t gate_dt, float scale) {
    memset(&A, 0, sizeof(A));
    A.B = s.B;
    A.N = s.N;
    A.H = s.H;
    A.Hk = s.Hk;
    A.dk = s.dk;
    A.dv = s.dv;
    A.nchunks = p.nchunks;
    A.nmats = bwd ? 3 : 2;
    A.nseg = p.nseg;
    A.seg_chunks = p.seg_chunks;
    A.mats = (char*)workspace + p.mats;
    A.fac = (float*)((char*)workspace + p.fac);
    A.segE = (float*)((char*)workspace + p.segE);
    A.segM = (float*)((char*)workspace + p.segM);
    A.segF = (float*)((char*)workspace + p.segF);
    A.s0t = (char*)workspace + p.s0t;
    A.ds1t = (char*)workspace + p.ds1t;
    A.et = (char*)workspace + p.et;
    A.dut = (char*)workspace + p.dut;
    A.state_lo = p.state / 2;  // bf16 elements
    A.rows_lo = p.rows / 2;
    A.out_bf16 = out_dt == RET_BF16;
    A.gate_bf16 = gate_dt == RET_BF16;
    A.scale = scale_of(scale, s.dk);
}

ret_status_t launch(const char* name, delta_kernel_t fn, dim3 grid, hipStream_t s, const Opts& op, const DeltaArgs& A,
                    int threads = kThreads) {
    LaunchTimer tm(name, s, op);
    hipLaunchKernelGGL(fn, grid, dim3(threads), 0, s, A);
    tm.done();
    return launch_status(name);
}

unsigned long long blocks(long long n, int per) { return (unsigned long long)((n + per - 1) / per); }

// Workgroups of the chains: a multiple of 8 segments (see DeltaBlock) times the column blocks of d_v, and in a local pass
// of the transition's d_k.
struct Grids {
    unsigned long long units, nv, nk, scan_y;
};
// RET_ERR_UNSUPPORTED where one of the call's launches would not run whole.
ret_status_t make_grids(const Shape& s, const Plan& p, const DeltaKernels& k, Grids* g) {
    const unsigned long long heads = (unsigned long long)s.B * s.H;
    *g = {blocks(heads * p.nseg, 8) * 8, blocks(s.dv, k.cols), blocks(s.dk, k.cols), blocks(s.dv, kScanCols)};
    const dim3 chunks = prep_grid(p, s);  // delta_prep's; delta_grad's is no larger
    const int threads = k.grad_threads > kThreads ? k.grad_threads : kThreads;
    const bool split = p.nseg > 1;
    if (!grid_fits(chunks.x, chunks.y, chunks.z, threads) ||
        !grid_fits(g->units * (g->nv + (split ? g->nk : 0)), 1, 1, k.threads) ||
        (split && !grid_fits(heads, g->scan_y, 1, k.scan_threads)))
        return fail(RET_ERR_UNSUPPORTED, "gated delta rule: B=%d N=%d H=%d d_v=%d in %d segments exceed a launch", s.B, s.N,
                    s.H, s.dv, p.nseg);
    return RET_OK;
}

}  // namespace

}  // namespace ret

using namespace ret;

extern "C" {

size_t ret_gated_delta_workspace_bytes(int B, int N, int H, int Hk, int dk, int dv, ret_dtype_t in_dt,
                                       const ret_options_t* opts) {
    const Shape s = {B, N, H, Hk, dk, dv};
    DeltaKernels k;
    if (check_shape(s, in_dt, RET_F32, RET_F32, kSeqMaxBH) != RET_OK) return 0;
    if (!delta_kernels_get(in_dt == RET_BF16, dk, dv, &k)) return 0;
    const Plan p = make_plan(s, k, in_dt, 0, resolve(opts));
    Grids G;
    return make_grids(s, p, k, &G) == RET_OK ? p.bytes : 0;
}

ret_status_t ret_gated_delta_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta, void* o,
                                 int B, int N, int H, int Hk, int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt,
                                 ret_dtype_t gate_dt, float scale, const int32_t* lengths, const float* state_in,
                                 float* state_out, void* workspace, size_t workspace_bytes, void* stream,
                                 const ret_options_t* opts) {
    const Shape s = {B, N, H, Hk, dk, dv};
    ret_status_t st = check_shape(s, in_dt, out_dt, gate_dt, kSeqMaxBH);
    if (st != RET_OK) return st;
    if (!q || !k || !v || !g || !beta || !o) return fail(RET_ERR_INVALID_ARG, "null q/k/v/g/beta/o pointer");
    if (!isfinite(scale)) return fail(RET_ERR_INVALID_ARG, "scale is not finite");
    DeltaKernels kn;
    if (!delta_kernels_get(in_dt == RET_BF16, dk, dv, &kn))
        return fail(RET_ERR_UNSUPPORTED, "gated delta rule: unsupported d_k=%d d_v=%d for %s input", dk, dv,
                    in_dt == RET_F32 ? "F32" : "BF16");
    const Opts op = resolve(opts);
    const Plan p = make_plan(s, kn, in_dt, 0, op);
    Grids G;
    if ((st = make_grids(s, p, kn, &G)) != RET_OK) return st;
    const size_t T = (size_t)B * N, ei = esize(in_dt), sb = (size_t)B * H * dk * dv * 4;
    const unsigned eg = esize(gate_dt);
    // state_out may be state_in (r[6]): every kernel that reads the latter has read it before the former is written,
    // except within a segment chain's first launches, which precede it
    const Buf w[] = {{"o", o, T * H * dv * esize(out_dt)}, {"state_out", state_out, sb, 1u << 6},
                     {"the workspace", workspace, workspace_bytes}};
    const Buf r[] = {{"q", q, T * Hk * dk * ei}, {"k", k, T * Hk * dk * ei}, {"v", v, T * H * dv * ei},
                     {"g", g, T * H * eg, 0, eg}, {"beta", beta, T * H * eg, 0, eg},
                     {"lengths", lengths, (size_t)B * 4, 0, 4}, {"state_in", state_in, sb}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    if (!workspace || workspace_bytes < p.bytes)
        return fail(RET_ERR_WORKSPACE, "gated delta rule: workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : 0, p.bytes);
    DeltaArgs A;
    fill(A, s, p, false, workspace, out_dt, gate_dt, scale);
    A.q = q;
    A.k = k;
    A.v = v;
    A.g = g;
    A.beta = beta;
    A.o = o;
    A.lengths = lengths;
    A.state_in = state_in;
    A.state_out = state_out;
    hipStream_t str = (hipStream_t)stream;
    const dim3 scan(B * H, (unsigned)G.scan_y), chain((unsigned)(G.units * G.nv));
    if ((st = launch("ret_delta_prep", kn.prep, prep_grid(p, s), str, op, A)) != RET_OK) return st;
    if (p.nseg > 1) {
        const dim3 local((unsigned)(G.units * (G.nv + G.nk)));
        if ((st = launch("ret_delta_local", kn.local, local, str, op, A, kn.threads)) != RET_OK) return st;
        if ((st = launch("ret_delta_scan", kn.scan, scan, str, op, A, kn.scan_threads)) != RET_OK) return st;
    }
    return launch("ret_delta_full", out_dt == RET_BF16 ? kn.full : kn.full_f32, chain, str, op, A, kn.threads);
}

size_t ret_gated_delta_bwd_workspace_bytes(int B, int N, int H, int Hk, int dk, int dv, ret_dtype_t in_dt,
                                           const ret_options_t* opts) {
    const Shape s = {B, N, H, Hk, dk, dv};
    DeltaKernels k;
    if (check_shape(s, in_dt, RET_F32, RET_F32, kSeqMaxBH) != RET_OK) return 0;
    if (!delta_kernels_get(in_dt == RET_BF16, dk, dv, &k)) return 0;
    const Plan p = make_plan(s, k, in_dt, in_dt == RET_BF16 ? 2 : 1, resolve(opts));
    Grids G;
    return make_grids(s, p, k, &G) == RET_OK ? p.bytes : 0;
}

ret_status_t ret_gated_delta_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                 const void* dout, void* dq, void* dk_out, void* dv_out, void* dg, void* dbeta, int B,
                                 int N, int H, int Hk, int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt,
                                 ret_dtype_t gate_dt, float scale, const int32_t* lengths, const float* state_in,
                                 const float* dstate_out, float* dstate_in, void* workspace, size_t workspace_bytes,
                                 void* stream, const ret_options_t* opts) {
    const Shape s = {B, N, H, Hk, dk, dv};
    ret_status_t st = check_shape(s, in_dt, out_dt, gate_dt, kSeqMaxBH);
    if (st != RET_OK) return st;
    if (!q || !k || !v || !g || !beta || !dout || !dq || !dk_out || !dv_out || !dg || !dbeta)
        return fail(RET_ERR_INVALID_ARG, "null q/k/v/g/beta/dout or gradient pointer");
    if (!isfinite(scale)) return fail(RET_ERR_INVALID_ARG, "scale is not finite");
    DeltaKernels kn;
    if (!delta_kernels_get(in_dt == RET_BF16, dk, dv, &kn))
        return fail(RET_ERR_UNSUPPORTED, "gated delta gradients: unsupported d_k=%d d_v=%d for %s input", dk, dv,
                    in_dt == RET_F32 ? "F32" : "BF16");
    const Opts op = resolve(opts);
    // gradients in fp32 from bf16 input: their type holds more than one rounding of the chains' states leaves
    const bool two = in_dt == RET_BF16 && (out_dt == RET_F32 || gate_dt == RET_F32);
    const Plan p = make_plan(s, kn, in_dt, two ? 2 : 1, op);
    Grids G;
    if ((st = make_grids(s, p, kn, &G)) != RET_OK) return st;
    const size_t T = (size_t)B * N, ei = esize(in_dt), eo = esize(out_dt), sb = (size_t)B * H * dk * dv * 4;
    const unsigned eg = esize(gate_dt);
    const Buf w[] = {{"dq", dq, T * Hk * dk * eo}, {"dk", dk_out, T * Hk * dk * eo}, {"dv", dv_out, T * H * dv * eo},
                     {"dg", dg, T * H * eg, 0, eg}, {"dbeta", dbeta, T * H * eg, 0, eg}, {"dstate_in", dstate_in, sb},
                     {"the workspace", workspace, workspace_bytes}};
    const Buf r[] = {{"q", q, T * Hk * dk * ei}, {"k", k, T * Hk * dk * ei}, {"v", v, T * H * dv * ei},
                     {"g", g, T * H * eg, 0, eg}, {"beta", beta, T * H * eg, 0, eg}, {"dout", dout, T * H * dv * ei},
                     {"lengths", lengths, (size_t)B * 4, 0, 4}, {"state_in", state_in, sb}, {"dstate_out", dstate_out, sb}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    if (!workspace || workspace_bytes < p.bytes)
        return fail(RET_ERR_WORKSPACE, "gated delta gradients: workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : 0, p.bytes);
    DeltaArgs A;
    fill(A, s, p, true, workspace, out_dt, gate_dt, scale);
    A.q = q;
    A.k = k;
    A.v = v;
    A.g = g;
    A.beta = beta;
    A.dout = dout;
    A.lengths = lengths;
    A.state_in = state_in;
    A.dstate_out = dstate_out;
    A.dstate_in = dstate_in;
    A.dq = dq;
    A.dk_ = dk_out;
    A.dv_ = dv_out;
    A.dg = dg;
    A.dbeta = dbeta;
    hipStream_t str = (hipStream_t)stream;
    const dim3 scan(B * H, (unsigned)G.scan_y), chain((unsigned)(G.units * G.nv));
    if ((st = launch("ret_delta_prep", kn.bprep, prep_grid(p, s), str, op, A)) != RET_OK) return st;
    if (p.nseg > 1) {
        const dim3 local((unsigned)(G.units * (G.nv + G.nk)));
        if ((st = launch("ret_delta_local", kn.blocal, local, str, op, A, kn.threads)) != RET_OK) return st;
        if ((st = launch("ret_delta_scan", kn.scan, scan, str, op, A, kn.scan_threads)) != RET_OK) return st;
    }
    if ((st = launch("ret_delta_states", two ? kn.states2 : kn.states, chain, str, op, A, kn.threads)) != RET_OK) return st;
    if (p.nseg > 1) {
        if ((st = launch("ret_delta_local_bwd", kn.rlocal, chain, str, op, A, kn.threads)) != RET_OK) return st;
        if ((st = launch("ret_delta_scan", kn.rscan, scan, str, op, A, kn.scan_threads)) != RET_OK) return st;
    }
    if ((st = launch("ret_delta_full_bwd", two ? kn.rfull2 : kn.rfull, chain, str, op, A, kn.threads)) != RET_OK) return st;
    const delta_kernel_t grad = H > Hk ? two ? kn.grad_group2 : kn.grad_group : two ? kn.grad2 : kn.grad;
    const int threads = two ? kn.grad2_threads : kn.grad_threads;
    return launch("ret_delta_grad", grad, dim3(p.nchunks, B * Hk), str, op, A, threads);
}

ret_status_t ret_gated_delta_step(const void* q, const void* k, const void* v, const void* g, const void* beta, void* o,
                                  float* state, int B, int H, int Hk, int dk, int dv, ret_dtype_t in_dt,
                                  ret_dtype_t out_dt, ret_dtype_t gate_dt, float scale, void* stream,
                                  const ret_options_t* opts) {
    const Shape s = {B, 1, H, Hk, dk, dv};
    ret_status_t st = check_shape(s, in_dt, out_dt, gate_dt, kStepMaxBH);
    if (st != RET_OK) return st;
    if (!q || !k || !v || !g || !beta || !o || !state)
        return fail(RET_ERR_INVALID_ARG, "null q/k/v/g/beta/o/state pointer");
    if (!isfinite(scale)) return fail(RET_ERR_INVALID_ARG, "scale is not finite");
    const delta_step_kernel_t fn = delta_step_kernel_get(in_dt == RET_BF16, dk);
    if (!fn || dv % 16)
        return fail(RET_ERR_UNSUPPORTED, "gated delta step: d_k=%d not in {16,32,64,128,256} or d_v=%d not a multiple of 16",
                    dk, dv);
    const unsigned long long col_blocks = blocks(dv, 64);
    const int threads = dk >= 32 ? 2 * dk : 64;
    if (!grid_fits(B * H, col_blocks, 1, threads))
        return fail(RET_ERR_UNSUPPORTED, "gated delta step: B=%d H=%d d_v=%d exceed a launch", B, H, dv);
    const size_t ei = esize(in_dt), ng = (size_t)B * H * esize(gate_dt);
    const unsigned eg = esize(gate_dt);
    const Buf w[] = {{"o", o, (size_t)B * H * dv * esize(out_dt)}, {"state", state, (size_t)B * H * dk * dv * 4}};
    const Buf r[] = {{"q", q, (size_t)B * Hk * dk * ei}, {"k", k, (size_t)B * Hk * dk * ei},
                     {"v", v, (size_t)B * H * dv * ei}, {"g", g, ng, 0, eg}, {"beta", beta, ng, 0, eg}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    DeltaStepArgs A = {q, k, v, g, beta, state, o, B, H, Hk, dv, out_dt == RET_BF16, gate_dt == RET_BF16,
                       scale_of(scale, dk)};
    hipStream_t str = (hipStream_t)stream;
    LaunchTimer tm("ret_delta_step", str, resolve(opts));
    hipLaunchKernelGGL(fn, dim3(B * H, (unsigned)col_blocks), dim3(threads), 0, str, A);
    tm.done();
    return launch_status("ret_delta_step");
}

}  // extern "C"
