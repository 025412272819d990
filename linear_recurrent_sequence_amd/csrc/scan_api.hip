// Entry points of the selective scan: argument checks, segment plan, workspace layout, launches.
#include <string.h>

#include <algorithm>

#include "host.h"
#include "rows.h"
#include "scan_bwd.h"
#include "scan_step.h"

namespace ret {

namespace {

size_t esize(ret_dtype_t t) { return t == RET_BF16 ? 2 : 4; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct Shape {
    int B, N, D, S, G;
};

ret_status_t check_shape(const Shape& s, ret_dtype_t in_dt, ret_dtype_t out_dt) {
    if (s.B <= 0 || s.N <= 0 || s.D <= 0 || s.S <= 0 || s.G <= 0)
        return fail(RET_ERR_INVALID_ARG, "sizes must be positive (B=%d N=%d D=%d S=%d G=%d)", s.B, s.N, s.D, s.S, s.G);
    for (ret_dtype_t t : {in_dt, out_dt})
        if (t != RET_F32 && t != RET_BF16) return fail(RET_ERR_INVALID_ARG, "bad dtype %d", (int)t);
    if (in_dt == RET_F32 && out_dt != RET_F32) return fail(RET_ERR_INVALID_ARG, "F32 input requires F32 output");
    if (s.D % s.G) return fail(RET_ERR_INVALID_ARG, "D=%d is not a multiple of G=%d", s.D, s.G);
    if (s.S != 8 && s.S != 16 && s.S != 32 && s.S != 64)
        return fail(RET_ERR_UNSUPPORTED, "selective scan: %d states are not 8, 16, 32 or 64", s.S);
    if (s.G > 1 && s.D / s.G % kScanCh)
        return fail(RET_ERR_UNSUPPORTED, "selective scan: groups of %d channels are not a multiple of %d", s.D / s.G,
                    kScanCh);
    if ((long long)s.B * s.N > 1LL << 36 || s.D > kScanMaxLd || s.N > INT32_MAX - 1024)
        return fail(RET_ERR_UNSUPPORTED, "selective scan: B=%d N=%d D=%d too large", s.B, s.N, s.D);
    return RET_OK;
}

// Rows apart of z, b and c: 0 stands for contiguous.
struct Rows {
    int64_t z, b, c;
};
ret_status_t check_rows(const Shape& s, Rows* r) {
    const int64_t gs = (int64_t)s.G * s.S;
    if (r->z == 0) r->z = s.D;
    if (r->b == 0) r->b = gs;
    if (r->c == 0) r->c = gs;
    if (r->z < s.D || r->b < gs || r->c < gs)
        return fail(RET_ERR_INVALID_ARG, "rows of z, b or c (%lld, %lld, %lld apart) are shorter than they are wide",
                    (long long)r->z, (long long)r->b, (long long)r->c);
    if (r->z > kScanMaxLd || r->b > kScanMaxLd || r->c > kScanMaxLd)
        return fail(RET_ERR_UNSUPPORTED, "rows of z, b or c are more than %lld elements apart", (long long)kScanMaxLd);
    return RET_OK;
}
size_t span(size_t rows, int64_t ld, int64_t width, size_t e) { return ((rows - 1) * ld + width) * e; }

bool vectors(const void* b, const void* c, const Rows& r, ret_dtype_t dt) {
    const uintptr_t a = 4 * esize(dt);
    return (uintptr_t)b % a == 0 && (uintptr_t)c % a == 0 && r.b % 4 == 0 && r.c % 4 == 0;
}

// How a sequence is cut up. Measured nanoseconds a token (bf16, with gate and skip), w the sequences' blocks of 16 channels:
// waves that walk a sequence whole take `walk` each and, all together, walk_all w; workgroups on chunks take `chunk` while the
// card holds them all (chunk_wgs), more in proportion; segments, which go over the tokens twice and start three kernels, take
// 22 us and seg_all w. The least of the three. Examples at 16 states, us (walk, chunks, segments): 512 tokens of 8192 channels
// 65, 38, 47; 8192 of 1024 992, 247, 84; 8192 of 4096 1012, 257, 260; 4 x 512 of 8192 100, 138, 142.
struct Cost {
    float walk, walk_all, chunk, chunk_wgs, seg_all;
};
constexpr Cost kCost[4] = {{99.f, 0.070f, 23.f, 310.f, 0.085f},   // 8 states
                           {122.f, 0.095f, 30.f, 230.f, 0.117f},  // 16
                           {200.f, 0.149f, 78.f, 400.f, 0.186f},  // 32
                           {370.f, 0.258f, 155.f, 378.f, 0.325f}};  // 64
// Waves that the segments are for (8 a SIMD: as many as run at once of the local pass, of the walk 5), tokens of a segment at
// least.
constexpr int kSegWaves = 8192, kSegLeast = 64;

struct Plan {
    bool walk;
    int nseg, seg_tokens, cblocks, wblocks;
    size_t seg_dt, bytes;
};
Plan make_plan(const Shape& s, const ScanKernels& k, const Opts& op) {
    Plan p;
    p.cblocks = (s.D + kScanCh - 1) / kScanCh;
    p.wblocks = (p.cblocks + kWalkWaves - 1) / kWalkWaves;
    const double w = (double)s.B * p.cblocks;
    const Cost& c = kCost[s.S == 8 ? 0 : s.S == 16 ? 1 : s.S == 32 ? 2 : 3];
    const double walk = s.N * std::max<double>(c.walk, c.walk_all * w);
    const double chunk = s.N * (double)c.chunk * std::max(1.0, w / c.chunk_wgs);
    const double seg = 22000.0 + s.N * c.seg_all * w;
    const bool split = op.segments > 1 || (op.segments == 0 && seg < std::min(walk, chunk));
    p.walk = op.variant == 1 || (op.variant != 2 && (split || walk <= chunk));
    const int unit = p.walk ? k.block : k.chunk, units = (s.N + unit - 1) / unit;
    long long n = op.segments > 0 ? op.segments : split ? std::min<long long>((long long)(kSegWaves / w), s.N / kSegLeast) : 1;
    if (n > units) n = units;
    if (n < 1) n = 1;
    const int per = (int)((units + n - 1) / n);
    p.seg_tokens = per * unit;
    p.nseg = (units + per - 1) / per;
    const size_t ds = (size_t)s.B * p.nseg * s.D;
    p.seg_dt = p.nseg > 1 ? round256(ds * s.S * 4) : 0;
    p.bytes = p.seg_dt + (p.nseg > 1 ? round256(ds * 4) : 256);
    return p;
}

// The gradients' local pass: from so many waves for each token of a chunk on, a wave does a chunk alone, which saves the join
// of the 8 (32 and 64 states: 4) that share a chunk below. Together and alone, us, at 16 states and 512 x 512 tokens x channels
// 8, 28; 2048 x 2048 26, 29; 4096 x 4096 91, 87; 2 x 2048 x 8192 190, 174; at 64 states 256 x 2048 24, 19; at 32 1024 x 2048
// 26, 24.
constexpr long long kLocalWaves = 40;

// Chunks of the gradients, and blocks of channels that a workgroup does one after another: the more, the smaller the partial
// sums of dB and dC, while about four workgroups a CU are left.
struct BwdPlan {
    int nchunks, blocks_g, parts_g, cblocks, lblocks;
    bool split;
    size_t seg_g, seg_dt, part_a, part_bc, bytes;
};
BwdPlan make_bwd_plan(const Shape& s, int chunk, int waves) {
    BwdPlan p;
    p.cblocks = (s.D + kScanCh - 1) / kScanCh;
    p.nchunks = (s.N + chunk - 1) / chunk;
    p.split = (long long)s.B * p.nchunks * p.cblocks < kLocalWaves * chunk;
    p.lblocks = p.split ? p.cblocks : (p.cblocks + waves - 1) / waves;
    p.blocks_g = (s.D / s.G + kScanCh - 1) / kScanCh;
    const long long units = (long long)s.B * p.nchunks * s.G * p.blocks_g;
    long long run = units / 1024;
    run = run < 1 ? 1 : run > 32 ? 32 : run;
    if (run > p.blocks_g) run = p.blocks_g;
    p.parts_g = (int)((p.blocks_g + run - 1) / run);
    const size_t dk = (size_t)s.B * p.nchunks * s.D;
    p.seg_g = round256(dk * s.S * 4);
    p.seg_dt = p.seg_g + round256(dk * s.S * 4);
    p.part_a = p.seg_dt + round256(dk * 4);
    p.part_bc = p.part_a + round256(dk * (s.S + 2) * 4);
    p.bytes = p.part_bc + round256((size_t)s.G * p.parts_g * s.B * s.N * 2 * s.S * 4);
    return p;
}

// How workgroups are dealt to the 8 XCDs. Without lengths: each gets a range. With lengths that would leave the XCDs that have
// the short sequences idle: where there are many segments they are dealt in turn; else the units of `channels` channels are, if
// that leaves lines of 128 bytes in one piece. Ranges and dealt, us, at 16 states, 8192 channels and sequences of 2741, 1500, 900
// and 100 tokens: forward 472, 410 (units; whole sequences take 475), gradients 2200, 1208 (segments; 2030 where only the units
// of the local pass can be dealt; whole ones take 2167). 4096 and 500 tokens of 1024 channels forward 79, 58.
constexpr long long kDealSegsLeast = 32;
ScanDeal deal(const int32_t* lengths, long long segs, int units, int channels, size_t e) {
    if (!lengths) return kDealRanges;
    if (segs >= kDealSegsLeast) return kDealSegs;
    return units % 8 == 0 && units / 8 * channels * e % 128 == 0 ? kDealUnits : kDealRanges;
}
unsigned long long deal_grid(ScanDeal d, int nseg, int B, int units) {
    const unsigned long long segs = (unsigned long long)deal_segs(d, nseg) * B;
    return d == kDealSegs ? (segs + 7) / 8 * 8 * units : (segs * units + 7) / 8 * 8;
}

// Grids and whether they fit; those that are dealt by deal() at their largest.
struct Grids {
    unsigned long long join, bc, cols;
};
ret_status_t fits(const Shape& s, bool ok) {
    if (ok) return RET_OK;
    return fail(RET_ERR_UNSUPPORTED, "selective scan: B=%d N=%d D=%d S=%d exceed a launch", s.B, s.N, s.D, s.S);
}
ret_status_t fwd_grids(const Shape& s, const Plan& p, const ScanKernels& k, Grids* g) {
    g->join = ((unsigned long long)s.D * s.S + 255) / 256;
    return fits(s, grid_fits(deal_grid(kDealSegs, p.nseg, s.B, p.wblocks), 1, 1, 64 * kWalkWaves) &&
                       (p.walk || grid_fits(deal_grid(kDealSegs, p.nseg, s.B, p.cblocks), 1, 1, k.threads)) &&
                       (p.nseg == 1 || grid_fits(g->join, s.B, 1, 256)));
}
ret_status_t bwd_grids(const Shape& s, const BwdPlan& p, int threads, Grids* g) {
    const long long segs = (long long)p.nchunks * s.B;
    g->join = ((unsigned long long)s.D * s.S + 255) / 256;
    g->bc = ((unsigned long long)s.B * s.N * 2 * s.S * s.G + kColSumThreads - 1) / kColSumThreads;
    g->cols = ((unsigned long long)s.D * (s.S + 2) + kColSumCols - 1) / kColSumCols;
    return fits(s, grid_fits(g->join, s.B, 2, 256) &&
                       grid_fits(deal_grid(kDealSegs, p.nchunks, s.B, p.lblocks), 1, 1, threads) &&
                       grid_fits(deal_grid(kDealSegs, p.nchunks, s.B, p.parts_g * s.G), 1, 1, threads) &&
                       grid_fits(g->bc + g->cols, 1, 1, kColSumThreads) && segs <= INT32_MAX / 2);
}

template <class K, class A>
ret_status_t launch(const char* name, K fn, dim3 grid, int threads, hipStream_t s, const Opts& op, const A& args) {
    LaunchTimer tm(name, s, op);
    hipLaunchKernelGGL(fn, grid, dim3(threads), 0, s, args);
    tm.done();
    return launch_status(name);
}

}  // namespace

}  // namespace ret

using namespace ret;

extern "C" {

size_t ret_selective_scan_workspace_bytes(int B, int N, int D, int S, int G, ret_dtype_t in_dt,
                                          const ret_options_t* opts) {
    const Shape s = {B, N, D, S, G};
    ScanKernels k;
    Grids g;
    if (check_shape(s, in_dt, RET_F32) != RET_OK || !scan_kernels_get(in_dt == RET_BF16, false, S, &k)) return 0;
    const Plan p = make_plan(s, k, resolve(opts));
    return fwd_grids(s, p, k, &g) == RET_OK ? p.bytes : 0;
}

ret_status_t ret_selective_scan_fwd(const void* u, const void* dt, const float* A, const void* b, int64_t b_ld,
                                    const void* c, int64_t c_ld, const float* d_skip, const void* z, int64_t z_ld,
                                    const float* dt_bias, void* y, int B, int N, int D, int S, int G, ret_dtype_t in_dt,
                                    ret_dtype_t out_dt, int softplus, const int32_t* lengths, const float* state_in,
                                    float* state_out, void* workspace, size_t workspace_bytes, void* stream,
                                    const ret_options_t* opts) {
    const Shape s = {B, N, D, S, G};
    Rows ld = {z_ld, b_ld, c_ld};
    ret_status_t st = check_shape(s, in_dt, out_dt);
    if (st != RET_OK || (st = check_rows(s, &ld)) != RET_OK) return st;
    if (!u || !dt || !A || !b || !c || !y) return fail(RET_ERR_INVALID_ARG, "null u/dt/A/b/c/y pointer");
    ScanKernels k;
    scan_kernels_get(in_dt == RET_BF16, out_dt == RET_BF16, S, &k);
    const Opts op = resolve(opts);
    const Plan p = make_plan(s, k, op);
    Grids g;
    if ((st = fwd_grids(s, p, k, &g)) != RET_OK) return st;
    const size_t rows = (size_t)B * N, e = esize(in_dt), sb = (size_t)B * D * S * 4, gs = (size_t)G * S;
    const unsigned ei = e, eo = esize(out_dt);
    const bool split = p.nseg > 1;
    // state_out may be state_in (r[8]): a workgroup reads its part before it writes it
    const Buf w[] = {{"y", y, rows * D * eo, 0, eo}, {"state_out", state_out, sb, 1u << 8},
                     {"the workspace", workspace, split ? workspace_bytes : 0}};
    const Buf r[] = {{"u", u, rows * D * e, 0, ei}, {"dt", dt, rows * D * e, 0, ei}, {"A", A, (size_t)D * S * 4},
                     {"b", b, span(rows, ld.b, gs, e), 0, ei}, {"c", c, span(rows, ld.c, gs, e), 0, ei},
                     {"d_skip", d_skip, (size_t)D * 4, 0, 4}, {"z", z, z ? span(rows, ld.z, D, e) : 0, 0, ei},
                     {"dt_bias", dt_bias, (size_t)D * 4, 0, 4}, {"state_in", state_in, sb},
                     {"lengths", lengths, (size_t)B * 4, 0, 4}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    if (split && (!workspace || workspace_bytes < p.bytes))
        return fail(RET_ERR_WORKSPACE, "selective scan: workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : 0, p.bytes);
    ScanArgs a;
    memset(&a, 0, sizeof(a));
    a.u = u, a.dt = dt, a.z = z, a.b = b, a.c = c, a.A = A, a.skip = d_skip, a.bias = dt_bias, a.lengths = lengths;
    a.state_in = state_in, a.state_out = state_out, a.y = y;
    a.seg_h = (float*)workspace, a.seg_dt = (float*)((char*)workspace + p.seg_dt);
    a.ldz = ld.z, a.ldb = ld.b, a.ldc = ld.c;
    a.B = B, a.N = N, a.D = D, a.G = G, a.nseg = p.nseg, a.seg_tokens = p.seg_tokens, a.cblocks = p.wblocks;
    a.softplus = softplus != 0, a.bc_vec = vectors(b, c, ld, in_dt);
    const long long segs = (long long)p.nseg * B;
    const ScanDeal dl = deal(lengths, segs, p.wblocks, kWalkWaves * kScanCh, e);
    const dim3 waves((unsigned)deal_grid(dl, p.nseg, B, p.wblocks));
    a.deal = dl;
    hipStream_t sm = (hipStream_t)stream;
    if (split) {
        if ((st = launch("ret_scan_local", k.local, waves, 64 * kWalkWaves, sm, op, a)) != RET_OK) return st;
        if ((st = launch("ret_scan_join", k.join, dim3((unsigned)g.join, B), 256, sm, op, a)) != RET_OK) return st;
    }
    if (p.walk) return launch("ret_scan_walk", k.walk, waves, 64 * kWalkWaves, sm, op, a);
    const ScanDeal dc = deal(lengths, segs, p.cblocks, kScanCh, e);
    a.cblocks = p.cblocks, a.deal = dc;
    return launch("ret_scan_chunks", k.chunks, dim3((unsigned)deal_grid(dc, p.nseg, B, p.cblocks)), k.threads, sm, op, a);
}

ret_status_t ret_selective_scan_step(const void* u, const void* dt, const float* A, const void* b, int64_t b_ld,
                                     const void* c, int64_t c_ld, const float* d_skip, const void* z, int64_t z_ld,
                                     const float* dt_bias, void* y, float* state, int B, int D, int S, int G,
                                     ret_dtype_t in_dt, ret_dtype_t out_dt, int softplus, void* stream,
                                     const ret_options_t* opts) {
    const Shape s = {B, 1, D, S, G};
    Rows ld = {z_ld, b_ld, c_ld};
    ret_status_t st = check_shape(s, in_dt, out_dt);
    if (st != RET_OK || (st = check_rows(s, &ld)) != RET_OK) return st;
    if (!u || !dt || !A || !b || !c || !y || !state) return fail(RET_ERR_INVALID_ARG, "null u/dt/A/b/c/y/state pointer");
    const int per = 1024 / S;
    const unsigned long long blocks = (D + per - 1) / per;
    // several sequences a workgroup while enough workgroups are left
    int seqs = 1;
    while (seqs < kScanStepSeqs && blocks * ((B + 2 * seqs - 1) / (2 * seqs)) >= kScanStepWgs) seqs *= 2;
    const unsigned long long wgs = blocks * ((B + seqs - 1) / seqs);
    if ((st = fits(s, grid_fits(wgs, 1, 1, 256))) != RET_OK) return st;
    const size_t n = (size_t)B * D, e = esize(in_dt), gs = (size_t)G * S;
    const unsigned ei = e, eo = esize(out_dt);
    const Buf w[] = {{"y", y, n * eo, 0, eo}, {"state", state, n * S * 4}};
    const Buf r[] = {{"u", u, n * e, 0, ei}, {"dt", dt, n * e, 0, ei}, {"A", A, (size_t)D * S * 4},
                     {"b", b, span(B, ld.b, gs, e), 0, ei}, {"c", c, span(B, ld.c, gs, e), 0, ei},
                     {"d_skip", d_skip, (size_t)D * 4, 0, 4}, {"z", z, z ? span(B, ld.z, D, e) : 0, 0, ei},
                     {"dt_bias", dt_bias, (size_t)D * 4, 0, 4}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    ScanStepArgs a = {u, dt, z, b, c, A, d_skip, dt_bias, state, y, ld.z, ld.b, ld.c, B, D, G, (int)blocks, seqs, softplus != 0,
                      vectors(b, c, ld, in_dt)};
    return launch("ret_scan_step", scan_step_kernel_get(in_dt == RET_BF16, out_dt == RET_BF16, S),
                  dim3((unsigned)wgs), 256, (hipStream_t)stream, resolve(opts), a);
}

size_t ret_selective_scan_bwd_workspace_bytes(int B, int N, int D, int S, int G, ret_dtype_t in_dt) {
    const Shape s = {B, N, D, S, G};
    ScanBwdKernels k;
    Grids g;
    if (check_shape(s, in_dt, RET_F32) != RET_OK || !scan_bwd_kernels_get(in_dt == RET_BF16, false, S, &k)) return 0;
    const BwdPlan p = make_bwd_plan(s, k.chunk, k.waves);
    return bwd_grids(s, p, 64 * k.waves, &g) == RET_OK ? p.bytes : 0;
}

ret_status_t ret_selective_scan_bwd(const void* u, const void* dt, const float* A, const void* b, int64_t b_ld,
                                    const void* c, int64_t c_ld, const float* d_skip, const void* z, int64_t z_ld,
                                    const float* dt_bias, const void* dy, void* du, void* ddt, float* dA, void* db,
                                    void* dc, float* dd_skip, void* dz, float* ddt_bias, int B, int N, int D, int S, int G,
                                    ret_dtype_t in_dt, ret_dtype_t out_dt, int softplus, const int32_t* lengths,
                                    const float* state_in, const float* dstate_out, float* dstate_in, void* workspace,
                                    size_t workspace_bytes, void* stream, const ret_options_t* opts) {
    const Shape s = {B, N, D, S, G};
    Rows ld = {z_ld, b_ld, c_ld};
    ret_status_t st = check_shape(s, in_dt, out_dt);
    if (st != RET_OK || (st = check_rows(s, &ld)) != RET_OK) return st;
    if (!u || !dt || !A || !b || !c || !dy || !du || !ddt || !db || !dc)
        return fail(RET_ERR_INVALID_ARG, "null u/dt/A/b/c/dy/du/ddt/db/dc pointer");
    if (dz && !z) return fail(RET_ERR_INVALID_ARG, "dz without z");
    if (dd_skip && !d_skip) return fail(RET_ERR_INVALID_ARG, "dd_skip without d_skip");
    ScanBwdKernels k;
    scan_bwd_kernels_get(in_dt == RET_BF16, out_dt == RET_BF16, S, &k);
    const Opts op = resolve(opts);
    const BwdPlan p = make_bwd_plan(s, k.chunk, k.waves);
    Grids g;
    if ((st = bwd_grids(s, p, 64 * k.waves, &g)) != RET_OK) return st;
    const size_t rows = (size_t)B * N, e = esize(in_dt), sb = (size_t)B * D * S * 4, gs = (size_t)G * S, nd = (size_t)D * 4;
    const unsigned ei = e, eo = esize(out_dt);
    const Buf w[] = {{"du", du, rows * D * eo, 0, eo}, {"ddt", ddt, rows * D * eo, 0, eo}, {"dA", dA, nd * S, 0, 4},
                     {"db", db, rows * gs * eo, 0, eo}, {"dc", dc, rows * gs * eo, 0, eo}, {"dd_skip", dd_skip, nd, 0, 4},
                     {"dz", dz, rows * D * eo, 0, eo}, {"ddt_bias", ddt_bias, nd, 0, 4}, {"dstate_in", dstate_in, sb},
                     {"the workspace", workspace, workspace_bytes}};
    const Buf r[] = {{"u", u, rows * D * e, 0, ei}, {"dt", dt, rows * D * e, 0, ei}, {"A", A, nd * S},
                     {"b", b, span(rows, ld.b, gs, e), 0, ei}, {"c", c, span(rows, ld.c, gs, e), 0, ei},
                     {"d_skip", d_skip, nd, 0, 4}, {"z", z, z ? span(rows, ld.z, D, e) : 0, 0, ei},
                     {"dt_bias", dt_bias, nd, 0, 4}, {"dy", dy, rows * D * e, 0, ei}, {"state_in", state_in, sb},
                     {"dstate_out", dstate_out, sb}, {"lengths", lengths, (size_t)B * 4, 0, 4}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    if (!workspace || workspace_bytes < p.bytes)
        return fail(RET_ERR_WORKSPACE, "selective scan gradients: workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : 0, p.bytes);
    ScanBwdArgs a;
    memset(&a, 0, sizeof(a));
    ScanArgs& f = a.f;
    f.u = u, f.dt = dt, f.z = z, f.b = b, f.c = c, f.A = A, f.skip = d_skip, f.bias = dt_bias, f.lengths = lengths;
    f.state_in = state_in, f.seg_h = (float*)workspace, f.seg_dt = (float*)((char*)workspace + p.seg_dt);
    f.ldz = ld.z, f.ldb = ld.b, f.ldc = ld.c;
    f.B = B, f.N = N, f.D = D, f.G = G, f.nseg = p.nchunks, f.seg_tokens = k.chunk, f.cblocks = p.lblocks;
    f.softplus = softplus != 0, f.bc_vec = vectors(b, c, ld, in_dt);
    const long long segs = (long long)p.nchunks * B;
    const ScanDeal dl = deal(lengths, segs, p.lblocks, p.split ? kScanCh : k.waves * kScanCh, e);
    const ScanDeal dg = deal(lengths, segs, p.parts_g * G, kScanCh, e);
    f.deal = dl, a.deal_parts = dg;
    a.dy = dy, a.dstate_out = dstate_out, a.dstate_in = dstate_in;
    a.seg_g = (float*)((char*)workspace + p.seg_g);
    a.part_a = (float*)((char*)workspace + p.part_a), a.part_bc = (float*)((char*)workspace + p.part_bc);
    a.du = du, a.ddt = ddt, a.dz = dz, a.db = db, a.dc = dc, a.parts_g = p.parts_g;
    a.bc_blocks = (unsigned)g.bc;
    a.cols = {a.part_a, dA, dd_skip, ddt_bias, (long long)D * (S + 2), (long long)D * S, D, B * p.nchunks};
    const bool cols = dA || dd_skip || ddt_bias;
    hipStream_t sm = (hipStream_t)stream;
    if ((st = launch("ret_scan_local_bwd", p.split ? k.local_split : k.local,
                     dim3((unsigned)deal_grid(dl, p.nchunks, B, p.lblocks)), 64 * k.waves, sm, op, a)) != RET_OK)
        return st;
    if ((st = launch("ret_scan_join_bwd", k.join, dim3((unsigned)g.join, B, 2), 256, sm, op, a)) != RET_OK) return st;
    if ((st = launch("ret_scan_grad", k.grad, dim3((unsigned)deal_grid(dg, p.nchunks, B, p.parts_g * G)), 64 * k.waves, sm, op,
                     a)) != RET_OK)
        return st;
    return launch("ret_scan_sums", k.sums, dim3((unsigned)(g.bc + (cols ? g.cols : 0))), kColSumThreads, sm, op, a);
}

}  // extern "C"
