// Short causal convolution per channel, with the activation fused: forward, gradients and one token.
//
//   x~ = the W - 1 inputs before the sequence (the state, or zeros), then x
//   pre_t = bias + sum_{j < W} w[j] x~_{t - W + 1 + j},  y_t = act(pre_t),  act the identity or silu
//   dpre_t = dy_t act'(pre_t),  dx~_t = sum_j w[j] dpre_{t + W - 1 - j},  dw[j] = sum_t dpre_t x~_{t - W + 1 + j}
//
// A thread owns V neighbouring channels and walks a strip of tokens with the last W - 1 inputs (and, for the gradients, the
// last W dpre) in registers, so that a strip reads its tokens once and W - 1 (2 W - 2) more of its neighbours'. Each kernel
// reads and writes its tensors once and is bound by HBM. The gradients' sums over tokens stay in registers over a
// workgroup's strips, meet in LDS and leave one partial row per workgroup, added up in a fixed order by a second kernel.
// 4 x 2048 tokens of 8192 channels, width 4: gradients 94 to 96 us in bf16, 5 of them for the sums, 4.5 TB/s of the 5.1 that a
// large copy reaches (the rows before and behind a strip come twice, mostly from L2); 214 in fp32, 132 in bf16 where 8190
// channels go one by one. 3 x 2741 tokens forward 66 us, in fp32 115.
#include <algorithm>

#include "host.h"
#include "rows.h"

namespace ret {

namespace {

// Tokens of a strip, at most, where the card is full, and at least: shorter ones where there are few, so that they run at
// once. Channels a thread: 4 (8 bytes of bf16), which leaves registers for more waves. Measured with 8192 channels in bf16,
// width 4: 4 x 2048 tokens back 97 us at 4 channels and strips of 128, 113 and 114 at 8 and 64; 108 at 4 and 64; 3 x 2741
// ragged ones forward 58 at 4 and 64, 61 at 4 and 32, 65 at 8 and 32.
constexpr int kConvStrip = 64, kConvStripLeast = 8, kConvBwdStrip = 128, kConvBwdStripLeast = 16;
constexpr int kConvWaves = 4;      // waves of a workgroup, each its own strips of the same 64 V channels
constexpr int kConvV = 4;  // channels a thread where rows move as vectors
// Sequences a thread of the single-token kernel, while so many workgroups are left: 128 sequences of 8192 channels 6.2 us with
// two, 7.0 with one, 7.8 and 9.7 with two and one at 8 channels a thread.
constexpr int kConvStepSeqs = 4, kConvStepWgs = 512;

struct ConvArgs {
    const void* x;          // rows of ld elements
    const float *w, *bias;  // [D][W], [D] or null
    const void* state_in;   // [B][W - 1][D], x's dtype, or null
    void* y;                // [B][N][D]
    void* state_out;        // as state_in, or null
    const int32_t* lengths;
    long long ld;
    int B, N, D, silu, strip, strips, cblocks;  // tokens of a strip, strips of a sequence
};
struct ConvBwdArgs {
    const void *dy, *x;
    const float *w, *bias;
    const void* state_in;
    const void* dstate_out;  // [B][W - 1][D], dx's dtype, or null
    void *dx, *dstate_in;
    float* partial;          // [parts][(W + 1) D]: dw, then dbias; or null
    const int32_t* lengths;
    long long ld;
    int B, N, D, silu, strip, strips, cblocks, parts;
};
struct ConvStepArgs {
    const void* x;
    const float *w, *bias;
    void *state, *y;
    long long ld;
    int B, D, silu, cblocks, seqs;
};

// V channels' weights [V][W] as w[j][v], and biases.
template <int V, int W>
__device__ __forceinline__ void load_weights(const float* w, const float* bias, long long c, int D, float (&o)[W][V],
                                             float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) o[j][v] = c < D ? w[(c + v) * W + j] : 0.f;
        b[v] = bias && c < D ? bias[c + v] : 0.f;
    }
}

// V values of a row as they lie in memory, so that a load is not waited for before its values are used.
template <int V, bool BF>
struct ConvRaw {
    typedef uint32_t word __attribute__((ext_vector_type(V / 2)));
    word r;
    __device__ __forceinline__ void load(const void* p, long long i) { r = *reinterpret_cast<const word*>((const uint16_t*)p + i); }
    __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            f[2 * e] = __uint_as_float(r[e] << 16);
            f[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
        }
    }
};
template <>
struct ConvRaw<1, true> {
    uint32_t r;
    __device__ __forceinline__ void load(const void* p, long long i) { r = ((const uint16_t*)p)[i]; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __uint_as_float(r << 16); }
};
template <int V>
struct ConvRaw<V, false> {  // fp32
    float r[V];
    __device__ __forceinline__ void load(const void* p, long long i) { row_load<V>(p, i, false, r); }
    __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = r[e];
    }
};

// Token t of x~ (t >= 1 - W) for V channels from c; zeros from n on.
template <int V, bool XB>
__device__ __forceinline__ void load_x(const void* x, const void* state, long long row0, long long ld, long long srow0,
                                       int D, long long c, int W, int t, int n, float (&f)[V]) {
    if (t >= 0 && t < n) {
        row_load<V>(x, (row0 + t) * ld + c, XB, f);
    } else if (t < 0 && state) {
        row_load<V>(state, (srow0 + W - 1 + t) * D + c, XB, f);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.f;
    }
}

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// The last four tokens of x~ are in a ring of four slots, token t0 + k in slot k % 4; four tokens a round, those of the next
// round asked for before this one's are used.
template <int V, int W, bool XB, bool YB>
__global__ __launch_bounds__(64 * kConvWaves) void conv_fwd_kernel(ConvArgs a) {
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cb = blockIdx.x % a.cblocks, rest = blockIdx.x / a.cblocks;
    const int groups = (a.strips + kConvWaves - 1) / kConvWaves;
    const int b = rest / groups, strip = rest % groups * kConvWaves + wv;
    const long long c = ((long long)cb * 64 + lane) * V;
    if (strip >= a.strips || c >= a.D) return;
    const int n = length_of(a.lengths, b, a.N), t0 = strip * a.strip;
    const int t1 = a.N - t0 < a.strip ? a.N : t0 + a.strip, live1 = t1 < n ? t1 : n;
    const long long row0 = (long long)b * a.N, srow0 = (long long)b * (W - 1);
    float w[W][V], bias[V], x[4][V];
    ConvRaw<V, XB> next[4];
    if (t0 < live1)
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i].load(a.x, (row0 + (t0 + i < n ? t0 + i : n - 1)) * a.ld + c);
    load_weights<V, W>(a.w, a.bias, c, a.D, w, bias);
#pragma unroll
    for (int i = 1; i < W; ++i)
        load_x<V, XB>(a.x, a.state_in, row0, a.ld, srow0, a.D, c, W, t0 - i, n, x[4 - i]);
    if (strip == 0 && a.state_out) {
        // the last W - 1 of x~ before token n; what of the old state stays is read before anything is written
        float s[W - 1][V];
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            load_x<V, XB>(a.x, a.state_in, row0, a.ld, srow0, a.D, c, W, n - (W - 1) + i, n, s[i]);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) row_store<V>(a.state_out, (srow0 + i) * a.D + c, XB, s[i]);
    }
    for (int t = t0; t < live1; t += 4) {
        ConvRaw<V, XB> now[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) now[i] = next[i];
        if (t + 4 < live1)
#pragma unroll
            for (int i = 0; i < 4; ++i) next[i].load(a.x, (row0 + (t + 4 + i < n ? t + 4 + i : n - 1)) * a.ld + c);
        auto round = [&](auto whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!decltype(whole)::value && t + k >= live1) break;
                now[k].get(x[k]);
                float y[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    y[v] = bias[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) y[v] = fmaf(w[j][v], x[(k - (W - 1) + j) & 3][v], y[v]);
                    if (a.silu) y[v] *= sigmoid_hw(y[v]);
                }
                row_store<V>(a.y, (row0 + t + k) * a.D + c, YB, y);
            }
        };
        if (t + 4 <= live1) round(Yes());
        else round(No());
    }
    float zero[V];
#pragma unroll
    for (int v = 0; v < V; ++v) zero[v] = 0.f;
    for (int t = live1 > t0 ? live1 : t0; t < t1; ++t) row_store<V>(a.y, (row0 + t) * a.D + c, YB, zero);
}

// Strips of a workgroup's waves: part p takes strips p kConvWaves + wave, then every parts kConvWaves further, over all
// sequences. A strip yields dx of tokens t0 - (W - 1) .. t1 - W: with dpre from t0 on that needs the W - 1 dpre before t0,
// computed again; the last strip of a sequence goes on to the end of dx with dpre of zero, the first starts in the state.
// Three waves a SIMD: of vectors at width 4 that spills 1 register in bf16, 6 with fp32 outputs and 77 in fp32 (120 bytes a
// lane), and 2 at width 3 in fp32.
template <int V, int W, bool XB, bool YB>
__global__ __launch_bounds__(64 * kConvWaves, 3) void conv_bwd_kernel(ConvBwdArgs a) {
    __shared__ float meet[kConvWaves - 1][64][V];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cb = blockIdx.x % a.cblocks, part = blockIdx.x / a.cblocks;
    const long long c = ((long long)cb * 64 + lane) * V;
    const bool in = c < a.D;
    float w[W][V], bias[V], dw[W][V], db[V];
    load_weights<V, W>(a.w, a.bias, c, a.D, w, bias);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    const long long all = (long long)a.B * a.strips;
    for (long long id = (long long)part * kConvWaves + wv; in && id < all; id += (long long)a.parts * kConvWaves) {
        const int b = (int)(id / a.strips), strip = (int)(id % a.strips);
        const int n = length_of(a.lengths, b, a.N), t0 = strip * a.strip;
        const bool last = strip == a.strips - 1;
        const int to = last ? a.N + W - 1 : t0 + a.strip;  // dpre of tokens t0 .. to
        const int whole = n < to ? n : to;
        const long long row0 = (long long)b * a.N, srow0 = (long long)b * (W - 1);
        float x[4][V], g[4][V];  // rings as in the forward: x~ and dpre
        ConvRaw<V, XB> nx[4], ny[4];
        auto ask = [&](int t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long row = row0 + (t + i < n ? t + i : n - 1);
                nx[i].load(a.x, row * a.ld + c);
                ny[i].load(a.dy, row * a.D + c);
            }
        };
        if (t0 < whole) ask(t0);
        // g[k] from dy: times act'(pre)
        auto through = [&](int k) {
            if (!a.silu) return;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float pre = bias[v];
#pragma unroll
                for (int j = 0; j < W; ++j) pre = fmaf(w[j][v], x[(k - (W - 1) + j) & 3][v], pre);
                const float s = sigmoid_hw(pre);
                g[k & 3][v] *= s * fmaf(pre, 1.f - s, 1.f);
            }
        };
        const int from = strip == 0 ? 0 : t0 - (W - 1);
        // x~ and dpre before t0
        {
            float before[W - 1][V];
#pragma unroll
            for (int i = 1; i < W; ++i)
                load_x<V, XB>(a.x, a.state_in, row0, a.ld, srow0, a.D, c, W, t0 - i, n, x[4 - i]);
            if (from < t0) {
                float y[W - 1][V];
#pragma unroll
                for (int i = 1; i < W; ++i) {
                    load_x<V, XB>(a.x, nullptr, row0, a.ld, srow0, a.D, c, W, t0 - (W - 1) - i, n, before[i - 1]);
                    load_x<V, XB>(a.dy, nullptr, row0, a.D, srow0, a.D, c, W, t0 - i, n, y[i - 1]);
                }
#pragma unroll
                for (int i = 1; i < W; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float d = y[i - 1][v];
                        if (a.silu) {
                            float pre = bias[v];
#pragma unroll
                            for (int j = 0; j < W; ++j) {  // token t0 - i - (W - 1) + j
                                const int back = i + W - 1 - j;
                                pre = fmaf(w[j][v], back < W ? x[(4 - back) & 3][v] : before[back >= W ? back - W : 0][v], pre);
                            }
                            const float s = sigmoid_hw(pre);
                            d *= s * fmaf(pre, 1.f - s, 1.f);
                        }
                        g[4 - i][v] = d;
                    }
            } else {
#pragma unroll
                for (int i = 1; i < W; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) g[4 - i][v] = 0.f;
            }
        }
        for (int t = t0; t < to; t += 4) {
            ConvRaw<V, XB> x0[4], y0[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x0[i] = nx[i], y0[i] = ny[i];
            if (t + 4 < whole) ask(t + 4);
            auto round = [&](auto all_there) {
                constexpr bool ALL = decltype(all_there)::value;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = t + k;
                    if (!ALL && at >= to) break;
                    if (ALL || at < n) {
                        x0[k].get(x[k]);
                        y0[k].get(g[k]);
                        through(k);
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            db[v] += g[k][v];
#pragma unroll
                            for (int j = 0; j < W; ++j)
                                dw[j][v] = fmaf(g[k][v], x[(k - (W - 1) + j) & 3][v], dw[j][v]);
                        }
                    } else {
#pragma unroll
                        for (int v = 0; v < V; ++v) x[k][v] = g[k][v] = 0.f;
                    }
                    float d[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        d[v] = 0.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) d[v] = fmaf(w[j][v], g[(k - j) & 3][v], d[v]);
                    }
                    const int o = at - (W - 1);  // the token that has all its dpre now
                    if (!ALL && o < n && a.dstate_out && o >= n - (W - 1)) {
                        float s[V];
                        row_load<V>(a.dstate_out, (srow0 + o - (n - (W - 1))) * a.D + c, YB, s);
#pragma unroll
                        for (int v = 0; v < V; ++v) d[v] += s[v];
                    }
                    if (ALL || o >= 0) {
                        if (!ALL && o >= n)
#pragma unroll
                            for (int v = 0; v < V; ++v) d[v] = 0.f;
                        row_store<V>(a.dx, (row0 + o) * a.D + c, YB, d);
                    } else if (a.dstate_in) {
                        row_store<V>(a.dstate_in, (srow0 + o + W - 1) * a.D + c, YB, d);
                    }
                }
            };
            if (t >= W - 1 && t + 4 <= whole) round(Yes());
            else round(No());
        }
    }
    if (!a.partial) return;
    float* out = a.partial + (long long)part * (W + 1) * a.D;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float(&mine)[V] = j < W ? dw[j < W ? j : 0] : db;
        __syncthreads();
        if (wv > 0)
#pragma unroll
            for (int v = 0; v < V; ++v) meet[wv - 1][lane][v] = mine[v];
        __syncthreads();
        if (wv == 0 && in)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float s = mine[v];
#pragma unroll
                for (int i = 0; i < kConvWaves - 1; ++i) s += meet[i][lane][v];
                if (j < W) out[(c + v) * W + j] = s;
                else out[(long long)W * a.D + c + v] = s;
            }
    }
}

// A thread owns V channels of `seqs` sequences (at most kConvStepSeqs), so that its weights are read once for all of them.
template <int V, int W, bool XB, bool YB>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepArgs a) {
    const int b0 = blockIdx.x / a.cblocks * a.seqs;
    const long long c = ((long long)(blockIdx.x % a.cblocks) * 256 + threadIdx.x) * V;
    if (c >= a.D) return;
    ConvRaw<V, XB> r[kConvStepSeqs][W];
#pragma unroll
    for (int e = 0; e < kConvStepSeqs; ++e) {
        const int b = b0 + e;
        if (e >= a.seqs || b >= a.B) break;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) r[e][i].load(a.state, ((long long)b * (W - 1) + i) * a.D + c);
        r[e][W - 1].load(a.x, b * a.ld + c);
    }
    float w[W][V], bias[V];
    load_weights<V, W>(a.w, a.bias, c, a.D, w, bias);
#pragma unroll
    for (int e = 0; e < kConvStepSeqs; ++e) {
        const int b = b0 + e;
        if (e >= a.seqs || b >= a.B) break;
        float x[W][V], y[V];
#pragma unroll
        for (int i = 0; i < W; ++i) r[e][i].get(x[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            y[v] = bias[v];
#pragma unroll
            for (int j = 0; j < W; ++j) y[v] = fmaf(w[j][v], x[j][v], y[v]);
            if (a.silu) y[v] *= sigmoid_hw(y[v]);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) row_store<V>(a.state, ((long long)b * (W - 1) + i) * a.D + c, XB, x[i + 1]);
        row_store<V>(a.y, (long long)b * a.D + c, YB, y);
    }
}

typedef void (*conv_fwd_t)(ConvArgs);
typedef void (*conv_bwd_t)(ConvBwdArgs);
typedef void (*conv_step_t)(ConvStepArgs);
struct ConvKernels {
    conv_fwd_t fwd;
    conv_bwd_t bwd;
    conv_step_t step;
};

template <int V, int W>
ConvKernels conv_of_types(bool xb, bool yb) {
    if (!xb) return {conv_fwd_kernel<V, W, false, false>, conv_bwd_kernel<V, W, false, false>, conv_step_kernel<V, W, false, false>};
    if (yb) return {conv_fwd_kernel<V, W, true, true>, conv_bwd_kernel<V, W, true, true>, conv_step_kernel<V, W, true, true>};
    return {conv_fwd_kernel<V, W, true, false>, conv_bwd_kernel<V, W, true, false>, conv_step_kernel<V, W, true, false>};
}

// vec: kConvV channels a thread as vectors (8 bytes in bf16, 16 in fp32), where every row starts on 16 bytes; else channel by
// channel.
ConvKernels conv_kernels_get(int W, bool vec, bool xb, bool yb) {
    if (W == 2) return vec ? conv_of_types<kConvV, 2>(xb, yb) : conv_of_types<1, 2>(xb, yb);
    if (W == 3) return vec ? conv_of_types<kConvV, 3>(xb, yb) : conv_of_types<1, 3>(xb, yb);
    return vec ? conv_of_types<kConvV, 4>(xb, yb) : conv_of_types<1, 4>(xb, yb);
}

size_t esize(ret_dtype_t t) { return t == RET_BF16 ? 2 : 4; }

// Tokens are int, and a strip's walk goes a few past the last.
bool conv_sizes_fit(int B, int N, int D) {
    return N <= INT32_MAX - 16 && (long long)B * N <= 1LL << 40 && D <= 1 << 28;
}

ret_status_t check_conv(const void* x, const void* w, const void* y, int B, int N, int D, int W, int64_t* ld,
                        ret_dtype_t in_dt, ret_dtype_t out_dt, int act) {
    if (!x || !w || !y) return fail(RET_ERR_INVALID_ARG, "null x/weight/output pointer");
    if (B <= 0 || N <= 0 || D <= 0)
        return fail(RET_ERR_INVALID_ARG, "sizes must be positive (B=%d N=%d D=%d)", B, N, D);
    for (ret_dtype_t t : {in_dt, out_dt})
        if (t != RET_F32 && t != RET_BF16) return fail(RET_ERR_INVALID_ARG, "bad dtype %d", (int)t);
    if (in_dt == RET_F32 && out_dt != RET_F32) return fail(RET_ERR_INVALID_ARG, "F32 input requires F32 output");
    if (act != RET_ACT_NONE && act != RET_ACT_SILU) return fail(RET_ERR_INVALID_ARG, "bad activation %d", act);
    if (W < 2 || W > 4) return fail(RET_ERR_UNSUPPORTED, "short convolution: width %d is not 2, 3 or 4", W);
    if (*ld == 0) *ld = D;
    if (*ld < D) return fail(RET_ERR_INVALID_ARG, "rows of x (%lld apart) are shorter than D=%d", (long long)*ld, D);
    if (!conv_sizes_fit(B, N, D) || *ld > 1LL << 32)
        return fail(RET_ERR_UNSUPPORTED, "short convolution: B=%d N=%d D=%d ld=%lld too large", B, N, D, (long long)*ld);
    return RET_OK;
}

bool conv_vec(const void* x, int D, int64_t ld) { return D % 8 == 0 && ld % 8 == 0 && aligned16(x); }

int64_t conv_cblocks(int D, int v) { return (D + 64 * v - 1) / (64 * v); }  // v: channels a thread

// Half of `most` and so on down to `least`, until there are two waves a SIMD.
int conv_strip(int B, int64_t N, int64_t cblocks, int most, int least) {
    while (most > least && cblocks * B * ((N + most - 1) / most) < 2048) most /= 2;
    return most;
}

struct ConvBwdPlan {
    int64_t cblocks, strips, parts;
    int strip;
};
ConvBwdPlan conv_bwd_plan(int B, int N, int D, bool vec) {
    ConvBwdPlan p;
    p.cblocks = conv_cblocks(D, vec ? kConvV : 1);
    p.strip = conv_strip(B, N, p.cblocks, kConvBwdStrip, kConvBwdStripLeast);
    p.strips = ((int64_t)N + p.strip - 1) / p.strip;
    const int64_t most = (B * p.strips + kConvWaves - 1) / kConvWaves, want = (1024 + p.cblocks - 1) / p.cblocks;
    p.parts = most < want ? most : want;
    return p;
}

}  // namespace

}  // namespace ret

using namespace ret;

extern "C" {

ret_status_t ret_short_conv_fwd(const void* x, int64_t x_ld, const float* weight, const float* bias, void* y, int B, int N,
                                int D, int W, ret_dtype_t in_dt, ret_dtype_t out_dt, int act, const int32_t* lengths,
                                const void* state_in, void* state_out, void* stream, const ret_options_t* opts) {
    ret_status_t st = check_conv(x, weight, y, B, N, D, W, &x_ld, in_dt, out_dt, act);
    if (st != RET_OK) return st;
    const bool vec = conv_vec(x, D, x_ld);
    const int64_t cblocks = conv_cblocks(D, vec ? kConvV : 1);
    const int strip = conv_strip(B, N, cblocks, kConvStrip, kConvStripLeast);
    const int64_t strips = ((int64_t)N + strip - 1) / strip;
    const unsigned long long wgs = (unsigned long long)cblocks * ((strips + kConvWaves - 1) / kConvWaves) * B;
    if (!grid_fits(wgs, 1, 1, 64 * kConvWaves))
        return fail(RET_ERR_UNSUPPORTED, "short convolution: B=%d N=%d D=%d exceed a launch", B, N, D);
    const size_t rows = (size_t)B * N, e = esize(in_dt), sb = (size_t)B * (W - 1) * D * e;
    const Buf w[] = {{"y", y, rows * D * esize(out_dt)}, {"state_out", state_out, sb, 1u << 3}};
    const Buf r[] = {{"x", x, ((rows - 1) * x_ld + D) * e, 0, (unsigned)e}, {"weight", weight, (size_t)D * W * 4},
                     {"bias", bias, (size_t)D * 4}, {"state_in", state_in, sb}, {"lengths", lengths, (size_t)B * 4, 0, 4}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    ConvArgs A = {x, weight, bias, state_in, y, state_out, lengths, x_ld, B, N, D, act == RET_ACT_SILU, strip, (int)strips,
                  (int)cblocks};
    hipStream_t s = (hipStream_t)stream;
    const Opts op = resolve(opts);
    LaunchTimer tm("ret_short_conv", s, op);
    hipLaunchKernelGGL(conv_kernels_get(W, vec, in_dt == RET_BF16, out_dt == RET_BF16).fwd, dim3((unsigned)wgs),
                       dim3(64 * kConvWaves), 0, s, A);
    tm.done();
    return launch_status("ret_short_conv");
}

size_t ret_short_conv_bwd_workspace_bytes(int B, int N, int D, int W) {
    if (B <= 0 || N <= 0 || D <= 0 || W < 2 || W > 4 || !conv_sizes_fit(B, N, D)) return 0;
    // either kernel's (x may be a slice that the vectors do not take)
    int64_t parts = conv_bwd_plan(B, N, D, false).parts;
    if (D % 8 == 0) parts = std::max(parts, conv_bwd_plan(B, N, D, true).parts);
    return (size_t)parts * (W + 1) * D * sizeof(float);
}

ret_status_t ret_short_conv_bwd(const void* dy, const void* x, int64_t x_ld, const float* weight, const float* bias,
                                void* dx, float* dweight, float* dbias, int B, int N, int D, int W, ret_dtype_t in_dt,
                                ret_dtype_t out_dt, int act, const int32_t* lengths, const void* state_in,
                                const void* dstate_out, void* dstate_in, void* workspace, size_t workspace_bytes,
                                void* stream, const ret_options_t* opts) {
    ret_status_t st = check_conv(x, weight, dx, B, N, D, W, &x_ld, in_dt, out_dt, act);
    if (st != RET_OK) return st;
    if (!dy) return fail(RET_ERR_INVALID_ARG, "null dy pointer");
    const bool vec = conv_vec(x, D, x_ld);
    const ConvBwdPlan p = conv_bwd_plan(B, N, D, vec);
    if (!grid_fits((unsigned long long)(p.cblocks * p.parts), 1, 1, 64 * kConvWaves))
        return fail(RET_ERR_UNSUPPORTED, "short convolution: B=%d N=%d D=%d exceed a launch", B, N, D);
    const bool cols = dweight || dbias;
    const size_t need = ret_short_conv_bwd_workspace_bytes(B, N, D, W);
    if (cols && (!workspace || workspace_bytes < need))
        return fail(RET_ERR_WORKSPACE, "short convolution gradients: workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : 0, need);
    const size_t rows = (size_t)B * N, e = esize(in_dt), eo = esize(out_dt), sn = (size_t)B * (W - 1) * D;
    const Buf w[] = {{"dx", dx, rows * D * eo}, {"dweight", dweight, (size_t)D * W * 4}, {"dbias", dbias, (size_t)D * 4},
                     {"dstate_in", dstate_in, sn * eo}, {"the workspace", workspace, cols ? workspace_bytes : 0}};
    const Buf r[] = {{"dy", dy, rows * D * e}, {"x", x, ((rows - 1) * x_ld + D) * e, 0, (unsigned)e},
                     {"weight", weight, (size_t)D * W * 4}, {"bias", bias, (size_t)D * 4}, {"state_in", state_in, sn * e},
                     {"dstate_out", dstate_out, sn * eo}, {"lengths", lengths, (size_t)B * 4, 0, 4}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    ConvBwdArgs A = {dy, x, weight, bias, state_in, dstate_out, dx, dstate_in, cols ? (float*)workspace : nullptr, lengths,
                     x_ld, B, N, D, act == RET_ACT_SILU, p.strip, (int)p.strips, (int)p.cblocks, (int)p.parts};
    hipStream_t s = (hipStream_t)stream;
    const Opts op = resolve(opts);
    {
        LaunchTimer tm("ret_short_conv_bwd", s, op);
        hipLaunchKernelGGL(conv_kernels_get(W, vec, in_dt == RET_BF16, out_dt == RET_BF16).bwd,
                           dim3((unsigned)(p.cblocks * p.parts)), dim3(64 * kConvWaves), 0, s, A);
        tm.done();
        if ((st = launch_status("ret_short_conv_bwd")) != RET_OK) return st;
    }
    if (!cols) return RET_OK;
    const long long n = (long long)(W + 1) * D;
    PartSumArgs P = {(const float*)workspace, dweight, dbias, nullptr, n, (long long)W * D, D, (int)p.parts};
    LaunchTimer tm("ret_column_sums", s, op);
    hipLaunchKernelGGL(part_sum_kernel_get(), dim3((unsigned)((n + kColSumCols - 1) / kColSumCols)), dim3(kColSumThreads),
                       0, s, P);
    tm.done();
    return launch_status("ret_column_sums");
}

ret_status_t ret_short_conv_step(const void* x, int64_t x_ld, const float* weight, const float* bias, void* y, void* state,
                                 int B, int D, int W, ret_dtype_t in_dt, ret_dtype_t out_dt, int act, void* stream,
                                 const ret_options_t* opts) {
    ret_status_t st = check_conv(x, weight, y, B, 1, D, W, &x_ld, in_dt, out_dt, act);
    if (st != RET_OK) return st;
    if (!state) return fail(RET_ERR_INVALID_ARG, "null state pointer");
    const bool vec = conv_vec(x, D, x_ld);
    const int per = 256 * (vec ? kConvV : 1);
    const unsigned long long cblocks = (D + per - 1) / per;
    int seqs = 1;
    while (seqs < kConvStepSeqs && cblocks * ((B + 2 * seqs - 1) / (2 * seqs)) >= kConvStepWgs) seqs *= 2;
    const unsigned long long wgs = cblocks * ((B + seqs - 1) / seqs);
    if (!grid_fits(wgs, 1, 1, 256))
        return fail(RET_ERR_UNSUPPORTED, "short convolution: B=%d D=%d exceed a launch", B, D);
    const size_t e = esize(in_dt);
    const Buf w[] = {{"y", y, (size_t)B * D * esize(out_dt)}, {"state", state, (size_t)B * (W - 1) * D * e}};
    const Buf r[] = {{"x", x, ((size_t)(B - 1) * x_ld + D) * e, 0, (unsigned)e}, {"weight", weight, (size_t)D * W * 4},
                     {"bias", bias, (size_t)D * 4}};
    if ((st = check_apart(w, r)) != RET_OK) return st;
    ConvStepArgs A = {x, weight, bias, state, y, x_ld, B, D, act == RET_ACT_SILU, (int)cblocks, seqs};
    hipStream_t s = (hipStream_t)stream;
    const Opts op = resolve(opts);
    LaunchTimer tm("ret_short_conv_step", s, op);
    hipLaunchKernelGGL(conv_kernels_get(W, vec, in_dt == RET_BF16, out_dt == RET_BF16).step,
                       dim3((unsigned)wgs), dim3(256), 0, s, A);
    tm.done();
    return launch_status("ret_short_conv_step");
}

}  // extern "C"
