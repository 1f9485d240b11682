// gma_conv.cu -- the short causal convolution per channel (gma_conv_forward, gma_conv_step,
// gma_conv_backward).
//
// p_t = sum_k w[k] x_{t-W+1+k} + bias, y = silu(p).  Bytes bound it: x is read and y written once, with
// about a dozen flops an element.  A thread keeps eight neighbouring channels and walks over a run of tokens
// with the last W - 1 inputs in registers, so each element is loaded once but for the W - 1 rows in
// front of a run; the accesses of a warp are 16 bytes a lane along the channels.
#include "block_common.cuh"

namespace gma {
namespace blk {
namespace {

// Tokens of one thread's run.  The rows in front of it are read a second time: (W - 1) / RUN extra.
constexpr int RUN = 16;
constexpr int THREADS = 128;

template <typename T> struct ConvArgs {
    int B, N, D, groups;        // groups = ceil(D / 8)
    Rows<const T> x;
    const float *w, *bias;
    const T *state_in;
    T *state_out;
    const int *lengths;
    Rows<T> y;
};

template <typename T, int W, bool VEC>
__device__ __forceinline__ void load_row(const ConvArgs<T> &a, int b, int t, int c0, int n, float (&v)[8])
{
    if (t >= 0) {
        load8<VEC>(a.x.at(b, t) + c0, n, v);
    } else if (a.state_in) {
        load8<VEC>(a.state_in + ((long long)b * (W - 1) + (t + W - 1)) * a.D + c0, n, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
}

template <int W> __device__ __forceinline__ void load_weights(const float *w, const float *bias, int c0, int n,
                                                              float (&wt)[8][W], float (&bs)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) wt[i][k] = i < n ? w[(long long)(c0 + i) * W + k] : 0.f;
        bs[i] = bias && i < n ? bias[c0 + i] : 0.f;
    }
}

template <typename T, int W, bool VEC, bool SILU>
__global__ void __launch_bounds__(THREADS) conv_forward_kernel(const ConvArgs<T> a)
{
    const int item = blockIdx.x * THREADS + threadIdx.x;
    const int g = item % a.groups, run = item / a.groups, b = blockIdx.y;
    const int len = row_length(a.lengths, b, a.N);
    const int c0 = g * 8, n = min(8, a.D - c0);
    const int t0 = run * RUN;
    // The state that follows: rows len - W + 1 .. len - 1, by the thread whose run holds the end.
    if (a.state_out && t0 <= len && len < t0 + RUN) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float v[8];
            load_row<T, W, VEC>(a, b, len - (W - 1) + k, c0, n, v);
            store8<VEC>(a.state_out + ((long long)b * (W - 1) + k) * a.D + c0, n, v);
        }
    }
    if (t0 >= len) return;
    float wt[8][W], bs[8], x[W][8];
    load_weights<W>(a.w, a.bias, c0, n, wt, bs);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_row<T, W, VEC>(a, b, t0 - (W - 1) + k, c0, n, x[k]);
#pragma unroll 4
    for (int s = 0; s < RUN; ++s) {
        const int t = t0 + s;
        if (t >= len) break;
        load8<VEC>(a.x.at(b, t) + c0, n, x[W - 1]);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float p = bs[i];
#pragma unroll
            for (int k = 0; k < W; ++k) p = fmaf(wt[i][k], x[k][i], p);
            y[i] = SILU ? silu(p) : p;
        }
        store8<VEC>(a.y.at(b, t) + c0, n, y);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = x[k + 1][i];
    }
}

// One token per batch row: the state's rows move up by one.  Each thread reads its channels of the
// state before it writes them, so state_out may be state_in.
template <typename T, int W, bool VEC, bool SILU>
__global__ void __launch_bounds__(THREADS) conv_step_kernel(const ConvArgs<T> a)
{
    const int item = blockIdx.x * THREADS + threadIdx.x;
    if (item >= a.groups) return;
    const int b = blockIdx.y, c0 = item * 8, n = min(8, a.D - c0);
    float wt[8][W], bs[8], x[W][8], y[8];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load8<VEC>(a.state_in + ((long long)b * (W - 1) + k) * a.D + c0, n, x[k]);
    load8<VEC>(a.x.at(b, 0) + c0, n, x[W - 1]);
    load_weights<W>(a.w, a.bias, c0, n, wt, bs);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store8<VEC>(a.state_out + ((long long)b * (W - 1) + k) * a.D + c0, n, x[k + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float p = bs[i];
#pragma unroll
        for (int k = 0; k < W; ++k) p = fmaf(wt[i][k], x[k][i], p);
        y[i] = SILU ? silu(p) : p;
    }
    store8<VEC>(a.y.at(b, 0) + c0, n, y);
}

template <typename T> struct ConvGradArgs {
    ConvArgs<T> f;
    Rows<const T> dy;
    Rows<T> dx;
    float *part;                // [runs * B][W + 1][groups * 8]
    int runs;
};

// Backward: with dp_t = dy_t silu'(p_t), dx_t = sum_k w[k] dp_{t+W-1-k}, dw[k] = sum_t dp_t x_{t-W+1+k},
// dbias = sum_t dp_t.  A thread's run of tokens needs p of the W - 1 tokens behind it too.  Each
// thread sums its run's share of dw and dbias in order and writes it to the workspace; a second
// kernel adds the runs up in a fixed order.
template <typename T, int W, bool VEC, bool SILU, int GRUN>
__global__ void __launch_bounds__(THREADS) conv_backward_kernel(const ConvGradArgs<T> g)
{
    const ConvArgs<T> &a = g.f;
    const int item = blockIdx.x * THREADS + threadIdx.x;
    const int grp = item % a.groups, run = item / a.groups, b = blockIdx.y;
    if (run >= g.runs) return;
    const int len = row_length(a.lengths, b, a.N);
    const int c0 = grp * 8, n = min(8, a.D - c0);
    const int t0 = run * GRUN;
    float dw[8][W], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[i][k] = 0.f;
    }
    if (t0 < len) {
        float wt[8][W], bs[8], x[W][8], dp[W][8];
        load_weights<W>(a.w, a.bias, c0, n, wt, bs);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) load_row<T, W, VEC>(a, b, t0 - (W - 1) + k, c0, n, x[k]);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) dp[k][i] = 0.f;
        // dp holds the last W tokens' dp: after token t, dx of token t - W + 1 is complete.
#pragma unroll 2
        for (int s = 0; s < GRUN + W - 1; ++s) {
            const int t = t0 + s;
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) dp[k][i] = dp[k + 1][i];
            if (t < len) {
                float d[8];
                load8<VEC>(a.x.at(b, t) + c0, n, x[W - 1]);
                load8<VEC>(g.dy.at(b, t) + c0, n, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (SILU) {
                        float p = bs[i];
#pragma unroll
                        for (int k = 0; k < W; ++k) p = fmaf(wt[i][k], x[k][i], p);
                        d[i] *= dsilu(p, sigmoid(p));
                    }
                    dp[W - 1][i] = d[i];
                }
                if (s < GRUN) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        db[i] += d[i];
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[i][k] = fmaf(d[i], x[k][i], dw[i][k]);
                    }
                }
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[k][i] = x[k + 1][i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dp[W - 1][i] = 0.f;
            }
            const int to = t - (W - 1);
            if (s >= W - 1 && to < len) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = 0.f;
                    // dp[j] is token to + j; tap k = W - 1 - j
#pragma unroll
                    for (int j = 0; j < W; ++j) v[i] = fmaf(wt[i][W - 1 - j], dp[j][i], v[i]);
                }
                store8<VEC>(g.dx.at(b, to) + c0, n, v);
            }
        }
    }
    float *out = g.part + (((long long)b * g.runs + run) * (W + 1)) * (a.groups * 8) + c0;
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k < W ? dw[i][k] : db[i];
        store8<true>(out + (long long)k * (a.groups * 8), 8, v);
    }
}

template <typename T> ConvArgs<T> args_of(const gma_conv_t &c)
{
    ConvArgs<T> a;
    a.B = c.B; a.N = c.N; a.D = c.D; a.groups = (c.D + 7) / 8;
    a.x = rows_of<const T>(c.x);
    a.w = c.weight; a.bias = c.bias;
    a.state_in = (const T *)c.state_in;
    a.state_out = (T *)c.state_out;
    a.lengths = c.lengths;
    a.y = rows_of<T>(c.y);
    return a;
}

bool vec_states(const gma_conv_t &c) { return c.D % 8 == 0 && opt_ok(c.state_in, 16) && opt_ok(c.state_out, 16); }

gma_status_t check(const gma_conv_t *c, bool need_out)
{
    if (!c) return GMA_ERR_INVALID_ARG;
    if (c->B < 1 || c->N < 1 || c->D < 1) return GMA_ERR_INVALID_ARG;
    if (c->dtype != GMA_F32 && c->dtype != GMA_BF16) return GMA_ERR_INVALID_ARG;
    if (c->flags & ~GMA_CONV_LINEAR) return GMA_ERR_INVALID_ARG;
    if (c->W < 2 || c->W > 4 || c->B > 65535 || c->D > (1 << 24) || c->N > (1 << 30)) return GMA_ERR_UNSUPPORTED_SHAPE;
    const size_t e = elem_size(c->dtype);
    if (!rows_ok(c->x, c->dtype, c->B, c->N, c->D, false)) return GMA_ERR_INVALID_ARG;
    if (need_out && !rows_ok(c->y, c->dtype, c->B, c->N, c->D, true)) return GMA_ERR_INVALID_ARG;
    if (!ptr_ok(c->weight, 4) || !opt_ok(c->bias, 4) || !opt_ok(c->state_in, e) || !opt_ok(c->state_out, e) ||
        !opt_ok(c->lengths, 4))
        return GMA_ERR_INVALID_ARG;
    return GMA_OK;
}

// Calls f(T{}, W, VEC, SILU) as template arguments.
template <typename F> gma_status_t dispatch(const gma_conv_t &c, bool vec, F f)
{
    const bool silu = !(c.flags & GMA_CONV_LINEAR);
    auto with_w = [&](auto tag) -> gma_status_t {
        using T = decltype(tag);
        auto with_vec = [&](auto wtag) -> gma_status_t {
            constexpr int W = decltype(wtag)::value;
            if (vec)
                return silu ? f(T{}, std::integral_constant<int, W>{}, std::true_type{}, std::true_type{})
                            : f(T{}, std::integral_constant<int, W>{}, std::true_type{}, std::false_type{});
            return silu ? f(T{}, std::integral_constant<int, W>{}, std::false_type{}, std::true_type{})
                        : f(T{}, std::integral_constant<int, W>{}, std::false_type{}, std::false_type{});
        };
        if (c.W == 2) return with_vec(std::integral_constant<int, 2>{});
        if (c.W == 3) return with_vec(std::integral_constant<int, 3>{});
        return with_vec(std::integral_constant<int, 4>{});
    };
    return c.dtype == GMA_BF16 ? with_w(__nv_bfloat16{}) : with_w(float{});
}

// Tokens of one thread's run in the backward pass.
constexpr int GRUN = 32;

int grad_runs(const gma_conv_t &c) { return (c.N + GRUN - 1) / GRUN; }

}  // namespace
}  // namespace blk
}  // namespace gma

using namespace gma;
using namespace gma::blk;

extern "C" {

gma_status_t gma_conv_forward(const gma_conv_t *c, gma_stream_t stream)
{
    gma_status_t r = check(c, true);
    if (r != GMA_OK) return r;
    if (c->state_out && c->state_out == c->state_in) return GMA_ERR_INVALID_ARG;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = vec_states(*c) && rows_vec(c->x, c->dtype) && rows_vec(c->y, c->dtype);
    return dispatch(*c, vec, [&](auto t, auto w, auto v, auto s) -> gma_status_t {
        using T = decltype(t);
        ConvArgs<T> a = args_of<T>(*c);
        // one run more when the sequence ends at the end of the last one (it writes the state)
        const long long runs = c->N / RUN + 1, items = runs * a.groups;
        const long long blocks = (items + THREADS - 1) / THREADS;
        if (blocks > 0x7fffffffll || items > 0x7fffff00ll) return GMA_ERR_UNSUPPORTED_SHAPE;
        GMA_LAUNCH(KID_CONV, st,
                   conv_forward_kernel<T, decltype(w)::value, decltype(v)::value, decltype(s)::value>
                   <<<dim3((unsigned)blocks, c->B), THREADS, 0, st>>>(a));
        return GMA_OK;
    });
}

gma_status_t gma_conv_step(const gma_conv_t *c, gma_stream_t stream)
{
    gma_status_t r = check(c, true);
    if (r != GMA_OK) return r;
    if (c->N != 1 || !c->state_in || !c->state_out || c->lengths) return GMA_ERR_INVALID_ARG;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = vec_states(*c) && rows_vec(c->x, c->dtype) && rows_vec(c->y, c->dtype);
    return dispatch(*c, vec, [&](auto t, auto w, auto v, auto s) -> gma_status_t {
        using T = decltype(t);
        ConvArgs<T> a = args_of<T>(*c);
        GMA_LAUNCH(KID_CONV_STEP, st,
                   conv_step_kernel<T, decltype(w)::value, decltype(v)::value, decltype(s)::value>
                   <<<dim3((a.groups + THREADS - 1) / THREADS, c->B), THREADS, 0, st>>>(a));
        return GMA_OK;
    });
}

size_t gma_conv_backward_workspace_size(const gma_conv_grad_t *g)
{
    if (!g || check(&g->fwd, false) != GMA_OK) return 0;
    const gma_conv_t &c = g->fwd;
    return align_up((size_t)grad_runs(c) * c.B * (c.W + 1) * ((c.D + 7) / 8 * 8) * sizeof(float), 256);
}

gma_status_t gma_conv_backward(const gma_conv_grad_t *g, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    if (!g) return GMA_ERR_INVALID_ARG;
    const gma_conv_t &c = g->fwd;
    gma_status_t r = check(&c, false);
    if (r != GMA_OK) return r;
    if (!rows_ok(g->dy, c.dtype, c.B, c.N, c.D, false) || !rows_ok(g->dx, c.dtype, c.B, c.N, c.D, true))
        return GMA_ERR_INVALID_ARG;
    if (!ptr_ok(g->dweight, 4) || !opt_ok(g->dbias, 4) || (c.bias && !g->dbias)) return GMA_ERR_INVALID_ARG;
    const long long runs = grad_runs(c), items = runs * ((c.D + 7) / 8);
    if (items > 0x7fffff00ll || runs * c.B > 0x7fffffffll) return GMA_ERR_UNSUPPORTED_SHAPE;
    if (!ws_ok(ws, ws_bytes, gma_conv_backward_workspace_size(g))) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = c.D % 8 == 0 && opt_ok(c.state_in, 16) && rows_vec(c.x, c.dtype) && rows_vec(g->dy, c.dtype) &&
                     rows_vec(g->dx, c.dtype);
    return dispatch(c, vec, [&](auto t, auto w, auto v, auto s) -> gma_status_t {
        using T = decltype(t);
        constexpr int W = decltype(w)::value;
        ConvGradArgs<T> a;
        a.f = args_of<T>(c);
        a.dy = rows_of<const T>(g->dy);
        a.dx = rows_of<T>(g->dx);
        a.part = (float *)ws;
        a.runs = (int)runs;
        GMA_LAUNCH(KID_CONV_BWD, st,
                   conv_backward_kernel<T, W, decltype(v)::value, decltype(s)::value, GRUN>
                   <<<dim3((unsigned)((items + THREADS - 1) / THREADS), c.B), THREADS, 0, st>>>(a));
        SumOut out[W + 1];
        for (int k = 0; k < W; ++k) out[k] = SumOut{g->dweight + k, W};
        out[W] = SumOut{g->dbias, 1};
        return sum_rows(a.part, runs * c.B, g->dbias ? W + 1 : W, W + 1, c.D, a.f.groups * 8, out, st);
    });
}

}  // extern "C"
