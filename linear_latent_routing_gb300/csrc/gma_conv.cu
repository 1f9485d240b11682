// gma_conv.cu -- the short causal convolution per channel (gma_conv_forward, gma_conv_step,
// gma_conv_backward).
//
// p_t = sum_k w[k] x_{t-W+1+k} + bias, y = silu(p).  Bytes bound it: x is read and y written once, with
// about a dozen flops an element.  A thread keeps four neighbouring channels and walks over a run of tokens
// with the last W inputs in registers, so each element is loaded once but for the W - 1 rows in
// front of a run; a warp's accesses are 256 neighbouring bytes of a row (bf16).  Four channels and not eight:
// the windows then take few enough registers for twice the warps, which hide the loads.  The window is a
// ring whose slots are fixed by unrolling a whole turn, so no value is moved.
// Measured (W = 4, bf16): forward 2 x 16384 x 2080 in 56 us (4.9 TB/s; eight channels a thread 71 us, with moved
// windows 150 us); backward 32 x 1024 x 512, half of it padding, 28 us (42 instructions an element at 128 registers),
// 4 x 16384 x 4096 324 us (5.0 TB/s).  In fp32 with W = 4 the backward kernel spills about 200 bytes a thread.
#include "block_common.cuh"

namespace gma {
namespace blk {
namespace {

constexpr int THREADS = 128, C = 4;

template <typename T> struct ConvArgs {
    int B, N, D, groups;        // groups = ceil(D / C)
    int run;                    // tokens of one thread's run
    bool zero;                  // zeros behind a sequence's last token
    Rows<const T> x;
    const float *w, *bias;
    const T *state_in;
    T *state_out;
    const int *lengths;
    Rows<T> y;
};

// Four neighbouring channels as two packed pairs.
template <typename T> struct Raw4;
template <> struct Raw4<__nv_bfloat16> {
    uint2 q;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { q = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void get(f2 (&v)[2]) const
    {
        v[0] = pack2(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u));
        v[1] = pack2(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
    }
};
template <> struct Raw4<float> {
    ulonglong2 q;
    __device__ __forceinline__ void load(const float *p) { q = *reinterpret_cast<const ulonglong2 *>(p); }
    __device__ __forceinline__ void get(f2 (&v)[2]) const { v[0] = q.x; v[1] = q.y; }
};
// VEC: all four exist and lie on an access's boundary; else the first n of them, one by one.
template <bool VEC, typename T> __device__ __forceinline__ void load4(const T *p, int n, f2 (&v)[2])
{
    if (VEC) {
        Raw4<T> r;
        r.load(p);
        r.get(v);
    } else {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = i < n ? to_f32<T>(p[i]) : 0.f;
        v[0] = pack2(s[0], s[1]);
        v[1] = pack2(s[2], s[3]);
    }
}
template <bool VEC> __device__ __forceinline__ void store4(__nv_bfloat16 *p, int n, const f2 (&v)[2])
{
    const float2 a = unpack2(v[0]), b = unpack2(v[1]);
    if (VEC) {
        uint2 q;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&q);
        h[0] = __floats2bfloat162_rn(a.x, a.y);
        h[1] = __floats2bfloat162_rn(b.x, b.y);
        *reinterpret_cast<uint2 *>(p) = q;
    } else {
        const float s[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(s[i]);
    }
}
template <bool VEC> __device__ __forceinline__ void store4(float *p, int n, const f2 (&v)[2])
{
    if (VEC) {
        *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v[0], v[1]);
    } else {
        const float2 a = unpack2(v[0]), b = unpack2(v[1]);
        const float s[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = s[i];
    }
}

// Row t of batch row b, or a row of the state in front (t < 0).
template <typename T, int W, bool VEC>
__device__ __forceinline__ void load_row(const ConvArgs<T> &a, int b, int t, int c0, int n, f2 (&v)[2])
{
    v[0] = v[1] = 0ull;
    if (t >= 0) load4<VEC>(a.x.at(b, t) + c0, n, v);
    else if (a.state_in) load4<VEC>(a.state_in + ((long long)b * (W - 1) + (t + W - 1)) * a.D + c0, n, v);
}

// wt[k]: tap k of the four channels.
template <int W> __device__ __forceinline__ void load_weights(const float *w, const float *bias, int c0, int n,
                                                              f2 (&wt)[W][2], f2 (&bs)[2])
{
    const float *p = w + (long long)c0 * W;
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            wt[k][i] = pack2(2 * i < n ? p[2 * i * W + k] : 0.f, 2 * i + 1 < n ? p[(2 * i + 1) * W + k] : 0.f);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        bs[i] = pack2(bias && 2 * i < n ? bias[c0 + 2 * i] : 0.f, bias && 2 * i + 1 < n ? bias[c0 + 2 * i + 1] : 0.f);
}

__device__ __forceinline__ f2 silu2(f2 v)
{
    const float2 x = unpack2(v);
    return pack2(silu(x.x), silu(x.y));
}
__device__ __forceinline__ f2 dsilu2(f2 v)
{
    const float2 x = unpack2(v);
    return pack2(dsilu(x.x, sigmoid(x.x)), dsilu(x.y, sigmoid(x.y)));
}

template <bool VEC, typename T>
__device__ __forceinline__ void zero_rows(const Rows<T> &r, int b, int from, int to, int c0, int n)
{
    const f2 none[2] = {0ull, 0ull};
    for (int t = from; t < to; ++t) store4<VEC>(r.at(b, t) + c0, n, none);
}

// Tokens whose loads are in flight together: whole turns of the ring.
template <int W> constexpr int flight() { return W == 3 ? 3 : 4; }

template <typename T, int W, bool VEC, bool SILU>
__global__ void __launch_bounds__(THREADS) conv_forward_kernel(const ConvArgs<T> a)
{
    constexpr int F = flight<W>();
    const int item = blockIdx.x * THREADS + threadIdx.x;
    const int g = item % a.groups, run = item / a.groups, b = blockIdx.y;
    const int len = row_length(a.lengths, b, a.N);
    const int c0 = g * C, n = min(C, a.D - c0);
    const int t0 = run * a.run, end = min(len, t0 + a.run);
    // The state that follows: rows len - W + 1 .. len - 1, by the thread whose run holds the end.
    if (a.state_out && t0 <= len && len < t0 + a.run) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            f2 v[2];
            load_row<T, W, VEC>(a, b, len - (W - 1) + k, c0, n, v);
            store4<VEC>(a.state_out + ((long long)b * (W - 1) + k) * a.D + c0, n, v);
        }
    }
    if (a.zero) zero_rows<VEC>(a.y, b, max(t0, len), min(t0 + a.run, a.N), c0, n);
    if (t0 >= len) return;
    f2 wt[W][2], bs[2], x[W][2];
    load_weights<W>(a.w, a.bias, c0, n, wt, bs);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_row<T, W, VEC>(a, b, t0 - (W - 1) + k, c0, n, x[k]);
    const T *xp = a.x.at(b, t0) + c0;
    T *yp = a.y.at(b, t0) + c0;
    Raw4<T> next[F];
    auto fetch = [&](int t) {
#pragma unroll
        for (int s = 0; s < F; ++s)
            if (VEC && t + s < end) next[s].load(xp + s * a.x.st);
    };
    fetch(t0);
    for (int t = t0; t < end; t += F) {
        Raw4<T> r[F];
#pragma unroll
        for (int s = 0; s < F; ++s) r[s] = next[s];
        const T *row = xp;
        xp += F * a.x.st;
        fetch(t + F);
#pragma unroll
        for (int s = 0; s < F; ++s)
            if (t + s < end) {
                f2(&in)[2] = x[(s + W - 1) % W];
                if (VEC) r[s].get(in);
                else load4<false>(row + s * a.x.st, n, in);
                f2 p[2] = {bs[0], bs[1]};
#pragma unroll
                for (int k = 0; k < W; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) p[i] = fma2(wt[k][i], x[(s + k) % W][i], p[i]);
                if (SILU) p[0] = silu2(p[0]), p[1] = silu2(p[1]);
                store4<VEC>(yp, n, p);
                yp += a.y.st;
            }
    }
}

// One token per batch row: the state's rows move up by one.  Each thread reads its channels of the
// state before it writes them, so state_out may be state_in.
template <typename T, int W, bool VEC, bool SILU>
__global__ void __launch_bounds__(THREADS) conv_step_kernel(const ConvArgs<T> a)
{
    const int item = blockIdx.x * THREADS + threadIdx.x;
    if (item >= a.groups) return;
    const int b = blockIdx.y, c0 = item * C, n = min(C, a.D - c0);
    f2 wt[W][2], bs[2], x[W][2];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load4<VEC>(a.state_in + ((long long)b * (W - 1) + k) * a.D + c0, n, x[k]);
    load4<VEC>(a.x.at(b, 0) + c0, n, x[W - 1]);
    load_weights<W>(a.w, a.bias, c0, n, wt, bs);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store4<VEC>(a.state_out + ((long long)b * (W - 1) + k) * a.D + c0, n, x[k + 1]);
    f2 p[2] = {bs[0], bs[1]};
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) p[i] = fma2(wt[k][i], x[k][i], p[i]);
    if (SILU) p[0] = silu2(p[0]), p[1] = silu2(p[1]);
    store4<VEC>(a.y.at(b, 0) + c0, n, p);
}

template <typename T> struct ConvGradArgs {
    ConvArgs<T> f;
    Rows<const T> dy;
    Rows<T> dx;
    float *part;                // [run blocks * B][W + 1][groups * C]
    int runs, gtiles, rtiles;   // blocks of 32 groups, of GWARPS runs
};

// Backward: with dp_t = dy_t silu'(p_t), dx_t = sum_k w[k] dp_{t+W-1-k}, dw[k] = sum_t dp_t x_{t-W+1+k},
// dbias = sum_t dp_t.  A thread's run of tokens needs p of the W - 1 tokens behind it too.  Each
// thread sums its run's share of dw and dbias in order, a block adds its warps (neighbouring runs of the
// same 128 channels) in order and writes one partial row, and sum_rows adds those in a fixed order.
constexpr int GWARPS = 8;
template <typename T, int W, bool VEC, bool SILU>
__global__ void __launch_bounds__(32 * GWARPS, 2) conv_backward_kernel(const ConvGradArgs<T> g)
{
    constexpr int F = flight<W>();
    const ConvArgs<T> &a = g.f;
    __shared__ __align__(16) float sums[W + 1][GWARPS][32 * C];
    let_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
    const int grp = blockIdx.x % g.gtiles * 32 + lane, rtile = blockIdx.x / g.gtiles, run = rtile * GWARPS + warp;
    const int len = grp < a.groups && run < g.runs ? row_length(a.lengths, b, a.N) : 0;
    const int c0 = grp * C, n = min(C, a.D - c0);
    const int t0 = run * a.run, end = min(len, t0 + a.run);
    if (a.zero && grp < a.groups && run < g.runs) zero_rows<VEC>(g.dx, b, max(t0, len), min(t0 + a.run, a.N), c0, n);
    f2 dw[W][2], db[2] = {0ull, 0ull};
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][0] = dw[k][1] = 0ull;
    if (t0 < len) {
        f2 wt[W][2], bs[2], x[W][2], dp[W][2];
        load_weights<W>(a.w, a.bias, c0, n, wt, bs);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) load_row<T, W, VEC>(a, b, t0 - (W - 1) + k, c0, n, x[k]);
#pragma unroll
        for (int k = 0; k < W; ++k) dp[k][0] = dp[k][1] = 0ull;
        const int last = end + W - 1;             // tokens whose dp this run's dx needs
        const T *xp = a.x.at(b, t0) + c0, *dyp = g.dy.at(b, t0) + c0;
        T *dxp = g.dx.at(b, t0) + c0;
        Raw4<T> xn[F], dn[F];
        auto fetch = [&](int t) {
#pragma unroll
            for (int s = 0; s < F; ++s)
                if (VEC && t + s < last && t + s < len) {
                    xn[s].load(xp + s * a.x.st);
                    dn[s].load(dyp + s * g.dy.st);
                }
        };
        fetch(t0);
        for (int t = t0; t < last; t += F) {
            Raw4<T> xr[F], dr[F];
#pragma unroll
            for (int s = 0; s < F; ++s) xr[s] = xn[s], dr[s] = dn[s];
            const T *xrow = xp, *drow = dyp;
            xp += F * a.x.st;
            dyp += F * g.dy.st;
            fetch(t + F);
#pragma unroll
            for (int s = 0; s < F; ++s)
                if (t + s < last) {
                    // the newest slot: x and dp of token t + s; (s + j) % W is token t + s - (W - 1) + j
                    f2(&d)[2] = dp[(s + W - 1) % W];
                    d[0] = d[1] = 0ull;
                    if (t + s < len) {
                        f2(&in)[2] = x[(s + W - 1) % W];
                        if (VEC) {
                            xr[s].get(in);
                            dr[s].get(d);
                        } else {
                            load4<false>(xrow + s * a.x.st, n, in);
                            load4<false>(drow + s * g.dy.st, n, d);
                        }
                        if (SILU) {
                            f2 p[2] = {bs[0], bs[1]};
#pragma unroll
                            for (int k = 0; k < W; ++k)
#pragma unroll
                                for (int i = 0; i < 2; ++i) p[i] = fma2(wt[k][i], x[(s + k) % W][i], p[i]);
#pragma unroll
                            for (int i = 0; i < 2; ++i) d[i] = mul2(d[i], dsilu2(p[i]));
                        }
                        if (t + s < end) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                db[i] = add2(db[i], d[i]);
#pragma unroll
                                for (int k = 0; k < W; ++k) dw[k][i] = fma2(d[i], x[(s + k) % W][i], dw[k][i]);
                            }
                        }
                    }
                    const int to = t + s - (W - 1);       // its dx is complete
                    if (to >= t0 && to < end) {
                        f2 v[2] = {0ull, 0ull};
#pragma unroll
                        for (int j = 0; j < W; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) v[i] = fma2(wt[W - 1 - j][i], dp[(s + j) % W][i], v[i]);
                        store4<VEC>(dxp, n, v);
                        dxp += g.dx.st;
                    }
                }
        }
    }
#pragma unroll
    for (int k = 0; k <= W; ++k) store4<true>(&sums[k][warp][lane * C], C, k < W ? dw[k < W ? k : 0] : db);
    __syncthreads();
    const int width = a.groups * C, first = blockIdx.x % g.gtiles * 32 * C;
    float *out = g.part + ((long long)b * g.rtiles + rtile) * (W + 1) * width + first;
    for (int i = threadIdx.x; i < (W + 1) * 32 * C; i += 32 * GWARPS) {
        const int k = i / (32 * C), at = i % (32 * C);
        if (first + at >= width) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < GWARPS; ++w) v += sums[k][w][at];
        out[(long long)k * width + at] = v;
    }
}

// Tokens of a thread's run: the rows in front of it are read a second time ((W - 1) / run extra), and its start and
// end cost as much as a few tokens, so runs as long as they can be with 768 threads an SM, up to 256.  2 x 16384 x 2080: 128 tokens
// 56 us, 64 tokens 58 us, 256 tokens (384 threads an SM) 68 us; backward 4 x 16384 x 4096: 256 tokens 324 us, 32 tokens
// 400 us, 512 tokens 354 us.
int run_of(const gma_conv_t &c)
{
    const long long groups = (long long)c.B * ((c.D + C - 1) / C);
    int run = 256;
    while (run > 8 && groups * ((c.N + run - 1) / run) < 152 * 768) run /= 2;
    return run;
}

template <typename T> ConvArgs<T> args_of(const gma_conv_t &c, int run)
{
    ConvArgs<T> a;
    a.run = run;
    a.zero = c.flags & GMA_ROWS_ZERO_TAIL;
    a.B = c.B; a.N = c.N; a.D = c.D; a.groups = (c.D + C - 1) / C;
    a.x = rows_of<const T>(c.x);
    a.w = c.weight; a.bias = c.bias;
    a.state_in = (const T *)c.state_in;
    a.state_out = (T *)c.state_out;
    a.lengths = c.lengths;
    a.y = rows_of<T>(c.y);
    return a;
}

// Whether accesses of four channels are aligned.
bool vec4(const gma_rows_t &r, int dtype)
{
    const size_t e = elem_size(dtype);
    return (((uintptr_t)r.ptr | (uintptr_t)(r.batch * e) | (uintptr_t)(r.token * e)) & (4 * e - 1)) == 0;
}
bool vec_states(const gma_conv_t &c)
{
    const size_t e = 4 * elem_size(c.dtype);
    return c.D % 4 == 0 && opt_ok(c.state_in, e) && opt_ok(c.state_out, e);
}

gma_status_t check(const gma_conv_t *c, bool need_out)
{
    if (!c) return GMA_ERR_INVALID_ARG;
    if (c->B < 1 || c->N < 1 || c->D < 1) return GMA_ERR_INVALID_ARG;
    if (c->dtype != GMA_F32 && c->dtype != GMA_BF16) return GMA_ERR_INVALID_ARG;
    if (c->flags & ~(GMA_CONV_LINEAR | GMA_ROWS_ZERO_TAIL)) return GMA_ERR_INVALID_ARG;
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

int grad_runs(const gma_conv_t &c)
{
    const int run = run_of(c);
    return (c.N + run - 1) / run;
}

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
    const bool vec = vec_states(*c) && vec4(c->x, c->dtype) && vec4(c->y, c->dtype);
    return dispatch(*c, vec, [&](auto t, auto w, auto v, auto s) -> gma_status_t {
        using T = decltype(t);
        const ConvArgs<T> a = args_of<T>(*c, run_of(*c));
        // one run more when the sequence ends at the end of the last one (it writes the state)
        const long long runs = c->N / a.run + 1, items = runs * a.groups;
        const long long blocks = (items + THREADS - 1) / THREADS;
        if (blocks > 0x7fffffffll || items > 0x7fffff00ll) return GMA_ERR_UNSUPPORTED_SHAPE;
        GMA_LAUNCH(KID_CONV, st,
                   conv_forward_kernel<T, decltype(w)::value, decltype(v)::value, decltype(s)::value>
                   <<<dim3((unsigned)blocks, c->B), THREADS, 0, st>>>(a));
        return GMA_OK;
    });
}

gma_status_t gma_conv_step(const gma_conv_t *conv, gma_stream_t stream)
{
    if (!conv) return GMA_ERR_INVALID_ARG;
    gma_conv_t one = *conv, *c = &one;       // its token strides are ignored
    one.x.token = one.y.token = 0;
    gma_status_t r = check(c, true);
    if (r != GMA_OK) return r;
    if (c->N != 1 || !c->state_in || !c->state_out || c->lengths) return GMA_ERR_INVALID_ARG;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = vec_states(*c) && vec4(c->x, c->dtype) && vec4(c->y, c->dtype);
    return dispatch(*c, vec, [&](auto t, auto w, auto v, auto s) -> gma_status_t {
        using T = decltype(t);
        const ConvArgs<T> a = args_of<T>(*c, 1);
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
    return align_up((size_t)((grad_runs(c) + GWARPS - 1) / GWARPS) * c.B * (c.W + 1) * ((c.D + C - 1) / C * C) * sizeof(float), 256);
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
    const long long runs = grad_runs(c), items = runs * ((c.D + C - 1) / C);
    if (items > 0x7fffff00ll || runs * c.B > 0x7fffffffll) return GMA_ERR_UNSUPPORTED_SHAPE;
    if (!ws_ok(ws, ws_bytes, gma_conv_backward_workspace_size(g))) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = vec_states(c) && vec4(c.x, c.dtype) && vec4(g->dy, c.dtype) &&
                     vec4(g->dx, c.dtype);
    return dispatch(c, vec, [&](auto t, auto w, auto v, auto s) -> gma_status_t {
        using T = decltype(t);
        constexpr int W = decltype(w)::value;
        ConvGradArgs<T> a;
        a.f = args_of<T>(c, run_of(c));
        a.dy = rows_of<const T>(g->dy);
        a.dx = rows_of<T>(g->dx);
        a.part = (float *)ws;
        a.runs = (int)runs;
        a.gtiles = (a.f.groups + 31) / 32;
        a.rtiles = (a.runs + GWARPS - 1) / GWARPS;
        GMA_LAUNCH(KID_CONV_BWD, st,
                   conv_backward_kernel<T, W, decltype(v)::value, decltype(s)::value>
                   <<<dim3((unsigned)(a.gtiles * a.rtiles), c.B), 32 * GWARPS, 0, st>>>(a));
        const long long width = a.f.groups * C;
        SumVec vecs[W + 1];
        for (int k = 0; k < W; ++k) vecs[k] = SumVec{a.part + k * width, (W + 1) * width, c.D, g->dweight + k, W};
        vecs[W] = SumVec{a.part + W * width, (W + 1) * width, c.D, g->dbias, 1};
        return sum_rows(vecs, g->dbias ? W + 1 : W, (long long)a.rtiles * c.B, st);
    });
}

}  // extern "C"
