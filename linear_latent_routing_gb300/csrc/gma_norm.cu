// gma_norm.cu -- the norms before and after a block, fused with its gate and residual scale
// (gma_norm_forward, gma_norm_backward).
//
//   a = o silu(gate);  v = w_post a rstd_g;  r' = residual + scale v;  h = w_pre r' rstd.
//
// Bytes bound both passes: every activation is read once and written once, and a row lives in
// registers between its two reductions.  A row is held by TPR threads (8 lanes of a warp up to a
// whole block, by the row's width), NV pieces of eight channels a thread; a block holds several
// narrow rows.  The mixers' layout [B][H][N][d] is read (and its gradient written) in place, head
// by head, so no transposition runs between a mixer and its norm.
#include "block_common.cuh"

namespace gma {
namespace blk {
namespace {

constexpr int MAX_WARPS = 32;

template <typename T, typename R> struct NormArgs {
    int N, d, D, group, tpr;      // tpr: threads per row
    long long rows;               // B * N
    float eps, inv_d, inv_group;
    Rows<const T> o;
    long long o_head;
    Rows<const T> gate;
    Rows<const R> residual;
    const float *w_post, *scale, *w_pre;
    Rows<R> r;
    Rows<T> h;
};

// Channels c0 .. c0 + 7 of token (b, t) in the head layout.  VEC: d is a multiple of eight.
template <bool VEC, typename T>
__device__ __forceinline__ void load_heads(const Rows<const T> &o, long long head, int d, int b, int t, int c0, int n,
                                           float (&v)[8])
{
    const T *p = o.at(b, t);
    if (VEC) {
        const int hd = c0 / d;
        load8<true>(p + hd * head + (c0 - hd * d), n, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i, hd = c / d;
            v[i] = i < n ? to_f32<T>(p[hd * head + (c - hd * d)]) : 0.f;
        }
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_heads(const Rows<T> &o, long long head, int d, int b, int t, int c0, int n,
                                            const float (&v)[8])
{
    T *p = o.at(b, t);
    if (VEC) {
        const int hd = c0 / d;
        store8<true>(p + hd * head + (c0 - hd * d), n, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i, hd = c / d;
            if (i < n) p[hd * head + (c - hd * d)] = from_f32<T>(v[i]);
        }
    }
}

template <bool VEC> __device__ __forceinline__ void load_param(const float *p, int c0, int n, float none, float (&v)[8])
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = none;
    } else {
        load8<VEC>(p + c0, n, v);
    }
}

// Sums of K values over a row's threads, the same bits in each of them.  `buf` is one of two
// buffers used in turn, so one barrier per sum is enough.
template <int K> __device__ __forceinline__ void row_sum(float (&v)[K], int tpr, float (*buf)[K])
{
    const int width = tpr < 32 ? tpr : 32;
    for (int off = width / 2; off; off >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, per = tpr >> 5, first = warp / per * per;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) buf[warp][k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = 0.f;
        for (int w = 0; w < per; ++w)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += buf[first + w][k];
    }
}

// Sum over the group that a thread's eight channels belong to: group / 8 neighbouring lanes (a power
// of two up to 32).
__device__ __forceinline__ float group_sum(float v, int lanes)
{
    for (int off = lanes / 2; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

template <typename T, typename R, bool VEC, int NV>
__global__ void __launch_bounds__(1024) norm_forward_kernel(const NormArgs<T, R> a)
{
    __shared__ float buf[2][MAX_WARPS][1];
    const int tid = threadIdx.x % a.tpr;
    const long long row = (long long)blockIdx.x * (blockDim.x / a.tpr) + threadIdx.x / a.tpr;
    const bool live = row < a.rows;
    const int b = live ? (int)(row / a.N) : 0, t = live ? (int)(row - (long long)b * a.N) : 0;
    float x[NV][8], rstd[NV];
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
        if (n > 0) {
            load_heads<VEC>(a.o, a.o_head, a.d, b, t, c0, n, x[j]);
            if (a.gate.p) {
                float g[8];
                load8<VEC>(a.gate.at(b, t) + c0, n, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] *= silu(g[i]);
            }
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[j][i], x[j][i], s);
        rstd[j] = s;
        ss[0] += s;
    }
    if (a.w_post) {
        if (a.group == a.D) {
            row_sum<1>(ss, a.tpr, buf[0]);
#pragma unroll
            for (int j = 0; j < NV; ++j) rstd[j] = rsqrtf(ss[0] * a.inv_group + a.eps);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) rstd[j] = rsqrtf(group_sum(rstd[j], a.group / 8) * a.inv_group + a.eps);
        }
    }
    float s2[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
        if (n > 0) {
            if (a.w_post) {
                float w[8];
                load8<VEC>(a.w_post + c0, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] *= rstd[j] * w[i];
            }
            if (a.residual.p) {
                float sc[8], r[8];
                load_param<VEC>(a.scale, c0, n, 1.f, sc);
                load8<VEC>(a.residual.at(b, t) + c0, n, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = fmaf(sc[i], x[j][i], r[i]);
            }
            store8<VEC>(a.r.at(b, t) + c0, n, x[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[j][i] = i < n ? to_f32<R>(from_f32<R>(x[j][i])) : 0.f;   // as stored
                s2[0] = fmaf(x[j][i], x[j][i], s2[0]);
            }
        }
    }
    if (!a.w_pre) return;
    row_sum<1>(s2, a.tpr, buf[1]);
    const float rs = rsqrtf(s2[0] * a.inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
        if (n > 0) {
            float w[8];
            load8<VEC>(a.w_pre + c0, n, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= x[j][i] * rs;
            store8<VEC>(a.h.at(b, t) + c0, n, w);
        }
    }
}

template <typename T, typename R> struct NormGradArgs {
    NormArgs<T, R> f;
    Rows<const R> dr;
    Rows<const T> dh;
    Rows<T> d_o;
    long long d_o_head;
    Rows<T> dgate;
    Rows<R> dresidual;
    float *part;                  // [blocks][3][pitch]: w_post, scale, w_pre
    int pitch;
};

// The adjoint, row by row, from the same inputs and the stored r':
//   dr' = dr + rstd2 (m - r' rstd2^2 mean(m r')),  m = w_pre dh;   dw_pre = sum dh r' rstd2;
//   dv = scale dr';  dscale = sum dr' v;  dw_post = sum dv a rstd;
//   da = rstd (q - a rstd^2 mean(q a)),  q = w_post dv;   do = da silu(gate), dgate = da o silu'(gate).
// Blocks walk over the rows with the parameter gradients of their channels in registers, add up
// their row lanes in order and leave one partial row each; sum_rows adds those in order.
template <typename T, typename R, bool VEC, int NV>
__global__ void __launch_bounds__(NV == 1 ? 256 : 1024) norm_backward_kernel(const NormGradArgs<T, R> g)
{
    extern __shared__ float part_s[];                      // [blockDim.x][8]
    __shared__ float buf[2][MAX_WARPS][3], buf2[2][MAX_WARPS][1];
    const NormArgs<T, R> &a = g.f;
    const int tid = threadIdx.x % a.tpr, lane_row = threadIdx.x / a.tpr, per = blockDim.x / a.tpr;
    float dwpost[NV][8], dscale[NV][8], dwpre[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dwpost[j][i] = dscale[j][i] = dwpre[j][i] = 0.f;
    int turn = 0;
    for (long long row0 = (long long)blockIdx.x * per; row0 < a.rows; row0 += (long long)gridDim.x * per, turn ^= 1) {
        const long long row = row0 + lane_row;
        const bool live = row < a.rows;
        const int b = live ? (int)(row / a.N) : 0, t = live ? (int)(row - (long long)b * a.N) : 0;
        float o[NV][8], gt[NV][8], rf[NV][8], dh[NV][8], dr[NV][8], gs[NV];
        float sums[3] = {0.f, 0.f, 0.f};                   // r'^2, m r', a^2
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[j][i] = gt[j][i] = rf[j][i] = dh[j][i] = dr[j][i] = 0.f;
            gs[j] = 0.f;
            if (n > 0) {
                load_heads<VEC>(a.o, a.o_head, a.d, b, t, c0, n, o[j]);
                if (a.gate.p) load8<VEC>(a.gate.at(b, t) + c0, n, gt[j]);
                if (g.dr.p) load8<VEC>(g.dr.at(b, t) + c0, n, dr[j]);
                if (g.dh.p) {
                    float w[8];
                    load8<VEC>(Rows<const R>{a.r.p, a.r.sb, a.r.st}.at(b, t) + c0, n, rf[j]);
                    load8<VEC>(g.dh.at(b, t) + c0, n, dh[j]);
                    load8<VEC>(a.w_pre + c0, n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sums[0] = fmaf(rf[j][i], rf[j][i], sums[0]);
                        sums[1] = fmaf(dh[j][i] * w[i], rf[j][i], sums[1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = a.gate.p ? o[j][i] * silu(gt[j][i]) : o[j][i];
                    gs[j] = fmaf(v, v, gs[j]);
                }
                sums[2] += gs[j];
            }
        }
        if (g.dh.p || (a.w_post && a.group == a.D)) row_sum<3>(sums, a.tpr, buf[turn]);
        const float rs2 = rsqrtf(sums[0] * a.inv_d + a.eps);
        const float k2 = rs2 * rs2 * sums[1] * a.inv_d;
        float rstd[NV], dots[NV], dot[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
            rstd[j] = 1.f;
            if (a.w_post)
                rstd[j] = rsqrtf((a.group == a.D ? sums[2] : group_sum(gs[j], a.group / 8)) * a.inv_group + a.eps);
            dots[j] = 0.f;
            if (n > 0) {
                if (g.dh.p) {
                    float w[8];
                    load8<VEC>(a.w_pre + c0, n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dwpre[j][i] = fmaf(dh[j][i] * rf[j][i], rs2, dwpre[j][i]);
                        dr[j][i] = fmaf(rs2, fmaf(-rf[j][i], k2, dh[j][i] * w[i]), dr[j][i]);
                    }
                }
                if (g.dresidual.p) store8<VEC>(g.dresidual.at(b, t) + c0, n, dr[j]);
                float w[8], sc[8];
                load_param<VEC>(a.w_post, c0, n, 1.f, w);
                load_param<VEC>(a.scale, c0, n, 1.f, sc);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = a.gate.p ? o[j][i] * silu(gt[j][i]) : o[j][i];
                    const float nrm = v * rstd[j], dv = dr[j][i] * sc[i];
                    dscale[j][i] = fmaf(dr[j][i], nrm * w[i], dscale[j][i]);
                    dwpost[j][i] = fmaf(dv, nrm, dwpost[j][i]);
                    dr[j][i] = dv * w[i];                  // q
                    dots[j] = fmaf(dr[j][i], v, dots[j]);
                }
                dot[0] += dots[j];
            }
        }
        if (a.w_post && a.group == a.D) row_sum<1>(dot, a.tpr, buf2[turn]);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
            float k1 = 0.f;
            if (a.w_post)
                k1 = rstd[j] * rstd[j] * a.inv_group * (a.group == a.D ? dot[0] : group_sum(dots[j], a.group / 8));
            if (n > 0) {
                float dov[8], dg[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = a.gate.p ? sigmoid(gt[j][i]) : 1.f, act = a.gate.p ? gt[j][i] * s : 1.f;
                    const float v = o[j][i] * act;
                    const float da = rstd[j] * fmaf(-v, k1, dr[j][i]);
                    dov[i] = da * act;
                    dg[i] = da * o[j][i] * dsilu(gt[j][i], s);
                }
                store_heads<VEC>(g.d_o, g.d_o_head, a.d, b, t, c0, n, dov);
                if (a.gate.p) store8<VEC>(g.dgate.at(b, t) + c0, n, dg);
            }
        }
    }
    // the block's row lanes, in order
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part_s[i * blockDim.x + threadIdx.x] = k == 0 ? dwpost[j][i] : k == 1 ? dscale[j][i] : dwpre[j][i];
            __syncthreads();
            const int c0 = (j * a.tpr + tid) * 8;
            for (int i = lane_row; i < 8; i += per) {
                float v = 0.f;
                for (int l = 0; l < per; ++l) v += part_s[i * blockDim.x + l * a.tpr + tid];
                if (c0 + i < a.D) g.part[((long long)blockIdx.x * 3 + k) * g.pitch + c0 + i] = v;
            }
        }
    }
}

// ------------------------------------------------------------------ host side
struct Plan {
    int tpr, nv, threads;
};

// Threads per row: enough for the row's pieces of eight channels, nv pieces a thread, a power of two
// from 8 on.  Blocks have 256 threads, or one row if that takes more.
Plan plan(int D, int nv)
{
    const int pieces = (D + 7) / 8;
    int tpr = 8;
    while (tpr * nv < pieces) tpr *= 2;
    return Plan{tpr, nv, tpr > 256 ? tpr : 256};
}

gma_status_t check(const gma_norm_t *n, bool forward)
{
    if (!n) return GMA_ERR_INVALID_ARG;
    if (n->B < 1 || n->N < 1 || n->H < 1 || n->d < 1 || !(n->eps >= 0.f)) return GMA_ERR_INVALID_ARG;
    if (n->dtype != GMA_F32 && n->dtype != GMA_BF16) return GMA_ERR_INVALID_ARG;
    if (n->residual.ptr && n->residual_dtype != GMA_F32 && n->residual_dtype != n->dtype) return GMA_ERR_INVALID_ARG;
    const long long D = (long long)n->H * n->d;
    if (D > 16384 || n->B > 65535 || n->N > (1 << 30)) return GMA_ERR_UNSUPPORTED_SHAPE;
    const int g = n->group;
    if (g != D && !((g == 8 || g == 16 || g == 32 || g == 64 || g == 128 || g == 256) && D % g == 0))
        return GMA_ERR_UNSUPPORTED_SHAPE;
    const int rd = n->residual.ptr ? n->residual_dtype : n->dtype;
    if (!n->w_post && !n->w_pre) return GMA_ERR_INVALID_ARG;
    if (n->scale && !n->residual.ptr) return GMA_ERR_INVALID_ARG;
    if (!opt_ok(n->w_post, 4) || !opt_ok(n->w_pre, 4) || !opt_ok(n->scale, 4)) return GMA_ERR_INVALID_ARG;
    if (n->o_head < 0 || !rows_ok(n->o, n->dtype, n->B, n->N, n->d, false)) return GMA_ERR_INVALID_ARG;
    if (n->gate.ptr && !rows_ok(n->gate, n->dtype, n->B, n->N, D, false)) return GMA_ERR_INVALID_ARG;
    if (forward) {
        if (n->residual.ptr && !rows_ok(n->residual, rd, n->B, n->N, D, false)) return GMA_ERR_INVALID_ARG;
        if (!rows_ok(n->r, rd, n->B, n->N, D, true)) return GMA_ERR_INVALID_ARG;
        if (n->w_pre && !rows_ok(n->h, n->dtype, n->B, n->N, D, true)) return GMA_ERR_INVALID_ARG;
    }
    return GMA_OK;
}

template <typename T, typename R> NormArgs<T, R> args_of(const gma_norm_t &n, int tpr)
{
    NormArgs<T, R> a;
    a.N = n.N; a.d = n.d; a.D = n.H * n.d; a.group = n.group; a.tpr = tpr;
    a.rows = (long long)n.B * n.N;
    a.eps = n.eps; a.inv_d = 1.f / a.D; a.inv_group = 1.f / n.group;
    a.o = rows_of<const T>(n.o); a.o_head = n.o_head;
    a.gate = rows_of<const T>(n.gate);
    a.residual = rows_of<const R>(n.residual);
    a.w_post = n.w_post; a.scale = n.scale; a.w_pre = n.w_pre;
    a.r = rows_of<R>(n.r);
    a.h = rows_of<T>(n.h);
    return a;
}

bool vec_given(const gma_rows_t &r, int dtype) { return !r.ptr || rows_vec(r, dtype); }

bool vec_common(const gma_norm_t &n)
{
    return n.d % 8 == 0 && rows_vec(n.o, n.dtype) && (n.o_head * elem_size(n.dtype)) % 16 == 0 &&
           vec_given(n.gate, n.dtype) && opt_ok(n.w_post, 16) && opt_ok(n.scale, 16) && opt_ok(n.w_pre, 16);
}

// Calls f(T{}, R{}, VEC, NV).
template <typename F> gma_status_t dispatch(const gma_norm_t &n, bool vec, int nv, F f)
{
    auto with_types = [&](auto t, auto r) -> gma_status_t {
        auto with_nv = [&](auto v) -> gma_status_t {
            if (nv == 1) return f(t, r, v, std::integral_constant<int, 1>{});
            return f(t, r, v, std::integral_constant<int, 2>{});
        };
        return vec ? with_nv(std::true_type{}) : with_nv(std::false_type{});
    };
    if (n.dtype == GMA_F32) return with_types(float{}, float{});
    if (n.residual.ptr && n.residual_dtype == GMA_F32) return with_types(__nv_bfloat16{}, float{});
    return with_types(__nv_bfloat16{}, __nv_bfloat16{});
}

// Two pieces a thread only where one would take more threads than a block has.
Plan plan_rows(int D) { return D > 8 * 1024 ? plan(D, 2) : plan(D, 1); }
Plan plan_grad(int D) { return D > 8 * 256 ? plan(D, 2) : plan(D, 1); }

int grad_blocks(const gma_norm_t &n, const Plan &p)
{
    const long long rows = (long long)n.B * n.N, per = p.threads / p.tpr;
    const long long want = 152ll * (1024 / p.threads);
    return (int)std::min((rows + per - 1) / per, want);
}

}  // namespace
}  // namespace blk
}  // namespace gma

using namespace gma;
using namespace gma::blk;

extern "C" {

gma_status_t gma_norm_forward(const gma_norm_t *n, gma_stream_t stream)
{
    gma_status_t r = check(n, true);
    if (r != GMA_OK) return r;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const int D = n->H * n->d, rd = n->residual.ptr ? n->residual_dtype : n->dtype;
    const Plan p = plan_rows(D);
    const bool vec = vec_common(*n) && vec_given(n->residual, rd) && rows_vec(n->r, rd) &&
                     (!n->w_pre || rows_vec(n->h, n->dtype));
    return dispatch(*n, vec, p.nv, [&](auto t, auto rt, auto v, auto nv) -> gma_status_t {
        using T = decltype(t);
        using R = decltype(rt);
        const NormArgs<T, R> a = args_of<T, R>(*n, p.tpr);
        const long long per = p.threads / p.tpr, blocks = (a.rows + per - 1) / per;
        if (blocks > 0x7fffffffll) return GMA_ERR_UNSUPPORTED_SHAPE;
        GMA_LAUNCH(KID_NORM, st,
                   norm_forward_kernel<T, R, decltype(v)::value, decltype(nv)::value>
                   <<<(unsigned)blocks, p.threads, 0, st>>>(a));
        return GMA_OK;
    });
}

size_t gma_norm_backward_workspace_size(const gma_norm_grad_t *g)
{
    if (!g || check(&g->fwd, false) != GMA_OK) return 0;
    const int D = g->fwd.H * g->fwd.d;
    return align_up((size_t)grad_blocks(g->fwd, plan_grad(D)) * 3 * ((D + 7) / 8 * 8) * sizeof(float), 256);
}

gma_status_t gma_norm_backward(const gma_norm_grad_t *g, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    if (!g) return GMA_ERR_INVALID_ARG;
    const gma_norm_t &n = g->fwd;
    gma_status_t r = check(&n, false);
    if (r != GMA_OK) return r;
    const int D = n.H * n.d, rd = n.residual.ptr ? n.residual_dtype : n.dtype;
    if (!g->dr.ptr && !g->dh.ptr) return GMA_ERR_INVALID_ARG;
    if (g->dr.ptr && !rows_ok(g->dr, rd, n.B, n.N, D, false)) return GMA_ERR_INVALID_ARG;
    if (g->dh.ptr && (!n.w_pre || !rows_ok(g->dh, n.dtype, n.B, n.N, D, false))) return GMA_ERR_INVALID_ARG;
    if (g->dh.ptr && !rows_ok(n.r, rd, n.B, n.N, D, false)) return GMA_ERR_INVALID_ARG;
    if (!rows_ok(g->d_o, n.dtype, n.B, n.N, n.d, true) || (n.H > 1 && g->d_o_head < n.d)) return GMA_ERR_INVALID_ARG;
    if (n.gate.ptr && !rows_ok(g->dgate, n.dtype, n.B, n.N, D, true)) return GMA_ERR_INVALID_ARG;
    if (g->dresidual.ptr && !rows_ok(g->dresidual, rd, n.B, n.N, D, true)) return GMA_ERR_INVALID_ARG;
    if ((n.w_post && !ptr_ok(g->dw_post, 4)) || (n.scale && !ptr_ok(g->dscale, 4)) ||
        (n.w_pre && !ptr_ok(g->dw_pre, 4)))
        return GMA_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, gma_norm_backward_workspace_size(g))) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const Plan p = plan_grad(D);
    const bool vec = vec_common(n) && vec_given(g->dr, rd) && vec_given(g->dh, n.dtype) &&
                     (!g->dh.ptr || rows_vec(n.r, rd)) && rows_vec(g->d_o, n.dtype) &&
                     (g->d_o_head * elem_size(n.dtype)) % 16 == 0 && (!n.gate.ptr || rows_vec(g->dgate, n.dtype)) &&
                     vec_given(g->dresidual, rd);
    return dispatch(n, vec, p.nv, [&](auto t, auto rt, auto v, auto nv) -> gma_status_t {
        using T = decltype(t);
        using R = decltype(rt);
        NormGradArgs<T, R> a;
        a.f = args_of<T, R>(n, p.tpr);
        a.dr = rows_of<const R>(g->dr);
        a.dh = rows_of<const T>(g->dh);
        a.d_o = rows_of<T>(g->d_o);
        a.d_o_head = g->d_o_head;
        a.dgate = rows_of<T>(g->dgate);
        a.dresidual = rows_of<R>(g->dresidual);
        a.part = (float *)ws;
        a.pitch = (D + 7) / 8 * 8;
        const int blocks = grad_blocks(n, p);
        GMA_LAUNCH(KID_NORM_BWD, st,
                   norm_backward_kernel<T, R, decltype(v)::value, decltype(nv)::value>
                   <<<blocks, p.threads, p.threads * 8 * sizeof(float), st>>>(a));
        SumOut out[3] = {{g->dw_post, 1}, {g->dscale, 1}, {g->dw_pre, 1}};
        for (int k = 0; k < 3; ++k) {      // neighbouring vectors that are wanted, in one launch
            if (!(k == 0 ? (const void *)n.w_post : k == 1 ? (const void *)n.scale : (const void *)n.w_pre)) continue;
            int e = k + 1;
            while (e < 3 && (e == 1 ? (const void *)n.scale : (const void *)n.w_pre)) ++e;
            const gma_status_t q = sum_rows(a.part + (size_t)k * a.pitch, blocks, e - k, 3, D, a.pitch, out + k, st);
            if (q != GMA_OK) return q;
            k = e - 1;
        }
        return GMA_OK;
    });
}

}  // extern "C"
