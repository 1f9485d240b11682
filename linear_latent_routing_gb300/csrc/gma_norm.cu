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
// Measured: per-head norm with a gate of 65536 x 2048 bf16 in 125 us (6.4 TB/s); both norms with gate, scale and an
// fp32 residual of 8192 x 2048 in 44 us (5.3 TB/s) forward and 81 us (4.6 TB/s) backward.  From 4097 channels on the
// backward kernels spill (about 430 bytes a thread, 2100 from 8193 on); those widths are not timed.
#include <algorithm>
#include <type_traits>

#include "block_common.cuh"

namespace gma {
namespace blk {
namespace {

constexpr int MAX_WARPS = 16;
constexpr int FORWARD_BLOCKS = 4, BACKWARD_BLOCKS = 2;   // blocks of 256 threads an SM, by their registers
constexpr int TWO_ROWS = 152 * 8;                        // blocks from which a thread takes two rows

// n / d for n < 2^31 by a multiplication (the divisor's rounded-up reciprocal): a row's batch row and token
// and a channel's head would otherwise take as many instructions as the row's arithmetic.
struct FastDiv {
    uint32_t d, m, s1, s2;
    __device__ __forceinline__ uint32_t div(uint32_t n) const
    {
        const uint32_t t = __umulhi(n, m);
        return (t + ((n - t) >> s1)) >> s2;
    }
};
FastDiv fast_div(uint32_t d)
{
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return FastDiv{d, (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l ? 1u : 0u, l ? l - 1 : 0u};
}

template <typename T, typename R> struct NormArgs {
    int N, D, group, tpr, tpr_log;   // tpr: threads per row, a power of two
    FastDiv by_n, by_d;
    int rows;                     // B * N
    float eps, inv_d, inv_group;
    Rows<const T> o;
    long long o_head;
    Rows<const T> gate;
    Rows<const R> residual;
    const float *w_post, *scale, *w_pre;
    Rows<R> r;
    Rows<T> h;
};

// Offset of channel c in a token of the head layout.
__device__ __forceinline__ long long head_offset(const FastDiv &by_d, long long head, int c)
{
    const int hd = by_d.div(c);
    return hd * head + (c - hd * (int)by_d.d);
}

// Channels c0 .. c0 + 7 of token (b, t) in the head layout.  VEC: d is a multiple of eight.
template <bool VEC, typename T>
__device__ __forceinline__ void load_heads(const Rows<const T> &o, long long head, const FastDiv &by_d, int b, int t, int c0, int n,
                                           float (&v)[8])
{
    const T *p = o.at(b, t);
    if (VEC) {
        load8<true>(p + head_offset(by_d, head, c0), n, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = i < n ? to_f32<T>(p[head_offset(by_d, head, c0 + i)]) : 0.f;
        }
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_heads(const Rows<T> &o, long long head, const FastDiv &by_d, int b, int t, int c0, int n,
                                            const float (&v)[8])
{
    T *p = o.at(b, t);
    if (VEC) {
        store8<true>(p + head_offset(by_d, head, c0), n, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < n) p[head_offset(by_d, head, c0 + i)] = from_f32<T>(v[i]);
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
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = tpr >> 5, first = warp & ~(per - 1);
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) buf[warp][k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = buf[first + (lane & (per - 1))][k];
        for (int off = per / 2; off; off >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    }
}

// Sum over the group that a thread's eight channels belong to: group / 8 neighbouring lanes (a power
// of two up to 32).
__device__ __forceinline__ float group_sum(float v, int lanes)
{
    for (int off = lanes / 2; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// A thread takes its pieces of ROWS rows at a time, so that the loads of all of them are in flight
// together: one row for few rows (latency), two where the GPU is full.
// GATED: a norm after a mixer, gate and w_post alone: nothing branches on what is given, and with 40 registers (bf16) six
// blocks run an SM (65536 x 2048 by heads: 161 -> 132 us, with the six blocks 125 us).  The same for the case where
// everything is given gained nothing.
template <typename T, bool GATED> constexpr int forward_blocks() { return GATED && sizeof(T) == 2 ? 6 : FORWARD_BLOCKS; }
template <typename T, typename R, bool VEC, int NV, int THREADS, int ROWS, bool GATED>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? forward_blocks<T, GATED>() : 1) norm_forward_kernel(const NormArgs<T, R> a)
{
    __shared__ float buf[2][MAX_WARPS][ROWS];
    const bool gate = GATED || a.gate.p, post = GATED || a.w_post, residual = !GATED && a.residual.p, pre = !GATED && a.w_pre;
    const int tid = threadIdx.x & (a.tpr - 1), lane_row = threadIdx.x >> a.tpr_log, per = THREADS >> a.tpr_log;
    int b[ROWS], t[ROWS];
    bool live[ROWS];
    float x[ROWS][NV][8], res[ROWS][NV][8], rstd[ROWS][NV], ss[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int row = (blockIdx.x * ROWS + r) * per + lane_row;
        live[r] = row < a.rows;
        b[r] = live[r] ? a.by_n.div(row) : 0;
        t[r] = live[r] ? row - b[r] * a.N : 0;
    }
    Raw8<T> on[ROWS][NV], gn[ROWS][NV];
    Raw8<R> rn[ROWS][NV];
    if (VEC) {
        long long head_at[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) head_at[j] = head_offset(a.by_d, a.o_head, (j * a.tpr + tid) * 8);
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c0 = (j * a.tpr + tid) * 8;
                if (!live[r] || c0 >= a.D) continue;
                on[r][j].load(a.o.at(b[r], t[r]) + head_at[j]);
                if (gate) gn[r][j].load(a.gate.at(b[r], t[r]) + c0);
                if (residual) rn[r][j].load(a.residual.at(b[r], t[r]) + c0);
            }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        ss[r] = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * a.tpr + tid) * 8, n = live[r] ? min(8, a.D - c0) : 0;
            float(&v)[8] = x[r][j];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = res[r][j][i] = 0.f;
            if (n > 0) {
                float g[8];
                if (VEC) {
                    on[r][j].get(v);
                    if (gate) gn[r][j].get(g);
                    if (residual) rn[r][j].get(res[r][j]);
                } else {
                    load_heads<false>(a.o, a.o_head, a.by_d, b[r], t[r], c0, n, v);
                    if (gate) load8<false>(a.gate.at(b[r], t[r]) + c0, n, g);
                    if (residual) load8<false>(a.residual.at(b[r], t[r]) + c0, n, res[r][j]);
                }
                if (gate) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= silu(g[i]);
                }
            }
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
            rstd[r][j] = s;
            ss[r] += s;
        }
    }
    if (post) {
        if (a.group == a.D) row_sum<ROWS>(ss, a.tpr, buf[0]);
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                rstd[r][j] = rsqrtf((a.group == a.D ? ss[r] : group_sum(rstd[r][j], a.group / 8)) * a.inv_group + a.eps);
    }
    float s2[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s2[r] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.tpr + tid) * 8, n = min(8, a.D - c0);
        if (n <= 0) continue;
        float w[8], sc[8];
        if (GATED) load8<VEC>(a.w_post + c0, n, w);
        else load_param<VEC>(a.w_post, c0, n, 1.f, w);
        if (!GATED) load_param<VEC>(a.scale, c0, n, 1.f, sc);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (!live[r]) continue;
            float(&v)[8] = x[r][j];
            if (post) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= rstd[r][j] * w[i];
            }
            if (residual) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = fmaf(sc[i], v[i], res[r][j][i]);
            }
            store8<VEC>(a.r.at(b[r], t[r]) + c0, n, v);
            if (pre) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = i < n ? to_f32<R>(from_f32<R>(v[i])) : 0.f;   // as stored
                    s2[r] = fmaf(v[i], v[i], s2[r]);
                }
            }
        }
    }
    if (!pre) return;
    row_sum<ROWS>(s2, a.tpr, buf[1]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.tpr + tid) * 8, n = min(8, a.D - c0);
        if (n <= 0) continue;
        float w[8];
        load8<VEC>(a.w_pre + c0, n, w);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (!live[r]) continue;
            const float rs = rsqrtf(s2[r] * a.inv_d + a.eps);
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = w[i] * x[r][j][i] * rs;
            store8<VEC>(a.h.at(b[r], t[r]) + c0, n, h);
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
// FULL: every input and parameter is there (a block in training), so nothing branches on them.
template <typename T, typename R, bool VEC, int NV, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? BACKWARD_BLOCKS : 1) norm_backward_kernel(const NormGradArgs<T, R> g)
{
    extern __shared__ float part_s[];                      // [8][THREADS]
    __shared__ float buf[2][MAX_WARPS][3], buf2[2][MAX_WARPS][1];
    constexpr bool AHEAD = VEC && NV == 1;        // wider rows have no registers left for it
    let_next();
    const NormArgs<T, R> &a = g.f;
    const bool gate = FULL || a.gate.p, has_dr = FULL || g.dr.p, has_dh = FULL || g.dh.p, post = FULL || a.w_post;
    const int tid = threadIdx.x & (a.tpr - 1), lane_row = threadIdx.x >> a.tpr_log, per = THREADS >> a.tpr_log;
    float dwpost[NV][8], dscale[NV][8], dwpre[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dwpost[j][i] = dscale[j][i] = dwpre[j][i] = 0.f;
    Raw8<T> on[NV], gn[NV], hn[NV];
    Raw8<R> dn[NV], rn[NV];
    const Rows<const R> kept{a.r.p, a.r.sb, a.r.st};
    long long head_at[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) head_at[j] = head_offset(a.by_d, a.o_head, (j * a.tpr + tid) * 8);
    auto fetch = [&](int row) {
        if (!AHEAD || row >= a.rows) return;
        const int b = a.by_n.div(row), t = row - b * a.N;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * a.tpr + tid) * 8;
            if (c0 >= a.D) continue;
            on[j].load(a.o.at(b, t) + head_at[j]);
            if (gate) gn[j].load(a.gate.at(b, t) + c0);
            if (has_dr) dn[j].load(g.dr.at(b, t) + c0);
            if (has_dh) {
                rn[j].load(kept.at(b, t) + c0);
                hn[j].load(g.dh.at(b, t) + c0);
            }
        }
    };
    const int step = gridDim.x * per;
    int row = blockIdx.x * per + lane_row;
    fetch(row);
    int turn = 0;
    for (int row0 = blockIdx.x * per; row0 < a.rows; row0 += step, row += step, turn ^= 1) {
        const bool live = row < a.rows;
        const int b = live ? a.by_n.div(row) : 0, t = live ? row - b * a.N : 0;
        // act[] = o silu(gate); by_o[], by_gate[]: its derivatives
        float act[NV][8], by_o[NV][8], by_gate[NV][8], rf[NV][8], dh[NV][8], dr[NV][8], gs[NV];
        float sums[3] = {0.f, 0.f, 0.f};                   // r'^2, m r', act^2
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) act[j][i] = by_o[j][i] = by_gate[j][i] = rf[j][i] = dh[j][i] = dr[j][i] = 0.f;
            gs[j] = 0.f;
            if (n > 0) {
                float o[8], gt[8];
                if (AHEAD) {
                    on[j].get(o);
                    if (gate) gn[j].get(gt);
                    if (has_dr) dn[j].get(dr[j]);
                    if (has_dh) {
                        rn[j].get(rf[j]);
                        hn[j].get(dh[j]);
                    }
                } else {
                    load_heads<VEC>(a.o, a.o_head, a.by_d, b, t, c0, n, o);
                    if (gate) load8<VEC>(a.gate.at(b, t) + c0, n, gt);
                    if (has_dr) load8<VEC>(g.dr.at(b, t) + c0, n, dr[j]);
                    if (has_dh) {
                        load8<VEC>(kept.at(b, t) + c0, n, rf[j]);
                        load8<VEC>(g.dh.at(b, t) + c0, n, dh[j]);
                    }
                }
                if (has_dh) {
                    float w[8];
                    load8<VEC>(a.w_pre + c0, n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sums[0] = fmaf(rf[j][i], rf[j][i], sums[0]);
                        sums[1] = fmaf(dh[j][i] * w[i], rf[j][i], sums[1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (gate) {
                        const float s = sigmoid(gt[i]);
                        by_o[j][i] = gt[i] * s;
                        by_gate[j][i] = o[i] * dsilu(gt[i], s);
                    } else {
                        by_o[j][i] = 1.f;
                    }
                    act[j][i] = o[i] * by_o[j][i];
                    gs[j] = fmaf(act[j][i], act[j][i], gs[j]);
                }
                sums[2] += gs[j];
            }
        }
        fetch(row + step);
        if (has_dh || (post && a.group == a.D)) row_sum<3>(sums, a.tpr, buf[turn]);
        const float rs2 = rsqrtf(sums[0] * a.inv_d + a.eps);
        const float k2 = rs2 * rs2 * sums[1] * a.inv_d;
        float rstd[NV], dots[NV], dot[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
            rstd[j] = 1.f;
            if (post)
                rstd[j] = rsqrtf((a.group == a.D ? sums[2] : group_sum(gs[j], a.group / 8)) * a.inv_group + a.eps);
            dots[j] = 0.f;
            if (n > 0) {
                if (has_dh) {
                    float w[8];
                    load8<VEC>(a.w_pre + c0, n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dwpre[j][i] = fmaf(dh[j][i] * rf[j][i], rs2, dwpre[j][i]);
                        dr[j][i] = fmaf(rs2, fmaf(-rf[j][i], k2, dh[j][i] * w[i]), dr[j][i]);
                    }
                }
                if (FULL || g.dresidual.p) store8<VEC>(g.dresidual.at(b, t) + c0, n, dr[j]);
                float w[8], sc[8];
                if (FULL) {
                    load8<VEC>(a.w_post + c0, n, w);
                    load8<VEC>(a.scale + c0, n, sc);
                } else {
                    load_param<VEC>(a.w_post, c0, n, 1.f, w);
                    load_param<VEC>(a.scale, c0, n, 1.f, sc);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float nrm = act[j][i] * rstd[j], dv = dr[j][i] * sc[i];
                    dscale[j][i] = fmaf(dr[j][i], nrm * w[i], dscale[j][i]);
                    dwpost[j][i] = fmaf(dv, nrm, dwpost[j][i]);
                    dr[j][i] = dv * w[i];                  // q
                    dots[j] = fmaf(dr[j][i], act[j][i], dots[j]);
                }
                dot[0] += dots[j];
            }
        }
        if (post && a.group == a.D) row_sum<1>(dot, a.tpr, buf2[turn]);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * a.tpr + tid) * 8, n = live ? min(8, a.D - c0) : 0;
            float k1 = 0.f;
            if (post)
                k1 = rstd[j] * rstd[j] * a.inv_group * (a.group == a.D ? dot[0] : group_sum(dots[j], a.group / 8));
            if (n > 0) {
                float dov[8], dg[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float da = rstd[j] * fmaf(-act[j][i], k1, dr[j][i]);
                    dov[i] = da * by_o[j][i];
                    dg[i] = da * by_gate[j][i];
                }
                store_heads<VEC>(g.d_o, g.d_o_head, a.by_d, b, t, c0, n, dov);
                if (gate) store8<VEC>(g.dgate.at(b, t) + c0, n, dg);
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
                part_s[i * THREADS + threadIdx.x] = k == 0 ? dwpost[j][i] : k == 1 ? dscale[j][i] : dwpre[j][i];
            __syncthreads();
            const int c0 = (j * a.tpr + tid) * 8;
            for (int i = lane_row; i < 8; i += per) {
                float v = 0.f;
                for (int l = 0; l < per; ++l) v += part_s[i * THREADS + l * a.tpr + tid];
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
// from 8 on.  Blocks have 256 threads, 512 where a row has more than 256 pieces of channels; a thread then
// has as many pieces as that takes (up to four, at 16384 channels).
Plan plan(int D)
{
    const int pieces = (D + 7) / 8;
    Plan p = {8, pieces > 1024 ? 4 : pieces > 512 ? 2 : 1, pieces > 256 ? 512 : 256};
    while (p.tpr * p.nv < pieces) p.tpr *= 2;
    return p;
}

// An output in place of an input: each thread reads its piece of a row before it writes that piece, so their rows have
// to be the same ones (a broadcast input's first row is also the others' input).
bool same_rows(const gma_rows_t &out, const gma_rows_t &in, int B, int N)
{
    return out.ptr != in.ptr || ((B == 1 || out.batch == in.batch) && (N == 1 || out.token == in.token));
}

gma_status_t check(const gma_norm_t *n, bool forward)
{
    if (!n) return GMA_ERR_INVALID_ARG;
    if (n->B < 1 || n->N < 1 || n->H < 1 || n->d < 1 || !(n->eps >= 0.f)) return GMA_ERR_INVALID_ARG;
    if (n->dtype != GMA_F32 && n->dtype != GMA_BF16) return GMA_ERR_INVALID_ARG;
    if (n->residual.ptr && n->residual_dtype != GMA_F32 && n->residual_dtype != n->dtype) return GMA_ERR_INVALID_ARG;
    const long long D = (long long)n->H * n->d;
    if (D > 16384 || (long long)n->B * n->N > (1ll << 30)) return GMA_ERR_UNSUPPORTED_SHAPE;
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
        if (!same_rows(n->r, n->residual, n->B, n->N)) return GMA_ERR_INVALID_ARG;
        if (n->w_pre && !rows_ok(n->h, n->dtype, n->B, n->N, D, true)) return GMA_ERR_INVALID_ARG;
    }
    return GMA_OK;
}

template <typename T, typename R> NormArgs<T, R> args_of(const gma_norm_t &n, int tpr)
{
    NormArgs<T, R> a;
    a.N = n.N; a.D = n.H * n.d; a.group = n.group; a.tpr = tpr; a.tpr_log = 0;
    while ((1 << a.tpr_log) < tpr) ++a.tpr_log;
    a.rows = n.B * n.N;
    a.by_n = fast_div(n.N);
    a.by_d = fast_div(n.d);
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

// Calls f(T{}, R{}, VEC, NV, THREADS).
template <typename F> gma_status_t dispatch(const gma_norm_t &n, bool vec, const Plan &p, F f)
{
    auto with_types = [&](auto t, auto r) -> gma_status_t {
        auto with_plan = [&](auto v) -> gma_status_t {
            typedef std::integral_constant<int, 512> Wide;
            if (p.threads == 256) return f(t, r, v, std::integral_constant<int, 1>{}, std::integral_constant<int, 256>{});
            if (p.nv == 1) return f(t, r, v, std::integral_constant<int, 1>{}, Wide{});
            if (p.nv == 2) return f(t, r, v, std::integral_constant<int, 2>{}, Wide{});
            return f(t, r, v, std::integral_constant<int, 4>{}, Wide{});
        };
        return vec ? with_plan(std::true_type{}) : with_plan(std::false_type{});
    };
    if (n.dtype == GMA_F32) return with_types(float{}, float{});
    if (n.residual.ptr && n.residual_dtype == GMA_F32) return with_types(__nv_bfloat16{}, float{});
    return with_types(__nv_bfloat16{}, __nv_bfloat16{});
}

// Blocks that walk over the rows: as many as run at once.
int blocks_of(const gma_norm_t &n, const Plan &p, int per_sm)
{
    const long long rows = (long long)n.B * n.N, per = p.threads / p.tpr;
    return (int)std::min((rows + per - 1) / per, 152ll * (p.threads == 256 ? per_sm : 1));
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
    const Plan p = plan(D);
    const bool vec = vec_common(*n) && vec_given(n->residual, rd) && rows_vec(n->r, rd) &&
                     (!n->w_pre || rows_vec(n->h, n->dtype));
    return dispatch(*n, vec, p, [&](auto t, auto rt, auto v, auto nv, auto threads) -> gma_status_t {
        using T = decltype(t);
        using R = decltype(rt);
        constexpr int TH = decltype(threads)::value;
        constexpr bool V = decltype(v)::value;
        constexpr int NV = decltype(nv)::value;
        const NormArgs<T, R> a = args_of<T, R>(*n, p.tpr);
        const int per = TH / p.tpr, blocks = (a.rows + per - 1) / per;
        // two rows a thread from two waves of blocks on
        constexpr bool narrow = V && NV == 1 && TH == 256;
        auto launch = [&](auto gated) -> gma_status_t {
            constexpr bool G = decltype(gated)::value;
            if (narrow && blocks > TWO_ROWS)
                GMA_LAUNCH(KID_NORM, st, norm_forward_kernel<T, R, V, NV, TH, narrow ? 2 : 1, G>
                                         <<<(unsigned)((blocks + 1) / 2), TH, 0, st>>>(a));
            else
                GMA_LAUNCH(KID_NORM, st, norm_forward_kernel<T, R, V, NV, TH, 1, G><<<(unsigned)blocks, TH, 0, st>>>(a));
            return GMA_OK;
        };
        constexpr bool plain = narrow && std::is_same<T, R>::value;      // no residual: r has o's type
        if (plain && n->gate.ptr && n->w_post && !n->residual.ptr && !n->w_pre) return launch(std::bool_constant<plain>{});
        return launch(std::false_type{});
    });
}

size_t gma_norm_backward_workspace_size(const gma_norm_grad_t *g)
{
    if (!g || check(&g->fwd, false) != GMA_OK) return 0;
    const int D = g->fwd.H * g->fwd.d;
    return align_up((size_t)blocks_of(g->fwd, plan(D), BACKWARD_BLOCKS) * 3 * ((D + 7) / 8 * 8) * sizeof(float), 256);
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
    if (g->dresidual.ptr && !same_rows(g->dresidual, g->dr, n.B, n.N)) return GMA_ERR_INVALID_ARG;
    if ((n.w_post && !ptr_ok(g->dw_post, 4)) || (n.scale && !ptr_ok(g->dscale, 4)) ||
        (n.w_pre && !ptr_ok(g->dw_pre, 4)))
        return GMA_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, gma_norm_backward_workspace_size(g))) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const Plan p = plan(D);
    const bool vec = vec_common(n) && vec_given(g->dr, rd) && vec_given(g->dh, n.dtype) &&
                     (!g->dh.ptr || rows_vec(n.r, rd)) && rows_vec(g->d_o, n.dtype) &&
                     (g->d_o_head * elem_size(n.dtype)) % 16 == 0 && (!n.gate.ptr || rows_vec(g->dgate, n.dtype)) &&
                     vec_given(g->dresidual, rd);
    return dispatch(n, vec, p, [&](auto t, auto rt, auto v, auto nv, auto threads) -> gma_status_t {
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
        constexpr int TH = decltype(threads)::value;
        const int blocks = blocks_of(n, p, BACKWARD_BLOCKS);
        constexpr bool V = decltype(v)::value;
        constexpr int NV = decltype(nv)::value;
        const bool full = V && NV == 1 && n.gate.ptr && g->dr.ptr && g->dh.ptr && n.w_post && n.scale && n.w_pre &&
                          g->dresidual.ptr;
        if (full)
            GMA_LAUNCH(KID_NORM_BWD, st,
                       norm_backward_kernel<T, R, V, NV, TH, V && NV == 1><<<blocks, TH, TH * 8 * sizeof(float), st>>>(a));
        else
            GMA_LAUNCH(KID_NORM_BWD, st,
                       norm_backward_kernel<T, R, V, NV, TH, false><<<blocks, TH, TH * 8 * sizeof(float), st>>>(a));
        const float *used[3] = {n.w_post, n.scale, n.w_pre};
        float *out[3] = {g->dw_post, g->dscale, g->dw_pre};
        SumVec vecs[3];
        int count = 0;
        for (int k = 0; k < 3; ++k)
            if (used[k]) vecs[count++] = SumVec{a.part + (size_t)k * a.pitch, 3ll * a.pitch, D, out[k], 1};
        return sum_rows(vecs, count, blocks, st);
    });
}

}  // extern "C"
