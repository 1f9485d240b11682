// gma_scan_bwd.cu -- the selective scan's backward pass (gma_scan_backward).
//
// With p_t the output before the gate, dp_t = dy_t silu(z_t) and g_t[n] = dL / dh_t[n],
//   g_t = c_t dp_t + r_t,   r_{t-1} = exp(delta_t A) g_t   (r behind the last token: dstate_out),
//   dc_t = sum_d dp_t h_t,   db_t = sum_d g_t delta_t u_t,   x_t = sum_n b_t g_t,   q_t[n] = r_{t-1} h_{t-1},
//   du = delta x + D dp,   ddelta = u x + sum_n A q,   dA = sum_t delta q,   ddt = ddelta sigmoid(dt + dt_bias).
// A block walks over its channels' tiles from the last to the first: each tile's states are computed
// again from the checkpoint in front of it, then the adjoint recurrence runs from the tile's end, both
// as a sequential pass over a lane's own tokens with a scan over the time lanes.  db and dc are sums
// over channels: a block adds up its own in shared memory, pair of states by pair of states, and
// leaves partial rows that a last kernel adds in a fixed order.
#include "scan_tile.cuh"

namespace gma {
namespace blk {
namespace {

template <typename T> struct GradArgs {
    ScanArgs<T> f;
    Rows<const T> dy;
    const float *dstate_out;
    Rows<T> du, ddt, dz, db, dc;
    float *da_log, *dd_skip, *ddt_bias, *dstate_in;
    float *bc_part;      // [G * tiles][B][N][2][S]
    float *a_part;       // [B][D][S]
    float *d_part;       // [2][B][D]: d_skip, dt_bias
};

template <class K> struct BackwardSmem {
    static constexpr int U = 0, DT = U + K::CHANNEL_FLOATS * 4, DP = DT + K::CHANNEL_FLOATS * 4;
    static constexpr int RED = (DP + K::CHANNEL_FLOATS * 4 + 15) / 16 * 16;
    static constexpr int PAIRS = RED + K::CH * K::TT * 16;
    // b, c; sums of delta q by lane; rate, state in front of the tile, adjoint behind it
    static size_t bytes(int S) { return PAIRS + (size_t)S * K::TT * 8 + (size_t)S * K::THREADS * 4 + (size_t)3 * K::CH * S * 4; }
};

template <typename T, class K, bool VEC, bool Z>
__global__ void __launch_bounds__(K::THREADS) scan_backward_kernel(const GradArgs<T> g)
{
    static_assert(K::TT == CKPT, "a tile starts at a checkpoint");
    extern __shared__ __align__(16) unsigned char smem[];
    const ScanArgs<T> &a = g.f;
    float *us = reinterpret_cast<float *>(smem + BackwardSmem<K>::U);
    float *dts = reinterpret_cast<float *>(smem + BackwardSmem<K>::DT);
    float *dps = reinterpret_cast<float *>(smem + BackwardSmem<K>::DP);
    ulonglong2 *red = reinterpret_cast<ulonglong2 *>(smem + BackwardSmem<K>::RED);
    f2 *bs = reinterpret_cast<f2 *>(smem + BackwardSmem<K>::PAIRS);
    f2 *cs = bs + a.S / 2 * K::TT;
    f2 *das = cs + a.S / 2 * K::TT;
    float *rate = reinterpret_cast<float *>(das + a.S / 2 * K::THREADS);
    float *hs = rate + K::CH * a.S, *rs = hs + K::CH * a.S;

    const int b = blockIdx.y, group = blockIdx.x / a.tiles, Dg = a.D / a.G;
    const int in_group = (blockIdx.x - group * a.tiles) * K::CH;
    const int c0 = group * Dg + in_group, nch = min(K::CH, Dg - in_group);
    const int len = row_length(a.lengths, b, a.N);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tl = lane % K::LT, ch = warp * K::CPW + lane / K::LT;
    const int nck = (a.N + CKPT - 1) / CKPT;

    for (int i = threadIdx.x; i < K::CH * a.S; i += K::THREADS) {
        const int k = i / a.S;
        const long long at = (long long)(c0 + k) * a.S + i % a.S;
        rate[i] = k < nch ? -expf(a.a_log[at]) * LOG2E : 0.f;
        hs[i] = 0.f;
        rs[i] = k < nch && g.dstate_out ? g.dstate_out[(long long)b * a.D * a.S + at] : 0.f;
    }
    for (int p = 0; p < a.S / 2; ++p) das[p * K::THREADS + threadIdx.x] = 0ull;
    const float skip = a.d_skip && ch < nch ? a.d_skip[c0 + ch] : 0.f;
    float dskip = 0.f, dbias = 0.f;

    for (int t0 = (len - 1) / K::TT * K::TT; t0 >= 0 && len > 0; t0 -= K::TT) {
        __syncthreads();
        for (int i = threadIdx.x; i < K::TT * (K::CH / 8); i += K::THREADS) {
            const int piece = i % (K::CH / 8), t = i / (K::CH / 8), n = min(8, nch - piece * 8);
            float u[8], d[8], y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = d[k] = y[k] = 0.f;
            if (t0 + t < len && n > 0) {
                const int c = c0 + piece * 8;
                load8<VEC>(a.u.at(b, t0 + t) + c, n, u);
                load8<VEC>(a.dt.at(b, t0 + t) + c, n, d);
                load8<VEC>(g.dy.at(b, t0 + t) + c, n, y);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    d[k] = k < n ? softplus(d[k] + (a.dt_bias ? a.dt_bias[c + k] : 0.f)) : 0.f;
                if (Z) {
                    float z[8];
                    load8<VEC>(a.z.at(b, t0 + t) + c, n, z);
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] *= silu(z[k]);
                }
            }
            const int at = K::pos(t);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                us[K::channel(piece * 8 + k) + at] = u[k];
                dts[K::channel(piece * 8 + k) + at] = d[k];
                dps[K::channel(piece * 8 + k) + at] = y[k];
            }
        }
        stage_pairs<K, T, VEC>(a.b, b, group * a.S, t0, len, a.S, bs);
        stage_pairs<K, T, VEC>(a.c, b, group * a.S, t0, len, a.S, cs);
        for (int i = threadIdx.x; i < nch * a.S; i += K::THREADS)
            hs[i] = a.ckpt[(((long long)b * nck + t0 / CKPT) * a.D + c0) * a.S + i];
        __syncthreads();

        float dt[K::TL], u[K::TL], dp[K::TL];
        lane_load<K>(dts + K::channel(ch), tl, dt);
        lane_load<K>(us + K::channel(ch), tl, u);
        lane_load<K>(dps + K::channel(ch), tl, dp);
        f2 x2[K::TL], q2[K::TL], y2[K::TL];           // sums over states of b g, A q, c h
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < K::TL; ++i) {
            total += dt[i];
            x2[i] = q2[i] = y2[i] = 0ull;
            dskip = fmaf(dp[i], u[i], dskip);
        }
        for (int p = 0; p < a.S / 2; ++p) {
            const f2 r2 = *reinterpret_cast<const f2 *>(rate + ch * a.S + 2 * p);
            f2 a2[K::TL], h2[K::TL], h = 0ull, r = 0ull;
#pragma unroll
            for (int q = 0; q < K::TL / 2; ++q) {
                f2 b2[2];
                pair_load<K>(bs, p, tl, q, b2[0], b2[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * q + e;
                    a2[i] = ex2_2(mul2(pack2(dt[i], dt[i]), r2));
                    h2[i] = mul2(b2[e], pack2(dt[i] * u[i], dt[i] * u[i]));
                    h = fma2(a2[i], h, h2[i]);
                }
            }
            const f2 decay = ex2_2(mul2(pack2(total, total), r2));
            f2 d1 = decay;
            scan_up<K::LT>(d1, h, tl);
            const f2 before = *reinterpret_cast<const f2 *>(hs + ch * a.S + 2 * p);
            d1 = __shfl_up_sync(0xffffffffu, d1, 1, K::LT);
            h = __shfl_up_sync(0xffffffffu, h, 1, K::LT);
            const f2 hin = tl ? fma2(d1, before, h) : before;
            h = hin;
#pragma unroll
            for (int i = 0; i < K::TL; ++i) {
                h = fma2(a2[i], h, h2[i]);
                h2[i] = h;
            }
#pragma unroll
            for (int q = K::TL / 2 - 1; q >= 0; --q) {
                f2 c2[2];
                pair_load<K>(cs, p, tl, q, c2[0], c2[1]);
#pragma unroll
                for (int e = 1; e >= 0; --e) {
                    const int i = 2 * q + e;
                    if (Z) y2[i] = fma2(c2[e], h2[i], y2[i]);
                    r = mul2(a2[i], fma2(c2[e], pack2(dp[i], dp[i]), r));
                }
            }
            d1 = decay;
            scan_down<K::LT>(d1, r, tl);
            f2 *carry = reinterpret_cast<f2 *>(rs + ch * a.S + 2 * p);
            const f2 behind = *carry;
            const f2 out = fma2(d1, behind, r);
            d1 = __shfl_down_sync(0xffffffffu, d1, 1, K::LT);
            r = __shfl_down_sync(0xffffffffu, r, 1, K::LT);
            r = tl < K::LT - 1 ? fma2(d1, behind, r) : behind;
            if (tl == 0) *carry = out;
            f2 da = das[p * K::THREADS + threadIdx.x];
#pragma unroll
            for (int q = K::TL / 2 - 1; q >= 0; --q) {
                f2 b2[2], c2[2];
                pair_load<K>(bs, p, tl, q, b2[0], b2[1]);
                pair_load<K>(cs, p, tl, q, c2[0], c2[1]);
#pragma unroll
                for (int e = 1; e >= 0; --e) {
                    const int i = 2 * q + e;
                    const f2 dp2 = pack2(dp[i], dp[i]);
                    const f2 gr = fma2(c2[e], dp2, r);
                    red[ch * K::TT + i * K::LT + tl] =
                        make_ulonglong2(mul2(gr, pack2(dt[i] * u[i], dt[i] * u[i])), mul2(h2[i], dp2));
                    x2[i] = fma2(gr, b2[e], x2[i]);
                    r = mul2(a2[i], gr);
                    const f2 w = mul2(r, i ? h2[i ? i - 1 : 0] : hin);
                    q2[i] = fma2(w, r2, q2[i]);
                    da = fma2(w, pack2(dt[i], dt[i]), da);
                }
            }
            das[p * K::THREADS + threadIdx.x] = da;
            __syncthreads();
            // the block's channels: a thread per token and {db, dc}
            for (int s = threadIdx.x; s < 2 * K::TT; s += K::THREADS) {
                const int j = s >> 1, t = (j % K::LT) * K::TL + j / K::LT;
                const f2 *col = reinterpret_cast<const f2 *>(red) + s;
                f2 v = 0ull;
#pragma unroll
                for (int k = 0; k < K::CH; ++k) v = add2(v, col[k * 2 * K::TT]);
                if (t0 + t < len)
                    *reinterpret_cast<f2 *>(g.bc_part + ((((long long)blockIdx.x * a.B + b) * a.N + t0 + t) * 2 + (s & 1)) * a.S +
                                            2 * p) = v;
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < K::TL; ++i) {
            const float2 xv = unpack2(x2[i]), qv = unpack2(q2[i]), yv = unpack2(y2[i]);
            const float x = xv.x + xv.y, pre = fmaf(skip, u[i], yv.x + yv.y);
            // sigmoid(raw) = 1 - exp(-softplus(raw))
            const float ddt = -expm1f(-dt[i]) * fmaf(x, u[i], (qv.x + qv.y) * 0.69314718055994531f);
            dbias += ddt;
            u[i] = fmaf(x, dt[i], skip * dp[i]);
            dt[i] = ddt;
            dp[i] = pre;
        }
        lane_store<K>(us + K::channel(ch), tl, u);
        lane_store<K>(dts + K::channel(ch), tl, dt);
        if (Z) lane_store<K>(dps + K::channel(ch), tl, dp);
        __syncthreads();
        for (int i = threadIdx.x; i < K::TT * (K::CH / 8); i += K::THREADS) {
            const int piece = i % (K::CH / 8), t = i / (K::CH / 8), n = min(8, nch - piece * 8);
            if (t0 + t >= len || n <= 0) continue;
            const int c = c0 + piece * 8, at = K::pos(t);
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = us[K::channel(piece * 8 + k) + at];
            store8<VEC>(g.du.at(b, t0 + t) + c, n, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = dts[K::channel(piece * 8 + k) + at];
            store8<VEC>(g.ddt.at(b, t0 + t) + c, n, v);
            if (Z) {
                float z[8], y[8];
                load8<VEC>(a.z.at(b, t0 + t) + c, n, z);
                load8<VEC>(g.dy.at(b, t0 + t) + c, n, y);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = y[k] * dps[K::channel(piece * 8 + k) + at] * dsilu(z[k], sigmoid(z[k]));
                store8<VEC>(g.dz.at(b, t0 + t) + c, n, v);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nch * a.S; i += K::THREADS) {
        const int k = i / a.S, n = i % a.S;
        // the channel's time lanes, in order
        const float *lanes = reinterpret_cast<const float *>(das + (n / 2) * K::THREADS + (k / K::CPW) * 32 + (k % K::CPW) * K::LT) + (n & 1);
        float v = 0.f;
#pragma unroll
        for (int l = 0; l < K::LT; ++l) v += lanes[2 * l];
        const long long at = ((long long)b * a.D + c0) * a.S + i;
        g.a_part[at] = v * rate[i] * 0.69314718055994531f;
        if (g.dstate_in) g.dstate_in[at] = rs[i];
    }
#pragma unroll
    for (int off = K::LT / 2; off; off >>= 1) {
        dskip += __shfl_xor_sync(0xffffffffu, dskip, off);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, off);
    }
    if (tl == 0 && ch < nch) {
        g.d_part[(long long)b * a.D + c0 + ch] = dskip;
        g.d_part[((long long)a.B + b) * a.D + c0 + ch] = dbias;
    }
}

// db and dc: the groups' blocks of channels in order; four states a thread.
template <typename T> __global__ void __launch_bounds__(256) scan_bc_kernel(const GradArgs<T> g)
{
    const ScanArgs<T> &a = g.f;
    const int per = 2 * a.S / 4;                              // threads per token and group
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int q = (int)(i % per);
    const long long tg = i / per;
    const int group = (int)(tg % a.G);
    const long long t = tg / a.G;
    const int b = blockIdx.y;
    if (t >= row_length(a.lengths, b, a.N)) return;
    const float4 *p = reinterpret_cast<const float4 *>(g.bc_part) + ((((long long)group * a.tiles * a.B + b) * a.N + t) * per + q);
    const long long step = (long long)a.B * a.N * per;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < a.tiles; ++k) {
        const float4 v = p[k * step];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    const int n = 4 * q < a.S ? 4 * q : 4 * q - a.S;
    T *out = (4 * q < a.S ? g.db : g.dc).at(b, (int)t) + group * a.S + n;
    out[0] = from_f32<T>(s.x); out[1] = from_f32<T>(s.y); out[2] = from_f32<T>(s.z); out[3] = from_f32<T>(s.w);
}

typedef Tile<16, 8, 8> BTile;

struct Layout {
    size_t bc, a, d, total;
};
Layout layout(const gma_scan_t &s)
{
    const long long tiles = (s.D / s.G + BTile::CH - 1) / BTile::CH;
    Layout l;
    l.bc = 0;
    l.a = align_up((size_t)s.G * tiles * s.B * s.N * 2 * s.S * sizeof(float), 256);
    l.d = l.a + align_up((size_t)s.B * s.D * s.S * sizeof(float), 256);
    l.total = l.d + align_up((size_t)2 * s.B * s.D * sizeof(float), 256);
    return l;
}

template <typename T, bool VEC, bool Z> gma_status_t launch_backward(const GradArgs<T> &g, cudaStream_t st)
{
    auto kern = scan_backward_kernel<T, BTile, VEC, Z>;
    const size_t smem = BackwardSmem<BTile>::bytes(g.f.S);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return GMA_ERR_CUDA;
    GMA_LAUNCH(KID_SCAN_BWD, st, kern<<<dim3(g.f.tiles * g.f.G, g.f.B), BTile::THREADS, smem, st>>>(g));
    return GMA_OK;
}

template <typename T> gma_status_t backward_of(const gma_scan_grad_t &s, char *ws, cudaStream_t st)
{
    const gma_scan_t &f = s.fwd;
    const Layout l = layout(f);
    GradArgs<T> g;
    g.f = scan_args<T>(f);
    g.f.tiles = (f.D / f.G + BTile::CH - 1) / BTile::CH;
    g.dy = rows_of<const T>(s.dy);
    g.dstate_out = s.dstate_out;
    g.du = rows_of<T>(s.du); g.ddt = rows_of<T>(s.ddt); g.dz = rows_of<T>(s.dz);
    g.db = rows_of<T>(s.db); g.dc = rows_of<T>(s.dc);
    g.da_log = s.da_log; g.dd_skip = s.dd_skip; g.ddt_bias = s.ddt_bias; g.dstate_in = s.dstate_in;
    g.bc_part = (float *)(ws + l.bc); g.a_part = (float *)(ws + l.a); g.d_part = (float *)(ws + l.d);
    const int dt = f.dtype;
    const bool vec = scan_vec(f) && rows_vec(s.dy, dt) && rows_vec(s.du, dt) && rows_vec(s.ddt, dt) &&
                     (!f.z.ptr || rows_vec(s.dz, dt));
    gma_status_t r;
    if (f.z.ptr) r = vec ? launch_backward<T, true, true>(g, st) : launch_backward<T, false, true>(g, st);
    else r = vec ? launch_backward<T, true, false>(g, st) : launch_backward<T, false, false>(g, st);
    if (r != GMA_OK) return r;
    const long long threads = (long long)f.N * f.G * (2 * f.S / 4);
    GMA_LAUNCH(KID_SCAN_BC, st,
               scan_bc_kernel<T><<<dim3((unsigned)((threads + 255) / 256), f.B), 256, 0, st>>>(g));
    const SumOut da = {s.da_log, 1};
    if ((r = sum_rows(g.a_part, f.B, 1, 1, f.D * f.S, f.D * f.S, &da, st)) != GMA_OK) return r;
    if (f.d_skip) {
        const SumOut o = {s.dd_skip, 1};
        if ((r = sum_rows(g.d_part, f.B, 1, 1, f.D, f.D, &o, st)) != GMA_OK) return r;
    }
    if (f.dt_bias) {
        const SumOut o = {s.ddt_bias, 1};
        if ((r = sum_rows(g.d_part + (size_t)f.B * f.D, f.B, 1, 1, f.D, f.D, &o, st)) != GMA_OK) return r;
    }
    return GMA_OK;
}

}  // namespace
}  // namespace blk
}  // namespace gma

using namespace gma;
using namespace gma::blk;

extern "C" {

size_t gma_scan_backward_workspace_size(const gma_scan_grad_t *g)
{
    if (!g || scan_check(&g->fwd, false) != GMA_OK) return 0;
    return layout(g->fwd).total;
}

gma_status_t gma_scan_backward(const gma_scan_grad_t *g, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    if (!g) return GMA_ERR_INVALID_ARG;
    const gma_scan_t &f = g->fwd;
    gma_status_t r = scan_check(&f, false);
    if (r != GMA_OK) return r;
    const long long B = f.B, N = f.N, D = f.D, GS = (long long)f.G * f.S;
    if (!f.checkpoints || !rows_ok(g->dy, f.dtype, B, N, D, false)) return GMA_ERR_INVALID_ARG;
    if (!rows_ok(g->du, f.dtype, B, N, D, true) || !rows_ok(g->ddt, f.dtype, B, N, D, true) ||
        (f.z.ptr && !rows_ok(g->dz, f.dtype, B, N, D, true)) || !rows_ok(g->db, f.dtype, B, N, GS, true) ||
        !rows_ok(g->dc, f.dtype, B, N, GS, true))
        return GMA_ERR_INVALID_ARG;
    if (!ptr_ok(g->da_log, 4) || (f.d_skip && !ptr_ok(g->dd_skip, 4)) || (f.dt_bias && !ptr_ok(g->ddt_bias, 4)) ||
        !opt_ok(g->dstate_out, 4) || !opt_ok(g->dstate_in, 4))
        return GMA_ERR_INVALID_ARG;
    if (D * f.S > 0x7fffffffll || N * f.G * f.S / 2 > 0x7fffffffll * 128) return GMA_ERR_UNSUPPORTED_SHAPE;
    if (!ws_ok(ws, ws_bytes, layout(f).total)) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    return f.dtype == GMA_BF16 ? backward_of<__nv_bfloat16>(*g, (char *)ws, st) : backward_of<float>(*g, (char *)ws, st);
}

}  // extern "C"
