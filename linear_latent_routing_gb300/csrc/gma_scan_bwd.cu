// gma_scan_bwd.cu -- the selective scan's backward pass (gma_scan_backward).
//
// With p_t the output before the gate, dp_t = dy_t silu(z_t) and g_t[n] = dL / dh_t[n],
//   g_t = c_t dp_t + r_t,   r_{t-1} = exp(delta_t A) g_t   (r behind the last token: dstate_out),
//   dc_t = sum_d dp_t h_t,   db_t = sum_d g_t delta_t u_t,   x_t = sum_n b_t g_t,   q_t[n] = r_{t-1} h_{t-1},
//   du = delta x + D dp,   ddelta = u x + sum_n A q,   dA = sum_t delta q,   ddt = ddelta sigmoid(dt + dt_bias).
// A block walks over its channels' tiles from the last to the first: each tile's states are computed
// again from the checkpoint in front of it, then the adjoint recurrence runs from the tile's end.  A lane
// owns TL neighbouring tokens of two channels (the two halves of its packed registers) and takes one state
// at a time: its tokens' states stay in registers between the two recurrences, and both are
// sequential over its own tokens with a scan of (decay, state) over the LT time lanes in between.
// db and dc are sums over channels: a block adds up its own in shared memory, state by state, and leaves
// partial sums that a last kernel adds in a fixed order.
#include "scan_tile.cuh"

namespace gma {
namespace blk {
namespace {

constexpr int LT = 16, TL = 8, TT = LT * TL;
static_assert(TT % CKPT == 0, "a tile starts at a checkpoint");
constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int SLOTS = WARPS * (32 / LT);        // lane groups of a block, two channels each
constexpr int CH = 2 * SLOTS;
constexpr int NB = 16;                          // states whose b and c are staged at a time

// A channel pair's tokens: token t = tl * TL + i at ((i / 2) * LT + tl) * 2 + i % 2, as pairs.
__device__ __forceinline__ int pos(int t) { return ((t % TL / 2) * LT + t / TL) * 2 + t % 2; }
constexpr int PITCH = TT + 2;                   // f2 between two channel pairs
constexpr int PAIRS = SLOTS * PITCH;

template <typename T> struct GradArgs {
    ScanArgs<T> f;
    Rows<const T> dy;
    const float *dstate_out;
    Rows<T> du, ddt, dz, db, dc;
    float *da_log, *dd_skip, *ddt_bias, *dstate_in;
    float2 *bc_part;     // [G * tiles][B][time tiles][S][TT]: db, dc in the order of pos()
    float *a_part;       // [B][D][S]
    float *d_part;       // [2][B][D]: d_skip, dt_bias
};

// Sums of delta over 1, 2, 4, ... lanes ending (up) or starting (down) at a lane: exp2(rate * sum) is the
// decay over them, so the scans over lanes exchange states alone.  FAR marks a window that leaves the
// tile: its decay is 0 (rates are kept at -1e-30 or below, a decay of exactly 1 for any real delta).
constexpr float FAR = 3e38f;
constexpr int STEPS = 4;
static_assert(LT == 1 << STEPS, "");
template <bool UP> __device__ __forceinline__ void windows(f2 total, int tl, f2 (&w)[STEPS], f2 &outside)
{
    f2 sum = total;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const bool in = UP ? tl >= 1 << k : tl + (1 << k) < LT;
        w[k] = in ? sum : pack2(FAR, FAR);
        const f2 far = UP ? __shfl_up_sync(0xffffffffu, sum, 1 << k, LT) : __shfl_down_sync(0xffffffffu, sum, 1 << k, LT);
        if (in) sum = add2(sum, far);
    }
    // everything before (or behind) the lane
    outside = UP ? __shfl_up_sync(0xffffffffu, sum, 1, LT) : __shfl_down_sync(0xffffffffu, sum, 1, LT);
    if (UP ? tl == 0 : tl == LT - 1) outside = 0ull;
}
// Inclusive scan of a lane's state, then the state that enters it, `edge` being what enters the tile.
template <bool UP> __device__ __forceinline__ f2 enter(f2 s, const f2 (&w)[STEPS], f2 outside, f2 inner, f2 r2, f2 edge)
{
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const f2 far = UP ? __shfl_up_sync(0xffffffffu, s, 1 << k, LT) : __shfl_down_sync(0xffffffffu, s, 1 << k, LT);
        s = fma2(ex2_2(mul2(w[k], r2)), far, s);
    }
    s = UP ? __shfl_up_sync(0xffffffffu, s, 1, LT) : __shfl_down_sync(0xffffffffu, s, 1, LT);
    return fma2(ex2_2(mul2(outside, r2)), edge, mul2(s, inner));
}

struct Smem {
    f2 us[PAIRS], dts[PAIRS], dps[PAIRS];
    f2 red[2][SLOTS][TT];                       // (db, dc) of a state, by lane group
    f2 bs[NB][TT], cs[NB][TT];                  // (b, b), (c, c)
    // then: sums of delta q by lane [S][THREADS], rate, state in front, adjoint behind [S][SLOTS], as pairs
};
size_t smem_bytes(int S) { return sizeof(Smem) + (size_t)S * THREADS * sizeof(f2) + (size_t)3 * S * SLOTS * sizeof(f2); }

template <typename T, bool VEC, bool Z>
__global__ void __launch_bounds__(THREADS) scan_backward_kernel(const GradArgs<T> g)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    const ScanArgs<T> &a = g.f;
    const int S = a.S, nb = S < NB ? S : NB;
    f2 *das = reinterpret_cast<f2 *>(raw + sizeof(Smem));
    f2 *rate = das + S * THREADS, *hs = rate + S * SLOTS, *rs = hs + S * SLOTS;

    const int b = blockIdx.y, group = blockIdx.x / a.tiles, Dg = a.D / a.G;
    const int in_group = (blockIdx.x - group * a.tiles) * CH;
    const int c0 = group * Dg + in_group, nch = min(CH, Dg - in_group);
    const int len = row_length(a.lengths, b, a.N);
    const int lane = threadIdx.x & 31, tl = lane % LT, slot = (threadIdx.x >> 5) * (32 / LT) + lane / LT;
    const int nck = (a.N + CKPT - 1) / CKPT, ntt = (a.N + TT - 1) / TT;

    for (int i = threadIdx.x; i < S * SLOTS; i += THREADS) {
        const int n = i / SLOTS, s = i % SLOTS;
        float v[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * s + e < nch) {
                const long long at = (long long)(c0 + 2 * s + e) * S + n;
                v[e] = fminf(-expf(a.a_log[at]) * LOG2E, -1e-30f);   // see FAR
                if (g.dstate_out) w[e] = g.dstate_out[(long long)b * a.D * S + at];
            }
        rate[i] = pack2(v[0], v[1]);
        rs[i] = pack2(w[0], w[1]);
    }
    for (int n = 0; n < S; ++n) das[n * THREADS + threadIdx.x] = 0ull;
    const int mine = nch - 2 * slot;                 // channels of this lane
    const f2 skip = pack2(a.d_skip && mine > 0 ? a.d_skip[c0 + 2 * slot] : 0.f,
                          a.d_skip && mine > 1 ? a.d_skip[c0 + 2 * slot + 1] : 0.f);
    f2 dskip = 0ull, dbias = 0ull;
    // 0 for the lane at the tile's edge, which has no neighbour there
    const f2 inner_up = tl ? pack2(1.f, 1.f) : 0ull, inner_down = tl < LT - 1 ? pack2(1.f, 1.f) : 0ull;

    // A thread stages and stores the same eight channels of UNITS tokens of every tile.
    constexpr int UNITS = TT * (CH / 8) / THREADS, STEP = TT / UNITS;
    const int piece = threadIdx.x % (CH / 8), token = threadIdx.x / (CH / 8);
    const int n8 = min(8, nch - piece * 8), cp = c0 + piece * 8;
    float bias[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) bias[k] = a.dt_bias && k < n8 ? a.dt_bias[cp + k] : 0.f;

    for (int t0 = (len - 1) / TT * TT; t0 >= 0 && len > 0; t0 -= TT) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const int t = token + j * STEP, at = pos(t);
            const bool on = t0 + t < len && n8 > 0;
            float u[8], d[8], y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = d[k] = y[k] = 0.f;
            if (on) {
                load8<VEC>(a.u.at(b, t0 + t) + cp, n8, u);
                load8<VEC>(a.dt.at(b, t0 + t) + cp, n8, d);
                load8<VEC>(g.dy.at(b, t0 + t) + cp, n8, y);
                if (Z) {
                    float z[8];
                    load8<VEC>(a.z.at(b, t0 + t) + cp, n8, z);
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] *= silu(z[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const float2 s = unpack2(softplus2(add2(pack2(d[k], d[k + 1]), pack2(bias[k], bias[k + 1]))));
                const int to = (piece * 4 + k / 2) * PITCH + at;
                sm.us[to] = pack2(u[k], u[k + 1]);
                sm.dts[to] = pack2(on && k < n8 ? s.x : 0.f, on && k + 1 < n8 ? s.y : 0.f);
                sm.dps[to] = pack2(y[k], y[k + 1]);
            }
        }
        for (int i = threadIdx.x; i < S * SLOTS; i += THREADS) {
            const int n = i / SLOTS, s = i % SLOTS;
            const float *ck = a.ckpt + (((long long)b * nck + t0 / CKPT) * a.D + c0 + 2 * s) * S + n;
            hs[i] = pack2(2 * s < nch ? ck[0] : 0.f, 2 * s + 1 < nch ? ck[S] : 0.f);
        }
        __syncthreads();

        f2 dt[TL], xu[TL], dp[TL], x2[TL], q2[TL], y2[TL], total = 0ull;
#pragma unroll
        for (int q = 0; q < TL / 2; ++q) {
            const int at = slot * PITCH + (q * LT + tl) * 2;
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sm.dts + at);
            const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(sm.us + at);
            const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(sm.dps + at);
            dt[2 * q] = v.x; dt[2 * q + 1] = v.y;
            xu[2 * q] = mul2(v.x, u.x); xu[2 * q + 1] = mul2(v.y, u.y);
            dp[2 * q] = p.x; dp[2 * q + 1] = p.y;
            dskip = fma2(p.x, u.x, dskip);
            dskip = fma2(p.y, u.y, dskip);
            total = add2(total, add2(v.x, v.y));
        }
#pragma unroll
        for (int i = 0; i < TL; ++i) x2[i] = q2[i] = y2[i] = 0ull;
        f2 up[STEPS], down[STEPS], before_sum, behind_sum;
        windows<true>(total, tl, up, before_sum);
        windows<false>(total, tl, down, behind_sum);
        float2 *part = g.bc_part + (((long long)blockIdx.x * a.B + b) * ntt + t0 / TT) * S * TT + threadIdx.x;

        for (int n0 = 0; n0 < S; n0 += nb) {
            if (n0) __syncthreads();
            for (int i = threadIdx.x; i < TT * (nb / 8); i += THREADS) {
                const int t = i % TT, k8 = i / TT * 8, at = pos(t);
                float v[8], w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = w[k] = 0.f;
                if (t0 + t < len) {
                    load8<VEC>(a.b.at(b, t0 + t) + group * S + n0 + k8, 8, v);
                    load8<VEC>(a.c.at(b, t0 + t) + group * S + n0 + k8, 8, w);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    sm.bs[k8 + k][at] = pack2(v[k], v[k]);
                    sm.cs[k8 + k][at] = pack2(w[k], w[k]);
                }
            }
            __syncthreads();
            for (int m = 0; m < nb; ++m) {
                const int n = n0 + m;
                const f2 r2 = rate[n * SLOTS + slot], before = hs[n * SLOTS + slot];
                const f2 *bl = sm.bs[m] + tl * 2, *cl = sm.cs[m] + tl * 2;
                f2 a2[TL], h2[TL], h = 0ull, r = 0ull;
#pragma unroll
                for (int q = 0; q < TL / 2; ++q) {
                    const ulonglong2 bv = *reinterpret_cast<const ulonglong2 *>(bl + q * LT * 2);
                    a2[2 * q] = ex2_2(mul2(dt[2 * q], r2));
                    a2[2 * q + 1] = ex2_2(mul2(dt[2 * q + 1], r2));
                    h2[2 * q] = mul2(bv.x, xu[2 * q]);
                    h2[2 * q + 1] = mul2(bv.y, xu[2 * q + 1]);
                    h = fma2(a2[2 * q], h, h2[2 * q]);
                    h = fma2(a2[2 * q + 1], h, h2[2 * q + 1]);
                }
                const f2 hin = enter<true>(h, up, before_sum, inner_up, r2, before);
                h = hin;
#pragma unroll
                for (int i = 0; i < TL; ++i) {
                    h = fma2(a2[i], h, h2[i]);
                    h2[i] = h;
                }
#pragma unroll
                for (int q = TL / 2 - 1; q >= 0; --q) {
                    const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(cl + q * LT * 2);
                    if (Z) {
                        y2[2 * q + 1] = fma2(cv.y, h2[2 * q + 1], y2[2 * q + 1]);
                        y2[2 * q] = fma2(cv.x, h2[2 * q], y2[2 * q]);
                    }
                    r = mul2(a2[2 * q + 1], fma2(cv.y, dp[2 * q + 1], r));
                    r = mul2(a2[2 * q], fma2(cv.x, dp[2 * q], r));
                }
                r = enter<false>(r, down, behind_sum, inner_down, r2, rs[n * SLOTS + slot]);
                f2 da = das[n * THREADS + threadIdx.x];
                f2 *red = sm.red[n & 1][slot] + tl * 2;
#pragma unroll
                for (int q = TL / 2 - 1; q >= 0; --q) {
                    const ulonglong2 bv = *reinterpret_cast<const ulonglong2 *>(bl + q * LT * 2);
                    const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(cl + q * LT * 2);
                    f2 sum[2];
#pragma unroll
                    for (int e = 1; e >= 0; --e) {
                        const int i = 2 * q + e;
                        const f2 gr = fma2(e ? cv.y : cv.x, dp[i], r);
                        const float2 db = unpack2(mul2(gr, xu[i])), dc = unpack2(mul2(h2[i], dp[i]));
                        sum[e] = pack2(db.x + db.y, dc.x + dc.y);
                        x2[i] = fma2(gr, e ? bv.y : bv.x, x2[i]);
                        r = mul2(a2[i], gr);
                        const f2 w = mul2(r, i ? h2[i ? i - 1 : 0] : hin);
                        q2[i] = fma2(w, r2, q2[i]);
                        da = fma2(w, dt[i], da);
                    }
                    *reinterpret_cast<ulonglong2 *>(red + q * LT * 2) = make_ulonglong2(sum[0], sum[1]);
                }
                das[n * THREADS + threadIdx.x] = da;
                if (tl == 0) rs[n * SLOTS + slot] = r;
                // The block's channels, a token a thread, in order.  The other half of `red` takes the next
                // state meanwhile, so one barrier a state is enough.
                __syncthreads();
                f2 v = 0ull;
#pragma unroll
                for (int k = 0; k < SLOTS; ++k) v = add2(v, sm.red[n & 1][k][threadIdx.x]);
                part[n * TT] = unpack2(v);
            }
        }
#pragma unroll
        for (int q = 0; q < TL / 2; ++q) {
            const int at = slot * PITCH + (q * LT + tl) * 2;
            const ulonglong2 uv = *reinterpret_cast<const ulonglong2 *>(sm.us + at);
            f2 du[2], dd[2], pre[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * q + e;
                const f2 u = e ? uv.y : uv.x;
                const float2 d = unpack2(dt[i]);
                // sigmoid(raw) = 1 - exp(-softplus(raw))
                const f2 slope = pack2(-expm1f(-d.x), -expm1f(-d.y));
                dd[e] = mul2(slope, fma2(x2[i], u, mul2(q2[i], pack2(0.69314718055994531f, 0.69314718055994531f))));
                dbias = add2(dbias, dd[e]);
                du[e] = fma2(x2[i], dt[i], mul2(skip, dp[i]));
                pre[e] = fma2(skip, u, y2[i]);
            }
            *reinterpret_cast<ulonglong2 *>(sm.us + at) = make_ulonglong2(du[0], du[1]);
            *reinterpret_cast<ulonglong2 *>(sm.dts + at) = make_ulonglong2(dd[0], dd[1]);
            if (Z) *reinterpret_cast<ulonglong2 *>(sm.dps + at) = make_ulonglong2(pre[0], pre[1]);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const int t = token + j * STEP, at = pos(t);
            if (t0 + t >= len || n8 <= 0) continue;
            float v[8];
            auto gather = [&](const f2 *tile) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 w = unpack2(tile[(piece * 4 + k) * PITCH + at]);
                    v[2 * k] = w.x;
                    v[2 * k + 1] = w.y;
                }
            };
            gather(sm.us);
            store8<VEC>(g.du.at(b, t0 + t) + cp, n8, v);
            gather(sm.dts);
            store8<VEC>(g.ddt.at(b, t0 + t) + cp, n8, v);
            if (Z) {
                float z[8], y[8];
                load8<VEC>(a.z.at(b, t0 + t) + cp, n8, z);
                load8<VEC>(g.dy.at(b, t0 + t) + cp, n8, y);
                gather(sm.dps);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= y[k] * dsilu(z[k], sigmoid(z[k]));
                store8<VEC>(g.dz.at(b, t0 + t) + cp, n8, v);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < S * SLOTS; i += THREADS) {
        const int n = i % S, s = i / S;
        // the pair's time lanes, in order
        const f2 *lanes = das + n * THREADS + s * LT;
        f2 v = 0ull;
#pragma unroll
        for (int l = 0; l < LT; ++l) v = add2(v, lanes[l]);
        const float2 da = unpack2(mul2(mul2(v, rate[n * SLOTS + s]), pack2(0.69314718055994531f, 0.69314718055994531f)));
        const float2 r = unpack2(rs[n * SLOTS + s]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * s + e < nch) {
                const long long at = ((long long)b * a.D + c0 + 2 * s + e) * S + n;
                g.a_part[at] = e ? da.y : da.x;
                if (g.dstate_in) g.dstate_in[at] = e ? r.y : r.x;
            }
    }
#pragma unroll
    for (int off = LT / 2; off; off >>= 1) {
        dskip = add2(dskip, __shfl_xor_sync(0xffffffffu, dskip, off));
        dbias = add2(dbias, __shfl_xor_sync(0xffffffffu, dbias, off));
    }
    if (tl == 0) {
        const float2 s = unpack2(dskip), t = unpack2(dbias);
        float *p = g.d_part + (long long)b * a.D + c0 + 2 * slot;
        if (mine > 0) p[0] = s.x, p[(long long)a.B * a.D] = t.x;
        if (mine > 1) p[1] = s.y, p[(long long)a.B * a.D + 1] = t.y;
    }
}

// db and dc: the groups' blocks of channels in order.  A block takes eight states of a time tile, a
// thread a token and four of them.
template <typename T> __global__ void __launch_bounds__(2 * TT) scan_bc_kernel(const GradArgs<T> g)
{
    const ScanArgs<T> &a = g.f;
    const int b = blockIdx.y, tile = blockIdx.x, group = blockIdx.z / (a.S / 8);
    const int n0 = blockIdx.z % (a.S / 8) * 8 + threadIdx.x / TT * 4, i = threadIdx.x % TT;
    const int len = row_length(a.lengths, b, a.N), ntt = (a.N + TT - 1) / TT;
    const int t = tile * TT + i;
    if (t >= len) return;
    const float2 *p = g.bc_part + ((((long long)group * a.tiles * a.B + b) * ntt + tile) * a.S + n0) * TT + pos(i);
    const long long step = (long long)a.B * ntt * a.S * TT;
    float2 s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < a.tiles; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 v = p[c * step + k * TT];
            s[k].x += v.x;
            s[k].y += v.y;
        }
    T *db = g.db.at(b, t) + group * a.S + n0, *dc = g.dc.at(b, t) + group * a.S + n0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        db[k] = from_f32<T>(s[k].x);
        dc[k] = from_f32<T>(s[k].y);
    }
}

struct Layout {
    size_t bc, a, d, total;
};
Layout layout(const gma_scan_t &s)
{
    const size_t tiles = (s.D / s.G + CH - 1) / CH, ntt = (s.N + TT - 1) / TT;
    Layout l;
    l.bc = 0;
    l.a = align_up(s.G * tiles * s.B * ntt * TT * 2 * s.S * sizeof(float), 256);
    l.d = l.a + align_up((size_t)s.B * s.D * s.S * sizeof(float), 256);
    l.total = l.d + align_up((size_t)2 * s.B * s.D * sizeof(float), 256);
    return l;
}

template <typename T, bool VEC, bool Z> gma_status_t launch_backward(const GradArgs<T> &g, cudaStream_t st)
{
    auto kern = scan_backward_kernel<T, VEC, Z>;
    const size_t smem = smem_bytes(g.f.S);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return GMA_ERR_CUDA;
    GMA_LAUNCH(KID_SCAN_BWD, st, kern<<<dim3(g.f.tiles * g.f.G, g.f.B), THREADS, smem, st>>>(g));
    return GMA_OK;
}

template <typename T> gma_status_t backward_of(const gma_scan_grad_t &s, char *ws, cudaStream_t st)
{
    const gma_scan_t &f = s.fwd;
    const Layout l = layout(f);
    GradArgs<T> g;
    g.f = scan_args<T>(f);
    g.f.tiles = (f.D / f.G + CH - 1) / CH;
    g.dy = rows_of<const T>(s.dy);
    g.dstate_out = s.dstate_out;
    g.du = rows_of<T>(s.du); g.ddt = rows_of<T>(s.ddt); g.dz = rows_of<T>(s.dz);
    g.db = rows_of<T>(s.db); g.dc = rows_of<T>(s.dc);
    g.da_log = s.da_log; g.dd_skip = s.dd_skip; g.ddt_bias = s.ddt_bias; g.dstate_in = s.dstate_in;
    g.bc_part = (float2 *)(ws + l.bc); g.a_part = (float *)(ws + l.a); g.d_part = (float *)(ws + l.d);
    const int dt = f.dtype;
    const bool vec = scan_vec(f) && rows_vec(s.dy, dt) && rows_vec(s.du, dt) && rows_vec(s.ddt, dt) &&
                     (!f.z.ptr || rows_vec(s.dz, dt));
    gma_status_t r;
    if (f.z.ptr) r = vec ? launch_backward<T, true, true>(g, st) : launch_backward<T, false, true>(g, st);
    else r = vec ? launch_backward<T, true, false>(g, st) : launch_backward<T, false, false>(g, st);
    if (r != GMA_OK) return r;
    GMA_LAUNCH(KID_SCAN_BC, st,
               scan_bc_kernel<T><<<dim3((f.N + TT - 1) / TT, f.B, f.G * (f.S / 8)), 2 * TT, 0, st>>>(g));
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
    if (D * f.S > 0x7fffffffll || GS / 8 > 65535) return GMA_ERR_UNSUPPORTED_SHAPE;
    if (!ws_ok(ws, ws_bytes, layout(f).total)) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    return f.dtype == GMA_BF16 ? backward_of<__nv_bfloat16>(*g, (char *)ws, st) : backward_of<float>(*g, (char *)ws, st);
}

}  // extern "C"
