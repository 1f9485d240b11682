// gma_scan_bwd.cu -- the selective scan's backward pass (gma_scan_backward).
//
// With p_t the output before the gate, dp_t = dy_t silu(z_t) and g_t[n] = dL / dh_t[n],
//   g_t = c_t dp_t + r_t,   r_{t-1} = exp(delta_t A) g_t   (r behind the last token: dstate_out),
//   dc_t = sum_d dp_t h_t,   db_t = sum_d g_t delta_t u_t,   x_t = sum_n b_t g_t,   q_t[n] = r_{t-1} h_{t-1},
//   du = delta x + D dp,   ddelta = u x + sum_n A q,   dA = sum_t delta q,   ddt = ddelta sigmoid(dt + dt_bias).
// In four launches:
//   1, 2. the adjoint r behind every chunk of 64 (or 16) tokens (each chunk's from zero, then joined);
//   3. every chunk: a warp walks over its channels' tokens forward from the checkpoint, keeping the state in
//      front of every eighth token in shared memory; then, eight tokens at a time from the last, it
//      computes their states again into registers and runs the adjoint back over them;
//   4. sums of the blocks' partial db and dc, and of the chunks' partial parameter gradients, in one launch.
// A lane holds eight states of a channel (S / 8 lanes a channel) and their eight tokens' history in 64
// registers, so that 12 warps fit an SM; x, q and p are added over a channel's lanes by shuffles.  db and dc are
// sums over channels: a warp passes its lanes' products through shared memory (lanes write rows, read
// columns), a block adds its warps, and step 4 the blocks, always in the same order.  The blocks' parts go through
// memory: S^2 / 128 bytes a (token, channel), 2 at 16 states and 32 at 64.
// Measured: 4 x 2048 x 1024 channels x 16 states, bf16 with a gate: 41 us, 10 us, 184 us and 10 us.  Step 3
// takes 422 instructions an element (three exponentials a state) at 50 % of the issue slots with 11 warps an SM; the
// shared-memory pipe binds it (76 % busy: 78 wavefronts a token of a warp, 32 of them the column sums').  Two channels
// of four states a lane halve those, but stage every value twice and spill more (this form spills 24 bytes a thread, with other
// types, states and rows 12 to 316): 224 us.  Tokens over lanes, as in
// gma_scan.cu, took 303 us.
#include "scan_args.cuh"

namespace gma {
namespace blk {
namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS, SUB = 8;
constexpr int NF = 4;                        // pairs of states of a lane
constexpr float LN2 = 0.69314718055994531f;

template <int S> struct Lane {
    static constexpr int SPLIT = S / 8, CHW = 32 / SPLIT, CH = WARPS * CHW;   // lanes of a channel; channels
};

template <typename T> struct GradArgs {
    ScanArgs<T> f;
    int chunks;
    Rows<const T> dy;
    Rows<T> du, ddt, dz, db, dc;
    float *state;        // [B][chunks][D][S]: the adjoint behind each chunk, then the chunk's sums for da_log
    float *skip, *bias;  // [B][chunks][D]: the chunk's sums for d_skip and dt_bias
    float *bc_part;      // [G * tiles][B][N][2 S]: per eight states, db then dc
};

// Four neighbouring channels, as they lie in memory until they are used (VEC), or the first n of them.
template <typename T, bool VEC> struct Raw4;
template <> struct Raw4<__nv_bfloat16, true> {
    uint2 q;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int) { q = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void get(float (&v)[4]) const
    {
        v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
        v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
    }
};
template <> struct Raw4<float, true> {
    float4 q;
    __device__ __forceinline__ void load(const float *p, int) { q = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w; }
};
template <typename T> struct Raw4<T, false> {
    float q[4];
    __device__ __forceinline__ void load(const T *p, int n)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = i < n ? to_f32<T>(p[i]) : 0.f;
    }
    __device__ __forceinline__ void get(float (&v)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = q[i];
    }
};
template <bool VEC> __device__ __forceinline__ void store4(__nv_bfloat16 *p, int n, const float (&v)[4])
{
    if (VEC) {
        uint2 q;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&q);
        h[0] = __floats2bfloat162_rn(v[0], v[1]);
        h[1] = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(p) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
}
template <bool VEC> __device__ __forceinline__ void store4(float *p, int n, const float (&v)[4])
{
    if (VEC) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = v[i];
    }
}

// Rows of products: 20 floats apart, so that lanes write them 16 bytes at a time without bank conflicts, and
// every block of rows that a half warp reads together with the one before half a line further.
constexpr int RED_ROW = 20;
template <int S> __device__ __forceinline__ int red_row(int r) { return r * RED_ROW + r / (S == 16 ? 16 : 8) * 16; }

// One warp's share of shared memory; CK: the chunk's tokens.
template <int S, int CK> struct WarpSmem {
    static constexpr int CHW = Lane<S>::CHW;
    f2 start[CK / SUB][NF][32];                                // the states in front of every eighth token
    float red[2][32 * RED_ROW + 48];                         // two tokens' products by lane, 16 values a row
    // eight tokens: delta; u, then du; dp, then ddelta; p
    float dt[SUB][CHW], u[SUB][CHW], dp[SUB][CHW], p[SUB][CHW];
};
template <int S, int CK> struct Smem {
    WarpSmem<S, CK> w[WARPS];
    f2 sums[WARPS][SUB][S];                                  // db and dc of eight tokens by warp
    float b[CK][S], c[CK][S];
};

template <typename T, int S, int CK, bool VEC, bool Z>
__global__ void __launch_bounds__(THREADS, 3) scan_backward_kernel(const GradArgs<T> g)
{
    constexpr int SPLIT = Lane<S>::SPLIT, CHW = Lane<S>::CHW, CH = Lane<S>::CH;
    extern __shared__ __align__(16) unsigned char raw[];
    typedef Smem<S, CK> Sm;
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    let_next();
    const ScanArgs<T> &a = g.f;
    const int b = blockIdx.z, k = blockIdx.y, t0 = k * CK;
    const int len = row_length(a.lengths, b, a.N), count = min(CK, len - t0);
    const int group = blockIdx.x / a.tiles, Dg = a.D / a.G;
    if (a.zero) {
        const int i0 = (blockIdx.x - group * a.tiles) * CH, rows = min(CK, a.N - t0);
        const float none[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i = threadIdx.x; i < rows * (CH / 4); i += THREADS) {
            const int t = i / (CH / 4), ch = i0 + i % (CH / 4) * 4, n = min(4, Dg - ch);
            if (t < count || n <= 0) continue;
            store4<VEC>(g.du.at(b, t0 + t) + group * Dg + ch, n, none);
            store4<VEC>(g.ddt.at(b, t0 + t) + group * Dg + ch, n, none);
            if (Z) store4<VEC>(g.dz.at(b, t0 + t) + group * Dg + ch, n, none);
        }
    }
    if (count <= 0) {                                        // no tokens here; the join has cleared `state`
        wait_previous();
        const int i = (blockIdx.x - group * a.tiles) * CH + threadIdx.x;
        const long long to = ((long long)b * g.chunks + k) * a.D + group * Dg + i;
        static_assert(CH <= THREADS, "a thread a channel");
        if (threadIdx.x < CH && i < Dg) g.skip[to] = g.bias[to] = 0.f;
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane / CHW;
    const int warp_ch = (blockIdx.x - group * a.tiles) * CH + warp * CHW;        // in the group
    const bool on = warp_ch + lane % CHW < Dg;
    const int c = group * Dg + warp_ch + lane % CHW;
    WarpSmem<S, CK> &ws = sm.w[warp];

    // b and c of the chunk
    for (int i = threadIdx.x; i < count * (S / 8); i += THREADS) {
        const int t = i / (S / 8), piece = i % (S / 8) * 8;
        float v[8];
        load8<VEC>(a.b.at(b, t0 + t) + group * S + piece, 8, v);
        store8<true>(&sm.b[t][piece], 8, v);
        load8<VEC>(a.c.at(b, t0 + t) + group * S + piece, 8, v);
        store8<true>(&sm.c[t][piece], 8, v);
    }
    for (int i = count * S + threadIdx.x; i < (count + SUB - 1) / SUB * SUB * S; i += THREADS)
        (&sm.b[0][0])[i] = (&sm.c[0][0])[i] = 0.f;

    f2 rate[NF], h[NF], r[NF], da[NF];
    const long long at = (long long)c * S + part * 8, nck = g.chunks;
    float *state = g.state + ((long long)b * nck + k) * a.D * S + at;
    {
        wait_previous();
        const float *ck = a.ckpt + ((long long)b * nck + k) * a.D * S + at;
#pragma unroll
        for (int j = 0; j < NF / 2; ++j) {
            const float4 v = on ? reinterpret_cast<const float4 *>(a.a_log + at)[j] : make_float4(0.f, 0.f, 0.f, 0.f);
            rate[2 * j] = on ? pack2(decay_rate(v.x), decay_rate(v.y)) : 0ull;
            rate[2 * j + 1] = on ? pack2(decay_rate(v.z), decay_rate(v.w)) : 0ull;
            ulonglong2 w = make_ulonglong2(0ull, 0ull), z = w;
            if (on) {
                w = reinterpret_cast<const ulonglong2 *>(ck)[j];
                z = reinterpret_cast<const ulonglong2 *>(state)[j];
            }
            h[2 * j] = w.x; h[2 * j + 1] = w.y;
            r[2 * j] = z.x; r[2 * j + 1] = z.y;
            da[2 * j] = da[2 * j + 1] = 0ull;
        }
    }

    // Staging: a lane takes four channels of a token, UNITS times, the same channels every time.
    constexpr int QUADS = CHW / 4, UNITS = QUADS >= 4 ? QUADS / 4 : 1;
    const int quad = lane % QUADS, first = lane / QUADS;                         // channels, token
    constexpr int TSTEP = 32 / QUADS;
    const int n4 = max(0, min(4, Dg - warp_ch - 4 * quad)), c4 = group * Dg + warp_ch + 4 * quad;
    float bias[4], dskip[4], dbias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = a.dt_bias && i < n4 ? a.dt_bias[c4 + i] : 0.f;
        dskip[i] = dbias[i] = 0.f;
    }
    auto put4 = [](float *to, const float (&v)[4]) { *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]); };
    auto get4 = [](const float *from, float (&v)[4]) {
        const float4 q = *reinterpret_cast<const float4 *>(from);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    };
    // The rows of eight tokens, loaded ahead of their use; then delta and u (and dp), zeros behind the
    // last token and for channels that are not there.  The pointers are at the lane's first token of the
    // eight that are fetched next, and of the eight that are worked on.
    Raw4<T, VEC> ur[UNITS], dr[UNITS], yr[UNITS], zr[UNITS];
    const int t_first = t0 + first;
    const T *up = a.u.at(b, t_first) + c4, *dtp = a.dt.at(b, t_first) + c4, *dyp = g.dy.at(b, t_first) + c4;
    const T *zp = Z ? a.z.at(b, t_first) + c4 : nullptr;
    auto move = [&](int eights) {
        up += eights * SUB * a.u.st;
        dtp += eights * SUB * a.dt.st;
        dyp += eights * SUB * g.dy.st;
        if (Z) zp += eights * SUB * a.z.st;
    };
    auto fetch = [&](int s, bool grad) {
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const int i = first + j * TSTEP;
            if (i >= SUB || s < 0 || s * SUB + i >= count || n4 <= 0) continue;
            ur[j].load(up + j * TSTEP * a.u.st, n4);
            dr[j].load(dtp + j * TSTEP * a.dt.st, n4);
            if (grad) {
                yr[j].load(dyp + j * TSTEP * g.dy.st, n4);
                if (Z) zr[j].load(zp + j * TSTEP * a.z.st, n4);
            }
        }
    };
    auto stage = [&](int s, bool grad) {
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const int i = first + j * TSTEP, t = s * SUB + i;
            if (i >= SUB) continue;
            float u[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
            if (t < count && n4 > 0) {
                ur[j].get(u);
                dr[j].get(d);
                if (grad) {
                    yr[j].get(y);
                    if (Z) {
                        float z[4];
                        zr[j].get(z);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] *= silu(z[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 v = unpack2(softplus2(pack2(d[e] + bias[e], d[e + 1] + bias[e + 1])));
                    d[e] = e < n4 ? v.x : 0.f;
                    d[e + 1] = e + 1 < n4 ? v.y : 0.f;
                }
            }
            put4(&ws.u[i][4 * quad], u);
            put4(&ws.dt[i][4 * quad], d);
            if (grad) {
                put4(&ws.dp[i][4 * quad], y);
#pragma unroll
                for (int e = 0; e < 4; ++e) dskip[e] = fmaf(y[e], u[e], dskip[e]);
            }
        }
    };
    const int subs = (count + SUB - 1) / SUB, lc = lane % CHW;
    const float skip_c = a.d_skip && on ? a.d_skip[c] : 0.f;
    fetch(0, subs == 1);
    __syncthreads();

    // forward: the state in front of every eighth token
    for (int s = 0;; ++s) {
#pragma unroll
        for (int j = 0; j < NF; ++j) ws.start[s][j][lane] = h[j];
        if (s == subs - 1) break;
        __syncwarp();
        stage(s, false);
        move(1);
        fetch(s + 1, s + 2 == subs);
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < SUB; ++i) {
            const float d = ws.dt[i][lc], x = d * ws.u[i][lc];
            const f2 d2 = pack2(d, d), x2 = pack2(x, x);
            const ulonglong2 *bp = reinterpret_cast<const ulonglong2 *>(&sm.b[s * SUB + i][part * 8]);
            const ulonglong2 b0 = bp[0], b1 = bp[1];
            h[0] = fma2(ex2_2(mul2(d2, rate[0])), h[0], mul2(x2, b0.x));
            h[1] = fma2(ex2_2(mul2(d2, rate[1])), h[1], mul2(x2, b0.y));
            h[2] = fma2(ex2_2(mul2(d2, rate[2])), h[2], mul2(x2, b1.x));
            h[3] = fma2(ex2_2(mul2(d2, rate[3])), h[3], mul2(x2, b1.y));
        }
    }

    // back, eight tokens at a time
    const int t_last = t_first + (subs - 1) * SUB;
    T *dup = g.du.at(b, t_last) + c4, *ddtp = g.ddt.at(b, t_last) + c4, *dzp = Z ? g.dz.at(b, t_last) + c4 : nullptr;
    for (int s = subs - 1; s >= 0; --s) {
        __syncthreads();                          // `sums` has been read
        stage(s, true);
        Raw4<T, VEC> dk[UNITS], yk[UNITS], zk[UNITS];
#pragma unroll
        for (int j = 0; j < UNITS; ++j) dk[j] = dr[j], yk[j] = yr[j], zk[j] = zr[j];
        move(-1);
        fetch(s - 1, true);
        __syncwarp();
        f2 hist[SUB + 1][NF];
#pragma unroll
        for (int j = 0; j < NF; ++j) hist[0][j] = ws.start[s][j][lane];
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            const float d = ws.dt[i][lc], x = d * ws.u[i][lc];
            const f2 d2 = pack2(d, d), x2 = pack2(x, x);
            const ulonglong2 *bp = reinterpret_cast<const ulonglong2 *>(&sm.b[s * SUB + i][part * 8]);
            const ulonglong2 b0 = bp[0], b1 = bp[1];
            hist[i + 1][0] = fma2(ex2_2(mul2(d2, rate[0])), hist[i][0], mul2(x2, b0.x));
            hist[i + 1][1] = fma2(ex2_2(mul2(d2, rate[1])), hist[i][1], mul2(x2, b0.y));
            hist[i + 1][2] = fma2(ex2_2(mul2(d2, rate[2])), hist[i][2], mul2(x2, b1.x));
            hist[i + 1][3] = fma2(ex2_2(mul2(d2, rate[3])), hist[i][3], mul2(x2, b1.y));
        }
#pragma unroll
        for (int i2 = SUB - 2; i2 >= 0; i2 -= 2) {
            float du[2], ddelta[2], pre[2];
#pragma unroll
            for (int e = 1; e >= 0; --e) {
                const int i = i2 + e;
                const float d = ws.dt[i][lc], uv = ws.u[i][lc], xu = d * uv, dpv = ws.dp[i][lc];
                const f2 d2 = pack2(d, d), xu2 = pack2(xu, xu), dp2 = pack2(dpv, dpv);
                const ulonglong2 *bp = reinterpret_cast<const ulonglong2 *>(&sm.b[s * SUB + i][part * 8]);
                const ulonglong2 *cp = reinterpret_cast<const ulonglong2 *>(&sm.c[s * SUB + i][part * 8]);
                const ulonglong2 b0 = bp[0], b1 = bp[1], v0 = cp[0], v1 = cp[1];
                const f2 bv[NF] = {b0.x, b0.y, b1.x, b1.y}, cv[NF] = {v0.x, v0.y, v1.x, v1.y};
                f2 x2 = 0ull, q2 = 0ull, p2 = 0ull, db[NF], dc[NF];
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    const f2 gr = fma2(cv[j], dp2, r[j]);
                    db[j] = mul2(gr, xu2);
                    dc[j] = mul2(hist[i + 1][j], dp2);
                    x2 = fma2(gr, bv[j], x2);
                    if (Z) p2 = fma2(cv[j], hist[i + 1][j], p2);
                    r[j] = mul2(ex2_2(mul2(d2, rate[j])), gr);
                    const f2 w = mul2(r[j], hist[i][j]);
                    q2 = fma2(w, rate[j], q2);
                    da[j] = fma2(w, d2, da[j]);
                }
                ulonglong2 *row = reinterpret_cast<ulonglong2 *>(ws.red[e] + red_row<S>(lane));
                row[0] = make_ulonglong2(db[0], db[1]);
                row[1] = make_ulonglong2(db[2], db[3]);
                row[2] = make_ulonglong2(dc[0], dc[1]);
                row[3] = make_ulonglong2(dc[2], dc[3]);
                const float2 xs = unpack2(x2), qs = unpack2(q2), ps = unpack2(p2);
                float xv = xs.x + xs.y, qv = qs.x + qs.y, pv = ps.x + ps.y;
#pragma unroll
                for (int off = CHW; off < 32; off *= 2) {
                    xv += __shfl_xor_sync(0xffffffffu, xv, off);
                    qv += __shfl_xor_sync(0xffffffffu, qv, off);
                    if (Z) pv += __shfl_xor_sync(0xffffffffu, pv, off);
                }
                du[e] = fmaf(xv, d, skip_c * dpv);
                ddelta[e] = fmaf(xv, uv, qv * LN2);
                if (Z) pre[e] = fmaf(skip_c, uv, pv);
            }
            __syncwarp();
            if (part == 0)                // behind the barrier: every lane of the channel has read u and dp
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    ws.u[i2 + e][lc] = du[e];
                    ws.dp[i2 + e][lc] = ddelta[e];
                    if (Z) ws.p[i2 + e][lc] = pre[e];
                }
            // columns: pair j of part `of` over that part's CHW lanes, eight of them a lane
            constexpr int COLS = 8 * SPLIT, PER = COLS <= 32 ? 1 : 2;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int m = 0; m < PER; ++m) {
                    const int col = COLS <= 32 ? lane % COLS : lane + 32 * m, from = COLS <= 32 ? lane / COLS * 8 : 0;
                    const f2 *src = reinterpret_cast<const f2 *>(ws.red[e] + red_row<S>(col / 8 * CHW + from) + col % 8 * 2);
                    f2 v = src[0];
#pragma unroll
                    for (int l = 1; l < (CHW < 8 ? CHW : 8); ++l) v = add2(v, src[RED_ROW / 2 * l]);
#pragma unroll
                    for (int off = COLS; off < 32; off *= 2) v = add2(v, __shfl_xor_sync(0xffffffffu, v, off));
                    if (COLS >= 32 || lane < COLS) sm.sums[warp][i2 + e][col] = v;
                }
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const int i = first + j * TSTEP, t = s * SUB + i;
            if (i >= SUB || t >= count || n4 <= 0) continue;
            float d[4], v[4];
            get4(&ws.u[i][4 * quad], v);
            store4<VEC>(dup + j * TSTEP * g.du.st, n4, v);
            dk[j].get(d);
            get4(&ws.dp[i][4 * quad], v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] *= sigmoid(d[e] + bias[e]);
                dbias[e] += e < n4 ? v[e] : 0.f;
            }
            store4<VEC>(ddtp + j * TSTEP * g.ddt.st, n4, v);
            if (Z) {
                float z[4], y[4];
                zk[j].get(z);
                yk[j].get(y);
                get4(&ws.p[i][4 * quad], v);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= y[e] * dsilu(z[e], sigmoid(z[e]));
                store4<VEC>(dzp + j * TSTEP * g.dz.st, n4, v);
            }
        }
        dup -= SUB * g.du.st;
        ddtp -= SUB * g.ddt.st;
        if (Z) dzp -= SUB * g.dz.st;
        // the block's warps
        __syncthreads();
        const long long row0 = ((long long)blockIdx.x * a.B + b) * a.N + t0 + s * SUB;
        for (int i = threadIdx.x; i < SUB * S; i += THREADS) {
            if (s * SUB + i / S >= count) continue;
            f2 v = sm.sums[0][i / S][i % S];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) v = add2(v, sm.sums[w][i / S][i % S]);
            *reinterpret_cast<f2 *>(g.bc_part + (row0 + i / S) * 2 * S + 2 * (i % S)) = v;
        }
    }

    // the chunk's sums for the parameters
    if (on) {
#pragma unroll
        for (int j = 0; j < NF / 2; ++j)
            reinterpret_cast<ulonglong2 *>(state)[j] =
                make_ulonglong2(mul2(mul2(da[2 * j], rate[2 * j]), pack2(LN2, LN2)),
                                mul2(mul2(da[2 * j + 1], rate[2 * j + 1]), pack2(LN2, LN2)));
    }
#pragma unroll
    for (int off = QUADS; off < 32; off *= 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dskip[e] += __shfl_xor_sync(0xffffffffu, dskip[e], off);
            dbias[e] += __shfl_xor_sync(0xffffffffu, dbias[e], off);
        }
    if (first == 0) {
        const long long to = ((long long)b * g.chunks + k) * a.D + c4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n4) {
                g.skip[to + e] = dskip[e];
                g.bias[to + e] = dbias[e];
            }
    }
}

// The parameters' sums (the first blocks), and db and dc: the groups' blocks of channels in order, four states a thread,
// `blocks` blocks a batch row and group.
template <typename T> __global__ void __launch_bounds__(256) scan_sums_kernel(const GradArgs<T> g, const SumList l, unsigned blocks)
{
    wait_previous();
    if (blockIdx.x < l.first[l.count]) {
        sum_rows_block(l, blockIdx.x);
        return;
    }
    const ScanArgs<T> &a = g.f;
    const int per = a.S / 2;                                  // float4 of a token and group
    const unsigned block = blockIdx.x - l.first[l.count], row = block / blocks;
    const long long i = (long long)(block - row * blocks) * 256 + threadIdx.x;
    const int q = (int)(i % per), b = row % a.B, group = row / a.B;
    const long long t = i / per;
    T *out = (q % 4 < 2 ? g.db : g.dc).at(b, (int)t) + group * a.S + q / 4 * 8 + q % 2 * 4;   // per eight states: db, then dc
    if (t >= row_length(a.lengths, b, a.N)) {
        if (a.zero && t < a.N) out[0] = out[1] = out[2] = out[3] = from_f32<T>(0.f);
        return;
    }
    const float4 *p = reinterpret_cast<const float4 *>(g.bc_part) + (((long long)group * a.tiles * a.B + b) * a.N + t) * per + q;
    const long long step = (long long)a.B * a.N * per;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < a.tiles; ++k) {
        const float4 v = p[k * step];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    out[0] = from_f32<T>(s.x); out[1] = from_f32<T>(s.y); out[2] = from_f32<T>(s.z); out[3] = from_f32<T>(s.w);
}

int channels_of(int S) { return S == 8 ? Lane<8>::CH : S == 16 ? Lane<16>::CH : S == 32 ? Lane<32>::CH : Lane<64>::CH; }

// Blocks of step 4 for db and dc of a batch row and group.
long long bc_blocks(const gma_scan_t &s) { return ((long long)s.N * (s.S / 2) + 255) / 256; }

struct Layout {
    size_t bc, state, total, skip, bias, size;
};
Layout layout(const gma_scan_t &s)
{
    const size_t tiles = (s.D / s.G + channels_of(s.S) - 1) / channels_of(s.S), chunks = (s.N + scan_spacing(s) - 1) / scan_spacing(s);
    const size_t row = align_up((size_t)s.B * chunks * s.D * sizeof(float), 256);
    Layout l;
    l.bc = 0;
    l.state = align_up(s.G * tiles * s.B * s.N * 2 * s.S * sizeof(float), 256);
    l.skip = l.state + align_up((size_t)s.B * chunks * s.D * s.S * sizeof(float), 256);
    l.bias = l.skip + row;
    l.total = l.bias;                        // read before the gradients of dt_bias are written
    l.size = l.bias + row;
    return l;
}

template <typename T, int S, int CK> gma_status_t launch_ck(const GradArgs<T> &g, bool vec, cudaStream_t st)
{
    const bool z = g.f.z.p != nullptr;
    auto kern = vec ? (z ? scan_backward_kernel<T, S, CK, true, true> : scan_backward_kernel<T, S, CK, true, false>)
                    : (z ? scan_backward_kernel<T, S, CK, false, true> : scan_backward_kernel<T, S, CK, false, false>);
    if (!allow_smem(kern, sizeof(Smem<S, CK>), sizeof(Smem<S, CK>))) return GMA_ERR_CUDA;
    GMA_LAUNCH(KID_SCAN_BWD, st,
               launch_pdl(kern, dim3(g.f.tiles * g.f.G, g.chunks, g.f.B), dim3(THREADS), sizeof(Smem<S, CK>), st, g));
    return GMA_OK;
}

template <typename T, int S> gma_status_t launch(const GradArgs<T> &g, bool vec, cudaStream_t st)
{
    return g.f.spacing == 16 ? launch_ck<T, S, 16>(g, vec, st) : launch_ck<T, S, 64>(g, vec, st);
}

template <typename T> gma_status_t backward_of(const gma_scan_grad_t &s, char *ws, cudaStream_t st)
{
    const gma_scan_t &f = s.fwd;
    const Layout l = layout(f);
    const int ch = channels_of(f.S);
    GradArgs<T> g;
    g.f = scan_args<T>(f);
    g.f.tiles = (f.D / f.G + ch - 1) / ch;
    g.chunks = (f.N + g.f.spacing - 1) / g.f.spacing;
    g.dy = rows_of<const T>(s.dy);
    g.du = rows_of<T>(s.du); g.ddt = rows_of<T>(s.ddt); g.dz = rows_of<T>(s.dz);
    g.db = rows_of<T>(s.db); g.dc = rows_of<T>(s.dc);
    g.bc_part = (float *)(ws + l.bc); g.state = (float *)(ws + l.state);
    g.skip = (float *)(ws + l.skip); g.bias = (float *)(ws + l.bias);
    gma_status_t r = scan_chunk_adjoint(s, g.state, (float *)(ws + l.total), st);
    if (r != GMA_OK) return r;
    const int dt = f.dtype;
    const bool vec = scan_vec(f) && rows_vec(s.dy, dt) && rows_vec(s.du, dt) && rows_vec(s.ddt, dt) &&
                     (!f.z.ptr || rows_vec(s.dz, dt));
    r = f.S == 8 ? launch<T, 8>(g, vec, st) : f.S == 16 ? launch<T, 16>(g, vec, st)
      : f.S == 32 ? launch<T, 32>(g, vec, st) : launch<T, 64>(g, vec, st);
    if (r != GMA_OK) return r;
    SumVec v[3] = {{g.state, (long long)f.D * f.S, (long long)f.D * f.S, s.da_log, 1}};
    int count = 1;
    if (f.d_skip) v[count++] = SumVec{g.skip, f.D, f.D, s.dd_skip, 1};
    if (f.dt_bias) v[count++] = SumVec{g.bias, f.D, f.D, s.ddt_bias, 1};
    const SumList sums = sum_list(v, count, (long long)f.B * g.chunks);
    const unsigned blocks = (unsigned)bc_blocks(f);
    GMA_LAUNCH(KID_SCAN_BC, st,
               launch_pdl(scan_sums_kernel<T>, dim3(sums.first[count] + blocks * f.B * f.G), dim3(256), 0, st, g, sums, blocks));
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
    return layout(g->fwd).size;
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
    if (D * f.S > 0x3fffffffll || f.G > 65535 || bc_blocks(f) * B * f.G > 0x3fffffffll || (N + scan_spacing(f) - 1) / scan_spacing(f) > 65535) return GMA_ERR_UNSUPPORTED_SHAPE;
    if (!ws_ok(ws, ws_bytes, layout(f).size)) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    return f.dtype == GMA_BF16 ? backward_of<__nv_bfloat16>(*g, (char *)ws, st) : backward_of<float>(*g, (char *)ws, st);
}

}  // extern "C"
