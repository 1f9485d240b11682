// gma_scan.cu -- the selective state space scan (gma_scan_forward) and its step for one token
// (gma_scan_step).
//
//   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t b_t[n] u_t,   y_t = (sum_n c_t[n] h_t[n] + D u_t) silu(z_t)
//
// The decay differs from channel to channel and state to state, so there is no matrix product in it:
// each (token, channel, state) takes one exponential and about five multiply-adds in fp32.  The kernel here
// spreads a tile's tokens over the lanes of a warp and needs one launch; it takes the calls with too few channels
// and tokens to fill the GPU in chunks (gma_scan_chunk.cu).  Latency bounds it there: 512 tokens of 1024
// channels x 16 states take 15 us, 32 tokens 12 us.  The step moves its state once: 128 x 2048 x 16 in 11 us
// (33.5 MB), 512 rows in 29 us (4.9 TB/s), one row of 1024 channels in the time of a launch.
#include <type_traits>

#include "scan_args.cuh"

namespace gma {
namespace blk {

static gma_status_t scan_sizes(const gma_scan_t &s)
{
    if (s.B < 1 || s.N < 1 || s.D < 1 || s.S < 1) return GMA_ERR_INVALID_ARG;
    const bool states = s.S == 8 || s.S == 16 || s.S == 32 || s.S == 64;
    return !states || s.B > 65535 || s.D > (1 << 24) || s.N > (1 << 30) ? GMA_ERR_UNSUPPORTED_SHAPE : GMA_OK;
}

gma_status_t scan_check(const gma_scan_t *s, bool out)
{
    if (!s || s->G < 1 || s->D < 1 || s->D % s->G) return GMA_ERR_INVALID_ARG;
    if (s->dtype != GMA_F32 && s->dtype != GMA_BF16) return GMA_ERR_INVALID_ARG;
    if (s->flags & ~GMA_ROWS_ZERO_TAIL || s->reserved) return GMA_ERR_INVALID_ARG;
    const gma_status_t sizes = scan_sizes(*s);
    if (sizes != GMA_OK) return sizes;
    const int dt = s->dtype;
    const long long B = s->B, N = s->N, D = s->D, GS = (long long)s->G * s->S;
    if (!rows_ok(s->u, dt, B, N, D, false) || !rows_ok(s->dt, dt, B, N, D, false) ||
        !rows_ok(s->b, dt, B, N, GS, false) || !rows_ok(s->c, dt, B, N, GS, false))
        return GMA_ERR_INVALID_ARG;
    if (s->z.ptr && !rows_ok(s->z, dt, B, N, D, false)) return GMA_ERR_INVALID_ARG;
    if (out && !rows_ok(s->y, dt, B, N, D, true)) return GMA_ERR_INVALID_ARG;
    // states are read and written in pairs and quadruples
    if (!ptr_ok(s->a_log, 16) || !opt_ok(s->d_skip, 4) || !opt_ok(s->dt_bias, 4) || !opt_ok(s->state_in, 16) ||
        !opt_ok(s->state_out, 16) || !opt_ok(s->checkpoints, 16) || !opt_ok(s->lengths, 4))
        return GMA_ERR_INVALID_ARG;
    return GMA_OK;
}

int scan_spacing(const gma_scan_t &s)
{
    const int lanes = s.S < 8 ? 1 : s.S / 8, channels = lanes < 32 ? 32 / lanes : 1;    // of a channel, of a warp
    return (double)s.B * ((s.N + 63) / 64) * ((s.D + channels - 1) / channels) < 152 * 6 ? 16 : 64;
}

bool scan_vec(const gma_scan_t &s)
{
    return (s.D / s.G) % 8 == 0 && rows_vec(s.u, s.dtype) && rows_vec(s.dt, s.dtype) &&
           (!s.z.ptr || rows_vec(s.z, s.dtype)) && rows_vec(s.b, s.dtype) && rows_vec(s.c, s.dtype);
}

namespace {

// ------------------------------------------------------------------ tokens over lanes
// A block takes CH channels of one group in one batch row, a warp each, and walks over the sequence in tiles of
// TT tokens.  A warp's lanes are time lanes, each of which owns TL neighbouring tokens: the recurrence is
// sequential over a lane's own tokens, with a scan of (decay, state) pairs over the lanes in between, so that a
// tile's exponentials are computed once and every warp has 32 lanes of independent work whatever the number of
// channels.  States n and n + 1 share packed fp32 pairs.
//
// Tiles lie in shared memory in the order the lanes read them, 16 bytes a lane without bank conflicts:
// token t = tl * TL + 4 q + e of a channel at (q * LT + tl) * 4 + e, and of a pair of states (2 q + e)
// at (q * LT + tl) * 2 + e.
constexpr int LT = 32, TL = 8, CH = 8;                      // time lanes, tokens of a lane, channels (one a warp)
constexpr int TT = LT * TL, THREADS = LT * CH;
static_assert(THREADS == TT && CH == 8, "a thread stages eight channels of one token");
constexpr int PITCH = TT + 4;                               // floats between two channels
__device__ __forceinline__ int pos(int t)
{
    const int tl = t / TL, i = t % TL;
    return ((i / 4) * LT + tl) * 4 + i % 4;
}
__device__ __forceinline__ int pos2(int t)
{
    const int tl = t / TL, i = t % TL;
    return ((i / 2) * LT + tl) * 2 + i % 2;
}

// One lane's TL values of a channel.
__device__ __forceinline__ void lane_load(const float *chan, int tl, float (&v)[TL])
{
#pragma unroll
    for (int q = 0; q < TL / 4; ++q) {
        const float4 x = *reinterpret_cast<const float4 *>(chan + (q * LT + tl) * 4);
        v[4 * q] = x.x; v[4 * q + 1] = x.y; v[4 * q + 2] = x.z; v[4 * q + 3] = x.w;
    }
}
__device__ __forceinline__ void lane_store(float *chan, int tl, const float (&v)[TL])
{
#pragma unroll
    for (int q = 0; q < TL / 4; ++q)
        *reinterpret_cast<float4 *>(chan + (q * LT + tl) * 4) =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
}

// One lane's TL values of a pair of states: two tokens of pair p.
__device__ __forceinline__ void pair_load(const f2 *tile, int p, int tl, int q, f2 &v0, f2 &v1)
{
    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(tile + p * TT + (q * LT + tl) * 2);
    v0 = x.x; v1 = x.y;
}

// Stages tokens t0 .. t0 + TT - 1 of b or c (S values a token) as pairs; zeros behind the last token.
template <typename T, bool VEC>
__device__ __forceinline__ void stage_pairs(const Rows<const T> &r, int b, int first, int t0, int len, int S, f2 *tile)
{
    const int pieces = S / 8;
    for (int i = threadIdx.x; i < TT * pieces; i += THREADS) {
        const int t = i % TT, piece = i / TT;
        float v[8];
        if (t0 + t < len) {
            load8<VEC>(r.at(b, t0 + t) + first + piece * 8, 8, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.f;
        }
        const int at = pos2(t);
#pragma unroll
        for (int k = 0; k < 4; ++k) tile[(piece * 4 + k) * TT + at] = pack2(v[2 * k], v[2 * k + 1]);
    }
}

// One step of a scan over the time lanes: takes (decay, state) of the lane `OFF` before, and where there is one,
// state += decay s and decay *= d.  The shuffle's own predicate tells.
template <int OFF> __device__ __forceinline__ void scan_step(f2 &decay, f2 &state)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 a, b, c, e;\n\t.reg .b64 d, s;\n\t"
                 "mov.b64 {a, b}, %1;\n\tmov.b64 {c, e}, %0;\n\t"
                 "shfl.sync.up.b32 a|p, a, %2, 0, 0xffffffff;\n\t"
                 "shfl.sync.up.b32 b, b, %2, 0, 0xffffffff;\n\t"
                 "shfl.sync.up.b32 c, c, %2, 0, 0xffffffff;\n\t"
                 "shfl.sync.up.b32 e, e, %2, 0, 0xffffffff;\n\t"
                 "mov.b64 d, {a, b};\n\tmov.b64 s, {c, e};\n\t"
                 "@p fma.rn.f32x2 %0, %1, s, %0;\n\t@p mul.rn.f32x2 %1, %1, d;\n\t}"
                 : "+l"(state), "+l"(decay)
                 : "n"(OFF));
}

// Inclusive scan over the time lanes.
__device__ __forceinline__ void scan_lanes(f2 &decay, f2 &state)
{
    scan_step<1>(decay, state);
    scan_step<2>(decay, state);
    scan_step<4>(decay, state);
    scan_step<8>(decay, state);
    scan_step<16>(decay, state);
}

struct ForwardSmem {
    static constexpr int U = 0;                                         // u, then p
    static constexpr int DT = U + CH * PITCH * 4;
    static constexpr int PAIRS = DT + CH * PITCH * 4;
    static_assert(PITCH % 4 == 0, "16-byte pieces");
    static size_t bytes(int S) { return PAIRS + (size_t)S * TT * 8 + (size_t)2 * CH * S * 4; }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(THREADS) scan_forward_kernel(const ScanArgs<T> a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    float *us = reinterpret_cast<float *>(smem + ForwardSmem::U);
    float *dts = reinterpret_cast<float *>(smem + ForwardSmem::DT);
    f2 *bs = reinterpret_cast<f2 *>(smem + ForwardSmem::PAIRS);
    f2 *cs = bs + a.S / 2 * TT;
    float *rate = reinterpret_cast<float *>(cs + a.S / 2 * TT);   // A log2(e), [CH][S]
    float *hs = rate + CH * a.S;                                   // the state before the tile, [CH][S]

    const int b = blockIdx.y, group = blockIdx.x / a.tiles, Dg = a.D / a.G;
    const int in_group = (blockIdx.x - group * a.tiles) * CH;
    const int c0 = group * Dg + in_group, nch = min(CH, Dg - in_group);
    const int len = row_length(a.lengths, b, a.N);
    const int ch = threadIdx.x / LT, tl = threadIdx.x % LT;
    const int nck = (a.N + a.spacing - 1) / a.spacing;

    for (int i = threadIdx.x; i < CH * a.S; i += THREADS) {
        const int k = i / a.S;
        const long long at = (long long)(c0 + k) * a.S + i % a.S;
        rate[i] = k < nch ? decay_rate(a.a_log[at]) : 0.f;
        hs[i] = k < nch && a.state_in ? a.state_in[(long long)b * a.D * a.S + at] : 0.f;
    }
    const float skip = a.d_skip && ch < nch ? a.d_skip[c0 + ch] : 0.f;

    // A thread stages the block's channels of one token of every tile, and loads the next tile's while it works on this one.
    const int token = threadIdx.x;
    float bias[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) bias[k] = a.dt_bias && k < nch ? a.dt_bias[c0 + k] : 0.f;
    Raw8<T> ur, dr, zr;
    auto fetch = [&](int t0) {
        ur.zero();
        dr.zero();
        if (VEC && t0 + token < len) {
            ur.load(a.u.at(b, t0 + token) + c0);
            dr.load(a.dt.at(b, t0 + token) + c0);
        }
    };
    fetch(0);

    for (int t0 = 0; t0 < len; t0 += TT) {
        const int t = t0 + token, at = pos(token);
        const bool on = t < len;
        __syncthreads();
        // u and delta of the tile, transposed; zeros behind the last token leave the state alone
        {
            float u[CH], d[CH];
            if (VEC) {
                ur.get(u);
                dr.get(d);
            } else {
                load8<false>(a.u.at(b, t) + c0, on ? nch : 0, u);
                load8<false>(a.dt.at(b, t) + c0, on ? nch : 0, d);
            }
#pragma unroll
            for (int k = 0; k < CH; k += 2) {
                const float2 s = unpack2(softplus2(add2(pack2(d[k], d[k + 1]), pack2(bias[k], bias[k + 1]))));
                us[k * PITCH + at] = u[k];
                us[(k + 1) * PITCH + at] = u[k + 1];
                dts[k * PITCH + at] = on && k < nch ? s.x : 0.f;
                dts[(k + 1) * PITCH + at] = on && k + 1 < nch ? s.y : 0.f;
            }
        }
        stage_pairs<T, VEC>(a.b, b, group * a.S, t0, len, a.S, bs);
        stage_pairs<T, VEC>(a.c, b, group * a.S, t0, len, a.S, cs);
        __syncthreads();
        fetch(t0 + TT);
        zr.zero();
        if (VEC && a.z.p && on) zr.load(a.z.at(b, t) + c0);

        {
            float dt[TL], u[TL];
            lane_load(dts + ch * PITCH, tl, dt);
            lane_load(us + ch * PITCH, tl, u);
            f2 dt2[TL], xu2[TL], y2[TL];
            float total = 0.f;
#pragma unroll
            for (int i = 0; i < TL; ++i) {
                total += dt[i];
                dt2[i] = pack2(dt[i], dt[i]);
                xu2[i] = pack2(dt[i] * u[i], dt[i] * u[i]);
                y2[i] = pack2(skip * u[i], 0.f);
            }
            const f2 total2 = pack2(total, total);
            const int start = t0 + tl * TL;
            const bool keep = a.ckpt && start % a.spacing == 0 && start < len && ch < nch;
            float *ck = keep ? a.ckpt + (((long long)b * nck + start / a.spacing) * a.D + c0 + ch) * a.S : nullptr;
            for (int p = 0; p < a.S / 2; ++p) {
                const f2 r2 = *reinterpret_cast<const f2 *>(rate + ch * a.S + 2 * p);
                f2 *h0 = reinterpret_cast<f2 *>(hs + ch * a.S + 2 * p);
                f2 a2[TL], x2[TL], h = 0ull;
#pragma unroll
                for (int q = 0; q < TL / 2; ++q) pair_load(bs, p, tl, q, x2[2 * q], x2[2 * q + 1]);
#pragma unroll
                for (int i = 0; i < TL; ++i) {
                    a2[i] = ex2_2(mul2(dt2[i], r2));
                    x2[i] = mul2(x2[i], xu2[i]);
                    h = fma2(a2[i], h, x2[i]);
                }
                f2 decay = ex2_2(mul2(total2, r2));
                scan_lanes(decay, h);
                const f2 before = *h0;
                const f2 d1 = __shfl_up_sync(0xffffffffu, decay, 1, LT);
                const f2 s1 = __shfl_up_sync(0xffffffffu, h, 1, LT);
                const f2 end = fma2(decay, before, h);
                h = tl ? fma2(d1, before, s1) : before;
                __syncwarp();                  // every lane has read h0
                if (tl == LT - 1) *h0 = end;
                if (keep) *reinterpret_cast<f2 *>(ck + 2 * p) = h;
#pragma unroll
                for (int q = 0; q < TL / 2; ++q) {
                    f2 c2[2];
                    pair_load(cs, p, tl, q, c2[0], c2[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        h = fma2(a2[2 * q + e], h, x2[2 * q + e]);
                        y2[2 * q + e] = fma2(c2[e], h, y2[2 * q + e]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < TL; ++i) {
                const float2 y = unpack2(y2[i]);
                u[i] = y.x + y.y;
            }
            lane_store(us + ch * PITCH, tl, u);
        }
        __syncthreads();
        if (on) {
            float y[CH];
#pragma unroll
            for (int k = 0; k < CH; ++k) y[k] = us[k * PITCH + at];
            if (a.z.p) {
                float z[CH];
                if (VEC) zr.get(z);
                else load8<false>(a.z.at(b, t) + c0, nch, z);
#pragma unroll
                for (int k = 0; k < CH; ++k) y[k] *= silu(z[k]);
            }
            store8<VEC>(a.y.at(b, t) + c0, nch, y);
        }
    }
    __syncthreads();
    if (a.zero)
        for (int t = len + token; t < a.N; t += THREADS) {
            const float none[CH] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            store8<VEC>(a.y.at(b, t) + c0, nch, none);
        }
    if (a.state_out)
        for (int i = threadIdx.x; i < nch * a.S; i += THREADS)
            a.state_out[((long long)b * a.D + c0) * a.S + i] = hs[i];
}

// One token: a lane holds four states of a channel, S / 4 lanes a channel.  The state is read and written once, which
// bounds it.  A block walks over batch rows, the next row's loads in flight, with its channels' rates computed once:
// 512 x 2048 x 16 in 29 us (a block for every two rows 38 us, every row 43 us), 128 in 11 us (13, 15).
__device__ __forceinline__ void quad(const __nv_bfloat16 *p, bool vec, float (&v)[4])
{
    if (vec) {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
        v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __bfloat162float(p[k]);
    }
}
__device__ __forceinline__ void quad(const float *p, bool vec, float (&v)[4])
{
    if (vec) {
        const float4 q = *reinterpret_cast<const float4 *>(p);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = p[k];
    }
}

constexpr int STEP_BLOCKS = 4;       // an SM
template <typename T, int S>
__global__ void __launch_bounds__(256, STEP_BLOCKS) scan_step_kernel(const ScanArgs<T> a, bool vec, int rows)
{
    constexpr int LPC = S / 4, CPB = 256 / LPC;
    const int d = blockIdx.x * CPB + threadIdx.x / LPC, q = threadIdx.x % LPC;
    const int b0 = blockIdx.y * rows, end = min(a.B, b0 + rows);
    const bool on = d < a.D;
    struct Row {
        float4 h;
        T u, dt, z;
        float b[4], c[4];
    };
    const int first = d / (a.D / a.G) * S + 4 * q;
    auto load = [&](int b, Row &r) {
        if (!on || b >= end) return;
        r.h = *reinterpret_cast<const float4 *>(a.state_in + ((long long)b * a.D + d) * S + 4 * q);
        r.u = a.u.at(b, 0)[d];
        r.dt = a.dt.at(b, 0)[d];
        if (a.z.p && q == 0) r.z = a.z.at(b, 0)[d];
        quad(a.b.at(b, 0) + first, vec, r.b);
        quad(a.c.at(b, 0) + first, vec, r.c);
    };
    Row cur, next;
    load(b0, cur);
    float rate[4] = {0.f, 0.f, 0.f, 0.f}, bias = 0.f, skip = 0.f;
    if (on) {
        const float4 v = *reinterpret_cast<const float4 *>(a.a_log + (long long)d * S + 4 * q);
        rate[0] = decay_rate(v.x); rate[1] = decay_rate(v.y);
        rate[2] = decay_rate(v.z); rate[3] = decay_rate(v.w);
        if (a.dt_bias) bias = a.dt_bias[d];
        if (a.d_skip) skip = a.d_skip[d];
    }
    for (int b = b0; b < end; ++b) {
        load(b + 1, next);
        float y = 0.f;
        if (on) {
            const float delta = softplus(to_f32<T>(cur.dt) + bias), xu = delta * to_f32<T>(cur.u);
            float h[4] = {cur.h.x, cur.h.y, cur.h.z, cur.h.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[k] = fmaf(ex2(rate[k] * delta), h[k], xu * cur.b[k]);
                y = fmaf(cur.c[k], h[k], y);
            }
            *reinterpret_cast<float4 *>(a.state_out + ((long long)b * a.D + d) * S + 4 * q) = make_float4(h[0], h[1], h[2], h[3]);
        }
#pragma unroll
        for (int off = LPC / 2; off; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (on && q == 0) {
            float v = fmaf(skip, to_f32<T>(cur.u), y);
            if (a.z.p) v *= silu(to_f32<T>(cur.z));
            a.y.at(b, 0)[d] = from_f32<T>(v);
        }
        cur = next;
    }
}

template <typename T, bool VEC> gma_status_t forward_of(const gma_scan_t &s, cudaStream_t st)
{
    ScanArgs<T> a = scan_args<T>(s);
    a.tiles = (s.D / s.G + CH - 1) / CH;
    const size_t smem = ForwardSmem::bytes(s.S);
    auto kern = scan_forward_kernel<T, VEC>;
    if (!allow_smem(kern, smem, ForwardSmem::bytes(MAX_S))) return GMA_ERR_CUDA;
    GMA_LAUNCH(KID_SCAN, st, kern<<<dim3(a.tiles * s.G, s.B), THREADS, smem, st>>>(a));
    return GMA_OK;
}

}  // namespace
}  // namespace blk
}  // namespace gma

using namespace gma;
using namespace gma::blk;

extern "C" {

int gma_scan_checkpoint_tokens(const gma_scan_t *s) { return s && scan_sizes(*s) == GMA_OK ? scan_spacing(*s) : 0; }

size_t gma_scan_checkpoint_size(const gma_scan_t *s)
{
    const int spacing = gma_scan_checkpoint_tokens(s);
    return spacing ? (size_t)s->B * ((s->N + spacing - 1) / spacing) * s->D * s->S * sizeof(float) : 0;
}

size_t gma_scan_workspace_size(const gma_scan_t *s)
{
    return scan_check(s, false) == GMA_OK && scan_chunked(*s) ? scan_chunk_workspace(*s) : 0;
}

gma_status_t gma_scan_forward(const gma_scan_t *s, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    gma_status_t r = scan_check(s, true);
    if (r != GMA_OK) return r;
    if (!ws_ok(ws, ws_bytes, gma_scan_workspace_size(s))) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    if (scan_chunked(*s)) return scan_chunk_forward(*s, ws, st);
    const bool vec = scan_vec(*s) && rows_vec(s->y, s->dtype);
    if (s->dtype == GMA_BF16)
        return vec ? forward_of<__nv_bfloat16, true>(*s, st) : forward_of<__nv_bfloat16, false>(*s, st);
    return vec ? forward_of<float, true>(*s, st) : forward_of<float, false>(*s, st);
}

gma_status_t gma_scan_step(const gma_scan_t *scan, gma_stream_t stream)
{
    if (!scan) return GMA_ERR_INVALID_ARG;
    gma_scan_t one = *scan, *s = &one;       // its token strides are ignored
    one.u.token = one.dt.token = one.z.token = one.b.token = one.c.token = one.y.token = 0;
    gma_status_t r = scan_check(s, true);
    if (r != GMA_OK) return r;
    if (s->N != 1 || !s->state_in || !s->state_out || s->lengths || s->checkpoints) return GMA_ERR_INVALID_ARG;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    auto run = [&](auto t) -> gma_status_t {
        using T = decltype(t);
        const ScanArgs<T> a = scan_args<T>(*s);
        const int cpb = 256 / (s->S / 4), tiles = (s->D + cpb - 1) / cpb;
        const bool vec = rows_vec(s->b, s->dtype) && rows_vec(s->c, s->dtype);
        // as many batch rows a block as leave STEP_BLOCKS blocks an SM
        const long long at_once = 152 * STEP_BLOCKS;
        const int rows = (int)(((long long)tiles * s->B + at_once - 1) / at_once);
        const dim3 grid(tiles, (s->B + rows - 1) / rows);
        auto launch = [&](auto n) -> gma_status_t {
            GMA_LAUNCH(KID_SCAN_STEP, st, scan_step_kernel<T, decltype(n)::value><<<grid, 256, 0, st>>>(a, vec, rows));
            return GMA_OK;
        };
        return s->S == 8 ? launch(std::integral_constant<int, 8>{}) : s->S == 16 ? launch(std::integral_constant<int, 16>{})
             : s->S == 32 ? launch(std::integral_constant<int, 32>{}) : launch(std::integral_constant<int, 64>{});
    };
    return s->dtype == GMA_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

}  // extern "C"
