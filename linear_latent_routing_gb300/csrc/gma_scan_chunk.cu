// gma_scan_chunk.cu -- the selective scan's forward pass in chunks of tokens, for states of up to 16.
//
// Lanes are channels (two a lane, whose u, dt, z and y are one 4-byte access), every warp walks over the
// tokens of one chunk with the 2 * S states in registers, and nothing is exchanged between lanes.
// The sequence is cut into chunks so that short batches fill the GPU too:
//   1. scan_chunk_state: each chunk's state from a zero start, and its sum of delta;
//   2. scan_chunk_join: over the chunks in order, state = exp(A sum delta) state + chunk's state;
//      what is in front of each chunk is its start (and a checkpoint for the backward pass);
//   3. scan_chunk_output: each chunk again from its start, with the output.
// One chunk needs step 3 alone.  Per (token, channel, state) steps 1 and 3 take two exponentials
// and about six instruction slots, of which the exponentials bind (one warp instruction in four cycles
// a scheduler).
#include "scan_tile.cuh"

namespace gma {
namespace blk {
namespace {

constexpr int CH_WARP = 64;          // channels of a warp
constexpr int STAGES = 3;            // of a warp's ring of staged tokens

// Tokens of a stage: 1 KB of each of u, dt and z.
template <typename T> constexpr int stage_tokens() { return 1024 / (CH_WARP * (int)sizeof(T)); }
constexpr int STAGE_BYTES = 3 * 1024;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;

__device__ __forceinline__ void cp_async16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T> struct ChunkArgs {
    ScanArgs<T> s;
    int chunk, chunks;               // tokens of a chunk, chunks of a sequence
    float *state;                    // [B][chunks][D][S]: chunk states, then starts
    float *total;                    // [B][chunks][D]: sums of delta
};

// Two neighbouring channels of a token, as they lie in memory until they are used.
template <typename T> struct Raw2;
template <> struct Raw2<__nv_bfloat16> {
    uint32_t w;
    template <bool VEC> __device__ __forceinline__ void load(const __nv_bfloat16 *p, int n)
    {
        if (VEC) {
            w = *reinterpret_cast<const uint32_t *>(p);
        } else {
            const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
            w = (n > 0 ? q[0] : 0u) | (n > 1 ? (uint32_t)q[1] << 16 : 0u);
        }
    }
    __device__ __forceinline__ float2 get() const { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
};
template <> struct Raw2<float> {
    float2 w;
    template <bool VEC> __device__ __forceinline__ void load(const float *p, int n)
    {
        if (VEC) w = *reinterpret_cast<const float2 *>(p);
        else w = make_float2(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f);
    }
    __device__ __forceinline__ float2 get() const { return w; }
};
template <bool VEC> __device__ __forceinline__ void store2(__nv_bfloat16 *p, int n, float2 v)
{
    if (VEC) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
    } else {
        if (n > 0) p[0] = __float2bfloat16_rn(v.x);
        if (n > 1) p[1] = __float2bfloat16_rn(v.y);
    }
}
template <bool VEC> __device__ __forceinline__ void store2(float *p, int n, float2 v)
{
    if (VEC) {
        *reinterpret_cast<float2 *>(p) = v;
    } else {
        if (n > 0) p[0] = v.x;
        if (n > 1) p[1] = v.y;
    }
}

// b or c of `count` tokens as fp32 rows of S.
template <typename T, int S>
__device__ __forceinline__ void stage_rows(const Rows<const T> &r, bool vec, int b, int first, int t0, int count, float *tile)
{
    for (int i = threadIdx.x; i < count * (S / 8); i += blockDim.x) {
        const int t = i / (S / 8), piece = i % (S / 8);
        float v[8];
        if (vec) load8<true>(r.at(b, t0 + t) + first + piece * 8, 8, v);
        else load8<false>(r.at(b, t0 + t) + first + piece * 8, 8, v);
        store8<true>(tile + t * S + piece * 8, 8, v);
    }
}

// The states' rates A log2(e), S / 2 pairs.
template <int S> __device__ __forceinline__ void load_rates(const float *a_log, long long at, bool on, f2 (&r)[S / 2])
{
#pragma unroll
    for (int q = 0; q < S / 4; ++q) {
        const float4 v = on ? reinterpret_cast<const float4 *>(a_log + at)[q] : make_float4(0.f, 0.f, 0.f, 0.f);
        r[2 * q] = on ? pack2(-expf(v.x) * LOG2E, -expf(v.y) * LOG2E) : 0ull;
        r[2 * q + 1] = on ? pack2(-expf(v.z) * LOG2E, -expf(v.w) * LOG2E) : 0ull;
    }
}
template <int S> __device__ __forceinline__ void load_state(const float *p, bool on, f2 (&h)[S / 2])
{
#pragma unroll
    for (int q = 0; q < S / 4; ++q) {
        ulonglong2 v = make_ulonglong2(0ull, 0ull);
        if (on) v = reinterpret_cast<const ulonglong2 *>(p)[q];
        h[2 * q] = v.x;
        h[2 * q + 1] = v.y;
    }
}
template <int S> __device__ __forceinline__ void store_state(float *p, bool on, const f2 (&h)[S / 2])
{
#pragma unroll
    for (int q = 0; q < S / 4; ++q)
        if (on) reinterpret_cast<ulonglong2 *>(p)[q] = make_ulonglong2(h[2 * q], h[2 * q + 1]);
}

// OUT: step 3 (states from `state`, or state_in for a single chunk), else step 1.
template <typename T, int S, bool VEC, bool OUT>
__global__ void __launch_bounds__(256, 2) scan_chunk_kernel(const ChunkArgs<T> g, bool vec_bc)
{
    extern __shared__ __align__(16) float rows_s[];
    const ScanArgs<T> &a = g.s;
    const int b = blockIdx.z, k = blockIdx.y, t0 = k * g.chunk;
    const int len = row_length(a.lengths, b, a.N);
    const int group = blockIdx.x / a.tiles, Dg = a.D / a.G;
    const int in_group = (blockIdx.x - group * a.tiles) * (blockDim.x * 2) + threadIdx.x * 2;
    const int n = min(2, Dg - in_group), c = group * Dg + in_group;
    const int count = min(g.chunk, len - t0);
    const bool only = g.chunks == 1;
    if (count <= 0) {
        // an empty sequence's state passes through
        if (OUT && only && a.state_out && a.state_out != a.state_in)
            for (int e = 0; e < n; ++e)
                for (int i = 0; i < S; ++i) {
                    const long long at = ((long long)b * a.D + c + e) * S + i;
                    a.state_out[at] = a.state_in ? a.state_in[at] : 0.f;
                }
        return;
    }
    float *bs = rows_s, *cs = rows_s + g.chunk * S;
    stage_rows<T, S>(a.b, vec_bc, b, group * S, t0, count, bs);
    if (OUT) stage_rows<T, S>(a.c, vec_bc, b, group * S, t0, count, cs);

    f2 r[2][S / 2], h[2][S / 2];
    float2 bias = make_float2(0.f, 0.f), skip = make_float2(0.f, 0.f), total = make_float2(0.f, 0.f);
    const long long row = ((long long)b * g.chunks + k) * a.D + c;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const bool on = e < n;
        load_rates<S>(a.a_log, (long long)(c + e) * S, on, r[e]);
        if (OUT && !only) load_state<S>(g.state + (row + e) * S, on, h[e]);
        else if (OUT && a.state_in) load_state<S>(a.state_in + ((long long)b * a.D + c + e) * S, on, h[e]);
        else load_state<S>(nullptr, false, h[e]);
        if (OUT && only && a.ckpt) store_state<S>(a.ckpt + ((long long)b * a.D + c + e) * S, on, h[e]);
    }
    if (n > 0 && a.dt_bias) bias.x = a.dt_bias[c];
    if (n > 1 && a.dt_bias) bias.y = a.dt_bias[c + 1];
    if (OUT && n > 0 && a.d_skip) skip.x = a.d_skip[c];
    if (OUT && n > 1 && a.d_skip) skip.y = a.d_skip[c + 1];
    __syncthreads();
    if (!VEC && n <= 0) return;

    T *yp = OUT ? a.y.at(b, t0) + c : nullptr;
    auto token = [&](int t, float2 uu, float2 dd, float2 zz) {
        const float2 dt = unpack2(softplus2(add2(pack2(dd.x, dd.y), pack2(bias.x, bias.y))));
        const float2 xu = make_float2(dt.x * uu.x, dt.y * uu.y);
        f2 y[2] = {0ull, 0ull};
        const f2 dt2[2] = {pack2(dt.x, dt.x), pack2(dt.y, dt.y)}, xu2[2] = {pack2(xu.x, xu.x), pack2(xu.y, xu.y)};
        if (!OUT) {
            total.x += dt.x;
            total.y += dt.y;
        }
#pragma unroll
        for (int q = 0; q < S / 4; ++q) {
            const ulonglong2 b2 = reinterpret_cast<const ulonglong2 *>(bs + t * S)[q];
            ulonglong2 c2;
            if (OUT) c2 = reinterpret_cast<const ulonglong2 *>(cs + t * S)[q];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                h[e][2 * q] = fma2(ex2_2(mul2(dt2[e], r[e][2 * q])), h[e][2 * q], mul2(xu2[e], b2.x));
                h[e][2 * q + 1] = fma2(ex2_2(mul2(dt2[e], r[e][2 * q + 1])), h[e][2 * q + 1], mul2(xu2[e], b2.y));
                if (OUT) {
                    y[e] = fma2(c2.x, h[e][2 * q], y[e]);
                    y[e] = fma2(c2.y, h[e][2 * q + 1], y[e]);
                }
            }
        }
        if (OUT) {
            const float2 y0 = unpack2(y[0]), y1 = unpack2(y[1]);
            float2 v = make_float2(fmaf(skip.x, uu.x, y0.x + y0.y), fmaf(skip.y, uu.y, y1.x + y1.y));
            if (a.z.p) {
                v.x *= silu(zz.x);
                v.y *= silu(zz.y);
            }
            if (!VEC || n > 0) store2<VEC>(yp, n, v);
            yp += a.y.st;
        }
    };
    if (VEC) {
        // A warp fetches its 64 channels of a stage's tokens, 16 bytes a lane, two stages ahead.
        constexpr int TOK = stage_tokens<T>(), ROW = CH_WARP * sizeof(T), SEGS = ROW / 16, PER = 32 / SEGS;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, seg = lane % SEGS, sub = lane / SEGS;
        unsigned char *ring = reinterpret_cast<unsigned char *>(rows_s) + ((OUT ? 2 : 1) * g.chunk * S * 4) + warp * RING_BYTES;
        const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
        const int first = in_group - 2 * lane + seg * (16 / (int)sizeof(T));          // channel in the group
        const bool mine = first < Dg;
        const T *up = a.u.at(b, t0) + group * Dg + first, *dp = a.dt.at(b, t0) + group * Dg + first;
        const T *zp = OUT && a.z.p ? a.z.at(b, t0) + group * Dg + first : nullptr;
        auto fetch = [&](int at, int stage) {
#pragma unroll
            for (int i = 0; i < TOK; i += PER) {
                const int t = at + i + sub;
                if (mine && t < count) {
                    const uint32_t to = ring_at + stage * STAGE_BYTES + (i + sub) * ROW + seg * 16;
                    cp_async16(to, up + t * a.u.st);
                    cp_async16(to + 1024, dp + t * a.dt.st);
                    if (zp) cp_async16(to + 2048, zp + t * a.z.st);
                }
            }
            cp_commit();
        };
        fetch(0, 0);
        fetch(TOK, 1);
        int stage = 0;
        for (int at = 0; at < count; at += TOK) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            fetch(at + 2 * TOK, stage == 0 ? 2 : stage - 1);
            const unsigned char *s = ring + stage * STAGE_BYTES + lane * 2 * sizeof(T);
#pragma unroll 2
            for (int i = 0; i < TOK; ++i) {
                if (at + i >= count) break;
                Raw2<T> u, d, z;
                u.template load<true>(reinterpret_cast<const T *>(s + i * ROW), 2);
                d.template load<true>(reinterpret_cast<const T *>(s + i * ROW + 1024), 2);
                if (OUT) z.template load<true>(reinterpret_cast<const T *>(s + i * ROW + 2048), 2);
                token(at + i, u.get(), d.get(), OUT ? z.get() : make_float2(0.f, 0.f));
            }
            stage = stage == 2 ? 0 : stage + 1;
        }
    } else {
        for (int t = 0; t < count; ++t) {
            Raw2<T> u, d, z;
            u.template load<false>(a.u.at(b, t0 + t) + c, n);
            d.template load<false>(a.dt.at(b, t0 + t) + c, n);
            if (OUT && a.z.p) z.template load<false>(a.z.at(b, t0 + t) + c, n);
            token(t, u.get(), d.get(), OUT && a.z.p ? z.get() : make_float2(0.f, 0.f));
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (!OUT) {
            store_state<S>(g.state + (row + e) * S, e < n, h[e]);
            if (e < n) g.total[row + e] = e ? total.y : total.x;
        } else if (only && a.state_out) {
            store_state<S>(a.state_out + ((long long)b * a.D + c + e) * S, e < n, h[e]);
        }
    }
}

// Step 2: four states a thread, the next chunks' loads in flight.
template <typename T, int S> __global__ void __launch_bounds__(128) scan_chunk_join_kernel(const ChunkArgs<T> g)
{
    constexpr int AHEAD = 8;
    const ScanArgs<T> &a = g.s;
    const int i = blockIdx.x * 128 + threadIdx.x, d = i / (S / 4), q = i % (S / 4), b = blockIdx.y;
    if (d >= a.D) return;
    const int len = row_length(a.lengths, b, a.N), count = (len + g.chunk - 1) / g.chunk;
    const long long at = ((long long)b * a.D + d) * S + 4 * q;
    const float4 al = *reinterpret_cast<const float4 *>(a.a_log + (long long)d * S + 4 * q);
    const float r[4] = {-expf(al.x) * LOG2E, -expf(al.y) * LOG2E, -expf(al.z) * LOG2E, -expf(al.w) * LOG2E};
    float4 h = a.state_in ? *reinterpret_cast<const float4 *>(a.state_in + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    float *state = g.state + ((long long)b * g.chunks * a.D + d) * S + 4 * q;
    const float *total = g.total + (long long)b * g.chunks * a.D + d;
    const long long step = (long long)a.D * S;
    const int nck = (a.N + CKPT - 1) / CKPT, per = CKPT / g.chunk;
    float *ck = a.ckpt ? a.ckpt + ((long long)b * nck * a.D + d) * S + 4 * q : nullptr;
    for (int k0 = 0; k0 < count; k0 += AHEAD) {
        float4 s[AHEAD];
        float tt[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (k0 + j < count) {
                s[j] = *reinterpret_cast<const float4 *>(state + (k0 + j) * step);
                tt[j] = total[(long long)(k0 + j) * a.D];
            }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (k0 + j < count) {
                *reinterpret_cast<float4 *>(state + (k0 + j) * step) = h;
                if (ck && (k0 + j) % per == 0) *reinterpret_cast<float4 *>(ck + (k0 + j) / per * step) = h;
                h.x = fmaf(ex2(tt[j] * r[0]), h.x, s[j].x);
                h.y = fmaf(ex2(tt[j] * r[1]), h.y, s[j].y);
                h.z = fmaf(ex2(tt[j] * r[2]), h.z, s[j].z);
                h.w = fmaf(ex2(tt[j] * r[3]), h.w, s[j].w);
            }
    }
    if (a.state_out) *reinterpret_cast<float4 *>(a.state_out + at) = h;
}

#ifndef CW
#define CW 12
#endif
// Tokens of a chunk: the longest of 128, 64 and 32 that still gives every SM 16 warps of work.
int chunk_of(const gma_scan_t &s)
{
    const long long warps = (long long)s.B * s.G * ((s.D / s.G + CH_WARP - 1) / CH_WARP);
    for (int c = CKPT; c > 32; c /= 2)
        if (warps * ((s.N + c - 1) / c) >= 152 * CW) return c;
    return 32;
}

template <typename T, int S, bool VEC> gma_status_t run(const gma_scan_t &s, char *ws, cudaStream_t st)
{
    ChunkArgs<T> g;
    g.s = scan_args<T>(s);
    g.chunk = chunk_of(s);
    g.chunks = (s.N + g.chunk - 1) / g.chunk;
    g.state = (float *)ws;
    g.total = (float *)(ws + align_up((size_t)s.B * g.chunks * s.D * S * sizeof(float), 256));
    const int warps = (s.D / s.G + CH_WARP - 1) / CH_WARP, per = warps < 8 ? warps : 8;
    g.s.tiles = (warps + per - 1) / per;
    const dim3 grid(g.s.tiles * s.G, g.chunks, s.B);
    const bool vec_bc = rows_vec(s.b, s.dtype) && rows_vec(s.c, s.dtype);
    const size_t rows = (size_t)g.chunk * S * sizeof(float), ring = VEC ? (size_t)per * RING_BYTES : 0;
    for (auto kern : {scan_chunk_kernel<T, S, VEC, false>, scan_chunk_kernel<T, S, VEC, true>})
        if (2 * rows + ring > 48 * 1024 &&
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(2 * rows + ring)) != cudaSuccess)
            return GMA_ERR_CUDA;
    if (g.chunks > 1) {
        GMA_LAUNCH(KID_SCAN_STATE, st, scan_chunk_kernel<T, S, VEC, false><<<grid, per * 32, rows + ring, st>>>(g, vec_bc));
        GMA_LAUNCH(KID_SCAN_JOIN, st,
                   scan_chunk_join_kernel<T, S><<<dim3((s.D * (S / 4) + 127) / 128, s.B), 128, 0, st>>>(g));
    }
    GMA_LAUNCH(KID_SCAN, st, scan_chunk_kernel<T, S, VEC, true><<<grid, per * 32, 2 * rows + ring, st>>>(g, vec_bc));
    return GMA_OK;
}

}  // namespace

bool scan_chunked(const gma_scan_t &s)
{
    return s.S <= 16 && (s.N + 31) / 32 <= 65535;
}

size_t scan_chunk_workspace(const gma_scan_t &s)
{
    const int chunk = chunk_of(s);
    const size_t chunks = (s.N + chunk - 1) / chunk;
    if (chunks == 1) return 0;
    return align_up((size_t)s.B * chunks * s.D * s.S * sizeof(float), 256) +
           align_up((size_t)s.B * chunks * s.D * sizeof(float), 256);
}

gma_status_t scan_chunk_forward(const gma_scan_t &s, void *ws, cudaStream_t st)
{
    const size_t pair = 2 * elem_size(s.dtype) - 1;
    const bool vec = (s.D / s.G) % 8 == 0 && rows_vec(s.u, s.dtype) && rows_vec(s.dt, s.dtype) &&
                     (!s.z.ptr || rows_vec(s.z, s.dtype)) &&
                     (((uintptr_t)s.y.ptr | (uintptr_t)(s.y.batch * elem_size(s.dtype)) |
                       (uintptr_t)(s.y.token * elem_size(s.dtype))) & pair) == 0;
    auto with = [&](auto t) -> gma_status_t {
        using T = decltype(t);
        if (s.S == 8) return vec ? run<T, 8, true>(s, (char *)ws, st) : run<T, 8, false>(s, (char *)ws, st);
        return vec ? run<T, 16, true>(s, (char *)ws, st) : run<T, 16, false>(s, (char *)ws, st);
    };
    return s.dtype == GMA_BF16 ? with(__nv_bfloat16{}) : with(float{});
}

}  // namespace blk
}  // namespace gma
