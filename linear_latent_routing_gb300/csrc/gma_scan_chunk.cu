// gma_scan_chunk.cu -- the selective scan's forward pass in chunks of tokens, and the adjoint behind every chunk of
// its backward pass.
//
// Lanes are channels, every warp walks over the tokens of one chunk with its states in registers, and
// nothing but y is exchanged between lanes: a lane holds the states of two channels (8 or 16 each, whose u, dt, z
// and y are one access) or 32 of one; with S = 64 two lanes share a channel.
// The sequence is cut into chunks so that short batches fill the GPU too:
//   1. scan_chunk_state: each chunk's state from a zero start, and its sum of delta;
//   2. scan_chunk_join: over the chunks in order, state = exp(A sum delta) state + chunk's state;
//      what is in front of each chunk is its start (and a checkpoint for the backward pass);
//   3. scan_chunk_output: each chunk again from its start, with the output.
// One chunk needs step 3 alone.  Per (token, channel, state) steps 1 and 3 take two exponentials
// (of 32 a clock and SM) and three and a half packed fp32 instructions; issue (62 % while an SM has work, 51 % of the
// elapsed time), the exponentials' pipe (53 and 43 %) and the last wave's empty places bind together.
// Measured: 65536 tokens of 2048 channels x 16 states, bf16 with a gate: 354 us, 32 us and 508 us (69 and 99
// instructions an element); 4 x 2048 x 1024: 37, 10 and 47 us.
#include "scan_args.cuh"

namespace gma {
namespace blk {
namespace {

template <int S> struct Lanes {
    static constexpr int CPL = S <= 16 ? 2 : 1;              // channels of a lane
    static constexpr int SL = S <= 32 ? S : 32;              // its states of each
    static constexpr int SPLIT = S / SL;                     // lanes of a channel
    static constexpr int CH_WARP = 32 * CPL / SPLIT;         // channels of a warp
};
constexpr int STAGES = 3;            // of a warp's ring of staged tokens

// Tokens of a stage: 1 KB of each of u, dt and z.
template <typename T, int S> struct Stage { static constexpr int TOKENS = 1024 / (Lanes<S>::CH_WARP * (int)sizeof(T)); };
constexpr int STAGE_BYTES = 3 * 1024;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int MAX_WARPS = 8, MAX_ROWS = 4096;      // of a block; of a chunk's b or c, in values
constexpr size_t MAX_SMEM = 2 * MAX_ROWS * sizeof(float) + MAX_WARPS * RING_BYTES;

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

// One or two (CPL) neighbouring channels of a staged token; storing, n of them exist.
template <int CPL> __device__ __forceinline__ float2 load_ch(const __nv_bfloat16 *p)
{
    if (CPL == 1) return make_float2(__bfloat162float(p[0]), 0.f);
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <int CPL> __device__ __forceinline__ float2 load_ch(const float *p)
{
    return CPL == 1 ? make_float2(p[0], 0.f) : *reinterpret_cast<const float2 *>(p);
}
template <int CPL, bool VEC> __device__ __forceinline__ void store_ch(__nv_bfloat16 *p, int n, float2 v)
{
    if (CPL == 2 && VEC) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
    } else {
        p[0] = __float2bfloat16_rn(v.x);
        if (CPL == 2 && n > 1) p[1] = __float2bfloat16_rn(v.y);
    }
}
template <int CPL, bool VEC> __device__ __forceinline__ void store_ch(float *p, int n, float2 v)
{
    if (CPL == 2 && VEC) {
        *reinterpret_cast<float2 *>(p) = v;
    } else {
        p[0] = v.x;
        if (CPL == 2 && n > 1) p[1] = v.y;
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

// A lane's states' rates A log2(e), in pairs.
template <int S> __device__ __forceinline__ void load_rates(const float *a_log, long long at, bool on, f2 (&r)[S / 2])
{
#pragma unroll
    for (int q = 0; q < S / 4; ++q) {
        const float4 v = on ? reinterpret_cast<const float4 *>(a_log + at)[q] : make_float4(0.f, 0.f, 0.f, 0.f);
        r[2 * q] = on ? pack2(decay_rate(v.x), decay_rate(v.y)) : 0ull;
        r[2 * q + 1] = on ? pack2(decay_rate(v.z), decay_rate(v.w)) : 0ull;
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

// STATE: step 1.  OUTPUT: step 3 (states from `state`, or state_in for a single chunk).  ADJOINT: step 1 of
// the backward pass, over the tokens from the last one back: r = exp(delta A) (c dp + r), where the rows
// of dy come in u's place.
enum Mode { STATE, OUTPUT, ADJOINT };
template <typename T, int S, bool VEC, Mode MODE>
__global__ void __launch_bounds__(256, 2) scan_chunk_kernel(const ChunkArgs<T> g, bool vec_bc)
{
    constexpr bool OUT = MODE == OUTPUT, ADJ = MODE == ADJOINT;
    constexpr int CPL = Lanes<S>::CPL, SL = Lanes<S>::SL, SPLIT = Lanes<S>::SPLIT, CH_WARP = Lanes<S>::CH_WARP;
    extern __shared__ __align__(16) float rows_s[];
    if (!OUT) let_next();                 // step 3 is a call's last launch
    const ScanArgs<T> &a = g.s;
    const int b = blockIdx.z, k = blockIdx.y, t0 = k * g.chunk;
    const int len = row_length(a.lengths, b, a.N);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = SPLIT == 2 ? lane >> 4 : 0;
    const int group = blockIdx.x / a.tiles, Dg = a.D / a.G;
    const int warp_ch = ((blockIdx.x - group * a.tiles) * (blockDim.x / 32) + warp) * CH_WARP;   // in the group
    const int in_group = warp_ch + (SPLIT == 2 ? lane & 15 : lane * CPL);
    const int n = max(0, min(CPL, Dg - in_group)), c = group * Dg + in_group;
    const int count = min(g.chunk, len - t0);
    const bool only = g.chunks == 1;
    const long long in_b = ((long long)b * a.D + c) * S + part * SL;      // states of this lane in [B][D][S]
    if (OUT && a.zero && n > 0 && part == 0)
        for (int t = max(count, 0); t < min(g.chunk, a.N - t0); ++t)
            store_ch<CPL, VEC>(a.y.at(b, t0 + t) + c, n, make_float2(0.f, 0.f));
    if (count <= 0) {
        if (OUT) wait_previous();
        // an empty sequence's state passes through
        if (OUT && k == 0 && a.state_out && a.state_out != a.state_in && only)
            for (int e = 0; e < n; ++e)
                for (int i = 0; i < SL; ++i)
                    a.state_out[in_b + e * S + i] = a.state_in ? a.state_in[in_b + e * S + i] : 0.f;
        return;
    }
    float *bs = rows_s, *cs = rows_s + g.chunk * S;
    stage_rows<T, S>(ADJ ? a.c : a.b, vec_bc, b, group * S, t0, count, bs);
    if (OUT) stage_rows<T, S>(a.c, vec_bc, b, group * S, t0, count, cs);
    bs += part * SL;
    cs += part * SL;

    f2 r[CPL][SL / 2], h[CPL][SL / 2];
    float2 bias = make_float2(0.f, 0.f), skip = make_float2(0.f, 0.f), total = make_float2(0.f, 0.f);
    const long long row = ((long long)b * g.chunks + k) * a.D + c;
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
        const bool on = e < n;
        load_rates<SL>(a.a_log, (long long)(c + e) * S + part * SL, on, r[e]);
        if (OUT && e == 0) wait_previous();
        if (OUT && !only) load_state<SL>(g.state + (row + e) * S + part * SL, on, h[e]);
        else if (OUT && a.state_in) load_state<SL>(a.state_in + in_b + e * S, on, h[e]);
        else load_state<SL>(nullptr, false, h[e]);
        if (OUT && only && a.ckpt) store_state<SL>(a.ckpt + in_b + e * S, on, h[e]);
    }
    if (n > 0 && a.dt_bias) bias.x = a.dt_bias[c];
    if (n > 1 && a.dt_bias) bias.y = a.dt_bias[c + 1];
    if (OUT && n > 0 && a.d_skip) skip.x = a.d_skip[c];
    if (OUT && n > 1 && a.d_skip) skip.y = a.d_skip[c + 1];
    __syncthreads();
    if (warp_ch >= Dg) return;

    T *yp = OUT ? a.y.at(b, t0) + c : nullptr;
    auto token = [&](int t, float2 uu, float2 dd, float2 zz) {
        const float2 dt = unpack2(softplus2(add2(pack2(dd.x, dd.y), pack2(bias.x, bias.y))));
        if (ADJ && a.z.p) uu = make_float2(uu.x * silu(zz.x), CPL == 2 ? uu.y * silu(zz.y) : 0.f);
        const float de[2] = {dt.x, dt.y}, xe[2] = {ADJ ? uu.x : dt.x * uu.x, ADJ ? uu.y : dt.y * uu.y};
        f2 y[CPL], dt2[CPL], xu2[CPL];
#pragma unroll
        for (int e = 0; e < CPL; ++e) {
            y[e] = 0ull;
            dt2[e] = pack2(de[e], de[e]);
            xu2[e] = pack2(xe[e], xe[e]);
        }
        if (!OUT) {
            total.x += dt.x;
            total.y += dt.y;
        }
#pragma unroll
        for (int q = 0; q < SL / 4; ++q) {
            const ulonglong2 b2 = reinterpret_cast<const ulonglong2 *>(bs + t * S)[q];
            ulonglong2 c2;
            if (OUT) c2 = reinterpret_cast<const ulonglong2 *>(cs + t * S)[q];
#pragma unroll
            for (int e = 0; e < CPL; ++e) {
                const f2 a0 = ex2_2(mul2(dt2[e], r[e][2 * q])), a1 = ex2_2(mul2(dt2[e], r[e][2 * q + 1]));
                if (ADJ) {
                    h[e][2 * q] = mul2(a0, fma2(xu2[e], b2.x, h[e][2 * q]));
                    h[e][2 * q + 1] = mul2(a1, fma2(xu2[e], b2.y, h[e][2 * q + 1]));
                } else {
                    h[e][2 * q] = fma2(a0, h[e][2 * q], mul2(xu2[e], b2.x));
                    h[e][2 * q + 1] = fma2(a1, h[e][2 * q + 1], mul2(xu2[e], b2.y));
                }
                if (OUT) {
                    y[e] = fma2(c2.x, h[e][2 * q], y[e]);
                    y[e] = fma2(c2.y, h[e][2 * q + 1], y[e]);
                }
            }
        }
        if (OUT) {
            const float2 y0 = unpack2(y[0]), y1 = CPL == 2 ? unpack2(y[CPL - 1]) : make_float2(0.f, 0.f);
            float2 v = make_float2(y0.x + y0.y, y1.x + y1.y);
            if (SPLIT == 2) v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
            v.x = fmaf(skip.x, uu.x, v.x);
            v.y = fmaf(skip.y, uu.y, v.y);
            if (a.z.p) {
                v.x *= silu(zz.x);
                if (CPL == 2) v.y *= silu(zz.y);
            }
            if (n > 0 && part == 0) store_ch<CPL, VEC>(yp, n, v);
            yp += a.y.st;
        }
    };
    constexpr int TOK = Stage<T, S>::TOKENS, ROW = CH_WARP * (int)sizeof(T), PIECE = 1024 / (int)sizeof(T);
    unsigned char *ring = reinterpret_cast<unsigned char *>(rows_s) + ((OUT ? 2 : 1) * g.chunk * S * 4) +
                          warp * (VEC ? RING_BYTES : STAGE_BYTES);
    auto tokens = [&](int at, int stage) {
        const T *s = reinterpret_cast<const T *>(ring + stage * STAGE_BYTES) + (in_group - warp_ch);
        const int m = min(TOK, count - at);
#pragma unroll 2
        for (int i = 0; i < m; ++i) {
            const T *p = s + i * CH_WARP;
            const float2 z = OUT || ADJ ? load_ch<CPL>(p + 2 * PIECE) : make_float2(0.f, 0.f);
            token(ADJ ? count - 1 - at - i : at + i, load_ch<CPL>(p), load_ch<CPL>(p + PIECE), z);
        }
    };
    if (VEC) {
        // A warp fetches its channels of a stage's tokens, 16 bytes a lane, two stages ahead.
        constexpr int SEGS = ROW / 16, PER = 32 / SEGS;
        const int seg = lane % SEGS, sub = lane / SEGS;
        const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
        const int first = warp_ch + seg * (16 / (int)sizeof(T));
        const bool mine = first < Dg;
        const T *up = a.u.at(b, t0) + group * Dg + first, *dp = a.dt.at(b, t0) + group * Dg + first;
        const T *zp = (OUT || ADJ) && a.z.p ? a.z.at(b, t0) + group * Dg + first : nullptr;
        auto fetch = [&](int at, int stage) {
#pragma unroll
            for (int i = 0; i < TOK; i += PER) {
                const int step = at + i + sub, t = ADJ ? count - 1 - step : step;
                if (mine && step < count) {
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
            tokens(at, stage);
            stage = stage == 2 ? 0 : stage + 1;
        }
    } else {
        // A lane copies its own channels, the loads of four or eight tokens at a time; token by token, each one's latency
        // was waited for (16384 x 1100 x 16: 559 -> 341 us).
        constexpr int BATCH = 8 / CPL;
        const T *up = a.u.at(b, t0) + c, *dp = a.dt.at(b, t0) + c, *zp = (OUT || ADJ) && a.z.p ? a.z.at(b, t0) + c : nullptr;
        T *to = reinterpret_cast<T *>(ring) + (in_group - warp_ch);
        for (int at = 0; at < count; at += TOK) {
            if (SPLIT == 2) __syncwarp();
#pragma unroll
            for (int i0 = 0; i0 < TOK; i0 += BATCH) {
                T v[BATCH][3][CPL];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int step = at + i0 + i;
                    const long long t = ADJ ? count - 1 - step : step;
#pragma unroll
                    for (int e = 0; e < CPL; ++e)
                        if (e < n && part == 0 && step < count) {
                            v[i][0][e] = up[t * a.u.st + e];
                            v[i][1][e] = dp[t * a.dt.st + e];
                            if (zp) v[i][2][e] = zp[t * a.z.st + e];
                        }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
#pragma unroll
                    for (int e = 0; e < CPL; ++e)
                        if (e < n && part == 0 && at + i0 + i < count) {
                            to[(i0 + i) * CH_WARP + e] = v[i][0][e];
                            to[(i0 + i) * CH_WARP + PIECE + e] = v[i][1][e];
                            if (zp) to[(i0 + i) * CH_WARP + 2 * PIECE + e] = v[i][2][e];
                        }
            }
            if (SPLIT == 2) __syncwarp();
            tokens(at, 0);
        }
    }
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
        if (!OUT) {
            store_state<SL>(g.state + (row + e) * S + part * SL, e < n, h[e]);
            if (e < n && part == 0) g.total[row + e] = e ? total.y : total.x;
        } else if (only && a.state_out) {
            store_state<SL>(a.state_out + in_b + e * S, e < n, h[e]);
        }
    }
}

// Step 2: one state a thread, the next chunks' loads in flight.  BACK: from the last chunk to the first, for
// the backward pass, whose `state_in` is dstate_out and `state_out` dstate_in; the rows of the chunks behind a
// sequence's end are cleared (they are added up later, with those of the others).
template <typename T, int S, bool BACK> __global__ void __launch_bounds__(128) scan_chunk_join_kernel(const ChunkArgs<T> g)
{
    constexpr int AHEAD = 16;
    let_next();
    const ScanArgs<T> &a = g.s;
    const int i = blockIdx.x * 128 + threadIdx.x, d = i / S, b = blockIdx.y;
    if (d >= a.D) return;
    const int len = row_length(a.lengths, b, a.N), count = (len + g.chunk - 1) / g.chunk;
    const long long step = (long long)a.D * S, at = b * step + i;
    const float r = decay_rate(a.a_log[i]);
    wait_previous();
    float h = a.state_in ? a.state_in[at] : 0.f;
    float *state = g.state + (long long)b * g.chunks * step + i;
    const float *total = g.total + (long long)b * g.chunks * a.D + d;
    // chunks between two checkpoints, a power of two
    const int nck = (a.N + a.spacing - 1) / a.spacing, per = max(1, a.spacing / g.chunk), per_log = 31 - __clz(per);
    float *ck = a.ckpt ? a.ckpt + (long long)b * nck * step + i : nullptr;
    for (int k0 = 0; k0 < count; k0 += AHEAD) {
        float s[AHEAD], tt[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (k0 + j < count) {
                const int k = BACK ? count - 1 - k0 - j : k0 + j;
                s[j] = state[k * step];
                tt[j] = total[(long long)k * a.D];
            }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (k0 + j < count) {
                const int k = BACK ? count - 1 - k0 - j : k0 + j;
                state[k * step] = h;
                if (ck && (k & (per - 1)) == 0) ck[(k >> per_log) * step] = h;
                h = fmaf(ex2(tt[j] * r), h, s[j]);
            }
    }
    if (BACK)
        for (int k = count; k < g.chunks; ++k) state[k * step] = 0.f;
    if (a.state_out) a.state_out[at] = h;
}

template <int S> int warps_of(const gma_scan_t &s) { return (s.D / s.G + Lanes<S>::CH_WARP - 1) / Lanes<S>::CH_WARP; }
int group_warps(const gma_scan_t &s)
{
    return s.S <= 16 ? warps_of<16>(s) : s.S == 32 ? warps_of<32>(s) : warps_of<64>(s);
}

// Blocks of up to eight warps over a group's channels, as even as they can be (260 channels of 32 a warp: 5 + 5, not 8 + 8).
struct Blocks {
    int tiles, warps;
};
Blocks blocks_of(const gma_scan_t &s)
{
    const int warps = group_warps(s), tiles = (warps + MAX_WARPS - 1) / MAX_WARPS;
    return Blocks{tiles, (warps + tiles - 1) / tiles};
}

// Tokens of a chunk, of 32, 64, 128 and 256: what takes least by (waves + 1/2) (chunk + 24), where a wave is
// the 304 blocks that run at once and 24 tokens' time goes into a chunk's start and the join.  A chunk's b and c
// stay within 32 KB (two blocks an SM), and a chunk does not step over a checkpoint.
int chunk_of(const gma_scan_t &s)
{
    const Blocks blocks = blocks_of(s);
    const double rows = (double)s.B * s.G * blocks.tiles * blocks.warps / 8;
    int best = 32;
    double least = 0;
    for (int c = 32; c <= 256 && c * s.S <= MAX_ROWS && !(s.checkpoints && c > scan_spacing(s)); c *= 2) {
        const double waves = rows * ((s.N + c - 1) / c) / 304 + 0.5, cost = (waves > 1 ? waves : 1) * (c + 24);
        if (c == 32 || cost < least) best = c, least = cost;
    }
    return best;
}

// The backward pass's adjoint behind every chunk.
template <typename T, int S, bool VEC>
gma_status_t run_adjoint(const gma_scan_grad_t &grad, float *state, float *total, cudaStream_t st)
{
    const gma_scan_t &s = grad.fwd;
    ChunkArgs<T> g;
    g.s = scan_args<T>(s);
    g.s.u = rows_of<const T>(grad.dy);
    g.s.state_in = grad.dstate_out;
    g.s.state_out = grad.dstate_in;
    g.s.ckpt = nullptr;
    g.chunk = g.s.spacing;
    g.chunks = (s.N + g.chunk - 1) / g.chunk;
    g.state = state;
    g.total = total;
    const Blocks blocks = blocks_of(s);
    const int per = blocks.warps;
    g.s.tiles = blocks.tiles;
    const size_t smem = (size_t)g.chunk * S * sizeof(float) + (size_t)per * (VEC ? RING_BYTES : STAGE_BYTES);
    auto kern = scan_chunk_kernel<T, S, VEC, ADJOINT>;
    if (!allow_smem(kern, smem, MAX_SMEM)) return GMA_ERR_CUDA;
    GMA_LAUNCH(KID_SCAN_ADJ, st, kern<<<dim3(g.s.tiles * s.G, g.chunks, s.B), per * 32, smem, st>>>(g, rows_vec(s.c, s.dtype)));
    GMA_LAUNCH(KID_SCAN_JOIN, st,
               launch_pdl(scan_chunk_join_kernel<T, S, true>, dim3((s.D * S + 127) / 128, s.B), dim3(128), 0, st, g));
    return GMA_OK;
}

template <typename T, int S, bool VEC> gma_status_t run(const gma_scan_t &s, char *ws, cudaStream_t st)
{
    ChunkArgs<T> g;
    g.s = scan_args<T>(s);
    g.chunk = chunk_of(s);
    g.chunks = (s.N + g.chunk - 1) / g.chunk;
    g.state = (float *)ws;
    g.total = (float *)(ws + align_up((size_t)s.B * g.chunks * s.D * S * sizeof(float), 256));
    const Blocks blocks = blocks_of(s);
    const int per = blocks.warps;
    g.s.tiles = blocks.tiles;
    const dim3 grid(g.s.tiles * s.G, g.chunks, s.B);
    const bool vec_bc = rows_vec(s.b, s.dtype) && rows_vec(s.c, s.dtype);
    const size_t rows = (size_t)g.chunk * S * sizeof(float), ring = (size_t)per * (VEC ? RING_BYTES : STAGE_BYTES);
    for (auto kern : {scan_chunk_kernel<T, S, VEC, STATE>, scan_chunk_kernel<T, S, VEC, OUTPUT>})
        if (!allow_smem(kern, 2 * rows + ring, MAX_SMEM)) return GMA_ERR_CUDA;
    if (g.chunks > 1) {
        GMA_LAUNCH(KID_SCAN_STATE, st, scan_chunk_kernel<T, S, VEC, STATE><<<grid, per * 32, rows + ring, st>>>(g, vec_bc));
        GMA_LAUNCH(KID_SCAN_JOIN, st,
                   launch_pdl(scan_chunk_join_kernel<T, S, false>, dim3((s.D * S + 127) / 128, s.B), dim3(128), 0, st, g));
    }
    if (g.chunks > 1)
        GMA_LAUNCH(KID_SCAN, st,
                   launch_pdl(scan_chunk_kernel<T, S, VEC, OUTPUT>, grid, dim3(per * 32), 2 * rows + ring, st, g, vec_bc));
    else
        GMA_LAUNCH(KID_SCAN, st, scan_chunk_kernel<T, S, VEC, OUTPUT><<<grid, per * 32, 2 * rows + ring, st>>>(g, vec_bc));
    return GMA_OK;
}

}  // namespace

// Worth it from six warps an SM on: with fewer, a warp's walk over its chunk takes as long as
// the whole call of the kernel that spreads a tile's tokens over lanes (512 tokens of 1024 channels: 33 us in
// three launches against 15 us).  That kernel walks over its tiles of 256 tokens one after another; a few channels over
// many thousand tokens are not measured on either side of the rule.
bool scan_chunked(const gma_scan_t &s)
{
    const long long warps = (long long)s.B * s.G * group_warps(s) * ((s.N + 31) / 32);
    return warps >= 152 * 6 && !(s.checkpoints && scan_spacing(s) < 32) && (s.N + 31) / 32 <= 65535 && (long long)s.D * s.S < (1ll << 31);
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
        if (s.S == 16) return vec ? run<T, 16, true>(s, (char *)ws, st) : run<T, 16, false>(s, (char *)ws, st);
        if (s.S == 32) return vec ? run<T, 32, true>(s, (char *)ws, st) : run<T, 32, false>(s, (char *)ws, st);
        return vec ? run<T, 64, true>(s, (char *)ws, st) : run<T, 64, false>(s, (char *)ws, st);
    };
    return s.dtype == GMA_BF16 ? with(__nv_bfloat16{}) : with(float{});
}

gma_status_t scan_chunk_adjoint(const gma_scan_grad_t &grad, float *state, float *total, cudaStream_t st)
{
    const gma_scan_t &s = grad.fwd;
    const bool vec = (s.D / s.G) % 8 == 0 && rows_vec(grad.dy, s.dtype) && rows_vec(s.dt, s.dtype) &&
                     (!s.z.ptr || rows_vec(s.z, s.dtype));
    auto with = [&](auto t) -> gma_status_t {
        using T = decltype(t);
#define GMA_ADJOINT(n) (vec ? run_adjoint<T, n, true>(grad, state, total, st) : run_adjoint<T, n, false>(grad, state, total, st))
        return s.S == 8 ? GMA_ADJOINT(8) : s.S == 16 ? GMA_ADJOINT(16) : s.S == 32 ? GMA_ADJOINT(32) : GMA_ADJOINT(64);
#undef GMA_ADJOINT
    };
    return s.dtype == GMA_BF16 ? with(__nv_bfloat16{}) : with(float{});
}

}  // namespace blk
}  // namespace gma
