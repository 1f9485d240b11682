// scan_tile.cuh -- the tile shared by the selective scan's forward and backward kernels.
//
// A block takes CH channels of one group in one batch row and walks over the sequence in tiles of
// TT = LT * TL tokens.  A warp's 32 lanes are CPW = 32 / LT channels times LT time lanes, each of which
// owns TL neighbouring tokens: the recurrence is sequential over a lane's own tokens, with a scan of
// (decay, state) pairs over the LT time lanes in between, so that a tile's exponentials are computed
// once and every warp has LT * CPW lanes of independent work whatever the number of channels.  States
// n and n + 1 share packed fp32 pairs.
//
// Tiles lie in shared memory in the order the lanes read them, 16 bytes a lane without bank conflicts:
// token t = tl * TL + 4 q + e of a channel at (q * LT + tl) * 4 + e, and of a pair of states (2 q + e)
// at (q * LT + tl) * 2 + e.
#pragma once

#include "block_common.cuh"

namespace gma {
namespace blk {

// Tokens between two checkpoints, and of a chunk of the backward pass: 64, or 16 where that leaves fewer than six
// warps an SM to walk over the chunks (2 x 301 x 384 channels: a walk over 64 tokens takes 33 us).
int scan_spacing(const gma_scan_t &s);

template <int LT_, int TL_, int WARPS_> struct Tile {
    static constexpr int LT = LT_, TL = TL_, WARPS = WARPS_;
    static constexpr int CPW = 32 / LT, CH = CPW * WARPS, TT = LT * TL, THREADS = 32 * WARPS;
    static constexpr int PITCH = TT + 4;                       // floats between two channels
    static constexpr int CHANNEL_FLOATS = CH * PITCH + CH / 8 * 16;
    static_assert(TL % 4 == 0 && CH % 8 == 0, "16-byte pieces");
    __host__ __device__ static constexpr int channel(int ch) { return ch * PITCH + ch / 8 * 16; }
    __device__ static __forceinline__ int pos(int t)
    {
        const int tl = t / TL, i = t % TL;
        return ((i / 4) * LT + tl) * 4 + i % 4;
    }
    __device__ static __forceinline__ int pos2(int t)
    {
        const int tl = t / TL, i = t % TL;
        return ((i / 2) * LT + tl) * 2 + i % 2;
    }
};

// One lane's TL values of a channel.
template <class K> __device__ __forceinline__ void lane_load(const float *chan, int tl, float (&v)[K::TL])
{
#pragma unroll
    for (int q = 0; q < K::TL / 4; ++q) {
        const float4 x = *reinterpret_cast<const float4 *>(chan + (q * K::LT + tl) * 4);
        v[4 * q] = x.x; v[4 * q + 1] = x.y; v[4 * q + 2] = x.z; v[4 * q + 3] = x.w;
    }
}
template <class K> __device__ __forceinline__ void lane_store(float *chan, int tl, const float (&v)[K::TL])
{
#pragma unroll
    for (int q = 0; q < K::TL / 4; ++q)
        *reinterpret_cast<float4 *>(chan + (q * K::LT + tl) * 4) =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
}

// One lane's TL values of a pair of states: two tokens of pair p.
template <class K> __device__ __forceinline__ void pair_load(const f2 *tile, int p, int tl, int q, f2 &v0, f2 &v1)
{
    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(tile + p * K::TT + (q * K::LT + tl) * 2);
    v0 = x.x; v1 = x.y;
}

// Stages tokens t0 .. t0 + TT - 1 of b or c (S values a token) as pairs; zeros behind the last token.
template <class K, typename T, bool VEC>
__device__ __forceinline__ void stage_pairs(const Rows<const T> &r, int b, int first, int t0, int len, int S, f2 *tile)
{
    const int pieces = S / 8;
    for (int i = threadIdx.x; i < K::TT * pieces; i += K::THREADS) {
        const int t = i % K::TT, piece = i / K::TT;
        float v[8];
        if (t0 + t < len) {
            load8<VEC>(r.at(b, t0 + t) + first + piece * 8, 8, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.f;
        }
        const int at = K::pos2(t);
#pragma unroll
        for (int k = 0; k < 4; ++k) tile[(piece * 4 + k) * K::TT + at] = pack2(v[2 * k], v[2 * k + 1]);
    }
}

// One step of a scan over lanes in groups of LT: takes (decay, state) of the lane `OFF` before (or
// behind), and where there is one, state += decay s and decay *= d.  The shuffle's own predicate tells.
template <int LT, int OFF, bool UP> __device__ __forceinline__ void scan_step(f2 &decay, f2 &state)
{
    constexpr int CLAMP = ((32 - LT) << 8) | (UP ? 0 : 31);
#define GMA_SCAN_STEP(MODE)                                                                        \
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 a, b, c, e;\n\t.reg .b64 d, s;\n\t"                 \
                 "mov.b64 {a, b}, %1;\n\tmov.b64 {c, e}, %0;\n\t"                                 \
                 "shfl.sync." MODE ".b32 a|p, a, %2, %3, 0xffffffff;\n\t"                          \
                 "shfl.sync." MODE ".b32 b, b, %2, %3, 0xffffffff;\n\t"                            \
                 "shfl.sync." MODE ".b32 c, c, %2, %3, 0xffffffff;\n\t"                            \
                 "shfl.sync." MODE ".b32 e, e, %2, %3, 0xffffffff;\n\t"                            \
                 "mov.b64 d, {a, b};\n\tmov.b64 s, {c, e};\n\t"                                   \
                 "@p fma.rn.f32x2 %0, %1, s, %0;\n\t@p mul.rn.f32x2 %1, %1, d;\n\t}"              \
                 : "+l"(state), "+l"(decay)                                                        \
                 : "n"(OFF), "n"(CLAMP))
    if (UP) GMA_SCAN_STEP("up");
    else GMA_SCAN_STEP("down");
#undef GMA_SCAN_STEP
}

// Inclusive scan over the time lanes, from the first one up or from the last one down.
template <int LT, bool UP> __device__ __forceinline__ void scan_lanes(f2 &decay, f2 &state)
{
    if (LT > 1) scan_step<LT, 1, UP>(decay, state);
    if (LT > 2) scan_step<LT, 2, UP>(decay, state);
    if (LT > 4) scan_step<LT, 4, UP>(decay, state);
    if (LT > 8) scan_step<LT, 8, UP>(decay, state);
    if (LT > 16) scan_step<LT, 16, UP>(decay, state);
}

template <typename T> struct ScanArgs {
    int B, N, D, S, G, tiles;      // tiles: blocks of CH channels per group
    Rows<const T> u, dt, z, b, c;
    const float *a_log, *d_skip, *dt_bias, *state_in;
    float *state_out;
    const int *lengths;
    Rows<T> y;
    float *ckpt;
    int spacing;                   // tokens between two checkpoints
    bool zero;                     // zeros behind a sequence's last token
};

template <typename T> inline ScanArgs<T> scan_args(const gma_scan_t &s)
{
    ScanArgs<T> a;
    a.B = s.B; a.N = s.N; a.D = s.D; a.S = s.S; a.G = s.G; a.tiles = 0;
    a.u = rows_of<const T>(s.u); a.dt = rows_of<const T>(s.dt); a.z = rows_of<const T>(s.z);
    a.b = rows_of<const T>(s.b); a.c = rows_of<const T>(s.c);
    a.a_log = s.a_log; a.d_skip = s.d_skip; a.dt_bias = s.dt_bias;
    a.state_in = s.state_in; a.state_out = s.state_out; a.lengths = s.lengths;
    a.y = rows_of<T>(s.y);
    a.ckpt = s.checkpoints;
    a.spacing = scan_spacing(s);
    a.zero = s.flags & GMA_ROWS_ZERO_TAIL;
    return a;
}

// Lets a kernel have the dynamic shared memory of a launch that wants `need` bytes (its static part is none).  The
// limit belongs to the kernel and is set to `most`, what the largest of its launches takes, by every call that needs
// more than the default: two host threads that each set their own call's would undo each other's.
template <typename... P> inline bool allow_smem(void (*kern)(P...), size_t need, size_t most)
{
    return need <= 48 * 1024 || cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) == cudaSuccess;
}
constexpr int MAX_S = 64;

// What every scan call needs; `out`: y is written.
gma_status_t scan_check(const gma_scan_t *s, bool out);
// 16-byte accesses to the rows of u, dt, z, b and c.
bool scan_vec(const gma_scan_t &s);

// The forward pass in chunks of tokens: whether it takes this call, its workspace, the call.
bool scan_chunked(const gma_scan_t &s);
size_t scan_chunk_workspace(const gma_scan_t &s);
gma_status_t scan_chunk_forward(const gma_scan_t &s, void *ws, cudaStream_t st);
// The adjoint behind every chunk of scan_spacing() tokens, state [B][chunks][D][S] (zeros behind a sequence's end), and
// dstate_in; total [B][chunks][D] is scratch.
gma_status_t scan_chunk_adjoint(const gma_scan_grad_t &grad, float *state, float *total, cudaStream_t st);

}  // namespace blk
}  // namespace gma
