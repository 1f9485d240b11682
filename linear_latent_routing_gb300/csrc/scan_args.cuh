// scan_args.cuh -- what the selective scan's translation units share: a call's arguments as the kernels take them,
// its checks, and the passes in chunks of tokens, which the forward and the backward call use.
#pragma once

#include "block_common.cuh"

namespace gma {
namespace blk {

// Tokens between two checkpoints, and of a chunk of the backward pass: 64, or 16 where that leaves fewer than six
// warps an SM to walk over the chunks (2 x 301 x 384 channels: a walk over 64 tokens takes 33 us).
int scan_spacing(const gma_scan_t &s);

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
