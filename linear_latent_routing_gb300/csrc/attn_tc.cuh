// attn_tc.cuh -- what the tensor-core attention kernels share: operand tiles of 128 rows in shared memory, their TMA loads and
// descriptors, and rows of tensor memory.
//
// A tile is 128 rows of up to 128 bf16 elements: one or two boxes of 64 columns (128 bytes a row, 128-byte swizzle), 16 KB
// each, columns behind the width and rows behind the tensor zero.  The same tile serves as a K-major operand (products over the
// width) and as an MN-major one (products over the rows).
#pragma once

#include <cuda.h>

#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace gma {
namespace att {

using namespace tc;
typedef __nv_bfloat16 bf16;

constexpr int TILE = 128;
constexpr uint32_t BOX = TILE * 128;          // bytes of 64 columns of a tile
constexpr uint32_t SMEM_MAX = 232448;         // 227 KB

// Descriptors of a tile as a K-major operand and as an MN-major one, and what one k-step (16 columns, 16 rows) adds to them: the
// address field counts 16 bytes, and tiles lie below 256 KB, so that a plain sum stays in it.
__device__ __forceinline__ uint64_t k_desc(uint32_t tile) { return smem_desc(tile, 16, 1024, SW_128B); }
__device__ __forceinline__ uint64_t mn_desc(uint32_t tile) { return smem_desc(tile, BOX, 1024, SW_128B); }
constexpr __host__ __device__ uint32_t k_step(int s) { return ((uint32_t)(s >> 2) * BOX + (uint32_t)(s & 3) * 32u) >> 4; }
constexpr __host__ __device__ uint32_t mn_step(int s) { return (uint32_t)(s * 16 * 128) >> 4; }

// A first operand in tensor memory, k-step s: each half of its columns lies at the first ones of its half.
__device__ __forceinline__ uint32_t half_col(int s) { return (uint32_t)(8 * s + (s >= 4 ? 32 : 0)); }

// D = A B^T over `steps` k-steps of two K-major tiles.
__device__ __forceinline__ void mma_tiles(uint32_t d, uint64_t a, uint64_t b, uint32_t id, int steps)
{
#pragma unroll
    for (int s = 0; s < TILE / 16; ++s)
        if (s < steps) mma_f16(d, a + k_step(s), b + k_step(s), id, s > 0);
}

// A place in a ring of tiles, and the parity of its turn.
struct RingPos {
    int s;
    uint32_t turn;
    __device__ __forceinline__ void step(int n, int slots)      // n <= slots
    {
        s += n;
        if (s >= slots) {
            s -= slots;
            turn ^= 1u;
        }
    }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)map) : "memory");
}

// One lane of a converged warp, the same one every time.  Where it issues the products the compiler knows that one thread does, and
// their operands stay in uniform registers.
__device__ __forceinline__ bool elect()
{
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

// Whole warps wait, and get one answer: every lane sees a barrier for itself, at a time of its own, and what follows (an elected lane's products,
// shuffles, tensor memory) wants all of them on the same path.
__device__ __forceinline__ bool bar_there(uint64_t *bar, uint32_t parity) { return __all_sync(~0u, mbar_test_wait(bar, parity)); }
__device__ __forceinline__ bool aborted(volatile int *abort) { return __any_sync(~0u, *abort != 0); }

// mbar_wait_abortable with a try that comes first and without the clock: most waits here are short or over, several of them a tile.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, WsHeader *hdr, unsigned where, volatile int *abort)
{
    if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(~0u, mbar_try_wait(bar, parity))) {
        if (aborted(abort)) return false;
        if (__any_sync(~0u, wait_expired(clock64() - t0, hdr))) {
            record_error(hdr, GMA_ERR_TIMEOUT, where);
            *abort = 1;
            return false;
        }
    }
    return true;
}

// The same for each lane by itself: for code that takes no branch by the answer before its lanes meet again.
__device__ __forceinline__ bool lane_wait(uint64_t *bar, uint32_t parity, WsHeader *hdr, unsigned where, volatile int *abort)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (wait_expired(clock64() - t0, hdr)) {
            record_error(hdr, GMA_ERR_TIMEOUT, where);
            *abort = 1;
            return false;
        }
    }
    return true;
}

// Zeros in rows `from` to 127 of a tile's boxes, by one warp; the tensor cores see them after the fence.
__device__ __forceinline__ void zero_rows(uint8_t *tile, int boxes, int from)
{
    const int lane = threadIdx.x & 31;
    for (int b = 0; b < boxes; ++b)
        for (int i = from * 8 + lane; i < TILE * 8; i += 32)
            *reinterpret_cast<uint4 *>(tile + b * BOX + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Columns [0, width) of this warp's lanes at `tl`, times f, as a row of bf16 (one row a thread; `valid`: it is there).
__device__ __forceinline__ void store_row(uint32_t tl, int width, float f, bool valid, bf16 *row, bool vec)
{
#pragma unroll 1
    for (int c = 0; c < width; c += 32) {
        uint32_t r[32];
        tmem_ld32(tl + c, r);
        tmem_ld_wait();
        if (!valid) continue;
        if (vec) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (c + 8 * q < width) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack_bf16(__uint_as_float(r[8 * q + 2 * e]) * f, __uint_as_float(r[8 * q + 2 * e + 1]) * f);
                    *reinterpret_cast<uint4 *>(row + c + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
                }
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (c + e < width) row[c + e] = __float2bfloat16_rn(__uint_as_float(r[e]) * f);
        }
    }
}

// The same without a factor as a row of fp32, columns up to the next multiple of four.
__device__ __forceinline__ void store_row_f32(uint32_t tl, int width, bool valid, float *row)
{
#pragma unroll 1
    for (int c = 0; c < width; c += 32) {
        uint32_t r[32];
        tmem_ld32(tl + c, r);
        tmem_ld_wait();
        if (!valid) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (c + 4 * q < width) *reinterpret_cast<uint4 *>(row + c + 4 * q) = make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
    }
}

// ------------------------------------------------------------------ host side
// Whether TMA can read these heads: bf16, 16-byte aligned strides that step.
bool tma_heads(const gma_heads_t &r, long long B, long long N, long long heads);
// Boxes of 64 columns x bh heads x bt tokens.
bool heads_map(CUtensorMap *m, const gma_heads_t &r, long long B, long long N, long long heads, int width, int bh, int bt);
// Whether rows of `width` can be stored 16 bytes at a time.
bool store_vec(const gma_heads_t &r, int width);

}  // namespace att
}  // namespace gma
