// attn_common.cuh -- what the softmax attention kernels behind gma_block.h share: heads with strides, the rows and
// keys of a sequence, the plan that cuts a call into work items, and the join of an item's parts.
#pragma once

#include <math.h>

#include "block_common.cuh"

namespace gma {
namespace att {

using blk::ex2;
using blk::LOG2E;
constexpr float LN2 = 0.6931471805599453f;
constexpr int SMS = 152;

// ------------------------------------------------------------------ tensors
template <typename T> struct Heads {
    T *p;
    long long sb, st, sh;   // element strides between batch rows, tokens and heads
    __device__ __forceinline__ T *at(long long b, long long t, int h) const { return p + b * sb + t * st + h * sh; }
};

template <typename T> inline Heads<T> heads_of(const gma_heads_t &r)
{
    return Heads<T>{(T *)r.ptr, (long long)r.batch, (long long)r.token, (long long)r.head};
}

// ------------------------------------------------------------------ sequences
struct Geo {
    int B, N, H, G, group, d, dv;
    int causal;
    float sl2;                     // scale * log2(e): scores in units of the exponent of two
    float scale;
    const int *lengths, *offsets;  // of the query rows
    // paged: the cache
    const int *cached, *table;     // null: the keys are the sequence's own rows
    long long table_stride;
    int table_pages, page, pages;
};

struct Seq {
    int b;             // batch row of the tensors (packed: 0)
    int row0;          // first row in it
    int n;             // query rows
    int L;             // keys
    int pos0;          // token of the first query row (negative: it comes before the first key)
    // keys that query row i sees: the first so many
    __device__ __forceinline__ int seen(const Geo &g, int i) const
    {
        return g.causal ? min(max(pos0 + i + 1, 0), L) : L;
    }
};

__device__ __forceinline__ Seq sequence(const Geo &g, int s)
{
    Seq q;
    if (g.offsets) {
        const int a = min(max(g.offsets[s], 0), g.N), e = min(max(g.offsets[s + 1], 0), g.N);
        q.b = 0; q.row0 = a; q.n = max(e - a, 0);
    } else {
        q.b = s; q.row0 = 0; q.n = blk::row_length(g.lengths, s, g.N);
    }
    if (g.cached) {
        q.L = (int)min((long long)max(g.cached[s], 0), (long long)g.table_pages * g.page);
        q.pos0 = q.L - q.n;
    } else {
        q.L = q.n;
        q.pos0 = 0;
    }
    return q;
}

// Where lse and the like of (row of the tensors, head) lie: [B][H][N], packed [H][N].
__device__ __forceinline__ long long stat_at(const Geo &g, const Seq &q, int h, int i)
{
    return ((long long)q.b * g.H + h) * g.N + q.row0 + i;
}

// The page and slot of key j of sequence s; the page is -1 where the table names none of the cache's.
__device__ __forceinline__ int page_of(const Geo &g, int s, int j, int *slot)
{
    const int at = j / g.page;
    *slot = j - at * g.page;
    const int p = g.table[(long long)s * g.table_stride + at];
    return p >= 0 && p < g.pages ? p : -1;
}

// ------------------------------------------------------------------ the plan
// A launch of one block cuts a call into items: a tile of query rows of one sequence (all heads alike) and a range of
// key tiles.  A row of the tile is a (token, head of a group of `pack`) pair, tokens outer.  Items come largest first,
// so that the last ones to start are short.  Tiles are narrow ones where wide ones would leave SMs without work, and
// items whose keys are more than an SM's share of the call are cut, their parts joined by the last one to finish.
struct Item {
    int seq, tok0;     // sequence, first token of the tile
    int t0, t1;        // key tiles
    int slot, parts;   // first slot of the parts' results, how many parts (1: no slot)
    int part, join;    // this part, counter of the parts that have finished
};

struct PlanHead {      // behind the workspace header
    int items;         // how many
    int tokens;        // tokens of a tile
    int pad[62];
};

constexpr int NEVER = 1 << 30;

struct Plan {          // host side: sizes and places in the workspace
    int pack, heads;           // query heads in a row tile, tiles' heads (grid: items * heads)
    int wide, narrow;          // tokens of a wide and of a narrow tile
    int key_shift;             // log2 of the keys of a key tile
    int blocks;                // that run at a time
    int least, fine;           // key tiles of a part, at least; of a block's share from which a part is half of it (0: no parts)
    int max_items, max_slots;  // of the list, and of the parts' results a head
    int rows;                  // rows of a part's results
    bool by_keys;              // items are tiles of keys, their cost the query tiles that see them (backward pass)
    size_t head_at, items_at, join_at, part_at, stat_at;
};

struct PlanArgs {
    Geo g;
    int wide, narrow, key_shift, blocks, least, fine, heads, max_items, max_slots, by_keys;
    WsHeader *hdr;
    PlanHead *head;
    Item *items;
    int *join;
};

Plan make_plan(const gma_attn_t &a, int pack, int wide_rows, int narrow_rows, int key_shift, int blocks, int least, int fine, Carve *ws);
PlanArgs plan_args(const Geo &g, const Plan &p, void *ws);
gma_status_t launch_plan(const PlanArgs &a, const PlanArgs *second, cudaStream_t st);

// ------------------------------------------------------------------ joining the parts of an item
// Part results: unnormalised sums over the part's keys relative to its maximum, [slot][head][rows][pitch] (dv rounded up to
// four), and per row the maximum (in units of the exponent of two; -inf: no key seen) and the sum, [slot][head][rows][2].
struct Parts {
    float *o, *stat;
    int rows, heads, dv, pitch;
    int *join;
    __device__ __forceinline__ float *o_at(int slot, int head, int row) const
    {
        return o + (((long long)slot * heads + head) * rows + row) * pitch;
    }
    __device__ __forceinline__ float *stat_at(int slot, int head, int row) const
    {
        return stat + (((long long)slot * heads + head) * rows + row) * 2;
    }
};

// Called by all threads of a block once its part lies in its slot: whether this block is the last of its item's.  The
// parts are then added in their order, whoever adds them.
__device__ __forceinline__ bool last_part(const Parts &p, const Item &it, int head, int *flag)
{
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) *flag = atomicAdd(p.join + (long long)it.join * p.heads + head, 1) == it.parts - 1;
    __syncthreads();
    const bool last = *flag != 0;
    if (last) __threadfence();
    return last;
}

// One warp's row of a joined item: lanes are parts for the weights, then four columns each for the sums, with the loads of sixteen parts
// in flight.
template <typename T>
__device__ __forceinline__ void join_row(const Parts &p, const Item &it, int head, int row, T *o, float *lse)
{
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int k = lane; k < it.parts; k += 32) m = fmaxf(m, __ldcg(p.stat_at(it.slot + k, head, row)));
#pragma unroll
    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, s));
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool mine = 4 * lane < p.dv;
    for (int k0 = 0; m != -INFINITY && k0 < it.parts; k0 += 32) {
        float w = 0.f;
        if (k0 + lane < it.parts) {
            const float2 s = __ldcg(reinterpret_cast<const float2 *>(p.stat_at(it.slot + k0 + lane, head, row)));
            w = ex2(s.x - m);
            l = fmaf(w, s.y, l);
        }
        const int n = min(32, it.parts - k0);
        for (int j0 = 0; j0 < n; j0 += 16) {
            float4 x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (mine && j0 + j < n) x[j] = __ldcg(reinterpret_cast<const float4 *>(p.o_at(it.slot + k0 + j0 + j, head, row)) + lane);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float f = __shfl_sync(~0u, w, j0 + j);
                if (f == 0.f || j0 + j >= n) continue;      // a part that saw nothing wrote no sums
                acc.x = fmaf(f, x[j].x, acc.x);
                acc.y = fmaf(f, x[j].y, acc.y);
                acc.z = fmaf(f, x[j].z, acc.z);
                acc.w = fmaf(f, x[j].w, acc.w);
            }
        }
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(~0u, l, s);
    const float inv = l > 0.f ? 1.f / l : 0.f, y[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (4 * lane + c < p.dv) o[4 * lane + c] = from_f32<T>(y[c] * inv);
    if (lse && lane == 0) *lse = l > 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
}

// ------------------------------------------------------------------ kernels
Geo geo_of(const gma_attn_t &a, const gma_attn_paged_t *paged);

// CUDA-core kernels, any type, stride and page.
size_t simt_workspace(const gma_attn_t &a, const gma_attn_paged_t *paged);
gma_status_t simt_forward(const gma_attn_t &a, const gma_attn_paged_t *paged, void *ws, cudaStream_t st);
size_t simt_backward_workspace(const gma_attn_grad_t &g);
gma_status_t simt_backward(const gma_attn_grad_t &g, void *ws, cudaStream_t st);

// delta = do . o of every row, in lse's layout.
gma_status_t launch_delta(const gma_attn_grad_t &g, float *delta, cudaStream_t st);

}  // namespace att
}  // namespace gma
