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

// Zeros in the rows of [rows][heads * width] that belong to no sequence, by warp `first` of `warps` (64 bits: a grid may have 2^31 blocks);
// `vec`: 16 bytes at a time.
template <typename T>
__device__ __forceinline__ void zero_dead_rows(const Geo &g, const Heads<T> &x, int heads, int width, int rows, long long first, long long warps,
                                               bool vec)
{
    constexpr int E = 16 / sizeof(T);
    const int lane = threadIdx.x & 31, a = g.offsets ? max(g.offsets[0], 0) : 0, e = g.offsets ? g.offsets[g.B] : 0;
    const int step = vec ? E : 1, each = width / step, all = heads * each;
    for (long long at_row = first; at_row < rows; at_row += warps) {
        const int r = (int)at_row;
        int b = 0, i = r;
        if (g.offsets) {
            if (r >= a && r < e) continue;
        } else {
            b = r / g.N;
            i = r - b * g.N;
            if (i < blk::row_length(g.lengths, b, g.N)) continue;
        }
        for (int c = lane; c < all; c += 32) {
            const int h = c / each;
            T *at = x.at(b, i, h) + (c - h * each) * step;
            if (vec) *reinterpret_cast<uint4 *>(at) = make_uint4(0, 0, 0, 0);
            else *at = from_f32<T>(0.f);
        }
    }
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
// so that the last ones to start are short.  Tiles are narrow ones where wide ones would leave SMs without work; over a cache,
// where few rows may face many keys, items are cut into parts, which a last launch joins.
struct Item {
    int seq, tok0;     // sequence, first token of the tile
    int t0, t1;        // key tiles
    int slot, parts;   // first slot of the parts' results, how many parts (1: no slot)
    int part, pad;     // this part
    Seq sq;            // the sequence: one access less between a block's start and its first tile
    int pad2[3];
};

static_assert(sizeof(Item) == 64, "four 16-byte accesses");
// (past the first-level cache, whose lines may be older than the launch that this one overlaps with)
__device__ __forceinline__ Item load_item(const Item *at)
{
    union {
        uint4 q[4];
        Item it;
    } u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u.q[i] = __ldcg(reinterpret_cast<const uint4 *>(at) + i);
    return u.it;
}

struct Join {          // an item that was cut
    int slot, parts;   // its parts' results
    int b, row, tokens; // batch row, first row and tokens of the tile
    int pad[3];
};

struct PlanHead {      // behind the workspace header
    int items;         // how many
    int tokens;        // tokens of a tile
    int ticket;        // of the next item, where blocks take them one after another
    int joins;         // items that were cut
    int pad[60];
};

struct Plan {          // host side: sizes and places in the workspace
    int pack, heads;           // query heads in a row tile, tiles' heads (grid: items * heads)
    int wide, narrow;          // tokens of a wide and of a narrow tile
    int key_shift;             // log2 of the keys of a key tile
    int blocks;                // that run at a time
    int max_items, max_slots;  // of the list, and of the parts' results a head (0: items are not cut)
    int rows;                  // rows of a part's results
    bool withhold;             // GMA_FLAG_TEST_WITHHOLD
    bool by_keys;              // items are tiles of keys, their cost the query tiles that see them (backward pass)
    size_t head_at, items_at, join_at, part_at, stat_at;
};

struct PlanArgs {
    Geo g;
    int wide, narrow, key_shift, blocks, heads, max_items, max_slots, by_keys;
    float part_cost;           // what a part costs beside its keys, in key tiles
    WsHeader *hdr;
    PlanHead *head;
    Item *items;
    Join *join;                // the items that were cut
    int short_waits;           // GMA_FLAG_TEST_WITHHOLD
};

Plan make_plan(const gma_attn_t &a, int pack, int wide_rows, int narrow_rows, int key_shift, int blocks, bool cut, Carve *ws);
PlanArgs plan_args(const Geo &g, const Plan &p, void *ws);
gma_status_t launch_plan(const PlanArgs &a, const PlanArgs *second, cudaStream_t st);

// ------------------------------------------------------------------ the parts of an item
// Part results: unnormalised sums over the part's keys relative to its maximum, [slot][head][rows][pitch] (dv rounded up to
// four), and per row the maximum (in units of the exponent of two; -inf: no key seen) and the sum, [slot][head][rows][2].
struct Parts {
    float *o, *stat;
    int rows, heads, dv, pitch;
    __device__ __forceinline__ float *o_at(int slot, int head, int row) const
    {
        return o + (((long long)slot * heads + head) * rows + row) * pitch;
    }
    __device__ __forceinline__ float *stat_at(int slot, int head, int row) const
    {
        return stat + (((long long)slot * heads + head) * rows + row) * 2;
    }
};

inline Parts parts_of(const Plan &p, const gma_attn_t &a, void *ws)
{
    return Parts{(float *)((char *)ws + p.part_at), (float *)((char *)ws + p.stat_at), p.rows, p.heads, a.dv, (a.dv + 3) & ~3};
}

// Adds up the parts of the items that the plan cut, in their order.
gma_status_t launch_join(const gma_attn_t &a, const Geo &g, const Plan &p, void *ws, cudaStream_t st);

// ------------------------------------------------------------------ the pieces of a group
// dk and dv of a head sum over its group's query heads.  Where that leaves SMs without work the group is cut into pieces, a block each, whose
// fp32 sums [piece][head][row][pitch] a last launch adds up in their order.
struct Pieces {
    int count;                  // 1: dk and dv are written at once
    float *k, *v;
    int k_pitch, v_pitch, heads;
    long long rows;
    __device__ __forceinline__ long long at(int piece, int head, long long row) const { return ((long long)piece * heads + head) * rows + row; }
    __device__ __forceinline__ float *k_at(int piece, int head, long long row) const { return k + at(piece, head, row) * k_pitch; }
    __device__ __forceinline__ float *v_at(int piece, int head, long long row) const { return v + at(piece, head, row) * v_pitch; }
};

struct PiecePlan {
    int count;
    size_t k_at, v_at;
};

// For tiles of so many keys that walk over rows by steps of so many, each of so many us.
PiecePlan plan_pieces(const gma_attn_t &a, int tile, int step, double step_us, Carve *ws);
Pieces pieces_of(const PiecePlan &p, const gma_attn_t &a, void *ws);
gma_status_t launch_pieces(const gma_attn_grad_t &g, const Pieces &p, cudaStream_t st);

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
