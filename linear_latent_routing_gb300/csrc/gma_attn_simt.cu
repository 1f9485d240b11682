// gma_attn_simt.cu -- softmax attention on the CUDA cores: fp32, and bf16 rows or pages that the tensor-core kernels
// cannot read (strides off 16 bytes, pages of odd sizes).
//
// Forward: a block takes R rows ((token, head of a group) pairs where the keys come from a cache) and walks over its keys 64
// at a time, with the running maximum and sum of each row in registers.  Scores are R / 16 x 4 a thread out of shared memory, four
// elements of the head at a time (R = 64: 8 loads of 16 bytes for 64 multiply-adds).  The next tile's rows are on their way by cp.async
// while one is worked on.  Calls of less than two blocks of 64 rows an SM take R = 32, single tokens R = 16: latency, not the fp32 pipe,
// bounds them.  Warps whose rows do not exist only copy.
//
// Measured in fp32: 4 x 2048 tokens, 8 heads of 128, causal, 1.01 ms (34 TFLOP/s of the CUDA cores' 74) and 5.0 ms backward (17 by five products a
// pair; seven are made), heads of 64 0.60 and 2.87 ms; 64 single tokens over 8192 cached ones each, 16 heads of 128 over 4, 1.04 ms (2.07 TB/s: the two
// warps whose rows exist work for all); three sequences of up to 301 tokens, 6 heads of 40, 23 us a call with its two launches.  In bf16 the same single
// tokens with pages of 24 take 2.4 ms (0.45 TB/s: two bytes a load, none ahead), against 0.19 ms with pages of 128 on the tensor cores.
#include <algorithm>

#include "attn_common.cuh"

namespace gma {
namespace att {
namespace {

constexpr int BR = 32;                // rows of a tile of the backward pass
constexpr int KT = 64;                // keys of a tile
constexpr int TH = 256;

template <typename T> struct Args {
    Geo g;
    Heads<const T> q, k, v;            // paged: k and v are the pages (batch: page, token: slot)
    Heads<T> o;
    float *lse;
    int pack, heads;
    int zero_rows, o_vec;              // rows of o to be looked through for such as belong to no sequence (0: none)
    const PlanHead *head;
    const Item *items;
    Parts parts;
    // backward
    Heads<const T> d_o;
    Heads<T> dq, dk, dv;
    const float *stat_lse, *delta;
    Pieces pieces;
};

constexpr __host__ __device__ int pitch_of(int width) { return (width + 3) / 4 * 4 + 4; }

__device__ __forceinline__ void copy16(float *dst, const void *src, bool is)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(is ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One row of `width` elements into shared memory as fp32 by the four threads of it; zeros behind the width and where it `is` not.
// VEC: fp32 rows on 16-byte boundaries, copied asynchronously.
template <bool VEC, typename T> __device__ __forceinline__ void stage_row(float *dst, const T *src, bool is, int width, int quarter)
{
    if (VEC) {
        for (int c = 4 * quarter; c < width; c += 16) copy16(dst + c, src + (is ? c : 0), is);
    } else {
        const int w4 = (width + 3) & ~3;
        for (int c = quarter; c < w4; c += 4) dst[c] = is && c < width ? to_f32<T>(src[c]) : 0.f;
    }
}

// Scores of rows RI ty + i against columns tx + 16 j of two staged tiles.
template <int RI>
__device__ __forceinline__ void products(const float *a, const float *b, int pitch, int width, int tx, int ty, float (&s)[RI][4])
{
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 2
    for (int c = 0; c < width; c += 4) {
        float4 x[RI], y[4];
#pragma unroll
        for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4 *>(a + (RI * ty + i) * pitch + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * pitch + c);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
    }
}

// acc[i][4 c + e] += sum_k p[row RI ty + i][k] x[k][64 c + 4 tx + e], over 64 k.
template <int RI>
__device__ __forceinline__ void accumulate(const float *p, const float *x, int pitch, int width, int tx, int ty, float (&acc)[RI][8])
{
#pragma unroll 2
    for (int k = 0; k < KT; k += 4) {
        float4 w[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) w[i] = *reinterpret_cast<const float4 *>(p + (RI * ty + i) * (KT + 4) + k);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (64 * c + 4 * tx >= width) break;
            const float *y = x + k * pitch + 64 * c + 4 * tx;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v = *reinterpret_cast<const float4 *>(y + e * pitch);
#pragma unroll
                for (int i = 0; i < RI; ++i) {
                    const float f = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
                    acc[i][4 * c] = fmaf(f, v.x, acc[i][4 * c]);
                    acc[i][4 * c + 1] = fmaf(f, v.y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(f, v.z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(f, v.w, acc[i][4 * c + 3]);
                }
            }
        }
    }
}

template <typename T, bool PAGED, bool VEC, int R>
__global__ void __launch_bounds__(TH, 1) attn_simt_kernel(const Args<T> a)
{
    constexpr int RI = R / 16;
    extern __shared__ __align__(16) float smem[];
    // beside the plan (no other kernel's results are read or written here)
    if (a.zero_rows)
        zero_dead_rows(a.g, a.o, a.g.H, a.g.dv, a.zero_rows, blockIdx.x * (TH / 32ll) + (threadIdx.x >> 5), gridDim.x * (TH / 32ll), a.o_vec);
    blk::wait_previous();
    if (PAGED) blk::let_next();
    const int rank = blockIdx.x / a.heads, head = blockIdx.x % a.heads;
    const Geo &g = a.g;
    const Item it = load_item(a.items + rank);       // beside the number of items
    if (rank >= a.head->items || it.part < 0) return;
    const Seq s = it.sq;
    const int pack = a.pack, kvh = pack == 1 ? head / g.group : head;
    const int tokens = min(a.head->tokens, s.n - it.tok0), rows = tokens * pack;
    const int qp = pitch_of(g.d), vp = pitch_of(g.dv);
    float *qs = smem, *ps = qs + R * qp, *ring = ps + R * (KT + 4);      // two stages of a tile of keys and one of values
    const int stage = KT * (qp + vp);
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4, mine = t >> 2, quarter = t & 3;
    // row r of the tile: token it.tok0 + r / pack, query head
    auto head_of = [&](int r) { return pack == 1 ? head : head * pack + r % pack; };
    const int end = min(it.t1 * KT, s.seen(g, it.tok0 + tokens - 1));
    // the page of this thread's row of a tile, fetched a tile ahead of the copy that needs it
    int slot = 0;
    auto page = [&](int k0) { return PAGED && k0 + mine < end ? page_of(g, it.seq, k0 + mine, &slot) : -1; };
    auto load = [&](int k0, int at, int p) {
        const bool is = k0 + mine < end && (!PAGED || p >= 0);
        const T *k, *v;
        if (PAGED) {
            k = a.k.at(is ? p : 0, is ? slot : 0, kvh);
            v = a.v.at(is ? p : 0, is ? slot : 0, kvh);
        } else {
            const long long row = s.row0 + (is ? k0 + mine : 0);
            k = a.k.at(s.b, row, kvh);
            v = a.v.at(s.b, row, kvh);
        }
        stage_row<VEC>(ring + at * stage + mine * qp, k, is, g.d, quarter);
        stage_row<VEC>(ring + at * stage + KT * qp + mine * vp, v, is, g.dv, quarter);
    };
    int k0 = it.t0 * KT, p = page(k0);
    if (mine < R) {
        const bool is = mine < rows;
        const int r = is ? mine : 0;
        stage_row<VEC>(qs + mine * qp, a.q.at(s.b, s.row0 + it.tok0 + r / pack, head_of(r)), is, g.d, quarter);
    }
    if (k0 < end) load(k0, 0, p);
    copies_commit();
    p = page(k0 + KT);
    int seen[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) seen[i] = RI * ty + i < rows ? s.seen(g, it.tok0 + (RI * ty + i) / pack) : 0;
    const bool busy = (t >> 5) * 2 * RI < rows;       // this warp's rows exist
    float m[RI], l[RI], acc[RI][8];
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
    }
    for (int at = 0; k0 < end; k0 += KT, at ^= 1) {
        if (k0 + KT < end) load(k0 + KT, at ^ 1, p);
        copies_commit();
        p = page(k0 + 2 * KT);
        copies_wait<1>();
        __syncthreads();
        if (busy) {
            const float *ks = ring + at * stage, *vs = ks + KT * qp;
            float x[RI][4];
            products<RI>(qs, ks, qp, g.d, tx, ty, x);
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = k0 + tx + 16 * j < seen[i] ? x[i][j] * g.sl2 : -INFINITY;
                    top = fmaxf(top, x[i][j]);
                }
#pragma unroll
                for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                const float now = fmaxf(m[i], top), base = now == -INFINITY ? 0.f : now, f = ex2(m[i] - base);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = ex2(x[i][j] - base);
                    sum += e;
                    ps[(RI * ty + i) * (KT + 4) + tx + 16 * j] = e;
                }
                l[i] = l[i] * f + sum;               // this thread's keys; the row's threads are added at the end
                m[i] = now;
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[i][c] *= f;
            }
            __syncwarp();                            // a warp reads the rows that it wrote
            accumulate<RI>(ps, vs, vp, g.dv, tx, ty, acc);
        }
        __syncthreads();
    }
    copies_wait<0>();
    const bool whole = it.parts == 1;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
#pragma unroll
        for (int o = 8; o; o >>= 1) l[i] += __shfl_xor_sync(~0u, l[i], o);
        const int r = RI * ty + i;
        if (r >= rows) continue;
        const int h = head_of(r), tok = it.tok0 + r / pack;
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        T *o = a.o.at(s.b, s.row0 + tok, h);
        float *part = whole ? nullptr : a.parts.o_at(it.slot + it.part, head, r);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int col = 64 * (c >> 2) + 4 * tx + (c & 3);
            if (col >= g.dv) continue;
            if (whole) o[col] = from_f32<T>(acc[i][c] * inv);
            else part[col] = acc[i][c];
        }
        if (tx) continue;
        if (whole) {
            if (a.lse) a.lse[stat_at(g, s, h, tok)] = l[i] > 0.f ? (m[i] + log2f(l[i])) * LN2 : -INFINITY;
        } else {
            float *st = a.parts.stat_at(it.slot + it.part, head, r);
            st[0] = m[i];
            st[1] = l[i];
        }
    }
}

// dq of 32 query rows of one head: ds = p (do . v - delta), dq = scale ds k over the keys that the rows see.
template <typename T, bool VEC> __global__ void __launch_bounds__(TH, 1) attn_simt_dq_kernel(const Args<T> a)
{
    constexpr int RI = BR / 16;
    extern __shared__ __align__(16) float smem[];
    // (the blocks before read the same results, and had waited for them when they let this kernel start; its last block waits for theirs)
    if (blockIdx.x == gridDim.x - 1) blk::wait_previous();
    const int rank = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
    const Geo &g = a.g;
    const Item it = load_item(a.items + rank);
    if (rank >= __ldcg(&a.head->items)) return;
    const Seq s = it.sq;
    const int kvh = h / g.group, rows = min(BR, s.n - it.tok0);
    const int qp = pitch_of(g.d), vp = pitch_of(g.dv), stage = KT * (qp + vp);
    float *qs = smem, *os = qs + BR * qp, *ps = os + BR * vp, *ring = ps + BR * (KT + 4);
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4, mine = t >> 2, quarter = t & 3;
    const int end = min(it.t1 * KT, s.L);
    auto load = [&](int k0, int at) {
        const bool is = k0 + mine < end;
        const long long row = s.row0 + (is ? k0 + mine : 0);
        stage_row<VEC>(ring + at * stage + mine * qp, a.k.at(s.b, row, kvh), is, g.d, quarter);
        stage_row<VEC>(ring + at * stage + KT * qp + mine * vp, a.v.at(s.b, row, kvh), is, g.dv, quarter);
    };
    if (mine < BR) {
        const bool is = mine < rows;
        const long long row = s.row0 + it.tok0 + (is ? mine : 0);
        stage_row<VEC>(qs + mine * qp, a.q.at(s.b, row, h), is, g.d, quarter);
        stage_row<VEC>(os + mine * vp, a.d_o.at(s.b, row, h), is, g.dv, quarter);
    }
    int k0 = it.t0 * KT;
    load(k0, 0);
    copies_commit();
    float lse2[RI], delta[RI], acc[RI][8];
    int seen[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const int r = RI * ty + i;
        const bool is = r < rows;
        const long long at = is ? stat_at(g, s, h, it.tok0 + r) : 0;
        seen[i] = is ? s.seen(g, it.tok0 + r) : 0;
        lse2[i] = is ? __ldcg(a.stat_lse + at) * LOG2E : 0.f;
        delta[i] = is ? __ldcg(a.delta + at) : 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
    }
    for (int at = 0; k0 < end; k0 += KT, at ^= 1) {
        if (k0 + KT < end) load(k0 + KT, at ^ 1);
        copies_commit();
        copies_wait<1>();
        __syncthreads();
        const float *ks = ring + at * stage, *vs = ks + KT * qp;
        float x[RI][4], y[RI][4];
        products<RI>(qs, ks, qp, g.d, tx, ty, x);
        products<RI>(os, vs, vp, g.dv, tx, ty, y);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = k0 + tx + 16 * j < seen[i] ? ex2(x[i][j] * g.sl2 - lse2[i]) : 0.f;
                ps[(RI * ty + i) * (KT + 4) + tx + 16 * j] = p == 0.f ? 0.f : p * (y[i][j] - delta[i]);
            }
        __syncwarp();
        accumulate<RI>(ps, ks, qp, g.d, tx, ty, acc);
        __syncthreads();
    }
    copies_wait<0>();
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        if (RI * ty + i >= rows) continue;
        T *dq = a.dq.at(s.b, s.row0 + it.tok0 + RI * ty + i, h);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int col = 64 * (c >> 2) + 4 * tx + (c & 3);
            if (col < g.d) dq[col] = from_f32<T>(acc[i][c] * g.scale);
        }
    }
}

// dk and dv of 32 keys of one head, over the query heads of its group (or of a piece of it) and the rows that see them: rows of the
// tiles are keys here, columns queries.
template <typename T, bool VEC> __global__ void __launch_bounds__(TH, 1) attn_simt_dkv_kernel(const Args<T> a)
{
    constexpr int RI = BR / 16;
    extern __shared__ __align__(16) float smem[];
    __shared__ float lse2[2][KT], delta[2][KT];
    blk::wait_previous();
    blk::let_next();       // what this kernel reads, the next one reads too: dq's blocks take the SMs that these leave
    const int parts = a.pieces.count, rank = blockIdx.x / a.heads, at_head = blockIdx.x - rank * a.heads, kvh = at_head / parts, piece = at_head - kvh * parts;
    const Geo &g = a.g;
    const Item it = load_item(a.items + rank);
    if (rank >= a.head->items) return;
    const Seq s = it.sq;
    const int rows = min(BR, s.n - it.tok0);
    const int qp = pitch_of(g.d), vp = pitch_of(g.dv), stage = KT * (qp + vp);
    float *ks = smem, *vs = ks + BR * qp, *ps = vs + BR * vp, *ds = ps + BR * (KT + 4), *ring = ds + BR * (KT + 4);
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4, mine = t >> 2, quarter = t & 3;
    const int first = it.t0 * KT, last = min(it.t1 * KT, s.n);
    auto load = [&](int h, int q0, int at) {
        const bool is = q0 + mine < last;
        const long long row = s.row0 + (is ? q0 + mine : 0);
        stage_row<VEC>(ring + at * stage + mine * qp, a.q.at(s.b, row, h), is, g.d, quarter);
        stage_row<VEC>(ring + at * stage + KT * qp + mine * vp, a.d_o.at(s.b, row, h), is, g.dv, quarter);
        if (quarter == 0) {
            const long long where = is ? stat_at(g, s, h, q0 + mine) : 0;
            lse2[at][mine] = is ? a.stat_lse[where] * LOG2E : 0.f;
            delta[at][mine] = is ? a.delta[where] : 0.f;
        }
    };
    if (mine < BR) {
        const bool is = mine < rows;
        const long long row = s.row0 + it.tok0 + (is ? mine : 0);
        stage_row<VEC>(ks + mine * qp, a.k.at(s.b, row, kvh), is, g.d, quarter);
        stage_row<VEC>(vs + mine * vp, a.v.at(s.b, row, kvh), is, g.dv, quarter);
    }
    float dk[RI][8], dv[RI][8];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) dk[i][c] = dv[i][c] = 0.f;
    int h = kvh * g.group + piece * (g.group / parts), q0 = first;
    const int heads_end = h + g.group / parts;
    load(h, q0, 0);
    copies_commit();
    for (int at = 0; h < heads_end; at ^= 1) {
        int next_h = h, next = q0 + KT;
        if (next >= last) {
            next = first;
            ++next_h;
        }
        if (next_h < heads_end) load(next_h, next, at ^ 1);
        copies_commit();
        copies_wait<1>();
        __syncthreads();
        const float *qs = ring + at * stage, *os = qs + KT * qp;
        const int have = min(KT, last - q0);
        float x[RI][4], y[RI][4];
        products<RI>(ks, qs, qp, g.d, tx, ty, x);
        products<RI>(vs, os, vp, g.dv, tx, ty, y);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = tx + 16 * j, key = it.tok0 + RI * ty + i;
                const float p = c < have && key < s.seen(g, q0 + c) ? ex2(x[i][j] * g.sl2 - lse2[at][c]) : 0.f;
                ps[(RI * ty + i) * (KT + 4) + c] = p;
                ds[(RI * ty + i) * (KT + 4) + c] = p == 0.f ? 0.f : p * (y[i][j] - delta[at][c]);
            }
        __syncwarp();
        accumulate<RI>(ps, os, vp, g.dv, tx, ty, dv);
        accumulate<RI>(ds, qs, qp, g.d, tx, ty, dk);
        __syncthreads();
        h = next_h;
        q0 = next;
    }
    copies_wait<0>();
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const int r = RI * ty + i;
        if (r >= rows) continue;
        if (parts > 1) {
            const long long row = (long long)s.b * g.N + s.row0 + it.tok0 + r;
            float *k = a.pieces.k_at(piece, kvh, row), *v = a.pieces.v_at(piece, kvh, row);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int col = 64 * (c >> 2) + 4 * tx + (c & 3);
                if (col < g.d) k[col] = dk[i][c];
                if (col < g.dv) v[col] = dv[i][c];
            }
            continue;
        }
        T *k = a.dk.at(s.b, s.row0 + it.tok0 + r, kvh), *v = a.dv.at(s.b, s.row0 + it.tok0 + r, kvh);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int col = 64 * (c >> 2) + 4 * tx + (c & 3);
            if (col < g.d) k[col] = from_f32<T>(dk[i][c] * g.scale);
            if (col < g.dv) v[col] = from_f32<T>(dv[i][c]);
        }
    }
}

// ------------------------------------------------------------------ host side
constexpr size_t MAX_SMEM = (size_t)(2 * 64 * 2 * 132 + 64 * 132 + 64 * 68) * sizeof(float);     // R = 64, 128 wide

template <typename... P> bool allow(void (*kern)(P...))
{
    // the same number from every call: the limit belongs to the kernel
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MAX_SMEM) == cudaSuccess;
}

// Rows of a forward tile: by the rows that there may be.
int rows_of(const gma_attn_t &a, int pack)
{
    const long long n = (long long)(a.offsets ? 1 : a.B) * a.N, each = (a.offsets ? n : (long long)a.N) * pack;
    if (each <= 16) return 16;
    return n * a.H / 64 < 2 * SMS ? 32 : 64;
}

Plan plan_of(const gma_attn_t &a, const gma_attn_paged_t *paged, int *rows, Carve *c)
{
    const int group = a.H / a.G;
    int pack = paged ? group : 1;
    *rows = rows_of(a, pack);
    if (pack > *rows) pack = 1;
    return make_plan(a, pack, *rows, *rows, 6, SMS, paged != nullptr, c);
}

// Rows of elements of e bytes on 16-byte boundaries; fp32 ones cp.async can copy.
bool vec_rows(const gma_heads_t &r, size_t e) { return (((uintptr_t)r.ptr | (uintptr_t)(r.batch * e) | (uintptr_t)(r.token * e) | (uintptr_t)(r.head * e)) & 15u) == 0; }
bool vec_heads(const gma_heads_t &r) { return vec_rows(r, 4); }

template <typename T>
Args<T> args_of(const gma_attn_t &a, const gma_attn_paged_t *paged, const Plan &p, void *ws)
{
    char *w = (char *)ws;
    Args<T> x = {};
    x.g = geo_of(a, paged);
    x.q = heads_of<const T>(a.q);
    x.k = heads_of<const T>(paged ? paged->k_pages : a.k);
    x.v = heads_of<const T>(paged ? paged->v_pages : a.v);
    x.o = heads_of<T>(a.o);
    x.lse = a.lse;
    x.pack = p.pack;
    x.heads = p.heads;
    x.zero_rows = (a.flags & GMA_ROWS_ZERO_TAIL) && (a.lengths || a.offsets) ? (a.offsets ? 1 : a.B) * a.N : 0;
    x.o_vec = a.dv % (int)(16 / sizeof(T)) == 0 && vec_rows(a.o, sizeof(T));
    x.head = (const PlanHead *)(w + p.head_at);
    x.items = (const Item *)(w + p.items_at);
    x.parts = parts_of(p, a, ws);
    return x;
}

template <typename T, bool PAGED, bool VEC>
gma_status_t forward(const gma_attn_t &a, const gma_attn_paged_t *paged, void *ws, cudaStream_t st)
{
    Carve c;
    int rows;
    const Plan p = plan_of(a, paged, &rows, &c);
    const Args<T> x = args_of<T>(a, paged, p, ws);
    gma_status_t r = launch_plan(plan_args(x.g, p, ws), nullptr, st);
    if (r != GMA_OK) return r;
    const int qp = pitch_of(a.d), vp = pitch_of(a.dv);
    const size_t smem = (size_t)(rows * (qp + KT + 4) + 2 * KT * (qp + vp)) * sizeof(float);
    const unsigned grid = (unsigned)p.max_items * p.heads;
    auto kern = rows == 64 ? attn_simt_kernel<T, PAGED, VEC, 64> : rows == 32 ? attn_simt_kernel<T, PAGED, VEC, 32> : attn_simt_kernel<T, PAGED, VEC, 16>;
    if (!allow(kern)) return GMA_ERR_CUDA;
    GMA_LAUNCH(KID_ATTN_SIMT, st, launch_pdl(kern, grid, TH, smem, st, x));
    return PAGED ? launch_join(a, x.g, p, ws, st) : GMA_OK;
}

struct GradPlan {
    Plan q, k;
    PiecePlan pieces;
    size_t delta_at;
};

GradPlan grad_plan(const gma_attn_t &a, Carve *c)
{
    GradPlan p;
    p.q = make_plan(a, 1, BR, BR, 6, SMS, false, c);
    gma_attn_t by = a;
    p.pieces = plan_pieces(a, BR, KT, 5., c);
    by.H = a.G * p.pieces.count;      // a tile of keys serves the group or a piece of it
    p.k = make_plan(by, 1, BR, BR, 6, SMS, false, c);
    p.k.by_keys = true;
    p.delta_at = c->take((size_t)(a.offsets ? 1 : a.B) * a.H * a.N * sizeof(float));
    return p;
}

template <typename T, bool VEC> gma_status_t backward(const gma_attn_grad_t &g, void *ws, cudaStream_t st)
{
    const gma_attn_t &a = g.fwd;
    Carve c;
    const GradPlan p = grad_plan(a, &c);
    Args<T> x = args_of<T>(a, nullptr, p.q, ws);
    x.d_o = heads_of<const T>(g.d_o);
    x.dq = heads_of<T>(g.dq); x.dk = heads_of<T>(g.dk); x.dv = heads_of<T>(g.dv);
    x.stat_lse = a.lse;
    float *delta = (float *)((char *)ws + p.delta_at);
    x.delta = delta;
    Args<T> y = x;
    y.heads = p.k.heads;
    y.pieces = pieces_of(p.pieces, a, ws);
    y.head = (const PlanHead *)((char *)ws + p.k.head_at);
    y.items = (const Item *)((char *)ws + p.k.items_at);
    const PlanArgs first = plan_args(x.g, p.q, ws);
    PlanArgs second = plan_args(x.g, p.k, ws);
    second.hdr = nullptr;
    gma_status_t r = launch_plan(first, &second, st);
    if (r != GMA_OK) return r;
    if ((r = launch_delta(g, delta, st)) != GMA_OK) return r;
    if (!allow(attn_simt_dq_kernel<T, VEC>) || !allow(attn_simt_dkv_kernel<T, VEC>)) return GMA_ERR_CUDA;
    const int both = pitch_of(a.d) + pitch_of(a.dv);
    const size_t tiles = (size_t)(BR + 2 * KT) * both * sizeof(float), square = BR * (KT + 4) * sizeof(float);
    GMA_LAUNCH(KID_ATTN_SIMT_DKV, st, launch_pdl(attn_simt_dkv_kernel<T, VEC>, (unsigned)p.k.max_items * p.k.heads, TH, tiles + 2 * square, st, y));
    GMA_LAUNCH(KID_ATTN_SIMT_DQ, st, launch_pdl(attn_simt_dq_kernel<T, VEC>, (unsigned)p.q.max_items * p.q.heads, TH, tiles + square, st, x));
    return launch_pieces(g, y.pieces, st);
}

}  // namespace

size_t simt_workspace(const gma_attn_t &a, const gma_attn_paged_t *paged)
{
    Carve c;
    int rows;
    plan_of(a, paged, &rows, &c);
    return c.total();
}

gma_status_t simt_forward(const gma_attn_t &a, const gma_attn_paged_t *p, void *ws, cudaStream_t st)
{
    if (a.dtype == GMA_BF16) return p ? forward<__nv_bfloat16, true, false>(a, p, ws, st) : forward<__nv_bfloat16, false, false>(a, p, ws, st);
    const bool vec = a.d % 4 == 0 && a.dv % 4 == 0 && vec_heads(a.q) && vec_heads(p ? p->k_pages : a.k) && vec_heads(p ? p->v_pages : a.v);
    if (p) return vec ? forward<float, true, true>(a, p, ws, st) : forward<float, true, false>(a, p, ws, st);
    return vec ? forward<float, false, true>(a, p, ws, st) : forward<float, false, false>(a, p, ws, st);
}

size_t simt_backward_workspace(const gma_attn_grad_t &g)
{
    Carve c;
    grad_plan(g.fwd, &c);
    return c.total();
}

gma_status_t simt_backward(const gma_attn_grad_t &g, void *ws, cudaStream_t st)
{
    const gma_attn_t &a = g.fwd;
    if (a.dtype == GMA_BF16) return backward<__nv_bfloat16, false>(g, ws, st);
    const bool vec = a.d % 4 == 0 && a.dv % 4 == 0 && vec_heads(a.q) && vec_heads(a.k) && vec_heads(a.v) && vec_heads(g.d_o);
    return vec ? backward<float, true>(g, ws, st) : backward<float, false>(g, ws, st);
}

}  // namespace att
}  // namespace gma
