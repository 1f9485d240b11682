// gma_attn_simt.cu -- softmax attention on the CUDA cores: fp32, and bf16 rows or pages that the tensor-core kernels
// cannot read (strides off 16 bytes, pages of odd sizes).
//
// Forward: a block takes 64 rows ((token, head of a group) pairs where the keys come from a cache) and walks over its keys 64
// at a time, with the running maximum and sum of each row in registers.  Scores are 4 x 4 a thread out of shared memory, four
// elements of the head at a time: 8 loads of 16 bytes for 64 multiply-adds, so that the fp32 pipe and not shared memory bounds it.
// Warps whose rows do not exist only copy.
#include <algorithm>

#include "attn_common.cuh"

namespace gma {
namespace att {
namespace {

constexpr int R = 64;                 // rows of a tile
constexpr int KT = 64;                // keys of a tile
constexpr int TH = 256;

template <typename T> struct Args {
    Geo g;
    Heads<const T> q, k, v;            // paged: k and v are the pages (batch: page, token: slot)
    Heads<T> o;
    float *lse;
    int pack, heads;
    const PlanHead *head;
    const Item *items;
    Parts parts;
    // backward
    Heads<const T> d_o;
    Heads<T> dq, dk, dv;
    const float *stat_lse, *delta;
};

constexpr __host__ __device__ int pitch_of(int width) { return (width + 3) / 4 * 4 + 4; }

// Rows of `width` elements into shared memory as fp32, zeros behind the width and for rows that `get` has not.
template <typename F> __device__ __forceinline__ void stage(float *dst, int rows, int width, int pitch, F get)
{
    const int w4 = (width + 3) & ~3;
    for (int i = threadIdx.x; i < rows * w4; i += TH) {
        const int r = i / w4, c = i - r * w4;
        dst[r * pitch + c] = c < width ? get(r, c) : 0.f;
    }
}

// Scores of rows 4 ty + i against columns tx + 16 j of two staged tiles.
__device__ __forceinline__ void products(const float *a, const float *b, int pitch, int width, int tx, int ty, float (&s)[4][4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int c = 0; c < width; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(a + (4 * ty + i) * pitch + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * pitch + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
    }
}

// acc[i][4 c + e] += sum_k p[row 4 ty + i][k] x[k][64 c + 4 tx + e], over 64 k.
__device__ __forceinline__ void accumulate(const float *p, const float *x, int pitch, int width, int tx, int ty, float (&acc)[4][8])
{
    for (int k = 0; k < KT; k += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4 *>(p + (4 * ty + i) * (KT + 4) + k);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (64 * c + 4 * tx >= width) break;
            const float *y = x + k * pitch + 64 * c + 4 * tx;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v = *reinterpret_cast<const float4 *>(y + e * pitch);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
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

template <typename T, bool PAGED>
__global__ void __launch_bounds__(TH, 2) attn_simt_kernel(const Args<T> a)
{
    extern __shared__ __align__(16) float smem[];
    __shared__ long long page_at[KT];            // page * 2^20 + slot of every key of the tile, or -1
    if (PAGED) blk::let_next();
    blk::wait_previous();
    const int rank = blockIdx.x / a.heads, head = blockIdx.x % a.heads;
    if (rank >= a.head->items) return;
    const Geo &g = a.g;
    const Item it = a.items[rank];
    if (it.part < 0) return;
    const Seq s = sequence(g, it.seq);
    const int pack = a.pack, kvh = pack == 1 ? head / g.group : head;
    const int tokens = min(a.head->tokens, s.n - it.tok0), rows = tokens * pack;
    const int qp = pitch_of(g.d), vp = pitch_of(g.dv);
    float *qs = smem, *ks = qs + R * qp, *vs = ks + KT * qp, *ps = vs + KT * vp;
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    // row r of the tile: token it.tok0 + r / pack, query head
    auto head_of = [&](int r) { return pack == 1 ? head : head * pack + r % pack; };
    stage(qs, R, g.d, qp, [&](int r, int c) {
        return r < rows ? to_f32<T>(a.q.at(s.b, s.row0 + it.tok0 + r / pack, head_of(r))[c]) : 0.f;
    });
    int seen[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) seen[i] = 4 * ty + i < rows ? s.seen(g, it.tok0 + (4 * ty + i) / pack) : 0;
    const bool busy = (t >> 5) * 8 < rows;       // this warp's rows exist
    float m[4], l[4], acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
    }
    const int end = min(it.t1 * KT, s.seen(g, it.tok0 + tokens - 1));
    for (int k0 = it.t0 * KT; k0 < end; k0 += KT) {
        __syncthreads();
        const int have = min(KT, end - k0);
        if (PAGED) {
            if (t < KT) {
                int slot = 0;
                const int p = t < have ? page_of(g, it.seq, k0 + t, &slot) : -1;
                page_at[t] = p < 0 ? -1 : (long long)p << 20 | slot;
            }
            __syncthreads();
        }
        auto element = [&](const Heads<const T> &x, int r, int c) -> float {
            if (r >= have) return 0.f;
            if (!PAGED) return to_f32<T>(x.at(s.b, s.row0 + k0 + r, kvh)[c]);
            const long long p = page_at[r];
            return p < 0 ? 0.f : to_f32<T>(x.at(p >> 20, p & 0xfffff, kvh)[c]);
        };
        stage(ks, KT, g.d, qp, [&](int r, int c) { return element(a.k, r, c); });
        stage(vs, KT, g.dv, vp, [&](int r, int c) { return element(a.v, r, c); });
        __syncthreads();
        if (!busy) continue;
        float x[4][4];
        products(qs, ks, qp, g.d, tx, ty, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
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
                const float p = ex2(x[i][j] - base);
                sum += p;
                ps[(4 * ty + i) * (KT + 4) + tx + 16 * j] = p;
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            l[i] = l[i] * f + sum;
            m[i] = now;
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[i][c] *= f;
        }
        __syncwarp();                            // a warp reads the rows that it wrote
        accumulate(ps, vs, vp, g.dv, tx, ty, acc);
    }
    const bool whole = it.parts == 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
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

// dq of 64 query rows of one head: ds = p (do . v - delta), dq = scale ds k over the keys that the rows see.
template <typename T> __global__ void __launch_bounds__(TH, 1) attn_simt_dq_kernel(const Args<T> a)
{
    extern __shared__ __align__(16) float smem[];
    blk::wait_previous();
    const int rank = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
    if (rank >= a.head->items) return;
    const Geo &g = a.g;
    const Item it = a.items[rank];
    const Seq s = sequence(g, it.seq);
    const int kvh = h / g.group, rows = min(R, s.n - it.tok0);
    const int qp = pitch_of(g.d), vp = pitch_of(g.dv);
    float *qs = smem, *os = qs + R * qp, *ks = os + R * vp, *vs = ks + KT * qp, *ps = vs + KT * vp;
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    stage(qs, R, g.d, qp, [&](int r, int c) { return r < rows ? to_f32<T>(a.q.at(s.b, s.row0 + it.tok0 + r, h)[c]) : 0.f; });
    stage(os, R, g.dv, vp, [&](int r, int c) { return r < rows ? to_f32<T>(a.d_o.at(s.b, s.row0 + it.tok0 + r, h)[c]) : 0.f; });
    float lse2[4], delta[4], acc[4][8];
    int seen[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        const bool is = r < rows;
        const long long at = is ? stat_at(g, s, h, it.tok0 + r) : 0;
        seen[i] = is ? s.seen(g, it.tok0 + r) : 0;
        lse2[i] = is ? a.stat_lse[at] * LOG2E : 0.f;
        delta[i] = is ? a.delta[at] : 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
    }
    const int end = min(it.t1 * KT, s.L);
    for (int k0 = it.t0 * KT; k0 < end; k0 += KT) {
        __syncthreads();
        const int have = min(KT, s.L - k0);
        stage(ks, KT, g.d, qp, [&](int r, int c) { return r < have ? to_f32<T>(a.k.at(s.b, s.row0 + k0 + r, kvh)[c]) : 0.f; });
        stage(vs, KT, g.dv, vp, [&](int r, int c) { return r < have ? to_f32<T>(a.v.at(s.b, s.row0 + k0 + r, kvh)[c]) : 0.f; });
        __syncthreads();
        float x[4][4], y[4][4];
        products(qs, ks, qp, g.d, tx, ty, x);
        products(os, vs, vp, g.dv, tx, ty, y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = k0 + tx + 16 * j < seen[i] ? ex2(x[i][j] * g.sl2 - lse2[i]) : 0.f;
                ps[(4 * ty + i) * (KT + 4) + tx + 16 * j] = p == 0.f ? 0.f : p * (y[i][j] - delta[i]);
            }
        __syncwarp();
        accumulate(ps, ks, qp, g.d, tx, ty, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (4 * ty + i >= rows) continue;
        T *dq = a.dq.at(s.b, s.row0 + it.tok0 + 4 * ty + i, h);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int col = 64 * (c >> 2) + 4 * tx + (c & 3);
            if (col < g.d) dq[col] = from_f32<T>(acc[i][c] * g.scale);
        }
    }
}

// dk and dv of 64 keys of one head, over the query heads of its group and the rows that see them: rows of the
// tiles are keys here, columns queries.
template <typename T> __global__ void __launch_bounds__(TH, 1) attn_simt_dkv_kernel(const Args<T> a)
{
    extern __shared__ __align__(16) float smem[];
    __shared__ float lse2[KT], delta[KT];
    blk::wait_previous();
    const int rank = blockIdx.x / a.heads, kvh = blockIdx.x % a.heads;
    if (rank >= a.head->items) return;
    const Geo &g = a.g;
    const Item it = a.items[rank];
    const Seq s = sequence(g, it.seq);
    const int rows = min(R, s.n - it.tok0);
    const int qp = pitch_of(g.d), vp = pitch_of(g.dv);
    float *ks = smem, *vs = ks + R * qp, *qs = vs + R * vp, *os = qs + KT * qp, *ps = os + KT * vp, *ds = ps + R * (KT + 4);
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    stage(ks, R, g.d, qp, [&](int r, int c) { return r < rows ? to_f32<T>(a.k.at(s.b, s.row0 + it.tok0 + r, kvh)[c]) : 0.f; });
    stage(vs, R, g.dv, vp, [&](int r, int c) { return r < rows ? to_f32<T>(a.v.at(s.b, s.row0 + it.tok0 + r, kvh)[c]) : 0.f; });
    float dk[4][8], dv[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) dk[i][c] = dv[i][c] = 0.f;
    for (int h = kvh * g.group; h < (kvh + 1) * g.group; ++h)
        for (int q0 = it.t0 * KT; q0 < min(it.t1 * KT, s.n); q0 += KT) {
            __syncthreads();
            const int have = min(KT, s.n - q0);
            stage(qs, KT, g.d, qp, [&](int r, int c) { return r < have ? to_f32<T>(a.q.at(s.b, s.row0 + q0 + r, h)[c]) : 0.f; });
            stage(os, KT, g.dv, vp, [&](int r, int c) { return r < have ? to_f32<T>(a.d_o.at(s.b, s.row0 + q0 + r, h)[c]) : 0.f; });
            if (t < have) {
                const long long at = stat_at(g, s, h, q0 + t);
                lse2[t] = a.stat_lse[at] * LOG2E;
                delta[t] = a.delta[at];
            }
            __syncthreads();
            float x[4][4], y[4][4];
            products(ks, qs, qp, g.d, tx, ty, x);
            products(vs, os, vp, g.dv, tx, ty, y);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = tx + 16 * j, key = it.tok0 + 4 * ty + i;
                    const float p = c < have && key < s.seen(g, q0 + c) ? ex2(x[i][j] * g.sl2 - lse2[c]) : 0.f;
                    ps[(4 * ty + i) * (KT + 4) + c] = p;
                    ds[(4 * ty + i) * (KT + 4) + c] = p == 0.f ? 0.f : p * (y[i][j] - delta[c]);
                }
            __syncwarp();
            accumulate(ps, os, vp, g.dv, tx, ty, dv);
            accumulate(ds, qs, qp, g.d, tx, ty, dk);
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= rows) continue;
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
constexpr size_t MAX_SMEM = (size_t)(4 * 64 * 132 + 2 * 64 * 68) * sizeof(float);

template <typename... P> bool allow(void (*kern)(P...))
{
    // the same number from every call: the limit belongs to the kernel
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MAX_SMEM) == cudaSuccess;
}

Plan plan_of(const gma_attn_t &a, const gma_attn_paged_t *paged, Carve *c)
{
    const int group = a.H / a.G, pack = paged && group <= R ? group : 1;
    return make_plan(a, pack, R, R, 6, SMS, paged != nullptr, c);
}

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
    x.head = (const PlanHead *)(w + p.head_at);
    x.items = (const Item *)(w + p.items_at);
    x.parts = parts_of(p, a, ws);
    return x;
}

template <typename T> gma_status_t forward(const gma_attn_t &a, const gma_attn_paged_t *paged, void *ws, cudaStream_t st)
{
    Carve c;
    const Plan p = plan_of(a, paged, &c);
    const Args<T> x = args_of<T>(a, paged, p, ws);
    gma_status_t r = launch_plan(plan_args(x.g, p, ws), nullptr, st);
    if (r != GMA_OK) return r;
    const size_t smem = (size_t)(2 * 64 * pitch_of(a.d) + 64 * pitch_of(a.dv) + 64 * 68) * sizeof(float);
    const unsigned grid = (unsigned)p.max_items * p.heads;
    if (paged) {
        if (!allow(attn_simt_kernel<T, true>)) return GMA_ERR_CUDA;
        GMA_LAUNCH(KID_ATTN_SIMT, st, launch_pdl(attn_simt_kernel<T, true>, grid, TH, smem, st, x));
        return launch_join(a, x.g, p, ws, st);
    } else {
        if (!allow(attn_simt_kernel<T, false>)) return GMA_ERR_CUDA;
        GMA_LAUNCH(KID_ATTN_SIMT, st, launch_pdl(attn_simt_kernel<T, false>, grid, TH, smem, st, x));
    }
    return GMA_OK;
}

struct GradPlan {
    Plan q, k;
    size_t delta_at;
};

GradPlan grad_plan(const gma_attn_t &a, Carve *c)
{
    GradPlan p;
    p.q = make_plan(a, 1, R, R, 6, SMS, false, c);
    gma_attn_t by = a;
    by.H = a.G;                       // a tile of keys serves the whole group
    p.k = make_plan(by, 1, R, R, 6, SMS, false, c);
    p.k.by_keys = true;
    p.delta_at = c->take((size_t)(a.offsets ? 1 : a.B) * a.H * a.N * sizeof(float));
    return p;
}

template <typename T> gma_status_t backward(const gma_attn_grad_t &g, void *ws, cudaStream_t st)
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
    y.head = (const PlanHead *)((char *)ws + p.k.head_at);
    y.items = (const Item *)((char *)ws + p.k.items_at);
    const PlanArgs first = plan_args(x.g, p.q, ws);
    PlanArgs second = plan_args(x.g, p.k, ws);
    second.hdr = nullptr;
    gma_status_t r = launch_plan(first, &second, st);
    if (r != GMA_OK) return r;
    if ((r = launch_delta(g, delta, st)) != GMA_OK) return r;
    if (!allow(attn_simt_dq_kernel<T>) || !allow(attn_simt_dkv_kernel<T>)) return GMA_ERR_CUDA;
    const size_t tiles = (size_t)(2 * 64 * pitch_of(a.d) + 2 * 64 * pitch_of(a.dv)) * sizeof(float), square = 64 * 68 * sizeof(float);
    GMA_LAUNCH(KID_ATTN_SIMT_DKV, st, launch_pdl(attn_simt_dkv_kernel<T>, (unsigned)p.k.max_items * p.k.heads, TH, tiles + 2 * square, st, y));
    GMA_LAUNCH(KID_ATTN_SIMT_DQ, st, launch_pdl(attn_simt_dq_kernel<T>, (unsigned)p.q.max_items * p.q.heads, TH, tiles + square, st, x));
    return GMA_OK;
}

}  // namespace

size_t simt_workspace(const gma_attn_t &a, const gma_attn_paged_t *paged)
{
    Carve c;
    plan_of(a, paged, &c);
    return c.total();
}

gma_status_t simt_forward(const gma_attn_t &a, const gma_attn_paged_t *paged, void *ws, cudaStream_t st)
{
    return a.dtype == GMA_BF16 ? forward<__nv_bfloat16>(a, paged, ws, st) : forward<float>(a, paged, ws, st);
}

size_t simt_backward_workspace(const gma_attn_grad_t &g)
{
    Carve c;
    grad_plan(g.fwd, &c);
    return c.total();
}

gma_status_t simt_backward(const gma_attn_grad_t &g, void *ws, cudaStream_t st)
{
    return g.fwd.dtype == GMA_BF16 ? backward<__nv_bfloat16>(g, ws, st) : backward<float>(g, ws, st);
}

}  // namespace att
}  // namespace gma
