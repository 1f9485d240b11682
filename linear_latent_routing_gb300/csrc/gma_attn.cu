// gma_attn.cu -- softmax attention: the entry points' checks, the plan of a call, and the small kernels around the
// products: tokens into the cache's pages, do . o of every row with zeros behind sequences in the gradients, dense copies, the join.
#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"
#include "attn_tc_host.cuh"

namespace gma {
namespace att {
namespace {

typedef __nv_bfloat16 bf16;
constexpr int PT = 256;                // threads of the plan's block
constexpr int SEQS = 1024;             // sequences that are held at a time
constexpr int CUTS = 2 * SMS + 2;      // tiles that are cut, at most
constexpr int BUCKETS = 1024;          // items are ordered by size up to so many key tiles
constexpr int TILES = 2048;            // tiles up to which cutting is looked at
constexpr int SIZES = 24;              // of parts that are tried
constexpr double REPACK_FROM = 5e5;     // rows x rows x heads
constexpr float ITEM_COST = 2.f;       // what an item costs beside its keys, in key tiles

// Exclusive sum over the block's threads; *all: the sum of all of them.
__device__ __forceinline__ int block_scan(int own, int *warps, int *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += up;
    }
    if (lane == 31) warps[warp] = sum;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < PT / 32; ++w) {
        const int x = warps[w];
        before += w < warp ? x : 0;
        total += x;
    }
    __syncthreads();
    *all = total;
    return before + sum - own;
}

// A thread a sequence (up to four of them) for their numbers of tiles, then a thread a tile (its sequence found by bisection) for everything
// else.  Up to SEQS sequences are read once, and up to TILES tiles looked up once; more are gone through again in every pass.
// Latency is all: 256 threads, whose barriers are cheap, a warp for each tile that is cut, and little code, since behind a long cache that has
// gone through L2 it comes from DRAM (one loop for the three passes, where each had a copy of its own).  65536 cached tokens of one sequence,
// 16 / 4 heads of 128: 43.7 -> 38.4 us a call; 512 sequences of 500 tokens but for one of 60000, when no more than 256 were cut: 439 -> 80 us.
__global__ void __launch_bounds__(PT) plan_kernel(const PlanArgs a0, const PlanArgs a1)
{
    const PlanArgs &a = blockIdx.x ? a1 : a0;
    __shared__ unsigned long long total;
    __shared__ int slots, joins, largest, warps[PT / 32], first[SEQS + 1], rows[SEQS], keys[SEQS], start_row[SEQS], costs[TILES], sizes[SIZES];
    __shared__ __align__(16) int hist[BUCKETS];
    __shared__ int cut_at[CUTS], cut_slot[CUTS], cut_tile[CUTS];
    __shared__ unsigned short seqs[TILES];
    __shared__ float times[SIZES];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, B = a.g.B, mask = (1 << a.key_shift) - 1;
    const int per = min((B + PT - 1) / PT, SEQS / PT), held = per * PT, mine = t * per;      // sequences a thread, at a time, this thread's first
    if (t == 0) { total = 0; slots = 0; joins = 0; largest = 0; }
    *reinterpret_cast<int4 *>(hist + 4 * t) = make_int4(0, 0, 0, 0);
    blk::wait_previous();
    blk::let_next();             // what came before is through, then: the next kernel's zeros need not wait
    if (a.hdr && t < (int)(sizeof(WsHeader) / 4)) reinterpret_cast<unsigned *>(a.hdr)[t] = t == 2 && a.short_waits;       // reserved[0]
    int tokens = a.wide;
    // reads the sequences from `base` on (or has them), and numbers their tiles
    auto number = [&](int base, bool have) {
        int own = 0, all;
        if (!have) __syncthreads();
#pragma unroll 1
        for (int k = mine; k < mine + per; ++k) {
            if (!have) {
                Seq q = {};
                if (base + k < B) q = sequence(a.g, base + k);
                rows[k] = q.n;
                keys[k] = q.L;
                start_row[k] = q.row0;
            }
            first[k] = own;                                          // of this thread's, so far
            own += (unsigned)(rows[k] + tokens - 1) / (unsigned)tokens;
        }
        const int at = block_scan(own, warps, &all);
#pragma unroll 1
        for (int k = mine; k < mine + per; ++k) first[k] += at;
        if (t == PT - 1) first[held] = all;
        __syncthreads();
        return all;
    };
    // wide tiles, or narrow ones where the wide ones are fewer than the SMs (4 x 2048 x 8 heads of 64, 256 wide tiles: 38 us with those, 43
    // with narrow ones)
    int count;
    for (bool again = false;; again = true) {
        count = 0;
        for (int base = 0; base < B; base += held) count += number(base, again && B <= held);
        if (again || (long long)count * a.heads >= SMS || a.narrow >= a.wide) break;
        tokens = a.narrow;
    }
    const bool table = B <= held && count <= TILES;      // costs and seqs hold all tiles, after the first pass
    // Three passes over the tiles: the work and the largest tile (where tiles may be cut; more of them than the table holds fill the GPU as they
    // are), how many items of each size, and the list.
    const bool cutting = a.max_slots && table && count;
    int share = 0x7fffffff;                              // a part's key tiles
#pragma unroll 1
    for (int pass = cutting ? 0 : 1; pass < 3; ++pass) {
        const bool known = table && (pass == 2 || (pass == 1 && cutting));
        unsigned long long work = 0;
        int most = 0;
#pragma unroll 1
        for (int base = 0; base < B; base += held) {
            if (B > held) number(base, false);
#pragma unroll 1
            for (int i = t; i < first[held]; i += PT) {
                int s = 0, cost;
                if (known) {
                    s = seqs[i];
                } else {
                    int hi = held;
                    while (hi - s > 1) {
                        const int mid = (s + hi) >> 1;
                        if (first[mid] <= i) s = mid; else hi = mid;
                    }
                }
                // (by_keys: query tiles of a tile of keys, from the first that sees it)
                const int n = rows[s], L = keys[s], tok = (i - first[s]) * tokens, pos0 = a.g.cached ? L - n : 0;
                const int from = a.by_keys && a.g.causal ? tok >> a.key_shift : 0;
                if (known) {
                    cost = costs[i];
                } else {
                    const int last = min(tok + tokens, n) - 1, seen = a.g.causal ? min(max(pos0 + last + 1, 0), L) : L;
                    cost = a.by_keys ? ((n + mask) >> a.key_shift) - from : max((seen + mask) >> a.key_shift, 1);
                    if (table) {
                        costs[i] = cost;
                        seqs[i] = (unsigned short)s;
                    }
                }
                if (pass == 0) {
                    work += cost;
                    most = max(most, cost);
                    continue;
                }
                const int parts = cost <= share ? 1 : (cost - 1) / share + 1, size = parts == 1 ? cost : (cost - 1) / parts + 1;
                const int at = atomicAdd(&hist[BUCKETS - 1 - min(size, BUCKETS - 1)], parts);
                if (pass == 1) continue;
                if (parts == 1) {
                    const Seq q{a.g.offsets ? 0 : base + s, start_row[s], n, L, pos0};
                    if (at < a.max_items) a.items[at] = Item{base + s, tok, from, from + cost, 0, 1, 0, 0, q, {}};
                } else {
                    const int cut = atomicAdd(&joins, 1), slot = atomicAdd(&slots, parts);
                    if (cut < CUTS) cut_at[cut] = at, cut_slot[cut] = slot, cut_tile[cut] = i;
                }
            }
        }
        if (pass == 0) {
            // the size of parts: an estimate of the time with SIZES sizes, from half a block's share of the call to five of them
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                work += __shfl_xor_sync(~0u, work, o);
                most = max(most, __shfl_xor_sync(~0u, most, o));
            }
            if (lane == 0 && work) {
                atomicAdd(&total, work);
                atomicMax(&largest, most);
            }
            __syncthreads();
            const float all = (float)total * a.heads, each = all / a.blocks;
            const int top = largest;
#pragma unroll 1
            for (int c = warp; c < SIZES; c += PT / 32) {
                const int size = max((int)ceilf(each * 0.5f * exp2f(c * (3.3f / (SIZES - 1)))), 1);
                const float inv = 1.f / size;
                int parts = 0, cut = 0;
#pragma unroll 1
                for (int i = lane; i < count; i += 32) {
                    // (an estimate: the quotient may be off by one)
                    const int k = costs[i] <= size ? 1 : (int)((costs[i] - 1) * inv) + 1;
                    parts += k;
                    if (k > 1) cut += k;
                }
                parts = __reduce_add_sync(~0u, parts);
                cut = __reduce_add_sync(~0u, cut);
                const float items = (float)parts * a.heads, extra = ITEM_COST * items + a.part_cost * cut * a.heads;
                const int cuts = top <= size ? 1 : (int)((top - 1) * inv) + 1;
                const float longest = (float)((top - 1) / cuts + 1) + ITEM_COST + (cuts > 1 ? a.part_cost : 0.f);
                const float mean = (all + extra) / items, waves = ceilf(items / a.blocks);
                // equal items run in whole waves; unequal ones, the longest first, fill the gaps
                const float time = longest < 1.2f * mean || items <= a.blocks ? waves * longest
                                                                              : fmaxf((all + extra) / a.blocks + 0.5f * mean, longest);
                if (lane == 0) times[c] = time, sizes[c] = size;
            }
            __syncthreads();
            // the largest of the best (times are not negative: their order is that of their bits)
            const unsigned time = lane < SIZES ? __float_as_uint(times[lane]) : ~0u, best = __reduce_min_sync(~0u, time);
            share = sizes[31 - __clz(__ballot_sync(~0u, time == best))];
        } else if (pass == 1) {
            // where the items of each size start, the largest first
            __syncthreads();
            const int4 h = *reinterpret_cast<const int4 *>(hist + 4 * t);
            const int at = block_scan(h.x + h.y + h.z + h.w, warps, &count);
            *reinterpret_cast<int4 *>(hist + 4 * t) = make_int4(at, at + h.x, at + h.x + h.y, at + h.x + h.y + h.z);
            __syncthreads();
        }
    }
    __syncthreads();
    // A warp a tile that is cut, a lane a part.  Cuts are within the bounds that the lists were made for (offsets that fall may make more tiles,
    // which are left out).
    const int cuts = min(min(joins, CUTS), a.max_slots);
#pragma unroll 1
    for (int c = warp; c < cuts; c += PT / 32) {
        const int i = cut_tile[c], s = seqs[i], cost = costs[i], at = cut_at[c], slot = cut_slot[c], n = rows[s], L = keys[s];
        const int tok = (i - first[s]) * tokens, parts = (cost - 1) / share + 1, size = (cost - 1) / parts + 1;
        const Seq q{a.g.offsets ? 0 : s, start_row[s], n, L, a.g.cached ? L - n : 0};
        const bool room = slot + parts <= a.max_slots && at + parts <= a.max_items;
#pragma unroll 1
        for (int p = lane; p < parts && at + p < a.max_items; p += 32)
            a.items[at + p] = Item{s, tok, min(p * size, cost), min((p + 1) * size, cost), room ? slot : 0, parts, room ? p : -1, 0, q, {}};
        if (lane == 0) a.join[c] = Join{slot, room ? parts : 0, q.b, q.row0 + tok, min(tokens, n - tok), {}};
    }
    if (t == 0) {
        a.head->items = min(count, a.max_items);
        a.head->tokens = tokens;
        a.head->ticket = a.blocks;       // a block's first item is that of its number
        a.head->joins = cuts;
    }
}

// A warp a row of a cut item: lanes are parts for the weights, then four columns each for the sums, with the loads of sixteen parts
// in flight.
template <typename T>
__global__ void __launch_bounds__(256) attn_join_kernel(const Geo g, const PlanHead *head, const Join *join, const Parts p, const Heads<T> out,
                                                        float *lse, int pack)
{
    const unsigned lane = threadIdx.x & 31, step = gridDim.x * 8;
    // (the plan was through when the kernel before let this one start)
    const unsigned rows = min((unsigned)__ldcg(&head->tokens) * pack, (unsigned)p.rows), n = (unsigned)__ldcg(&head->joins) * p.heads * rows;
    // Rows that are fewer than the blocks lie on SMs of their own (16 rows of 38 parts each in two blocks took 2 us more: one token over 65536); more of
    // them fill the first blocks, which start on the first SMs that are free (32 x 6 drafted tokens 2 us less than over all blocks).
    unsigned i = n <= gridDim.x ? (threadIdx.x >> 5) * gridDim.x + blockIdx.x : blockIdx.x * 8 + (threadIdx.x >> 5);
    auto entry = [&]() {
        const int4 *at = reinterpret_cast<const int4 *>(join + min(i, n - 1) / rows / p.heads);
        const int4 x = __ldcg(at), y = __ldcg(at + 1);
        return Join{x.x, x.y, x.z, x.w, y.x, {}};
    };
    Join it = {};
    if (i < n) it = entry();
    blk::wait_previous();
    for (; i < n; i += step, it = entry()) {
        const unsigned hj = i / rows, row = i - hj * rows, j = hj / p.heads, hd = hj - j * p.heads;
        const int tok = row / pack, h = pack == 1 ? hd : hd * pack + row % pack;
        if (tok >= it.tokens) continue;
        const float *stat = p.stat_at(it.slot, hd, row), *part = p.o_at(it.slot, hd, row) + 4 * lane;
        const long long stat_step = (long long)p.heads * p.rows * 2, part_step = (long long)p.heads * p.rows * p.pitch;
        const bool mine = 4 * lane < p.dv;
        float m = -INFINITY, l = 0.f;            // so far
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < it.parts; k0 += 32) {
            // a first batch of sums, on its way beside the weights
            const int n = min(32, it.parts - k0);
            float4 x[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (mine && k < n) x[k] = *reinterpret_cast<const float4 *>(part + (k0 + k) * part_step);
            float2 s = make_float2(-INFINITY, 0.f);
            if ((int)lane < n) s = *reinterpret_cast<const float2 *>(stat + (k0 + lane) * stat_step);
            float top = s.x;
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            const float now = fmaxf(m, top), base = now == -INFINITY ? 0.f : now, f0 = ex2(m - base);
            const float w = ex2(s.x - base);     // of a part that saw nothing: 0, and it wrote no sums
            m = now;
            l = l * f0 + w * s.y;
            acc.x *= f0; acc.y *= f0; acc.z *= f0; acc.w *= f0;
            for (int k1 = 0; k1 < n; k1 += 16) {
                if (k1) {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (mine && k1 + k < n) x[k] = *reinterpret_cast<const float4 *>(part + (k0 + k1 + k) * part_step);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float f = __shfl_sync(~0u, w, k1 + k);
                    if (f == 0.f) continue;
                    acc.x = fmaf(f, x[k].x, acc.x);
                    acc.y = fmaf(f, x[k].y, acc.y);
                    acc.z = fmaf(f, x[k].z, acc.z);
                    acc.w = fmaf(f, x[k].w, acc.w);
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
        const float inv = l > 0.f ? 1.f / l : 0.f, y[4] = {acc.x, acc.y, acc.z, acc.w};
        T *o = out.at(it.b, it.row + tok, h);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if ((int)(4 * lane + c) < p.dv) o[4 * lane + c] = from_f32<T>(y[c] * inv);
        if (lse && lane == 0) lse[((long long)it.b * g.H + h) * g.N + it.row + tok] = l > 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
    }
}

// Rows that see at most so many keys have a delta of their own in the backward pass of bf16 tensors.  A stored o is off by 2^-9 of itself in the
// mean, and do . o with it, which over few keys is not small beside ds = p (do . v - delta); delta = sum p do . v / sum p is the same and reads no o.
// How far dq is off (normwise; the rounding of dq alone 1.66e-3), with do . o for all rows and so: 200 sequences of 2 tokens 3.65e-3 and 2.34e-3,
// 20 of 33 2.72e-3 and 2.40e-3, 2 of 1000 2.46e-3 and 2.40e-3.  Rows over 17 keys with do . o: 2.54e-3; up to 32 keys cost train steps of
// 64 x 100 x 16 heads of 128 11 us more.
constexpr int FEW = 16;

struct FewArgs {
    Heads<const bf16> q, k, v;
    const float *lse;
    unsigned blocks;           // the first ones of the launch, 0: none
    int pairs;                 // two neighbouring elements lie on 4-byte boundaries
};

// Those rows' delta: a warp a sequence and head, by mma.sync.  16 x 16 scores are too small for tcgen05, whose loads, barriers and tensor memory take
// longer than the products; latency is all, and the blocks of the other rows run beside these (5 blocks an SM for their sake: 4 x 2048 tokens, forward
// and backward, 131.5 us without and 131.0 with it; as a launch of its own 144).
template <bool PAIR> __device__ __forceinline__ void delta_of_few(const Geo &g, const FewArgs &a, const Heads<const bf16> &d_o, float *delta)
{
    const int lane = threadIdx.x & 31, gr = lane >> 2, t2 = 2 * (lane & 3);
    const long long tiles = (long long)g.B * g.H;
    // elements c and c + 1 of a row, zeros behind its width and where it `is` not; without branches, so that the loads of a product are on their way
    // together
    auto pair = [&](const bf16 *row, int c, int width, bool is) -> uint32_t {
        const bool lo = is && c < width, hi = is && c + 1 < width;
        if (PAIR) {
            const uint32_t x = *reinterpret_cast<const uint32_t *>(row + (lo ? c : 0));
            return lo ? x : 0u;
        }
        const uint32_t x = __bfloat16_as_ushort(row[lo ? c : 0]), y = __bfloat16_as_ushort(row[hi ? c + 1 : 0]);
        return (lo ? x : 0u) | (hi ? y : 0u) << 16;
    };
    for (long long w = blockIdx.x * 8ll + (threadIdx.x >> 5); w < tiles; w += a.blocks * 8ll) {
        const int h = (int)(w % g.H), kvh = h / g.group, i0 = gr, i1 = gr + 8;
        const Seq s = sequence(g, (int)(w / g.H));
        const int rows = g.causal || s.n <= FEW ? min(s.n, FEW) : 0;      // and keys
        if (!rows) continue;
        // rows i0 (the first two of four) and i1 of x times the keys' rows of y, columns 8 n + t2 and the next one
        auto product = [&](const Heads<const bf16> &x, const Heads<const bf16> &y, int width, float (&d)[2][4]) {
            const bf16 *x0 = x.at(s.b, s.row0 + (i0 < rows ? i0 : 0), h), *x1 = x.at(s.b, s.row0 + (i1 < rows ? i1 : 0), h), *yn[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                yn[n] = y.at(s.b, s.row0 + (8 * n + gr < rows ? 8 * n + gr : 0), kvh);
#pragma unroll
                for (int c = 0; c < 4; ++c) d[n][c] = 0.f;
            }
#pragma unroll 1
            for (int c0 = 0; c0 < width; c0 += 16) {
                const int c = c0 + t2;
                const uint32_t a0 = pair(x0, c, width, i0 < rows), a1 = pair(x1, c, width, i1 < rows);
                const uint32_t a2 = pair(x0, c + 8, width, i0 < rows), a3 = pair(x1, c + 8, width, i1 < rows);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const bool is = 8 * n + gr < rows;
                    const uint32_t b0 = pair(yn[n], c, width, is), b1 = pair(yn[n], c + 8, width, is);
                    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                        : "+f"(d[n][0]), "+f"(d[n][1]), "+f"(d[n][2]), "+f"(d[n][3])
                        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
                }
            }
        };
        float score[2][4], dp[2][4];
        product(a.q, a.k, g.d, score);
        product(d_o, a.v, g.dv, dp);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = half ? i1 : i0, seen = i < rows ? (g.causal ? i + 1 : s.n) : 0;
            const long long at = stat_at(g, s, h, i < rows ? i : 0);
            const float lse2 = a.lse[at] * LOG2E;
            float sum = 0.f, dot = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float p = 8 * n + t2 + c < seen ? ex2(score[n][2 * half + c] * g.sl2 - lse2) : 0.f;
                    sum += p;
                    dot = fmaf(p, dp[n][2 * half + c], dot);
                }
#pragma unroll
            for (int o = 2; o; o >>= 1) {
                sum += __shfl_xor_sync(~0u, sum, o);
                dot += __shfl_xor_sync(~0u, dot, o);
            }
            if (i < rows && t2 == 0) delta[at] = dot / sum;
        }
    }
}

// Whether row i of the packed tensors, which belongs to a sequence, sees few keys.
__device__ __forceinline__ bool sees_few(const Geo &g, int i)
{
    int lo = 0, hi = g.B;              // the last sequence that starts at or before the row: empty ones may share a start
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.offsets[mid] <= i) lo = mid; else hi = mid;
    }
    const int start = max(g.offsets[lo], 0);
    return g.causal ? i - start < FEW : min(g.offsets[lo + 1], g.N) - start <= FEW;
}

// delta = do . o, and zeros in the gradients' rows that belong to no sequence: LANES lanes a (row, head), eight elements each (VEC) or every LANES-th.
template <typename T, bool VEC, int LANES>
__global__ void __launch_bounds__(256, 5) attn_delta_kernel(const Geo g, const Heads<const T> o, const Heads<const T> d_o, float *delta,
                                                         long long rows, const Heads<T> dq, const Heads<T> dk, const Heads<T> dv, int zero,
                                                         const FewArgs few)
{
    const int lane = threadIdx.x % LANES;
    blk::let_next();
    if constexpr (sizeof(T) == 2) {
        if (blockIdx.x < few.blocks) {
            if (few.pairs) delta_of_few<true>(g, few, d_o, delta);
            else delta_of_few<false>(g, few, d_o, delta);
            blk::wait_previous();
            return;
        }
    }
    const unsigned block = blockIdx.x - few.blocks, blocks = gridDim.x - few.blocks;
    for (long long r0 = block * (256ll / LANES); r0 < rows; r0 += blocks * (256ll / LANES)) {
        const long long r = r0 + threadIdx.x / LANES;         // heads inner: neighbouring rows of lanes read neighbouring heads
        bool is = r < rows;
        const long long bi = r / g.H;
        const int h = (int)(r - bi * g.H), b = (int)(bi / g.N);
        const long long i = bi - (long long)b * g.N;
        if (is) is = g.offsets ? i >= max(g.offsets[0], 0) && i < g.offsets[g.B] : i < blk::row_length(g.lengths, b, g.N);
        // the gradients' rows that belong to no sequence
        if (zero && !is && r < rows) {
            auto clear = [&](T *at, int width) {
                constexpr int E = 16 / sizeof(T);
                if (zero > 1)
                    for (int c = lane * E; c < width; c += LANES * E) *reinterpret_cast<uint4 *>(at + c) = make_uint4(0, 0, 0, 0);
                else
                    for (int c = lane; c < width; c += LANES) at[c] = from_f32<T>(0.f);
            };
            clear(dq.at(b, i, h), g.d);
            if (h < g.G) {
                clear(dk.at(b, i, h), g.d);
                clear(dv.at(b, i, h), g.dv);
            }
        }
        float s = 0.f;
        if (is) {
            const T *x = o.at(b, i, h), *y = d_o.at(b, i, h);
            if (VEC) {
                if (8 * lane < g.dv) {
                    float u[8], v[8];
                    blk::load8<true>(x + 8 * lane, 8, u);
                    blk::load8<true>(y + 8 * lane, 8, v);
#pragma unroll
                    for (int c = 0; c < 8; ++c) s = fmaf(u[c], v[c], s);
                }
            } else {
                for (int c = lane; c < g.dv; c += LANES) s = fmaf(to_f32<T>(x[c]), to_f32<T>(y[c]), s);
            }
        }
#pragma unroll
        for (int m = LANES / 2; m; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
        bool mine = is;
        if (few.blocks && is) mine = g.offsets ? !sees_few(g, (int)i) : g.causal ? i >= FEW : blk::row_length(g.lengths, b, g.N) > FEW;
        if (mine && lane == 0) delta[((long long)b * g.H + h) * g.N + i] = s;
    }
    blk::wait_previous();
}

// dk and dv of a head from its group's pieces: a warp a (row, head), four columns a lane.
template <typename T>
__global__ void __launch_bounds__(256) attn_pieces_kernel(const Geo g, const Pieces p, const Heads<T> dk, const Heads<T> dv)
{
    const int lane = threadIdx.x & 31;
    const long long all = p.rows * g.G;
    blk::wait_previous();
    for (long long i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < all; i += gridDim.x * 8ll) {
        const long long r = i / g.G, tok = r % g.N;
        const int h = (int)(i - r * g.G), b = (int)(r / g.N);
        if (g.offsets ? tok < max(g.offsets[0], 0) || tok >= g.offsets[g.B] : tok >= blk::row_length(g.lengths, b, g.N)) continue;
        auto sum = [&](const float *at, int pitch, int width, float f, T *out) {
            if (4 * lane >= width) return;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < p.count; ++k) {
                const float4 x = *reinterpret_cast<const float4 *>(at + p.at(k, h, r) * pitch + 4 * lane);
                s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
            }
            const float y[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (4 * lane + c < width) out[4 * lane + c] = from_f32<T>(y[c] * f);
        };
        sum(p.k, p.k_pitch, g.d, g.scale, dk.at(b, tok, h));
        sum(p.v, p.v_pitch, g.dv, 1.f, dv.at(b, tok, h));
    }
}

// The new tokens' keys and values into their slots: a warp a (token, head), both tensors.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) attn_append_kernel(const Geo g, const Heads<const T> k, const Heads<const T> v, const Heads<T> kp,
                                                          const Heads<T> vp, long long rows)
{
    const int lane = threadIdx.x & 31;
    blk::let_next();             // the plan of a call on the cache, which waits for this one's end
    for (long long r = blockIdx.x * 8ll + (threadIdx.x >> 5); r < rows; r += gridDim.x * 8ll) {
        const int h = (int)(r % g.G);
        const long long tok = r / g.G;
        int s, i;
        if (g.offsets) {               // the last sequence that starts at or before the row
            int lo = 0, hi = g.B;      // empty ones may share a start: the last of them holds the row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (g.offsets[mid] <= tok) lo = mid; else hi = mid;
            }
            s = lo;
        } else {
            s = (int)(tok / g.N);
        }
        const Seq q = sequence(g, s);
        i = (int)(g.offsets ? tok - q.row0 : tok - (long long)s * g.N);
        const int j = q.pos0 + i;
        if (i < 0 || i >= q.n || j < 0 || j >= q.L) continue;
        int slot;
        const int p = page_of(g, s, j, &slot);
        if (p < 0) continue;
        const T *ks = k.at(q.b, q.row0 + i, h), *vs = v.at(q.b, q.row0 + i, h);
        T *kd = kp.at(p, slot, h), *vd = vp.at(p, slot, h);
        if (VEC) {
            constexpr int E = 16 / sizeof(T);
            for (int c = lane * E; c < g.d; c += 32 * E) *reinterpret_cast<uint4 *>(kd + c) = *reinterpret_cast<const uint4 *>(ks + c);
            for (int c = lane * E; c < g.dv; c += 32 * E) *reinterpret_cast<uint4 *>(vd + c) = *reinterpret_cast<const uint4 *>(vs + c);
        } else {
            for (int c = lane; c < g.d; c += 32) kd[c] = ks[c];
            for (int c = lane; c < g.dv; c += 32) vd[c] = vs[c];
        }
    }
}

// Rows of up to four tensors into dense ones whose heads start on 16-byte boundaries: a warp a (row, head).
struct Repack {
    Heads<const bf16> from[4];
    bf16 *to[4];
    int heads[4], width[4], pitch[4], first[5];      // first: (row, head) pairs of the tensors before, divided by the rows
    int count;
};
__global__ void __launch_bounds__(256) attn_repack_kernel(const Repack x, int N, long long rows)
{
    const int lane = threadIdx.x & 31;
    const long long all = rows * x.first[x.count];
    for (long long i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < all; i += gridDim.x * 8ll) {
        int k = 0;
        while (k + 1 < x.count && i >= rows * x.first[k + 1]) ++k;
        const long long j = i - rows * x.first[k], r = j / x.heads[k], b = r / N;
        const int h = (int)(j - r * x.heads[k]);
        const bf16 *s = x.from[k].at(b, r - b * N, h);
        bf16 *d = x.to[k] + j * x.pitch[k];
        for (int c = lane; c < x.width[k]; c += 32) d[c] = s[c];
    }
}

unsigned row_blocks(long long rows) { return (unsigned)std::min<long long>((rows + 7) / 8, SMS * 16); }

// ------------------------------------------------------------------ checks
// One of [B][N][heads][width]: aligned to its elements, strides that are not negative; outputs' rows apart.
bool heads_ok(const gma_heads_t &r, int dtype, long long B, long long N, long long heads, long long width, bool out)
{
    if (!r.ptr || ((uintptr_t)r.ptr & (blk::elem_size(dtype) - 1)) || r.batch < 0 || r.token < 0 || r.head < 0) return false;
    if (!out) return true;
    // each stride that is used steps over the extent of the smaller ones
    struct Dim { long long size, stride; } dims[3] = {{heads, r.head}, {N, r.token}, {B, r.batch}};
    std::sort(dims, dims + 3, [](const Dim &x, const Dim &y) { return x.stride < y.stride; });
    long long extent = width;
    for (const Dim &m : dims) {
        if (m.size <= 1) continue;
        if (m.stride < extent) return false;
        extent += (m.size - 1) * m.stride;
    }
    return true;
}

bool heads_vec(const gma_heads_t &r, int dtype)
{
    const size_t e = blk::elem_size(dtype);
    return (((uintptr_t)r.ptr | (uintptr_t)(r.batch * e) | (uintptr_t)(r.token * e) | (uintptr_t)(r.head * e)) & 15u) == 0;
}

gma_status_t check_sizes(const gma_attn_t *a, uint32_t flags)
{
    if (!a || a->reserved || (a->flags & ~flags)) return GMA_ERR_INVALID_ARG;
    if (a->B < 1 || a->N < 1 || a->H < 1 || a->G < 1 || a->d < 1 || a->dv < 1 || a->H % a->G) return GMA_ERR_INVALID_ARG;
    if (a->dtype != GMA_BF16 && a->dtype != GMA_F32) return GMA_ERR_INVALID_ARG;
    if (!(a->scale >= 1e-12f) || !(a->scale <= 1e12f)) return GMA_ERR_INVALID_ARG;
    if (a->lengths && a->offsets) return GMA_ERR_INVALID_ARG;
    if (!blk::opt_ok(a->lengths, 4) || !blk::opt_ok(a->offsets, 4) || !blk::opt_ok(a->lse, 4)) return GMA_ERR_INVALID_ARG;
    if (a->d > 128 || a->dv > 128 || a->H > 4096 || a->B > 65535) return GMA_ERR_UNSUPPORTED_SHAPE;
    const long long rows = (a->offsets ? 1 : (long long)a->B) * a->N;
    if (rows > (1 << 28) || rows * a->H > (1ll << 34)) return GMA_ERR_UNSUPPORTED_SHAPE;       // tiles times heads stay below 2^31
    return GMA_OK;
}

// Batch rows that the tensors have.
long long batches(const gma_attn_t &a) { return a.offsets ? 1 : a.B; }

gma_status_t check(const gma_attn_t *a, bool out)
{
    gma_status_t r = check_sizes(a, GMA_ATTN_CAUSAL | GMA_ROWS_ZERO_TAIL | GMA_FLAG_TEST_WITHHOLD);
    if (r != GMA_OK) return r;
    const long long B = batches(*a), N = a->N;
    if (!heads_ok(a->q, a->dtype, B, N, a->H, a->d, false) || !heads_ok(a->k, a->dtype, B, N, a->G, a->d, false) ||
        !heads_ok(a->v, a->dtype, B, N, a->G, a->dv, false) || !heads_ok(a->o, a->dtype, B, N, a->H, a->dv, out))
        return GMA_ERR_INVALID_ARG;
    return GMA_OK;
}

gma_status_t check_grad(const gma_attn_grad_t *g)
{
    if (!g) return GMA_ERR_INVALID_ARG;
    const gma_attn_t &a = g->fwd;
    gma_status_t r = check(&a, false);
    if (r != GMA_OK) return r;
    const long long B = batches(a), N = a.N;
    if (!a.lse || !heads_ok(g->d_o, a.dtype, B, N, a.H, a.dv, false) || !heads_ok(g->dq, a.dtype, B, N, a.H, a.d, true) ||
        !heads_ok(g->dk, a.dtype, B, N, a.G, a.d, true) || !heads_ok(g->dv, a.dtype, B, N, a.G, a.dv, true))
        return GMA_ERR_INVALID_ARG;
    return GMA_OK;
}

// `attend`: q and o are used, otherwise k and v.
gma_status_t check_paged(const gma_attn_paged_t *p, bool attend)
{
    if (!p || p->reserved) return GMA_ERR_INVALID_ARG;
    const gma_attn_t &a = p->attn;
    gma_status_t r = check_sizes(&a, GMA_ROWS_ZERO_TAIL | GMA_FLAG_TEST_WITHHOLD);
    if (r != GMA_OK) return r;
    if (p->pages < 1 || p->page < 1 || p->table_pages < 1 || p->table_stride < 0) return GMA_ERR_INVALID_ARG;
    if (!blk::ptr_ok(p->table, 4) || !blk::ptr_ok(p->cached, 4)) return GMA_ERR_INVALID_ARG;
    if (p->page > 65536 || (long long)p->pages * p->page >= (1ll << 40) || (long long)p->table_pages * p->page > (1 << 28))
        return GMA_ERR_UNSUPPORTED_SHAPE;
    const long long B = batches(a), N = a.N;
    if (!heads_ok(p->k_pages, a.dtype, p->pages, p->page, a.G, a.d, !attend) ||
        !heads_ok(p->v_pages, a.dtype, p->pages, p->page, a.G, a.dv, !attend))
        return GMA_ERR_INVALID_ARG;
    if (attend && (!heads_ok(a.q, a.dtype, B, N, a.H, a.d, false) || !heads_ok(a.o, a.dtype, B, N, a.H, a.dv, true)))
        return GMA_ERR_INVALID_ARG;
    if (!attend && (!heads_ok(a.k, a.dtype, B, N, a.G, a.d, false) || !heads_ok(a.v, a.dtype, B, N, a.G, a.dv, false)))
        return GMA_ERR_INVALID_ARG;
    return GMA_OK;
}

}  // namespace

Geo geo_of(const gma_attn_t &a, const gma_attn_paged_t *p)
{
    Geo g = {};
    g.B = a.B; g.N = a.N; g.H = a.H; g.G = a.G; g.group = a.H / a.G; g.d = a.d; g.dv = a.dv;
    g.causal = p || (a.flags & GMA_ATTN_CAUSAL);
    g.scale = a.scale;
    g.sl2 = a.scale * LOG2E;
    g.lengths = a.lengths; g.offsets = a.offsets;
    if (p) {
        g.cached = p->cached; g.table = p->table; g.table_stride = p->table_stride;
        g.table_pages = p->table_pages; g.page = p->page; g.pages = p->pages;
    }
    return g;
}

Plan make_plan(const gma_attn_t &a, int pack, int wide_rows, int narrow_rows, int key_shift, int blocks, bool cut, Carve *ws)
{
    Plan p = {};
    p.withhold = (a.flags & GMA_FLAG_TEST_WITHHOLD) != 0;
    p.pack = pack;
    p.heads = a.H / pack;
    p.narrow = std::max(narrow_rows / pack, 1);
    p.wide = p.narrow * (wide_rows / narrow_rows);
    p.key_shift = key_shift;
    p.blocks = blocks;
    // tiles of n rows and of every sequence's last rows; wide tiles are the fewer
    const long long n = (long long)a.N * batches(a);
    long long narrow = n / p.narrow + a.B, wide = n / p.wide + a.B;
    // narrow ones are taken where the wide ones are fewer than the SMs, so that they are at most twice as many and one
    const long long most = std::max(wide, std::min(narrow, (long long)(wide_rows / narrow_rows + 1) * (SMS / p.heads + 1)));
    // the call's work is `blocks` shares and a part at least half of one; items longer than a part make at most twice as many
    const long long extra = cut ? 4ll * blocks / p.heads + 2 : 0;
    p.max_items = (int)(most + extra);
    p.max_slots = (int)extra;
    p.rows = std::min(p.wide, a.N) * pack;          // a tile does not span sequences (packed: N rows in all)
    p.head_at = ws->take(sizeof(PlanHead));
    p.items_at = ws->take((size_t)p.max_items * sizeof(Item));
    p.join_at = ws->take((size_t)p.max_slots * sizeof(Join));
    p.stat_at = ws->take((size_t)p.max_slots * p.heads * p.rows * 2 * sizeof(float));
    p.part_at = ws->take((size_t)p.max_slots * p.heads * p.rows * ((a.dv + 3) & ~3) * sizeof(float));
    return p;
}

PlanArgs plan_args(const Geo &g, const Plan &p, void *ws)
{
    char *w = (char *)ws;
    // a part's cost, in key tiles: its chain into the join and its rows (1 and 3 for the first, 2 as it is: 32 single tokens over up to 2048, 8 heads
    // of 64: 32.7, 30.5 and 30.5 us)
    const float part_cost = 2.f + p.rows / 64.f;
    return PlanArgs{g, p.wide, p.narrow, p.key_shift, p.blocks, p.heads, p.max_items, p.max_slots, p.by_keys, part_cost, (WsHeader *)ws,
                    (PlanHead *)(w + p.head_at), (Item *)(w + p.items_at), (Join *)(w + p.join_at), p.withhold};
}

gma_status_t launch_plan(const PlanArgs &a, const PlanArgs *second, cudaStream_t st)
{
    GMA_LAUNCH(KID_ATTN_PLAN, st, launch_pdl(plan_kernel, second ? 2 : 1, PT, 0, st, a, second ? *second : a));
    return GMA_OK;
}

gma_status_t launch_join(const gma_attn_t &a, const Geo &g, const Plan &p, void *ws, cudaStream_t st)
{
    const char *w = (const char *)ws;
    const PlanHead *head = (const PlanHead *)(w + p.head_at);
    const Join *join = (const Join *)(w + p.join_at);
    const Parts parts = parts_of(p, a, ws);
    // as many rows as there may be in the parts
    const unsigned blocks = (unsigned)std::min<long long>(((long long)p.max_slots / 2 * p.heads * p.rows + 7) / 8, 4 * SMS);
    if (a.dtype == GMA_BF16)
        GMA_LAUNCH(KID_ATTN_JOIN, st, launch_pdl(attn_join_kernel<bf16>, blocks, 256, 0, st, g, head, join, parts, heads_of<bf16>(a.o), a.lse, p.pack));
    else
        GMA_LAUNCH(KID_ATTN_JOIN, st, launch_pdl(attn_join_kernel<float>, blocks, 256, 0, st, g, head, join, parts, heads_of<float>(a.o), a.lse, p.pack));
    return GMA_OK;
}

// An estimate of the time in steps, by sequences of equal length: the longest block's, or an SM's share of this kernel's and dq's (three quarters of
// it), whose blocks fill the gaps; pieces add the sums' stores and loads and a launch.  us of a backward pass without and with pieces, bf16, causal:
// 1 x 2048 x 16 heads of 128 over 2 187 and 75, 1 x 4096 x 16 of 64 over 1 574 and 142, 1 x 8192 x 16 of 128 over 2 851 and 606,
// 1 x 4096 x 16 of 128 over 4 233 and 194, fp32 5 x 200 x 4 of 48 over 2 60 and 39; not taken for 1 x 2048 x 16 of 128 over 8: 67 and 81.
PiecePlan plan_pieces(const gma_attn_t &a, int tile, int step, double step_us, Carve *ws)
{
    const int group = a.H / a.G;
    const long long rows = batches(a) * a.N, n = a.offsets ? (a.N + a.B - 1) / a.B : a.N, tiles = (n + tile - 1) / tile * a.B * a.G;
    const double steps = (double)((n + step - 1) / step), longest = steps * group;
    const double share = 1.75 * (a.flags & GMA_ATTN_CAUSAL ? (steps + 1) / 2 : steps) * group * tiles / SMS;
    const int width = ((a.d + 3) & ~3) + ((a.dv + 3) & ~3);
    PiecePlan p = {1, 0, 0};
    double best = std::max(longest, share) + 2;
    for (int c = 2; c <= std::min(group, 64); ++c) {
        if (group % c) continue;
        const double time = std::max(longest / c + 2, share + (tiles * c > SMS ? longest / c / 24 : 0.)) +
                            (6 + (double)(rows * a.G * c * width) * 8 / 3e6) / step_us;
        if (time < best) {
            best = time;
            p.count = c;
        }
    }
    if (p.count == 1) return p;
    p.k_at = ws->take((size_t)p.count * a.G * rows * ((a.d + 3) & ~3) * sizeof(float));
    p.v_at = ws->take((size_t)p.count * a.G * rows * ((a.dv + 3) & ~3) * sizeof(float));
    return p;
}

Pieces pieces_of(const PiecePlan &p, const gma_attn_t &a, void *ws)
{
    return Pieces{p.count, (float *)((char *)ws + p.k_at), (float *)((char *)ws + p.v_at), (a.d + 3) & ~3, (a.dv + 3) & ~3, a.G, batches(a) * a.N};
}

gma_status_t launch_pieces(const gma_attn_grad_t &g, const Pieces &p, cudaStream_t st)
{
    if (p.count == 1) return GMA_OK;
    const gma_attn_t &a = g.fwd;
    const Geo geo = geo_of(a, nullptr);
    const unsigned blocks = row_blocks(p.rows * a.G);
    if (a.dtype == GMA_BF16)
        GMA_LAUNCH(KID_ATTN_PIECES, st, launch_pdl(attn_pieces_kernel<bf16>, blocks, 256, 0, st, geo, p, heads_of<bf16>(g.dk), heads_of<bf16>(g.dv)));
    else
        GMA_LAUNCH(KID_ATTN_PIECES, st, launch_pdl(attn_pieces_kernel<float>, blocks, 256, 0, st, geo, p, heads_of<float>(g.dk), heads_of<float>(g.dv)));
    return GMA_OK;
}

gma_status_t launch_delta(const gma_attn_grad_t &g, float *delta, cudaStream_t st)
{
    const gma_attn_t &a = g.fwd;
    const Geo geo = geo_of(a, nullptr);
    const long long rows = batches(a) * a.H * a.N;
    const bool vec = a.dv % 8 == 0 && heads_vec(a.o, a.dtype) && heads_vec(g.d_o, a.dtype);
    // rows of no sequence in the gradients: none to clear, element by element, 16 bytes at a time
    const int e16 = 16 / (int)blk::elem_size(a.dtype);
    const int zero = !((a.flags & GMA_ROWS_ZERO_TAIL) && (a.lengths || a.offsets)) ? 0
                     : a.d % e16 == 0 && a.dv % e16 == 0 && heads_vec(g.dq, a.dtype) && heads_vec(g.dk, a.dtype) && heads_vec(g.dv, a.dtype) ? 2 : 1;
    // rows that see few keys: the first of causal sequences, all of short ones
    FewArgs few = {heads_of<const bf16>(a.q), heads_of<const bf16>(a.k), heads_of<const bf16>(a.v), a.lse, 0, 0};
    if (a.dtype == GMA_BF16 && (geo.causal || a.N <= FEW || a.lengths || a.offsets)) {
        auto even = [](const gma_heads_t &x) { return (((uintptr_t)x.ptr | (uintptr_t)(x.batch * 2) | (uintptr_t)(x.token * 2) | (uintptr_t)(x.head * 2)) & 3u) == 0; };
        few.blocks = (unsigned)std::min<long long>(((long long)a.B * a.H + 7) / 8, SMS * 16);
        few.pairs = a.d % 2 == 0 && a.dv % 2 == 0 && even(a.q) && even(a.k) && even(a.v) && even(g.d_o);
    }
    auto launch = [&](auto type, auto v, auto lanes) -> gma_status_t {
        using T = decltype(type);
        constexpr int LANES = decltype(lanes)::value;
        const unsigned blocks = few.blocks + (unsigned)std::min<long long>((rows + 256 / LANES - 1) / (256 / LANES), SMS * 32);
        GMA_LAUNCH(KID_ATTN_DELTA, st, launch_pdl(attn_delta_kernel<T, decltype(v)::value, LANES>, blocks, 256, 0, st, geo, heads_of<const T>(a.o),
                                                  heads_of<const T>(g.d_o), delta, rows, heads_of<T>(g.dq), heads_of<T>(g.dk), heads_of<T>(g.dv),
                                                  zero, few));
        return GMA_OK;
    };
    using Yes = std::true_type;
    using No = std::false_type;
    if (!vec)
        return a.dtype == GMA_BF16 ? launch(bf16(), No(), std::integral_constant<int, 32>()) : launch(float(), No(), std::integral_constant<int, 32>());
    if (a.dv <= 64)
        return a.dtype == GMA_BF16 ? launch(bf16(), Yes(), std::integral_constant<int, 8>()) : launch(float(), Yes(), std::integral_constant<int, 8>());
    return a.dtype == GMA_BF16 ? launch(bf16(), Yes(), std::integral_constant<int, 16>()) : launch(float(), Yes(), std::integral_constant<int, 16>());
}

// bf16 calls on whole sequences whose rows TMA cannot read: dense copies in the workspace, behind what the kernels take of it.
namespace {

struct Packed {
    gma_heads_t q, k, v, d_o;
    size_t bytes;
};

Packed pack_places(const gma_attn_t &a, bool grad, size_t at, void *ws)
{
    Packed p = {};
    const int64_t rows = batches(a) * a.N;
    size_t off = align_up(at, 256);
    auto take = [&](int heads, int width) {
        const int64_t pitch = (width + 7) & ~7;
        const gma_heads_t h = {(char *)ws + off, a.N * (heads * pitch), heads * pitch, pitch};      // 64 bits from the first product on
        off = align_up(off + (size_t)(rows * heads * pitch) * sizeof(bf16), 256);
        return h;
    };
    p.q = take(a.H, a.d);
    p.k = take(a.G, a.d);
    p.v = take(a.G, a.dv);
    if (grad) p.d_o = take(a.H, a.dv);
    p.bytes = off;
    return p;
}

gma_status_t launch_repack(const gma_attn_t &a, const gma_heads_t *d_o, const Packed &p, cudaStream_t st)
{
    Repack x = {};
    auto add = [&](const gma_heads_t &from, const gma_heads_t &to, int heads, int width) {
        const int k = x.count++;
        x.from[k] = heads_of<const bf16>(from);
        x.to[k] = (bf16 *)to.ptr;
        x.heads[k] = heads;
        x.width[k] = width;
        x.pitch[k] = (int)to.head;
        x.first[k + 1] = x.first[k] + heads;
    };
    add(a.q, p.q, a.H, a.d);
    add(a.k, p.k, a.G, a.d);
    add(a.v, p.v, a.G, a.dv);
    if (d_o) add(*d_o, p.d_o, a.H, a.dv);
    const long long rows = batches(a) * a.N;
    GMA_LAUNCH(KID_ATTN_REPACK, st, attn_repack_kernel<<<row_blocks(rows * x.first[x.count]), 256, 0, st>>>(x, a.N, rows));
    return GMA_OK;
}

gma_attn_t with(const gma_attn_t &a, const Packed &p)
{
    gma_attn_t b = a;
    b.q = p.q;
    b.k = p.k;
    b.v = p.v;
    return b;
}

// Copies cost a launch and the rows' bytes, the CUDA cores' products more than that from some scores on.  Both sides, forward and backward
// in us: 2 x 128 x 8 heads of 63 (2.6e5) 23 and 46 with copies, 20 and 46 without; 2 x 256 x 8 (1e6) 27 and 50 against 31 and 77;
// 4 x 2048 x 8 of 117 170 and 403 against 1314 and 6391.
bool repacks(const gma_attn_t &a)
{
    return a.dtype == GMA_BF16 && (double)batches(a) * a.N * a.N * a.H >= REPACK_FROM;
}

}  // namespace

}  // namespace att
}  // namespace gma

using namespace gma;
using namespace gma::att;

extern "C" {

size_t gma_attn_workspace_size(const gma_attn_t *a)
{
    if (check(a, true) != GMA_OK) return 0;
    if (tc_takes(*a, nullptr)) return tc_workspace(*a, nullptr);
    return repacks(*a) ? pack_places(*a, false, tc_workspace(*a, nullptr), nullptr).bytes : simt_workspace(*a, nullptr);
}

gma_status_t gma_attn_forward(const gma_attn_t *a, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    gma_status_t r = check(a, true);
    if (r != GMA_OK) return r;
    if (!blk::ws_ok(ws, ws_bytes, gma_attn_workspace_size(a))) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    if (tc_takes(*a, nullptr)) return tc_forward(*a, nullptr, ws, st);
    if (!repacks(*a)) return simt_forward(*a, nullptr, ws, st);
    const Packed p = pack_places(*a, false, tc_workspace(*a, nullptr), ws);
    if ((r = launch_repack(*a, nullptr, p, st)) != GMA_OK) return r;
    return tc_forward(with(*a, p), nullptr, ws, st);
}

size_t gma_attn_backward_workspace_size(const gma_attn_grad_t *g)
{
    if (check_grad(g) != GMA_OK) return 0;
    if (tc_takes_backward(*g)) return tc_backward_workspace(*g);
    return repacks(g->fwd) ? pack_places(g->fwd, true, tc_backward_workspace(*g), nullptr).bytes : simt_backward_workspace(*g);
}

gma_status_t gma_attn_backward(const gma_attn_grad_t *g, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    gma_status_t r = check_grad(g);
    if (r != GMA_OK) return r;
    if (!blk::ws_ok(ws, ws_bytes, gma_attn_backward_workspace_size(g))) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const gma_attn_t &a = g->fwd;
    if (tc_takes_backward(*g)) return tc_backward(*g, ws, st);
    if (!repacks(a)) return simt_backward(*g, ws, st);
    const Packed p = pack_places(a, true, tc_backward_workspace(*g), ws);
    if ((r = launch_repack(a, &g->d_o, p, st)) != GMA_OK) return r;
    gma_attn_grad_t packed = *g;
    packed.fwd = with(a, p);
    packed.d_o = p.d_o;
    return tc_backward(packed, ws, st);
}

gma_status_t gma_attn_append(const gma_attn_paged_t *p, gma_stream_t stream)
{
    gma_status_t r = check_paged(p, false);
    if (r != GMA_OK) return r;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    const gma_attn_t &a = p->attn;
    const Geo g = geo_of(a, p);
    const long long rows = batches(a) * a.N * a.G;
    const int e = 16 / (int)blk::elem_size(a.dtype);
    const bool vec = a.d % e == 0 && a.dv % e == 0 && heads_vec(a.k, a.dtype) && heads_vec(a.v, a.dtype) && heads_vec(p->k_pages, a.dtype) &&
                     heads_vec(p->v_pages, a.dtype);
    auto launch = [&](auto type, auto v) -> gma_status_t {
        using T = decltype(type);
        GMA_LAUNCH(KID_ATTN_APPEND, st, attn_append_kernel<T, decltype(v)::value><<<row_blocks(rows), 256, 0, st>>>(
                                            g, heads_of<const T>(a.k), heads_of<const T>(a.v), heads_of<T>(p->k_pages), heads_of<T>(p->v_pages), rows));
        return GMA_OK;
    };
    if (a.dtype == GMA_BF16)
        return vec ? launch(__nv_bfloat16(), std::true_type()) : launch(__nv_bfloat16(), std::false_type());
    return vec ? launch(float(), std::true_type()) : launch(float(), std::false_type());
}

size_t gma_attn_paged_workspace_size(const gma_attn_paged_t *p)
{
    return check_paged(p, true) != GMA_OK ? 0 : tc_takes(p->attn, p) ? tc_workspace(p->attn, p) : simt_workspace(p->attn, p);
}

gma_status_t gma_attn_paged(const gma_attn_paged_t *p, void *ws, size_t ws_bytes, gma_stream_t stream)
{
    gma_status_t r = check_paged(p, true);
    if (r != GMA_OK) return r;
    if (!blk::ws_ok(ws, ws_bytes, gma_attn_paged_workspace_size(p))) return GMA_ERR_WORKSPACE;
    if ((r = usable_device()) != GMA_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    if (tc_takes(p->attn, p)) return tc_forward(p->attn, p, ws, st);
    return simt_forward(p->attn, p, ws, st);
}

}  // extern "C"
