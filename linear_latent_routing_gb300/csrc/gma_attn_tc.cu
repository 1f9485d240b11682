// gma_attn_tc.cu -- softmax attention on the tensor cores (tcgen05), bf16: whole sequences, and new tokens over a cache of pages.
//
// A block runs two streams of 128 query rows against key tiles of 128, each with its scores and its output in tensor
// memory (S0 S1 O0 O1, 512 columns): while one stream's warps take exponentials the tensor cores work for the other.
// An item of more than 128 rows gives each stream its own rows, and both read every key tile; an item of fewer (few new
// tokens) gives both the same rows and each every other key tile, and their results are joined in shared memory at the end.
// Keys and values pass through one ring of tiles.  P, rounded to bf16 (half a step, 2^-8 relative, which leaves the result's
// own rounding as large; its sum is taken before that, in fp32), replaces S in tensor memory as the second product's
// first operand.  The maximum that the exponentials are relative to is moved only when it would grow by more than 2^8, so that
// the output is rarely rescaled: fp32 sums do not mind the factor, and bf16 holds p at any scale.
//
// Blocks stay, one an SM, and take items from the plan's list, the largest first: the next item's queries and keys are on their way while the
// last rows of one are written.
//
// Warps: 0-3 and 4-7 the streams (a thread a row), 8 issues the products, 9 loads, 10 and 11 write zeros where rows belong to no sequence.
//
// Measured, calls one after another: 32768 tokens, 16 heads of 128 over 4, causal 2.71 ms for seconds on end (1620 TFLOP/s; the power limit lowers
// the clock to 1.9 GHz), 2.57 for some of them (1710), 8192 tokens 201 us (1370; the kernel alone 189, tensor pipe 64 % busy), 4 x 4096 x 16 heads of 64
// 179 us (770; at 8192 tokens tensor pipe 40 %, exponentials' pipe 37 %).  At 128 columns the
// products' warp and the two streams' turns bound it, at 64 the turn of a stream as such: wait, load, maximum, 128 exponentials a thread,
// store, hand over, which two streams do not cover when the products take half as long.  64 sequences x 8192 cached tokens in pages of 128: 6.2
// TB/s in the kernel (5.6 the call from a cold cache); pages of 16 cost 6 to 17 % (boxes of 2 KB).
#include "attn_tc.cuh"
#include "attn_tc_host.cuh"

namespace gma {

namespace tck {
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                  const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();
}  // namespace tck

namespace att {
namespace {

constexpr int THREADS = 384;
constexpr int MAX_SLOTS = 10;
constexpr float GROW = 8.f;                  // by so much (in powers of two) the maximum may lag

struct TcArgs {
    Geo g;
    Heads<bf16> o;
    float *lse;
    int pack, heads;           // query heads in a row tile, heads of the grid
    int o_vec;
    int zero_rows;             // of o, to be looked through for such as belong to no sequence (0: none)
    PlanHead *head;
    const Item *items;
    Parts parts;
    WsHeader *hdr;
    int q_boxes, v_boxes;      // boxes of 64 columns of q and k, of v
    uint32_t slot_bytes;
    int slots;
    int page_rows, tile_pages; // rows of a page's box, such boxes in a tile
    int page_shift;            // pages are powers of two
    int withhold;              // GMA_FLAG_TEST_WITHHOLD: a block's first tile of keys is never loaded
};

// An item of one head as its block's warps see it.
struct Job {
    Seq sq;
    int seq, tok0, tokens;     // sequence, first token, tokens (0: no more jobs)
    int t0, t1, e0;            // key tiles, and where stream 0's end if it has rows of its own
    int two;                   // each stream has its own rows
    int head, kvh;
    int slot, parts, part;
};

// shared memory: query tiles, the ring, the barriers
struct Bars {
    uint64_t q, q_free, full[MAX_SLOTS], empty[MAX_SLOTS], s[2], p[2], o[2], job[2], job_free[2], sync, drain;
    uint32_t tmem;
    int abort;
    Job jobs[2];
    float merge[TILE][2];
};

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// exp2(s sl2 - m) of a row's scores as bf16 pairs into tensor memory, and their sums in fp32.
__device__ __forceinline__ void exponentials(const uint32_t (&r)[4][32], uint32_t ts, float sl2, float m, blk::f2 (&sum)[2])
{
    const float base = m == -INFINITY ? 0.f : -m;
    const blk::f2 scale = blk::pack2(sl2, sl2), shift = blk::pack2(base, base);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const blk::f2 y =
                blk::ex2_2(blk::fma2(blk::pack2(__uint_as_float(r[c][2 * e]), __uint_as_float(r[c][2 * e + 1])), scale, shift));
            sum[e & 1] = blk::add2(sum[e & 1], y);
            const float2 z = blk::unpack2(y);
            p[e] = pack_bf16(z.x, z.y);
        }
        tmem_st16(ts + 16 * c, p);
    }
}

template <bool PAGED>
__global__ void __launch_bounds__(THREADS, 1) attn_tc_kernel(const TcArgs a, const __grid_constant__ CUtensorMap qmap,
                                                             const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t q_tile = (uint32_t)a.q_boxes * BOX;
    uint8_t *ring = smem + 2 * q_tile;
    Bars *bars = reinterpret_cast<Bars *>(ring + (size_t)a.slots * a.slot_bytes);
    volatile int *abort = &bars->abort;
    // the warp's number and what its roles go by as values that the compiler knows to be uniform: the products' operands then stay in uniform
    // registers, and their warp gets by with fewer issue slots beside the streams' (32768-token prompt 2818 -> 2701 us)
    const int t = threadIdx.x, warp = __shfl_sync(~0u, t >> 5, 0), lane = t & 31;
    if (t == 256) {
        mbar_init(&bars->q, 1);
        mbar_init(&bars->q_free, 1);
        for (int i = 0; i < a.slots; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&bars->s[w], 1);
            mbar_init(&bars->p[w], TILE);
            mbar_init(&bars->o[w], 1);
            mbar_init(&bars->job[w], 1);
            mbar_init(&bars->job_free[w], 9);
        }
        mbar_init(&bars->sync, 256);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&bars->tmem, 512);
    if (t == 288) {
        prefetch_map(&qmap);
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, bars->tmem, 0);
    const uint32_t sb = smem_u32(smem), rb = smem_u32(ring);
    const Geo &g = a.g;
    const int pack = a.pack, per = TILE / pack;                  // tokens of a row tile
    int js = 0;                                                  // the job at hand, and the parity of its turn
    uint32_t jt = 0;

    if (warp == 8) {
        // ================================================================ products
        reg_dec<88>();
        const uint32_t id_s = idesc_f16(TILE, TILE, 1, 1, 0, 0), id_o = idesc_f16(TILE, (uint32_t)(g.dv + 15) & ~15u, 1, 1, 0, 1);
        const int ksteps = (g.d + 15) >> 4;
        const uint64_t q_desc = k_desc(sb);
        bool ok = true;
        uint32_t turn[2] = {0, 0}, qt = 0;         // parities of the streams' tiles and of the query tiles
        RingPos v{1, 0}, kb{0, 0};
        while ((ok = bar_wait(&bars->job[js], jt, a.hdr, 210, abort))) {
            const Job &job = bars->jobs[js];
            if (!job.tokens) break;
            const int t0 = __shfl_sync(~0u, job.t0, 0), t1 = __shfl_sync(~0u, job.t1, 0), e0 = __shfl_sync(~0u, job.e0, 0), L = __shfl_sync(~0u, job.sq.L, 0);
            const bool two = __shfl_sync(~0u, job.two, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->job_free[js]);
            js ^= 1;
            if (!js) jt ^= 1u;
            if (t1 <= t0) continue;
            if (!(ok = bar_wait(&bars->q, qt, a.hdr, 200, abort))) break;
            qt ^= 1u;
            bool begun[2] = {false, false};
            const uint64_t q_next = two ? q_tile >> 4 : 0;
            const int step = two ? 1 : 2;
            auto loaded = [&](const RingPos &r) { return bar_wait(&bars->full[r.s], r.turn, a.hdr, 201, abort); };
            // S_w = Q_w K^T; after a tile's last one it is given back, after the job's last one the queries too
            auto put_scores = [&](int w, const RingPos &k, bool last, int kt) {
                mma_tiles(tmem + w * TILE, q_desc + (w ? q_next : 0), k_desc(rb + (uint32_t)k.s * a.slot_bytes), id_s, ksteps);
                mma_commit(&bars->s[w]);
                if (last) {
                    mma_commit(&bars->empty[k.s]);
                    if (kt + 1 == t1) mma_commit(&bars->q_free);
                }
            };
            auto scores = [&](int w, const RingPos &k, bool last, int kt) {
                if (elect()) put_scores(w, k, last, kt);
            };
            // O_w += P_w V
            auto put_output = [&](int w, const RingPos &v, bool last) {
                const uint64_t desc = mn_desc(rb + (uint32_t)v.s * a.slot_bytes);
                const uint32_t p = tmem + w * TILE, o = tmem + 256 + w * TILE;
#pragma unroll
                for (int s = 0; s < TILE / 16; ++s) mma_f16_tmem_a(o, p + 8 * s, desc + mn_step(s), id_o, s > 0 || begun[w]);
                if (last) mma_commit(&bars->empty[v.s]);
            };
            // the keys that the next scores take
            RingPos k = kb;
            if (!(ok = loaded(k))) break;
            if (t0 < e0) scores(0, k, !two, t0);
            if (two) scores(1, k, true, t0);
            k.step(2, a.slots);
            if (!two) {
                if (t0 + 1 < t1) {
                    if (!(ok = loaded(k))) break;
                    scores(1, k, true, t0 + 1);
                }
                k.step(2, a.slots);
            }
            bool go = true;                        // a lane's own waits have not given up
            for (int kt = t0; kt < t1; ++kt) {
                const int next = kt + step, have = L - kt * TILE;
                bool v_there = false, k_there = false;
                // values behind the sequence's end meet probabilities of zero, and may be anything
                if (have < TILE) {
                    if (!(ok = loaded(v))) break;
                    zero_rows(ring + (size_t)v.s * a.slot_bytes, a.v_boxes, have);
                    v_there = true;
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (two ? w == 0 && kt >= e0 : w != ((kt - t0) & 1)) continue;
                    const bool last = !two || w == 1, more = next < (two && w == 0 ? e0 : t1);
                    // A barrier that is through costs some 80 cycles to find so, and this warp's time is what bounds the loop: the three that the
                    // products wait for are asked at once.  Keys that are not there yet do not keep the first product.  Every lane asks and waits
                    // for itself, and all of them meet at elect(), whatever they were told; the elected one goes by its own answers.  (A vote on the
                    // answers: 32768-token prompt 2940 us, of all three at once 2846, without 2690.)
                    const bool p_now = mbar_test_wait(&bars->p[w], turn[w]);
                    const bool v_now = v_there || mbar_test_wait(&bars->full[v.s], v.turn);
                    const bool k_now = !more || k_there || mbar_test_wait(&bars->full[k.s], k.turn);
                    go = go && (v_now || lane_wait(&bars->full[v.s], v.turn, a.hdr, 201, abort));
                    go = go && (p_now || lane_wait(&bars->p[w], turn[w], a.hdr, 202, abort));
                    tc_fence_after();
                    if (elect() && go) {
                        put_output(w, v, last);
                        if (!more) mma_commit(&bars->o[w]);
                        else if (k_now || lane_wait(&bars->full[k.s], k.turn, a.hdr, 201, abort)) put_scores(w, k, last, next);
                    }
                    v_there = true;
                    k_there = k_there || more;
                    begun[w] = true;
                    turn[w] ^= 1u;
                }
                v.step(2, a.slots);
                k.step(2, a.slots);
                kb.step(2, a.slots);
            }
            ok = ok && !aborted(abort);
            if (!ok) break;
        }
        // after a wait that gave up: products in flight end before their operands and results go
        if (aborted(abort)) {
            if (elect()) mma_commit(&bars->drain);
            mbar_wait(&bars->drain, 0, a.hdr, 209);
        }
    } else if (warp == 9) {
        // ================================================================ jobs and loads
        reg_dec<88>();
        blk::wait_previous();
        if (PAGED) blk::let_next();
        Item it = load_item(a.items + blockIdx.x / a.heads);       // beside the number of items: the list has a place for every block's first
        const int all = a.head->items * a.heads, tile_tokens = a.head->tokens;
        bool ok = true;
        int issued = 0, queries = 0;
        RingPos r{0, 1};
        uint32_t qt = 1;
        jt = 1;
        int ticket = blockIdx.x;                   // the plan's counter starts behind these
        while (true) {
            Job job;
            job.tokens = 0;
            if (ticket < all) {
                const int rank = ticket / a.heads;
                job.head = ticket - rank * a.heads;
                job.sq = it.sq;
                job.seq = it.seq;
                job.tok0 = it.tok0;
                job.tokens = min(tile_tokens, job.sq.n - it.tok0);
                job.two = job.tokens > per;
                job.kvh = pack == 1 ? job.head / g.group : job.head;
                job.t0 = it.t0;
                job.t1 = it.part < 0 ? it.t0 : min(it.t1, (job.sq.seen(g, it.tok0 + job.tokens - 1) + TILE - 1) / TILE);
                job.e0 = job.two ? min(job.t1, (job.sq.seen(g, it.tok0 + per - 1) + TILE - 1) / TILE) : job.t1;
                job.slot = it.slot;
                job.parts = it.parts;
                job.part = it.part;
            }
            if (!(ok = bar_wait(&bars->job_free[js], jt, a.hdr, 211, abort))) break;
            if (lane == 0) bars->jobs[js] = job;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->job[js]);
            js ^= 1;
            if (!js) jt ^= 1u;
            if (!job.tokens) break;
            const Seq &sq = job.sq;
            const int t0 = job.t0, t1 = job.t1;
            // the page of this lane's box of a tile
            auto page_entry = [&](int kt) {
                const int j = kt * TILE + lane * a.page_rows;
                if (lane >= a.tile_pages || j >= sq.L) return 0;
                return g.table[(long long)job.seq * g.table_stride + (j >> a.page_shift)];
            };
            if (t1 > t0) {
                int entry = PAGED ? page_entry(t0) : 0;
                if (!(ok = bar_wait(&bars->q_free, qt, a.hdr, 212, abort))) break;
                qt ^= 1u;
                if (lane == 0) {
                    const uint32_t box = (uint32_t)(per * pack) * 128u;
                    const int tiles = job.two ? 2 : 1;
                    mbar_arrive_expect_tx(&bars->q, box * tiles * a.q_boxes);
                    for (int w = 0; w < tiles; ++w)
                        for (int b = 0; b < a.q_boxes; ++b)
                            tma_load_4d(sb + w * q_tile + b * BOX, &qmap, &bars->q, 64 * b, job.head * pack, sq.row0 + job.tok0 + w * per, sq.b);
                }
                ++queries;
                for (int kt = t0; ok && kt < t1; ++kt) {
                    const int have = min(sq.L - kt * TILE, TILE), boxes = PAGED ? (have + a.page_rows - 1) / a.page_rows : 1;
                    const int in_page = PAGED ? (kt * TILE) & (g.page - 1) : 0;
                    const int ahead = PAGED && kt + 1 < t1 ? page_entry(kt + 1) : 0;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!(ok = bar_wait(&bars->empty[r.s], r.turn, a.hdr, 203, abort))) break;
                        const uint32_t dst = rb + (uint32_t)r.s * a.slot_bytes;
                        uint64_t *full = &bars->full[r.s];
                        const int nb = half ? a.v_boxes : a.q_boxes;
                        const CUtensorMap *map = half ? &vmap : &kmap;
                        const bool held = a.withhold && !issued;
                        if (lane == 0 && !held) mbar_arrive_expect_tx(full, PAGED ? (uint32_t)(boxes * a.page_rows * 128 * nb) : BOX * nb);
                        __syncwarp();
                        if (PAGED) {
                            // an entry that names no page: a coordinate behind the pool, which reads as zeros
                            const int page = entry >= 0 && entry < g.pages ? entry : g.pages;
                            if (lane < boxes && !held)
                                for (int b = 0; b < nb; ++b)
                                    tma_load_4d(dst + b * BOX + lane * a.page_rows * 128, map, full, 64 * b, job.kvh, in_page, page);
                        } else if (lane == 0 && !held) {
                            for (int b = 0; b < nb; ++b) tma_load_4d(dst + b * BOX, map, full, 64 * b, job.kvh, sq.row0 + kt * TILE, sq.b);
                        }
                        ++issued;
                        r.step(1, a.slots);
                    }
                    entry = ahead;
                }
                if (!ok) break;
            }
            // taken when this one's last tiles are on their way, not before: a block with a long item would hold on to a second one
            if (lane == 0) ticket = atomicAdd(&a.head->ticket, 1);
            ticket = __shfl_sync(~0u, ticket, 0);
            if (ticket < all) it = load_item(a.items + ticket / a.heads);
        }
        // loads that no product waited for (a wait gave up) end before the block does
        if (aborted(abort)) {
            if (queries) mbar_wait(&bars->q, (uint32_t)(queries - 1) & 1u, a.hdr, 204);
            for (int c = issued > a.slots ? issued - a.slots : 0; c < issued; ++c)
                mbar_wait(&bars->full[c % a.slots], (uint32_t)(c / a.slots) & 1u, a.hdr, 205);
        }
    } else if (warp < 8) {
        // ================================================================ a stream's rows (registers: 256 x 208 + 128 x 88 = 384 x 168)
        reg_inc<208>();
        const int w = warp >> 2, row = t & (TILE - 1);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + w * TILE, to = tmem + lanes + 256 + w * TILE;
        uint32_t st = 0, ot[2] = {0, 0}, yt = 0;   // parities of this stream's scores, of both streams' results, of their meetings
        auto streams_sync = [&]() {
            mbar_arrive(&bars->sync);
            const bool met = bar_wait(&bars->sync, yt, a.hdr, 214, abort);
            yt ^= 1u;
            return met;
        };
        while (bar_wait(&bars->job[js], jt, a.hdr, 213, abort)) {
            const Job &job = bars->jobs[js];
            if (!job.tokens) break;
            const bool two = job.two;
            const int tok = job.tok0 + (two ? w * per : 0) + row / pack;
            const bool valid = row < per * pack && tok < job.tok0 + job.tokens;
            const bool busy = __any_sync(~0u, valid);
            const int seen = valid ? job.sq.seen(g, tok) : job.sq.L;
            const int step = two ? 1 : 2, begin = two ? job.t0 : job.t0 + w, end = two && w == 0 ? job.e0 : job.t1;
            float m = -INFINITY;
            blk::f2 sum[2] = {blk::pack2(0.f, 0.f), blk::pack2(0.f, 0.f)};
            bool ok = true;
            int n = 0;
            for (int kt = begin; kt < end; kt += step, ++n) {
                if (!(ok = bar_wait(&bars->s[w], st, a.hdr, 206, abort))) break;
                st ^= 1u;
                tc_fence_after();
                if (busy) {
                    const int lim = seen - kt * TILE;
                    const bool edge = __any_sync(~0u, lim < TILE);
                    uint32_t r[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, r[c]);
                    tmem_ld_wait();
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * c + e >= lim) r[c][e] = 0xff800000u;
                    }
                    float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) x[c] = max3(x[c], __uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1]));
                    }
                    // (a row that does not exist holds the next sequence's queries, or what was left in shared memory: it must not move the
                    // others' maximum, by which their probabilities are rounded)
                    const float top = valid ? fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * g.sl2 : -INFINITY;
                    // the maximum that the exponentials are relative to moves rarely, and with it what was summed up so far
                    if (__any_sync(~0u, top > m + GROW)) {
                        const float now = fmaxf(m, top), f = now == -INFINITY ? 1.f : ex2(m - now);
                        m = now;
                        const blk::f2 ff = blk::pack2(f, f);
                        sum[0] = blk::mul2(sum[0], ff);
                        sum[1] = blk::mul2(sum[1], ff);
                        if (n) {
#pragma unroll 1
                            for (int c = 0; c < g.dv; c += 16) {
                                uint32_t v[16];
                                tmem_ld16(to + c, v);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                                tmem_st16(to + c, v);
                            }
                        }
                    }
                    exponentials(r, ts, g.sl2, m, sum);
                    tmem_st_wait();
                }
                tc_fence_before();
                mbar_arrive(&bars->p[w]);
            }
            if (!ok) break;
            const float2 la = blk::unpack2(blk::add2(sum[0], sum[1]));
            float l = la.x + la.y;
            const bool shared = !two && job.t1 - job.t0 > 1;        // both streams have parts of the same rows
            if (n && !bar_wait(&bars->o[w], ot[w], a.hdr, 207, abort)) break;
            if (shared && w == 0 && !bar_wait(&bars->o[1], ot[1], a.hdr, 208, abort)) break;
            if (two ? job.e0 > job.t0 : job.t1 > job.t0) ot[0] ^= 1u;
            if (two ? job.t1 > job.t0 : shared) ot[1] ^= 1u;
            tc_fence_after();
            float mine = 1.f, theirs = 0.f;                         // factors of the streams' sums
            if (shared) {
                if (w == 1) {
                    bars->merge[row][0] = m;
                    bars->merge[row][1] = l;
                }
                if (!streams_sync()) break;
                if (w == 0) {
                    const float m1 = bars->merge[row][0], l1 = bars->merge[row][1], now = fmaxf(m, m1);
                    mine = now == -INFINITY ? 0.f : ex2(m - now);
                    theirs = now == -INFINITY ? 0.f : ex2(m1 - now);
                    l = l * mine + l1 * theirs;
                    m = now;
                }
            }
            const bool whole = job.parts == 1;
            if (busy && (two || w == 0) && job.part >= 0) {
                const int h = pack == 1 ? job.head : job.head * pack + row % pack;
                const int item_row = (two ? w * per * pack : 0) + row;
                const float f = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
                mine *= f;
                theirs *= f;
                bf16 *out = a.o.at(job.sq.b, job.sq.row0 + (valid ? tok : job.tok0), h);
                float *part = whole ? nullptr : a.parts.o_at(job.slot + job.part, job.head, valid ? item_row : 0);
                if (valid) {
                    if (whole) {
                        if (a.lse) a.lse[stat_at(g, job.sq, h, tok)] = l > 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
                    } else {
                        float *stat = a.parts.stat_at(job.slot + job.part, job.head, item_row);
                        stat[0] = l > 0.f ? m : -INFINITY;
                        stat[1] = l;
                    }
                }
#pragma unroll 1
                for (int c = 0; c < g.dv; c += 32) {
                    uint32_t v[32];
                    float y[32];
                    if (n) {
                        tmem_ld32(to + c, v);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = n && mine != 0.f ? __uint_as_float(v[e]) * mine : 0.f;
                    if (shared) {
                        tmem_ld32(to + TILE + c, v);                // the other stream's rows lie in the same lanes
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = theirs != 0.f ? fmaf(__uint_as_float(v[e]), theirs, y[e]) : y[e];
                    }
                    if (!valid) continue;
                    if (!whole) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (c + 4 * q < g.dv) *reinterpret_cast<float4 *>(part + c + 4 * q) = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
                    } else if (a.o_vec) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (c + 8 * q < g.dv)
                                *reinterpret_cast<uint4 *>(out + c + 8 * q) =
                                    make_uint4(pack_bf16(y[8 * q], y[8 * q + 1]), pack_bf16(y[8 * q + 2], y[8 * q + 3]),
                                               pack_bf16(y[8 * q + 4], y[8 * q + 5]), pack_bf16(y[8 * q + 6], y[8 * q + 7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c + e < g.dv) out[c + e] = __float2bfloat16_rn(y[e]);
                    }
                }
            }
            // the next job's products over these results, and its exchange, wait for all that read this one's
            tc_fence_before();
            if (shared && !streams_sync()) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->job_free[js]);
            js ^= 1;
            if (!js) jt ^= 1u;
        }
    } else {
        reg_dec<88>();
        // the output's rows that belong to no sequence (no other kernel's results are read or written here)
        if (a.zero_rows) zero_dead_rows(g, a.o, g.H, g.dv, a.zero_rows, blockIdx.x * 2 + (warp - 10), gridDim.x * 2, a.o_vec);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

}  // namespace

// ------------------------------------------------------------------ host side
bool tma_heads(const gma_heads_t &r, long long B, long long N, long long heads)
{
    auto fits = [](long long size, long long stride) { return size <= 1 || (stride > 0 && stride % 8 == 0 && stride < (1ll << 38)); };
    return ((uintptr_t)r.ptr & 15u) == 0 && fits(heads, r.head) && fits(N, r.token) && fits(B, r.batch);
}

bool heads_map(CUtensorMap *m, const gma_heads_t &r, long long B, long long N, long long heads, int width, int bh, int bt)
{
    const tck::EncodeTiledFn fn = tck::encode_fn();
    if (!fn) return false;
    auto bytes = [](long long size, long long stride) { return (cuuint64_t)(size > 1 ? stride * 2 : 16); };
    const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)N, (cuuint64_t)B};
    const cuuint64_t strides[3] = {bytes(heads, r.head), bytes(N, r.token), bytes(B, r.batch)};
    const cuuint32_t box[4] = {64, (cuuint32_t)bh, (cuuint32_t)bt, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r.ptr, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool store_vec(const gma_heads_t &r, int width)
{
    return width % 8 == 0 && (((uintptr_t)r.ptr | (uintptr_t)(r.batch * 2) | (uintptr_t)(r.token * 2) | (uintptr_t)(r.head * 2)) & 15u) == 0;
}

namespace {

Plan plan_of(const gma_attn_t &a, const gma_attn_paged_t *paged, Carve *c)
{
    const int group = a.H / a.G, pack = paged && group <= TILE ? group : 1;
    return make_plan(a, pack, 2 * TILE, TILE, 7, SMS, paged != nullptr, c);
}

}  // namespace

bool tc_takes(const gma_attn_t &a, const gma_attn_paged_t *p)
{
    if (a.dtype != GMA_BF16) return false;
    const long long B = a.offsets ? 1 : a.B;
    if (!tma_heads(a.q, B, a.N, a.H)) return false;
    if (!p) return tma_heads(a.k, B, a.N, a.G) && tma_heads(a.v, B, a.N, a.G);
    return p->page >= 8 && (p->page & (p->page - 1)) == 0 && tma_heads(p->k_pages, p->pages, p->page, a.G) &&
           tma_heads(p->v_pages, p->pages, p->page, a.G);
}

size_t tc_workspace(const gma_attn_t &a, const gma_attn_paged_t *paged)
{
    Carve c;
    plan_of(a, paged, &c);
    return c.total();
}

gma_status_t tc_forward(const gma_attn_t &a, const gma_attn_paged_t *p, void *ws, cudaStream_t st)
{
    Carve c;
    const Plan pl = plan_of(a, p, &c);
    char *w = (char *)ws;
    TcArgs x = {};
    x.g = geo_of(a, p);
    x.o = heads_of<bf16>(a.o);
    x.lse = a.lse;
    x.pack = pl.pack;
    x.heads = pl.heads;
    x.o_vec = store_vec(a.o, a.dv);
    x.zero_rows = (a.flags & GMA_ROWS_ZERO_TAIL) && (a.lengths || a.offsets) ? (a.offsets ? 1 : a.B) * a.N : 0;
    x.head = (PlanHead *)(w + pl.head_at);
    x.items = (const Item *)(w + pl.items_at);
    x.parts = parts_of(pl, a, ws);
    x.hdr = (WsHeader *)ws;
    x.withhold = pl.withhold;
    x.q_boxes = (a.d + 63) / 64;
    x.v_boxes = (a.dv + 63) / 64;
    x.slot_bytes = BOX * (uint32_t)(x.q_boxes > x.v_boxes ? x.q_boxes : x.v_boxes);
    const uint32_t fixed = 2 * BOX * (uint32_t)x.q_boxes + 1024 + (uint32_t)sizeof(Bars);
    x.slots = (int)((SMEM_MAX - fixed) / x.slot_bytes);
    if (x.slots > MAX_SLOTS) x.slots = MAX_SLOTS;
    const uint32_t smem = fixed + (uint32_t)x.slots * x.slot_bytes;
    x.page_rows = p ? (p->page < TILE ? p->page : TILE) : TILE;
    x.tile_pages = TILE / x.page_rows;
    while (p && (1 << x.page_shift) < p->page) ++x.page_shift;
    const long long B = a.offsets ? 1 : a.B;
    CUtensorMap qm, km, vm;
    const int per = TILE / pl.pack;
    if (!heads_map(&qm, a.q, B, a.N, a.H, a.d, pl.pack, per)) return GMA_ERR_CUDA;
    if (p ? !heads_map(&km, p->k_pages, p->pages, p->page, a.G, a.d, 1, x.page_rows) || !heads_map(&vm, p->v_pages, p->pages, p->page, a.G, a.dv, 1, x.page_rows)
          : !heads_map(&km, a.k, B, a.N, a.G, a.d, 1, TILE) || !heads_map(&vm, a.v, B, a.N, a.G, a.dv, 1, TILE))
        return GMA_ERR_CUDA;
    gma_status_t r = launch_plan(plan_args(x.g, pl, ws), nullptr, st);
    if (r != GMA_OK) return r;
    // blocks stay and take items until there are no more
    const long long most = (long long)pl.max_items * pl.heads;
    const unsigned grid = most < SMS ? (unsigned)most : SMS;
    auto kern = p ? attn_tc_kernel<true> : attn_tc_kernel<false>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MAX) != cudaSuccess) return GMA_ERR_CUDA;
    GMA_LAUNCH(KID_ATTN, st, launch_pdl(kern, grid, THREADS, smem, st, x, qm, km, vm));
    return p ? launch_join(a, x.g, pl, ws, st) : GMA_OK;
}

}  // namespace att
}  // namespace gma
