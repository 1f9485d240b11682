// gma_attn_tc_bwd.cu -- backward pass of softmax attention over whole sequences on the tensor cores (tcgen05), bf16.
//
// Scores are computed again from q, k and the rows' log-sum-exp, once with keys as rows (dk, dv) and once with queries as rows
// (dq): seven products of a tile instead of five, but every sum is one block's in one order, without atomics and without an
// fp32 copy of dq, so that repeated calls give the same bits.
//
// dk, dv: a block owns 128 keys of one key head and walks over the query tiles that see them, of every query head of the group or, where that
// leaves SMs without work, of a piece of it.
//   S^T = K Q^T - lse / scale, dP^T = V dO^T - delta, P^T = exp(scale S^T), dS^T = P^T dP^T, dV += P^T dO, dK += dS^T Q.
// lse and delta belong to the columns here.  Read from shared memory they doubled the time of the exponentials (whose loads wait behind the
// products'); so they are a k-step of the products, in three bf16 terms each.
// Tensor memory: S^T | dP^T | dV | dK, 128 columns each.  P^T and dS^T, rounded to bf16 (half a step, 2^-8 relative), take the place of
// S^T and dP^T as first operands.  The products' order hides the warps' work: while they take exponentials the tensor cores run dK
// of the tile before and dP^T of this one, while they form dS^T they run dV of this tile and S^T of the next.
//
// dq: a block owns 128 query rows of one head and walks over their key tiles.  Tensor memory: S | S | dP | dQ; S of the next tile
// and dQ of the tile before run while the warps form dS of this one, in place of its S.
//
// Warps: 0-3 and 4-7 each take half a tile's columns (a thread a row), 8 issues the products, 9 loads.
//
// Measured: 8192 tokens, 16 heads of 128 over 4, causal: dk and dv 333 us, dq 254 us alone, 565 us together with the plan and delta (dq's blocks take
// the SMs that the others leave; 1220 TFLOP/s by five products a tile, 1700 by the seven that are made), tensor pipe 78 and 72 % busy; 4 x 4096 x 16
// heads of 64 558 us.  The chain scores - exponentials - products of one tile bounds both.  At 128 columns there is no second tile to work on
// meanwhile: tensor memory is full, and shared memory holds two query tiles.  At 64 columns 128 columns of tensor memory are free in dk and dv, 64 in
// dq, which this order of products does not use.
#include "attn_tc.cuh"
#include "attn_tc_host.cuh"

namespace gma {
namespace att {
namespace {

constexpr int THREADS = 384;
constexpr int STAGES = 4, SLOTS = 5;         // at most

struct GradArgs {
    Geo g;
    Heads<bf16> dq, dk, dv;
    const float *lse, *delta;
    const PlanHead *q_head, *k_head;
    const Item *q_items, *k_items;
    int q_vec, k_vec, v_vec;     // 16-byte stores
    WsHeader *hdr;
    int q_boxes, v_boxes;
    int stages, k_slots, v_slots; // of the two kernels' rings
    Pieces pieces;
    int withhold;                 // GMA_FLAG_TEST_WITHHOLD: a block's own tiles are never loaded
};

// A row's statistic enters its products as one more k-step: three bf16 terms that add up to it in fp32's 24 bits, against ones.
// Tiles of 128 rows of 16 (K-major, 32-byte swizzle), 4 KB.
constexpr uint32_t EXTRA = TILE * 32;
__device__ __forceinline__ uint64_t extra_desc(uint32_t tile) { return smem_desc(tile, 16, 256, SW_32B); }
__device__ __forceinline__ void put_extra(uint8_t *tile, int row, float x)
{
    const bf16 hi = __float2bfloat16_rn(x);
    const float r1 = x - __bfloat162float(hi);
    const bf16 mid = __float2bfloat16_rn(r1), lo = __float2bfloat16_rn(r1 - __bfloat162float(mid));
    const uint32_t a = (uint32_t)__bfloat16_as_ushort(hi) | (uint32_t)__bfloat16_as_ushort(mid) << 16, b = __bfloat16_as_ushort(lo);
    *reinterpret_cast<uint4 *>(tile + row * 32 + (((row >> 2) & 1) << 4)) = make_uint4(a, b, 0, 0);
}

// 32 columns' values back as bf16 pairs in 16 columns.
__device__ __forceinline__ void put_pairs(uint32_t at, const blk::f2 (&v)[16])
{
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 x = blk::unpack2(v[e]);
        w[e] = pack_bf16(x.x, x.y);
    }
    tmem_st16(at, w);
}
__device__ __forceinline__ blk::f2 pair_of(const uint32_t (&r)[32], int e)
{
    return blk::pack2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
}

// ------------------------------------------------------------------ dk, dv
struct KeyBars {
    uint64_t kv, fq[STAGES], fo[STAGES], eq[STAGES], eo[STAGES], s, dp, p, ds, done, drain;
    uint32_t tmem;
    int abort;
};

__global__ void __launch_bounds__(THREADS, 1) attn_dkv_kernel(const GradArgs a, const __grid_constant__ CUtensorMap qmap,
                                                              const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                                                              const __grid_constant__ CUtensorMap omap)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t q_tile = (uint32_t)a.q_boxes * BOX, v_tile = (uint32_t)a.v_boxes * BOX, stage = q_tile + v_tile;
    uint8_t *ring = smem + stage;                                // K and V lie before it
    uint8_t *ones = ring + (size_t)a.stages * stage, *extra = ones + EXTRA;      // extra: of each stage, -lse / scale and -delta
    KeyBars *bars = reinterpret_cast<KeyBars *>(extra + (size_t)a.stages * 2 * EXTRA);
    volatile int *abort = &bars->abort;
    const int t = threadIdx.x, warp = __shfl_sync(~0u, t >> 5, 0), lane = t & 31;      // uniform, as the compiler knows
    if (t == 256) {
        mbar_init(&bars->kv, 1);
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&bars->fq[i], 2);
            mbar_init(&bars->fo[i], 1);
            mbar_init(&bars->eq[i], 1);
            mbar_init(&bars->eo[i], 1);
        }
        mbar_init(&bars->s, 1);
        mbar_init(&bars->dp, 1);
        mbar_init(&bars->p, 256);
        mbar_init(&bars->ds, 256);
        mbar_init(&bars->done, 1);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    blk::wait_previous();
    blk::let_next();       // what this kernel reads, the next one reads too: dq's blocks take the SMs that these leave
    const Geo &g = a.g;
    const int parts = a.pieces.count, rank = blockIdx.x / (g.G * parts), at = blockIdx.x - rank * g.G * parts;
    const int kvh = at / parts, piece = at - kvh * parts, heads = g.group / parts;
    if (rank >= a.k_head->items) return;
    if (warp == 8) tmem_alloc(&bars->tmem, 512);
    const Item it = load_item(a.k_items + rank);
    const Seq sq = it.sq;
    const int tiles = __shfl_sync(~0u, it.t1 - it.t0, 0), steps = tiles * heads;
    for (int i = t; i < TILE; i += THREADS) {
        *reinterpret_cast<uint4 *>(ones + i * 32 + (((i >> 2) & 1) << 4)) = make_uint4(0x3f803f80u, 0x3f80u, 0, 0);
        *reinterpret_cast<uint4 *>(ones + i * 32 + ((((i >> 2) & 1) ^ 1) << 4)) = make_uint4(0, 0, 0, 0);
    }
    for (int i = t; i < a.stages * 2 * TILE; i += THREADS)
        *reinterpret_cast<uint4 *>(extra + i * 32 + ((((i >> 2) & 1) ^ 1) << 4)) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, bars->tmem, 0), sb = smem_u32(smem), rb = smem_u32(ring);

    if (warp == 8) {
        const uint32_t id_s = idesc_f16(TILE, TILE, 1, 1, 0, 0);
        const uint32_t id_v = idesc_f16(TILE, (uint32_t)(g.dv + 15) & ~15u, 1, 1, 0, 1), id_k = idesc_f16(TILE, (uint32_t)(g.d + 15) & ~15u, 1, 1, 0, 1);
        const int kq = (g.d + 15) >> 4, ko = (g.dv + 15) >> 4;
        bool ok = bar_wait(&bars->kv, 0, a.hdr, 220, abort);
        const uint64_t kd = k_desc(sb), vd = k_desc(sb + q_tile), ones_desc = extra_desc(smem_u32(ones));
        const uint32_t xb = smem_u32(extra);
        // the steps whose scores and whose dP come next, and the one at hand; rows that a step's tile has
        RingPos rs{0, 0}, rp{0, 0}, rc{0, 0};
        int js = 0, jp = 0;
        auto rows = [&](int j) { return sq.n - (it.t0 + j) * TILE; };
        // rows behind the sequence's end meet zeros of P and dS, and may be anything
        auto q_there = [&]() { return bar_wait(&bars->fq[rs.s], rs.turn, a.hdr, 221, abort); };
        auto o_there = [&]() { return bar_wait(&bars->fo[rp.s], rp.turn, a.hdr, 222, abort); };
        auto scores = [&]() {
            if (rows(js) < TILE) zero_rows(ring + rs.s * stage, a.q_boxes, rows(js));
            if (++js == tiles) js = 0;
            if (elect()) {
                mma_tiles(tmem, kd, k_desc(rb + rs.s * stage), id_s, kq);
                mma_f16(tmem, ones_desc, extra_desc(xb + rs.s * 2 * EXTRA), id_s, 1u);
                mma_commit(&bars->s);
            }
            rs.step(1, a.stages);
        };
        auto dprobs = [&]() {
            if (rows(jp) < TILE) zero_rows(ring + rp.s * stage + q_tile, a.v_boxes, rows(jp));
            if (++jp == tiles) jp = 0;
            if (elect()) {
                mma_tiles(tmem + 128, vd, k_desc(rb + rp.s * stage + q_tile), id_s, ko);
                mma_f16(tmem + 128, ones_desc, extra_desc(xb + rp.s * 2 * EXTRA + EXTRA), id_s, 1u);
                mma_commit(&bars->dp);
            }
            rp.step(1, a.stages);
        };
        // A barrier that is through costs some 80 cycles to find so, and this warp's time bounds the loop: the two that a pair of products waits
        // for are asked at once.  A tile that is not there yet does not keep the first of the pair (waited for before it, 8192 x 16 heads
        // of 128 take 389 us instead of 350).
        if ((ok = ok && q_there())) scores();
        if ((ok = ok && o_there())) dprobs();
        for (int i = 0; ok && i < steps; ++i) {
            const bool more = i + 1 < steps;
            bool now = bar_there(&bars->p, i & 1), there = bar_there(&bars->fq[rs.s], rs.turn);
            if (!now && !(ok = bar_wait(&bars->p, i & 1, a.hdr, 223, abort))) break;
            tc_fence_after();
            if (elect()) {
                const uint64_t o = mn_desc(rb + rc.s * stage + q_tile);
#pragma unroll
                for (int s = 0; s < 8; ++s) mma_f16_tmem_a(tmem + 256, tmem + half_col(s), o + mn_step(s), id_v, i > 0 || s > 0);
                mma_commit(&bars->eo[rc.s]);
            }
            if (more) {
                if (!there && !(ok = q_there())) break;
                scores();
            }
            now = bar_there(&bars->ds, i & 1);
            there = bar_there(&bars->fo[rp.s], rp.turn);
            if (!now && !(ok = bar_wait(&bars->ds, i & 1, a.hdr, 224, abort))) break;
            tc_fence_after();
            if (elect()) {
                const uint64_t q = mn_desc(rb + rc.s * stage);
#pragma unroll
                for (int s = 0; s < 8; ++s) mma_f16_tmem_a(tmem + 384, tmem + 128 + half_col(s), q + mn_step(s), id_k, i > 0 || s > 0);
                mma_commit(&bars->eq[rc.s]);
            }
            if (more) {
                if (!there && !(ok = o_there())) break;
                dprobs();
            }
            rc.step(1, a.stages);
        }
        if (ok && elect()) mma_commit(&bars->done);
        if (aborted(abort)) {
            if (elect()) mma_commit(&bars->drain);
            mbar_wait(&bars->drain, 0, a.hdr, 225);
        }
    } else if (warp == 9) {
        if (lane == 0 && !a.withhold) {
            mbar_arrive_expect_tx(&bars->kv, stage);
            for (int b = 0; b < a.q_boxes; ++b) tma_load_4d(sb + b * BOX, &kmap, &bars->kv, 64 * b, kvh, sq.row0 + it.tok0, sq.b);
            for (int b = 0; b < a.v_boxes; ++b) tma_load_4d(sb + q_tile + b * BOX, &vmap, &bars->kv, 64 * b, kvh, sq.row0 + it.tok0, sq.b);
        }
        bool ok = true;
        int issued_q = 0, issued_o = 0;
        RingPos r{0, 1};
        const float inv_scale = 1.f / g.scale;
        int h = kvh * g.group + piece * heads, j = 0;
        for (int i = 0; ok && i < steps; ++i) {
            const int q0 = (it.t0 + j) * TILE, s = r.s;
            const uint32_t free = r.turn;
            // this tile's statistics, on their way while its place is waited for
            float l[4], e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = q0 + lane + 32 * k;
                const long long at = row < sq.n ? stat_at(g, sq, h, row) : 0;
                l[k] = row < sq.n ? -a.lse[at] * inv_scale : 0.f;
                e[k] = row < sq.n ? -a.delta[at] : 0.f;
            }
            if (!(ok = bar_wait(&bars->eq[s], free, a.hdr, 226, abort))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->fq[s], q_tile);
                for (int b = 0; b < a.q_boxes; ++b) tma_load_4d(rb + s * stage + b * BOX, &qmap, &bars->fq[s], 64 * b, h, sq.row0 + q0, sq.b);
            }
            issued_q = i + 1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                put_extra(extra + s * 2 * EXTRA, lane + 32 * k, l[k]);
                put_extra(extra + s * 2 * EXTRA + EXTRA, lane + 32 * k, e[k]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->fq[s]);
            if (!(ok = bar_wait(&bars->eo[s], free, a.hdr, 227, abort))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->fo[s], v_tile);
                for (int b = 0; b < a.v_boxes; ++b) tma_load_4d(rb + s * stage + q_tile + b * BOX, &omap, &bars->fo[s], 64 * b, h, sq.row0 + q0, sq.b);
            }
            issued_o = i + 1;
            r.step(1, a.stages);
            if (++j == tiles) {
                j = 0;
                ++h;
            }
        }
        if (aborted(abort)) {          // loads that no product waited for
            mbar_wait(&bars->kv, 0, a.hdr, 228);
            for (int i = issued_q > a.stages ? issued_q - a.stages : 0; i < issued_q; ++i)
                mbar_wait(&bars->fq[i % a.stages], (uint32_t)(i / a.stages) & 1u, a.hdr, 229);
            for (int i = issued_o > a.stages ? issued_o - a.stages : 0; i < issued_o; ++i)
                mbar_wait(&bars->fo[i % a.stages], (uint32_t)(i / a.stages) & 1u, a.hdr, 230);
        }
    } else if (warp < 8) {
        const int w = warp >> 2, row = t & (TILE - 1), key = it.tok0 + row;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 64 * w, td = ts + 128;
        bool ok = true;
        int j = 0;
        const blk::f2 scale = blk::pack2(g.sl2, g.sl2);
        for (int i = 0; i < steps; ++i) {
            const int q0 = (it.t0 + j) * TILE + 64 * w;
            if (++j == tiles) j = 0;
            // columns that this row's key is seen by, of those that are there: [from, to)
            const int from = g.causal ? key - q0 : 0, to = sq.n - q0;
            const bool edge = __any_sync(~0u, from > 0 || to < 64);
            if (!(ok = bar_wait(&bars->s, i & 1, a.hdr, 232, abort))) break;
            tc_fence_after();
            blk::f2 p[2][16];
            {
                uint32_t r[2][32];
                tmem_ld32(ts, r[0]);
                tmem_ld32(ts + 32, r[1]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[c][e] = blk::ex2_2(blk::mul2(pair_of(r[c], e), scale));
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int col = 32 * c + 2 * e;
                            const float2 x = blk::unpack2(p[c][e]);
                            p[c][e] = blk::pack2(col >= from && col < to ? x.x : 0.f, col + 1 >= from && col + 1 < to ? x.y : 0.f);
                        }
                    }
                    put_pairs(ts + 16 * c, p[c]);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars->p);
            if (!(ok = bar_wait(&bars->dp, i & 1, a.hdr, 233, abort))) break;
            tc_fence_after();
            uint32_t r[2][32];
            tmem_ld32(td, r[0]);
            tmem_ld32(td + 32, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int e = 0; e < 16; ++e) p[c][e] = blk::mul2(p[c][e], pair_of(r[c], e));
                put_pairs(td + 16 * c, p[c]);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars->ds);
        }
        if (ok && bar_wait(&bars->done, 0, a.hdr, 234, abort)) {
            tc_fence_after();
            const bool valid = key < sq.n;
            const int r = sq.row0 + (valid ? key : it.tok0);
            if (parts > 1) {
                const long long at = (long long)sq.b * g.N + r;
                if (w == 0) store_row_f32(tmem + lanes + 256, g.dv, valid, a.pieces.v_at(piece, kvh, at));
                else store_row_f32(tmem + lanes + 384, g.d, valid, a.pieces.k_at(piece, kvh, at));
            } else if (w == 0) store_row(tmem + lanes + 256, g.dv, 1.f, valid, a.dv.at(sq.b, r, kvh), a.v_vec);
            else store_row(tmem + lanes + 384, g.d, g.scale, valid, a.dk.at(sq.b, r, kvh), a.k_vec);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ dq
struct QueryBars {
    uint64_t q, fk[SLOTS], ek[SLOTS], fv[SLOTS], ev[SLOTS], s[2], dp, ds, done, drain;
    uint32_t tmem;
    int abort;
};

__global__ void __launch_bounds__(THREADS, 1) attn_dq_kernel(const GradArgs a, const __grid_constant__ CUtensorMap qmap,
                                                             const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                                                             const __grid_constant__ CUtensorMap omap)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t q_tile = (uint32_t)a.q_boxes * BOX, v_tile = (uint32_t)a.v_boxes * BOX;
    uint8_t *ring = smem + q_tile + v_tile;
    uint8_t *vring = ring + (size_t)a.k_slots * q_tile;
    QueryBars *bars = reinterpret_cast<QueryBars *>(vring + (size_t)a.v_slots * v_tile);
    volatile int *abort = &bars->abort;
    const int t = threadIdx.x, warp = __shfl_sync(~0u, t >> 5, 0), lane = t & 31;      // uniform, as the compiler knows
    if (t == 256) {
        mbar_init(&bars->q, 1);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&bars->fk[i], 1);
            mbar_init(&bars->ek[i], 1);
            mbar_init(&bars->fv[i], 1);
            mbar_init(&bars->ev[i], 1);
        }
        mbar_init(&bars->s[0], 1);
        mbar_init(&bars->s[1], 1);
        mbar_init(&bars->dp, 1);
        mbar_init(&bars->ds, 256);
        mbar_init(&bars->done, 1);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    // (the blocks before read the same results, and had waited for them when they let this kernel start; its last block waits for theirs)
    if (blockIdx.x == gridDim.x - 1) blk::wait_previous();
    const Geo &g = a.g;
    const int rank = blockIdx.x / g.H, h = blockIdx.x % g.H, kvh = h / g.group;
    if (rank >= __ldcg(&a.q_head->items)) return;
    if (warp == 8) tmem_alloc(&bars->tmem, 512);
    const Item it = load_item(a.q_items + rank);
    const Seq sq = it.sq;
    const int tiles = __shfl_sync(~0u, it.t1 - it.t0, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, bars->tmem, 0), sb = smem_u32(smem), rb = smem_u32(ring), vb = smem_u32(vring);

    if (warp == 8) {
        const uint32_t id_s = idesc_f16(TILE, TILE, 1, 1, 0, 0), id_q = idesc_f16(TILE, (uint32_t)(g.d + 15) & ~15u, 1, 1, 0, 1);
        const int kq = (g.d + 15) >> 4, ko = (g.dv + 15) >> 4;
        bool ok = bar_wait(&bars->q, 0, a.hdr, 240, abort);
        const uint64_t qd = k_desc(sb), od = k_desc(sb + q_tile);
        // the ring's places of the keys whose scores come next, of the values whose dP does, and of the keys at hand
        RingPos rk{0, 0}, rv{0, 0}, rc{0, 0};
        // keys behind the sequence's end meet zeros of dS, and may be anything
        auto keys = [&](int j, bool there) {
            if (!there && !bar_wait(&bars->fk[rk.s], rk.turn, a.hdr, 241, abort)) return false;
            const int have = sq.L - (it.t0 + j) * TILE;
            if (have < TILE) zero_rows(ring + (size_t)rk.s * q_tile, a.q_boxes, have);
            return true;
        };
        auto put_scores = [&](int j) {
            mma_tiles(tmem + 128 * (j & 1), qd, k_desc(rb + (uint32_t)rk.s * q_tile), id_s, kq);
            mma_commit(&bars->s[j & 1]);
        };
        auto put_dprobs = [&]() {
            mma_tiles(tmem + 256, od, k_desc(vb + (uint32_t)rv.s * v_tile), id_s, ko);
            mma_commit(&bars->dp);
            mma_commit(&bars->ev[rv.s]);
        };
        auto put_dq = [&](int j) {
            const uint64_t k = mn_desc(rb + (uint32_t)rc.s * q_tile);
            const uint32_t ds = tmem + 128 * (j & 1);
#pragma unroll
            for (int s = 0; s < 8; ++s) mma_f16_tmem_a(tmem + 384, ds + half_col(s), k + mn_step(s), id_q, j > 0 || s > 0);
            mma_commit(&bars->ek[rc.s]);
        };
        auto values = [&]() { return bar_wait(&bars->fv[rv.s], rv.turn, a.hdr, 250, abort); };
        if ((ok = ok && keys(0, false) && values()) && elect()) {
            put_scores(0);
            put_dprobs();
        }
        rk.step(1, a.k_slots);
        rv.step(1, a.v_slots);
        if (ok && tiles > 1 && (ok = keys(1, false))) {
            if (elect()) put_scores(1);
            rk.step(1, a.k_slots);
        }
        // dP of the next tile, dQ of this one and S of the one after next follow one another, their barriers asked at once: each costs some 80
        // cycles to find that it is through, and this warp's time bounds the loop (4 x 4096 x 16 heads of 64: 268 -> 252 us)
        for (int j = 0; ok && j < tiles; ++j) {
            const bool more = j + 1 < tiles, after = j + 2 < tiles;
            const bool now = bar_there(&bars->ds, j & 1);
            const bool v_there = !more || bar_there(&bars->fv[rv.s], rv.turn);
            const bool k_there = !after || bar_there(&bars->fk[rk.s], rk.turn);
            if (!v_there && !(ok = values())) break;
            if (!now && !(ok = bar_wait(&bars->ds, j & 1, a.hdr, 242, abort))) break;
            tc_fence_after();
            if (k_there) {
                if (after && !(ok = keys(j + 2, true))) break;
                if (elect()) {
                    if (more) put_dprobs();
                    put_dq(j);
                    if (after) put_scores(j + 2);
                }
            } else {
                if (elect()) {
                    if (more) put_dprobs();
                    put_dq(j);
                }
                if (!(ok = keys(j + 2, false))) break;
                if (elect()) put_scores(j + 2);
            }
            rv.step(1, a.v_slots);
            rc.step(1, a.k_slots);
            if (after) rk.step(1, a.k_slots);
        }
        if (ok && elect()) mma_commit(&bars->done);
        if (aborted(abort)) {
            if (elect()) mma_commit(&bars->drain);
            mbar_wait(&bars->drain, 0, a.hdr, 243);
        }
    } else if (warp == 9) {
        if (lane == 0 && !a.withhold) {
            mbar_arrive_expect_tx(&bars->q, q_tile + v_tile);
            for (int b = 0; b < a.q_boxes; ++b) tma_load_4d(sb + b * BOX, &qmap, &bars->q, 64 * b, h, sq.row0 + it.tok0, sq.b);
            for (int b = 0; b < a.v_boxes; ++b) tma_load_4d(sb + q_tile + b * BOX, &omap, &bars->q, 64 * b, h, sq.row0 + it.tok0, sq.b);
        }
        // keys wait for the products of two tiles before their place is free, values for one: rings of their own
        bool ok = true;
        int keys = 0, values = 0;
        RingPos rk{0, 1}, rv{0, 1};
        for (int j = 0; ok && j < tiles; ++j) {
            const int row = sq.row0 + (it.t0 + j) * TILE;
            if (!(ok = bar_wait(&bars->ek[rk.s], rk.turn, a.hdr, 244, abort))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->fk[rk.s], q_tile);
                for (int b = 0; b < a.q_boxes; ++b) tma_load_4d(rb + rk.s * q_tile + b * BOX, &kmap, &bars->fk[rk.s], 64 * b, kvh, row, sq.b);
            }
            ++keys;
            rk.step(1, a.k_slots);
            if (!(ok = bar_wait(&bars->ev[rv.s], rv.turn, a.hdr, 251, abort))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->fv[rv.s], v_tile);
                for (int b = 0; b < a.v_boxes; ++b) tma_load_4d(vb + rv.s * v_tile + b * BOX, &vmap, &bars->fv[rv.s], 64 * b, kvh, row, sq.b);
            }
            ++values;
            rv.step(1, a.v_slots);
        }
        if (aborted(abort)) {
            mbar_wait(&bars->q, 0, a.hdr, 245);
            for (int c = keys > a.k_slots ? keys - a.k_slots : 0; c < keys; ++c)
                mbar_wait(&bars->fk[c % a.k_slots], (uint32_t)(c / a.k_slots) & 1u, a.hdr, 246);
            for (int c = values > a.v_slots ? values - a.v_slots : 0; c < values; ++c)
                mbar_wait(&bars->fv[c % a.v_slots], (uint32_t)(c / a.v_slots) & 1u, a.hdr, 252);
        }
    } else if (warp < 8) {
        const int w = warp >> 2, row = t & (TILE - 1), tok = it.tok0 + row;
        const bool valid = tok < sq.n;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int seen = valid ? sq.seen(g, tok) : sq.L;
        const long long at = valid ? stat_at(g, sq, h, tok) : 0;
        const float lse2 = valid ? __ldcg(a.lse + at) * LOG2E : 0.f, delta = valid ? __ldcg(a.delta + at) : 0.f;
        const blk::f2 scale = blk::pack2(g.sl2, g.sl2), less = blk::pack2(-lse2, -lse2), minus = blk::pack2(-delta, -delta);
        bool ok = true;
        for (int j = 0; j < tiles; ++j) {
            const uint32_t ts = tmem + lanes + 128 * (j & 1) + 64 * w, td = tmem + lanes + 256 + 64 * w;
            if (!(ok = bar_wait(&bars->s[j & 1], (j >> 1) & 1, a.hdr, 247, abort))) break;
            tc_fence_after();
            const int lim = seen - (it.t0 + j) * TILE - 64 * w;
            const bool edge = __any_sync(~0u, lim < 64);
            blk::f2 p[2][16];
            {
                uint32_t r[2][32];
                tmem_ld32(ts, r[0]);
                tmem_ld32(ts + 32, r[1]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[c][e] = blk::ex2_2(blk::fma2(pair_of(r[c], e), scale, less));
            }
            if (!(ok = bar_wait(&bars->dp, j & 1, a.hdr, 248, abort))) break;
            tc_fence_after();
            uint32_t r[2][32];
            tmem_ld32(td, r[0]);
            tmem_ld32(td + 32, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int e = 0; e < 16; ++e) p[c][e] = blk::mul2(p[c][e], blk::add2(pair_of(r[c], e), minus));
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int col = 32 * c + 2 * e;
                        const float2 x = blk::unpack2(p[c][e]);
                        p[c][e] = blk::pack2(col < lim ? x.x : 0.f, col + 1 < lim ? x.y : 0.f);
                    }
                }
                put_pairs(ts + 16 * c, p[c]);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars->ds);
        }
        if (ok && bar_wait(&bars->done, 0, a.hdr, 249, abort)) {
            tc_fence_after();
            // each half of the warps takes half of the columns
            const int from = 64 * w, width = min(g.d - from, 64);
            if (width > 0)
                store_row(tmem + lanes + 384 + from, width, g.scale, valid, a.dq.at(sq.b, sq.row0 + (valid ? tok : it.tok0), h) + from, a.q_vec);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

struct GradPlan {
    Plan q, k;
    PiecePlan pieces;
    size_t delta_at;
};

GradPlan grad_plan(const gma_attn_t &a, Carve *c)
{
    GradPlan p;
    p.q = make_plan(a, 1, TILE, TILE, 7, SMS, false, c);
    gma_attn_t by = a;
    p.pieces = plan_pieces(a, TILE, TILE, 1.5, c);
    by.H = a.G * p.pieces.count;      // a tile of keys serves the group or a piece of it
    p.k = make_plan(by, 1, TILE, TILE, 7, SMS, false, c);
    p.k.by_keys = true;
    p.delta_at = c->take((size_t)(a.offsets ? 1 : a.B) * a.H * a.N * sizeof(float));
    return p;
}

}  // namespace

bool tc_takes_backward(const gma_attn_grad_t &g)
{
    const gma_attn_t &a = g.fwd;
    const long long B = a.offsets ? 1 : a.B;
    return tc_takes(a, nullptr) && tma_heads(g.d_o, B, a.N, a.H);
}

size_t tc_backward_workspace(const gma_attn_grad_t &g)
{
    Carve c;
    grad_plan(g.fwd, &c);
    return c.total();
}

gma_status_t tc_backward(const gma_attn_grad_t &g, void *ws, cudaStream_t st)
{
    const gma_attn_t &a = g.fwd;
    Carve c;
    const GradPlan p = grad_plan(a, &c);
    char *w = (char *)ws;
    GradArgs x = {};
    x.g = geo_of(a, nullptr);
    x.dq = heads_of<bf16>(g.dq); x.dk = heads_of<bf16>(g.dk); x.dv = heads_of<bf16>(g.dv);
    x.lse = a.lse;
    float *delta = (float *)(w + p.delta_at);
    x.delta = delta;
    x.q_head = (const PlanHead *)(w + p.q.head_at);
    x.k_head = (const PlanHead *)(w + p.k.head_at);
    x.q_items = (const Item *)(w + p.q.items_at);
    x.k_items = (const Item *)(w + p.k.items_at);
    x.q_vec = store_vec(g.dq, a.d);
    x.k_vec = store_vec(g.dk, a.d);
    x.v_vec = store_vec(g.dv, a.dv);
    x.hdr = (WsHeader *)ws;
    x.withhold = p.q.withhold;
    x.pieces = pieces_of(p.pieces, a, ws);
    x.q_boxes = (a.d + 63) / 64;
    x.v_boxes = (a.dv + 63) / 64;
    const uint32_t pair = BOX * (uint32_t)(x.q_boxes + x.v_boxes), k_fixed = pair + EXTRA + 1024 + (uint32_t)sizeof(KeyBars),
                   q_fixed = pair + 1024 + (uint32_t)sizeof(QueryBars);
    const uint32_t k_stage = pair + 2 * EXTRA;
    x.stages = (int)((SMEM_MAX - k_fixed) / k_stage);
    if (x.stages > STAGES) x.stages = STAGES;
    const uint32_t q_room = SMEM_MAX - q_fixed;
    x.v_slots = (int)(q_room / pair);                             // and one more of keys, where there is room
    if (x.v_slots > SLOTS - 1) x.v_slots = SLOTS - 1;
    x.k_slots = x.v_slots + (q_room - x.v_slots * pair >= BOX * (uint32_t)x.q_boxes ? 1 : 0);
    const uint32_t q_ring = BOX * (uint32_t)(x.k_slots * x.q_boxes + x.v_slots * x.v_boxes);
    const long long B = a.offsets ? 1 : a.B;
    CUtensorMap qm, km, vm, om;
    if (!heads_map(&qm, a.q, B, a.N, a.H, a.d, 1, TILE) || !heads_map(&km, a.k, B, a.N, a.G, a.d, 1, TILE) ||
        !heads_map(&vm, a.v, B, a.N, a.G, a.dv, 1, TILE) || !heads_map(&om, g.d_o, B, a.N, a.H, a.dv, 1, TILE))
        return GMA_ERR_CUDA;
    const PlanArgs first = plan_args(x.g, p.q, ws);
    PlanArgs second = plan_args(x.g, p.k, ws);
    second.hdr = nullptr;
    gma_status_t r = launch_plan(first, &second, st);
    if (r != GMA_OK) return r;
    if ((r = launch_delta(g, delta, st)) != GMA_OK) return r;
    if (cudaFuncSetAttribute(attn_dkv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MAX) != cudaSuccess ||
        cudaFuncSetAttribute(attn_dq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MAX) != cudaSuccess)
        return GMA_ERR_CUDA;
    GMA_LAUNCH(KID_ATTN_DKV, st, launch_pdl(attn_dkv_kernel, (unsigned)p.k.max_items * p.k.heads, THREADS, k_fixed + x.stages * k_stage, st, x, qm, km, vm, om));
    GMA_LAUNCH(KID_ATTN_DQ, st, launch_pdl(attn_dq_kernel, (unsigned)p.q.max_items * a.H, THREADS, q_fixed + q_ring, st, x, qm, km, vm, om));
    return launch_pieces(g, x.pieces, st);
}

}  // namespace att
}  // namespace gma
