// gma_blocksum.cu -- sums over rows of per-block partial results (parameter gradients), in a fixed
// order, so that they repeat bit for bit.  304 rows of 3 x 2048 sums take 5 us, most of it the launch's.
#include "block_common.cuh"

namespace gma {
namespace blk {
namespace {

struct SumList {
    SumVec v[MAX_SUMS];
    unsigned first[MAX_SUMS + 1];        // first block of each vector
    int count;
};

// 32 columns a block (one 128-byte line a row), eight warps of four independent sums each over every
// 32nd row, then the warps in order.  The partial rows were just written and come from L2.
__global__ void __launch_bounds__(256) sum_rows_kernel(const SumList l, long long rows)
{
    __shared__ float s[8][33];
    wait_previous();
    int k = 0;
#pragma unroll
    for (int j = 1; j < MAX_SUMS; ++j)
        if (j < l.count && blockIdx.x >= l.first[j]) k = j;
    const SumVec v = l.v[k];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long i = (long long)(blockIdx.x - l.first[k]) * 32 + lane;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < v.n) {
        const float *p = v.part + i;
        long long r = warp;
        for (; r + 24 < rows; r += 32)
#pragma unroll
            for (int u = 0; u < 4; ++u) a[u] += p[(r + 8 * u) * v.row_stride];
        for (; r < rows; r += 8) a[0] += p[r * v.row_stride];
    }
    s[warp][lane] = (a[0] + a[1]) + (a[2] + a[3]);
    __syncthreads();
    if (warp == 0 && i < v.n) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += s[w][lane];
        v.out[i * v.out_stride] = t;
    }
}

}  // namespace

gma_status_t sum_rows(const SumVec *vecs, int count, long long rows, cudaStream_t st)
{
    SumList l = {};
    unsigned blocks = 0;
    for (int k = 0; k < count; ++k) {
        l.v[k] = vecs[k];
        l.first[k] = blocks;
        blocks += (unsigned)((vecs[k].n + 31) / 32);
    }
    l.count = count;
    if (blocks == 0) return GMA_OK;
    GMA_LAUNCH(KID_SUM_ROWS, st, launch_pdl(sum_rows_kernel, dim3(blocks), dim3(256), 0, st, l, rows));
    return GMA_OK;
}

}  // namespace blk
}  // namespace gma
