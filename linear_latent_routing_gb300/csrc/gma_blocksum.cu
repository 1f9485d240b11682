// gma_blocksum.cu -- sums over rows of per-block partial results (parameter gradients), in a fixed
// order, so that they repeat bit for bit.
#include "block_common.cuh"

namespace gma {
namespace blk {
namespace {

struct SumOuts {
    SumOut o[MAX_SUMS];
};

// 32 columns a block (one 128-byte line a row), eight warps of four independent sums each over every
// 32nd row, then the warps in order.  The partial rows were just written and come from L2.
__global__ void __launch_bounds__(256) sum_rows_kernel(const float *part, long long rows, long long row_stride, int n,
                                                       int pitch, const SumOuts outs)
{
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane, k = blockIdx.y;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < n) {
        const float *p = part + (long long)k * pitch + i;
        long long r = warp;
        for (; r + 24 < rows; r += 32)
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] += p[(r + 8 * u) * row_stride];
        for (; r < rows; r += 8) v[0] += p[r * row_stride];
    }
    s[warp][lane] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (warp == 0 && i < n) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += s[w][lane];
        outs.o[k].p[i * outs.o[k].stride] = t;
    }
}

}  // namespace

gma_status_t sum_rows(const float *part, long long rows, int K, int per_row, int n, int pitch, const SumOut *out,
                      cudaStream_t st)
{
    SumOuts o = {};
    for (int k = 0; k < K; ++k) o.o[k] = out[k];
    GMA_LAUNCH(KID_SUM_ROWS, st,
               sum_rows_kernel<<<dim3((n + 31) / 32, K), 256, 0, st>>>(part, rows, (long long)per_row * pitch, n, pitch, o));
    return GMA_OK;
}

}  // namespace blk
}  // namespace gma
