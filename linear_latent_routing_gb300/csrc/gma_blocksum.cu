// gma_blocksum.cu -- sums over rows of per-block partial results (parameter gradients), in a fixed
// order, so that they repeat bit for bit.  304 rows of 3 x 2048 sums take 5 us, most of it the launch's.
#include "block_common.cuh"

namespace gma {
namespace blk {
namespace {

__global__ void __launch_bounds__(256) sum_rows_kernel(const SumList l)
{
    wait_previous();
    sum_rows_block(l, blockIdx.x);
}

}  // namespace

SumList sum_list(const SumVec *vecs, int count, long long rows)
{
    SumList l = {};
    unsigned blocks = 0;
    for (int k = 0; k < count; ++k) {
        l.v[k] = vecs[k];
        l.first[k] = blocks;
        blocks += (unsigned)((vecs[k].n + 31) / 32);
    }
    l.count = count;
    l.first[count] = blocks;
    l.rows = rows;
    return l;
}

gma_status_t sum_rows(const SumVec *vecs, int count, long long rows, cudaStream_t st)
{
    const SumList l = sum_list(vecs, count, rows);
    if (l.first[count] == 0) return GMA_OK;
    GMA_LAUNCH(KID_SUM_ROWS, st, launch_pdl(sum_rows_kernel, dim3(l.first[count]), dim3(256), 0, st, l));
    return GMA_OK;
}

}  // namespace blk
}  // namespace gma
