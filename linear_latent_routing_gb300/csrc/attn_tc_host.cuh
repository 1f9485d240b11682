// attn_tc_host.cuh -- the tensor-core attention's calls.
#pragma once

#include "attn_common.cuh"

namespace gma {
namespace att {

// Whether the tensor-core kernels take this call as it lies.
bool tc_takes(const gma_attn_t &a, const gma_attn_paged_t *paged);
size_t tc_workspace(const gma_attn_t &a, const gma_attn_paged_t *paged);
gma_status_t tc_forward(const gma_attn_t &a, const gma_attn_paged_t *paged, void *ws, cudaStream_t st);
bool tc_takes_backward(const gma_attn_grad_t &g);
size_t tc_backward_workspace(const gma_attn_grad_t &g);
gma_status_t tc_backward(const gma_attn_grad_t &g, void *ws, cudaStream_t st);

}  // namespace att
}  // namespace gma
