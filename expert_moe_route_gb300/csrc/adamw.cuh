// Launchers of the optimiser kernels (adamw.cu).
#pragma once

#include "common.cuh"

namespace moe {

size_t grad_norm_ws_bytes(const moe_adamw_tensor_t* x, int n);
cudaError_t launch_grad_norm(const moe_adamw_tensor_t* x, int n, double max_norm, float* norm,
                             void* ws, cudaStream_t s);
cudaError_t launch_adamw(const moe_adamw_tensor_t* x, int n, const moe_adamw_t& h,
                         const float* norm, cudaStream_t s);

}  // namespace moe
