// Launchers of routing by scores (route_scores.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

struct ScoresArgs {
  const void* logits;
  long long ld;
  int dtype, T, E, R;
  moe_router_t router;
  const float* bias;        // [E] or null
};
cudaError_t launch_route_scores(const ScoresArgs& a, int32_t* topk_idx, float* topk_w,
                                cudaStream_t s);
cudaError_t launch_route_scores_bwd(const ScoresArgs& a, const int32_t* topk_idx, const float* dw,
                                    void* dlogits, long long ld_dlogits, cudaStream_t s);

}  // namespace moe
