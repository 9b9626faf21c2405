// C ABI of routing by scores and of the experts' products on block-scaled fp8 (declared in
// include/moe.h): argument checks, workspace layout, launches on the caller's stream.
#include <math.h>

#include "kernels.h"
#include "product_fp8.cuh"
#include "route_scores.cuh"
#include "rows.cuh"

using namespace moe;

namespace {

constexpr size_t kErrBytes = 256;   // device error word, at the start of a workspace

inline cudaStream_t S(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool known(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F16 || dtype == MOE_F32; }

#define MOE_NEED(expr)                    \
  do {                                    \
    const moe_status_t st_ = (expr);      \
    if (st_ != MOE_OK) return st_;        \
  } while (0)

// A matrix of `rows` rows that must be there when it has any.
moe_status_t matrix_check(const void* p, long long ld, long long rows, int d, int es) {
  if (rows == 0) return MOE_OK;
  if (!p || ld < d) return MOE_ERR_INVALID_ARG;
  if (ld >= (1LL << 40) / rows) return MOE_ERR_UNSUPPORTED;
  return aligned(p, es) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status_t router_check(const moe_router_t* r, int T, int E, int R, int dtype) {
  if (!r || T < 0 || E <= 0 || R <= 0 || !known(dtype)) return MOE_ERR_INVALID_ARG;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (R > 32 || E > 1024 || r->groups > 32) return MOE_ERR_UNSUPPORTED;
  if ((long long)T * R >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if (r->groups <= 0 || E % r->groups != 0) return MOE_ERR_INVALID_ARG;
  if (r->top_groups <= 0 || r->top_groups > r->groups) return MOE_ERR_INVALID_ARG;
  const int per_group = E / r->groups;
  if (r->group_keys < 1 || r->group_keys > 2 || (r->groups > 1 && r->group_keys > per_group))
    return MOE_ERR_INVALID_ARG;
  if (R > r->top_groups * per_group) return MOE_ERR_INVALID_ARG;
  return isfinite(r->scale) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// One group: its worth is never asked for.
moe_router_t settled(const moe_router_t& r) {
  moe_router_t s = r;
  if (s.groups == 1) s.group_keys = 1;
  return s;
}

moe_status_t product_sizes(int N, int n, int K, int E) {
  if (N < 0 || n <= 0 || K <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (n % 16 != 0 || K % 16 != 0 || E > 1024 || N > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (n > (1 << 26) || K > (1 << 26)) return MOE_ERR_UNSUPPORTED;
  if ((long long)n * K >= (1LL << 40) / E || (long long)N * (n > K ? n : K) >= (1LL << 40))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The three products: a, b and their scales in the order of ProductArgs.
moe_status_t product(const ProductArgs& p, void* ws, size_t* ws_bytes, unsigned flags,
                     moe_stream_t stream) {
  MOE_NEED(product_sizes(p.N, p.n, p.K, p.E));
  if (!ws_bytes) return MOE_ERR_INVALID_ARG;
  const size_t need = kErrBytes + product_fp8_parts_bytes(p.N, p.n, p.K, p.E);
  if (!ws) {
    *ws_bytes = need;
    return MOE_OK;
  }
  if (*ws_bytes < need || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  const bool dw = p.mode == PRODUCT_DW;
  if (!known(p.out_dtype) || (!p.offsets && p.E != 1)) return MOE_ERR_INVALID_ARG;
  if (p.N > 0 && (!p.a || !p.sa)) return MOE_ERR_INVALID_ARG;
  if ((p.N > 0 || !dw) && (!p.b || !p.sb)) return MOE_ERR_INVALID_ARG;
  const int cols = p.mode == PRODUCT ? p.n : p.K;
  MOE_NEED(matrix_check(p.out, p.ld_out, dw ? (long long)p.E * p.n : p.N, cols,
                        dw ? 16 : dtype_bytes(p.out_dtype)));
  if (!aligned(p.a, 16) || !aligned(p.b, 16) || !aligned(p.sa, 4) || !aligned(p.sb, dw ? 16 : 4) ||
      !aligned(p.offsets, 4))
    return MOE_ERR_UNSUPPORTED;
  int* err = static_cast<int*>(ws);
  if (flags & MOE_CHECK) {          // otherwise nobody reads the word
    const cudaError_t e = cudaMemsetAsync(err, 0, sizeof(int), S(stream));
    if (e != cudaSuccess) return cuda_failed(e);
  }
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kErrBytes);
  return finish(launch_product_fp8(p, parts, err, S(stream)), err, flags, S(stream));
}

}  // namespace

extern "C" {

moe_status_t moe_route_scores(const void* logits, long long ld_logits, int dtype,
                              const float* bias, int T, int E, int R, const moe_router_t* router,
                              int32_t* topk_idx, float* topk_w, moe_stream_t stream) {
  MOE_NEED(router_check(router, T, E, R, dtype));
  MOE_NEED(matrix_check(logits, ld_logits, T, E, dtype_bytes(dtype)));
  if (T > 0 && (!topk_idx || !topk_w)) return MOE_ERR_INVALID_ARG;
  if (!aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4)) return MOE_ERR_UNSUPPORTED;
  const ScoresArgs a{logits, ld_logits, dtype, T, E, R, settled(*router), bias};
  return finish(launch_route_scores(a, topk_idx, topk_w, S(stream)), nullptr, 0, S(stream));
}

moe_status_t moe_route_scores_bwd(const void* logits, long long ld_logits, int dtype,
                                  const int32_t* topk_idx, const float* dw, int T, int E, int R,
                                  const moe_router_t* router, void* dlogits,
                                  long long ld_dlogits, moe_stream_t stream) {
  MOE_NEED(router_check(router, T, E, R, dtype));
  MOE_NEED(matrix_check(logits, ld_logits, T, E, dtype_bytes(dtype)));
  MOE_NEED(matrix_check(dlogits, ld_dlogits, T, E, dtype_bytes(dtype)));
  if (T > 0 && (!topk_idx || !dw)) return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_idx, 4) || !aligned(dw, 4)) return MOE_ERR_UNSUPPORTED;
  const ScoresArgs a{logits, ld_logits, dtype, T, E, R, settled(*router), nullptr};
  return finish(launch_route_scores_bwd(a, topk_idx, dw, dlogits, ld_dlogits, S(stream)), nullptr,
                0, S(stream));
}

moe_status_t moe_quantize_fp8(const void* x, long long ldx, int dtype, int N, int K,
                              uint8_t* row_codes, float* row_scales, uint8_t* col_codes,
                              float* col_scales, moe_stream_t stream) {
  if (N < 0 || K <= 0 || !known(dtype)) return MOE_ERR_INVALID_ARG;
  if ((row_codes == nullptr) != (row_scales == nullptr) ||
      (col_codes == nullptr) != (col_scales == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (N > 0 && !row_codes && !col_codes) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || N > (1 << 30) || (long long)N * K >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  MOE_NEED(matrix_check(x, ldx, N, K, dtype_bytes(dtype)));
  if (!aligned(row_codes, 16) || !aligned(col_codes, 16) || !aligned(row_scales, 4) ||
      !aligned(col_scales, 4))
    return MOE_ERR_UNSUPPORTED;
  const QuantizeArgs a{x, ldx, dtype, N, K, row_codes, row_scales, col_codes, col_scales};
  return finish(launch_quantize_fp8(a, S(stream)), nullptr, 0, S(stream));
}

moe_status_t moe_quantize_fp8_tiles(const void* w, int dtype, int E, int n, int K, uint8_t* codes,
                                    float* scales, moe_stream_t stream) {
  if (E < 0 || n <= 0 || K <= 0 || !known(dtype)) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || (long long)n * K >= (1LL << 40) / (E > 0 ? E : 1)) return MOE_ERR_UNSUPPORTED;
  if (E > 0 && (!w || !codes || !scales)) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, dtype_bytes(dtype)) || !aligned(codes, 16) || !aligned(scales, 4))
    return MOE_ERR_UNSUPPORTED;
  return finish(launch_quantize_fp8_tiles(w, dtype, E, n, K, codes, scales, S(stream)), nullptr, 0,
                S(stream));
}

moe_status_t moe_product_fp8(const uint8_t* xq, const float* xs, const int32_t* offsets, int N,
                             int n, int K, int E, const uint8_t* wq, const float* wscale,
                             void* out, long long ld_out, int out_dtype, void* ws,
                             size_t* ws_bytes, unsigned flags, moe_stream_t stream) {
  return product({PRODUCT, N, n, K, E, xq, xs, wq, wscale, offsets, out, ld_out, out_dtype, false},
                 ws, ws_bytes, flags, stream);
}

moe_status_t moe_product_fp8_dx(const uint8_t* dyq, const float* dys, const int32_t* offsets,
                                int N, int n, int K, int E, const uint8_t* wq,
                                const float* wscale, void* dx, long long ld_dx, int dx_dtype,
                                void* ws, size_t* ws_bytes, unsigned flags, moe_stream_t stream) {
  return product({PRODUCT_DX, N, n, K, E, dyq, dys, wq, wscale, offsets, dx, ld_dx, dx_dtype, false},
                 ws, ws_bytes, flags, stream);
}

moe_status_t moe_product_fp8_dw(const uint8_t* dyq, const float* dys, const uint8_t* xq,
                                const float* xs, const int32_t* offsets, int N, int n, int K,
                                int E, void* dw, int dw_dtype, void* ws, size_t* ws_bytes,
                                unsigned flags, moe_stream_t stream) {
  return product({PRODUCT_DW, N, n, K, E, dyq, dys, xq, xs, offsets, dw, K, dw_dtype,
                  (flags & MOE_ACCUMULATE) != 0},
                 ws, ws_bytes, flags, stream);
}

}  // extern "C"
