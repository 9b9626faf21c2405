// Launchers of the experts' products on block-scaled fp8 operands (product_fp8.cu)
// and of their quantiser (quantize_fp8.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

enum ProductMode : int { PRODUCT = 0, PRODUCT_DX = 1, PRODUCT_DW = 2 };

// One call.  PRODUCT: a = x [N, K], b = w [E, n, K], out [N, n].  PRODUCT_DX:
// a = dy [N, n], b = w, out = dx [N, K].  PRODUCT_DW: a = dy [N, n], b = x [N, K],
// out = dw [E, n, K].  Scales: a, and b of PRODUCT_DW, as the quantiser's rows
// (columns for PRODUCT_DW); w in tiles.
struct ProductArgs {
  int mode, N, n, K, E;
  const uint8_t* a;
  const float* sa;
  const uint8_t* b;
  const float* sb;
  const int32_t* offsets;   // [E + 1] on the device, or null: one expert of N rows
  void* out;
  long long ld_out;
  int out_dtype;
  bool accumulate;
};

// Bytes of partial sums that a call of any mode on these sizes may need.
size_t product_fp8_parts_bytes(int N, int n, int K, int E);
cudaError_t launch_product_fp8(const ProductArgs& a, float* parts, int* err, cudaStream_t s);

struct QuantizeArgs {
  const void* x;            // [n, K] rows, ldx apart
  long long ldx;
  int dtype;
  long long n;
  int K;
  uint8_t* row_codes;       // null: not wanted
  float* row_scales;        // [n, ceil(K / 128)]
  uint8_t* col_codes;
  float* col_scales;        // [ceil(n / 128), K]
};
cudaError_t launch_quantize_fp8(const QuantizeArgs& a, cudaStream_t s);
// x [E, n, K] dense; scales [E, ceil(n / 128), ceil(K / 128)]
cudaError_t launch_quantize_fp8_tiles(const void* x, int dtype, int E, int n, int K,
                                      uint8_t* codes, float* scales, cudaStream_t s);

}  // namespace moe
