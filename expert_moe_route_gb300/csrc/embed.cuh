// Launchers of the embedding kernels (embed.cu).
#pragma once

#include "rows.cuh"

namespace moe {

struct EmbedArgs {
  const void* ids;
  int ids_bytes;     // 4 or 8
  long long n;
  int V, d;
  float scale;
  int in_dtype, out_dtype;
  RowsIn in;         // lookup: table [V, d]; gradient: dout [n, d]
  RowsOut out;       // lookup: out [n, d]; gradient: dtable [V, d]
  bool accumulate;   // gradient: dtable += instead of =
};
cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t s);
size_t embed_bwd_ws_bytes(long long n, int d);
cudaError_t launch_embed_bwd(const EmbedArgs& a, void* ws, int* err, cudaStream_t s);

}  // namespace moe
