// C ABI of the operators around the layer in a training step (declared in
// include/moe.h): argument checks, workspace layout, launches on the caller's
// stream.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "adamw.cuh"
#include "embed.cuh"
#include "kernels.h"
#include "permute.cuh"
#include "sort.cuh"

using namespace moe;

namespace {

constexpr size_t kErrBytes = 256;   // device error word, at the start of a workspace

inline cudaStream_t S(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool known(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F16 || dtype == MOE_F32; }

cudaError_t init_sort() {
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = sort_set_limits();
    if (e != cudaSuccess) return e;
    done[dev] = 1;
  }
  return cudaSuccess;
}

moe_status_t sort_check(int T, int R, int E, int align) {
  if (T < 0 || R <= 0 || E <= 0 || align <= 0) return MOE_ERR_INVALID_ARG;
  if (R > 32 || E > 1024 || align > 4096) return MOE_ERR_UNSUPPORTED;
  if ((long long)T * R >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

long long rows_bound(int T, int R, int E, int align, int capacity) {
  const long long n = (long long)T * R;
  const long long most = (n + std::min<long long>(E, n) * (align - 1)) / align * align;
  if (capacity <= 0) return most;
  const long long each = ((long long)capacity + align - 1) / align * align;
  return std::min(most, E * each);
}

// Checks of the four row-moving calls.  tok and other: [T, d]; rows sides: [N, d].
moe_status_t rows_check(int T, int d, int R, int N, int dtype) {
  if (T < 0 || d <= 0 || R <= 0 || N < 0 || !known(dtype)) return MOE_ERR_INVALID_ARG;
  if (R > 32 || (long long)T * R >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if ((long long)std::max(T, N) * d >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A matrix of `rows` rows that must be there when it has any.
moe_status_t matrix_check(const void* p, long long ld, long long rows, int d, int es) {
  if (rows == 0) return MOE_OK;
  if (!p || ld < d) return MOE_ERR_INVALID_ARG;
  if (ld >= (1LL << 40) / rows) return MOE_ERR_UNSUPPORTED;
  return aligned(p, es) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status_t list_check(const moe_adamw_tensor_t* x, int n, bool grads_only) {
  if (n < 0 || (n > 0 && !x)) return MOE_ERR_INVALID_ARG;
  for (int k = 0; k < n; ++k) {
    const moe_adamw_tensor_t& t = x[k];
    if (t.n < 0) return MOE_ERR_INVALID_ARG;
    if (t.g_dtype != MOE_BF16 && t.g_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
    if (t.n >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
    if (t.n > 0 && !t.g) return MOE_ERR_INVALID_ARG;
    if (!aligned(t.g, dtype_bytes(t.g_dtype))) return MOE_ERR_UNSUPPORTED;
    if (grads_only) continue;
    if (t.p_dtype != MOE_BF16 && t.p_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
    if (t.state_bits != 8 && t.state_bits != 32) return MOE_ERR_UNSUPPORTED;
    if (t.master && t.p_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (!isfinite(t.weight_decay)) return MOE_ERR_INVALID_ARG;
    if (t.n > 0 && (!t.p || !t.m || !t.v)) return MOE_ERR_INVALID_ARG;
    if (t.n > 0 && t.state_bits == 8 && (!t.m_scale || !t.v_scale)) return MOE_ERR_INVALID_ARG;
    const int sb = t.state_bits / 8;
    if (!aligned(t.p, dtype_bytes(t.p_dtype)) || !aligned(t.master, 4) || !aligned(t.m, sb) ||
        !aligned(t.v, sb) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
      return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

#define MOE_NEED(expr)                    \
  do {                                    \
    const moe_status_t st_ = (expr);      \
    if (st_ != MOE_OK) return st_;        \
  } while (0)

}  // namespace

extern "C" {

long long moe_sort_rows_bound(int T, int R, int E, int align, int capacity) {
  return sort_check(T, R, E, align) == MOE_OK ? rows_bound(T, R, E, align, capacity) : -1;
}

moe_status_t moe_sort(const int32_t* topk_idx, int T, int E, int R, int align, int capacity, int N,
                      int32_t* counts, int32_t* offsets, int32_t* row_slot, int32_t* slot_row,
                      void* ws, size_t* ws_bytes, unsigned flags, moe_stream_t stream) {
  MOE_NEED(sort_check(T, R, E, align));
  if (!ws_bytes) return MOE_ERR_INVALID_ARG;
  if (!ws) {
    *ws_bytes = kErrBytes;
    return MOE_OK;
  }
  const long long bound = rows_bound(T, R, E, align, capacity);
  if (bound >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if (N < bound) return MOE_ERR_INVALID_ARG;
  if (*ws_bytes < kErrBytes || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  if (!counts || !offsets || (T > 0 && (!topk_idx || !slot_row)) || (N > 0 && !row_slot))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_idx, 4) || !aligned(counts, 4) || !aligned(offsets, 4) ||
      !aligned(row_slot, 4) || !aligned(slot_row, 4))
    return MOE_ERR_UNSUPPORTED;
  cudaError_t e = init_sort();
  if (e != cudaSuccess) return cuda_failed(e);
  int* err = static_cast<int*>(ws);
  e = launch_sort_slots(topk_idx, T * R, E, align, capacity, N, counts, offsets, row_slot,
                        slot_row, err, S(stream));
  return finish(e, err, flags, S(stream));
}

moe_status_t moe_permute(const void* x, long long ldx, const float* w, const int32_t* row_slot,
                         const int32_t* slot_row, int T, int d, int R, int N, int dtype,
                         void* rows, long long ld_rows, moe_stream_t stream) {
  MOE_NEED(rows_check(T, d, R, N, dtype));
  const int es = dtype_bytes(dtype);
  MOE_NEED(matrix_check(x, ldx, T, d, es));
  MOE_NEED(matrix_check(rows, ld_rows, N, d, es));
  if ((T > 0 && !slot_row) || (N > 0 && !row_slot)) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(slot_row, 4) || !aligned(row_slot, 4)) return MOE_ERR_UNSUPPORTED;
  const PermuteArgs a{T, d, R, N, dtype, {x, ldx}, w, row_slot, slot_row, {nullptr, 0},
                      {rows, ld_rows}, nullptr};
  return finish(launch_spread(a, S(stream)), nullptr, 0, S(stream));
}

moe_status_t moe_permute_bwd(const void* drows, long long ld_drows, const int32_t* slot_row,
                             const float* w, const void* x, long long ldx, int T, int d, int R,
                             int N, int dtype, void* dx, long long ld_dx, float* dw,
                             moe_stream_t stream) {
  MOE_NEED(rows_check(T, d, R, N, dtype));
  const int es = dtype_bytes(dtype);
  MOE_NEED(matrix_check(drows, ld_drows, N, d, es));
  MOE_NEED(matrix_check(dx, ld_dx, T, d, es));
  if ((dw == nullptr) != (x == nullptr) && T > 0) return MOE_ERR_INVALID_ARG;
  if (dw) MOE_NEED(matrix_check(x, ldx, T, d, es));
  if (T > 0 && !slot_row) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(slot_row, 4) || !aligned(dw, 4)) return MOE_ERR_UNSUPPORTED;
  const PermuteArgs a{T, d, R, N, dtype, {drows, ld_drows}, w, nullptr, slot_row, {x, ldx},
                      {dx, ld_dx}, dw};
  return finish(launch_collect(a, S(stream)), nullptr, 0, S(stream));
}

moe_status_t moe_unpermute(const void* rows, long long ld_rows, const int32_t* slot_row,
                           const float* w, int T, int d, int R, int N, int dtype, void* y,
                           long long ldy, moe_stream_t stream) {
  MOE_NEED(rows_check(T, d, R, N, dtype));
  const int es = dtype_bytes(dtype);
  MOE_NEED(matrix_check(rows, ld_rows, N, d, es));
  MOE_NEED(matrix_check(y, ldy, T, d, es));
  if (T > 0 && !slot_row) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(slot_row, 4)) return MOE_ERR_UNSUPPORTED;
  const PermuteArgs a{T, d, R, N, dtype, {rows, ld_rows}, w, nullptr, slot_row, {nullptr, 0},
                      {y, ldy}, nullptr};
  return finish(launch_collect(a, S(stream)), nullptr, 0, S(stream));
}

moe_status_t moe_unpermute_bwd(const void* dy, long long ld_dy, const int32_t* row_slot,
                               const int32_t* slot_row, const float* w, const void* rows,
                               long long ld_rows, int T, int d, int R, int N, int dtype,
                               void* drows, long long ld_drows, float* dw, moe_stream_t stream) {
  MOE_NEED(rows_check(T, d, R, N, dtype));
  const int es = dtype_bytes(dtype);
  MOE_NEED(matrix_check(dy, ld_dy, T, d, es));
  MOE_NEED(matrix_check(drows, ld_drows, N, d, es));
  if ((dw == nullptr) != (rows == nullptr) && T > 0 && N > 0) return MOE_ERR_INVALID_ARG;
  if (dw) MOE_NEED(matrix_check(rows, ld_rows, N, d, es));
  if ((T > 0 && !slot_row) || (N > 0 && !row_slot)) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(slot_row, 4) || !aligned(row_slot, 4) || !aligned(dw, 4))
    return MOE_ERR_UNSUPPORTED;
  const PermuteArgs a{T, d, R, N, dtype, {dy, ld_dy}, w, row_slot, slot_row, {rows, ld_rows},
                      {drows, ld_drows}, dw};
  return finish(launch_spread(a, S(stream)), nullptr, 0, S(stream));
}

moe_status_t moe_embed(const void* ids, int ids_bytes, long long n, const void* table,
                       long long ld_table, int V, int d, int table_dtype, float scale, void* out,
                       long long ld_out, int out_dtype, moe_stream_t stream) {
  if (n < 0 || V <= 0 || d <= 0 || !known(table_dtype) || !known(out_dtype) ||
      (ids_bytes != 4 && ids_bytes != 8))
    return MOE_ERR_INVALID_ARG;
  if (n >= (1LL << 31) || n * d >= (1LL << 40) || (long long)V * d >= (1LL << 40))
    return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!ids) return MOE_ERR_INVALID_ARG;
  MOE_NEED(matrix_check(table, ld_table, V, d, dtype_bytes(table_dtype)));
  MOE_NEED(matrix_check(out, ld_out, n, d, dtype_bytes(out_dtype)));
  if (!aligned(ids, ids_bytes)) return MOE_ERR_UNSUPPORTED;
  const EmbedArgs a{ids, ids_bytes, n, V, d, scale, table_dtype, out_dtype, {table, ld_table},
                    {out, ld_out}, false};
  return finish(launch_embed(a, S(stream)), nullptr, 0, S(stream));
}

moe_status_t moe_embed_bwd(const void* dout, long long ld_dout, const void* ids, int ids_bytes,
                           long long n, int V, int d, int dout_dtype, float scale, void* dtable,
                           long long ld_dtable, int dtable_dtype, void* ws, size_t* ws_bytes,
                           unsigned flags, moe_stream_t stream) {
  if (n < 0 || V <= 0 || d <= 0 || !known(dout_dtype) || !known(dtable_dtype) ||
      (ids_bytes != 4 && ids_bytes != 8))
    return MOE_ERR_INVALID_ARG;
  if (n >= (1LL << 30) || V > (1 << 30) || n * d >= (1LL << 40) || (long long)V * d >= (1LL << 40))
    return MOE_ERR_UNSUPPORTED;
  if (!ws_bytes) return MOE_ERR_INVALID_ARG;
  const size_t need = kErrBytes + embed_bwd_ws_bytes(n, d);
  if (!ws) {
    *ws_bytes = need;
    return MOE_OK;
  }
  if (*ws_bytes < need || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  if (n > 0 && !ids) return MOE_ERR_INVALID_ARG;
  MOE_NEED(matrix_check(dout, ld_dout, n, d, dtype_bytes(dout_dtype)));
  MOE_NEED(matrix_check(dtable, ld_dtable, V, d, dtype_bytes(dtable_dtype)));
  if (!aligned(ids, ids_bytes)) return MOE_ERR_UNSUPPORTED;
  const cudaError_t e = init_sort();
  if (e != cudaSuccess) return cuda_failed(e);
  const EmbedArgs a{ids, ids_bytes, n, V, d, scale, dout_dtype, dtable_dtype, {dout, ld_dout},
                    {dtable, ld_dtable}, (flags & MOE_ACCUMULATE) != 0};
  int* err = static_cast<int*>(ws);
  return finish(launch_embed_bwd(a, static_cast<uint8_t*>(ws) + kErrBytes, err, S(stream)), err,
                flags, S(stream));
}

moe_status_t moe_grad_norm(const moe_adamw_tensor_t* tensors, int n_tensors, double max_norm,
                           float* norm, void* ws, size_t* ws_bytes, moe_stream_t stream) {
  MOE_NEED(list_check(tensors, n_tensors, true));
  if (!ws_bytes || isnan(max_norm)) return MOE_ERR_INVALID_ARG;
  const size_t need = grad_norm_ws_bytes(tensors, n_tensors);
  if (!ws) {
    *ws_bytes = need;
    return MOE_OK;
  }
  if (*ws_bytes < need || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  if (!norm) return MOE_ERR_INVALID_ARG;
  if (!aligned(norm, 16)) return MOE_ERR_UNSUPPORTED;
  return finish(launch_grad_norm(tensors, n_tensors, max_norm, norm, ws, S(stream)), nullptr, 0,
                S(stream));
}

moe_status_t moe_adamw_step(const moe_adamw_tensor_t* tensors, int n_tensors,
                            const moe_adamw_t* settings, const float* norm, moe_stream_t stream) {
  MOE_NEED(list_check(tensors, n_tensors, false));
  if (!settings) return MOE_ERR_INVALID_ARG;
  const moe_adamw_t& h = *settings;
  if (!isfinite(h.lr) || !(h.beta1 >= 0 && h.beta1 < 1) || !(h.beta2 >= 0 && h.beta2 < 1) ||
      !((float)h.eps >= FLT_MIN) || !isfinite((float)h.eps) || h.step < 1)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(norm, 16)) return MOE_ERR_UNSUPPORTED;
  return finish(launch_adamw(tensors, n_tensors, h, norm, S(stream)), nullptr, 0, S(stream));
}

}  // extern "C"
