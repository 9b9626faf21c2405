// Rows to and from expert order, with the gate weights and their gradients.
// With row(t, r) = slot_row[t*R + r] (a slot without a row contributes nothing):
//   spread:   rows[row(t, r)] = w[t, r] x[t]            moe_permute
//             dw[t, r] = <x[t], other[row(t, r)]>       moe_unpermute_bwd, x = dy
//   collect:  y[t] = sum_r w[t, r] rows[row(t, r)]      moe_unpermute
//             dw[t, r] = <other[t], rows[row(t, r)]>    moe_permute_bwd
// fp32 products and sums in r order, one rounding at the store; dot products are
// summed per thread over its columns, then over the threads in a fixed order, so
// every result is bitwise reproducible.
//
// Both are bound by HBM.  A group of threads (a warp for short rows, a block for
// long ones) owns a token: x[t] is read once for its R rows (row by row it would
// be read R times, from all over the sorted order).
#include <algorithm>

#include "kernels.h"
#include "permute.cuh"

namespace moe {

namespace {
constexpr int PT = 256;              // threads per block
constexpr int kMaxR = 32;

// Sums each of acc[0..RM) over the warp: every exchange halves the values a lane
// still holds, RM - 1 + log2(32 / RM) shuffles instead of 5 RM.  Lane
// r * (32 / RM) ends with the sum of acc[r] in acc[0].
template <int RM>
__device__ __forceinline__ void warp_sums(float (&acc)[RM]) {
  const int lane = threadIdx.x & 31;
  int off = 16;
#pragma unroll
  for (int n = RM; n > 1; n /= 2, off /= 2) {
    const bool hi = lane & off;
#pragma unroll
    for (int i = 0; i < RM / 2; ++i) {
      if (i >= n / 2) break;
      const float send = hi ? acc[i] : acc[i + n / 2];
      const float keep = hi ? acc[i + n / 2] : acc[i];
      acc[i] = keep + __shfl_xor_sync(kFull, send, off);
    }
  }
#pragma unroll
  for (; off > 0; off /= 2) acc[0] += __shfl_xor_sync(kFull, acc[0], off);
}

// dw[r] = acc[r] summed over the group (32 or PT threads); slots without a row
// get 0.  Ends with the group's threads in step when G > 32.
template <int G, int RM>
__device__ __forceinline__ void store_dots(float (&acc)[RM], const int* rows_s, int R, float* red,
                                           float* dw) {
  constexpr int STEP = 32 / RM;
  const int lane = threadIdx.x & 31, gt = threadIdx.x % G;
  warp_sums<RM>(acc);
  const int r = lane / STEP;
  if (G == 32) {
    if (lane % STEP == 0 && r < R) dw[r] = rows_s[r] >= 0 ? acc[0] : 0.f;
    return;
  }
  if (lane % STEP == 0) red[gt / 32 * RM + r] = acc[0];
  __syncthreads();
  if (gt < R) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < G / 32; ++w) s += red[w * RM + gt];
    dw[gt] = rows_s[gt] >= 0 ? s : 0.f;
  }
}

template <typename T, int W, int G, int RM, bool DOTS>
__global__ void __launch_bounds__(PT) spread_kernel(
    const T* __restrict__ x, long long ldx, const float* __restrict__ w,
    const int32_t* __restrict__ row_slot, const int32_t* __restrict__ slot_row, int T_, int d,
    int R, int N, const T* __restrict__ other, long long ldo, T* __restrict__ rows,
    long long ldr, float* __restrict__ dw) {
  constexpr int NG = PT / G;
  __shared__ int rows_s[NG][kMaxR];
  __shared__ float w_s[NG][kMaxR];
  __shared__ float red[DOTS && G > 32 ? PT / 32 * RM : 1];
  using V = Vec<T, W>;
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  auto sync = [] { if (G == 32) __syncwarp(); else __syncthreads(); };
  for (long long t = (long long)blockIdx.x * NG + grp; t < T_; t += (long long)gridDim.x * NG) {
    if (gt < R) {
      const int row = slot_row[t * R + gt];
      rows_s[grp][gt] = (unsigned)row < (unsigned)N ? row : -1;
      w_s[grp][gt] = w ? w[t * R + gt] : 1.f;
    }
    sync();
    float acc[RM];
#pragma unroll
    for (int r = 0; r < RM; ++r) acc[r] = 0.f;
    for (int v = gt; v < nv; v += G) {
      float g[W];
      V::unpack(V::load(x + t * ldx + (long long)v * W), g);
#pragma unroll
      for (int r0 = 0; r0 < RM; r0 += 4) {
        if (r0 >= R) break;
        typename V::Raw q[4];
        if (DOTS) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = r0 + u < R ? rows_s[grp][r0 + u] : -1;
            q[u] = row >= 0 ? V::load(other + row * ldo + (long long)v * W) : V::zero();
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = r0 + u;
          if (r >= R) break;
          const int row = rows_s[grp][r];
          if (row < 0) continue;
          const float wr = w_s[grp][r];
          float out[W];
#pragma unroll
          for (int j = 0; j < W; ++j) out[j] = wr * g[j];
          V::store(rows + row * ldr + (long long)v * W, V::pack(out));
          if (DOTS) {
            float o[W];
            V::unpack(q[u], o);
#pragma unroll
            for (int j = 0; j < W; ++j) acc[r] = fmaf(g[j], o[j], acc[r]);
          }
        }
      }
    }
    if (DOTS) store_dots<G, RM>(acc, rows_s[grp], R, red, dw + t * R);
    sync();
  }
  // Rows without a slot are zero.  They come in runs (the ends of segments), so
  // neighbouring rows go to different groups; a group looks at 32 rows at a time.
  const int lane = threadIdx.x & 31;
  const long long groups = (long long)gridDim.x * NG;
  for (long long i = (long long)blockIdx.x * NG + grp; i < N; i += groups * 32) {
    const long long mine = i + lane * groups;
    unsigned empty = __ballot_sync(kFull, mine < N && row_slot[mine] < 0);
    while (empty) {
      const long long row = i + (__ffs(empty) - 1) * groups;
      empty &= empty - 1;
      for (int v = gt; v < nv; v += G) V::store(rows + row * ldr + (long long)v * W, V::zero());
    }
  }
}

template <typename T, int W, int G, int RM, bool DOTS>
__global__ void __launch_bounds__(PT) collect_kernel(
    const T* __restrict__ rows, long long ldr, const int32_t* __restrict__ slot_row,
    const float* __restrict__ w, int T_, int d, int R, int N, const T* __restrict__ other,
    long long ldo, T* __restrict__ y, long long ldy, float* __restrict__ dw) {
  constexpr int NG = PT / G;
  __shared__ int rows_s[NG][kMaxR];
  __shared__ float w_s[NG][kMaxR];
  __shared__ float red[DOTS && G > 32 ? PT / 32 * RM : 1];
  using V = Vec<T, W>;
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  auto sync = [] { if (G == 32) __syncwarp(); else __syncthreads(); };
  for (long long t = (long long)blockIdx.x * NG + grp; t < T_; t += (long long)gridDim.x * NG) {
    if (gt < R) {
      const int row = slot_row[t * R + gt];
      rows_s[grp][gt] = (unsigned)row < (unsigned)N ? row : -1;
      w_s[grp][gt] = w ? w[t * R + gt] : 1.f;
    }
    sync();
    float acc[RM];
#pragma unroll
    for (int r = 0; r < RM; ++r) acc[r] = 0.f;
    for (int v = gt; v < nv; v += G) {
      float sum[W], g[W];
#pragma unroll
      for (int j = 0; j < W; ++j) sum[j] = 0.f;
      if (DOTS) V::unpack(V::load(other + t * ldo + (long long)v * W), g);
#pragma unroll
      for (int r0 = 0; r0 < RM; r0 += 8) {
        if (r0 >= R) break;
        typename V::Raw q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int row = r0 + u < R ? rows_s[grp][r0 + u] : -1;
          q[u] = row >= 0 ? V::load(rows + row * ldr + (long long)v * W) : V::zero();
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = r0 + u;
          if (r >= R || rows_s[grp][r] < 0) continue;
          const float wr = w_s[grp][r];
          float o[W];
          V::unpack(q[u], o);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            sum[j] = fmaf(wr, o[j], sum[j]);
            if (DOTS) acc[r] = fmaf(g[j], o[j], acc[r]);
          }
        }
      }
      V::store(y + t * ldy + (long long)v * W, V::pack(sum));
    }
    if (DOTS) store_dots<G, RM>(acc, rows_s[grp], R, red, dw + t * R);
    sync();
  }
}

template <typename T, int W, int G, int RM>
cudaError_t spread_t(const PermuteArgs& a, cudaStream_t s) {
  const long long units = std::max<long long>(a.T, (a.N + 7) / 8);
  const int blocks = (int)((units + PT / G - 1) / (PT / G));
  if (a.dw)
    spread_kernel<T, W, G, RM, true><<<blocks, PT, 0, s>>>(
        (const T*)a.tok.p, a.tok.ld, a.w, a.row_slot, a.slot_row, a.T, a.d, a.R, a.N,
        (const T*)a.other.p, a.other.ld, (T*)a.out.p, a.out.ld, a.dw);
  else
    spread_kernel<T, W, G, RM, false><<<blocks, PT, 0, s>>>(
        (const T*)a.tok.p, a.tok.ld, a.w, a.row_slot, a.slot_row, a.T, a.d, a.R, a.N, nullptr, 0,
        (T*)a.out.p, a.out.ld, nullptr);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int W, int G, int RM>
cudaError_t collect_t(const PermuteArgs& a, cudaStream_t s) {
  const int blocks = (int)(((long long)a.T + PT / G - 1) / (PT / G));
  if (a.dw)
    collect_kernel<T, W, G, RM, true><<<blocks, PT, 0, s>>>(
        (const T*)a.tok.p, a.tok.ld, a.slot_row, a.w, a.T, a.d, a.R, a.N, (const T*)a.other.p,
        a.other.ld, (T*)a.out.p, a.out.ld, a.dw);
  else
    collect_kernel<T, W, G, RM, false><<<blocks, PT, 0, s>>>(
        (const T*)a.tok.p, a.tok.ld, a.slot_row, a.w, a.T, a.d, a.R, a.N, nullptr, 0,
        (T*)a.out.p, a.out.ld, nullptr);
  count_launches(1);
  return cudaGetLastError();
}

// A block per token for rows of over 128 accesses, a warp for shorter ones.  At
// T = 16384, d = 4096 bf16 a block takes 362 us for moe_unpermute_bwd and a warp
// 373, at T = 4096, d = 2048 moe_permute_bwd 29 and 40 us: a warp's rows wait for
// one another.
template <typename T, int W> cudaError_t by_shape(const PermuteArgs& a, bool spread, cudaStream_t s) {
  const bool wide = a.d / W > 128;
  if (a.R <= 8) {
    if (spread) return wide ? spread_t<T, W, PT, 8>(a, s) : spread_t<T, W, 32, 8>(a, s);
    return wide ? collect_t<T, W, PT, 8>(a, s) : collect_t<T, W, 32, 8>(a, s);
  }
  if (spread) return wide ? spread_t<T, W, PT, 32>(a, s) : spread_t<T, W, 32, 32>(a, s);
  return wide ? collect_t<T, W, PT, 32>(a, s) : collect_t<T, W, 32, 32>(a, s);
}

template <typename T> cudaError_t by_width(const PermuteArgs& a, bool spread, cudaStream_t s) {
  const RowsIn in[] = {a.tok, a.other};
  const RowsOut out[] = {a.out};
  const int b = access_bytes(a.dtype, a.d, in, 2, out, 1);
  if (b == 16) return by_shape<T, 16 / sizeof(T)>(a, spread, s);
  if (b == 4) return by_shape<T, 4 / sizeof(T)>(a, spread, s);
  return by_shape<T, 1>(a, spread, s);
}

cudaError_t by_type(const PermuteArgs& a, bool spread, cudaStream_t s) {
  if (a.dtype == MOE_BF16) return by_width<__nv_bfloat16>(a, spread, s);
  if (a.dtype == MOE_F16) return by_width<__half>(a, spread, s);
  return by_width<float>(a, spread, s);
}
}  // namespace

cudaError_t launch_spread(const PermuteArgs& a, cudaStream_t s) {
  if (a.N == 0 && (a.T == 0 || !a.dw)) return cudaSuccess;
  return by_type(a, true, s);
}
cudaError_t launch_collect(const PermuteArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  return by_type(a, false, s);
}

}  // namespace moe
