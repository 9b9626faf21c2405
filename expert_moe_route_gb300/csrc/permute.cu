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
// Both are bound by HBM.  A group of threads owns a token: x[t] is read once for
// its R rows (row by row it would be read R times, from all over the sorted
// order).
#include <algorithm>

#include "kernels.h"
#include "permute.cuh"

namespace moe {

namespace {
constexpr int PT = 256;              // threads per block
constexpr int kMaxR = 32;
constexpr int kGroup = 128;          // threads per token of a long row
// Threads of a block whose groups of G own a token each.
constexpr int threads_of(int G) { return G > PT / 8 ? G : PT; }

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

// dw[r] = acc[r] summed over the group (32 or kGroup threads); slots without a row
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

// Rows without a slot are zero.  They come in runs (the ends of segments), so
// neighbouring rows go to different groups; a group looks at 32 rows at a time.
template <typename T, int G, int BT>
__device__ __forceinline__ void zero_rows(const int32_t* __restrict__ row_slot, int N, int d,
                                          T* __restrict__ rows, long long ldr) {
  constexpr int NG = BT / G;
  const int grp = threadIdx.x / G, gt = threadIdx.x % G, lane = threadIdx.x & 31;
  const long long groups = (long long)gridDim.x * NG;
  for (long long i = (long long)blockIdx.x * NG + grp; i < N; i += groups * 32) {
    const long long mine = i + lane * groups;
    unsigned empty = __ballot_sync(kFull, mine < N && row_slot[mine] < 0);
    while (empty) {
      const long long row = i + (__ffs(empty) - 1) * groups;
      empty &= empty - 1;
      zero_span<T, G>(rows + row * ldr, d, gt);
    }
  }
}

// Spread without dot products: a warp takes 32 * kWide accesses of a token's row
// and writes them to its R rows, 2 KB apiece where the row is long: the loads are
// in flight together and a few tokens still fill the card.  T = 16384, d = 4096,
// R = 8, weighted, segments of 128: 198 us for 1.34 GB; T = 128, d = 7168, 4864 rows:
// 13 us, of which the zero rows are four fifths.
constexpr int kWide = 4;

template <typename T, int W>
__global__ void __launch_bounds__(PT) spread_kernel(
    const T* __restrict__ x, long long ldx, const float* __restrict__ w,
    const int32_t* __restrict__ row_slot, const int32_t* __restrict__ slot_row, int T_, int d,
    int R, int N, int cols, T* __restrict__ rows, long long ldr) {
  using V = Vec<T, W>;
  const int lane = threadIdx.x & 31;
  const int nv = d / W;
  const long long unit = (long long)blockIdx.x * (PT / 32) + threadIdx.x / 32;
  const long long t = unit / cols;
  if (t < T_) {
    const int v0 = (int)(unit % cols) * (32 * kWide) + lane;
    int my_row = -1;
    float my_w = 1.f;
    if (lane < R) {
      my_row = slot_row[t * R + lane];
      if (w) my_w = w[t * R + lane];
    }
    typename V::Raw q[kWide];
#pragma unroll
    for (int u = 0; u < kWide; ++u)
      q[u] = v0 + 32 * u < nv ? V::load(x + t * ldx + (long long)(v0 + 32 * u) * W) : V::zero();
    for (int r = 0; r < R; ++r) {
      const int row = __shfl_sync(kFull, my_row, r);
      const float wr = __shfl_sync(kFull, my_w, r);
      if ((unsigned)row >= (unsigned)N) continue;
      T* dst = rows + row * ldr;
#pragma unroll
      for (int u = 0; u < kWide; ++u) {
        if (v0 + 32 * u >= nv) break;
        if (w) {
          float f[W];
          V::unpack(q[u], f);
#pragma unroll
          for (int j = 0; j < W; ++j) f[j] *= wr;
          V::store(dst + (long long)(v0 + 32 * u) * W, V::pack(f));
        } else {
          V::store(dst + (long long)(v0 + 32 * u) * W, q[u]);
        }
      }
    }
  }
  // a warp a row up to 2 KB (1024 tokens over 512 experts in segments of 128, with the
  // plan: d 512 18.6 us, a block 38.9; d 1024 29.1, 41.9), a block for longer ones (d 2048
  // 52.9, a warp 50.3; 128 tokens over 256 experts, d 7168: 78.8, 76.3)
  if (d * sizeof(T) > 2048) zero_rows<T, PT, PT>(row_slot, N, d, rows, ldr);
  else zero_rows<T, 32, PT>(row_slot, N, d, rows, ldr);
}

// Spread with dot products: a group of threads owns a token.
template <typename T, int W, int G, int RM>
__global__ void __launch_bounds__(threads_of(G)) spread_dots_kernel(
    const T* __restrict__ x, long long ldx, const float* __restrict__ w,
    const int32_t* __restrict__ row_slot, const int32_t* __restrict__ slot_row, int T_, int d,
    int R, int N, const T* __restrict__ other, long long ldo, T* __restrict__ rows,
    long long ldr, float* __restrict__ dw) {
  constexpr int BT = threads_of(G), NG = BT / G;
  __shared__ int rows_s[NG][kMaxR];
  __shared__ float w_s[NG][kMaxR];
  __shared__ float red[G > 32 ? G / 32 * RM : 1];
  using V = Vec<T, W>;
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  auto sync = [] { if (G == 32) __syncwarp(); else __syncthreads(); };
  const long long t = (long long)blockIdx.x * NG + grp;
  if (t < T_) {
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
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = r0 + u < R ? rows_s[grp][r0 + u] : -1;
          q[u] = row >= 0 ? V::load(other + row * ldo + (long long)v * W) : V::zero();
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = r0 + u;
          if (r >= R) break;
          const int row = rows_s[grp][r];
          if (row < 0) continue;
          const float wr = w_s[grp][r];
          float out[W], o[W];
          V::unpack(q[u], o);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            out[j] = wr * g[j];
            acc[r] = fmaf(g[j], o[j], acc[r]);
          }
          V::store(rows + row * ldr + (long long)v * W, V::pack(out));
        }
      }
    }
    store_dots<G, RM>(acc, rows_s[grp], R, red, dw + t * R);
  }
  zero_rows<T, G, BT>(row_slot, N, d, rows, ldr);
}

template <typename T, int W, int G, int RM, bool DOTS>
__global__ void __launch_bounds__(threads_of(G)) collect_kernel(
    const T* __restrict__ rows, long long ldr, const int32_t* __restrict__ slot_row,
    const float* __restrict__ w, int T_, int d, int R, int N, const T* __restrict__ other,
    long long ldo, T* __restrict__ y, long long ldy, float* __restrict__ dw) {
  constexpr int BT = threads_of(G), NG = BT / G;
  __shared__ int rows_s[NG][kMaxR];
  __shared__ float w_s[NG][kMaxR];
  __shared__ float red[DOTS && G > 32 ? G / 32 * RM : 1];
  using V = Vec<T, W>;
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  auto sync = [] { if (G == 32) __syncwarp(); else __syncthreads(); };
  const long long t = (long long)blockIdx.x * NG + grp;
  if (t < T_) {
    if (gt < R) {
      const int row = slot_row[t * R + gt];
      rows_s[grp][gt] = (unsigned)row < (unsigned)N ? row : -1;
      w_s[grp][gt] = w ? w[t * R + gt] : 1.f;
    }
    sync();
    float acc[RM];
#pragma unroll
    for (int r = 0; r < RM; ++r) acc[r] = 0.f;
    // eight row accesses in flight: RB rows of a column, C columns
    constexpr int RB = RM < 8 ? RM : 8, C = 8 / RB;
    for (int v0 = gt; v0 < nv; v0 += G * C) {
      float sum[C][W];
      typename V::Raw mine[DOTS ? C : 1];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int v = v0 + c * G;
#pragma unroll
        for (int j = 0; j < W; ++j) sum[c][j] = 0.f;
        if (DOTS) mine[c] = v < nv ? V::load(other + t * ldo + (long long)v * W) : V::zero();
      }
#pragma unroll
      for (int r0 = 0; r0 < RM; r0 += RB) {
        if (r0 >= R) break;
        typename V::Raw q[C][RB];
#pragma unroll
        for (int u = 0; u < RB; ++u) {
          const int row = r0 + u < R ? rows_s[grp][r0 + u] : -1;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int v = v0 + c * G;
            q[c][u] = row >= 0 && v < nv ? V::load(rows + row * ldr + (long long)v * W) : V::zero();
          }
        }
#pragma unroll
        for (int u = 0; u < RB; ++u) {
          const int r = r0 + u;
          if (r >= R || rows_s[grp][r] < 0) continue;
          const float wr = w_s[grp][r];
#pragma unroll
          for (int c = 0; c < C; ++c) {
            float o[W], g[W];
            V::unpack(q[c][u], o);
            if (DOTS) V::unpack(mine[c], g);
#pragma unroll
            for (int j = 0; j < W; ++j) {
              sum[c][j] = fmaf(wr, o[j], sum[c][j]);
              if (DOTS) acc[r] = fmaf(g[j], o[j], acc[r]);
            }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (v0 + c * G < nv) V::store(y + t * ldy + (long long)(v0 + c * G) * W, V::pack(sum[c]));
    }
    if (DOTS) store_dots<G, RM>(acc, rows_s[grp], R, red, dw + t * R);
  }
}

// Blocks that look for rows without a slot: eight an SM, or one for 32 rows.
long long blocks_for_zeros(int N) { return std::max((N + 31LL) / 32, std::min<long long>(N, 152 * 8)); }

template <typename T, int W>
cudaError_t spread_t(const PermuteArgs& a, cudaStream_t s) {
  const int cols = std::max(1, (a.d / W + 32 * kWide - 1) / (32 * kWide));
  const long long units = ((long long)a.T * cols + PT / 32 - 1) / (PT / 32);
  const int blocks = (int)std::max(units, blocks_for_zeros(a.N));
  spread_kernel<T, W><<<blocks, PT, 0, s>>>((const T*)a.tok.p, a.tok.ld, a.w, a.row_slot,
                                            a.slot_row, a.T, a.d, a.R, a.N, cols, (T*)a.out.p,
                                            a.out.ld);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int W, int G, int RM>
cudaError_t spread_dots_t(const PermuteArgs& a, cudaStream_t s) {
  constexpr int BT = threads_of(G);
  const long long units = ((long long)a.T + BT / G - 1) / (BT / G);
  const int blocks = (int)std::max(units, blocks_for_zeros(a.N));
  spread_dots_kernel<T, W, G, RM><<<blocks, BT, 0, s>>>(
      (const T*)a.tok.p, a.tok.ld, a.w, a.row_slot, a.slot_row, a.T, a.d, a.R, a.N,
      (const T*)a.other.p, a.other.ld, (T*)a.out.p, a.out.ld, a.dw);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int W, int G, int RM>
cudaError_t collect_t(const PermuteArgs& a, cudaStream_t s) {
  constexpr int BT = threads_of(G);
  const int blocks = (int)(((long long)a.T + BT / G - 1) / (BT / G));
  if (a.dw)
    collect_kernel<T, W, G, RM, true><<<blocks, BT, 0, s>>>(
        (const T*)a.tok.p, a.tok.ld, a.slot_row, a.w, a.T, a.d, a.R, a.N, (const T*)a.other.p,
        a.other.ld, (T*)a.out.p, a.out.ld, a.dw);
  else
    collect_kernel<T, W, G, RM, false><<<blocks, BT, 0, s>>>(
        (const T*)a.tok.p, a.tok.ld, a.slot_row, a.w, a.T, a.d, a.R, a.N, nullptr, 0,
        (T*)a.out.p, a.out.ld, nullptr);
  count_launches(1);
  return cudaGetLastError();
}

// A block of 128 per token for rows of over 128 accesses, a warp for shorter ones
// (d = 512, T = 16384, R = 8, moe_unpermute_bwd: 51 us, a block 72) unless the tokens
// are so few that a warp each does not fill the card (d = 1024, T = 512: 6.2 us, a
// warp 10.3).
// moe_permute_bwd, T = 4096, d = 2048, R = 6: 23 us (a warp 40, a block of 256 29:
// few blocks fit an SM and each waits for its one round of loads);
// moe_unpermute_bwd, T = 16384, d = 4096, R = 8: 356 us (373, 361);
// moe_unpermute, T = 65536, d = 7168, R = 8: 1.16 ms (1.23, 1.17).  A block takes one
// token: persistent blocks were 5 to 15% slower, with or without the next token's
// plan read ahead.
template <typename T, int W> cudaError_t by_shape(const PermuteArgs& a, bool spread, cudaStream_t s) {
  if (spread && !a.dw) return spread_t<T, W>(a, s);
  const bool wide = a.d / W > 128 || (a.d / W > 32 && a.T < 152 * 16);
  if (spread) {
    if (a.R <= 8) return wide ? spread_dots_t<T, W, kGroup, 8>(a, s) : spread_dots_t<T, W, 32, 8>(a, s);
    return wide ? spread_dots_t<T, W, kGroup, 32>(a, s) : spread_dots_t<T, W, 32, 32>(a, s);
  }
  if (a.R <= 2) return wide ? collect_t<T, W, kGroup, 2>(a, s) : collect_t<T, W, 32, 2>(a, s);
  if (a.R <= 8) return wide ? collect_t<T, W, kGroup, 8>(a, s) : collect_t<T, W, 32, 8>(a, s);
  return wide ? collect_t<T, W, kGroup, 32>(a, s) : collect_t<T, W, 32, 32>(a, s);
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
