// Embedding lookup with a scale, and the table's gradient.
//   out[i] = scale * table[ids[i]]                         (zero for ids outside [0, V))
//   dtable[v] (+)= scale * sum_{i : ids[i] == v} dout[i]
// The gradient sorts the positions by id (sort.cu), so every table row is
// written once by one owner and equal ids are summed in position order: no
// atomics, bitwise reproducible.  The ids of text follow a power law, and the
// commonest may own a tenth of all positions: the sorted list is cut into
// pieces of kPiece positions, a piece that lies inside one row is summed by a
// group of its own into the workspace, and a row's owner adds the pieces and
// the ragged ends in order.
//
// Bound by HBM: n rows read, V rows (or, accumulating, the distinct ones) written.
#include "embed.cuh"
#include "kernels.h"
#include "sort.cuh"

namespace moe {

namespace {
constexpr int ET = 256;
constexpr int kPiece = 64;

// A group of G threads copies kRows rows side by side, so that a thread has that
// many loads in flight although a row is only one or two accesses a thread.
constexpr int kRows = 4;

template <typename T, typename O, int W, int G, typename I>
__global__ void __launch_bounds__(ET) embed_kernel(const I* __restrict__ ids, long long n,
                                                   const T* __restrict__ table, long long ldt,
                                                   int V, int d, float scale, O* __restrict__ out,
                                                   long long ldo) {
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  const long long i0 = ((long long)blockIdx.x * (ET / G) + grp) * kRows;
  const T* src[kRows];
  bool live[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const I id = i0 + u < n ? ids[i0 + u] : (I)-1;
    live[u] = id >= 0 && id < (I)V;
    src[u] = table + (live[u] ? (long long)id : 0) * ldt;
  }
  for (int v = gt; v < nv; v += G) {
    typename Vec<T, W>::Raw q[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      q[u] = live[u] ? Vec<T, W>::load(src[u] + (long long)v * W) : Vec<T, W>::zero();
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (i0 + u >= n) break;
      float f[W];
      Vec<T, W>::unpack(q[u], f);
#pragma unroll
      for (int j = 0; j < W; ++j) f[j] = live[u] ? f[j] * scale : 0.f;
      Vec<O, W>::store(out + (i0 + u) * ldo + (long long)v * W, Vec<O, W>::pack(f));
    }
  }
}

// First of the n sorted positions whose id is >= v.
__device__ __forceinline__ int first_at(const int2* __restrict__ sorted, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (sorted[mid].x < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// acc += dout rows of sorted[lo..hi), in order.
template <typename T, int W>
__device__ __forceinline__ void add_rows(const int2* __restrict__ sorted, int lo, int hi,
                                         const T* __restrict__ dout, long long ldd, int v,
                                         float* acc) {
  for (int k = lo; k < hi; k += 8) {
    typename Vec<T, W>::Raw q[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      q[u] = k + u < hi ? Vec<T, W>::load(dout + (long long)sorted[k + u].y * ldd + (long long)v * W)
                        : Vec<T, W>::zero();
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (k + u >= hi) break;
      float f[W];
      Vec<T, W>::unpack(q[u], f);
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] += f[j];
    }
  }
}

// partial[k] = sum of piece k, for the pieces inside one row.  There are few
// pieces, so a warp takes 32 accesses of a row, not a group the whole row.
template <typename T, int W>
__global__ void __launch_bounds__(ET) pieces_kernel(const int2* __restrict__ sorted,
                                                    const int32_t* __restrict__ live,
                                                    const T* __restrict__ dout, long long ldd,
                                                    int d, int cols, float* __restrict__ partial) {
  const int lane = threadIdx.x & 31;
  const int pieces = *live / kPiece;
  const long long unit = (long long)blockIdx.x * (ET / 32) + threadIdx.x / 32;
  const int k = (int)(unit / cols), v = (int)(unit % cols) * 32 + lane;
  if (k >= pieces) return;
  const int lo = k * kPiece;
  if (sorted[lo].x != sorted[lo + kPiece - 1].x || v >= d / W) return;
  float acc[W];
#pragma unroll
  for (int j = 0; j < W; ++j) acc[j] = 0.f;
  add_rows<T, W>(sorted, lo, lo + kPiece, dout, ldd, v, acc);
  Vec<float, W>::store(partial + (long long)k * d + (long long)v * W, Vec<float, W>::pack(acc));
}

// A group of G threads owns kOwn neighbouring rows of the table.
constexpr int kOwn = 8;

template <typename T, typename O, int W, int G, bool ADD>
__global__ void __launch_bounds__(ET) table_rows_kernel(
    const int2* __restrict__ sorted, const int32_t* __restrict__ live,
    const T* __restrict__ dout, long long ldd, const float* __restrict__ partial, int V, int d,
    float scale, O* __restrict__ dtable, long long ldt) {
  constexpr int NG = ET / G;
  __shared__ int start_s[NG][kOwn + 1];
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  const long long r0 = ((long long)blockIdx.x * NG + grp) * kOwn;
  if (gt <= kOwn)
    start_s[grp][gt] = first_at(sorted, *live, (int)min((long long)V, r0 + gt));
  if (G == 32) __syncwarp();
  else __syncthreads();
  for (int k = 0; k < kOwn; ++k) {
    const long long r = r0 + k;
    if (r >= V) return;
    const int lo = start_s[grp][k], hi = start_s[grp][k + 1];
    if (ADD && lo == hi) continue;
    const int p0 = (lo + kPiece - 1) / kPiece, p1 = hi / kPiece;   // whole pieces in the row
    const int head = p0 < p1 ? p0 * kPiece : hi;
    for (int v = gt; v < nv; v += G) {
      float acc[W];
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] = 0.f;
      add_rows<T, W>(sorted, lo, head, dout, ldd, v, acc);
      for (int p = p0; p < p1; ++p) {
        float part[W];
        Vec<float, W>::unpack(Vec<float, W>::load(partial + (long long)p * d + (long long)v * W), part);
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] += part[j];
      }
      if (p0 < p1) add_rows<T, W>(sorted, p1 * kPiece, hi, dout, ldd, v, acc);
      O* dst = dtable + r * ldt + (long long)v * W;
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] *= scale;
      if (ADD) {
        float old[W];
        Vec<O, W>::unpack(Vec<O, W>::load_rw(dst), old);
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] += old[j];
      }
      Vec<O, W>::store(dst, Vec<O, W>::pack(acc));
    }
  }
}

int blocks_for(long long units, int per_block) { return (int)((units + per_block - 1) / per_block); }

template <typename T, typename O, int W, int G>
cudaError_t embed_t(const EmbedArgs& a, cudaStream_t s) {
  const int blocks = blocks_for(a.n, ET / G * kRows);
  if (a.ids_bytes == 8)
    embed_kernel<T, O, W, G, int64_t><<<blocks, ET, 0, s>>>(
        (const int64_t*)a.ids, a.n, (const T*)a.in.p, a.in.ld, a.V, a.d, a.scale, (O*)a.out.p,
        a.out.ld);
  else
    embed_kernel<T, O, W, G, int32_t><<<blocks, ET, 0, s>>>(
        (const int32_t*)a.ids, a.n, (const T*)a.in.p, a.in.ld, a.V, a.d, a.scale, (O*)a.out.p,
        a.out.ld);
  count_launches(1);
  return cudaGetLastError();
}

size_t sort_bytes(long long n) { return align_up((size_t)n * sizeof(int2), 256); }

template <typename T, typename O, int W, int G>
cudaError_t table_t(const EmbedArgs& a, void* ws, int* err, cudaStream_t s) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  int2* scratch = reinterpret_cast<int2*>(p);
  int2* sorted = reinterpret_cast<int2*>(p + sort_bytes(a.n));
  int32_t* live = reinterpret_cast<int32_t*>(p + 2 * sort_bytes(a.n));
  float* partial = reinterpret_cast<float*>(p + 2 * sort_bytes(a.n) + 256);
  cudaError_t e = launch_sort_ids(a.ids, a.ids_bytes, (int)a.n, a.V, scratch, sorted, live, err, s);
  if (e != cudaSuccess) return e;
  const long long pieces = a.n / kPiece;
  const int cols = blocks_for(a.d / W, 32);
  if (pieces > 0)
    pieces_kernel<T, W><<<blocks_for(pieces * cols, ET / 32), ET, 0, s>>>(
        sorted, live, (const T*)a.in.p, a.in.ld, a.d, cols, partial);
  const int blocks = blocks_for(a.V, ET / G * kOwn);
  if (a.accumulate)
    table_rows_kernel<T, O, W, G, true><<<blocks, ET, 0, s>>>(
        sorted, live, (const T*)a.in.p, a.in.ld, partial, a.V, a.d, a.scale, (O*)a.out.p,
        a.out.ld);
  else
    table_rows_kernel<T, O, W, G, false><<<blocks, ET, 0, s>>>(
        sorted, live, (const T*)a.in.p, a.in.ld, partial, a.V, a.d, a.scale, (O*)a.out.p,
        a.out.ld);
  count_launches(pieces > 0 ? 2 : 1);
  return cudaGetLastError();
}

template <typename T, typename O, int W>
cudaError_t by_length(const EmbedArgs& a, bool grad, void* ws, int* err, cudaStream_t s) {
  if (a.d / W > 64)
    return grad ? table_t<T, O, W, ET>(a, ws, err, s) : embed_t<T, O, W, ET>(a, s);
  return grad ? table_t<T, O, W, 32>(a, ws, err, s) : embed_t<T, O, W, 32>(a, s);
}

// Elements per access: 8 where both sides' rows are 16-byte aligned, 2 where a
// pair is aligned, else 1.
int width(const EmbedArgs& a) {
  const int si = dtype_bytes(a.in_dtype), so = dtype_bytes(a.out_dtype);
  for (int w : {8, 2}) {
    const int bi = w * si < 16 ? w * si : 16, bo = w * so < 16 ? w * so : 16;
    if (a.d % w == 0 && (uintptr_t)a.in.p % bi == 0 && a.in.ld * si % bi == 0 &&
        (uintptr_t)a.out.p % bo == 0 && a.out.ld * so % bo == 0)
      return w;
  }
  return 1;
}

template <typename T, typename O>
cudaError_t by_width(const EmbedArgs& a, bool grad, void* ws, int* err, cudaStream_t s) {
  switch (width(a)) {
    case 8: return by_length<T, O, 8>(a, grad, ws, err, s);
    case 2: return by_length<T, O, 2>(a, grad, ws, err, s);
    default: return by_length<T, O, 1>(a, grad, ws, err, s);
  }
}

template <typename T>
cudaError_t by_out(const EmbedArgs& a, bool grad, void* ws, int* err, cudaStream_t s) {
  if (a.out_dtype == MOE_BF16) return by_width<T, __nv_bfloat16>(a, grad, ws, err, s);
  if (a.out_dtype == MOE_F16) return by_width<T, __half>(a, grad, ws, err, s);
  return by_width<T, float>(a, grad, ws, err, s);
}

cudaError_t by_type(const EmbedArgs& a, bool grad, void* ws, int* err, cudaStream_t s) {
  if (a.in_dtype == MOE_BF16) return by_out<__nv_bfloat16>(a, grad, ws, err, s);
  if (a.in_dtype == MOE_F16) return by_out<__half>(a, grad, ws, err, s);
  return by_out<float>(a, grad, ws, err, s);
}
}  // namespace

cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  return by_type(a, false, nullptr, nullptr, s);
}

size_t embed_bwd_ws_bytes(long long n, int d) {
  return 2 * sort_bytes(n) + 256 + align_up((size_t)(n / kPiece) * d * sizeof(float), 256);
}

cudaError_t launch_embed_bwd(const EmbedArgs& a, void* ws, int* err, cudaStream_t s) {
  return by_type(a, true, ws, err, s);
}

}  // namespace moe
