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

template <typename T, typename O, int W, int G, typename I>
__global__ void __launch_bounds__(ET) embed_kernel(const I* __restrict__ ids, long long n,
                                                   const T* __restrict__ table, long long ldt,
                                                   int V, int d, float scale, O* __restrict__ out,
                                                   long long ldo) {
  constexpr int NG = ET / G;
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  for (long long i = (long long)blockIdx.x * NG + grp; i < n; i += (long long)gridDim.x * NG) {
    const I id = ids[i];
    const bool live = id >= 0 && id < (I)V;
    const T* src = table + (live ? (long long)id : 0) * ldt;
    O* dst = out + i * ldo;
    for (int v0 = gt; v0 < nv; v0 += G * 4) {
      typename Vec<T, W>::Raw q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int v = v0 + u * G;
        q[u] = live && v < nv ? Vec<T, W>::load(src + (long long)v * W) : Vec<T, W>::zero();
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int v = v0 + u * G;
        if (v >= nv) break;
        float f[W];
        Vec<T, W>::unpack(q[u], f);
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = live ? f[j] * scale : 0.f;
        Vec<O, W>::store(dst + (long long)v * W, Vec<O, W>::pack(f));
      }
    }
  }
}

// start[v] = first sorted position whose id is >= v, v = 0..V.
__global__ void __launch_bounds__(ET) starts_kernel(const int2* __restrict__ sorted,
                                                    const int32_t* __restrict__ live, int V,
                                                    int32_t* __restrict__ start) {
  const int n = *live;
  for (long long v = blockIdx.x * (long long)ET + threadIdx.x; v <= V;
       v += (long long)gridDim.x * ET) {
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (sorted[mid].x < (int)v) lo = mid + 1;
      else hi = mid;
    }
    start[v] = lo;
  }
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

// partial[k] = sum of piece k, for the pieces inside one row.
template <typename T, int W, int G>
__global__ void __launch_bounds__(ET) pieces_kernel(const int2* __restrict__ sorted,
                                                    const int32_t* __restrict__ live,
                                                    const T* __restrict__ dout, long long ldd,
                                                    int d, float* __restrict__ partial) {
  constexpr int NG = ET / G;
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  const int pieces = *live / kPiece;
  for (int k = blockIdx.x * NG + grp; k < pieces; k += gridDim.x * NG) {
    const int lo = k * kPiece;
    if (sorted[lo].x != sorted[lo + kPiece - 1].x) continue;
    for (int v = gt; v < nv; v += G) {
      float acc[W];
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] = 0.f;
      add_rows<T, W>(sorted, lo, lo + kPiece, dout, ldd, v, acc);
#pragma unroll
      for (int j = 0; j < W; ++j) partial[(long long)k * d + v * W + j] = acc[j];
    }
  }
}

template <typename T, typename O, int W, int G, bool ADD>
__global__ void __launch_bounds__(ET) table_rows_kernel(
    const int2* __restrict__ sorted, const int32_t* __restrict__ start,
    const T* __restrict__ dout, long long ldd, const float* __restrict__ partial, int V, int d,
    float scale, O* __restrict__ dtable, long long ldt) {
  constexpr int NG = ET / G;
  const int grp = threadIdx.x / G, gt = threadIdx.x % G;
  const int nv = d / W;
  for (long long r = (long long)blockIdx.x * NG + grp; r < V; r += (long long)gridDim.x * NG) {
    const int lo = start[r], hi = start[r + 1];
    if (ADD && lo == hi) continue;
    const int p0 = (lo + kPiece - 1) / kPiece, p1 = hi / kPiece;   // whole pieces in the row
    const int head = p0 < p1 ? p0 * kPiece : hi;
    for (int v = gt; v < nv; v += G) {
      float acc[W];
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] = 0.f;
      add_rows<T, W>(sorted, lo, head, dout, ldd, v, acc);
      for (int p = p0; p < p1; ++p)
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] += partial[(long long)p * d + v * W + j];
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

int grid_for(long long units) { return (int)(units < 152 * 8 ? units : 152 * 8); }

template <typename T, typename O, int W, int G>
cudaError_t embed_t(const EmbedArgs& a, cudaStream_t s) {
  const int blocks = grid_for((a.n + ET / G - 1) / (ET / G));
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
  int32_t* start = live + 64;
  float* partial = reinterpret_cast<float*>(p + 2 * sort_bytes(a.n) +
                                            align_up(sizeof(int32_t) * (64 + (size_t)a.V + 1), 256));
  cudaError_t e = launch_sort_ids(a.ids, a.ids_bytes, (int)a.n, a.V, scratch, sorted, live, err, s);
  if (e != cudaSuccess) return e;
  starts_kernel<<<grid_for((a.V + (long long)ET) / ET), ET, 0, s>>>(sorted, live, a.V, start);
  const int pieces = (int)(a.n / kPiece);
  if (pieces > 0)
    pieces_kernel<T, W, G><<<grid_for((pieces + ET / G - 1) / (ET / G)), ET, 0, s>>>(
        sorted, live, (const T*)a.in.p, a.in.ld, a.d, partial);
  const int blocks = grid_for(((long long)a.V + ET / G - 1) / (ET / G));
  if (a.accumulate)
    table_rows_kernel<T, O, W, G, true><<<blocks, ET, 0, s>>>(
        sorted, start, (const T*)a.in.p, a.in.ld, partial, a.V, a.d, a.scale, (O*)a.out.p,
        a.out.ld);
  else
    table_rows_kernel<T, O, W, G, false><<<blocks, ET, 0, s>>>(
        sorted, start, (const T*)a.in.p, a.in.ld, partial, a.V, a.d, a.scale, (O*)a.out.p,
        a.out.ld);
  count_launches(pieces > 0 ? 3 : 2);
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

size_t embed_bwd_ws_bytes(long long n, int V, int d) {
  return 2 * sort_bytes(n) + align_up(sizeof(int32_t) * (64 + (size_t)V + 1), 256) +
         align_up((size_t)(n / kPiece) * d * sizeof(float), 256);
}

cudaError_t launch_embed_bwd(const EmbedArgs& a, void* ws, int* err, cudaStream_t s) {
  return by_type(a, true, ws, err, s);
}

}  // namespace moe
