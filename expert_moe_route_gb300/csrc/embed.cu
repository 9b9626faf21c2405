// Embedding lookup with a scale, and the table's gradient.
//   out[i] = scale * table[ids[i]]                         (zero for ids outside [0, V))
//   dtable[v] (+)= scale * sum_{i : ids[i] == v} dout[i]
// The gradient sorts the positions by id (sort.cu), so every table row is
// written once by one owner and equal ids are summed in position order: bitwise
// reproducible (the one atomic hands out list slots in any order).  The ids of text follow a power law, and the
// commonest may own a tenth of all positions, so the work is cut by positions of
// the sorted list, not by rows.
//
// Bound by HBM: n rows read, V rows (or, accumulating, the distinct ones) written.
#include "embed.cuh"
#include "kernels.h"
#include "sort.cuh"

namespace moe {

namespace {
constexpr int ET = 256;
constexpr int kPiece = 32;

// A group of G threads copies kRows rows side by side, so that a thread has that
// many loads in flight although a row is only one or two accesses a thread.  Bound
// by HBM: 32768 ids, V = 65536, d = 4096 bf16 (354 MB) 57 us; one row at a time 64.
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

// First sorted position whose id is >= v.
__device__ __forceinline__ int first_at(const int2* sorted, const SortedHead* head, int shift,
                                        int v) {
  int lo = head->top[v >> shift], hi = head->top[(v >> shift) + 1];
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (sorted[mid].x < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// A row that spans pieces: its first piece, its id, how many pieces it touches.
struct Span {
  int first, id, pieces, pad;
};

// The sorted list is cut into pieces of kPiece positions.  A warp takes a piece
// and 32 accesses of the row length, walks the positions and writes a table row
// where one ends.  A row that goes past the piece's end leaves its part in
// parts[2 k + 1] and k in `spans`, one that came in from the piece before in
// parts[2 k] (as does one that fills the whole piece); joined_kernel adds those.
//
// The rows come by asynchronous copies into shared memory, sixteen in flight a
// warp: held in registers they left 15 warps an SM (91 registers; now 24 warps,
// 50).  16384 ids, 65536 x 4096 fp32: 174 us for 1.18 GB, most of it zeros;
// 49999 ids added into 32003 x 2048: 62 us for 0.33 GB, bound by latency.
//
// What the kernel before wrote is read with plain loads (no __restrict__, no
// __ldg): a load of constant data might be moved above wait_for_previous().
constexpr int RT = 128;          // threads a block of rows_kernel
// Whole gradients in a graph, A: 16384 ids, 65536 x 4096, overwritten, 193 us; B: 49999 ids
// added into 32003 x 2048, 88 us.
constexpr int kFlight = 16;      // positions whose rows a warp has in flight (8: A 209, B 86)
constexpr int kGroup = 4;        // positions waited for together (2: B 94, 8: 89; A the same)
constexpr int kOwn = 8;          // rows a warp looks through for rows without a token (4: A 186,
                                 // 16: 209)
constexpr int kLong = 4;         // a row of more pieces is joined by a block (2: B 89, 16: 91)

// Copies of a lane's accesses: 4, 8 or 16 bytes on their way into shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from),
                 "n"(BYTES < 4 ? 4 : BYTES) : "memory");
}

template <typename T, typename O, int W, bool ADD>
__global__ void __launch_bounds__(RT) rows_kernel(
    const int2* sorted, SortedHead* head, int shift, const T* __restrict__ dout, long long ldd,
    int V, int d, int cols, int piece_blocks, float scale, O* dtable, long long ldt, float* parts,
    Span* spans) {
  using In = typename Vec<T, W>::Raw;
  constexpr bool kAsync = sizeof(In) >= 4;   // a 2-byte access has no asynchronous copy
  __shared__ In slots[RT / 32][kFlight][32];
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int nv = d / W;
  if ((int)blockIdx.x >= piece_blocks) {   // rows without a token are zero
    const long long r0 = ((long long)(blockIdx.x - piece_blocks) * (RT / 32) + wid) * kOwn;
    const long long r = r0 + lane;
    const int lo = lane > kOwn ? 0 : r < V ? first_at(sorted, head, shift, (int)r) : head->live;
    const int hi = __shfl_down_sync(kFull, lo, 1);
    for (int k = 0; k < kOwn && r0 + k < V; ++k) {
      if (__shfl_sync(kFull, lo, k) != __shfl_sync(kFull, hi, k)) continue;
      O* dst = dtable + (r0 + k) * ldt;
      if (W * sizeof(O) >= 16)
        for (int v = lane; v < nv; v += 32)
          Vec<O, W>::store(dst + (long long)v * W, Vec<O, W>::zero());
      else
        zero_span<O, 32>(dst, d, lane);
    }
    return;
  }
  const int n = head->live;
  const long long unit = (long long)blockIdx.x * (RT / 32) + wid;
  const int k = (int)(unit / cols), v = (int)(unit % cols) * 32 + lane;
  const int p0 = k * kPiece, count = min(kPiece, n - p0);
  if (count <= 0) return;
  // lane l holds position p0 + l and whether its row ends there
  const int2 kv = lane < count ? sorted[p0 + lane] : make_int2(-1, 0);
  const int before = p0 > 0 ? sorted[p0 - 1].x : -1;
  const int after = p0 + count < n ? sorted[p0 + count].x : -1;
  const bool here = v < nv;
  const T* const column = dout + (long long)v * W;
  In(&slot)[kFlight][32] = slots[wid];
  auto fetch = [&](int i0) {             // positions i0 .. i0 + kGroup - 1; one commit
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const int i = i0 + u;
      const int at = __shfl_sync(kFull, kv.y, i & 31);
      if (here && i < count) {
        const T* from = column + (long long)at * ldd;
        if (kAsync) copy_async<sizeof(In)>(&slot[i % kFlight][lane], from);
        else slot[i % kFlight][lane] = Vec<T, W>::load(from);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kFlight; i += kGroup) fetch(i);
  int next = __shfl_down_sync(kFull, kv.x, 1);
  if (lane == count - 1) next = after;
  const unsigned ends = __ballot_sync(kFull, lane < count && next != kv.x);
  bool inherited = __shfl_sync(kFull, kv.x, 0) == before;   // the row began in an earlier piece
  // one warp of a piece's notes the row that goes on from here: short ones from
  // the front of `spans`, long ones from its back
  if (v == 0 && !(ends >> (count - 1) & 1) && !(inherited && ends == 0)) {
    const int end = after + 1 < V ? first_at(sorted, head, shift, after + 1) : n;
    const int pieces = (end - 1) / kPiece - k + 1;
    const int at = pieces > kLong ? (n - 1) / kPiece - atomicAdd(&head->long_spans, 1)
                                  : atomicAdd(&head->spans, 1);
    spans[at] = {k, after, pieces, 0};
  }
  float acc[W];
#pragma unroll
  for (int j = 0; j < W; ++j) acc[j] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += kGroup) {
    typename Vec<O, W>::Raw old[ADD ? kGroup : 1];   // what the rows that end here hold
    if (ADD) {
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const int id = __shfl_sync(kFull, kv.x, i0 + u);
        old[u] = here && (ends >> (i0 + u) & 1)
                     ? Vec<O, W>::load_rw(dtable + id * ldt + (long long)v * W)
                     : Vec<O, W>::zero();
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kFlight / kGroup - 1) : "memory");
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const int i = i0 + u;
      if (i >= count) break;
      float f[W];        // lanes past the row's end sum what is there and store nothing
      Vec<T, W>::unpack(slot[i % kFlight][lane], f);
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] += f[j];
      const bool ended = ends >> i & 1;
      if (!ended && i != count - 1) continue;
      const int id = __shfl_sync(kFull, kv.x, i);
      if (here && (inherited || !ended)) {
        Vec<float, W>::store(parts + (2LL * k + (inherited ? 0 : 1)) * d + (long long)v * W,
                             Vec<float, W>::pack(acc));
      } else if (here) {
        if (ADD) Vec<O, W>::unpack(old[ADD ? u : 0], f);
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = ADD ? acc[j] * scale + f[j] : acc[j] * scale;
        Vec<O, W>::store(dtable + id * ldt + (long long)v * W, Vec<O, W>::pack(acc));
      }
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] = 0.f;
      inherited = false;
    }
    fetch(i0 + kFlight);
  }
}

// acc += parts [a, b) of a row that spans pieces, 32 accesses of it.
template <int W>
__device__ __forceinline__ void add_parts(const Span& sp, int a, int b, int d, int v,
                                          const float* parts, float* acc) {
  for (int i0 = a; i0 < b; i0 += 4) {
    typename Vec<float, W>::Raw q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u;
      const long long slot = i == 0 ? 2LL * sp.first + 1 : 2LL * (sp.first + i);
      q[u] = i < b ? Vec<float, W>::load_rw(parts + slot * d + (long long)v * W)
                   : Vec<float, W>::zero();
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i0 + u >= b) break;
      float f[W];
      Vec<float, W>::unpack(q[u], f);
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] += f[j];
    }
  }
}

// Rows that span pieces: a warp adds the parts of 32 accesses of a row, in order;
// of a long row a block, its warps contiguous ranges of the parts, then the warps'
// sums in order.  Latency: 6 to 12 us at the sizes above.
template <typename O, int W, bool ADD>
__global__ void __launch_bounds__(ET) joined_kernel(const SortedHead* head, int d, int cols,
                                                    float scale, O* dtable, long long ldt,
                                                    const float* parts, const Span* spans) {
  __shared__ float red[ET / 32][32][W + (W > 1)];
  wait_for_previous();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  auto put = [&](int id, int v, const typename Vec<O, W>::Raw& before, float* acc) {
    float old[W];
    if (ADD) Vec<O, W>::unpack(before, old);
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = ADD ? acc[j] * scale + old[j] : acc[j] * scale;
    Vec<O, W>::store(dtable + id * ldt + (long long)v * W, Vec<O, W>::pack(acc));
  };
  auto get = [&](int id, int v) {
    return ADD ? Vec<O, W>::load_rw(dtable + id * ldt + (long long)v * W) : Vec<O, W>::zero();
  };
  const int last = (head->live - 1) / kPiece;
  for (long long task = blockIdx.x; task < (long long)head->long_spans * cols; task += gridDim.x) {
    const Span sp = spans[last - task / cols];
    const int v = (int)(task % cols) * 32 + lane;
    const bool here = v < d / W;
    const int share = (sp.pieces + ET / 32 - 1) / (ET / 32);
    const int a = min(sp.pieces, wid * share), b = min(sp.pieces, a + share);
    float acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.f;
    if (here) add_parts<W>(sp, a, b, d, v, parts, acc);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < W; ++j) red[wid][lane][j] = acc[j];
    __syncthreads();
    if (wid > 0 || !here) continue;
    const auto old = get(sp.id, v);
    for (int w = 1; w < ET / 32; ++w)
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] += red[w][lane][j];
    put(sp.id, v, old, acc);
  }
  const long long warps = (long long)gridDim.x * (ET / 32);
  for (long long task = (long long)blockIdx.x * (ET / 32) + wid;
       task < (long long)head->spans * cols; task += warps) {
    const Span sp = spans[task / cols];
    const int v = (int)(task % cols) * 32 + lane;
    if (v >= d / W) continue;
    const auto old = get(sp.id, v);
    float acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.f;
    add_parts<W>(sp, 0, sp.pieces, d, v, parts, acc);
    put(sp.id, v, old, acc);
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

// The workspace of a gradient: unsorted pairs, then (byte offsets) these.
struct TableWs {
  size_t sorted, head, spans, parts, total;
};
TableWs table_ws(long long n, int d) {
  const size_t pairs = align_up((size_t)n * sizeof(int2), 256), pieces = blocks_for(n, kPiece);
  TableWs w;
  w.sorted = pairs;
  w.head = w.sorted + pairs;
  w.spans = w.head + align_up(sizeof(SortedHead), 256);
  w.parts = w.spans + align_up(pieces * sizeof(Span), 256);
  w.total = w.parts + align_up(pieces * 2 * d * sizeof(float), 256);
  return w;
}

template <typename T, typename O, int W, bool ADD>
cudaError_t table_t(const EmbedArgs& a, void* ws, int* err, cudaStream_t s) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  const TableWs at = table_ws(a.n, a.d);
  int2* scratch = reinterpret_cast<int2*>(p);
  int2* sorted = reinterpret_cast<int2*>(p + at.sorted);
  SortedHead* head = reinterpret_cast<SortedHead*>(p + at.head);
  Span* spans = reinterpret_cast<Span*>(p + at.spans);
  float* parts = reinterpret_cast<float*>(p + at.parts);
  int shift = 0;
  cudaError_t e =
      launch_sort_ids(a.ids, a.ids_bytes, (int)a.n, a.V, scratch, sorted, head, &shift, err, s);
  if (e != cudaSuccess) return e;
  const int pieces = blocks_for(a.n, kPiece), cols = blocks_for(a.d / W, 32);
  const int piece_blocks = blocks_for((long long)pieces * cols, RT / 32);
  const int blocks = piece_blocks + (ADD ? 0 : blocks_for(a.V, RT / 32 * kOwn));
  if (blocks > 0)
    e = launch_after(rows_kernel<T, O, W, ADD>, blocks, RT, s, sorted, head, shift,
                     (const T*)a.in.p, a.in.ld, a.V, a.d, cols, piece_blocks, a.scale,
                     (O*)a.out.p, a.out.ld, parts, spans);
  if (e == cudaSuccess && pieces > 1) {
    const long long most = (long long)(pieces - 1) * cols;
    e = launch_after(joined_kernel<O, W, ADD>, (int)(most < 152 * 4 ? most : 152 * 4), ET, s,
                     head, a.d, cols, a.scale, (O*)a.out.p, a.out.ld, parts, spans);
  }
  count_launches((blocks > 0) + (pieces > 1));
  return e;
}

template <typename T, typename O, int W>
cudaError_t by_length(const EmbedArgs& a, bool grad, void* ws, int* err, cudaStream_t s) {
  if (grad)
    return a.accumulate ? table_t<T, O, W, true>(a, ws, err, s)
                        : table_t<T, O, W, false>(a, ws, err, s);
  // A block copies four rows of more than 64 accesses, a warp four shorter ones.  32768 ids,
  // bf16: d 256 4.3 us (a block 10.1), 512 9.8 (12.8), 768 14.6 (a warp 13.4), 1024 17.0
  // (17.4), 4096 58 (63); 1000 ids, where a warp a row leaves SMs idle: d 1024 2.0 (3.4).
  return a.d / W > 64 ? embed_t<T, O, W, ET>(a, s) : embed_t<T, O, W, 32>(a, s);
}

// Elements per access: the most of 8, 4, 2 and 1 that both sides' rows are aligned
// to, up to 16 bytes of the input.
int width(const EmbedArgs& a) {
  const int si = dtype_bytes(a.in_dtype), so = dtype_bytes(a.out_dtype);
  for (int w = 16 / si; w > 1; w /= 2)
    if (a.d % w == 0 && (uintptr_t)a.in.p % (w * si) == 0 && a.in.ld % w == 0 &&
        (uintptr_t)a.out.p % (w * so) == 0 && a.out.ld % w == 0)
      return w;
  return 1;
}

template <typename T, typename O>
cudaError_t by_width(const EmbedArgs& a, bool grad, void* ws, int* err, cudaStream_t s) {
  switch (width(a)) {
    case 8:
      if constexpr (sizeof(T) == 2) return by_length<T, O, 8>(a, grad, ws, err, s);
      [[fallthrough]];
    case 4: return by_length<T, O, 4>(a, grad, ws, err, s);
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

size_t embed_bwd_ws_bytes(long long n, int d) { return table_ws(n, d).total; }

cudaError_t launch_embed_bwd(const EmbedArgs& a, void* ws, int* err, cudaStream_t s) {
  return by_type(a, true, ws, err, s);
}

}  // namespace moe
