// Stable counting sort on one thread-block cluster, for the slots of an expert
// sort (moe_sort) and for the token ids of an embedding gradient.
//
// Keys are cut into contiguous shares, one per CTA of the cluster, and each
// share into contiguous ranges, one per warp.  Every warp counts its range's
// keys into its own row of a shared-memory table [32 warps][bins]; a prefix
// over the warps, then over the CTAs (each CTA reads the others' totals through
// distributed shared memory) and over the bins gives every warp its first
// position in every bin.  The warps then walk their ranges once more:
// __match_any_sync ranks equal keys inside a group of 32, so positions follow
// the keys' order and no atomic decides one.
//
// One launch does the whole plan.  Separate histogram, scan and rank launches
// cost about 2 us each in launch latency; the cluster barrier costs well under
// one.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "sort.cuh"

namespace moe {

namespace {
constexpr int ST = 1024;          // threads per CTA
constexpr int SW = ST / 32;       // warps per CTA
constexpr int kMaxCluster = 8;

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster(const int* local, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];"
               : "=r"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Exclusive scan over the block's threads of one value each; total in *total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) warp_sums[wid] = incl;
  __syncthreads();
  if (wid == 0) {
    int ws = lane < SW ? warp_sums[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kFull, ws, off);
      if (lane >= off) ws += o;
    }
    warp_sums[lane] = ws;
  }
  __syncthreads();
  const int before = (wid > 0 ? warp_sums[wid - 1] : 0) + incl - v;
  *total = warp_sums[SW - 1];
  __syncthreads();
  return before;
}

// Shared-memory table of one pass over `bins` bins (at most ST).
struct Table {
  int* wcnt;    // [SW][bins] counts, then each warp's offset inside the CTA's part of a bin
  int* mine;    // [bins] this CTA's counts (read by the other CTAs)
  int* below;   // [bins] keys of the bin in earlier CTAs
};

// Counts are in t.wcnt: fills mine and below and returns this thread's bin total
// over the cluster (threads past `bins` get 0).  The other CTAs' shared memory
// has been read: a cluster barrier must follow before this CTA leaves or
// changes `mine`.
__device__ int cluster_totals(const Table& t, int bins, uint32_t rank, uint32_t nr) {
  const int b = threadIdx.x;
  __syncthreads();
  if (b < bins) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < SW; ++w) {
      const int c = t.wcnt[w * bins + b];
      t.wcnt[w * bins + b] = run;
      run += c;
    }
    t.mine[b] = run;
  }
  cluster_arrive();
  cluster_wait();
  int total = 0, before = 0;
  if (b < bins) {
    for (uint32_t r = 0; r < nr; ++r) {
      const int c = ld_cluster(t.mine + b, r);
      if (r < rank) before += c;
      total += c;
    }
    t.below[b] = before;
  }
  return total;
}

// Position of `key` (this lane's, -1 for none) among the keys of its bin in the
// warp's range so far; counts them in `my`.
__device__ __forceinline__ int warp_rank(int key, int* my) {
  const int lane = threadIdx.x & 31;
  const unsigned peers = __match_any_sync(kFull, key);
  int pos = 0;
  if (key >= 0) pos = my[key] + __popc(peers & ((1u << lane) - 1u));
  __syncwarp();
  if (key >= 0 && lane == __ffs(peers) - 1) my[key] += __popc(peers);
  __syncwarp();
  return pos;
}

// ---------------------------------------------------------------- expert sort
__global__ void __launch_bounds__(ST) sort_slots_kernel(
    const int32_t* __restrict__ idx, int n, int share, int E, int align, int capacity, int N,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ row_slot,
    int32_t* __restrict__ slot_row, int* __restrict__ err) {
  extern __shared__ int sm[];
  __shared__ int warp_sums[32];
  __shared__ int bad_s;
  const uint32_t rank = cluster_rank(), nr = cluster_size();
  Table t{sm, sm + SW * E, sm + SW * E + E};
  int* kept_s = sm + SW * E + 2 * E;   // [E]
  int* off_s = kept_s + E;             // [E]
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) bad_s = 0;
  for (int i = tid; i < SW * E; i += ST) t.wcnt[i] = 0;
  __syncthreads();
  const long long c0 = (long long)rank * share;
  const int per_warp = share / SW;
  const long long w0 = c0 + (long long)wid * per_warp;
  const long long w1 = min((long long)n, w0 + per_warp);
  int* my = t.wcnt + wid * E;
  bool bad = false;
  for (long long g = w0; g < w1; g += 32) {
    const long long i = g + lane;
    if (i < w1) {
      const int e = idx[i];
      if ((unsigned)e < (unsigned)E) atomicAdd(&my[e], 1);
      else bad |= e != -1;
    }
  }
  if (bad) atomicOr(&bad_s, 1);
  const int total = cluster_totals(t, E, rank, nr);
  if (rank == 0 && tid == 0) {
    int any = 0;
    for (uint32_t r = 0; r < nr; ++r) any |= ld_cluster(&bad_s, r);
    *err = any ? kErrBadRouting : 0;
  }
  cluster_arrive();
  const int kept = capacity > 0 ? min(total, capacity) : total;
  const int padded = (kept + align - 1) / align * align;
  int end;
  const int off = block_scan(tid < E ? padded : 0, warp_sums, &end);
  if (tid < E) {
    kept_s[tid] = kept;
    off_s[tid] = off;
    if (rank == 0) {
      counts[tid] = kept;
      offsets[tid] = off;
    }
  }
  if (rank == 0 && tid == 0) offsets[E] = end;
  __syncthreads();
  for (long long g = w0; g < w1; g += 32) {
    const long long i = g + lane;
    int e = i < w1 ? idx[i] : -1;
    if ((unsigned)e >= (unsigned)E) e = -1;
    const int pos = warp_rank(e, my);
    if (i >= w1) continue;
    int row = -1;
    if (e >= 0) {
      const int p = t.below[e] + pos;
      if (p < kept_s[e]) row = off_s[e] + p;
    }
    slot_row[i] = row;
    if (row >= 0) row_slot[row] = (int)i;
  }
  // rows without a slot: the ends of the segments, and what follows the last one
  for (int e = (int)rank * SW + wid; e < E; e += (int)nr * SW) {
    const int last = e + 1 < E ? off_s[e + 1] : end;
    for (int r = off_s[e] + kept_s[e] + lane; r < last; r += 32) row_slot[r] = -1;
  }
  for (int r = end + (int)rank * ST + tid; r < N; r += (int)nr * ST) row_slot[r] = -1;
  cluster_wait();   // no CTA leaves while another still reads its totals
}

// ---------------------------------------------------------------- id sort
template <typename I>
__global__ void __launch_bounds__(ST) sort_ids_kernel(
    const I* __restrict__ ids, int n, int V, int bits, int passes, int2* a, int2* b,
    int32_t* __restrict__ live_out, int* __restrict__ err) {
  extern __shared__ int sm[];
  __shared__ int warp_sums[32];
  __shared__ int bad_s;
  const uint32_t rank = cluster_rank(), nr = cluster_size();
  const int bins = 1 << bits;
  Table t{sm, sm + SW * bins, sm + SW * bins + bins};
  int* off_s = sm + SW * bins + 2 * bins;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) bad_s = 0;
  int count = n;                 // keys of this pass
  bool bad = false;
  for (int p = 0; p < passes; ++p) {
    // sources and destinations alternate so that the last pass writes b
    int2* dst = (passes - 1 - p) & 1 ? a : b;
    const int2* src = dst == a ? b : a;
    const int shift = p * bits;
    for (int i = tid; i < SW * bins; i += ST) t.wcnt[i] = 0;
    __syncthreads();
    const int per_warp = ((count + (int)nr * SW - 1) / ((int)nr * SW) + 31) / 32 * 32;
    const long long w0 = ((long long)rank * SW + wid) * per_warp;
    const long long w1 = min((long long)count, w0 + per_warp);
    int* my = t.wcnt + wid * bins;
    for (long long i = w0 + lane; i < w1; i += 32) {
      int key;
      if (p == 0) {
        const I id = ids[i];
        if (id >= (I)V) bad = true;
        key = id >= 0 && id < (I)V ? (int)id : -1;
      } else {
        key = __ldcg(&src[i]).x;
      }
      if (key >= 0) atomicAdd(&my[(key >> shift) & (bins - 1)], 1);
    }
    if (p == 0 && bad) atomicOr(&bad_s, 1);
    const int total = cluster_totals(t, bins, rank, nr);
    int live;
    const int off = block_scan(tid < bins ? total : 0, warp_sums, &live);
    if (tid < bins) off_s[tid] = off + t.below[tid];
    if (p == 0 && rank == 0 && tid == 0) {
      int any = 0;
      for (uint32_t r = 0; r < nr; ++r) any |= ld_cluster(&bad_s, r);
      *err = any ? kErrBadRouting : 0;
      *live_out = live;
    }
    __syncthreads();
    for (long long g = w0; g < w1; g += 32) {
      const long long i = g + lane;
      int2 kv = make_int2(-1, (int)i);
      if (i < w1) {
        if (p == 0) {
          const I id = ids[i];
          if (id >= 0 && id < (I)V) kv.x = (int)id;
        } else {
          kv = __ldcg(&src[i]);
        }
      }
      const int bin = kv.x >= 0 ? (kv.x >> shift) & (bins - 1) : -1;
      const int pos = warp_rank(bin, my);
      if (bin >= 0) __stcg(&dst[off_s[bin] + pos], kv);
    }
    count = live;
    cluster_arrive();   // the totals are read, this pass's pairs written
    cluster_wait();
  }
}

int cluster_for(long long n) {
  int c = 1;
  while (c < kMaxCluster && n > (long long)c * 4 * ST) c *= 2;
  return c;
}

cudaError_t launch_cluster(const void* f, int ctas, size_t smem, void** args, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(ST);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, f, args);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t table_bytes(int bins, int extra) { return sizeof(int) * (size_t)bins * (SW + 2 + extra); }
}  // namespace

cudaError_t sort_set_smem_limits() {
  const int most = (int)table_bytes(1024, 2);
  cudaError_t e = cudaFuncSetAttribute((const void*)sort_slots_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute((const void*)sort_ids_kernel<int32_t>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute((const void*)sort_ids_kernel<int64_t>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  return e;
}

cudaError_t launch_sort_slots(const int32_t* idx, int n, int E, int align, int capacity, int N,
                              int32_t* counts, int32_t* offsets, int32_t* row_slot,
                              int32_t* slot_row, int* err, cudaStream_t s) {
  const int ctas = cluster_for(n);
  int share = (int)((((long long)n + ctas - 1) / ctas + ST - 1) / ST * ST);
  void* args[] = {&idx, &n, &share, &E, &align, &capacity, &N, &counts, &offsets, &row_slot,
                  &slot_row, &err};
  return launch_cluster((const void*)sort_slots_kernel, ctas, table_bytes(E, 2), args, s);
}

cudaError_t launch_sort_ids(const void* ids, int ids_bytes, int n, int V, int2* scratch,
                            int2* sorted, int32_t* live, int* err, cudaStream_t s) {
  int key_bits = 1;
  while (key_bits < 31 && (1LL << key_bits) < V) ++key_bits;
  int passes = (key_bits + 9) / 10;
  int bits = (key_bits + passes - 1) / passes;
  const int ctas = cluster_for(n);
  void* args[] = {&ids, &n, &V, &bits, &passes, &scratch, &sorted, &live, &err};
  return launch_cluster(ids_bytes == 8 ? (const void*)sort_ids_kernel<int64_t>
                                       : (const void*)sort_ids_kernel<int32_t>,
                        ctas, table_bytes(1 << bits, 1), args, s);
}

}  // namespace moe
