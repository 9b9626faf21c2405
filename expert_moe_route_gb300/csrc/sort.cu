// Stable counting sort on one thread-block cluster, for the slots of an expert
// sort (moe_sort) and for the token ids of an embedding gradient.
//
// Keys are cut into contiguous shares, one per CTA of the cluster, and each
// share into contiguous ranges, one per warp.  Every warp counts its range's
// keys into its own row of a shared-memory table [16 warps][bins]; a prefix
// over the warps, then over the CTAs (each CTA reads the others' totals through
// distributed shared memory) and over the bins gives every warp its first
// position in every bin.  The warps then walk their ranges once more: ballots
// rank equal keys inside a group of 32, so positions follow the keys' order and
// no atomic decides one.
//
// One launch does the whole plan: separate histogram, scan and rank launches
// would add their latencies.  Bound by latency, 1024 slots over 256 experts take
// 4.2 us, 131072 over 128 12.5 us, 524288 over 256 37 us (3% of moving their rows
// of 7168 bf16).
#include "common.cuh"
#include "kernels.h"
#include "sort.cuh"

namespace moe {

namespace {
constexpr int ST = 512;           // threads per CTA
constexpr int SW = ST / 32;       // warps per CTA
constexpr int kMaxCluster = 16;   // a cluster of more than 8 CTAs is an opt-in
constexpr int kBatch = 8;         // groups of 32 keys whose loads are in flight together

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
__device__ __forceinline__ int2 ld_cluster2(const int* local, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
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
  int mine = lane < SW ? warp_sums[lane] : 0;
#pragma unroll
  for (int off = 1; off < SW; off <<= 1) {
    const int o = __shfl_up_sync(kFull, mine, off);
    if (lane >= off) mine += o;
  }
  *total = __shfl_sync(kFull, mine, SW - 1);
  const int before = __shfl_sync(kFull, mine, wid > 0 ? wid - 1 : 0);
  return (wid > 0 ? before : 0) + incl - v;
}

// Shared-memory table of one pass over `bins` bins (even, at most 2 ST: thread t
// owns bins 2 t and 2 t + 1).
struct Table {
  int* wcnt;    // [SW][bins] counts, then each warp's offset inside the CTA's part of a bin
  int* mine;    // [bins] this CTA's counts (read by the other CTAs)
  int* below;   // [bins] keys of the bin in earlier CTAs
};

// Counts are in t.wcnt: fills mine and below and returns the totals over the
// cluster of this thread's two bins (0 past `bins`).  The other CTAs' shared
// memory has been read: a cluster barrier must follow before this CTA leaves or
// changes `mine`.
__device__ __forceinline__ int2 cluster_totals(const Table& t, int bins, uint32_t rank,
                                               uint32_t nr) {
  const int b = threadIdx.x * 2;
  int2 run = make_int2(0, 0);
  __syncthreads();
  if (b < bins) {
    int2 c[SW];
#pragma unroll
    for (int w = 0; w < SW; ++w) c[w] = *reinterpret_cast<const int2*>(t.wcnt + w * bins + b);
#pragma unroll
    for (int w = 0; w < SW; ++w) {
      *reinterpret_cast<int2*>(t.wcnt + w * bins + b) = run;
      run.x += c[w].x;
      run.y += c[w].y;
    }
    *reinterpret_cast<int2*>(t.mine + b) = run;
  }
  if (nr == 1) {
    if (b < bins) *reinterpret_cast<int2*>(t.below + b) = make_int2(0, 0);
    return run;
  }
  cluster_arrive();
  cluster_wait();
  int2 total = make_int2(0, 0), before = make_int2(0, 0);
  if (b < bins) {
    int2 c[kMaxCluster];          // all reads in flight together
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r)
      c[r] = r < nr ? ld_cluster2(t.mine + b, r) : make_int2(0, 0);
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r) {
      if (r < rank) {
        before.x += c[r].x;
        before.y += c[r].y;
      }
      total.x += c[r].x;
      total.y += c[r].y;
    }
    *reinterpret_cast<int2*>(t.below + b) = before;
  }
  return total;
}

// Position of `key` (this lane's, -1 for none, else below 2^bits) among the keys of
// its bin in the warp's range so far; counts them in `my`.  A ballot per bit finds
// the equal keys; __match_any_sync took 44 us, this 37, for 524288 keys.
__device__ __forceinline__ int warp_rank(int key, int* my, int bits) {
  const int lane = threadIdx.x & 31;
  unsigned peers = __ballot_sync(kFull, key >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool one = key >> b & 1;
    const unsigned ones = __ballot_sync(kFull, one);
    peers &= one ? ones : ~ones;
  }
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
  const int bins = (E + 1) & ~1, bits = 32 - __clz(E - 1);
  Table t{sm, sm + SW * bins, sm + SW * bins + bins};
  int* room_s = sm + SW * bins + 2 * bins;   // [bins] rows left for this CTA's part of the bin (<= 0: none)
  int* off_s = room_s + bins;                // [bins] first row of this CTA's part of the bin
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) bad_s = 0;
  for (int i = tid; i < SW * bins / 2; i += ST) reinterpret_cast<int2*>(t.wcnt)[i] = make_int2(0, 0);
  // rows without a slot keep this; the others are written after the cluster's barrier
  for (long long r = (long long)rank * ST + tid; r < N; r += (long long)nr * ST) row_slot[r] = -1;
  const int per_warp = share / SW;
  const long long w0 = (long long)rank * share + (long long)wid * per_warp;
  const long long w1 = min((long long)n, w0 + per_warp);
  int* my = t.wcnt + wid * bins;
  auto load = [&](long long g, int* e) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const long long i = g + 32 * j + lane;
      e[j] = i < w1 ? __ldg(idx + i) : -1;
    }
  };
  bool bad = false;
  int early[kBatch];            // the first batch stays in registers for the second walk
  load(w0, early);
  __syncthreads();
  for (long long g = w0; g < w1; g += 32 * kBatch) {
    int e[kBatch];
    if (g == w0) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) e[j] = early[j];
    } else {
      load(g, e);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (g + 32 * j >= w1) break;
      if ((unsigned)e[j] < (unsigned)E) atomicAdd(&my[e[j]], 1);
      else bad |= e[j] != -1;
    }
  }
  if (bad) atomicOr(&bad_s, 1);
  const int2 total = cluster_totals(t, bins, rank, nr);
  if (rank == 0 && tid == 0) {
    int any = 0;
    for (uint32_t r = 0; r < nr; ++r) any |= ld_cluster(&bad_s, r);
    *err = any ? kErrBadRouting : 0;
  }
  if (nr > 1) cluster_arrive();
  const int b = tid * 2;
  int2 kept, padded;
  kept.x = capacity > 0 ? min(total.x, capacity) : total.x;
  kept.y = capacity > 0 ? min(total.y, capacity) : total.y;
  // kept + align may reach 2^31, what is left of it after rounding does not
  padded.x = (int)(((unsigned)kept.x + align - 1) / align * align);
  padded.y = (int)(((unsigned)kept.y + align - 1) / align * align);
  int end;
  const int off = block_scan(padded.x + padded.y, warp_sums, &end);
  if (b < bins) {
    const int2 before = *reinterpret_cast<const int2*>(t.below + b);
    // ranks go up to 2^31 also where a limit keeps the rows few: a slot's rank is
    // compared with the room before the bin's first row is added to it
    *reinterpret_cast<int2*>(room_s + b) = make_int2(kept.x - before.x, kept.y - before.y);
    *reinterpret_cast<int2*>(off_s + b) =
        make_int2(off + min(before.x, kept.x), off + padded.x + min(before.y, kept.y));
    if (rank == 0) {
      counts[b] = kept.x;
      offsets[b] = off;
      if (b + 1 < E) {
        counts[b + 1] = kept.y;
        offsets[b + 1] = off + padded.x;
      }
    }
  }
  if (rank == 0 && tid == 0) offsets[E] = end;
  __syncthreads();
  for (long long g = w0; g < w1; g += 32 * kBatch) {
    int e[kBatch];
    if (g == w0) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) e[j] = early[j];
    } else {
      load(g, e);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const long long i = g + 32 * j + lane;
      if (g + 32 * j >= w1) break;       // the same for the whole warp
      if ((unsigned)e[j] >= (unsigned)E) e[j] = -1;
      const int pos = warp_rank(e[j], my, bits);
      int row = -1;
      if (e[j] >= 0 && pos < room_s[e[j]]) row = off_s[e[j]] + pos;
      if (i < w1) slot_row[i] = row;
      if (row >= 0) row_slot[row] = (int)i;
    }
  }
  if (nr > 1) cluster_wait();   // no CTA leaves while another still reads its totals
}

// ---------------------------------------------------------------- id sort
template <typename I>
__global__ void __launch_bounds__(ST) sort_ids_kernel(
    const I* __restrict__ ids, int n, int V, int bits, int passes, int2* a, int2* b,
    SortedHead* __restrict__ head, int* __restrict__ err) {
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
    for (int i = tid; i < SW * bins / 2; i += ST)
      reinterpret_cast<int2*>(t.wcnt)[i] = make_int2(0, 0);
    const int per_warp = ((count + (int)nr * SW - 1) / ((int)nr * SW) + 31) / 32 * 32;
    const long long w0 = ((long long)rank * SW + wid) * per_warp;
    const long long w1 = min((long long)count, w0 + per_warp);
    int* my = t.wcnt + wid * bins;
    auto load = [&](long long g, int2* kv) {   // (id, position); id -1: none
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const long long i = g + 32 * j + lane;
        kv[j] = make_int2(-1, (int)i);
        if (i >= w1) continue;
        if (p == 0) {
          const I id = ids[i];
          if (id >= (I)V) bad = true;
          else if (id >= 0) kv[j].x = (int)id;
        } else {
          kv[j] = __ldcg(&src[i]);
        }
      }
    };
    int2 early[kBatch];           // the first batch stays in registers for the second walk
    load(w0, early);
    __syncthreads();
    for (long long g = w0; g < w1; g += 32 * kBatch) {
      int2 kv[kBatch];
      if (g == w0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) kv[j] = early[j];
      } else {
        load(g, kv);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (kv[j].x >= 0) atomicAdd(&my[(kv[j].x >> shift) & (bins - 1)], 1);
    }
    if (p == 0 && bad) atomicOr(&bad_s, 1);
    const int2 total = cluster_totals(t, bins, rank, nr);
    int live;
    const int off = block_scan(total.x + total.y, warp_sums, &live);
    if (tid * 2 < bins) {
      off_s[tid * 2] = off + t.below[tid * 2];
      off_s[tid * 2 + 1] = off + total.x + t.below[tid * 2 + 1];
      if (rank == 0 && p == passes - 1) {
        head->top[tid * 2] = off;
        head->top[tid * 2 + 1] = off + total.x;
      }
    }
    if (p == 0 && rank == 0 && tid == 0) {
      int any = 0;
      for (uint32_t r = 0; r < nr; ++r) any |= ld_cluster(&bad_s, r);
      *err = any ? kErrBadRouting : 0;
      head->live = live;
      head->spans = head->long_spans = 0;
      head->top[bins] = live;
    }
    __syncthreads();
    for (long long g = w0; g < w1; g += 32 * kBatch) {
      int2 kv[kBatch];
      if (g == w0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) kv[j] = early[j];
      } else {
        load(g, kv);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (g + 32 * j >= w1) break;     // the same for the whole warp
        const int bin = kv[j].x >= 0 ? (kv[j].x >> shift) & (bins - 1) : -1;
        const int pos = warp_rank(bin, my, bits);
        if (bin >= 0) __stcg(&dst[off_s[bin] + pos], kv[j]);
      }
    }
    count = live;
    if (nr > 1) {
      cluster_arrive();   // the totals are read, this pass's pairs written
      cluster_wait();
    } else {
      __syncthreads();
    }
  }
}

int g_max_cluster[64];   // per device: CTAs a cluster of these kernels may have

int max_cluster() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 8;
  return g_max_cluster[dev] > 0 ? g_max_cluster[dev] : 8;
}

// Two keys a thread before the cluster grows.  4096 slots over 256 experts: 5.4 us (one
// key 5.0, four 6.3); 1024 slots: 3.9 (one 4.5: two CTAs and their barriers); 16384 over
// 64: 5.2 (5.2, 6.1); a gradient by 4096 ids of 32003: 21.5 (20.8, 23.5).
int cluster_for(long long n) {
  const int most = max_cluster();
  int c = 1;
  while (c < most && n > (long long)c * 2 * ST) c *= 2;
  return c;
}

cudaLaunchConfig_t cluster_config(int ctas, size_t smem, cudaLaunchAttribute* at, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(ST);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

cudaError_t launch_cluster(const void* f, int ctas, size_t smem, void** args, cudaStream_t s) {
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = cluster_config(ctas, smem, at, s);
  const cudaError_t e = cudaLaunchKernelExC(&cfg, f, args);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t table_bytes(int bins, int extra) { return sizeof(int) * (size_t)bins * (SW + 2 + extra); }
}  // namespace

cudaError_t sort_set_limits() {
  const int most = (int)table_bytes(1024, 2);
  bool wide = true;
  for (const void* f : {(const void*)sort_slots_kernel, (const void*)sort_ids_kernel<int32_t>,
                        (const void*)sort_ids_kernel<int64_t>}) {
    cudaError_t e =
        cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    const cudaLaunchConfig_t cfg = cluster_config(kMaxCluster, most, at, nullptr);
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, f, &cfg) != cudaSuccess || fit < 1) {
      (void)cudaGetLastError();
      wide = false;
    }
  }
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev >= 0 && dev < 64) g_max_cluster[dev] = wide ? kMaxCluster : 8;
  return e;
}

cudaError_t launch_sort_slots(const int32_t* idx, int n, int E, int align, int capacity, int N,
                              int32_t* counts, int32_t* offsets, int32_t* row_slot,
                              int32_t* slot_row, int* err, cudaStream_t s) {
  const int ctas = cluster_for(n);
  int share = (int)((((long long)n + ctas - 1) / ctas + ST - 1) / ST * ST);
  void* args[] = {&idx, &n, &share, &E, &align, &capacity, &N, &counts, &offsets, &row_slot,
                  &slot_row, &err};
  return launch_cluster((const void*)sort_slots_kernel, ctas, table_bytes((E + 1) & ~1, 2), args,
                        s);
}

cudaError_t launch_sort_ids(const void* ids, int ids_bytes, int n, int V, int2* scratch,
                            int2* sorted, SortedHead* head, int* shift, int* err, cudaStream_t s) {
  int key_bits = 1;
  while (key_bits < 31 && (1LL << key_bits) < V) ++key_bits;
  int passes = (key_bits + 9) / 10;
  int bits = (key_bits + passes - 1) / passes;
  *shift = (passes - 1) * bits;
  const int ctas = cluster_for(n);
  void* args[] = {&ids, &n, &V, &bits, &passes, &scratch, &sorted, &head, &err};
  return launch_cluster(ids_bytes == 8 ? (const void*)sort_ids_kernel<int64_t>
                                       : (const void*)sort_ids_kernel<int32_t>,
                        ctas, table_bytes(1 << bits, 1), args, s);
}

}  // namespace moe
