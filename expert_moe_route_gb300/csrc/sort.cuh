// Launchers of the cluster counting sort (sort.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Per-device set-up (shared memory, cluster size) before the first launch.
cudaError_t sort_set_limits();
// The plan of moe_sort; writes every entry of counts, offsets, row_slot [N],
// slot_row [n] and the error word.
cudaError_t launch_sort_slots(const int32_t* idx, int n, int E, int align, int capacity, int N,
                              int32_t* counts, int32_t* offsets, int32_t* row_slot,
                              int32_t* slot_row, int* err, cudaStream_t s);
// What a sort of ids leaves beside the sorted pairs.
struct SortedHead {
  int32_t live;        // pairs
  int32_t spans, long_spans;   // 0: counters for the kernels that follow
  int32_t top[1025];   // first pair whose id >> shift is at least the index
};
// sorted[0 .. head->live): (id, position) of the ids inside [0, V), by id, equal ids
// by position.  scratch and sorted hold n pairs each.  Ids >= V set the error word.
// *shift (host): that of head->top.
cudaError_t launch_sort_ids(const void* ids, int ids_bytes, int n, int V, int2* scratch,
                            int2* sorted, SortedHead* head, int* shift, int* err, cudaStream_t s);

}  // namespace moe
