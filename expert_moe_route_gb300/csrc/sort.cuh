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
// sorted[0 .. *live): (id, position) of the ids inside [0, V), by id, equal ids by
// position.  scratch and sorted hold n pairs each.  Ids >= V set the error word.
cudaError_t launch_sort_ids(const void* ids, int ids_bytes, int n, int V, int2* scratch,
                            int2* sorted, int32_t* live, int* err, cudaStream_t s);

}  // namespace moe
