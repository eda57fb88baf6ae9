// Which positions a sequence's moved entries go to, and where in its row of nodes each of them looks (include/pace_draft.h:
// pace_cache_move with nodes).  Used by the kernel; host code, too, so that its ends can be checked on the CPU.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pace {

struct MoveRange {
  int64_t start, first, end;    // entries go to positions first .. end - 1, the i-th to start + i
  int64_t base;                 // where the steps begin: the first position's tile of 16
  int32_t count;
};

// False where nothing is moved; then there need not be a node to read.  limit: positions of the page table.
__host__ __device__ inline bool move_range(int32_t start, int32_t count, int32_t T, int64_t limit, MoveRange& r) {
  r.start = start;
  r.count = count < 0 ? 0 : count < T ? count : T;
  r.first = start > 0 ? start : 0;
  r.end = r.start + r.count < limit ? r.start + r.count : limit;
  r.base = r.first & ~(int64_t)15;
  return r.first < r.end;
}

// The place in the row of nodes for position pos: in [0, count) whatever pos is.
__host__ __device__ inline int64_t node_place(const MoveRange& r, int64_t pos) {
  const int64_t i = pos - r.start, last = (int64_t)r.count - 1;
  return i < 0 ? 0 : i < last ? i : last;
}

}  // namespace pace
