// A ring of rows in shared memory that one thread fills by bulk copies and a whole block
// empties in step.
#pragma once

#include "internal.h"
#include "tc_ptx.cuh"

namespace nabla {

constexpr int kMaxStages = 4;

struct RowRing {
  uint64_t full[kMaxStages];  // a stage's row has arrived
  int abort;
  int stages;
};

// The wait for a row that is not there yet.  A thread whose wait gives up leaves (barriers and
// shuffles go on without it, and the status says that the results are void); thread 0, which
// alone asks for rows, first lets its copies in flight land, those of the stages from here on.
// (A loop that went on with a flag beside it took 1.4 times as long at 8192 columns: spills.)
template <uint64_t kLimit = tc::kWaitNs>
__device__ __noinline__ void wait_for_row(uint64_t *bar, uint32_t phase, RowRing *r, int *status) {
  if (tc::mbar_wait(bar, phase, &r->abort, status, kDevTimeout, kLimit)) return;
  if (threadIdx.x == 0)
    for (int i = 0; i < r->stages; ++i) {  // (one not asked for again is waited for in vain)
      tc::mbar_wait(bar, phase, nullptr, status, kDevTimeout, kLimit);
      if (++bar == r->full + r->stages) bar = r->full, phase ^= 1u;
    }
  asm volatile("exit;");
}

}  // namespace nabla
