// What the cross-attention kernels share: how query rows are packed into tiles and
// how a batch's states are cut into tiles.
//
// The heads of a group (G = h / hk) read the same keys, so their rows go into one
// tile: a 64-row subtile holds tq = 64 / G tokens of all G heads of the group, row
// r = (token) * G + (head in the group); rows from tq * G on (G not dividing 64) stay
// zero.  One K/V tile then serves all the heads that share it, and a single token of a
// grouped model fills G rows instead of one.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "internal.h"
#include "tc_ptx.cuh"

namespace nabla {
namespace cross {

constexpr int kTile = 128;  // states per tile

struct Packing {
  int G, tq, nsub;  // heads per group, tokens per 64-row subtile, subtiles per (b, key head)
};
inline Packing packing(const CrossShape &s) {
  Packing p;
  p.G = s.h / s.hk;
  p.tq = 64 / p.G;
  p.nsub = (s.Sq + p.tq - 1) / p.tq;
  return p;
}

// One thread's wait, and a whole warp's.  A lane whose wait gave up waits no more but goes
// on through its loops, over whatever the buffers hold: later waits return at once, the
// role meets its barriers, and the status word says that the results are void.  So the
// lanes need no vote on each wait, which cost the softmax warps 100 cycles and more.
__device__ __forceinline__ bool thread_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                            int *status) {
  return tc::mbar_wait_small(bar, parity, abort, status, kDevTimeout);
}
__device__ __forceinline__ void warp_wait(bool &live, uint64_t *bar, uint32_t parity,
                                          volatile int *abort, int *status) {
  if (live) live = tc::mbar_wait_small(bar, parity, abort, status, kDevTimeout);
  __syncwarp();
}

// The work units of a kernel, numbered with the run of the split axis first, then the
// tile, the key head and the batch; a CTA takes every gridDim.x-th.  The divisions are
// done once, for the CTA's first unit (and on the host, for the step): a unit of a few
// tiles is short enough for them to show.
struct Walk {
  int sp, t, j, b;
};
struct WalkStep {
  int nsplit, nt, hk;  // radices
  int sp, t, j, b;     // digits of gridDim.x
};
inline WalkStep walk_step(unsigned grid, int nsplit, int nt, int hk) {
  WalkStep s{nsplit, nt, hk, 0, 0, 0, 0};
  s.sp = (int)(grid % nsplit);
  grid /= nsplit;
  s.t = (int)(grid % nt);
  grid /= nt;
  s.j = (int)(grid % hk);
  s.b = (int)(grid / hk);
  return s;
}
__device__ __forceinline__ Walk walk_start(const WalkStep &s, uint32_t u) {
  Walk w;
  w.sp = (int)(u % (uint32_t)s.nsplit);
  u /= (uint32_t)s.nsplit;
  w.t = (int)(u % (uint32_t)s.nt);
  u /= (uint32_t)s.nt;
  w.j = (int)(u % (uint32_t)s.hk);
  w.b = (int)(u / (uint32_t)s.hk);
  return w;
}
__device__ __forceinline__ void walk_next(const WalkStep &s, Walk &w) {
  w.sp += s.sp;
  w.t += s.t;
  w.j += s.j;
  w.b += s.b;
  if (w.sp >= s.nsplit) w.sp -= s.nsplit, ++w.t;
  if (w.t >= s.nt) w.t -= s.nt, ++w.j;
  if (w.j >= s.hk) w.j -= s.hk, ++w.b;
}

__device__ __forceinline__ int batch_len(const int32_t *kv_len, int b, int Sk) {
  if (!kv_len) return Sk;
  const int n = __ldg(kv_len + b);
  return n < 0 ? 0 : n > Sk ? Sk : n;
}

// A lane reports a kv_len outside [0, Sk] (it is used clamped).
__device__ __forceinline__ void check_len(const int32_t *kv_len, int b, int Sk, int *status) {
  if (kv_len && (kv_len[b] < 0 || kv_len[b] > Sk)) atomicCAS(status, kDevOk, kDevBadIndex);
}

// ---------------------------------------------------------------- host side
// [B, S, heads, D] bf16 with strides as a 4-D tensor (D, heads, S, B); box = 64 columns
// of `bh` heads of `tokens` tokens.
inline bool cross_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, const void *ptr,
                      int B, int S, int heads, int D, const nabla_strides &st, int bh,
                      int tokens) {
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)st.head * 2, (cuuint64_t)st.token * 2,
                           (cuuint64_t)st.batch * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)bh, (cuuint32_t)tokens, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace cross
}  // namespace nabla
