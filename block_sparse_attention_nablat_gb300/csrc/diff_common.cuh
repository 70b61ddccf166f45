// What the differential-attention kernels share.  A head's D columns of q and k hold the
// two maps' d = D / 2 side by side, so all else is as in the cross attention: the packing
// of the rows that share a key head into tiles, strides, lengths and runs.
#pragma once

#include "cross_common.cuh"
#include "internal.h"

namespace nabla {
namespace diff {

constexpr int kStates = 64;  // states per tile

// 16-state MMA steps of tile t of a batch with `len` states: 4, or fewer in its last tile.
__device__ __forceinline__ int steps16(int len, int t) {
  const int left = len - t * kStates;
  return left >= kStates ? 4 : (left + 15) >> 4;
}

// Rows [rows, end) of a tile (128 bytes a row and box) as zeros; a whole warp.
template <int kBoxes>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int box, int rows, int end) {
  const int n16 = (end - rows) * 8;
  for (int c = 0; c < kBoxes; ++c)
    for (int e = threadIdx.x & 31; e < n16; e += 32)
      *reinterpret_cast<uint4 *>(tile + c * box + rows * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
  tc::fence_async_smem();
  __syncwarp();
}

// Whether a barrier's phase is over, for one thread.  A wait costs some 130 cycles even where
// it is; asked for several barriers at once, or ahead of other work, the answers come together.
__device__ __forceinline__ bool is_over(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// A whole warp's wait, `over` saying whether it was asked already and is.
__device__ __forceinline__ void wait_unless(bool over, bool &live, uint64_t *bar, uint32_t parity,
                                            volatile int *abort, int *status) {
  if (!__all_sync(0xffffffffu, over)) cross::warp_wait(live, bar, parity, abort, status);
}

// 16-column step kk (of all D columns) of a K-major tile of `box` bytes a box.
__device__ __forceinline__ uint64_t k_step(int kk, int box) {
  return (uint64_t)(((kk >> 2) * box + (kk & 3) * 32) >> 4);
}

// ---- How the forward's units (128 packed rows of a batch and key head, `per` of them a
// batch) are dealt out.  The first `whole` go round the CTAs, so that those at work share a
// few heads' states in L2.  The others, a round or two of them, are laid end to end, every
// unit as long as its batch has state tiles (one, where it has none), and cut into kCtas
// equal pieces: however the lengths differ, every CTA gets the same.  A CTA's piece begins and
// ends inside a unit; those parts' results go to its two places in the workspace.
constexpr int kCtas = 152;  // GB300's SMs

__device__ __forceinline__ int weight(const int32_t *kv_len, int b, int Sk) {
  const int n = (cross::batch_len(kv_len, b, Sk) + kStates - 1) / kStates;
  return n > 0 ? n : 1;
}

struct Span {  // tile t of unit `unit` of batch b
  int b, unit, t;
};

// All of a warp: the length of all units, and where position `at` lies.
__device__ __forceinline__ long span_total(const int32_t *kv_len, int B, int Sk, int per) {
  if (!kv_len) return (long)B * per * weight(nullptr, 0, Sk);
  long n = 0;
  for (int b = threadIdx.x & 31; b < B; b += 32) n += weight(kv_len, b, Sk);
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * per;
}
__device__ __forceinline__ Span span_find(const int32_t *kv_len, int B, int Sk, int per, long at) {
  if (!kv_len) {
    const int w = weight(nullptr, 0, Sk);
    const long u = at / w;
    return Span{(int)(u / per), (int)(u % per), (int)(at - u * w)};
  }
  const int lane = threadIdx.x & 31;
  long base = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int w = b0 + lane < B ? weight(kv_len, b0 + lane, Sk) : 0;
    long end = (long)w * per;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    const uint32_t in = __ballot_sync(0xffffffffu, at < base + end);
    if (in) {
      const int l = __ffs(in) - 1, wl = __shfl_sync(0xffffffffu, w, l);
      const long rest = at - base - __shfl_sync(0xffffffffu, end - (long)w * per, l);
      return Span{b0 + l, (int)(rest / wl), (int)(rest % wl)};
    }
    base += __shfl_sync(0xffffffffu, end, 31);
  }
  return Span{B, 0, 0};  // the end
}
// The position of unit `u`.
__device__ __forceinline__ long span_of_unit(const int32_t *kv_len, int Sk, int per, long u) {
  const int b = (int)(u / per), lane = threadIdx.x & 31;
  if (!kv_len) return u * weight(nullptr, 0, Sk);
  long n = 0;
  for (int i = lane; i < b; i += 32) n += weight(kv_len, i, Sk);
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  const long in = u - (long)b * per;
  return n * per + (in ? in * weight(kv_len, b, Sk) : 0);
}
// Where the piece of CTA c begins, of `n` positions from p0 on.
__device__ __forceinline__ long piece(long p0, long n, int c) {
  // (a division of 64 bits takes several times as long, and they come one after another)
  return p0 + (n < (1L << 24) ? (long)((uint32_t)n * (uint32_t)c / kCtas) : n * c / kCtas);
}

}  // namespace diff
}  // namespace nabla
