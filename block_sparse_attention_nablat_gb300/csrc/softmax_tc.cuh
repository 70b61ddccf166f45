// Softmax pieces of the tcgen05 attention kernels: 32 scores of a row in registers.
#pragma once

#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace nabla {
namespace cross {

using tcattn::add2;
using tcattn::f2;
using tcattn::fma2;
using tcattn::max3;
using tcattn::unf2;

// 32 scores -> P = 2^(s * sl2 - m) in bf16 pairs (16 words); sums in acc0, acc1.
__device__ __forceinline__ void x_exp(const uint32_t (&r)[32], uint64_t sc2, uint64_t nm2,
                                      uint64_t &acc0, uint64_t &acc1, uint32_t (&pk)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float x0, x1, y0, y1;
    unf2(fma2(f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), sc2, nm2), x0, x1);
    unf2(fma2(f2(__uint_as_float(r[2 * i + 2]), __uint_as_float(r[2 * i + 3])), sc2, nm2), y0,
         y1);
    x0 = tc::ex2(x0);
    x1 = tc::ex2(x1);
    y0 = tc::ex2(y0);
    y1 = tc::ex2(y1);
    acc0 = add2(acc0, f2(x0, x1));
    acc1 = add2(acc1, f2(y0, y1));
    pk[i] = tc::pack_bf16x2(x0, x1);
    pk[i + 1] = tc::pack_bf16x2(y0, y1);
  }
}

// Scores from column `valid` on (past the batch's states) as -inf, whatever was computed
// there.
__device__ __forceinline__ void x_mask(int valid, uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = i < valid ? r[i] : 0xff800000u;
}

__device__ __forceinline__ void x_max(const uint32_t (&r)[32], float &a0, float &a1) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    a0 = max3(a0, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
    a1 = max3(a1, __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
  }
}

}  // namespace cross
}  // namespace nabla
