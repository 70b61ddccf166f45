// The fp32 cross-attention kernels' shared pieces (256 threads as 16 x 16; thread
// (ty, tx) owns rows ty + 16 a and, of a product's columns, tx + 16 c or 4 tx + 64 e).
#pragma once

#include "attn_common.cuh"
#include "cross_common.cuh"
#include "internal.h"

namespace nabla {
namespace cross {

using tcattn::f2;
using tcattn::fma2;
using tcattn::unf2;

constexpr int kCols = 64;  // states per tile

struct SimtParams {
  const void *q, *k, *v, *dout;
  nabla_strides q_st, k_st, v_st, dout_st;
  const float *lse, *delta;  // backward, packed rows [B, hk, nsub, 64]
  float *out, *out2;         // o; dq; dk and dv (or their parts)
  float *lse_out;
  float *po, *plse;  // runs (forward) or tiles (dq of few rows): their parts
  const int32_t *kv_len;
  int B, Sq, Sk, h, hk, G, tq, nsub, nsplit;
  float scale, scale_log2;
  int *status;
};

inline SimtParams simt_params(const CrossArgs &a) {
  SimtParams p{};
  const Packing pk = packing(a.s);
  p.q = a.q, p.k = a.k, p.v = a.v, p.dout = a.dout;
  p.q_st = a.q_st, p.k_st = a.k_st, p.v_st = a.v_st, p.dout_st = a.dout_st;
  p.kv_len = a.kv_len;
  p.B = a.s.B, p.Sq = a.s.Sq, p.Sk = a.s.Sk, p.h = a.s.h, p.hk = a.s.hk;
  p.G = pk.G, p.tq = pk.tq, p.nsub = pk.nsub, p.nsplit = 1;
  p.scale = a.scale;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  return p;
}

struct Side {
  const float *p;
  nabla_strides st;
};

struct PackedRow {
  int token, head;
  bool ok;
};
__device__ __forceinline__ PackedRow packed_row(const SimtParams &P, int j, int sub, int r) {
  const int t = r / P.G;
  PackedRow w;
  w.head = j * P.G + (r - t * P.G);
  w.token = sub * P.tq + t;
  w.ok = t < P.tq && w.token < P.Sq;
  return w;
}

// 16 bytes to shared memory, asynchronously, so that a tile's copies are all in flight
// together (as loads and stores: 731 us against 633 for one token each against 16 x 4096
// states in one run, 24 heads on 8, D 128); zeros if !ok.
__device__ __forceinline__ void copy16(float *dst, const float *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>  // all but the last N groups committed
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// M packed query rows from row r0 of subtile `sub` (rows that are none: zeros).
template <int D, int M>
__device__ __forceinline__ void load_rows(float *dst, const Side &x, const SimtParams &P, int b,
                                          int j, int sub, int r0) {
  constexpr int kVec = D / 4;
  for (int e = threadIdx.x; e < M * kVec; e += 256) {
    const int r = e / kVec, c = (e - r * kVec) * 4;
    const PackedRow w = packed_row(P, j, sub, r0 + r);
    copy16(dst + r * (D + 4) + c,
           w.ok ? x.p + b * x.st.batch + w.token * x.st.token + w.head * x.st.head + c : x.p, w.ok);
  }
}

// States k0 .. k0 + 63 of key head j (from `len` on: zeros, whatever memory holds).
template <int D>
__device__ __forceinline__ void load_states(float *dst, const float *x, const nabla_strides &st,
                                            int b, int j, int k0, int len) {
  constexpr int kVec = D / 4;
  for (int e = threadIdx.x; e < kCols * kVec; e += 256) {
    const int r = e / kVec, c = (e - r * kVec) * 4;
    const bool ok = k0 + r < len;
    copy16(dst + r * (D + 4) + c,
           ok ? x + b * st.batch + (int64_t)(k0 + r) * st.token + j * st.head + c : x, ok);
  }
}

// s[a][c] = <X row ty + 16 a, Y row tx + 16 c> over D columns (rows D + 4 apart).
template <int D, int A>
__device__ __forceinline__ void dot_rows(const float *X, const float *Y, int ty, int tx,
                                         float (&s)[A][4]) {
  uint64_t acc[A][4];
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = 0ull;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    ulonglong2 x[A], y[4];
#pragma unroll
    for (int a = 0; a < A; ++a)
      x[a] = *reinterpret_cast<const ulonglong2 *>(X + (ty + 16 * a) * (D + 4) + d);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      y[c] = *reinterpret_cast<const ulonglong2 *>(Y + (tx + 16 * c) * (D + 4) + d);
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[a][c] = fma2(x[a].x, y[c].x, acc[a][c]);
        acc[a][c] = fma2(x[a].y, y[c].y, acc[a][c]);
      }
  }
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float lo, hi;
      unf2(acc[a][c], lo, hi);
      s[a][c] = lo + hi;
    }
}

// acc[a][e] += sum_u W[ty + 16 a][u] Y[u][4 tx + 64 e .. + 3] over 64 rows u of Y
// (W's rows 68 apart, Y's D + 4).
template <int D, int A>
__device__ __forceinline__ void mul_rows(const float *W, const float *Y, int ty, int tx,
                                         uint64_t (&acc)[A][D / 64][2]) {
#pragma unroll 2
  for (int u = 0; u < kCols; u += 4) {
    float4 w[A];
#pragma unroll
    for (int a = 0; a < A; ++a)
      w[a] = *reinterpret_cast<const float4 *>(W + (ty + 16 * a) * (kCols + 4) + u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ulonglong2 y[D / 64];
#pragma unroll
      for (int e = 0; e < D / 64; ++e)
        y[e] = *reinterpret_cast<const ulonglong2 *>(Y + (u + i) * (D + 4) + 4 * tx + 64 * e);
#pragma unroll
      for (int a = 0; a < A; ++a) {
        const float p = i == 0 ? w[a].x : i == 1 ? w[a].y : i == 2 ? w[a].z : w[a].w;
        const uint64_t p2 = f2(p, p);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
          acc[a][e][0] = fma2(p2, y[e].x, acc[a][e][0]);
          acc[a][e][1] = fma2(p2, y[e].y, acc[a][e][1]);
        }
      }
    }
  }
}

// The same, summed apart first.
template <int D, int A>
__device__ __forceinline__ void add_rows(const float *W, const float *Y, int ty, int tx,
                                         uint64_t (&acc)[A][D / 64][2]) {
  uint64_t t[A][D / 64][2];
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int e = 0; e < D / 64; ++e) t[a][e][0] = t[a][e][1] = 0ull;
  mul_rows<D, A>(W, Y, ty, tx, t);
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      acc[a][e][0] = tcattn::add2(acc[a][e][0], t[a][e][0]);
      acc[a][e][1] = tcattn::add2(acc[a][e][1], t[a][e][1]);
    }
}

}  // namespace cross
}  // namespace nabla
