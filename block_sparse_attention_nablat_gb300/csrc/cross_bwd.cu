// The parts of the cross attention backward around its products: the rows' lse and delta
// in packed order (before), and the sum of the dK / dV runs (after).
#include <cuda_bf16.h>

#include "cross_common.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace nabla {
namespace {

__device__ __forceinline__ float dot8(const float *a, const float *b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 x = *reinterpret_cast<const float4 *>(a + i);
    const float4 y = *reinterpret_cast<const float4 *>(b + i);
    s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
  }
  return s;
}
__device__ __forceinline__ float dot8(const __nv_bfloat16 *a, const __nv_bfloat16 *b) {
  const uint4 x = *reinterpret_cast<const uint4 *>(a), y = *reinterpret_cast<const uint4 *>(b);
  const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), s);
    s = fmaf(__uint_as_float(u[i] & 0xffff0000u), __uint_as_float(v[i] & 0xffff0000u), s);
  }
  return s;
}

// -lse and -delta = -<dout, o> of the packed rows [B, hk, nsub, 64]: -inf and 0 where a
// row is none or has no states, so that its P is 0.  A block takes a 64-row subtile,
// D / 8 lanes a row, 16 bytes of bf16 a lane; HBM-bound (o and dout read once), so a
// thread's rows are all in flight at once.
template <typename T, int D>
__global__ void __launch_bounds__(256)
    cross_prep_kernel(const T *__restrict__ o, const nabla_strides o_st,
                      const T *__restrict__ dout, const nabla_strides g_st,
                      const float *__restrict__ lse, int Sq, int h, int hk, int G, int tq,
                      int nsub, float *__restrict__ nlse, float *__restrict__ ndelta) {
  constexpr int kLanes = D / 8, kPass = 256 / kLanes, kRows = 64 / kPass;
  const int lane = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  pdl_launch_dependents();
  const uint32_t bj = blockIdx.x / (uint32_t)nsub, sub = blockIdx.x - bj * nsub;
  const uint32_t b = bj / (uint32_t)hk, j = bj - b * hk;
  o += b * o_st.batch + lane * 8;
  dout += b * g_st.batch + lane * 8;
  lse += (size_t)b * h * Sq;
  pdl_wait();
  float s[kRows], l[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t r = r0 + i * kPass, t = r / (uint32_t)G;
    const int token = (int)(sub * tq + t), hh = (int)(j * G + r - t * G);
    s[i] = 0.f;
    l[i] = -INFINITY;
    if (t < (uint32_t)tq && token < Sq) {
      s[i] = dot8(dout + token * g_st.token + hh * g_st.head,
                  o + token * o_st.token + hh * o_st.head);
      if (lane == 0) l[i] = lse[(size_t)hh * Sq + token];
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
#pragma unroll
    for (int x = kLanes / 2; x; x >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], x);
    if (lane == 0) {
      const size_t row = (size_t)blockIdx.x * 64 + r0 + i * kPass;
      nlse[row] = l[i] == -INFINITY ? -INFINITY : -l[i];
      ndelta[row] = -s[i];
    }
  }
}

// dK and dV: the runs' fp32 sums added up in order and rounded; 0 past the length (where
// no run wrote anything).
template <typename T>
__global__ void __launch_bounds__(256)
    cross_dkv_join_kernel(const float *__restrict__ part, int nsplit, int Sk, int row, long n4,
                          const int32_t *kv_len, T *dk, T *dv) {
  pdl_launch_dependents();
  pdl_wait();
  const long i = (long)blockIdx.x * 256 + threadIdx.x;  // four columns of dK, then of dV
  if (i >= 2 * n4) return;
  const bool v = i >= n4;
  const long e = (v ? i - n4 : i) * 4, state = e / row;
  const long b = state / Sk;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (state - b * Sk < cross::batch_len(kv_len, (int)b, Sk)) {
    for (int k = 0; k < nsplit; ++k) {
      const float4 p =
          *reinterpret_cast<const float4 *>(part + ((size_t)k * 2 + v) * (size_t)n4 * 4 + e);
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
  }
  T *o = (v ? dv : dk) + e;
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2 *>(o) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                               *reinterpret_cast<const uint32_t *>(&hi));
  } else {
    *reinterpret_cast<float4 *>(o) = s;
  }
}

template <typename T, int D>
cudaError_t launch_prep(const CrossArgs &a, const cross::Packing &pk, int nsub, float *nlse,
                        float *ndelta, cudaStream_t st) {
  const long blocks = (long)a.s.B * a.s.hk * nsub;
  return launch_pdl(cross_prep_kernel<T, D>, dim3((unsigned)blocks), dim3(256), 0, st,
                    static_cast<const T *>(a.of), a.o_st, static_cast<const T *>(a.dout), a.dout_st,
                    (const float *)a.lse, a.s.Sq, a.s.h, a.s.hk, pk.G, pk.tq, nsub, nlse, ndelta);
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

struct BwdLayout {
  int nsub;  // subtiles per (batch, key head), a whole number of 128-row tiles
  size_t nlse, ndelta, part, qpart, total;
};
BwdLayout bwd_layout(const CrossShape &s, nabla_dtype dt) {
  BwdLayout w;
  w.nsub = (cross::packing(s).nsub + 1) / 2 * 2;
  const size_t rows = round_up((size_t)s.B * s.hk * w.nsub * 64 * sizeof(float));
  const int n = cross_few_rows(s, dt) ? 1 : cross_dkv_splits(s, dt);
  w.nlse = 0;
  w.ndelta = rows;
  w.part = 2 * rows;
  w.total = w.part + (n > 1 ? round_up((size_t)n * 2 * s.B * s.Sk * s.hk * s.D * sizeof(float))
                            : 0);
  w.qpart = w.total;
  if (dt == NABLA_BF16 && cross_dq_splits(s) > 1)
    w.total += round_up((size_t)cross_dq_splits(s) * s.B * s.Sq * s.h * s.D * sizeof(float));
  if (cross_few_rows(s, dt))
    w.total += round_up((size_t)((s.Sk + 63) / 64) * s.B * s.h * s.Sq * s.D * sizeof(float));
  return w;
}

}  // namespace

bool cross_few_rows(const CrossShape &s, nabla_dtype dt) {
  return dt == NABLA_F32 && (long)s.Sq * (s.h / s.hk) <= 16;
}

cudaError_t launch_cross_dkv_join(const CrossArgs &a, nabla_dtype dt, const float *part,
                                  int nsplit, cudaStream_t st) {
  const long n4 = (long)a.s.B * a.s.Sk * a.s.hk * a.s.D / 4;
  const dim3 grid((unsigned)((2 * n4 + 255) / 256));
  if (dt == NABLA_BF16)
    return launch_pdl(cross_dkv_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, part, nsplit,
                      a.s.Sk, a.s.hk * a.s.D, n4, a.kv_len, static_cast<__nv_bfloat16 *>(a.dk),
                      static_cast<__nv_bfloat16 *>(a.dv));
  return launch_pdl(cross_dkv_join_kernel<float>, grid, dim3(256), 0, st, part, nsplit, a.s.Sk,
                    a.s.hk * a.s.D, n4, a.kv_len, static_cast<float *>(a.dk),
                    static_cast<float *>(a.dv));
}

// Runs of query tiles the dK / dV units are split into.  Cost in steps: the waves of units
// over GB300's 152 SMs times a unit's steps (and what it takes to start and end one), and
// the runs' sums written and read back.  A step is a 128 x 128 tile in bf16, about a
// microsecond, in which 6 MB move; in fp32 64 x 64 on CUDA cores, about 15.
int cross_dkv_splits(const CrossShape &s, nabla_dtype dt) {
  const bool tc = dt == NABLA_BF16;
  const int tile = tc ? cross::kTile : 64, nsub = cross::packing(s).nsub;
  const long units = (long)s.B * s.hk * ((s.Sk + tile - 1) / tile);
  const int nq = tc ? (nsub + 1) / 2 : nsub;
  const double start = tc ? 2.0 : 0.2, moved = tc ? 6.0e6 : 90.0e6;
  int best = 1;
  double least = 0.0;
  for (int n = 1; n <= nq && n <= 64; ++n) {
    const double waves = (double)((units * n + 151) / 152);
    double cost = waves * ((nq + n - 1) / n + start);
    if (n > 1) cost += start + (double)units * n * tile * s.D * 2 * 4 * 2 / moved;
    if (n == 1 || cost < least) {
      best = n;
      least = cost;
    }
  }
  return best;
}

// Runs of state tiles the bf16 dQ units are split into: as in the forward, only where they
// still go on the SMs in one wave, four tiles at least.  (Whole backward, D 128, us, in runs
// and whole: 2 x 6 tokens, 4553 states, 24 heads: 115, 141; 1 x 8192, 1 head: 25, 77;
// 300 x 4096, 8 heads: 45, 60.)
int cross_dq_splits(const CrossShape &s) {
  const long units = (long)s.B * s.hk * ((cross::packing(s).nsub + 1) / 2);
  const long runs = 152 / units, tiles = (s.Sk + cross::kTile - 1) / cross::kTile;
  const long n = runs < tiles / 4 ? runs : tiles / 4;
  return n < 2 ? 1 : (int)n;
}

size_t cross_bwd_workspace(const CrossShape &s, nabla_dtype dt) { return bwd_layout(s, dt).total; }

cudaError_t launch_cross_bwd(const CrossArgs &a, nabla_dtype dt, cudaStream_t st) {
  const BwdLayout w = bwd_layout(a.s, dt);
  char *ws = static_cast<char *>(a.workspace);
  float *nlse = reinterpret_cast<float *>(ws + w.nlse);
  float *ndelta = reinterpret_cast<float *>(ws + w.ndelta);
  float *part = reinterpret_cast<float *>(ws + w.part);
  const cross::Packing pk = cross::packing(a.s);
  cudaError_t e;
  if (dt == NABLA_BF16)
    e = a.s.D == 64 ? launch_prep<__nv_bfloat16, 64>(a, pk, w.nsub, nlse, ndelta, st)
                    : launch_prep<__nv_bfloat16, 128>(a, pk, w.nsub, nlse, ndelta, st);
  else
    e = a.s.D == 64 ? launch_prep<float, 64>(a, pk, w.nsub, nlse, ndelta, st)
                    : launch_prep<float, 128>(a, pk, w.nsub, nlse, ndelta, st);
  if (e != cudaSuccess) return e;
  float *qpart = reinterpret_cast<float *>(ws + w.qpart);
  return dt == NABLA_BF16 ? launch_cross_bwd_tc(a, nlse, ndelta, part, qpart, st)
                          : launch_cross_bwd_simt(a, nlse, ndelta, part, w.nsub, st);
}

}  // namespace nabla
