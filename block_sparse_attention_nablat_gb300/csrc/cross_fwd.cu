// The cross attention forward's runs: how many a batch's states are split into when there
// are few rows, and the kernel that joins them.
#include <cuda_bf16.h>

#include "cross_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace nabla {
namespace {

template <typename T>
struct JoinParams {
  const float *po, *plse;  // [nsplit, B, h, Sq, D], [nsplit, B, h, Sq] (base 2)
  T *o;
  float *lse;
  long rows;  // B h Sq
  int Sq, h, nsplit;
};

// o = sum_i 2^(lse_i - lse) o_i.  A warp per row; four runs are read at a time, since a
// row's loads are all that this short kernel waits for.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_combine_kernel(const JoinParams<T> P) {
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const long row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= P.rows) return;
  float m = -INFINITY;
  for (int i = lane; i < P.nsplit; i += 32) m = fmaxf(m, P.plse[(size_t)i * P.rows + row]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  constexpr int kV = D / 32;
  float acc[kV], l = 0.f;
#pragma unroll
  for (int e = 0; e < kV; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < P.nsplit; i0 += 4) {
    float li[4], src[4][kV];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      li[x] = i0 + x < P.nsplit ? P.plse[(size_t)(i0 + x) * P.rows + row] : -INFINITY;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int e = 0; e < kV; ++e)
        src[x][e] = li[x] == -INFINITY  // no states in this run: nothing was written
                        ? 0.f
                        : P.po[((size_t)(i0 + x) * P.rows + row) * D + lane * kV + e];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float w = li[x] == -INFINITY ? 0.f : exp2f(li[x] - m);
      l += w;
#pragma unroll
      for (int e = 0; e < kV; ++e) acc[e] = fmaf(w, src[x][e], acc[e]);
    }
  }
  const float inv = l > 0.f ? 1.0f / l : l;  // 0 for no states; NaN stays
  const long bh = row / P.Sq, token = row - bh * P.Sq, b = bh / P.h, hh = bh - b * P.h;
  T *dst = P.o + ((b * P.Sq + token) * P.h + hh) * D + lane * kV;
#pragma unroll
  for (int e = 0; e < kV; e += 2) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint32_t *>(dst + e) = tc::pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    else
      *reinterpret_cast<float2 *>(dst + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
  }
  if (P.lse && lane == 0) P.lse[row] = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
}

template <typename T, int D>
cudaError_t launch_join(const CrossArgs &a, int nsplit, cudaStream_t st) {
  const CrossShape &s = a.s;
  const long rows = (long)s.B * s.h * s.Sq;
  const CrossRuns r = cross_runs(a, nsplit);
  const JoinParams<T> p{r.po, r.plse, static_cast<T *>(a.o), a.lse, rows, s.Sq, s.h, nsplit};
  return launch_pdl(cross_combine_kernel<T, D>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0,
                    st, p);
}

}  // namespace

// Sized for GB300's 152 SMs, so that the workspace depends on the shape alone.
//
// bf16: a unit (128 packed rows of one batch and key head) streams its keys and values at
// up to 1/128 of the HBM's rate, and starting a run and joining the runs cost a few
// microseconds.  So 1 run, unless two or more fill the SMs in one wave; runs of four
// tiles at least.  One token each, D 128, us: 16 x 4096 states, 24 heads on 8: 43 whole,
// 48 in 2 runs, 53 in 5; 8 x 4096: 32 whole, 27 in 2, 30 in 4; 1 x 8192, 24 heads: 24 in 6,
// 26 in 12, 32 in 26; 1 head: 12 in 16, 14 in 32, 21 in 64.
//
// fp32: cross_simt_plan.
int cross_fwd_splits(const CrossShape &s, nabla_dtype dt) {
  const bool few = cross_few_rows(s, dt);
  if (dt == NABLA_F32 && !few) return cross_simt_plan(s).nsplit;
  // fp32, few rows: 64-state tiles, a unit per key head
  const long units = (long)s.B * s.hk * (few ? 1 : (cross::packing(s).nsub + 1) / 2);
  const long tiles = few ? (s.Sk + 63) / 64 : (s.Sk + cross::kTile - 1) / cross::kTile;
  auto runs = [&](long room) {
    const long n = room / units < tiles / 4 ? room / units : tiles / 4;
    return n < 2 ? 1 : (int)n;
  };
  if (!few) return runs(152);
  const int two = runs(304);
  if (s.Sq * (s.h / s.hk) <= 8) return two;  // two CTAs on an SM
  // More than 8 rows are held in registers, which leaves one CTA an SM: one wave of longer
  // runs, or two of shorter ones where those fill the SMs better.  (D 128, us in one wave
  // and in two: 9 rows x 8192 states, 8 heads: 42, 52; 16 x 2048, 24 heads: 44, 56; D 64:
  // 10 x 8192, 100 heads: 316 whole, 222 in 3 runs; 16 x 8192, 60 heads: 216, 183.)
  const int one = runs(152);
  return 2 * ((tiles + two - 1) / two) < (tiles + one - 1) / one ? two : one;
}

// Rows per CTA (16 A) and runs of the fp32 kernel's walk over the states, by the time they
// take: a 64-state tile costs about 8, 9, 11.5 us (A = 1, 2, 4; D 128) where CTAs are alone
// on their SMs, 10, 11, 14 where two share one, and joining n runs 3 + n / 5; runs only
// while they still go two to an SM.  (Forward, D 128, us for A = 1, 2, 4: 2 x 500 x 77
// tokens, 6 heads on 2: 34, 26, 29; 4096 x 512, 24 heads: 1698, 975, 672.)
CrossSimtPlan cross_simt_plan(const CrossShape &s) {
  const cross::Packing pk = cross::packing(s);
  const int rows = (s.Sq < pk.tq ? s.Sq : pk.tq) * pk.G;  // of the largest subtile
  const int tiles = (s.Sk + 63) / 64;
  CrossSimtPlan best{4, 1};
  double least = 0.0;
  for (int x = 2; x >= 0; --x) {
    const int A = 1 << x;
    const double alone = A == 1 ? 8.0 : A == 2 ? 9.0 : 11.5;
    const double shared = A == 1 ? 10.0 : A == 2 ? 11.0 : 14.0;
    const long units = (long)s.B * s.hk * pk.nsub * ((rows + 16 * A - 1) / (16 * A));
    for (int n = 1; n == 1 || (n <= tiles && units * n <= 304); ++n) {
      const long full = units * n / 304, rest = units * n % 304;
      const double wave = full * shared + (rest == 0 ? 0.0 : rest <= 152 ? alone : shared);
      const double cost = wave * ((tiles + n - 1) / n) + (n > 1 ? 3.0 + 0.2 * n : 0.0);
      if ((A == 4 && n == 1) || cost < least) {
        best = CrossSimtPlan{A, n};
        least = cost;
      }
    }
  }
  return best;
}

size_t cross_fwd_workspace(const CrossShape &s, nabla_dtype dt) {
  const int n = cross_fwd_splits(s, dt);
  return n > 1 ? (size_t)n * s.B * s.h * s.Sq * (s.D + 1) * sizeof(float) : 0;
}

CrossRuns cross_runs(const CrossArgs &a, int nsplit) {
  if (nsplit == 1) return CrossRuns{nullptr, nullptr};
  float *po = static_cast<float *>(a.workspace);
  return CrossRuns{po, po + (size_t)nsplit * a.s.B * a.s.h * a.s.Sq * a.s.D};
}

cudaError_t launch_cross_combine(const CrossArgs &a, nabla_dtype dt, int nsplit,
                                 cudaStream_t st) {
  if (dt == NABLA_BF16)
    return a.s.D == 64 ? launch_join<__nv_bfloat16, 64>(a, nsplit, st)
                       : launch_join<__nv_bfloat16, 128>(a, nsplit, st);
  return a.s.D == 64 ? launch_join<float, 64>(a, nsplit, st)
                     : launch_join<float, 128>(a, nsplit, st);
}

}  // namespace nabla
