// The differential attention forward's runs: how many a batch's states are split into when
// there are few rows, and the kernel that joins them.
#include <cuda_bf16.h>

#include "diff_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace nabla {
namespace {

template <typename T>
struct JoinParams {
  const float *po, *plse;  // [nsplit, 2, B, h, Sq, D], [nsplit, 2, B, h, Sq] (base 2)
  const float *lam;
  T *o, *o2;
  float *lse;  // [B, h, 2, Sq]
  long rows;   // B h Sq
  int Sq, h, nsplit, lam_step;
};

// o_m = sum_i 2^(lse_mi - lse_m) o_mi, o = o_1 - lam o_2.  A warp per row, 16 bytes a lane
// (at D 64 half of them have none); four runs are read at a time.
template <typename T, int D>
__global__ void __launch_bounds__(256) diff_join_kernel(const JoinParams<T> P) {
  const int lane = threadIdx.x & 31, col = lane * 4;
  pdl_launch_dependents();
  pdl_wait();
  const long row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= P.rows) return;
  const long bh = row / P.Sq, token = row - bh * P.Sq, b = bh / P.h, hh = bh - b * P.h;
  float4 o[2];
  float lse[2];
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    float m = -INFINITY;
    for (int i = lane; i < P.nsplit; i += 32)
      m = fmaxf(m, P.plse[((size_t)i * 2 + map) * P.rows + row]);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int i0 = 0; i0 < P.nsplit; i0 += 4) {
      float li[4];
      float4 src[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        li[x] = i0 + x < P.nsplit ? P.plse[((size_t)(i0 + x) * 2 + map) * P.rows + row]
                                  : -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        src[x] = li[x] == -INFINITY || col >= D  // no states in this run: nothing was written
                     ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : *reinterpret_cast<const float4 *>(
                           P.po + (((size_t)(i0 + x) * 2 + map) * P.rows + row) * D + col);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float w = li[x] == -INFINITY ? 0.f : exp2f(li[x] - m);
        l += w;
        acc.x = fmaf(w, src[x].x, acc.x);
        acc.y = fmaf(w, src[x].y, acc.y);
        acc.z = fmaf(w, src[x].z, acc.z);
        acc.w = fmaf(w, src[x].w, acc.w);
      }
    }
    const float inv = l > 0.f ? 1.0f / l : l;  // 0 for no states; NaN stays
    o[map] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    lse[map] = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
  }
  if (P.lse && lane < 2) P.lse[(bh * 2 + lane) * P.Sq + token] = lane ? lse[1] : lse[0];
  if (col >= D) return;
  const float lam = P.lam[hh * P.lam_step];
  const float4 d = make_float4(fmaf(-lam, o[1].x, o[0].x), fmaf(-lam, o[1].y, o[0].y),
                               fmaf(-lam, o[1].z, o[0].z), fmaf(-lam, o[1].w, o[0].w));
  const long to = ((b * P.Sq + token) * P.h + hh) * D + col;
  auto put = [](T *p, const float4 &v) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2 *>(p) =
          make_uint2(tc::pack_bf16x2(v.x, v.y), tc::pack_bf16x2(v.z, v.w));
    else
      *reinterpret_cast<float4 *>(p) = v;
  };
  put(P.o + to, d);
  if (P.o2) put(P.o2 + to, o[1]);
}

template <typename T, int D>
cudaError_t launch_join(const DiffArgs &a, int nsplit, cudaStream_t st) {
  const CrossShape &s = a.x.s;
  const long rows = (long)s.B * s.h * s.Sq;
  const CrossRuns r = diff_runs(a, nsplit);
  const JoinParams<T> p{r.po, r.plse, a.lam, static_cast<T *>(a.x.o), static_cast<T *>(a.o2),
                        a.x.lse, rows, s.Sq, s.h, nsplit, a.lam_n > 1 ? 1 : 0};
  return launch_pdl(diff_join_kernel<T, D>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, p);
}

}  // namespace

// Sized for GB300's 152 SMs, so that the workspace depends on the shape alone.  bf16: runs
// only where two or more of every unit go on the SMs in one wave, 512 states at least.  fp32:
// as in the cross attention, whose tiles' costs have the same proportions.
int diff_fwd_splits(const CrossShape &s, nabla_dtype dt) {
  if (dt == NABLA_F32) return cross_simt_plan(s).nsplit;
  const long units = (long)s.B * s.hk * ((cross::packing(s).nsub + 1) / 2);
  const long tiles = (s.Sk + diff::kStates - 1) / diff::kStates;
  const long n = 152 / units < tiles / 8 ? 152 / units : tiles / 8;
  return n < 2 ? 1 : (int)n;
}

size_t diff_fwd_workspace(const CrossShape &s, nabla_dtype dt) {
  const int n = diff_fwd_splits(s, dt);
  return n > 1 ? (size_t)n * 2 * s.B * s.h * s.Sq * (s.D + 1) * sizeof(float) : 0;
}

CrossRuns diff_runs(const DiffArgs &a, int nsplit) {
  if (nsplit == 1) return CrossRuns{nullptr, nullptr};
  const CrossShape &s = a.x.s;
  float *po = static_cast<float *>(a.x.workspace);
  return CrossRuns{po, po + (size_t)nsplit * 2 * s.B * s.h * s.Sq * s.D};
}

cudaError_t launch_diff_join(const DiffArgs &a, nabla_dtype dt, int nsplit, cudaStream_t st) {
  if (dt == NABLA_BF16)
    return a.x.s.D == 64 ? launch_join<__nv_bfloat16, 64>(a, nsplit, st)
                         : launch_join<__nv_bfloat16, 128>(a, nsplit, st);
  return a.x.s.D == 64 ? launch_join<float, 64>(a, nsplit, st)
                       : launch_join<float, 128>(a, nsplit, st);
}

}  // namespace nabla
