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
  const float *po, *plse;  // [nsplit, 2, rows, D], [nsplit, 2, rows] (base 2)
  const float *lam;
  T *o, *o2;
  float *lse;  // [B, h, 2, Sq]
  long rows;   // B h Sq, in that order, or (packed) the packed rows of the units from `first`
  long first;
  int Sq, h, hk, nsplit, lam_step, G, tq, nqt;
};

// o_m = sum_i 2^(lse_mi - lse_m) o_mi, o = o_1 - lam o_2.  A warp per row, 16 bytes a lane
// (at D 64 half of them have none); four runs are read at a time.
template <typename T, int D, bool kPacked>
__global__ void __launch_bounds__(256)
    diff_join_kernel(const __grid_constant__ JoinParams<T> P) {
  const int lane = threadIdx.x & 31, col = lane * 4;
  pdl_launch_dependents();
  pdl_wait();
  const long row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= P.rows) return;
  long b, hh, token;
  if (kPacked) {
    const long unit = P.first + (row >> 7), bj = unit / P.nqt, qt = unit - bj * P.nqt;
    const int r = (int)(row & 127), t = (r & 63) / P.G;
    b = bj / P.hk;
    hh = (bj - b * P.hk) * P.G + (r & 63) - t * P.G;
    token = (qt * 2 + (r >> 6)) * P.tq + t;
    if (t >= P.tq || token >= P.Sq) return;  // none
  } else {
    const long bh = row / P.Sq;
    token = row - bh * P.Sq;
    b = bh / P.h;
    hh = bh - b * P.h;
  }
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
  if (P.lse && lane < 2) P.lse[((b * P.h + hh) * 2 + lane) * P.Sq + token] = lane ? lse[1] : lse[0];
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
cudaError_t launch_join(const DiffArgs &a, const DiffRuns &r, cudaStream_t st) {
  const CrossShape &s = a.x.s;
  const cross::Packing pk = cross::packing(s);
  JoinParams<T> p{};
  p.po = r.po, p.plse = r.plse, p.lam = a.lam;
  p.o = static_cast<T *>(a.x.o), p.o2 = static_cast<T *>(a.o2), p.lse = a.x.lse;
  p.rows = r.rows, p.first = r.plan.whole;
  p.Sq = s.Sq, p.h = s.h, p.hk = s.hk, p.nsplit = r.plan.runs, p.lam_step = a.lam_n > 1 ? 1 : 0;
  p.G = pk.G, p.tq = pk.tq, p.nqt = (pk.nsub + 1) / 2;
  const dim3 grid((unsigned)((r.rows + 7) / 8));
  return r.plan.packed ? launch_pdl(diff_join_kernel<T, D, true>, grid, dim3(256), 0, st, p)
                       : launch_pdl(diff_join_kernel<T, D, false>, grid, dim3(256), 0, st, p);
}

}  // namespace

// How the forward's states are split into runs.  Sized for GB300's 152 SMs, so that the
// workspace depends on the shape alone.
//
// bf16: units of 128 packed rows go on the SMs in rounds; those of the last one, where they
// leave SMs idle, are split into as many runs as fill them (512 states each at least: a run
// costs some 2 us and the join 4).  8192 x 8192 states, 12 heads: 768 units, the last 8 in 19
// runs.  Few rows: runs of 512 states, or longer ones where those are many.  fp32: as in the
// cross attention, whose tiles' costs have the same proportions.
DiffPlan diff_fwd_plan(const CrossShape &s, nabla_dtype dt) {
  if (diff_few_rows(s)) {
    const long runs = (s.Sk + 511) / 512, room = 152L * 16 / ((long)s.B * s.hk);
    return {0, 0, runs <= 1 || room <= 1 ? 1 : (int)(runs < room ? runs : room), false};
  }
  if (dt == NABLA_F32) return {0, 0, cross_simt_plan(s).nsplit, false};
  const long units = (long)s.B * s.hk * ((cross::packing(s).nsub + 1) / 2);
  const long tiles = (s.Sk + diff::kStates - 1) / diff::kStates;
  const long rest = units % 152, room = rest ? 152 / rest : 1;
  const long n = room < tiles / 8 ? room : tiles / 8;
  return n < 2 ? DiffPlan{units, 0, 1, true} : DiffPlan{units - rest, rest, (int)n, true};
}

namespace {
// Rows of a run's partial results.
long run_rows(const CrossShape &s, const DiffPlan &p) {
  return p.packed ? p.rest * 128 : (long)s.B * s.h * s.Sq;
}
}  // namespace

size_t diff_fwd_workspace(const CrossShape &s, nabla_dtype dt) {
  const DiffPlan p = diff_fwd_plan(s, dt);
  return p.runs > 1 ? (size_t)p.runs * 2 * run_rows(s, p) * (s.D + 1) * sizeof(float) : 0;
}

DiffRuns diff_runs(const DiffArgs &a, nabla_dtype dt) {
  DiffRuns r{};
  r.plan = diff_fwd_plan(a.x.s, dt);
  if (r.plan.runs == 1) return r;
  r.rows = run_rows(a.x.s, r.plan);
  r.po = static_cast<float *>(a.x.workspace);
  r.plse = r.po + (size_t)r.plan.runs * 2 * r.rows * a.x.s.D;
  return r;
}

cudaError_t launch_diff_join(const DiffArgs &a, nabla_dtype dt, const DiffRuns &r,
                             cudaStream_t st) {
  if (dt == NABLA_BF16)
    return a.x.s.D == 64 ? launch_join<__nv_bfloat16, 64>(a, r, st)
                         : launch_join<__nv_bfloat16, 128>(a, r, st);
  return a.x.s.D == 64 ? launch_join<float, 64>(a, r, st)
                       : launch_join<float, 128>(a, r, st);
}

}  // namespace nabla
