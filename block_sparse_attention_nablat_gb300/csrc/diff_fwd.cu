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
  long rows;   // B h Sq
  int Sq, h, nsplit, lam_step;
};

// o_m = sum_i 2^(lse_mi - lse_m) o_mi, o = o_1 - lam o_2.  A warp per row, 16 bytes a lane
// (at D 64 half of them have none); four runs are read at a time.
template <typename T, int D>
__global__ void __launch_bounds__(256)
    diff_join_kernel(const __grid_constant__ JoinParams<T> P) {
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
  const long rows = (long)s.B * s.h * s.Sq;
  const JoinParams<T> p{r.po, r.plse, a.lam, static_cast<T *>(a.x.o), static_cast<T *>(a.o2),
                        a.x.lse, rows, s.Sq, s.h, r.runs, a.lam_n > 1 ? 1 : 0};
  return launch_pdl(diff_join_kernel<T, D>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, p);
}

// The parts of the tcgen05 kernel's units: blockIdx.y = c - 1 joins the unit that the pieces
// of CTAs c - 1 and c share, if c is the first to go on with it; a warp per packed row.
struct StreamParams {
  const float *po, *plse;  // [kCtas, 2 places, 2 maps, 128, D] and [.., 128]
  const float *lam;
  __nv_bfloat16 *o, *o2;
  float *lse;
  const int32_t *kv_len;
  int lam_step, B, Sq, Sk, h, hk, G, tq, nqt;
  long whole;
};

template <int D>
__global__ void __launch_bounds__(256)
    diff_stream_join_kernel(const __grid_constant__ StreamParams P) {
  __shared__ int place[diff::kCtas];  // of the parts: CTA * 2 + its place
  __shared__ int count, batch, unit;
  const int lane = threadIdx.x & 31, col = lane * 4, c = blockIdx.y + 1;
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), t = (r & 63) / P.G;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x < 32) {  // the unit and its parts
    const int per = P.nqt * P.hk;
    const long p0 = diff::span_of_unit(P.kv_len, P.Sk, per, P.whole);
    const long n = diff::span_total(P.kv_len, P.B, P.Sk, per) - p0;
    const long from = diff::piece(p0, n, c), prev = diff::piece(p0, n, c - 1);
    int parts = 0;
    if (from < p0 + n && from != prev) {
      const diff::Span at = diff::span_find(P.kv_len, P.B, P.Sk, per, from);
      const long begin = from - at.t, end = begin + diff::weight(P.kv_len, at.b, P.Sk);
      // (one that begins here has no part before; or an earlier block joins it)
      if (at.t > 0 && prev <= begin) {
        for (int i0 = c - 1; i0 < diff::kCtas; i0 += 32) {
          const int i = i0 + lane;
          const long a = i < diff::kCtas ? diff::piece(p0, n, i) : end;
          const bool in = a < end, some = in && a != diff::piece(p0, n, i + 1);
          const uint32_t mask = __ballot_sync(0xffffffffu, some);
          // its second place, where the CTA's piece began before this unit
          if (some) place[parts + __popc(mask & ((1u << lane) - 1u))] = i * 2 + (a < begin);
          parts += __popc(mask);
          if (!__any_sync(0xffffffffu, in && i == i0 + 31)) break;
        }
        batch = at.b;
        unit = at.unit;
      }
    }
    if (lane == 0) count = parts;
  }
  __syncthreads();
  if (count == 0) return;
  const int j = unit / P.nqt, qt = unit - j * P.nqt;
  const int token = (qt * 2 + (r >> 6)) * P.tq + t, hh = j * P.G + (r & 63) - t * P.G;
  if (t >= P.tq || token >= P.Sq) return;  // none
  float4 o[2];
  float lse[2];
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    auto row = [&](int i) { return (size_t)place[i] * 256 + map * 128 + r; };
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < count; i += 32) m = fmaxf(m, P.plse[row(i)]);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < count; i0 += 4) {
      float li[4];
      float4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        li[e] = i0 + e < count ? P.plse[row(i0 + e)] : -INFINITY;
        x[e] = i0 + e < count && col < D
                   ? *reinterpret_cast<const float4 *>(P.po + row(i0 + e) * D + col)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = li[e] == -INFINITY ? 0.f : exp2f(li[e] - m);
        l += w;
        acc.x = fmaf(w, x[e].x, acc.x);
        acc.y = fmaf(w, x[e].y, acc.y);
        acc.z = fmaf(w, x[e].z, acc.z);
        acc.w = fmaf(w, x[e].w, acc.w);
      }
    }
    const float inv = l > 0.f ? 1.0f / l : l;  // NaN stays
    o[map] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    lse[map] = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
  }
  if (P.lse && lane < 2)
    P.lse[(((size_t)batch * P.h + hh) * 2 + lane) * P.Sq + token] = lane ? lse[1] : lse[0];
  if (col >= D) return;
  const float lam = P.lam[hh * P.lam_step];
  const size_t to = (((size_t)batch * P.Sq + token) * P.h + hh) * D + col;
  auto put = [](__nv_bfloat16 *p, const float4 &v) {
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(tc::pack_bf16x2(v.x, v.y), tc::pack_bf16x2(v.z, v.w));
  };
  put(P.o + to, make_float4(fmaf(-lam, o[1].x, o[0].x), fmaf(-lam, o[1].y, o[0].y),
                            fmaf(-lam, o[1].z, o[0].z), fmaf(-lam, o[1].w, o[0].w)));
  if (P.o2) put(P.o2 + to, o[1]);
}

}  // namespace

// How the forward is split.  Sized for GB300's 152 SMs, so that the workspace depends on the
// shape alone.
//
// bf16: units of 128 packed rows that go round the SMs, and from 1024 states on a last round
// or two cut into equal pieces (below that a unit costs less than joining its parts).  Few
// rows: runs of 512 states, or longer ones where those are many.  fp32: runs as in the cross
// attention, whose tiles' costs have the same proportions.
DiffPlan diff_fwd_plan(const CrossShape &s, nabla_dtype dt) {
  if (diff_few_rows(s, dt)) {
    const long runs = (s.Sk + 511) / 512, room = 152L * 16 / ((long)s.B * s.hk);
    return {0, runs <= 1 || room <= 1 ? 1 : (int)(runs < room ? runs : room), false};
  }
  if (dt == NABLA_F32) return {0, cross_simt_plan(s).nsplit, false};
  const long units = (long)s.B * s.hk * ((cross::packing(s).nsub + 1) / 2);
  if (s.Sk < 1024) return {units, 1, false};
  return {units < 2 * diff::kCtas ? 0 : (units / diff::kCtas - 1) * diff::kCtas, 1, true};
}

DiffRuns diff_runs(const DiffArgs &a, nabla_dtype dt) {
  const CrossShape &s = a.x.s;
  const DiffPlan p = diff_fwd_plan(s, dt);
  DiffRuns r{p.runs, nullptr, nullptr};
  if (p.runs == 1 && !p.cut) return r;
  const size_t rows = p.cut ? diff::kCtas * 2 * 256 : (size_t)p.runs * 2 * s.B * s.h * s.Sq;
  r.po = static_cast<float *>(a.x.workspace);
  r.plse = r.po + rows * s.D;
  return r;
}

size_t diff_fwd_workspace(const CrossShape &s, nabla_dtype dt) {
  const DiffPlan p = diff_fwd_plan(s, dt);
  if (p.cut) return (size_t)diff::kCtas * 2 * 256 * (s.D + 1) * sizeof(float);
  return p.runs > 1 ? (size_t)p.runs * 2 * s.B * s.h * s.Sq * (s.D + 1) * sizeof(float) : 0;
}

cudaError_t launch_diff_stream_join(const DiffArgs &a, const DiffRuns &r, cudaStream_t st) {
  const CrossShape &s = a.x.s;
  const cross::Packing pk = cross::packing(s);
  const StreamParams p{r.po, r.plse, a.lam, static_cast<__nv_bfloat16 *>(a.x.o),
                       static_cast<__nv_bfloat16 *>(a.o2), a.x.lse, a.x.kv_len,
                       a.lam_n > 1 ? 1 : 0, s.B, s.Sq, s.Sk, s.h, s.hk, pk.G, pk.tq,
                       (pk.nsub + 1) / 2, diff_fwd_plan(s, NABLA_BF16).whole};
  // blocks of eight packed rows, as many as a unit can have
  const int used = s.Sq < pk.tq ? s.Sq * pk.G : s.Sq < 2 * pk.tq ? 64 + (s.Sq - pk.tq) * pk.G : 128;
  const dim3 grid((unsigned)((used + 7) / 8), diff::kCtas - 1);
  return s.D == 64 ? launch_pdl(diff_stream_join_kernel<64>, grid, dim3(256), 0, st, p)
                   : launch_pdl(diff_stream_join_kernel<128>, grid, dim3(256), 0, st, p);
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
