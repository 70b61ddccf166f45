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

// o_m = sum_i 2^(lse_mi - lse_m) o_mi, o = o_1 - lam o_2.  kG warps per row, 16 bytes a lane
// (at D 64 half of them have none), each of them every kG-th run, four at a time.
template <typename T, int D, int kG>
__global__ void __launch_bounds__(256)
    diff_join_kernel(const __grid_constant__ JoinParams<T> P) {
  __shared__ float4 part[kG > 1 ? kG : 1][2][32];
  __shared__ float part_l[kG > 1 ? kG : 1][2];
  const int lane = threadIdx.x & 31, col = lane * 4, g = (threadIdx.x >> 5) % kG;
  pdl_launch_dependents();
  pdl_wait();
  const long row = (long)blockIdx.x * (8 / kG) + (threadIdx.x >> 5) / kG;
  if (row >= P.rows) return;
  const long bh = row / P.Sq, token = row - bh * P.Sq, b = bh / P.h, hh = bh - b * P.h;
  float4 o[2];
  float lse[2], top[2], sum[2];
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    float m = -INFINITY;
    for (int i = lane; i < P.nsplit; i += 32)
      m = fmaxf(m, P.plse[((size_t)i * 2 + map) * P.rows + row]);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int i0 = g; i0 < P.nsplit; i0 += 4 * kG) {
      float li[4];
      float4 src[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = i0 + x * kG;
        li[x] = i < P.nsplit ? P.plse[((size_t)i * 2 + map) * P.rows + row] : -INFINITY;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        src[x] = li[x] == -INFINITY || col >= D  // no states in this run: nothing was written
                     ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : *reinterpret_cast<const float4 *>(
                           P.po + (((size_t)(i0 + x * kG) * 2 + map) * P.rows + row) * D + col);
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
    o[map] = acc, sum[map] = l, top[map] = m;
    if constexpr (kG > 1) {
      part[g][map][lane] = acc;
      if (lane == 0) part_l[g][map] = l;
    }
  }
  if constexpr (kG > 1) {
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int map = 0; map < 2; ++map)
#pragma unroll
      for (int i = 1; i < kG; ++i) {
        const float4 x = part[i][map][lane];
        o[map].x += x.x, o[map].y += x.y, o[map].z += x.z, o[map].w += x.w;
        sum[map] += part_l[i][map];
      }
  }
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    const float l = sum[map], inv = l > 0.f ? 1.0f / l : l;  // 0 for no states; NaN stays
    o[map] = make_float4(o[map].x * inv, o[map].y * inv, o[map].z * inv, o[map].w * inv);
    lse[map] = l > 0.f ? top[map] + log2f(l) : l == 0.f ? -INFINITY : l;
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
  // A block a row where the SMs hold them all at once (one token of 24 heads on 8, 8192
  // states: 11.2 us, a warp a row 20.6; but 64 x 32 rows 41 against 35).
  if (rows <= 152 * 8)
    return launch_pdl(diff_join_kernel<T, D, 8>, dim3((unsigned)rows), dim3(256), 0, st, p);
  return launch_pdl(diff_join_kernel<T, D, 1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st,
                    p);
}

// The parts of the tcgen05 kernel's units: blockIdx.y = c - 1 joins the unit that the pieces
// of CTAs c - 1 and c share, if c is the first to go on with it.  A thread takes kQ times four
// columns of one of the first `rows` packed rows, kE parts at a time; lanes have rows, which
// the parts hold four columns at a time side by side, so a warp reads 512 bytes at once.
struct StreamParams {
  const float *po, *plse;  // [kCtas, 2 places, 2 maps, D / 4, 128, 4] and [.., 2 maps, 128]
  const float *lam;
  __nv_bfloat16 *o, *o2;
  float *lse;
  const int32_t *kv_len;
  int lam_step, B, Sq, Sk, h, hk, G, tq, nqt, rows;
  long whole;
};

template <int D, int kQ, int kE>
__global__ void __launch_bounds__(256, 2)
    diff_stream_join_kernel(const __grid_constant__ StreamParams P) {
  __shared__ int place[diff::kCtas];  // of the parts: CTA * 2 + its place
  __shared__ int count, batch, unit;
  const int lane = threadIdx.x & 31, c = blockIdx.y + 1;
  const int teams = 256 / P.rows, team = threadIdx.x / P.rows;
  const int r = threadIdx.x - team * P.rows, t = (r & 63) / P.G;
  const int quad = (blockIdx.x * teams + team) * kQ;  // of the columns
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
  if (team >= teams || quad >= D / 4 || t >= P.tq || token >= P.Sq) return;  // none
  const float lam = P.lam[hh * P.lam_step];
  float o[2][4 * kQ], lse[2];
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    auto log_sum = [&](int i) { return P.plse[(size_t)place[i] * 256 + map * 128 + r]; };
    float4 x[kE][kQ];
    auto load = [&](int i0) {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int i = i0 + e < count ? i0 + e : count - 1;
        const float4 *from = reinterpret_cast<const float4 *>(P.po) +
                             (((size_t)place[i] * 2 + map) * (D / 4) + quad) * 128 + r;
#pragma unroll
        for (int y = 0; y < kQ; ++y) x[e][y] = from[y * 128];
      }
    };
    load(0);
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < count; ++i) m = fmaxf(m, log_sum(i));
#pragma unroll
    for (int y = 0; y < 4 * kQ; ++y) o[map][y] = 0.f;
    for (int i0 = 0; i0 < count; i0 += kE) {
      if (i0) load(i0);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float li = i0 + e < count ? log_sum(i0 + e) : -INFINITY;
        if (li == -INFINITY) continue;
        const float w = exp2f(li - m);
        l += w;
#pragma unroll
        for (int y = 0; y < kQ; ++y) {
          o[map][4 * y] = fmaf(w, x[e][y].x, o[map][4 * y]);
          o[map][4 * y + 1] = fmaf(w, x[e][y].y, o[map][4 * y + 1]);
          o[map][4 * y + 2] = fmaf(w, x[e][y].z, o[map][4 * y + 2]);
          o[map][4 * y + 3] = fmaf(w, x[e][y].w, o[map][4 * y + 3]);
        }
      }
    }
    const float inv = l > 0.f ? 1.0f / l : l;  // NaN stays
#pragma unroll
    for (int y = 0; y < 4 * kQ; ++y) o[map][y] *= inv;
    lse[map] = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
  }
  if (P.lse && quad == 0) {
    float *to = P.lse + ((size_t)batch * P.h + hh) * 2 * P.Sq + token;
    to[0] = lse[0];
    to[P.Sq] = lse[1];
  }
  const size_t to = (((size_t)batch * P.Sq + token) * P.h + hh) * D + quad * 4;
  auto put = [](__nv_bfloat16 *p, const float (&v)[4 * kQ]) {
    uint32_t w[2 * kQ];
#pragma unroll
    for (int y = 0; y < 2 * kQ; ++y) w[y] = tc::pack_bf16x2(v[2 * y], v[2 * y + 1]);
    if constexpr (kQ == 1)
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else
#pragma unroll
      for (int y = 0; y < 2 * kQ; y += 4)
        *reinterpret_cast<uint4 *>(p + 2 * y) = make_uint4(w[y], w[y + 1], w[y + 2], w[y + 3]);
  };
  if (P.o2) put(P.o2 + to, o[1]);
#pragma unroll
  for (int y = 0; y < 4 * kQ; ++y) o[0][y] = fmaf(-lam, o[1][y], o[0][y]);
  put(P.o + to, o[0]);
}

}  // namespace

// How the forward is split.  Sized for GB300's 152 SMs, so that the workspace depends on the
// shape alone.
//
// bf16: units of 128 packed rows that go round the SMs; the last round or two are cut into
// equal pieces where that spares every SM at least 28 tiles of 64 states, 18 us, about what
// the parts and their join cost.  (us, whole and cut; D 128: 8192 tokens, 12 heads, 1536
// states 99, 101, 2048 states 128, 126; 64 tokens, 24 heads on 8, 2048 states 24.3, 25.0,
// 4096 states 44, 27.)  Where lengths differ they are taken to be half of Sk on average.  (One
// token of 24 heads on 8, 16 ragged batches: 2048 states 25.0, 26.3, 4096 states 45.6, 42.0,
// 8192 states 85, 66.)
//
// Few rows: runs of 256 states above 512 (one batch, 16 heads, us: 512 states whole 6.9, in two
// 8.7; 1024 in four 8.4, in two 10.3), longer ones where two CTAs an SM are all there is room
// for (16 batches, 16 heads, 1024 states: whole 23.1, in two 29.3; 4 batches, 8 heads, 4096
// states: in 9 12.6, in 16 15.9).  Where lengths differ, runs of 2048 or eight CTAs an SM at
// least, so that the longest batch holds up no one (8 batches of up to 32768, 12 heads: in 12
// 133 us, in 3 153; 64 of up to 2048, 4 heads: whole 28.9, in two 35).
//
// fp32 of more rows: rows a CTA and runs as in the cross attention.  (us, as chosen, then
// otherwise: 1024 x 257, 2 heads of 64, in 5 runs 24, in 3 27; 4096 x 512, 4 heads of 128, whole
// 184, in 4 199; 8192 x 128, 2 heads of 64, whole 30, in two 48.  At D 128 an SM holds one CTA of
// 64 rows, where those costs count on two: 2 x 500 x 77, 6 heads on 2, in two 36, whole 26.)
DiffPlan diff_fwd_plan(const CrossShape &s, nabla_dtype dt, bool ragged) {
  if (diff_few_rows(s, dt)) {
    const long heads = (long)s.B * s.hk, least = (s.Sk + 255) / 256;
    long runs = s.Sk <= 512 ? 1 : least < 304 / heads ? least : 304 / heads;
    const long more = s.Sk / 2048 < 1216 / heads ? s.Sk / 2048 : 1216 / heads;
    if (ragged && runs < more) runs = more;
    return {0, runs < 1 ? 1 : (int)runs, false};
  }
  if (dt == NABLA_F32) return {0, cross_simt_plan(s).nsplit, false};
  const long units = (long)s.B * s.hk * ((cross::packing(s).nsub + 1) / 2);
  const long tiles = (s.Sk + diff::kStates - 1) / diff::kStates;
  const long over = units % diff::kCtas;  // of a round: the others idle meanwhile
  double idle = over ? 1.0 - (double)over / diff::kCtas : 0.0;
  if (ragged && idle < 0.5) idle = 0.5;
  if (idle * (double)tiles < 28.0) return {units, 1, false};
  return {units < 2 * diff::kCtas ? 0 : (units / diff::kCtas - 1) * diff::kCtas, 1, true};
}

DiffRuns diff_runs(const DiffArgs &a, nabla_dtype dt) {
  const CrossShape &s = a.x.s;
  const DiffPlan p = diff_fwd_plan(s, dt, a.x.kv_len != nullptr);
  DiffRuns r{p.runs, nullptr, nullptr};
  if (p.runs == 1 && !p.cut) return r;
  const size_t rows = p.cut ? diff::kCtas * 2 * 256 : (size_t)p.runs * 2 * s.B * s.h * s.Sq;
  r.po = static_cast<float *>(a.x.workspace);
  r.plse = r.po + rows * s.D;
  return r;
}

size_t diff_fwd_workspace(const CrossShape &s, nabla_dtype dt) {
  const DiffPlan p = diff_fwd_plan(s, dt, true);  // cut wherever equal lengths are
  if (p.cut) return (size_t)diff::kCtas * 2 * 256 * (s.D + 1) * sizeof(float);
  return p.runs > 1 ? (size_t)p.runs * 2 * s.B * s.h * s.Sq * (s.D + 1) * sizeof(float) : 0;
}

cudaError_t launch_diff_stream_join(const DiffArgs &a, const DiffRuns &r, cudaStream_t st) {
  const CrossShape &s = a.x.s;
  const cross::Packing pk = cross::packing(s);
  // few rows: more threads for each
  const int used = s.Sq <= pk.tq ? s.Sq * pk.G : 128, rows = used <= 32 ? used : 128;
  const StreamParams p{r.po, r.plse, a.lam, static_cast<__nv_bfloat16 *>(a.x.o),
                       static_cast<__nv_bfloat16 *>(a.o2), a.x.lse, a.x.kv_len,
                       a.lam_n > 1 ? 1 : 0, s.B, s.Sq, s.Sk, s.h, s.hk, pk.G, pk.tq,
                       (pk.nsub + 1) / 2, rows,
                       diff_fwd_plan(s, NABLA_BF16, a.x.kv_len != nullptr).whole};
  const int threads = s.D / (rows < 128 ? 4 : 16), teams = 256 / rows;  // of a row, a block's
  const dim3 grid((unsigned)((threads + teams - 1) / teams), diff::kCtas - 1);
  auto kern = s.D == 64 ? (rows < 128 ? diff_stream_join_kernel<64, 1, 8>
                                      : diff_stream_join_kernel<64, 4, 2>)
                        : (rows < 128 ? diff_stream_join_kernel<128, 1, 8>
                                      : diff_stream_join_kernel<128, 4, 2>);
  return launch_pdl(kern, grid, dim3(256), 0, st, p);
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
