// K9f -- fp32 cross attention forward on CUDA cores (tcgen05 has no fp32 MMA and tf32
// would not hold fp32 accuracy).
//
// One CTA per (batch, key head, run of packed query rows; cross_common.cuh), 256
// threads as 16 x 16.  It walks the batch's states in tiles of 64: scores, online
// softmax (running maximum and sum per row, base 2 with the scale folded in), O += P V.
// Thread (ty, tx) owns rows ty + 16 a and, of the scores, columns tx + 16 c; of O,
// columns 4 tx + 64 e .. + 3.  Both products read shared memory in 16-byte pieces (the
// scores along D, P V along the states) and multiply pairs (fma.rn.f32x2), so a warp
// issues 32 pair-FMAs for 12 wavefronts of shared memory.  P takes over K's tile, which
// leaves room for two CTAs per SM at D = 128.
// 64 rows a CTA, or 32 or 16 where 64 would leave SMs without work (short queries); where
// those are still few the states are split into runs (cross_combine joins them).
// 4096 x 512 tokens, 24 heads, D 128: 646 us, 40 TFLOP/s of about 75.  Shared memory's data
// path is busy 73% of the time and the FMA pipe 62%, with 15 warps an SM to keep both: of 7.3
// warps waiting an issue, 1.6 wait for the FMA pipe, 1.3 for shared memory, 1.1 for a fixed
// latency and 0.4 for the tiles' copies and barriers.
#include <cfloat>

#include "attn_common.cuh"
#include "cross_common.cuh"
#include "cross_simt.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace nabla {
namespace {

using namespace cross;

template <int D, int A>
constexpr int fwd_smem() {
  return (16 * A + 2 * kCols) * (D + 4) * (int)sizeof(float);
}
// Tiles whose O is summed in registers before it goes to the sum so far, which lies where
// the rows go: one running sum over 7200 states was off by 2.2e-6 of its norm, this one is
// by 0.6e-6.  (Kept in shared memory it left one CTA an SM: 4096 x 512 tokens, 24 heads,
// D 128 took 757 us instead of 646.)
constexpr int kFold = 8;

template <int D, int A>
__global__ void __launch_bounds__(256, 2)
    cross_attn_simt_kernel(const SimtParams P) {
  constexpr int M = 16 * A, LD = D + 4, LP = kCols + 4, E = D / 64;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Ks = Qs + M * LD, *Vs = Ks + kCols * LD, *Ps = Ks;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int parts = 64 / M;
  const int sp = (int)(blockIdx.x % P.nsplit);
  const long blk = blockIdx.x / P.nsplit;
  const int part = (int)(blk % parts);
  const long su = blk / parts;
  const int sub = (int)(su % P.nsub);
  const long bj = su / P.nsub;
  const int b = (int)(bj / P.hk), j = (int)(bj - (long)b * P.hk);
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0) check_len(P.kv_len, b, P.Sk, P.status);
  if (!packed_row(P, j, sub, part * M).ok) return;  // nor is any later row of the tile
  const int len = batch_len(P.kv_len, b, P.Sk), tiles = (len + kCols - 1) / kCols;
  const int t0 = (int)((long)tiles * sp / P.nsplit), t1 = (int)((long)tiles * (sp + 1) / P.nsplit);
  const Side q{static_cast<const float *>(P.q), P.q_st};
  load_rows<D, M>(Qs, q, P, b, j, sub, part * M);
  copy_commit();

  float m_run[A], l_run[A], beta[A];  // beta: what O so far is to be scaled by
  uint64_t acc[A][E][2];
  bool folded = false;
  auto place = [&](const PackedRow &r) {  // the thread's columns of a row of o, or of a run's
    const size_t row = ((size_t)b * P.h + r.head) * P.Sq + r.token;
    return (P.nsplit > 1 ? P.po + ((size_t)sp * P.B * P.h * P.Sq + row) * D
                         : P.out + (((size_t)b * P.Sq + r.token) * P.h + r.head) * D) +
           4 * tx;
  };
  auto fold = [&](bool last) {  // O so far += acc; the last time acc += O so far
#pragma unroll
    for (int a = 0; a < A; ++a) {
      const PackedRow r = packed_row(P, j, sub, part * M + ty + 16 * a);
      if (r.ok) {
        float *o = place(r);
        const uint64_t b2 = f2(beta[a], beta[a]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          ulonglong2 *at = reinterpret_cast<ulonglong2 *>(o + 64 * e), w;
          if (folded) {
            w = *at;
            acc[a][e][0] = fma2(w.x, b2, acc[a][e][0]);
            acc[a][e][1] = fma2(w.y, b2, acc[a][e][1]);
          }
          if (last) continue;
          w.x = acc[a][e][0], w.y = acc[a][e][1];
          *at = w;
          acc[a][e][0] = acc[a][e][1] = 0ull;
        }
      }
      beta[a] = 1.f;
    }
    folded = true;
  };
#pragma unroll
  for (int a = 0; a < A; ++a) {
    m_run[a] = -FLT_MAX;
    l_run[a] = 0.f;
    beta[a] = 1.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[a][e][0] = acc[a][e][1] = 0ull;
  }
  for (int k0 = t0 * kCols; k0 < t1 * kCols; k0 += kCols) {
    __syncthreads();  // the last tile's P and V are no longer read
    load_states<D>(Ks, static_cast<const float *>(P.k), P.k_st, b, j, k0, len);
    copy_commit();
    load_states<D>(Vs, static_cast<const float *>(P.v), P.v_st, b, j, k0, len);
    copy_commit();
    copy_wait<1>();  // Q, K
    __syncthreads();
    float s[A][4];
    dot_rows<D, A>(Qs, Ks, ty, tx, s);
    copy_wait<0>();
    __syncthreads();  // V is there; K is no longer read: P takes its place
#pragma unroll
    for (int a = 0; a < A; ++a) {
      float mx = -FLT_MAX;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[a][c] *= P.scale_log2;
        if (k0 + tx + 16 * c < len) mx = fmaxf(mx, s[a][c]);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m_run[a], mx);
      const float alpha = exp2f(m_run[a] - m_new);
      m_run[a] = m_new;
      float ps = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = k0 + tx + 16 * c < len ? exp2f(s[a][c] - m_new) : 0.f;
        Ps[(ty + 16 * a) * LP + tx + 16 * c] = p;
        ps += p;
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
      l_run[a] = l_run[a] * alpha + ps;
      beta[a] *= alpha;
      const uint64_t al2 = f2(alpha, alpha);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        acc[a][e][0] = fma2(acc[a][e][0], al2, 0ull);
        acc[a][e][1] = fma2(acc[a][e][1], al2, 0ull);
      }
    }
    __syncwarp();  // a row's P comes from the 16 lanes that use it
    mul_rows<D, A>(Ps, Vs, ty, tx, acc);
    if ((k0 / kCols - t0 + 1) % kFold == 0 && k0 + kCols < t1 * kCols) fold(false);
  }
  if (folded) fold(true);
#pragma unroll
  for (int a = 0; a < A; ++a) {
    const PackedRow r = packed_row(P, j, sub, part * M + ty + 16 * a);
    if (!r.ok) continue;
    const float l = l_run[a], inv = l > 0.f ? 1.0f / l : l;
    const size_t row = ((size_t)b * P.h + r.head) * P.Sq + r.token;
    const size_t run = (size_t)sp * P.B * P.h * P.Sq + row;  // of a run's sums
    float *lse = P.nsplit > 1 ? P.plse + run : P.lse_out ? P.lse_out + row : nullptr;
    if (lse && tx == 0) *lse = l > 0.f ? m_run[a] + log2f(l) : l == 0.f ? -INFINITY : l;
    if (P.nsplit > 1 && t0 == t1) continue;  // not read
    float *o = place(r);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float4 w;
      unf2(acc[a][e][0], w.x, w.y);
      unf2(acc[a][e][1], w.z, w.w);
      *reinterpret_cast<float4 *>(o + 64 * e) =
          make_float4(w.x * inv, w.y * inv, w.z * inv, w.w * inv);
    }
  }
}

// Few rows (at most 16 packed rows a key head: single tokens).  The mapping above reads a
// tile out of shared memory once for every pair of rows' warp, 10 us a tile whether its
// rows are there or not; here a tile is read once, and the work goes with the rows.  One
// token each against 16 x 4096 states, 24 heads on 8, D 128: 97 us, 5.5 TB/s (324 above).
//   scores: four threads a state, a quarter of D each; its piece of K stays in registers
//           while the rows pass by;
//   softmax: thread (ty, tx), as above;
//   O: a warp takes eight states, a lane four columns of all rows; the warps' sums are
//           added at the end.
// The next tile's K is loaded behind the softmax and O, its V behind the scores.
template <int D>
struct Few {
  // K rows 64 bytes apart modulo 128, so the two states of eight lanes meet no bank twice
  static constexpr int LK = D + 16, LP = kCols + 4;
  static constexpr int kOffV = kCols * LK, kOffQ = kOffV + kCols * D, kOffS = kOffQ + 16 * D;
  static constexpr int kOffA = kOffS + 16 * LP, kFloats = kOffA + 48;
};

template <int D, int kR>
__global__ void __launch_bounds__(256) cross_few_attn_kernel(const SimtParams P) {
  using F = Few<D>;
  constexpr int kPieces = D / 16, kSets = 256 / (D / 4);  // 16-byte pieces a thread; sets of O
  extern __shared__ __align__(16) float sm[];
  float *Ks = sm, *Vs = sm + F::kOffV, *Qs = sm + F::kOffQ, *Ss = sm + F::kOffS,
        *al = sm + F::kOffA;  // and l, m
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int sp = (int)(blockIdx.x % P.nsplit);
  const long bj = blockIdx.x / P.nsplit;
  const int b = (int)(bj / P.hk), j = (int)(bj - (long)b * P.hk), rows = P.Sq * P.G;
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0) check_len(P.kv_len, b, P.Sk, P.status);
  const int len = batch_len(P.kv_len, b, P.Sk), tiles = (len + kCols - 1) / kCols;
  const int t0 = (int)((long)tiles * sp / P.nsplit), t1 = (int)((long)tiles * (sp + 1) / P.nsplit);
  const float *k = static_cast<const float *>(P.k) + b * P.k_st.batch + j * P.k_st.head;
  const float *v = static_cast<const float *>(P.v) + b * P.v_st.batch + j * P.v_st.head;
  auto load = [&](float *dst, int pitch, const float *src, int64_t token, int t) {
    if (t < t1)
#pragma unroll
      for (int e = tid; e < kCols * (D / 4); e += 256) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        const bool ok = t * kCols + r < len;
        copy16(dst + r * pitch + c, ok ? src + (int64_t)(t * kCols + r) * token + c : src, ok);
      }
    copy_commit();
  };
  for (int e = tid; e < 16 * (D / 4); e += 256) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    const PackedRow w = packed_row(P, j, 0, r);
    const float *q = static_cast<const float *>(P.q);
    copy16(Qs + r * D + c,
           w.ok ? q + b * P.q_st.batch + w.token * P.q_st.token + w.head * P.q_st.head + c : q,
           w.ok);
  }
  load(Ks, F::LK, k, P.k_st.token, t0);
  load(Vs, D, v, P.v_st.token, t0);
  float m_run = -FLT_MAX, l_run = 0.f;
  uint64_t acc[kR][2];
#pragma unroll
  for (int r = 0; r < kR; ++r) acc[r][0] = acc[r][1] = 0ull;
  const int state = tid >> 2, quarter = tid & 3;
  const int set = tid / (D / 4), col = (tid % (D / 4)) * 4;  // O: states of this set, 4 columns
  for (int t = t0; t < t1; ++t) {
    copy_wait<1>();
    __syncthreads();  // Q and K are there
    {
      ulonglong2 kk[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        kk[i] = *reinterpret_cast<const ulonglong2 *>(Ks + state * F::LK + (quarter + 4 * i) * 4);
      for (int r = 0; r < rows; ++r) {
        uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const ulonglong2 q =
              *reinterpret_cast<const ulonglong2 *>(Qs + r * D + (quarter + 4 * i) * 4);
          s0 = fma2(q.x, kk[i].x, s0);
          s1 = fma2(q.y, kk[i].y, s1);
        }
        float a, c, e, f;
        unf2(s0, a, c);
        unf2(s1, e, f);
        float s = (a + c) + (e + f);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (quarter == 0) Ss[r * F::LP + state] = s * P.scale_log2;
      }
    }
    __syncthreads();  // the scores are there, K is no longer read
    load(Ks, F::LK, k, P.k_st.token, t + 1);
    if ((ty & ~1) < rows) {  // a warp's two rows
      float s[4], mx = -FLT_MAX;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[c] = Ss[ty * F::LP + tx + 16 * c];
        if (t * kCols + tx + 16 * c < len) mx = fmaxf(mx, s[c]);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m_run, mx), alpha = exp2f(m_run - m_new);
      m_run = m_new;
      float ps = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = t * kCols + tx + 16 * c < len ? exp2f(s[c] - m_new) : 0.f;
        Ss[ty * F::LP + tx + 16 * c] = p;
        ps += p;
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
      l_run = l_run * alpha + ps;
      if (tx == 0) al[ty] = alpha;
    }
    copy_wait<1>();
    __syncthreads();  // P and V are there
    constexpr int kOwn = kCols / kSets;  // states of a set: 8, or 4
    uint64_t part[kR][2];
#pragma unroll
    for (int r = 0; r < kR; ++r) part[r][0] = part[r][1] = 0ull;
#pragma unroll
    for (int u = 0; u < kOwn; u += 4) {
      ulonglong2 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[i] = *reinterpret_cast<const ulonglong2 *>(Vs + (set * kOwn + u + i) * D + col);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r >= rows) break;
        const float4 p4 = *reinterpret_cast<const float4 *>(Ss + r * F::LP + set * kOwn + u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = i == 0 ? p4.x : i == 1 ? p4.y : i == 2 ? p4.z : p4.w;
          part[r][0] = fma2(f2(p, p), y[i].x, part[r][0]);
          part[r][1] = fma2(f2(p, p), y[i].y, part[r][1]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (r >= rows) break;
      const uint64_t a2 = f2(al[r], al[r]);
      acc[r][0] = fma2(acc[r][0], a2, part[r][0]);
      acc[r][1] = fma2(acc[r][1], a2, part[r][1]);
    }
    __syncthreads();  // V and P are no longer read
    load(Vs, D, v, P.v_st.token, t + 1);
  }
  copy_wait<0>();
  __syncthreads();
  // the warps' sums, over K and V: [warp][row][D]
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    if (r >= rows) break;
    ulonglong2 w;
    w.x = acc[r][0], w.y = acc[r][1];
    if (D == 64) {  // a warp's two sets
      w.x = tcattn::add2(w.x, __shfl_xor_sync(0xffffffffu, w.x, 16));
      w.y = tcattn::add2(w.y, __shfl_xor_sync(0xffffffffu, w.y, 16));
    }
    if ((tid & 31) < D / 4)
      *reinterpret_cast<ulonglong2 *>(sm + ((tid >> 5) * kR + r) * D + col) = w;
  }
  if (tx == 0 && ty < rows) al[16 + ty] = l_run, al[32 + ty] = m_run;
  __syncthreads();
  for (int e = tid; e < rows * (D / 4); e += 256) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 x = *reinterpret_cast<const float4 *>(sm + (i * kR + r) * D + c);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    const PackedRow w = packed_row(P, j, 0, r);
    const float l = al[16 + r], inv = l > 0.f ? 1.0f / l : l;
    const size_t row = ((size_t)b * P.h + w.head) * P.Sq + w.token;
    const size_t run = (size_t)sp * P.B * P.h * P.Sq + row;  // of a run's sums
    float *lse = P.nsplit > 1 ? P.plse + run : P.lse_out ? P.lse_out + row : nullptr;
    if (lse && c == 0) *lse = l > 0.f ? al[32 + r] + log2f(l) : l == 0.f ? -INFINITY : l;
    if (P.nsplit > 1 && t0 == t1) continue;  // not read
    float *o = P.nsplit > 1 ? P.po + run * D
                            : P.out + (((size_t)b * P.Sq + w.token) * P.h + w.head) * D;
    *reinterpret_cast<float4 *>(o + c) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
  }
}

template <int D, int kR>
cudaError_t launch_few(const SimtParams &p, cudaStream_t st) {
  static_assert(8 * kR * D <= Few<D>::kOffQ, "the warps' sums go over K and V");
  auto kern = cross_few_attn_kernel<D, kR>;
  const int smem = Few<D>::kFloats * (int)sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)((long)p.B * p.hk * p.nsplit)), dim3(256), smem, st, p);
}

// Rows held in registers: with 16 a CTA is alone on its SM.
template <int D>
cudaError_t launch_few_rows(const SimtParams &p, int rows, cudaStream_t st) {
  return rows <= 4   ? launch_few<D, 4>(p, st)
         : rows <= 8 ? launch_few<D, 8>(p, st)
                     : launch_few<D, 16>(p, st);
}

template <int D, int A>
cudaError_t launch_f(const SimtParams &p, long subs, cudaStream_t st) {
  auto kern = cross_attn_simt_kernel<D, A>;
  const int smem = fwd_smem<D, A>();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)(subs * (4 / A) * p.nsplit)), dim3(256), smem, st, p);
}

template <int D>
cudaError_t launch_a(const SimtParams &p, int A, long subs, cudaStream_t st) {
  return A == 1   ? launch_f<D, 1>(p, subs, st)
         : A == 2 ? launch_f<D, 2>(p, subs, st)
                  : launch_f<D, 4>(p, subs, st);
}

}  // namespace

cudaError_t launch_cross_attn_simt(const CrossArgs &a, cudaStream_t st) {
  SimtParams p = simt_params(a);
  p.out = static_cast<float *>(a.o);
  p.lse_out = a.lse;
  p.nsplit = cross_fwd_splits(a.s, NABLA_F32);
  const CrossRuns runs = cross_runs(a, p.nsplit);
  p.po = runs.po, p.plse = runs.plse;
  const long subs = (long)a.s.B * a.s.hk * p.nsub;
  cudaError_t e;
  if (cross_few_rows(a.s, NABLA_F32)) {
    const int rows = a.s.Sq * p.G;
    e = a.s.D == 64 ? launch_few_rows<64>(p, rows, st) : launch_few_rows<128>(p, rows, st);
  } else {
    const int A = cross_simt_plan(a.s).A;
    e = a.s.D == 64 ? launch_a<64>(p, A, subs, st) : launch_a<128>(p, A, subs, st);
  }
  if (e != cudaSuccess || p.nsplit == 1) return e;
  return launch_cross_combine(a, NABLA_F32, p.nsplit, st);
}

}  // namespace nabla
