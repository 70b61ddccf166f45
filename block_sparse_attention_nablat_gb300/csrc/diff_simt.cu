// K12f, K13f -- fp32 differential attention, forward and backward, on CUDA cores: the tiles,
// threads and products of the fp32 cross attention (cross_simt.cuh), with the two maps'
// scores over half of the columns each.
//
//  * Forward: one CTA per (batch, key head, run of packed query rows, run of states).  A
//    tile's scores of both maps are formed, each has its running maximum and sum; P_1, then
//    P_2 lie over K's tile for O_m += P_m V.  The two O are subtracted at the end.
//  * dQ: dz_1 = P_1 (dout v^T - delta_1), dz_2 = -lam P_2 (dout v^T - delta_2); a thread's
//    columns of q lie in one map's half, so one product with K serves both.
//  * dK, dV: the same with the axes exchanged; dV takes P_1 - lam P_2.
// A tile's sums of the backward are added up apart and then to the total.
//
// Bound by shared memory: a step of 64 x 64 takes 6.7 us in dQ and 10 in dK / dV at D 64, 12
// and 16 at D 128, and loads what it needs before it begins.  So few rows have their states (dQ)
// or their rows (dK, dV) split over CTAs; 16 rows a CTA in place of 64 took 4.8 us a step and
// four times the steps.
// 512 x 2048, 2 heads, D 64: backward 92 us; 1024 x 1024, 4 heads: 162 us, D 128: 255 us.
#include <cfloat>

#include "attn_common.cuh"
#include "cross_simt.cuh"
#include "diff_common.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace nabla {
namespace {

using namespace cross;

struct DiffSimt {
  SimtParams x;             // lse, delta: unused
  const float *lam;
  int lam_step;
  float *o2;                // forward, or null
  const float *rows;        // backward: -lse_1, -lse_2, -delta_1, -delta_2 (and -lam) of the packed rows
  size_t nrows;             // rows of each
};

// s[a][c] = <X row ty + 16 a, Y row tx + 16 c> over the d columns from X and Y on.
template <int D, int A>
__device__ __forceinline__ void dot_half(const float *X, const float *Y, int ty, int tx,
                                         float (&s)[A][4]) {
  uint64_t acc[A][4];
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = 0ull;
#pragma unroll 4
  for (int d = 0; d < D / 2; d += 4) {
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

// add_rows with W1 for the columns of the first map and W2 for the second's.
template <int D, int A>
__device__ __forceinline__ void add_maps(const float *W1, const float *W2, const float *Y, int ty,
                                         int tx, uint64_t (&acc)[A][D / 64][2]) {
  constexpr int E = D / 64;
  uint64_t t[A][E][2];
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int e = 0; e < E; ++e) t[a][e][0] = t[a][e][1] = 0ull;
  const float *W[E];
#pragma unroll
  for (int e = 0; e < E; ++e) W[e] = 4 * tx + 64 * e < D / 2 ? W1 : W2;
#pragma unroll 2
  for (int u = 0; u < kCols; u += 4) {
    float4 w[A][E];
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
      for (int e = 0; e < E; ++e)
        w[a][e] = *reinterpret_cast<const float4 *>(W[e] + (ty + 16 * a) * (kCols + 4) + u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const ulonglong2 y =
            *reinterpret_cast<const ulonglong2 *>(Y + (u + i) * (D + 4) + 4 * tx + 64 * e);
#pragma unroll
        for (int a = 0; a < A; ++a) {
          const float4 &q = w[a][e];
          const float p = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
          const uint64_t p2 = f2(p, p);
          t[a][e][0] = fma2(p2, y.x, t[a][e][0]);
          t[a][e][1] = fma2(p2, y.y, t[a][e][1]);
        }
      }
    }
  }
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      acc[a][e][0] = tcattn::add2(acc[a][e][0], t[a][e][0]);
      acc[a][e][1] = tcattn::add2(acc[a][e][1], t[a][e][1]);
    }
}

template <int D, int A>
constexpr int fwd_smem() {
  return (16 * A + 2 * kCols) * (D + 4) * (int)sizeof(float);
}

template <int D, int A>
__global__ void __launch_bounds__(256, A == 4 && D == 128 ? 1 : 2)
    diff_attn_simt_kernel(const __grid_constant__ DiffSimt S) {
  constexpr int M = 16 * A, LD = D + 4, LP = kCols + 4, E = D / 64;
  const SimtParams &P = S.x;
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
  load_rows<D, M>(Qs, Side{static_cast<const float *>(P.q), P.q_st}, P, b, j, sub, part * M);
  copy_commit();
  float m_run[2][A], l_run[2][A];
  uint64_t acc[2][A][E][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int a = 0; a < A; ++a) {
      m_run[m][a] = -FLT_MAX;
      l_run[m][a] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[m][a][e][0] = acc[m][a][e][1] = 0ull;
    }
  for (int k0 = t0 * kCols; k0 < t1 * kCols; k0 += kCols) {
    __syncthreads();  // the last tile's P and V are no longer read
    load_states<D>(Ks, static_cast<const float *>(P.k), P.k_st, b, j, k0, len);
    copy_commit();
    load_states<D>(Vs, static_cast<const float *>(P.v), P.v_st, b, j, k0, len);
    copy_commit();
    copy_wait<1>();  // Q, K
    __syncthreads();
    float s[2][A][4];
    dot_half<D, A>(Qs, Ks, ty, tx, s[0]);
    dot_half<D, A>(Qs + D / 2, Ks + D / 2, ty, tx, s[1]);
    copy_wait<0>();
    __syncthreads();  // V is there; K is no longer read: P takes its place
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int a = 0; a < A; ++a) {
        float mx = -FLT_MAX;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[m][a][c] *= P.scale_log2;
          if (k0 + tx + 16 * c < len) mx = fmaxf(mx, s[m][a][c]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_new = fmaxf(m_run[m][a], mx), alpha = exp2f(m_run[m][a] - m_new);
        m_run[m][a] = m_new;
        float ps = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = k0 + tx + 16 * c < len ? exp2f(s[m][a][c] - m_new) : 0.f;
          Ps[(ty + 16 * a) * LP + tx + 16 * c] = p;
          ps += p;
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l_run[m][a] = l_run[m][a] * alpha + ps;
        const uint64_t al2 = f2(alpha, alpha);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          acc[m][a][e][0] = fma2(acc[m][a][e][0], al2, 0ull);
          acc[m][a][e][1] = fma2(acc[m][a][e][1], al2, 0ull);
        }
      }
      __syncwarp();  // a row's P comes from the 16 lanes that use it
      mul_rows<D, A>(Ps, Vs, ty, tx, acc[m]);
      __syncwarp();  // and is no longer read
    }
  }
  copy_wait<0>();  // Q's, where there were no states
  const size_t all = (size_t)P.B * P.h * P.Sq;
#pragma unroll
  for (int a = 0; a < A; ++a) {
    const PackedRow r = packed_row(P, j, sub, part * M + ty + 16 * a);
    if (!r.ok) continue;
    const size_t row = ((size_t)b * P.h + r.head) * P.Sq + r.token;
    const size_t dense = (((size_t)b * P.Sq + r.token) * P.h + r.head) * D + 4 * tx;
    float inv[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float l = l_run[m][a];
      inv[m] = l > 0.f ? 1.0f / l : l;
      float *lse = P.nsplit > 1 ? P.plse + ((size_t)sp * 2 + m) * all + row
                   : P.lse_out  ? P.lse_out + (((size_t)b * P.h + r.head) * 2 + m) * P.Sq + r.token
                                : nullptr;
      if (lse && tx == 0) *lse = l > 0.f ? m_run[m][a] + log2f(l) : l == 0.f ? -INFINITY : l;
    }
    if (P.nsplit > 1 && t0 == t1) continue;  // not read
    const float lam = S.lam[r.head * S.lam_step];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float4 w[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        unf2(acc[m][a][e][0], w[m].x, w[m].y);
        unf2(acc[m][a][e][1], w[m].z, w[m].w);
        w[m].x *= inv[m], w[m].y *= inv[m], w[m].z *= inv[m], w[m].w *= inv[m];
      }
      if (P.nsplit > 1) {
        float *po = P.po + ((size_t)sp * 2 * all + row) * D + 4 * tx + 64 * e;
        *reinterpret_cast<float4 *>(po) = w[0];
        *reinterpret_cast<float4 *>(po + all * D) = w[1];
        continue;
      }
      *reinterpret_cast<float4 *>(P.out + dense + 64 * e) =
          make_float4(fmaf(-lam, w[1].x, w[0].x), fmaf(-lam, w[1].y, w[0].y),
                      fmaf(-lam, w[1].z, w[0].z), fmaf(-lam, w[1].w, w[0].w));
      if (S.o2) *reinterpret_cast<float4 *>(S.o2 + dense + 64 * e) = w[1];
    }
  }
}

// ---------------------------------------------------------------- backward

template <int D>
constexpr int dq_smem() {  // q, dout, K, V, dz of both maps
  return ((2 * 64 + 2 * kCols) * (D + 4) + 2 * 64 * (kCols + 4)) * (int)sizeof(float);
}

// CTA: run `sp` of a batch's state tiles over a subtile of 64 packed rows.
template <int D>
__global__ void __launch_bounds__(256) diff_dq_simt_kernel(const __grid_constant__ DiffSimt S) {
  constexpr int A = 4, M = 64, LD = D + 4, LP = kCols + 4, E = D / 64;
  const SimtParams &P = S.x;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Gs = Qs + M * LD, *Ks = Gs + M * LD, *Vs = Ks + kCols * LD,
        *Z1 = Vs + kCols * LD, *Z2 = Z1 + M * LP;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int sp = (int)(blockIdx.x % P.nsplit);
  const long su = blockIdx.x / P.nsplit;
  const int sub = (int)(su % P.nsub);
  const long bj = su / P.nsub;
  const int b = (int)(bj / P.hk), j = (int)(bj - (long)b * P.hk);
  pdl_launch_dependents();
  pdl_wait();
  const size_t row0 = (size_t)(bj * P.nsub + sub) * 64;
  const int len = batch_len(P.kv_len, b, P.Sk), tiles = (len + kCols - 1) / kCols;
  const int u0 = (int)((long)tiles * sp / P.nsplit) * kCols;
  const int u1 = (int)((long)tiles * (sp + 1) / P.nsplit) * kCols;
  // no rows, or a run without states, whose dQ is not read
  if (sub * P.tq >= P.Sq || (P.nsplit > 1 && u0 == u1)) return;
  load_rows<D, M>(Qs, Side{static_cast<const float *>(P.q), P.q_st}, P, b, j, sub, 0);
  load_rows<D, M>(Gs, Side{static_cast<const float *>(P.dout), P.dout_st}, P, b, j, sub, 0);
  copy_commit();
  float n[4][A], lam[A];
  uint64_t acc[A][E][2];
#pragma unroll
  for (int a = 0; a < A; ++a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i][a] = S.rows[i * S.nrows + row0 + ty + 16 * a];
    const PackedRow r = packed_row(P, j, sub, ty + 16 * a);
    lam[a] = r.ok ? S.lam[r.head * S.lam_step] : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[a][e][0] = acc[a][e][1] = 0ull;
  }
  for (int k0 = u0; k0 < u1; k0 += kCols) {
    __syncthreads();
    load_states<D>(Ks, static_cast<const float *>(P.k), P.k_st, b, j, k0, len);
    load_states<D>(Vs, static_cast<const float *>(P.v), P.v_st, b, j, k0, len);
    copy_commit();
    copy_wait<0>();
    __syncthreads();
    float s[A][4], dp[A][4];
    dot_rows<D, A>(Gs, Vs, ty, tx, dp);
    dot_half<D, A>(Qs, Ks, ty, tx, s);
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p =
            k0 + tx + 16 * c < len ? exp2f(fmaf(s[a][c], P.scale_log2, n[0][a])) : 0.f;
        Z1[(ty + 16 * a) * LP + tx + 16 * c] = p * (dp[a][c] + n[2][a]);
      }
    dot_half<D, A>(Qs + D / 2, Ks + D / 2, ty, tx, s);
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p =
            k0 + tx + 16 * c < len ? exp2f(fmaf(s[a][c], P.scale_log2, n[1][a])) : 0.f;
        Z2[(ty + 16 * a) * LP + tx + 16 * c] = -lam[a] * p * (dp[a][c] + n[3][a]);
      }
    __syncwarp();  // a row's dz comes from the 16 lanes that use it
    add_maps<D, A>(Z1, Z2, Ks, ty, tx, acc);
  }
  copy_wait<0>();  // q's and dout's, where there were no states
  const float scale = P.nsplit > 1 ? 1.f : P.scale;  // parts are scaled when they are joined
  float *out = P.out + (P.nsplit > 1 ? sp * (size_t)P.B * P.Sq * P.h * D : 0);
#pragma unroll
  for (int a = 0; a < A; ++a) {
    const PackedRow r = packed_row(P, j, sub, ty + 16 * a);
    if (!r.ok) continue;
    float *o = out + (((size_t)b * P.Sq + r.token) * P.h + r.head) * D + 4 * tx;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float4 w;
      unf2(acc[a][e][0], w.x, w.y);
      unf2(acc[a][e][1], w.z, w.w);
      *reinterpret_cast<float4 *>(o + 64 * e) =
          make_float4(w.x * scale, w.y * scale, w.z * scale, w.w * scale);
    }
  }
}

template <int D>
constexpr int dkv_smem() {  // K, V, q, dout; P^T and dz^T (one array in turn); the rows' numbers
  return (4 * 64 * (D + 4) + 3 * 64 * (kCols + 4) + 5 * 64) * (int)sizeof(float);
}

template <int D>
__global__ void __launch_bounds__(256) diff_dkv_simt_kernel(const __grid_constant__ DiffSimt S) {
  constexpr int LD = D + 4, LP = kCols + 4, E = D / 64;
  const SimtParams &P = S.x;
  extern __shared__ __align__(16) float sm[];
  float *Ks = sm, *Vs = Ks + 64 * LD, *Qs = Vs + 64 * LD, *Gs = Qs + 64 * LD, *Ps = Gs + 64 * LD,
        *Z1 = Ps + 64 * LP, *Z2 = Z1 + 64 * LP, *ls = Z2 + 64 * LP;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int nkt = (P.Sk + kCols - 1) / kCols;
  const int sp = (int)(blockIdx.x % P.nsplit);
  const long ku = blockIdx.x / P.nsplit;
  const int kt = (int)(ku % nkt);
  const long bj = ku / nkt;
  const int b = (int)(bj / P.hk), j = (int)(bj - (long)b * P.hk);
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0) check_len(P.kv_len, b, P.Sk, P.status);
  const int len = batch_len(P.kv_len, b, P.Sk), k0 = kt * kCols;
  if (P.nsplit > 1 && k0 >= len) return;  // the join writes the zeros
  load_states<D>(Ks, static_cast<const float *>(P.k), P.k_st, b, j, k0, len);
  load_states<D>(Vs, static_cast<const float *>(P.v), P.v_st, b, j, k0, len);
  copy_commit();
  uint64_t dk[4][E][2], dv[4][E][2];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int e = 0; e < E; ++e)
      dk[a][e][0] = dk[a][e][1] = dv[a][e][0] = dv[a][e][1] = 0ull;
  const int s0 = (int)((long)P.nsub * sp / P.nsplit);
  const int s1 = (int)((long)P.nsub * (sp + 1) / P.nsplit);
  for (int sub = s0; sub < s1 && k0 < len && sub * P.tq < P.Sq; ++sub) {
    __syncthreads();
    load_rows<D, 64>(Qs, Side{static_cast<const float *>(P.q), P.q_st}, P, b, j, sub, 0);
    load_rows<D, 64>(Gs, Side{static_cast<const float *>(P.dout), P.dout_st}, P, b, j, sub, 0);
    copy_commit();
    const size_t row0 = (size_t)(bj * P.nsub + sub) * 64;
    ls[tid] = S.rows[(tid >> 6) * S.nrows + row0 + (tid & 63)];
    if (tid < 64) {
      const PackedRow r = packed_row(P, j, sub, tid);
      ls[256 + tid] = r.ok ? S.lam[r.head * S.lam_step] : 0.f;
    }
    copy_wait<0>();
    __syncthreads();
    float s[4][4], dp[4][4], p1[4][4];  // rows: states ty + 16 a; columns: query rows tx + 16 c
    dot_rows<D, 4>(Vs, Gs, ty, tx, dp);
    dot_half<D, 4>(Ks, Qs, ty, tx, s);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c;
        p1[a][c] = k0 + ty + 16 * a < len ? exp2f(fmaf(s[a][c], P.scale_log2, ls[col])) : 0.f;
        Z1[(ty + 16 * a) * LP + col] = p1[a][c] * (dp[a][c] + ls[128 + col]);
      }
    dot_half<D, 4>(Ks + D / 2, Qs + D / 2, ty, tx, s);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c;
        const float p2 =
            k0 + ty + 16 * a < len
                ? ls[256 + col] * exp2f(fmaf(s[a][c], P.scale_log2, ls[64 + col]))
                : 0.f;
        Ps[(ty + 16 * a) * LP + col] = p1[a][c] - p2;
        Z2[(ty + 16 * a) * LP + col] = -p2 * (dp[a][c] + ls[192 + col]);
      }
    __syncwarp();  // a row's P and dz come from the 16 lanes that use them
    add_rows<D, 4>(Ps, Gs, ty, tx, dv);
    add_maps<D, 4>(Z1, Z2, Qs, ty, tx, dk);
  }
  copy_wait<0>();
  const size_t all = (size_t)P.B * P.Sk * P.hk * D;
  float *odk = P.nsplit > 1 ? P.out + (size_t)sp * 2 * all : P.out;
  float *odv = P.nsplit > 1 ? odk + all : P.out2;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int state = k0 + ty + 16 * a;
    if (state >= P.Sk) continue;
    const size_t at = (((size_t)b * P.Sk + state) * P.hk + j) * D + 4 * tx;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float4 w;
      unf2(dk[a][e][0], w.x, w.y);
      unf2(dk[a][e][1], w.z, w.w);
      *reinterpret_cast<float4 *>(odk + at + 64 * e) =
          make_float4(w.x * P.scale, w.y * P.scale, w.z * P.scale, w.w * P.scale);
      unf2(dv[a][e][0], w.x, w.y);
      unf2(dv[a][e][1], w.z, w.w);
      *reinterpret_cast<float4 *>(odv + at + 64 * e) = w;
    }
  }
}

// ---------------------------------------------------------------- launches

template <class K>
cudaError_t launch_with(K kern, long blocks, int smem, const DiffSimt &p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), smem, st, p);
}

template <int D>
cudaError_t launch_fwd(const DiffSimt &p, int A, long subs, cudaStream_t st) {
  const long n = subs * (4 / A) * p.x.nsplit;
  return A == 1   ? launch_with(diff_attn_simt_kernel<D, 1>, n, fwd_smem<D, 1>(), p, st)
         : A == 2 ? launch_with(diff_attn_simt_kernel<D, 2>, n, fwd_smem<D, 2>(), p, st)
                  : launch_with(diff_attn_simt_kernel<D, 4>, n, fwd_smem<D, 4>(), p, st);
}

template <int D>
cudaError_t launch_bwd(const DiffArgs &a, DiffSimt p, float *part, int nsplit, float *qpart,
                       int qsplit, cudaStream_t st) {
  const int nkt = (a.x.s.Sk + kCols - 1) / kCols;
  p.x.nsplit = nsplit;
  p.x.out = nsplit > 1 ? part : static_cast<float *>(a.x.dk);
  p.x.out2 = static_cast<float *>(a.x.dv);
  cudaError_t e = launch_with(diff_dkv_simt_kernel<D>, (long)a.x.s.B * a.x.s.hk * nkt * nsplit,
                              dkv_smem<D>(), p, st);
  if (e == cudaSuccess && nsplit > 1) e = launch_cross_dkv_join(a.x, NABLA_F32, part, nsplit, st);
  if (e != cudaSuccess) return e;
  p.x.nsplit = qsplit;
  p.x.out = qsplit > 1 ? qpart : static_cast<float *>(a.x.dq);
  e = launch_with(diff_dq_simt_kernel<D>, (long)a.x.s.B * a.x.s.hk * p.x.nsub * qsplit,
                  dq_smem<D>(), p, st);
  return e != cudaSuccess || qsplit == 1 ? e : launch_diff_dq_sum(a, NABLA_F32, qpart, qsplit, st);
}

DiffSimt diff_simt(const DiffArgs &a) {
  DiffSimt p{};
  p.x = simt_params(a.x);
  p.lam = a.lam;
  p.lam_step = a.lam_n > 1 ? 1 : 0;
  return p;
}

}  // namespace

cudaError_t launch_diff_attn_simt(const DiffArgs &a, cudaStream_t st) {
  DiffSimt p = diff_simt(a);
  p.x.out = static_cast<float *>(a.x.o);
  p.x.lse_out = a.x.lse;
  p.o2 = static_cast<float *>(a.o2);
  const DiffRuns runs = diff_runs(a, NABLA_F32);
  p.x.nsplit = runs.runs, p.x.po = runs.po, p.x.plse = runs.plse;
  const long subs = (long)a.x.s.B * a.x.s.hk * p.x.nsub;
  const int A = cross_simt_plan(a.x.s).A;
  const cudaError_t e =
      a.x.s.D == 64 ? launch_fwd<64>(p, A, subs, st) : launch_fwd<128>(p, A, subs, st);
  if (e != cudaSuccess || p.x.nsplit == 1) return e;
  return launch_diff_join(a, NABLA_F32, runs, st);
}

cudaError_t launch_diff_bwd_simt(const DiffArgs &a, const DiffRows &r, float *part, int nsplit,
                                 float *qpart, int qsplit, cudaStream_t st) {
  DiffSimt p = diff_simt(a);
  p.rows = r.rows;
  p.nrows = r.nrows;
  p.x.nsub = r.nsub;  // of the rows' layout; a subtile past the last token is skipped
  return a.x.s.D == 64 ? launch_bwd<64>(a, p, part, nsplit, qpart, qsplit, st)
                       : launch_bwd<128>(a, p, part, nsplit, qpart, qsplit, st);
}

}  // namespace nabla
