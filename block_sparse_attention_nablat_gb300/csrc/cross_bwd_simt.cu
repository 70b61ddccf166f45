// K10f -- fp32 cross attention backward on CUDA cores, the products laid out as in the
// fp32 forward (cross_simt.cuh): 256 threads as 16 x 16, tiles of 64 packed query rows and
// 64 states, pairs multiplied along the contracted axis.
//
//  * dQ: one CTA per subtile of query rows (64, or 16 of them where that leaves SMs idle);
//    it walks the batch's states, forms dz = P (dout v^T - delta) and adds dz k.
//  * dK, dV: one CTA per (batch, key head, 64 states, run of subtiles); K and V stay, the
//    subtiles pass by, P^T and dz^T give dV += P^T dout and dK += dz^T q.  Runs are added
//    up by cross_dkv_join.
//  * Few rows (at most 16 packed rows a key head: single tokens): one CTA per (batch, key
//    head, 64 states) forms dK and dV whole and its part of dQ, which cross_dq_join adds
//    up; K and V are read once.  Four tokens in all against 2862 states each, 24 heads of
//    64: the two kernels above take 1065 us, these 67.
// A tile's sums are added up apart and then to the total: over thousands of states one
// running sum would lose two bits.
// P = 2^(scale log2(e) <q, k> - lse) with the rows' -lse and -delta in packed order.
// 4096 x 512 tokens, 24 heads, D 128: 2.31 ms, 39 TFLOP/s of the seven products formed (z and
// dP in both kernels; 28 of the five that are needed, of about 75).  The 162 and 166 registers
// and 170 KB of shared memory leave 8 warps an SM, which keep neither pipe full: FMA 54%
// active, shared memory's data path 67%; of 3.5 warps waiting an issue, 0.7 wait for
// each, 1.1 for a fixed latency, 0.2 for copies and barriers.  The two need nothing of each
// other, so dQ starts on the SMs that dK and dV leave idle (500 x 77, batch 2, 6 heads on
// 2: 66 us; one after the other, with runs sized for 128-row steps, 109).
#include "attn_common.cuh"
#include "cross_common.cuh"
#include "cross_simt.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace nabla {
namespace {

using namespace cross;

template <int D, int A>
constexpr int dq_smem() {  // q, dout, K, V, dz
  return (2 * 16 * A + 2 * kCols) * (D + 4) * (int)sizeof(float) +
         16 * A * (kCols + 4) * (int)sizeof(float);
}

template <int D, int A>
__global__ void __launch_bounds__(256)
    cross_dq_simt_kernel(const SimtParams P) {
  constexpr int M = 16 * A, LD = D + 4, LP = kCols + 4, E = D / 64;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Gs = Qs + M * LD, *Ks = Gs + M * LD, *Vs = Ks + kCols * LD,
        *Zs = Vs + kCols * LD;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int parts = 64 / M, part = (int)(blockIdx.x % parts);
  const long su = blockIdx.x / parts;
  const int sub = (int)(su % P.nsub);
  const long bj = su / P.nsub;
  const int b = (int)(bj / P.hk), j = (int)(bj - (long)b * P.hk);
  pdl_launch_dependents();  // no wait: dkv's blocks launched this one after theirs
  if (tid == 0) check_len(P.kv_len, b, P.Sk, P.status);
  if (!packed_row(P, j, sub, part * M).ok) {  // nor is any later row of the tile
    pdl_wait();
    return;
  }
  const int len = batch_len(P.kv_len, b, P.Sk);
  load_rows<D, M>(Qs, Side{static_cast<const float *>(P.q), P.q_st}, P, b, j, sub, part * M);
  load_rows<D, M>(Gs, Side{static_cast<const float *>(P.dout), P.dout_st}, P, b, j, sub, part * M);
  float nl[A], nd[A];
#pragma unroll
  for (int a = 0; a < A; ++a) {
    const long r = (bj * P.nsub + sub) * 64 + part * M + ty + 16 * a;
    nl[a] = __ldcg(P.lse + r);  // written two kernels ago, without a wait in between
    nd[a] = __ldcg(P.delta + r);
  }
  uint64_t acc[A][E][2];
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[a][e][0] = acc[a][e][1] = 0ull;
  for (int k0 = 0; k0 < len; k0 += kCols) {
    __syncthreads();
    load_states<D>(Ks, static_cast<const float *>(P.k), P.k_st, b, j, k0, len);
    copy_commit();  // with q and dout
    load_states<D>(Vs, static_cast<const float *>(P.v), P.v_st, b, j, k0, len);
    copy_commit();
    copy_wait<1>();
    __syncthreads();
    float s[A][4], dp[A][4];
    dot_rows<D, A>(Qs, Ks, ty, tx, s);
    copy_wait<0>();
    __syncthreads();
    dot_rows<D, A>(Gs, Vs, ty, tx, dp);
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = k0 + tx + 16 * c < len ? exp2f(fmaf(s[a][c], P.scale_log2, nl[a])) : 0.f;
        Zs[(ty + 16 * a) * LP + tx + 16 * c] = p * (dp[a][c] + nd[a]);
      }
    __syncwarp();  // a row's dz comes from the 16 lanes that use it
    add_rows<D, A>(Zs, Ks, ty, tx, acc);
  }
#pragma unroll
  for (int a = 0; a < A; ++a) {
    const PackedRow r = packed_row(P, j, sub, part * M + ty + 16 * a);
    if (!r.ok) continue;
    float *o = P.out + (((size_t)b * P.Sq + r.token) * P.h + r.head) * D + 4 * tx;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float4 w;
      unf2(acc[a][e][0], w.x, w.y);
      unf2(acc[a][e][1], w.z, w.w);
      *reinterpret_cast<float4 *>(o + 64 * e) =
          make_float4(w.x * P.scale, w.y * P.scale, w.z * P.scale, w.w * P.scale);
    }
  }
  pdl_wait();  // whoever waits for this kernel waits for dK and dV
}

template <int D>
constexpr int dkv_smem() {  // K, V, q, dout; P^T and dz^T; lse and delta
  return 4 * 64 * (D + 4) * (int)sizeof(float) + 2 * 64 * (kCols + 4) * (int)sizeof(float) +
         128 * (int)sizeof(float);
}

template <int D>
__global__ void __launch_bounds__(256)
    cross_dkv_simt_kernel(const SimtParams P) {
  constexpr int LD = D + 4, LP = kCols + 4, E = D / 64;
  extern __shared__ __align__(16) float sm[];
  float *Ks = sm, *Vs = Ks + 64 * LD, *Qs = Vs + 64 * LD, *Gs = Qs + 64 * LD, *Ps = Gs + 64 * LD,
        *Zs = Ps + 64 * LP, *ls = Zs + 64 * LP;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int nkt = (P.Sk + kCols - 1) / kCols;
  const int sp = (int)(blockIdx.x % P.nsplit);
  const long ku = blockIdx.x / P.nsplit;
  const int kt = (int)(ku % nkt);
  const long bj = ku / nkt;
  const int b = (int)(bj / P.hk), j = (int)(bj - (long)b * P.hk);
  pdl_wait();
  pdl_launch_dependents();  // dQ, which needs no more than this kernel
  const int len = batch_len(P.kv_len, b, P.Sk), k0 = kt * kCols;
  if (P.nsplit > 1 && k0 >= len) return;  // the join writes the zeros
  load_states<D>(Ks, static_cast<const float *>(P.k), P.k_st, b, j, k0, len);
  load_states<D>(Vs, static_cast<const float *>(P.v), P.v_st, b, j, k0, len);
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
    if (tid < 128) ls[tid] = (tid < 64 ? P.lse : P.delta)[(bj * P.nsub + sub) * 64 + (tid & 63)];
    copy_wait<0>();
    __syncthreads();
    float s[4][4], dp[4][4];  // rows: states ty + 16 a; columns: query rows tx + 16 c
    dot_rows<D, 4>(Ks, Qs, ty, tx, s);
    dot_rows<D, 4>(Vs, Gs, ty, tx, dp);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c;
        const float p =
            k0 + ty + 16 * a < len ? exp2f(fmaf(s[a][c], P.scale_log2, ls[col])) : 0.f;
        Ps[(ty + 16 * a) * LP + col] = p;
        Zs[(ty + 16 * a) * LP + col] = p * (dp[a][c] + ls[64 + col]);
      }
    __syncwarp();  // a row's P and dz come from the 16 lanes that use them
    add_rows<D, 4>(Ps, Gs, ty, tx, dv);
    add_rows<D, 4>(Zs, Qs, ty, tx, dk);
  }
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

template <int D>
constexpr int few_smem() {  // K, V; q, dout; P and dz
  return (2 * kCols + 2 * 16) * (D + 4) * (int)sizeof(float) +
         2 * 16 * (kCols + 4) * (int)sizeof(float);
}

// out2 = dv, out = dk, po = the tiles' parts of dq [tiles, B hk, Sq G, D] (unscaled).
template <int D>
__global__ void __launch_bounds__(256) cross_few_simt_kernel(const SimtParams P) {
  constexpr int LD = D + 4, LP = kCols + 4, E = D / 64;
  extern __shared__ __align__(16) float sm[];
  float *Ks = sm, *Vs = Ks + kCols * LD, *Qs = Vs + kCols * LD, *Gs = Qs + 16 * LD,
        *Ps = Gs + 16 * LD, *Zs = Ps + 16 * LP;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int nkt = (P.Sk + kCols - 1) / kCols, rows = P.Sq * P.G;
  const int kt = (int)(blockIdx.x % nkt);
  const long bj = blockIdx.x / nkt;
  const int b = (int)(bj / P.hk), j = (int)(bj - (long)b * P.hk);
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0 && kt == 0) check_len(P.kv_len, b, P.Sk, P.status);
  const int len = batch_len(P.kv_len, b, P.Sk), k0 = kt * kCols;
  uint64_t dk[4][E][2], dv[4][E][2];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int e = 0; e < E; ++e)
      dk[a][e][0] = dk[a][e][1] = dv[a][e][0] = dv[a][e][1] = 0ull;
  if (k0 < len) {
    load_rows<D, 16>(Qs, Side{static_cast<const float *>(P.q), P.q_st}, P, b, j, 0, 0);
    load_rows<D, 16>(Gs, Side{static_cast<const float *>(P.dout), P.dout_st}, P, b, j, 0, 0);
    load_states<D>(Ks, static_cast<const float *>(P.k), P.k_st, b, j, k0, len);
    load_states<D>(Vs, static_cast<const float *>(P.v), P.v_st, b, j, k0, len);
    copy_commit();
    const float nl = P.lse[bj * P.nsub * 64 + ty], nd = P.delta[bj * P.nsub * 64 + ty];
    copy_wait<0>();
    __syncthreads();
    if ((ty & ~1) < rows) {  // a warp's two rows
      float s[1][4], dp[1][4];
      dot_rows<D, 1>(Qs, Ks, ty, tx, s);
      dot_rows<D, 1>(Gs, Vs, ty, tx, dp);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c;
        const float p = k0 + col < len ? exp2f(fmaf(s[0][c], P.scale_log2, nl)) : 0.f;
        Ps[ty * LP + col] = p;
        Zs[ty * LP + col] = p * (dp[0][c] + nd);
      }
      __syncwarp();
      uint64_t dq[1][E][2];
#pragma unroll
      for (int e = 0; e < E; ++e) dq[0][e][0] = dq[0][e][1] = 0ull;
      mul_rows<D, 1>(Zs, Ks, ty, tx, dq);
      if (ty < rows) {
        float *o = P.po + (((size_t)kt * P.B * P.hk + bj) * rows + ty) * D + 4 * tx;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float4 w;
          unf2(dq[0][e][0], w.x, w.y);
          unf2(dq[0][e][1], w.z, w.w);
          *reinterpret_cast<float4 *>(o + 64 * e) = w;
        }
      }
    }
    __syncthreads();
    for (int r = 0; r < rows; ++r) {
      ulonglong2 q[E], g[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[e] = *reinterpret_cast<const ulonglong2 *>(Qs + r * LD + 4 * tx + 64 * e);
        g[e] = *reinterpret_cast<const ulonglong2 *>(Gs + r * LD + 4 * tx + 64 * e);
      }
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float p = Ps[r * LP + ty + 16 * a], z = Zs[r * LP + ty + 16 * a];
        const uint64_t p2 = f2(p, p), z2 = f2(z, z);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          dv[a][e][0] = fma2(p2, g[e].x, dv[a][e][0]);
          dv[a][e][1] = fma2(p2, g[e].y, dv[a][e][1]);
          dk[a][e][0] = fma2(z2, q[e].x, dk[a][e][0]);
          dk[a][e][1] = fma2(z2, q[e].y, dk[a][e][1]);
        }
      }
    }
  }
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
      *reinterpret_cast<float4 *>(P.out + at + 64 * e) =
          make_float4(w.x * P.scale, w.y * P.scale, w.z * P.scale, w.w * P.scale);
      unf2(dv[a][e][0], w.x, w.y);
      unf2(dv[a][e][1], w.z, w.w);
      *reinterpret_cast<float4 *>(P.out2 + at + 64 * e) = w;
    }
  }
}

// dq of the few rows: the tiles' parts added up in order.  A thread per four columns.
template <int D>
__global__ void __launch_bounds__(64) cross_dq_join_kernel(const SimtParams P, float *dq) {
  const int rows = P.Sq * P.G;
  const long i = (long)blockIdx.x * 64 + threadIdx.x;
  const long row = i / (D / 4);
  const int c = (int)(i % (D / 4)) * 4;
  pdl_launch_dependents();
  pdl_wait();
  if (row >= (long)P.B * P.hk * rows) return;
  const long bj = row / rows;
  const int r = (int)(row - bj * rows), b = (int)(bj / P.hk), j = (int)(bj - (long)b * P.hk);
  const int tiles = (batch_len(P.kv_len, b, P.Sk) + kCols - 1) / kCols;
  const size_t step = (size_t)P.B * P.hk * rows * D;
  const float *p = P.po + (size_t)row * D + c;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int t = 0; t < tiles; ++t) {
    const float4 x = *reinterpret_cast<const float4 *>(p + t * step);
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
  }
  const PackedRow w = packed_row(P, j, 0, r);
  *reinterpret_cast<float4 *>(dq + (((size_t)b * P.Sq + w.token) * P.h + w.head) * D + c) =
      make_float4(s.x * P.scale, s.y * P.scale, s.z * P.scale, s.w * P.scale);
}

template <int D>
cudaError_t launch_few(const CrossArgs &a, SimtParams p, float *part, cudaStream_t st) {
  auto kern = cross_few_simt_kernel<D>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem<D>());
  if (e != cudaSuccess) return e;
  p.out = static_cast<float *>(a.dk);
  p.out2 = static_cast<float *>(a.dv);
  p.po = part;
  const long units = (long)p.B * p.hk * ((p.Sk + kCols - 1) / kCols);
  e = launch_pdl(kern, dim3((unsigned)units), dim3(256), few_smem<D>(), st, p);
  if (e != cudaSuccess) return e;
  const long n = (long)p.B * p.h * p.Sq * (D / 4);
  return launch_pdl(cross_dq_join_kernel<D>, dim3((unsigned)((n + 63) / 64)), dim3(64), 0, st, p,
                    static_cast<float *>(a.dq));
}

template <int D, int A>
cudaError_t launch_dq(const SimtParams &p, cudaStream_t st) {
  auto kern = cross_dq_simt_kernel<D, A>;
  const int smem = dq_smem<D, A>();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long subs = (long)p.B * p.hk * p.nsub;
  return launch_pdl(kern, dim3((unsigned)(subs * (4 / A))), dim3(256), smem, st, p);
}

template <int D>
cudaError_t launch_d(const CrossArgs &a, SimtParams p, float *part, int nsplit, cudaStream_t st) {
  auto kern = cross_dkv_simt_kernel<D>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dkv_smem<D>());
  if (e != cudaSuccess) return e;
  p.nsplit = nsplit;
  p.out = nsplit > 1 ? part : static_cast<float *>(a.dk);
  p.out2 = static_cast<float *>(a.dv);
  const long units = (long)p.B * p.hk * ((p.Sk + kCols - 1) / kCols) * nsplit;
  e = launch_pdl(kern, dim3((unsigned)units), dim3(256), dkv_smem<D>(), st, p);
  if (e != cudaSuccess) return e;
  p.out = static_cast<float *>(a.dq);
  // 16 rows a CTA only where 64 would leave most SMs idle: beside dK and dV, whose blocks
  // fill SMs too, 96 CTAs of 64 rows do better than 384 of 16 (66 against 75 us in all at
  // 2 x 500 x 77 tokens, 6 heads on 2)
  const bool few = (long)p.B * p.hk * p.nsub < 64;
  e = few ? launch_dq<D, 1>(p, st) : launch_dq<D, 4>(p, st);
  if (e != cudaSuccess || nsplit == 1) return e;
  return launch_cross_dkv_join(a, NABLA_F32, part, nsplit, st);
}

}  // namespace

cudaError_t launch_cross_bwd_simt(const CrossArgs &a, const float *nlse, const float *ndelta,
                                  float *part, int nsub, cudaStream_t st) {
  SimtParams p = simt_params(a);
  p.lse = nlse;
  p.delta = ndelta;
  p.nsub = nsub;  // the packed rows' own, a whole number of pairs
  if (cross_few_rows(a.s, NABLA_F32))
    return a.s.D == 64 ? launch_few<64>(a, p, part, st) : launch_few<128>(a, p, part, st);
  const int nsplit = cross_dkv_splits(a.s, NABLA_F32);
  return a.s.D == 64 ? launch_d<64>(a, p, part, nsplit, st)
                     : launch_d<128>(a, p, part, nsplit, st);
}

}  // namespace nabla
