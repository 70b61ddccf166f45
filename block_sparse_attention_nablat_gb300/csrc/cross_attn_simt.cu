// K9f -- fp32 cross attention forward on CUDA cores (tcgen05 has no fp32 MMA and tf32
// would not hold fp32 accuracy).
//
// One CTA per (batch, key head, run of packed query rows; cross_common.cuh), 256
// threads as 16 x 16.  It walks the batch's states in tiles of 64: scores, online
// softmax (running maximum and sum per row, base 2 with the scale folded in), O += P V.
// Thread (ty, tx) owns rows ty + 16 a and, of the scores, columns tx + 16 c; of O,
// columns 4 tx + 64 e .. + 3.  Both products read shared memory in 16-byte pieces (the
// scores along D, P V along the states) and multiply pairs (fma.rn.f32x2), so a warp
// issues 32 pair-FMAs for 12 wavefronts of shared memory and the FMA pipe bounds the
// kernel.  P takes over K's tile, which leaves room for two CTAs per SM at D = 128.
// 64 rows a CTA, or 32 or 16 where 64 would leave SMs without work (short queries); where
// those are still few the states are split into runs (cross_combine joins them).
// 4096 x 512 tokens, 24 heads, D 128: 646 us, 40 TFLOP/s (the pipe's peak is about 75).
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

  float m_run[A], l_run[A];
  uint64_t acc[A][E][2];
#pragma unroll
  for (int a = 0; a < A; ++a) {
    m_run[a] = -FLT_MAX;
    l_run[a] = 0.f;
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
      const uint64_t al2 = f2(alpha, alpha);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        acc[a][e][0] = fma2(acc[a][e][0], al2, 0ull);
        acc[a][e][1] = fma2(acc[a][e][1], al2, 0ull);
      }
    }
    __syncwarp();  // a row's P comes from the 16 lanes that use it
    mul_rows<D, A>(Ps, Vs, ty, tx, acc);
  }
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
    float *o = (P.nsplit > 1 ? P.po + run * D
                             : P.out + (((size_t)b * P.Sq + r.token) * P.h + r.head) * D) +
               4 * tx;
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
  const CrossSimtPlan plan = cross_simt_plan(a.s);
  p.nsplit = plan.nsplit;
  const CrossRuns runs = cross_runs(a, p.nsplit);
  p.po = runs.po, p.plse = runs.plse;
  const long subs = (long)a.s.B * a.s.hk * p.nsub;
  const cudaError_t e = a.s.D == 64 ? launch_a<64>(p, plan.A, subs, st)
                                    : launch_a<128>(p, plan.A, subs, st);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  return launch_cross_combine(a, NABLA_F32, p.nsplit, st);
}

}  // namespace nabla
