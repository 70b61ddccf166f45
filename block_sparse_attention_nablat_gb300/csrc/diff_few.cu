// K12s -- differential attention forward of few rows: a single packed row a key head (one token)
// in bf16, up to four in fp32.
//
// Bound by the bytes of K and V.  D columns of a state lie over the lanes of a group, 16
// bytes a lane (bf16, D 128: 16 lanes, two states a warp and load), the first half of the
// lanes holding map 1's columns of K, the others map 2's.  A group walks its own states
// with its own running maxima and sums: no barrier but at the end.  A lane's pieces come by
// asynchronous copies into places of its own in shared memory, three steps of eight copies
// ahead, 190 KB under way on an SM.  Scores: products of the
// lane's columns, added up over the half group; then every lane has its own map's P, takes
// the other's from the other half, and adds both times its columns of V.  The groups of a CTA
// are joined in shared memory at the end, CTAs (runs of a batch's states) by diff_join.
// 16 x 1000 states at most, half of them there, 16 heads, D 128, bf16: 21 us, 3.2 TB/s.
#include <cuda_bf16.h>

#include <cfloat>
#include <type_traits>

#include "attn_common.cuh"
#include "diff_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace nabla {
namespace {

using tcattn::add2;
using tcattn::f2;
using tcattn::fma2;
using tcattn::unf2;

struct FewParams {
  const void *q, *k, *v;
  nabla_strides q_st, k_st, v_st;
  const float *lam;
  const int32_t *kv_len;
  void *o, *o2;
  float *lse;         // [B, h, 2, Sq]
  float *po, *plse;   // runs
  int lam_step, B, Sq, Sk, h, hk, G, nsplit;
  float scale_log2;
  int *status;
};

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 16 bytes as fp32 pairs.
__device__ __forceinline__ void widen(const uint4 &r, uint64_t (&v)[4], __nv_bfloat16) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void widen(const uint4 &r, uint64_t (&v)[2], float) {
  v[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
  v[1] = f2(__uint_as_float(r.z), __uint_as_float(r.w));
}
__device__ __forceinline__ void put(__nv_bfloat16 *p, const float4 &v) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(tc::pack_bf16x2(v.x, v.y), tc::pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void put(float *p, const float4 &v) {
  *reinterpret_cast<float4 *>(p) = v;
}

constexpr int kAhead = 4, kDepth = 3;  // states of a group in a step; steps copied ahead

template <typename T, int D, int kR>
constexpr int few_smem() {
  constexpr int groups = 256 / (D * (int)sizeof(T) / 16);
  constexpr int copies = kDepth * 2 * kAhead * 256 * 16, sums = kR * groups * 2 * (D + 4) * 4;
  return copies > sums ? copies : sums;
}

__device__ __forceinline__ void copy16(uint4 *to, const void *from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(to)), "l"(from),
               "r"(on ? 16 : 0)
               : "memory");
}

// CTA: run `sp` of the states of batch b and key head j; kR: rows at most.
template <typename T, int D, int kR>
__global__ void __launch_bounds__(256, kR == 4 ? 1 : 2)
    diff_few_kernel(const __grid_constant__ FewParams P) {
  constexpr int kCols = 16 / (int)sizeof(T), kPairs = kCols / 2;  // columns a lane
  constexpr int kLanes = D / kCols, kHalf = kLanes / 2;           // of a group, of a map's half
  constexpr int kGroups = 256 / kLanes;
  __shared__ float ml[kGroups][2][kR][2];                         // maximum and sum
  // The copies' places, [step in turn][K's, V's][thread]; in the end the groups' sums,
  // [row][group][map][D + 4].
  extern __shared__ __align__(16) uint4 ring[];
  float *sums = reinterpret_cast<float *>(ring);
  __shared__ float total[2][kR][2];                               // of all groups
  const int tid = threadIdx.x, lane = tid % kLanes, group = tid / kLanes;
  const bool second = lane >= kHalf;
  const int sp = (int)(blockIdx.x % P.nsplit);
  const int bj = (int)(blockIdx.x / P.nsplit), b = bj / P.hk, j = bj - b * P.hk;
  const int rows = P.Sq * P.G;
  const int64_t kst = P.k_st.token * kGroups, vst = P.v_st.token * kGroups;
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0) cross::check_len(P.kv_len, b, P.Sk, P.status);
  const int len = cross::batch_len(P.kv_len, b, P.Sk);
  const int u0 = (int)((long)len * sp / P.nsplit), u1 = (int)((long)len * (sp + 1) / P.nsplit);
  const T *k = static_cast<const T *>(P.k) + b * P.k_st.batch + j * P.k_st.head + lane * kCols;
  const T *v = static_cast<const T *>(P.v) + b * P.v_st.batch + j * P.v_st.head + lane * kCols;
  uint64_t q[kR][kPairs], own[kR][kPairs], other[kR][kPairs];  // O of this lane's map, the other's
  float m[kR], l[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int t = r / P.G, hh = j * P.G + r - t * P.G;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows)
      w = *reinterpret_cast<const uint4 *>(static_cast<const T *>(P.q) + b * P.q_st.batch +
                                           t * P.q_st.token + hh * P.q_st.head + lane * kCols);
    widen(w, q[r], T());
    const uint64_t s2 = f2(P.scale_log2, P.scale_log2);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      q[r][i] = mul2(q[r][i], s2);  // scores come in base 2
      own[r][i] = other[r][i] = 0ull;
    }
    m[r] = -FLT_MAX;
    l[r] = 0.f;
  }
  constexpr int kStep = kGroups * kAhead;
  const int steps = (u1 - u0 + kStep - 1) / kStep;
  const T *kn = k + (int64_t)(u0 + group) * P.k_st.token;  // of the next step to be copied
  const T *vn = v + (int64_t)(u0 + group) * P.v_st.token;
  int ask = 0;
  auto request = [&]() {
    uint4 *to = ring + (ask % kDepth) * 2 * kAhead * 256 + tid;
    const int u = u0 + group + ask * kStep;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const bool on = u + a * kGroups < u1;
      copy16(to + a * 256, on ? kn + a * kst : k, on);
      copy16(to + (kAhead + a) * 256, on ? vn + a * vst : v, on);
    }
    kn += kAhead * kst;
    vn += kAhead * vst;
    ++ask;
  };
  // Step i: kAhead states of every group; kFull: all of them are there.
  auto step = [&](int i, auto full) {
    constexpr bool kFull = decltype(full)::value;
    const int u = u0 + i * kStep + group;
    uint4 kr[kAhead], vr[kAhead];
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    const uint4 *from = ring + (i % kDepth) * 2 * kAhead * 256 + tid;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) kr[a] = from[a * 256];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) vr[a] = from[(kAhead + a) * 256];
    // the pieces are in registers (this thread's, whose places these are)
    asm volatile("" ::"r"(kr[kAhead - 1].w), "r"(vr[kAhead - 1].w) : "memory");
    if (ask < steps) request();
    asm volatile("cp.async.commit_group;" ::: "memory");
    float s[kAhead][kR];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      uint64_t kk[kPairs];
      widen(kr[a], kk, T());
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        uint64_t t = mul2(q[r][0], kk[0]);
#pragma unroll
        for (int i = 1; i < kPairs; ++i) t = fma2(q[r][i], kk[i], t);
        float x, y;
        unf2(t, x, y);
        s[a][r] = x + y;
      }
    }
#pragma unroll
    for (int o = kHalf / 2; o; o >>= 1)
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
#pragma unroll
        for (int r = 0; r < kR; ++r) s[a][r] += __shfl_xor_sync(0xffffffffu, s[a][r], o);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float top = m[r];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (kFull || u + a * kGroups < u1) top = fmaxf(top, s[a][r]);
      // the maximum rises seldom: O is scaled only where it does in a lane of the warp
      if (__any_sync(0xffffffffu, top > m[r])) {
        const float by = tc::ex2(m[r] - top), by_other = __shfl_xor_sync(0xffffffffu, by, kHalf);
        m[r] = top;
        l[r] *= by;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          own[r][i] = mul2(own[r][i], f2(by, by));
          other[r][i] = mul2(other[r][i], f2(by_other, by_other));
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        s[a][r] = kFull || u + a * kGroups < u1 ? tc::ex2(s[a][r] - top) : 0.f;
        l[r] += s[a][r];
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      uint64_t vv[kPairs];
      widen(vr[a], vv, T());
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const float p = s[a][r], p_other = __shfl_xor_sync(0xffffffffu, p, kHalf);
        const uint64_t p2 = f2(p, p), p2_other = f2(p_other, p_other);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          own[r][i] = fma2(p2, vv[i], own[r][i]);
          other[r][i] = fma2(p2_other, vv[i], other[r][i]);
        }
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    if (i < steps) request();
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    if (u0 + (i + 1) * kStep <= u1)
      step(i, std::true_type());
    else
      step(i, std::false_type());
  }
  // the groups' sums of a row, scaled to their common maximum
  if (lane % kHalf == 0)
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      ml[group][second][r][0] = m[r];
      ml[group][second][r][1] = l[r];
    }
  __syncthreads();
  if (tid < 2 * kR) {
    const int map = tid / kR, r = tid % kR;
    float top = -FLT_MAX, sum = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) top = fmaxf(top, ml[g][map][r][0]);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float w = tc::ex2(ml[g][map][r][0] - top);
      sum = fmaf(ml[g][map][r][1], w, sum);
      ml[g][map][r][0] = w;
    }
    total[map][r][0] = top;
    total[map][r][1] = sum;
  }
  __syncthreads();
  const size_t all = (size_t)P.B * P.h * P.Sq;
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      const float w = ml[group][map][r][0];
      float *to = sums + ((r * kGroups + group) * 2 + map) * (D + 4) + lane * kCols;
#pragma unroll
      for (int i = 0; i < kPairs; i += 2) {
        float4 x;
        unf2(mul2((map == 1) == second ? own[r][i] : other[r][i], f2(w, w)), x.x, x.y);
        unf2(mul2((map == 1) == second ? own[r][i + 1] : other[r][i + 1], f2(w, w)), x.z, x.w);
        *reinterpret_cast<float4 *>(to + 2 * i) = x;
      }
    }
  __syncthreads();
  auto place = [&](int r, int &hh, int &t) {
    t = r / P.G;
    hh = j * P.G + r - t * P.G;
    return ((size_t)b * P.h + hh) * P.Sq + t;
  };
  if (tid < 2 * rows) {
    const int map = tid & 1, r = tid >> 1;
    int hh, t;
    const size_t row = place(r, hh, t);
    const float s = total[map][r][1];
    const float lse = s > 0.f ? total[map][r][0] + log2f(s) : s == 0.f ? -INFINITY : s;
    if (P.nsplit > 1)
      P.plse[((size_t)sp * 2 + map) * all + row] = lse;
    else if (P.lse)
      P.lse[(((size_t)b * P.h + hh) * 2 + map) * P.Sq + t] = lse;
  }
  for (int e = tid; e < rows * (D / 4); e += 256) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    float4 o[2];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float4 y = *reinterpret_cast<const float4 *>(
            sums + ((r * kGroups + g) * 2 + map) * (D + 4) + c);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      const float sum = total[map][r][1], inv = sum > 0.f ? 1.0f / sum : sum;
      o[map] = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    }
    int hh, t;
    const size_t row = place(r, hh, t);
    if (P.nsplit > 1) {
      if (u0 < u1) {  // (a run without states is not read)
        float *po = P.po + ((size_t)sp * 2 * all + row) * D + c;
        put(po, o[0]);
        put(po + all * D, o[1]);
      }
      continue;
    }
    const float lam = P.lam[hh * P.lam_step];
    const size_t to = (((size_t)b * P.Sq + t) * P.h + hh) * D + c;
    put(static_cast<T *>(P.o) + to,
        make_float4(fmaf(-lam, o[1].x, o[0].x), fmaf(-lam, o[1].y, o[0].y),
                    fmaf(-lam, o[1].z, o[0].z), fmaf(-lam, o[1].w, o[0].w)));
    if (P.o2) put(static_cast<T *>(P.o2) + to, o[1]);
  }
}

template <typename T, int D, int kR>
cudaError_t launch_few(const FewParams &p, cudaStream_t st) {
  auto kern = diff_few_kernel<T, D, kR>;
  constexpr int smem = few_smem<T, D, kR>();
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)((long)p.B * p.hk * p.nsplit)), dim3(256), smem, st, p);
}

template <int D>
cudaError_t launch_rows(const FewParams &p, cudaStream_t st) {  // fp32
  const int rows = p.Sq * p.G;
  return rows == 1   ? launch_few<float, D, 1>(p, st)
         : rows == 2 ? launch_few<float, D, 2>(p, st)
         : rows == 3 ? launch_few<float, D, 3>(p, st)
                     : launch_few<float, D, 4>(p, st);
}

}  // namespace

// fp32: up to four rows (24 heads on 8, 16 x 1000 states: 29 us, 118 in the general form).
// bf16: a single row; the tensor cores' form takes two and more in the time of one, and its
// pieces are equal (D 128, us here and there: 1 row, 1 x 8192 states, 8 heads 21, 28; 16 x 1000,
// 16 heads 21, 23; 4 x 100 3.7, 5.8; 3 rows, 16 x 4096, 24 heads 56, 44; 16 x 128 8.0, 7.1).
bool diff_few_rows(const CrossShape &s, nabla_dtype dt) {
  return (long)s.Sq * (s.h / s.hk) <= (dt == NABLA_F32 ? 4 : 1);
}

cudaError_t launch_diff_few(const DiffArgs &a, nabla_dtype dt, cudaStream_t st) {
  const CrossShape &s = a.x.s;
  FewParams p{};
  p.q = a.x.q, p.k = a.x.k, p.v = a.x.v;
  p.q_st = a.x.q_st, p.k_st = a.x.k_st, p.v_st = a.x.v_st;
  p.lam = a.lam, p.lam_step = a.lam_n > 1 ? 1 : 0;
  p.kv_len = a.x.kv_len;
  p.o = a.x.o, p.o2 = a.o2, p.lse = a.x.lse;
  p.B = s.B, p.Sq = s.Sq, p.Sk = s.Sk, p.h = s.h, p.hk = s.hk, p.G = s.h / s.hk;
  p.scale_log2 = a.x.scale * 1.4426950408889634f;
  p.status = a.x.status;
  const DiffRuns runs = diff_runs(a, dt);
  p.nsplit = runs.runs, p.po = runs.po, p.plse = runs.plse;
  cudaError_t e;
  if (dt == NABLA_BF16)
    e = s.D == 64 ? launch_few<__nv_bfloat16, 64, 1>(p, st)
                  : launch_few<__nv_bfloat16, 128, 1>(p, st);
  else
    e = s.D == 64 ? launch_rows<64>(p, st) : launch_rows<128>(p, st);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  return launch_diff_join(a, dt, runs, st);
}

}  // namespace nabla
