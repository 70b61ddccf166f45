// K12s -- differential attention forward of few rows: up to eight packed rows a key head in
// bf16, up to four in fp32, as a step that asks for one token has them.  Bound by the bytes of
// K and V: every warp or group of lanes walks its own states with its own running maxima and
// sums and no barrier but at the end, its tiles coming by asynchronous copies into places of
// its own in shared memory, three ahead, 190 KB under way on an SM.  The warps of a CTA are
// joined in shared memory, CTAs (runs of a batch's states) by diff_join.
//
// bf16: a warp takes tiles of 16 states.  They are the rows of its tensor instructions and the
// query rows their eight columns, S_m^T = K_m Q_m^T and O_m^T += V^T P_m^T, so that a tile is
// 24 instructions and nothing is padded to the 128 rows of a tcgen05 tile, whose step takes 0.6
// us whatever the rows.  One token of 24 heads on 8, 16 ragged batches of up to 4096 states: 32
// us, 4.3 TB/s, where the tcgen05 kernel takes 42; 16 heads, 64 x 4096 states 302 us, 7.1 TB/s;
// 1 x 8192 states 11 us.
//
// fp32: D columns of a state lie over the lanes of a group, 16 bytes a lane, the first half of
// the lanes holding map 1's columns of K, the others map 2's.  Scores: products of the lane's
// columns, added up over the half group; then every lane has its own map's P, takes the
// other's from the other half, and adds both times its columns of V.
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
__device__ __forceinline__ void widen(const uint4 &r, uint64_t (&v)[2]) {
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

template <int D, int kR>
constexpr int few_smem() {
  constexpr int groups = 256 / (D / 4);
  constexpr int copies = kDepth * 2 * kAhead * 256 * 16, sums = kR * groups * 2 * (D + 4) * 4;
  return copies > sums ? copies : sums;
}

__device__ __forceinline__ void copy16(uint4 *to, const void *from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(to)), "l"(from),
               "r"(on ? 16 : 0)
               : "memory");
}

// The rows' results out of a CTA, from their maxima and sums `total` and the sums of P V that
// at(row, map, column) gives; `some`: its run has states.
template <typename T, int D, int kR, int kThreads, class At>
__device__ __forceinline__ void store_rows(const FewParams &P, const float (&total)[2][kR][2],
                                           int sp, int b, int j, bool some, const At &at) {
  const int tid = threadIdx.x, rows = P.Sq * P.G;
  const size_t all = (size_t)P.B * P.h * P.Sq;
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
  for (int e = tid; e < rows * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    float4 o[2];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      const float4 x = at(r, map, c);
      const float sum = total[map][r][1], inv = sum > 0.f ? 1.0f / sum : sum;
      o[map] = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    }
    int hh, t;
    const size_t row = place(r, hh, t);
    if (P.nsplit > 1) {
      if (some) {  // (a run without states is not read)
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

// CTA: run `sp` of the states of batch b and key head j; kR: rows at most.
template <int D, int kR>
__global__ void __launch_bounds__(256, kR == 4 ? 1 : 2)
    diff_few_kernel(const __grid_constant__ FewParams P) {
  using T = float;
  constexpr int kCols = 4, kPairs = 2;                   // columns a lane
  constexpr int kLanes = D / kCols, kHalf = kLanes / 2;  // of a group, of a map's half
  constexpr int kGroups = 256 / kLanes;
  __shared__ float ml[kGroups][2][kR][2];                // maximum and sum
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
    widen(w, q[r]);
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
      widen(kr[a], kk);
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
      widen(vr[a], vv);
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
  store_rows<T, D, kR, 256>(P, total, sp, b, j, u0 < u1, [&](int r, int map, int c) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float4 y = *reinterpret_cast<const float4 *>(
          sums + ((r * kGroups + g) * 2 + map) * (D + 4) + c);
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    return x;
  });
}

// ---- bf16, up to eight rows: states along the tensor instructions' 16 rows, the query rows
// along their 8 columns.

constexpr int kRows = 8, kRowWarps = 4, kTile = 16;

template <int D>
struct RCfg {
  static constexpr int kBytes = kTile * D * 2;         // of K's or V's tile
  static constexpr int kDepth = D == 128 ? 3 : 6;      // tiles copied ahead by a warp
  static constexpr int kWarp = kDepth * 2 * kBytes;    // of shared memory
  static constexpr int kSmem = kRowWarps * kWarp;
  static_assert(kWarp >= 2 * kRows * (D + 4) * 4, "the warp's sums take its copies' place");
};

__device__ __forceinline__ void ldmatrix(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // of 8 x 8
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// c += a b, 16 x 8 by a depth of 16.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// CTA: run `sp` of the states of batch b and key head j.  A warp takes every fourth tile of
// 16 states, with its own maxima and sums: S_m^T = K_m Q_m^T, O_m^T += V^T P_m^T.
template <int D>
__global__ void __launch_bounds__(kRowWarps * 32, 2)
    diff_rows_kernel(const __grid_constant__ FewParams P) {
  using C = RCfg<D>;
  using T = __nv_bfloat16;
  constexpr int kSteps = D / 32, kCols = D / 16;  // depth of a map's scores, 16 columns of V
  __shared__ float ml[kRowWarps][2][kRows][2], total[2][kRows][2];
  extern __shared__ __align__(16) uint8_t rows_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = lane & 3, g8 = lane >> 2;
  const int sp = (int)(blockIdx.x % P.nsplit);
  const int bj = (int)(blockIdx.x / P.nsplit), b = bj / P.hk, j = bj - b * P.hk;
  const int rows = P.Sq * P.G;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) cross::check_len(P.kv_len, b, P.Sk, P.status);
  const int len = cross::batch_len(P.kv_len, b, P.Sk);
  const int u0 = (int)((long)len * sp / P.nsplit), u1 = (int)((long)len * (sp + 1) / P.nsplit);
  uint8_t *ring = rows_smem + warp * C::kWarp;
  // copies: 16 bytes a lane, a state's D columns by D / 8 lanes; a tile's pieces are swizzled
  // by their state, so that eight states' pieces of the same columns lie in different banks
  constexpr int kPieces = D / 8, kLoads = kTile * kPieces / 32, kStride = 32 / kPieces;
  const int cs = lane / kPieces, cp = lane % kPieces;  // state and piece of this lane's first
  const T *k = static_cast<const T *>(P.k) + b * P.k_st.batch + j * P.k_st.head + cp * 8;
  const T *v = static_cast<const T *>(P.v) + b * P.v_st.batch + j * P.v_st.head + cp * 8;
  const int tiles = (u1 - u0 + kTile - 1) / kTile;
  const int steps = tiles > warp ? (tiles - warp + kRowWarps - 1) / kRowWarps : 0;
  auto request = [&](int i) {
    const int u = u0 + (i * kRowWarps + warp) * kTile + cs;
    uint8_t *to = ring + (i % C::kDepth) * 2 * C::kBytes;
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int s = cs + x * kStride;
      const bool on = u + x * kStride < u1;
      const int64_t at = on ? u + x * kStride : 0;
      const int off = s * (D * 2) + ((cp ^ (s & 7)) << 4);
      copy16(reinterpret_cast<uint4 *>(to + off), k + at * P.k_st.token, on);
      copy16(reinterpret_cast<uint4 *>(to + C::kBytes + off), v + at * P.v_st.token, on);
    }
  };
#pragma unroll
  for (int i = 0; i < C::kDepth; ++i) {
    if (i < steps) request(i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Q^T: this lane's columns 16 x + 2 q4 (+ 8) of row g8
  uint32_t q[kCols][2];
  {
    const int t = g8 / P.G, hh = j * P.G + g8 - t * P.G;
    const T *from = static_cast<const T *>(P.q) + b * P.q_st.batch + t * P.q_st.token +
                    hh * P.q_st.head + 2 * q4;
#pragma unroll
    for (int x = 0; x < kCols; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        q[x][i] = g8 < rows ? *reinterpret_cast<const uint32_t *>(from + 16 * x + 8 * i) : 0u;
  }
  float o[2][kCols][4], m[2][2], l[2][2];
#pragma unroll
  for (int map = 0; map < 2; ++map) {
#pragma unroll
    for (int x = 0; x < kCols; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[map][x][i] = 0.f;
    m[map][0] = m[map][1] = -FLT_MAX;
    l[map][0] = l[map][1] = 0.f;
  }
  // this lane's row of ldmatrix's four 8 x 8 pieces: K's in the order of the product's rows
  // first, V's (transposed) in that of its columns
  const int mi = lane >> 3, ri = lane & 7;
  const uint32_t ring_at = tc::smem_u32(ring);
  const uint32_t k_row = (uint32_t)(ri + (mi & 1) * 8) * (D * 2), k_piece = (uint32_t)mi >> 1;
  const uint32_t v_row = (uint32_t)(ri + (mi >> 1) * 8) * (D * 2), v_piece = (uint32_t)mi & 1;
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::kDepth - 1) : "memory");
    __syncwarp();
    const uint32_t at = ring_at + (uint32_t)(i % C::kDepth) * 2 * C::kBytes;
    const int u = u0 + (i * kRowWarps + warp) * kTile + g8;
    uint32_t pt[2][2];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = map * kSteps; x < (map + 1) * kSteps; ++x) {
        uint32_t a[4];
        ldmatrix(at + k_row + (((2 * x + k_piece) ^ (uint32_t)ri) << 4), a);
        mma16(s, a, q[x][0], q[x][1]);
      }
      // states u and u + 8, rows 2 q4 and the next
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[e] = u + (e >> 1) * 8 < u1 ? s[e] * P.scale_log2 : -INFINITY;
      float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
      // the maximum is only the exponents' bias: it is raised where a P would pass 2^8
      if (__any_sync(0xffffffffu, top[0] > m[map][0] + 8.f || top[1] > m[map][1] + 8.f)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2)
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], d));
          top[e] = fmaxf(top[e], m[map][e]);
          const float by = tc::ex2(m[map][e] - top[e]);
          m[map][e] = top[e];
          l[map][e] *= by;
#pragma unroll
          for (int x = 0; x < kCols; ++x) {
            o[map][x][e] *= by;
            o[map][x][e + 2] *= by;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] = tc::ex2(s[e] - m[map][e & 1]);
        l[map][e & 1] += s[e];
      }
      pt[map][0] = transposed(tc::pack_bf16x2(s[0], s[1]));
      pt[map][1] = transposed(tc::pack_bf16x2(s[2], s[3]));
    }
#pragma unroll
    for (int x = 0; x < kCols; ++x) {
      uint32_t a[4];
      ldmatrix_trans(at + C::kBytes + v_row + (((2 * x + v_piece) ^ (uint32_t)ri) << 4), a);
      mma16(o[0][x], a, pt[0][0], pt[0][1]);
      mma16(o[1][x], a, pt[1][0], pt[1][1]);
    }
    __syncwarp();  // the tile has been read
    if (i + C::kDepth < steps) request(i + C::kDepth);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the warps' sums, [map][row][D + 4] in the place of their copies
  float *sums = reinterpret_cast<float *>(ring);
  constexpr int LD = D + 4;
#pragma unroll
  for (int map = 0; map < 2; ++map) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[map][e] += __shfl_xor_sync(0xffffffffu, l[map][e], d);
      if (g8 == 0) {
        ml[warp][map][2 * q4 + e][0] = m[map][e];
        ml[warp][map][2 * q4 + e][1] = l[map][e];
      }
    }
#pragma unroll
    for (int x = 0; x < kCols; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sums[(map * kRows + 2 * q4 + (e & 1)) * LD + 16 * x + g8 + (e >> 1) * 8] = o[map][x][e];
  }
  __syncthreads();
  if (threadIdx.x < 2 * kRows) {
    const int map = threadIdx.x / kRows, r = threadIdx.x % kRows;
    float top = -FLT_MAX, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, ml[w][map][r][0]);
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      const float by = tc::ex2(ml[w][map][r][0] - top);
      sum = fmaf(ml[w][map][r][1], by, sum);
      ml[w][map][r][0] = by;
    }
    total[map][r][0] = top;
    total[map][r][1] = sum;
  }
  __syncthreads();
  store_rows<T, D, kRows, kRowWarps * 32>(P, total, sp, b, j, u0 < u1, [&](int r, int map, int c) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      const float by = ml[w][map][r][0];
      const float4 y = *reinterpret_cast<const float4 *>(rows_smem + w * C::kWarp +
                                                         ((map * kRows + r) * LD + c) * 4);
      x.x = fmaf(by, y.x, x.x), x.y = fmaf(by, y.y, x.y);
      x.z = fmaf(by, y.z, x.z), x.w = fmaf(by, y.w, x.w);
    }
    return x;
  });
}

template <int D>
cudaError_t launch_bf16(const FewParams &p, cudaStream_t st) {
  auto kern = diff_rows_kernel<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)((long)p.B * p.hk * p.nsplit)), dim3(kRowWarps * 32),
                    RCfg<D>::kSmem, st, p);
}

template <int D, int kR>
cudaError_t launch_few(const FewParams &p, cudaStream_t st) {
  auto kern = diff_few_kernel<D, kR>;
  constexpr int smem = few_smem<D, kR>();
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)((long)p.B * p.hk * p.nsplit)), dim3(256), smem, st, p);
}

template <int D>
cudaError_t launch_rows(const FewParams &p, cudaStream_t st) {  // fp32
  const int rows = p.Sq * p.G;
  return rows == 1   ? launch_few<D, 1>(p, st)
         : rows == 2 ? launch_few<D, 2>(p, st)
         : rows == 3 ? launch_few<D, 3>(p, st)
                     : launch_few<D, 4>(p, st);
}

}  // namespace

// fp32: up to four rows (24 heads on 8, 16 x 1000 states: 29 us, 118 in the general form).
// bf16: as many as a tensor instruction has columns (eight tokens, 2 x 4096 states, 8 heads:
// 12 us, the tcgen05 kernel 21).
bool diff_few_rows(const CrossShape &s, nabla_dtype dt) {
  return (long)s.Sq * (s.h / s.hk) <= (dt == NABLA_F32 ? 4 : 8);
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
    e = s.D == 64 ? launch_bf16<64>(p, st) : launch_bf16<128>(p, st);
  else
    e = s.D == 64 ? launch_rows<64>(p, st) : launch_rows<128>(p, st);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  return launch_diff_join(a, dt, runs, st);
}

}  // namespace nabla
