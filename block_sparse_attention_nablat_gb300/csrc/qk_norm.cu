// K8 -- RMS norm of queries and keys per head with the position rotation in the
// same pass, and its gradient.
//
// A row x (one head of one token, D columns) becomes z = Rot(y), y = w x r with
// r = 1 / sqrt(mean(x^2) + eps); Rot turns the first R columns in pairs (a, b) ->
// (a c - b s, a s + b c) by the token's angles.  With dy = Rot^T dz and g = w dy:
//   dx = r (g - x r^2 mean(g x)),   dw = sum over all rows of dy x r.
// Everything between the load and the one rounding at the store is fp32.
//
// HBM-bound: a row is read once and written once (backward: x and dz read, dx
// written).  A lane holds 8 adjacent columns (one 16-byte load of bf16), D / 8
// lanes hold a row and a warp 32 / (D / 8) rows at a time, so the norm's sum is
// log2(D / 8) shuffles and no shared memory is touched.  A warp's item is a run of
// one token's heads, so the token's angles and the weights are read once per item
// and stay in registers.  At 32768 tokens, 24 + 24 heads, D 128, bf16: 123 us, 6.6 TB/s
// of rows read and written (97% of a plain copy's rate); backward 208 us, 5.8 TB/s (86%:
// its 128 registers a thread leave fewer loads in flight).  The backward's warps step over
// items by an even number, so one only ever gets q's or k's: with 32 + 4 heads of 64 (4 x 6483
// tokens) the warps of the k side are done early, and it takes 98 us of 53.
#include <cuda_bf16.h>

#include "internal.h"
#include "pdl.cuh"
#include "vec8.cuh"

namespace nabla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Weights of this lane's columns (1 where the caller gave none).
__device__ __forceinline__ void load_weight(const void *w, nabla_dtype wdt, int col,
                                            float (&v)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
  } else if (wdt == NABLA_BF16) {
    load8(static_cast<const __nv_bfloat16 *>(w) + col, v);
  } else {
    load8(static_cast<const float *>(w) + col, v);
  }
}

// The rotation of one lane's 8 columns.  Pairs: c[j], s[j] (j < 4) turn columns 2j
// and 2j + 1.  Halves: column j of this lane pairs with column j of lane `partner`
// (R / 2 columns on), and the sign of the second product is folded into s.  Lanes
// beyond R keep c = 1, s = 0, with themselves as partner.  R is a multiple of 16, so
// a lane lies wholly in the first half, the second half or beyond.
struct Turn {
  float c[8], s[8];
  int partner;
};

template <bool kPairs>
__device__ __forceinline__ Turn load_turn(const float *cos_t, const float *sin_t, long at, int R,
                                          int col, int lane, bool on) {
  Turn t;
  t.partner = lane;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    t.c[j] = 1.f;
    t.s[j] = 0.f;
  }
  const int half = R >> 1;
  if (!kPairs && col < R) t.partner = col < half ? lane + (half >> 3) : lane - (half >> 3);
  if (!on || col >= R) return t;
  if (kPairs) {
    const float4 c = *reinterpret_cast<const float4 *>(cos_t + at * half + (col >> 1));
    const float4 s = *reinterpret_cast<const float4 *>(sin_t + at * half + (col >> 1));
    t.c[0] = c.x, t.c[1] = c.y, t.c[2] = c.z, t.c[3] = c.w;
    t.s[0] = s.x, t.s[1] = s.y, t.s[2] = s.z, t.s[3] = s.w;
  } else {
    const bool second = col >= half;
    const long i = at * half + (second ? col - half : col);
    load8(cos_t + i, t.c);
    load8(sin_t + i, t.s);
    if (!second)
#pragma unroll
      for (int j = 0; j < 8; ++j) t.s[j] = -t.s[j];
  }
  return t;
}

// kBack: the transpose (the angles negated).
template <bool kPairs, bool kBack>
__device__ __forceinline__ void turn8(float (&y)[8], const Turn &t) {
  if (kPairs) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = y[2 * j], b = y[2 * j + 1], s = kBack ? -t.s[j] : t.s[j];
      y[2 * j] = fmaf(a, t.c[j], -(b * s));
      y[2 * j + 1] = fmaf(a, s, b * t.c[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float o = __shfl_sync(0xffffffffu, y[j], t.partner);
      y[j] = fmaf(y[j], t.c[j], o * (kBack ? -t.s[j] : t.s[j]));
    }
  }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Side {  // q or k
  const void *x, *dz;
  void *out;  // z, or dx
  const void *w;
  nabla_strides x_st, z_st, o_st;  // of x, dz and out
  int h, chunks;                   // heads, items per token (few heads: tokens per item)
};

struct QkParams {
  Side side[2];
  nabla_dtype wdt;
  const float *cos_t, *sin_t;
  const int32_t *pos;
  long tokens, items;  // B * S; tokens * (chunks of both sides)
  long first;          // few heads: items of q, the first ones
  int S, rows, R, heads_per_item;
  float eps;
  float *partial;  // backward: [grid][2][D] column sums
  int *status;
};

struct Item {
  int side, h0, h1;
  long b, s, at;
  bool turn;
};

// The item's token, its run of heads and its row of the rotation table.
__device__ __forceinline__ Item decode_item(const QkParams &P, long i) {
  const int per = P.side[0].chunks + P.side[1].chunks;
  const long t = i / per;
  int c = (int)(i - t * per);
  Item it;
  it.side = c >= P.side[0].chunks;
  if (it.side) c -= P.side[0].chunks;
  it.h0 = c * P.heads_per_item;
  it.h1 = min(it.h0 + P.heads_per_item, P.side[it.side].h);
  it.b = t / P.S;
  it.s = t - it.b * P.S;
  it.at = P.pos && P.R ? P.pos[t] : it.s;
  it.turn = P.R > 0;
  if (P.pos && P.R && (it.at < 0 || it.at >= P.rows)) {  // normed, not rotated, and reported
    if ((threadIdx.x & 31) == 0) atomicCAS(P.status, kDevOk, kDevBadIndex);
    it.turn = false;
  }
  return it;
}

// kDense: every tensor's heads lie D apart, so a row's place is an immediate offset from
// the item's first (with strides in registers instead the backward took 336 us where this
// one took 237 then, 32768 tokens, 24 + 24 heads, D 128).
template <typename T, int D, bool kPairs, bool kDense>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const __grid_constant__ QkParams P) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAhead = 4;
  const int lane = threadIdx.x & 31, col = (lane % kLanes) * 8, sub = lane / kLanes;
  pdl_launch_dependents();
  pdl_wait();
  const long stride = (long)gridDim.x * kWarps;
  for (long i = (long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < P.items; i += stride) {
    const Item it = decode_item(P, i);
    const Side &sd = P.side[it.side];
    const int64_t xh = kDense ? D : sd.x_st.head, oh = kDense ? D : sd.o_st.head;
    const T *x = static_cast<const T *>(sd.x) + it.b * sd.x_st.batch + it.s * sd.x_st.token +
                 (it.h0 + sub) * xh + col;
    T *o = static_cast<T *>(sd.out) + it.b * sd.o_st.batch + it.s * sd.o_st.token +
           (it.h0 + sub) * oh + col;
    float w[8];
    load_weight(sd.w, P.wdt, col, w);
    const Turn t = load_turn<kPairs>(P.cos_t, P.sin_t, it.at, P.R, col, lane, it.turn);
    for (int hb = it.h0; hb < it.h1; hb += kRows * kAhead) {
      Raw<T> in[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        in[a] = load_raw(x + a * kRows * xh, hb + a * kRows + sub < it.h1);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (hb + a * kRows >= it.h1) break;  // the same for the whole warp
        float y[8], ss = 0.f;
        unpack8(in[a], y);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
        const float r = rsqrtf(fmaf(row_sum<kLanes>(ss), 1.f / D, P.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= r * w[j];
        turn8<kPairs, false>(y, t);
        if (hb + a * kRows + sub < it.h1) store8(o + a * kRows * oh, y);
      }
      x += kRows * kAhead * xh;
      o += kRows * kAhead * oh;
    }
  }
}

// A block's sums of dy x r, its warps' added in order, to its row of `partial`.
template <int D>
__device__ __forceinline__ void put_sums(const float (&acc)[2][8], float (*sums)[2 * D],
                                         float *partial) {
  constexpr int kLanes = D / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = (lane % kLanes) * 8, sub = lane / kLanes;
  if (!partial) return;
#pragma unroll
  for (int sd = 0; sd < 2; ++sd)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = acc[sd][j];
#pragma unroll
      for (int o = 16; o >= kLanes; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (sub == 0) sums[warp][sd * D + col + j] = v;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += sums[k][c];
    partial[(size_t)blockIdx.x * 2 * D + c] = v;
  }
}

// dx row by row as above; every warp keeps the column sums of dy x r of both sides
// in registers over all its items, the block joins its warps' sums in a fixed order
// and writes one row per block, and qk_dw_kernel adds the rows.  Items are dealt out
// by index alone, so dw is the same from run to run.
template <typename T, int D, bool kPairs, bool kDense>
__global__ void __launch_bounds__(kThreads)
    qk_norm_bwd_kernel(const __grid_constant__ QkParams P) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAhead = sizeof(T) == 2 ? 4 : 2;
  __shared__ float sums[kWarps][2 * D];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31, col = (lane % kLanes) * 8, sub = lane / kLanes;
  pdl_launch_dependents();
  pdl_wait();
  float acc[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[0][j] = acc[1][j] = 0.f;
  const long stride = (long)gridDim.x * kWarps;
  for (long i = (long)blockIdx.x * kWarps + warp; i < P.items; i += stride) {
    const Item it = decode_item(P, i);
    const Side &sd = P.side[it.side];
    const int64_t xh = kDense ? D : sd.x_st.head, zh = kDense ? D : sd.z_st.head,
                  oh = kDense ? D : sd.o_st.head;
    const T *x = static_cast<const T *>(sd.x) + it.b * sd.x_st.batch + it.s * sd.x_st.token +
                 (it.h0 + sub) * xh + col;
    const T *dz = static_cast<const T *>(sd.dz) + it.b * sd.z_st.batch + it.s * sd.z_st.token +
                  (it.h0 + sub) * zh + col;
    T *o = static_cast<T *>(sd.out) + it.b * sd.o_st.batch + it.s * sd.o_st.token +
           (it.h0 + sub) * oh + col;
    float w[8], part[8];
    load_weight(sd.w, P.wdt, col, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) part[j] = 0.f;
    const Turn t = load_turn<kPairs>(P.cos_t, P.sin_t, it.at, P.R, col, lane, it.turn);
    for (int hb = it.h0; hb < it.h1; hb += kRows * kAhead) {
      Raw<T> xin[kAhead], zin[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const bool on = hb + a * kRows + sub < it.h1;
        xin[a] = load_raw(x + a * kRows * xh, on);
        zin[a] = load_raw(dz + a * kRows * zh, on);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (hb + a * kRows >= it.h1) break;  // the same for the whole warp
        float xv[8], g[8], ss = 0.f, dot = 0.f;
        unpack8(xin[a], xv);
        unpack8(zin[a], g);
        turn8<kPairs, true>(g, t);  // dy
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(xv[j], xv[j], ss);
          dot = fmaf(g[j] * w[j], xv[j], dot);
        }
        const float r = rsqrtf(fmaf(row_sum<kLanes>(ss), 1.f / D, P.eps));
        const float m = row_sum<kLanes>(dot) * (1.f / D) * r * r;
        const bool on = hb + a * kRows + sub < it.h1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (on) part[j] = fmaf(g[j] * r, xv[j], part[j]);
          g[j] = r * fmaf(-xv[j], m, g[j] * w[j]);
        }
        if (on) store8(o + a * kRows * oh, g);
      }
      x += kRows * kAhead * xh;
      dz += kRows * kAhead * zh;
      o += kRows * kAhead * oh;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[0][j] += it.side ? 0.f : part[j];
      acc[1][j] += it.side ? part[j] : 0.f;
    }
  }
  put_sums<D>(acc, sums, P.partial);
}

// The same for few heads, where one token's rows would leave most of a warp's loads unused:
// an item is a run of tokens whose rows one pass of the warp takes, each with its own
// angles.
struct FewItem {
  int side, rows;   // rows of the run
  long t0, b0, s0;  // its first token
};
__device__ __forceinline__ FewItem few_item(const QkParams &P, long i) {
  FewItem it;
  it.side = i >= P.first;
  const Side &sd = P.side[it.side];
  it.t0 = (it.side ? i - P.first : i) * sd.chunks;
  it.rows = (int)min((long)sd.chunks, P.tokens - it.t0) * sd.h;
  it.b0 = it.t0 / P.S;
  it.s0 = it.t0 - it.b0 * P.S;
  return it;
}
struct FewRow {
  long b, s, at;
  int head;
  bool on, turn;
};
__device__ __forceinline__ FewRow few_row(const QkParams &P, const FewItem &it, int r, bool lead) {
  const uint32_t h = (uint32_t)P.side[it.side].h, dt = (uint32_t)r / h;
  FewRow w;
  w.on = r < it.rows;
  w.head = r - (int)(dt * h);
  const uint32_t st = (uint32_t)it.s0 + dt, db = st / (uint32_t)P.S;
  w.b = it.b0 + db;
  w.s = st - db * (uint32_t)P.S;
  w.at = w.s;
  w.turn = w.on && P.R > 0;
  if (w.turn && P.pos) {
    w.at = P.pos[it.t0 + dt];
    if (w.at < 0 || w.at >= P.rows) {  // normed, not rotated, and reported
      if (lead) atomicCAS(P.status, kDevOk, kDevBadIndex);
      w.turn = false;
    }
  }
  return w;
}
__device__ __forceinline__ int64_t row_at(const nabla_strides &st, const FewRow &w) {
  return w.b * st.batch + w.s * st.token + w.head * st.head;
}

template <typename T, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads) qk_few_kernel(const __grid_constant__ QkParams P) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAhead = 4;
  const int lane = threadIdx.x & 31, col = (lane % kLanes) * 8, sub = lane / kLanes;
  pdl_launch_dependents();
  pdl_wait();
  const long stride = (long)gridDim.x * kWarps;
  for (long i = (long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < P.items; i += stride) {
    const FewItem it = few_item(P, i);
    const Side &sd = P.side[it.side];
    Raw<T> in[kAhead];
    Turn t[kAhead];
    T *o[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const FewRow w = few_row(P, it, a * kRows + sub, col == 0);
      in[a] = load_raw(static_cast<const T *>(sd.x) + row_at(sd.x_st, w) + col, w.on);
      t[a] = load_turn<kPairs>(P.cos_t, P.sin_t, w.at, P.R, col, lane, w.turn);
      o[a] = w.on ? static_cast<T *>(sd.out) + row_at(sd.o_st, w) + col : nullptr;
    }
    float w[8];
    load_weight(sd.w, P.wdt, col, w);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (a * kRows >= it.rows) break;  // the same for the whole warp
      float y[8], ss = 0.f;
      unpack8(in[a], y);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
      const float r = rsqrtf(fmaf(row_sum<kLanes>(ss), 1.f / D, P.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= r * w[j];
      turn8<kPairs, false>(y, t[a]);
      if (o[a]) store8(o[a], y);
    }
  }
}

template <typename T, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads) qk_few_bwd_kernel(const __grid_constant__ QkParams P) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAhead = sizeof(T) == 2 ? 4 : 2;
  __shared__ float sums[kWarps][2 * D];
  const int lane = threadIdx.x & 31, col = (lane % kLanes) * 8, sub = lane / kLanes;
  pdl_launch_dependents();
  pdl_wait();
  float acc[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[0][j] = acc[1][j] = 0.f;
  const long stride = (long)gridDim.x * kWarps;
  for (long i = (long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < P.items; i += stride) {
    const FewItem it = few_item(P, i);
    const Side &sd = P.side[it.side];
    Raw<T> xin[kAhead], zin[kAhead];
    Turn t[kAhead];
    T *o[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const FewRow w = few_row(P, it, a * kRows + sub, col == 0);
      xin[a] = load_raw(static_cast<const T *>(sd.x) + row_at(sd.x_st, w) + col, w.on);
      zin[a] = load_raw(static_cast<const T *>(sd.dz) + row_at(sd.z_st, w) + col, w.on);
      t[a] = load_turn<kPairs>(P.cos_t, P.sin_t, w.at, P.R, col, lane, w.turn);
      o[a] = w.on ? static_cast<T *>(sd.out) + row_at(sd.o_st, w) + col : nullptr;
    }
    float w[8], part[8];
    load_weight(sd.w, P.wdt, col, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) part[j] = 0.f;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (a * kRows >= it.rows) break;  // the same for the whole warp
      float xv[8], g[8], ss = 0.f, dot = 0.f;
      unpack8(xin[a], xv);
      unpack8(zin[a], g);
      turn8<kPairs, true>(g, t[a]);  // dy
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(xv[j], xv[j], ss);
        dot = fmaf(g[j] * w[j], xv[j], dot);
      }
      const float r = rsqrtf(fmaf(row_sum<kLanes>(ss), 1.f / D, P.eps));
      const float m = row_sum<kLanes>(dot) * (1.f / D) * r * r;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (o[a]) part[j] = fmaf(g[j] * r, xv[j], part[j]);
        g[j] = r * fmaf(-xv[j], m, g[j] * w[j]);
      }
      if (o[a]) store8(o[a], g);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[0][j] += it.side ? 0.f : part[j];
      acc[1][j] += it.side ? part[j] : 0.f;
    }
  }
  put_sums<D>(acc, sums, P.partial);
}

// dw: the blocks' rows added up, 32 columns a block, 32 rows at a time.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const float *__restrict__ partial, int rows,
                                                     int D, void *dwq, void *dwk,
                                                     nabla_dtype wdt) {
  __shared__ float sums[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r0 = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  float v = 0.f;
  for (int r = r0; r < rows; r += 32) v += partial[(size_t)r * 2 * D + c];
  sums[r0][threadIdx.x & 31] = v;
  __syncthreads();
  if (r0) return;
  v = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) v += sums[k][threadIdx.x];
  void *dw = c < D ? dwq : dwk;
  if (!dw) return;
  const int at = c < D ? c : c - D;
  if (wdt == NABLA_BF16)
    static_cast<__nv_bfloat16 *>(dw)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float *>(dw)[at] = v;
}

// Blocks of the backward at most: enough warps to keep HBM busy, few enough rows of
// partial sums (the workspace holds this many).
constexpr int kBwdBlocksPerSm = 4, kBwdBlocksMost = 1024;

enum Kind { kDenseHeads, kStrided, kFewHeads };

template <typename T, int D, bool kPairs>
cudaError_t launch_few(const QkParams &p, bool bwd, unsigned grid, cudaStream_t st) {
  if (bwd) return launch_pdl(qk_few_bwd_kernel<T, D, kPairs>, grid, kThreads, 0, st, p);
  return launch_pdl(qk_few_kernel<T, D, kPairs>, grid, kThreads, 0, st, p);
}

template <typename T, int D, bool kPairs, bool kDense>
cudaError_t launch_typed(const QkParams &p, bool bwd, unsigned grid, cudaStream_t st) {
  if (bwd) return launch_pdl(qk_norm_bwd_kernel<T, D, kPairs, kDense>, grid, kThreads, 0, st, p);
  return launch_pdl(qk_norm_kernel<T, D, kPairs, kDense>, grid, kThreads, 0, st, p);
}

template <typename T, int D>
cudaError_t launch_dim(const QkParams &p, bool pairs, bool bwd, Kind kind, unsigned grid,
                       cudaStream_t st) {
  if (kind == kFewHeads)
    return pairs ? launch_few<T, D, true>(p, bwd, grid, st)
                 : launch_few<T, D, false>(p, bwd, grid, st);
  if (kind == kDenseHeads)
    return pairs ? launch_typed<T, D, true, true>(p, bwd, grid, st)
                 : launch_typed<T, D, false, true>(p, bwd, grid, st);
  return pairs ? launch_typed<T, D, true, false>(p, bwd, grid, st)
               : launch_typed<T, D, false, false>(p, bwd, grid, st);
}

template <typename T>
cudaError_t launch_dtype(const QkParams &p, int D, bool pairs, bool bwd, Kind kind, unsigned grid,
                         cudaStream_t st) {
  return D == 64 ? launch_dim<T, 64>(p, pairs, bwd, kind, grid, st)
                 : launch_dim<T, 128>(p, pairs, bwd, kind, grid, st);
}

}  // namespace

size_t qk_norm_bwd_workspace(int D) {
  return (size_t)kBwdBlocksMost * 2 * D * sizeof(float);
}

cudaError_t launch_qk_norm(const QkNormArgs &a, cudaStream_t st) {
  const bool bwd = a.dz[0] != nullptr;
  QkParams p{};
  p.wdt = a.wdt;
  p.cos_t = a.cos_t;
  p.sin_t = a.sin_t;
  p.pos = a.pos;
  p.tokens = (long)a.B * a.S;
  p.S = a.S;
  p.rows = a.rope_rows;
  p.R = a.R;
  p.eps = a.eps;
  p.status = a.status;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // Heads per item: all of a token's heads of one side, or, where that leaves the GPU
  // short of warps, as few as one pass of the warp takes.
  const int pass = 32 / (a.D / 8) * (bwd && a.dt == NABLA_F32 ? 2 : 4);
  const int most = a.h[0] > a.h[1] ? a.h[0] : a.h[1];
  int hpi = most;
  if (p.tokens * 2 < (long)sms * 64) hpi = pass;
  p.heads_per_item = hpi;
  p.items = 0;
  // Few heads: runs of tokens, where several tokens' rows go into a pass: four, two where
  // there is more work to a row's angles, eight where the angles take more registers.  (D 128, forward / backward, us, as runs of
  // tokens against a token an item: 9 x 13717 tokens, 1 + 1 heads, pairs 41 / 51 against
  // 90 / 172, halves 62 / 113 against 102 / 189; 98304 tokens, 4 + 4 heads, pairs 121 / 149
  // against 101 / 189, halves 168 / 304 against 115 / 206.)
  const bool few = most * (a.interleaved ? (bwd ? 2 : 4) : 8) <= pass;
  bool dense = true;
  for (int i = 0; i < 2; ++i) {
    Side &s = p.side[i];
    s.x = a.x[i];
    s.dz = a.dz[i];
    s.out = a.out[i];
    s.w = a.w[i];
    s.x_st = a.x_st[i];
    s.z_st = a.dz_st[i];
    s.o_st = a.out_st[i];
    if (a.h[i] > 1 && (s.x_st.head != a.D || s.o_st.head != a.D || (bwd && s.z_st.head != a.D)))
      dense = false;
    s.h = a.h[i];
    if (few) {
      s.chunks = a.h[i] ? pass / a.h[i] : 1;
      if (a.h[i]) p.items += (p.tokens + s.chunks - 1) / s.chunks;
      if (i == 0) p.first = p.items;
    } else {
      s.chunks = (a.h[i] + hpi - 1) / hpi;
      p.items += p.tokens * s.chunks;
    }
  }
  const long need = (p.items + kWarps - 1) / kWarps;
  long cap = bwd ? (long)sms * kBwdBlocksPerSm : (long)sms * 64;
  if (bwd && cap > kBwdBlocksMost) cap = kBwdBlocksMost;
  const unsigned grid = (unsigned)(need < cap ? need : cap);
  if (bwd && (a.dw[0] || a.dw[1])) p.partial = static_cast<float *>(a.workspace);
  const Kind kind = few ? kFewHeads : dense ? kDenseHeads : kStrided;
  e = a.dt == NABLA_BF16 ? launch_dtype<__nv_bfloat16>(p, a.D, a.interleaved, bwd, kind, grid, st)
                         : launch_dtype<float>(p, a.D, a.interleaved, bwd, kind, grid, st);
  if (e != cudaSuccess || !p.partial) return e;
  return launch_pdl(qk_dw_kernel, dim3(2 * a.D / 32), dim3(1024), 0, st,
                    (const float *)p.partial, (int)grid, a.D, a.dw[0], a.dw[1], a.wdt);
}

}  // namespace nabla
