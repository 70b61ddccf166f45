// The parts of the differential attention backward around its products: the rows' numbers in
// packed order (before), and lam's gradient (after).
#include <cuda_bf16.h>

#include "diff_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"
#include "vec8.cuh"

namespace nabla {
namespace {

constexpr int kRowsArrays = 5;

// -lse_1, -lse_2, -delta_1, -delta_2 and -lam of the packed rows [B, hk, nsub, 64], with
// delta_2 = <dout, o2> and delta_1 = <dout, o> + lam delta_2; -inf and 0 where a row is none
// or has no states, so that its P is 0.  A block takes a 64-row subtile, D / 8 lanes a row;
// HBM-bound (o, o2 and dout read once), so a thread's rows are all in flight at once.
template <typename T>
struct PrepParams {
  const T *o, *o2, *dout;
  nabla_strides o_st, o2_st, g_st;
  const float *lse, *lam;  // [B, h, 2, Sq]
  float *rows;
  size_t nrows;
  unsigned *counter;
  int lam_step, Sq, h, hk, G, tq, nsub;
};

template <typename T, int D>
__global__ void __launch_bounds__(256) diff_prep_kernel(const __grid_constant__ PrepParams<T> P) {
  constexpr int kLanes = D / 8, kPass = 256 / kLanes, kRows = 64 / kPass;
  __shared__ float out[kRowsArrays][64];
  const int lane = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  pdl_launch_dependents();
  // blocks side by side take the heads of the same tokens, which lie side by side
  const uint32_t bs = blockIdx.x / (uint32_t)P.hk, j = blockIdx.x - bs * P.hk;
  const uint32_t b = bs / (uint32_t)P.nsub, sub = bs - b * P.nsub;
  const T *o = P.o + b * P.o_st.batch + lane * 8, *o2 = P.o2 + b * P.o2_st.batch + lane * 8;
  const T *g = P.dout + b * P.g_st.batch + lane * 8;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.counter = 0;  // of lam_kernel's blocks
  Raw<T> a[kRows], c[kRows], d[kRows];
  float n[kRows][3];  // -lse_1, -lse_2, lam
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t r = r0 + i * kPass, t = r / (uint32_t)P.G;
    const int token = (int)(sub * P.tq + t), hh = (int)(j * P.G + r - t * P.G);
    const bool ok = t < (uint32_t)P.tq && token < P.Sq;
    a[i] = load_raw(o + token * P.o_st.token + hh * P.o_st.head, ok);
    c[i] = load_raw(o2 + token * P.o2_st.token + hh * P.o2_st.head, ok);
    d[i] = load_raw(g + token * P.g_st.token + hh * P.g_st.head, ok);
    n[i][0] = n[i][1] = -INFINITY;
    n[i][2] = 0.f;
    if (ok) {
      const float *l = P.lse + ((size_t)b * P.h + hh) * 2 * P.Sq + token;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float v = l[(size_t)m * P.Sq];
        if (v != -INFINITY) n[i][m] = -v;
      }
      n[i][2] = P.lam[hh * P.lam_step];
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float x[8], y[8], z[8], s = 0.f, s2 = 0.f;
    unpack8(a[i], x);
    unpack8(c[i], y);
    unpack8(d[i], z);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s = fmaf(z[e], x[e], s);
      s2 = fmaf(z[e], y[e], s2);
    }
#pragma unroll
    for (int e = kLanes / 2; e; e >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, e);
      s2 += __shfl_xor_sync(0xffffffffu, s2, e);
    }
    if (lane < kRowsArrays) {
      const float v = lane == 0   ? n[i][0]
                      : lane == 1 ? n[i][1]
                      : lane == 2 ? -fmaf(n[i][2], s2, s)
                      : lane == 3 ? -s2
                                  : -n[i][2];
      out[lane][r0 + i * kPass] = v;
    }
  }
  __syncthreads();
  const size_t row0 = ((size_t)(b * P.hk + j) * P.nsub + sub) * 64;
  for (int e = threadIdx.x; e < kRowsArrays * 64; e += 256)
    P.rows[(e >> 6) * P.nrows + row0 + (e & 63)] = out[e >> 6][e & 63];
}

// dQ of runs of state tiles: their sums added up in order, scaled and rounded.  A thread per
// four columns.
template <typename T>
__global__ void __launch_bounds__(256)
    diff_dq_sum_kernel(const float *part, int nsplit, int Sq, int Sk, const int32_t *kv_len,
                       float scale, long n4, int row, T *dq) {
  pdl_launch_dependents();
  pdl_wait();
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const long e = i * 4;
  const int b = (int)(e / row / Sq);
  const int tiles = (cross::batch_len(kv_len, b, Sk) + diff::kStates - 1) / diff::kStates;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int sp = 0; sp < nsplit; ++sp) {
    if ((long)tiles * sp / nsplit == (long)tiles * (sp + 1) / nsplit) continue;  // no states
    const float4 x = *reinterpret_cast<const float4 *>(part + (size_t)sp * n4 * 4 + e);
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
  }
  s = make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale);
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4 *>(dq + e) = s;
  else
    *reinterpret_cast<uint2 *>(dq + e) =
        make_uint2(tc::pack_bf16x2(s.x, s.y), tc::pack_bf16x2(s.z, s.w));
}

// A sum in two floats, the second holding what the additions to the first rounded off (Knuth's
// two-sum): the rows' numbers cancel, and 64-bit additions take 2 to 6 us more here.
struct Sum {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum &o) {
    lo += o.lo;
    add(o.hi);
  }
  __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
  __device__ __forceinline__ void over_warp() {
#pragma unroll
    for (int o = 16; o; o >>= 1)
      add(Sum{__shfl_xor_sync(0xffffffffu, hi, o), __shfl_xor_sync(0xffffffffu, lo, o)});
  }
};

// lam's gradient: `sign` times the sum of the rows' numbers ([runs][nrows]; 0 where a row is
// none).  Block (j, c): chunk c of key head j's subtiles, four at a time; lane r of a subtile
// adds up the numbers of head r % G, a warp a head's lanes, to part [h][chunks].  The block that
// is done last adds those up, in order, so that the sum is the same whichever it is.
//
// bf16: minus the sums of P_2 Y from the dQ kernel, since o2 is rounded.  fp32: the rows'
// -delta_2 = -<dout, o2>, where P_2 rebuilt from an fp32 log-sum-exp is off by 2e-7 in a whole
// row at once (2 x 500 x 77, 6 heads on 2 of 128: the gradient off by 2.2e-7 of the rows' norm
// against 4.6e-7; with sums in fp32 3.2e-7).
struct LamParams {
  const float *rows;
  size_t nrows;
  int runs, B, h, hk, G, tq, nsub, each;
  Sum *part;
  float *dlam, sign;
  unsigned *counter;
};

__global__ void __launch_bounds__(256) lam_kernel(const LamParams P) {
  __shared__ Sum sums[256];
  __shared__ bool last;
  const int j = blockIdx.x, chunk = blockIdx.y, chunks = gridDim.y, r = threadIdx.x & 63;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  const long n = (long)P.B * P.nsub, e0 = n * chunk / chunks, e1 = n * (chunk + 1) / chunks;
  pdl_wait();
  const long count = (e1 - e0) * P.runs;
  Sum v{0.f, 0.f};
  for (long k0 = threadIdx.x >> 6; k0 < count; k0 += 4 * 8) {
    float x[8];  // under way together
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t k = (uint32_t)k0 + 4 * i, run = k % (uint32_t)P.runs;
      const uint32_t e = (uint32_t)e0 + k / (uint32_t)P.runs, b = e / (uint32_t)P.nsub;
      const size_t row = ((size_t)(b * P.hk + j) * P.nsub + e - b * P.nsub) * 64 + r;
      x[i] = k < count ? P.rows[run * P.nrows + row] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v.add(x[i]);
  }
  sums[threadIdx.x] = v;
  __syncthreads();
  for (int i = warp; i < P.G; i += 8) {  // head i of the group
    v = Sum{0.f, 0.f};
    for (int t = lane; t < 4 * P.tq; t += 32) v.add(sums[(t & 3) * 64 + (t >> 2) * P.G + i]);
    v.over_warp();
    if (lane == 0) P.part[(size_t)(j * P.G + i) * chunks + chunk] = v;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(P.counter, 1u) + 1u == gridDim.x * gridDim.y;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // a warp for each head, the lanes along its chunks; one weight: the heads' sums in order
  Sum all{0.f, 0.f};
  for (int i = warp; i < P.h; i += 8) {
    v = Sum{0.f, 0.f};
    for (int c = lane; c < chunks; c += 32) {
      const float2 p = __ldcg(reinterpret_cast<const float2 *>(P.part + (size_t)i * chunks + c));
      v.add(Sum{p.x, p.y});
    }
    v.over_warp();
    all.add(v);
    if (P.each && lane == 0) P.dlam[i] = P.sign * v.value();
  }
  if (P.each) return;
  if (lane == 0) sums[warp] = all;
  __syncthreads();
  if (threadIdx.x) return;
  v = Sum{0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) v.add(sums[i]);
  P.dlam[0] = P.sign * v.value();
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Runs of state tiles the fp32 dQ units (64 packed rows) are split into.  Cost in steps of a
// 64 x 64 tile, about 6 us (12 at D 128), in which 24 MB move: as cross_dkv_splits.  (Whole
// backward, D 64, us, in runs and whole: 512 x 2048, 2 heads 92, 281; 256 x 1024, 4 heads 55,
// 148; 2048 x 256, 2 heads 57, 66; D 128: 1024 x 1024, 4 heads 254, 349.  Furthest from the best
// of those tried: 64 x 4096, 4 heads of 64, in 16 runs 72, in 32 65.)
int simt_dq_splits(const CrossShape &s, int nsub) {
  const long units = (long)s.B * s.hk * nsub;
  const int tiles = (s.Sk + 63) / 64;
  int best = 1;
  double least = 0.0;
  for (int n = 1; n <= tiles && n <= 64; ++n) {
    double cost = (double)((units * n + 151) / 152) * ((tiles + n - 1) / n + 0.5);
    if (n > 1) cost += 1.0 + (double)units * n * 64 * s.D * 4 * 2 / 24.0e6;
    if (n == 1 || cost < least) {
      best = n;
      least = cost;
    }
  }
  return best;
}

struct BwdLayout {
  int nsub;  // subtiles per (batch, key head), a whole number of 128-row tiles
  size_t nrows;
  int nsplit, qsplit, truns, chunks;
  size_t rows, t2, part, qpart, lam, counter, total;
};
BwdLayout bwd_layout(const CrossShape &s, nabla_dtype dt) {
  BwdLayout w;
  w.nsub = (cross::packing(s).nsub + 1) / 2 * 2;
  w.nrows = (size_t)s.B * s.hk * w.nsub * 64;
  // Runs of dK / dV, and of dQ in bf16, as in the cross attention's backward: its units' steps
  // and sums are in about the same proportions.  (Whole backward, us, as chosen, then with
  // others.  dK / dV: 32768 x 512, 12 heads of 128, 3 runs 472, 2 564, 6 483; 8192 x 8192 whole
  // 1550, 2 1599; 65536 x 128, 1 head of 64, 64 runs 67, 32 77; 8 x 3000 x 200, 5 heads of 64,
  // whole 110, 3 104, the furthest from the best of those tried; fp32: 2 x 500 x 77, 6 heads on 2
  // of 128, 12 79, 8 95, 20 97.  dQ: 500 x 4000, 4 heads of 128, 8 runs 51, whole 85, 12 64.)
  w.nsplit = cross_dkv_splits(s, dt);
  w.qsplit = dt == NABLA_BF16 ? cross_dq_splits(s) : simt_dq_splits(s, w.nsub);
  w.truns = dt == NABLA_BF16 ? 2 * w.qsplit : 0;
  // 16 subtiles a chunk: four loads a thread and run
  const size_t chunks = ((size_t)s.B * w.nsub + 15) / 16;
  w.chunks = chunks > 64 ? 64 : (int)chunks;
  w.rows = 0;
  w.t2 = round_up(kRowsArrays * w.nrows * sizeof(float));
  w.part = w.t2 + round_up(w.truns * w.nrows * sizeof(float));
  w.qpart = w.part + (w.nsplit > 1 ? round_up((size_t)w.nsplit * 2 * s.B * s.Sk * s.hk * s.D *
                                              sizeof(float))
                                   : 0);
  w.lam = w.qpart + (w.qsplit > 1 ? round_up((size_t)w.qsplit * s.B * s.Sq * s.h * s.D *
                                             sizeof(float))
                                  : 0);
  w.counter = w.lam + round_up((size_t)s.h * w.chunks * sizeof(Sum));
  w.total = w.counter + 256;
  return w;
}

template <typename T, int D>
cudaError_t launch_prep(const DiffArgs &a, const DiffRows &r, float *rows, unsigned *counter,
                        cudaStream_t st) {
  const CrossShape &s = a.x.s;
  const cross::Packing pk = cross::packing(s);
  PrepParams<T> p{};
  p.o = static_cast<const T *>(a.x.of), p.o2 = static_cast<const T *>(a.o2f);
  p.dout = static_cast<const T *>(a.x.dout);
  p.o_st = a.x.o_st, p.o2_st = a.o2_st, p.g_st = a.x.dout_st;
  p.lse = a.x.lse, p.lam = a.lam, p.lam_step = a.lam_n > 1 ? 1 : 0;
  p.rows = rows, p.nrows = r.nrows, p.counter = counter;
  p.Sq = s.Sq, p.h = s.h, p.hk = s.hk, p.G = pk.G, p.tq = pk.tq, p.nsub = r.nsub;
  return launch_pdl(diff_prep_kernel<T, D>, dim3((unsigned)((long)s.B * s.hk * r.nsub)), dim3(256),
                    0, st, p);
}

}  // namespace

cudaError_t launch_diff_dq_sum(const DiffArgs &a, nabla_dtype dt, const float *part, int nsplit,
                               cudaStream_t st) {
  const CrossShape &s = a.x.s;
  const long n4 = (long)s.B * s.Sq * s.h * (s.D / 4);
  const dim3 grid((unsigned)((n4 + 255) / 256));
  if (dt == NABLA_BF16)
    return launch_pdl(diff_dq_sum_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, part, nsplit,
                      s.Sq, s.Sk, a.x.kv_len, a.x.scale, n4, s.h * s.D,
                      static_cast<__nv_bfloat16 *>(a.x.dq));
  return launch_pdl(diff_dq_sum_kernel<float>, grid, dim3(256), 0, st, part, nsplit, s.Sq, s.Sk,
                    a.x.kv_len, a.x.scale, n4, s.h * s.D, static_cast<float *>(a.x.dq));
}

size_t diff_bwd_workspace(const CrossShape &s, nabla_dtype dt) { return bwd_layout(s, dt).total; }

cudaError_t launch_diff_bwd(const DiffArgs &a, nabla_dtype dt, cudaStream_t st) {
  const CrossShape &s = a.x.s;
  const BwdLayout w = bwd_layout(s, dt);
  char *ws = static_cast<char *>(a.x.workspace);
  auto at = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
  unsigned *counter = reinterpret_cast<unsigned *>(ws + w.counter);
  const DiffRows r{at(w.rows), w.nrows, at(w.t2), w.nsub};
  cudaError_t e;
  if (dt == NABLA_BF16)
    e = s.D == 64 ? launch_prep<__nv_bfloat16, 64>(a, r, at(w.rows), counter, st)
                  : launch_prep<__nv_bfloat16, 128>(a, r, at(w.rows), counter, st);
  else
    e = s.D == 64 ? launch_prep<float, 64>(a, r, at(w.rows), counter, st)
                  : launch_prep<float, 128>(a, r, at(w.rows), counter, st);
  if (e != cudaSuccess) return e;
  e = dt == NABLA_BF16
          ? launch_diff_bwd_tc(a, r, at(w.part), w.nsplit, at(w.qpart), w.qsplit, st)
          : launch_diff_bwd_simt(a, r, at(w.part), w.nsplit, at(w.qpart), w.qsplit, st);
  if (e != cudaSuccess) return e;
  const cross::Packing pk = cross::packing(s);
  LamParams p{r.t2, w.nrows, w.truns, s.B, s.h, s.hk, pk.G, pk.tq, w.nsub,
              a.lam_n > 1 ? 1 : 0, reinterpret_cast<Sum *>(ws + w.lam), a.dlam, -1.f,
              counter};
  if (dt == NABLA_F32) p.rows = r.rows + 3 * w.nrows, p.runs = 1, p.sign = 1.f;  // -delta_2
  return launch_pdl(lam_kernel, dim3((unsigned)s.hk, (unsigned)w.chunks), dim3(256), 0, st, p);
}

}  // namespace nabla
