// K11 -- what lies between two branches of a transformer block: the residual plus a
// branch's output, normed, gated and scaled, and the adaptive norm the next branch reads;
// and its gradient.
//
//   s = x + rs gate Np(u) pw,   y = N(s) w (1 + scale) + shift
//   N(t) = t / sqrt(mean t^2 + eps)  or  (t - mean t) / sqrt(var t + eps)
// With d = dy w (1 + scale), n = N(s), r = 1 / sqrt(...), m(.) a row's mean:
//   ds = dsum + r (d - [m(d)] - n m(d n)),   dx = ds,   e = rs gate pw ds,
//   du = ru (e - [m(e)] - nu m(e nu))  (or e),   dgate = rs pw sum ds nu,
//   dscale = w sum dy n,  dshift = sum dy,  dw = sum dy (1 + scale) n,  dpw = sum rs gate ds nu,
// [.] for the layer norm; the sums run over the tokens that share the row of the
// modulation, those of dw and dpw over all.
//
// HBM-bound: x, u read and s, y written once (backward: s, u, dsum, dy read, dx, du
// written).  Variances are summed about each warp's own mean and joined exactly, so a large
// mean cancels no digits of the squares.  The mean itself is an fp32 number: a normed value is
// off by some 2^-24 |mean| / deviation, as it is in elementary fp32 operations (2048 columns, a
// mean of 1000 deviations: 2.3e-5 on average, 9e-5 at most; there 2.3e-5 and 8e-5).
//
// Forward: a warp holds a row (up to 8 vectors of 8 columns a lane; few columns: 8 or 16
// lanes, many: two to eight warps), so its norms need no barrier, and an SM's 16 warps have
// enough rows in flight without loading ahead.  The modulations of a block's rows lie in
// shared memory as fp32, w (1 + scale), rs gate pw and shift, until the block comes to
// another row of them; where such a row has fewer tokens than that is worth they are read
// with every token.  98304 x 1536, norms before and after: 203 us, 5.9 TB/s (88% of a copy's);
// 32768 x 2048, the norm alone: 45 us, 6.0 TB/s; 16 rows of 2048: 3 us in a graph.
//
// Backward: three sums a column stay in registers, so a team of threads holds a row, 8
// columns a thread, a whole block above 256 columns.  Its rows come by bulk copies into a
// ring in shared memory, several rows ahead, which takes no registers; the warps exchange
// their sums once a norm.  Sums over tokens: every team adds up its run's, a modulation row
// at a time.  A row whose tokens all lie in the run is finished there, the others' parts (of
// the run's first and last row of modulations) go to the workspace and are added up in
// order by a second kernel, as are the teams' sums for the weights.  65536 x 2048: 282 us,
// 5.7 TB/s (84%); instructions are issued in 54% of the cycles, which it shares the bound with.
#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "row_ring.cuh"
#include "tc_ptx.cuh"
#include "vec8.cuh"

namespace nabla {
namespace {

using tcattn::add2;
using tcattn::f2;
using tcattn::fma2;
using tcattn::unf2;

constexpr int kTeamBlock = 128;  // backward: threads of a block of several teams
// Threads of a forward block: two blocks an SM leave a thread 128 registers, or 168 where a
// lane holds eight vectors of both x and u (with 128 it spills 350 bytes).
template <int N, bool kU>
constexpr int kFwdBlock = N == 8 && kU ? 192 : 256;
// Blocks of 256 threads on an SM: rows of few vectors need more of them under way (16.8 M
// elements, two blocks against four: C 256 41 us against 29; against three: C 512 28.6
// against 25.3).
template <int N>
constexpr int kFwdPerSm = N == 1 ? 4 : N == 2 ? 3 : 2;
// Blocks of a row each on an SM, with up to 256 threads or up to 512: registers that let one
// more of them in (304 rows of 4096, bf16: 4.2 us against 6.5).
template <int N, int kSpread>
constexpr int kSpreadPerSm = N == 2 ? 1 : kSpread == 256 ? 3 : 2;

struct Mod {  // a modulation: `rows` rows, `st` elements apart
  const void *p;
  int64_t st;
};

struct NormParams {
  const void *x, *u, *dsum, *dy;  // x: backward: the sum
  void *s, *y;                    // forward
  void *dx, *du;                  // backward
  int64_t x_b, x_t, u_b, u_t, ds_b, ds_t, dy_b, dy_t, s_b, s_t, y_b, y_t, dx_b, dx_t, du_b, du_t;
  const void *w, *pw;
  Mod gate, scale, shift;
  void *dgate, *dscale, *dshift;  // [rows, C]
  float *part;                    // [teams][2][3][C]: sums dy n, dy, ds nu of unfinished rows
  float *wpart;                   // [teams][2][C]: the teams' dw and dpw
  nabla_dtype wdt, mdt;
  long T, n;  // tokens; tokens that share a row of the modulations
  int S, C, L;  // tokens of a batch; columns; rows of a run
  int norm, post;  // 0: none, 1: RMS, 2: layer
  int stages;      // backward: rows of the ring
  float rs, eps;
  int *status;
};

__device__ __forceinline__ void load_vec(const void *p, nabla_dtype dt, int64_t at, bool on,
                                         float otherwise, float (&v)[8]) {
  if (!p || !on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = otherwise;
  } else if (dt == NABLA_BF16) {
    load8(static_cast<const __nv_bfloat16 *>(p) + at, v);
  } else {
    load8(static_cast<const float *>(p) + at, v);
  }
}
__device__ __forceinline__ void store_vec(void *p, nabla_dtype dt, int64_t at,
                                          const float (&v)[8]) {
  if (dt == NABLA_BF16)
    store8(static_cast<__nv_bfloat16 *>(p) + at, v);
  else
    store8(static_cast<float *>(p) + at, v);
}

// Eight columns as four fp32 pairs: the pair instructions halve the kernels' arithmetic,
// which as single ones took longer than the rows' way in and out.
using V8 = uint64_t[4];

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float a) { return f2(a, a); }
__device__ __forceinline__ float total(uint64_t v) {
  float a, b;
  unf2(v, a, b);
  return a + b;
}
__device__ __forceinline__ void pairs(const float (&f)[8], V8 &v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void singles(const V8 &v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unf2(v[i], f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw<T> &r, V8 &v) {
  float f[8];
  unpack8(r, f);
  pairs(f, v);
}

// The sums a row's norm needs: its mean (0 for the RMS norm), squares about it, and, of
// the gradient, the sums of d and of d (t - mean).
struct Sums {
  float mean, sq, d, dt;
};

// Shared memory of a block: the warps' sums and column counts.
struct Box {
  Sums of[2][2][16];  // [row in turn][norm][warp]
  float cols[16];
};

// A team: kTeam lanes of a warp, or (0) the whole block.
template <int kTeam, int N, int kBlock>
struct Team {
  static constexpr int kLanes = kTeam ? kTeam : 32;
  long id;
  int size, lane, warps;
  int col[N];
  bool on[N];  // the columns exist
  float own, per;  // columns of this thread's warp, or of the team in it; 1 / own
  Box *box;

  __device__ __forceinline__ Team(int C, Box *b) : box(b) {
    size = kTeam ? kTeam : (int)blockDim.x;
    warps = kTeam ? 1 : (int)blockDim.x >> 5;
    lane = kTeam ? (int)threadIdx.x % kLanes : (int)threadIdx.x;
    id = kTeam ? (long)blockIdx.x * (kBlock / kLanes) + (int)threadIdx.x / kLanes : blockIdx.x;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      col[i] = (lane + i * size) * 8;
      on[i] = col[i] < C;
      n += __popc(__ballot_sync(0xffffffffu, on[i])) * 8;
    }
    own = kTeam ? (float)C : (float)n;
    per = 1.f / own;
    if (warps > 1) {
      if ((threadIdx.x & 31) == 0) box->cols[threadIdx.x >> 5] = own;
      __syncthreads();
    }
  }

  __device__ __forceinline__ float sum(float v) const {
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }

  // The row's sums from its warps'.
  __device__ __forceinline__ Sums join(const Sums &v, int turn, int which, float inv) const {
    if (kTeam || warps == 1) return v;
    Sums *b = box->of[turn][which];
    if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
    __syncthreads();
    // A lane per warp, in both halves of the warp.  First about warp 0's mean, from which the
    // others' differ little: four sums at once, two in each half, whose eighths share them out.
    const int l = threadIdx.x & 15;
    const bool hi = threadIdx.x & 16, odd = threadIdx.x & 8;
    const Sums a = l < warps ? b[l] : Sums{0.f, 0.f, 0.f, 0.f};
    const float n = l < warps ? box->cols[l] : 0.f, mean0 = b[0].mean, off = a.mean - mean0;
    const float x = hi ? a.d : n * off;
    const float y = fmaf(off, x, hi ? a.dt : a.sq);
    float z = (odd ? y : x) + __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
#pragma unroll
    for (int o = 4; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float first = __shfl_sync(0xffffffffu, z, 0), sq = __shfl_sync(0xffffffffu, z, 8);
    const float d = __shfl_sync(0xffffffffu, z, 16), dt = __shfl_sync(0xffffffffu, z, 24);
    const float by = first * inv;  // then about the row's
    return Sums{mean0 + by, fmaf(-by, first, sq), d, fmaf(-by, d, dt)};
  }

  // Takes this warp's mean (layer; else 0) off v, whose columns that do not exist stay 0,
  // and returns it with the squares.
  __device__ __forceinline__ Sums center(V8 (&v)[N], bool layer) const {
    Sums r{0.f, 0.f, 0.f, 0.f};
    if (layer) {
      uint64_t t = 0ull;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) t = add2(t, v[i][j]);
      r.mean = sum(total(t)) * per;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint64_t off = both(on[i] ? -r.mean : 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], off);
      }
    }
    uint64_t t = 0ull;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) t = fma2(v[i][j], v[i][j], t);
    r.sq = total(t);
    return r;
  }
  // This thread's squares (center()'s, of one row) as the warp's.
  __device__ __forceinline__ void sum_squares(Sums &r) const { r.sq = sum(r.sq); }
  // The sums of d and of d v of this warp, v centred, and of its squares.  Three sums a step
  // would be 15 shuffles; here the halves of the warp first share out two pairs of values,
  // then the quarters one.
  __device__ __forceinline__ void products(const V8 (&d)[N], const V8 (&v)[N], Sums &r) const {
    uint64_t a = 0ull, b = 0ull;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a = add2(a, d[i][j]);
        b = fma2(d[i][j], v[i][j], b);
      }
    r.d = total(a);
    r.dt = total(b);
    if (kLanes < 32) {
      r.sq = sum(r.sq), r.d = sum(r.d), r.dt = sum(r.dt);
      return;
    }
    const bool hi = threadIdx.x & 16, odd = threadIdx.x & 8;
    // lanes 0-15: sq, d; lanes 16-31: dt (and nothing)
    const float x = (hi ? r.dt : r.sq) + __shfl_xor_sync(0xffffffffu, hi ? r.sq : r.dt, 16);
    const float y = (hi ? 0.f : r.d) + __shfl_xor_sync(0xffffffffu, hi ? r.d : 0.f, 16);
    // lanes 0-7: sq, 8-15: d, 16-23: dt
    float z = (odd ? y : x) + __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
#pragma unroll
    for (int o = 4; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    r.sq = __shfl_sync(0xffffffffu, z, 0);
    r.d = __shfl_sync(0xffffffffu, z, 8);
    r.dt = __shfl_sync(0xffffffffu, z, 16);
  }
};

// A run's rows: place of the next row to be loaded, and the tokens left in its row of the
// modulations.
struct Place {
  long b;
  int s;
  __device__ __forceinline__ void next(int S) {
    if (++s == S) s = 0, ++b;
  }
};

template <typename T, int N, class Tm>
__device__ __forceinline__ void fetch(const void *p, int64_t bst, int64_t tst, const Place &at,
                                      const Tm &tm, bool on, Raw<T> (&r)[N]) {
  const T *row = static_cast<const T *>(p) + at.b * bst + at.s * tst;
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = load_raw(row + tm.col[i], on && tm.on[i]);
}
template <typename T, int N, class Tm>
__device__ __forceinline__ void put(void *p, int64_t bst, int64_t tst, const Place &at,
                                    const Tm &tm, const V8 (&v)[N]) {
  T *row = static_cast<T *>(p) + at.b * bst + at.s * tst;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (tm.on[i]) {
      float f[8];
      singles(v[i], f);
      store8(row + tm.col[i], f);
    }
}

// up = w (1 + scale) and by = rs gate pw of the team's columns in row `m` of the modulations
// (0 for columns that do not exist).
template <int N, class Tm>
__device__ __forceinline__ void load_mods(const NormParams &P, const Tm &tm, long m, V8 (&up)[N],
                                          V8 (&by)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float a[8], t[8];
    load_vec(P.w, P.wdt, tm.col[i], tm.on[i], 1.f, a);
    load_vec(P.scale.p, P.mdt, m * P.scale.st + tm.col[i], tm.on[i], 0.f, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] *= 1.f + t[j];
    pairs(a, up[i]);
    load_vec(P.pw, P.wdt, tm.col[i], tm.on[i], 1.f, a);
    load_vec(P.gate.p, P.mdt, m * P.gate.st + tm.col[i], tm.on[i], 1.f, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] *= tm.on[i] ? P.rs * t[j] : 0.f;
    pairs(a, by[i]);
  }
}

// kShared: the modulations of a block's rows in shared memory, [up, by, add][C], halves of
// every eight columns apart.
// kSpread: few rows; a block a row, with as many threads as that takes, up to kSpread.
// kU: there is a branch's output.
template <typename T, int kTeam, int N, bool kShared, int kSpread, bool kU>
__global__ void __launch_bounds__(kSpread ? kSpread : kFwdBlock<N, kU>,
                                  kSpread ? kSpreadPerSm<N, kSpread> : kFwdPerSm<N>)
    block_norm_kernel(const __grid_constant__ NormParams P) {
  __shared__ Box box;
  extern __shared__ __align__(16) float mods[];
  pdl_launch_dependents();
  const Team<kTeam, N, kFwdBlock<N, kU>> tm(P.C, &box);
  constexpr int kTeams = kTeam ? kFwdBlock<N, kU> / (kTeam ? kTeam : 1) : 1;
  const uint32_t team = kTeam ? threadIdx.x / tm.kLanes : 0;
  pdl_wait();
  const uint32_t first = blockIdx.x * (uint32_t)P.L;
  const uint32_t end = first + P.L < P.T ? first + P.L : (uint32_t)P.T;
  const float inv = 1.f / (float)P.C;
  // The first four of every eight columns, then the others: lanes 16 bytes apart, so that a
  // warp's read meets every bank once.
  auto put_mod = [&](int which, int c, const float (&v)[8]) {
    float *to = mods + which * P.C + c / 2;
    *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(to + P.C / 2) = make_float4(v[4], v[5], v[6], v[7]);
  };
  int turn = 0;
  for (uint32_t g0 = first, g1; g0 < end; g0 = g1) {
    g1 = end;
    if (kShared) {  // the block's next row of the modulations
      const uint32_t m = g0 / (uint32_t)P.n, last = (m + 1) * (uint32_t)P.n;
      g1 = last < end ? last : end;
      __syncthreads();  // the last one's are no longer read
      for (int c = threadIdx.x * 8; c < P.C; c += blockDim.x * 8) {
        float a[8], t[8];
        load_vec(P.w, P.wdt, c, true, 1.f, a);
        load_vec(P.scale.p, P.mdt, m * P.scale.st + c, true, 0.f, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] *= 1.f + t[j];
        put_mod(0, c, a);
        load_vec(P.pw, P.wdt, c, true, 1.f, a);
        load_vec(P.gate.p, P.mdt, m * P.gate.st + c, true, 1.f, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] *= P.rs * t[j];
        put_mod(1, c, a);
        load_vec(P.shift.p, P.mdt, m * P.shift.st + c, true, 0.f, t);
        put_mod(2, c, t);
      }
      __syncthreads();
    }
#pragma unroll 1
    for (uint32_t r0 = g0; r0 < g1; r0 += kTeams, turn ^= 1) {
      const uint32_t row = r0 + team;
      const bool live = row < g1;
      const Place at{(long)(row / (uint32_t)P.S), (int)(row % (uint32_t)P.S)};
      const uint32_t m = kShared || !live ? 0 : row / (uint32_t)P.n;
      Raw<T> xr[N], ur[N];
      fetch<T, N>(P.x, P.x_b, P.x_t, at, tm, live, xr);
      if (kU) fetch<T, N>(P.u, P.u_b, P.u_t, at, tm, live, ur);
      // eight columns of up, by or add
      auto mod = [&](int which, int i, V8 &v) {
        float a[8], t[8];
        if (kShared) {
          const float *from = mods + which * P.C + tm.col[i] / 2;
          if (tm.on[i]) {
            const ulonglong2 lo = *reinterpret_cast<const ulonglong2 *>(from);
            const ulonglong2 hi = *reinterpret_cast<const ulonglong2 *>(from + P.C / 2);
            v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
          }
          return;
        }
        const bool on = live && tm.on[i];
        if (which == 2) {
          load_vec(P.shift.p, P.mdt, m * P.shift.st + tm.col[i], on, 0.f, a);
        } else {
          const Mod &f = which ? P.gate : P.scale;
          load_vec(which ? P.pw : P.w, P.wdt, tm.col[i], on, 1.f, a);
          load_vec(f.p, P.mdt, m * f.st + tm.col[i], on, which ? 1.f : 0.f, t);
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] *= which ? P.rs * t[j] : 1.f + t[j];
        }
        pairs(a, v);
      };
      V8 s[N];
      if (kU) {
#pragma unroll
        for (int i = 0; i < N; ++i) unpack(ur[i], s[i]);
        float off = 0.f, r = 1.f;  // the normed row: r s + off
        if (P.post) {
          Sums w = tm.center(s, P.post == 2);
          tm.sum_squares(w);
          const Sums q = tm.join(w, turn, 0, inv);
          r = rsqrtf(fmaf(q.sq, inv, P.eps));
          off = (w.mean - q.mean) * r;
        }
        const uint64_t r2 = both(r), off2 = both(off);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          V8 x, by;
          unpack(xr[i], x);
          mod(1, i, by);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = tm.on[i] ? fma2(fma2(s[i][j], r2, off2), by[j], x[j]) : 0ull;
        }
        if (live) put<T, N>(P.s, P.s_b, P.s_t, at, tm, s);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) unpack(xr[i], s[i]);
      }
      if (P.norm) {
        Sums w = tm.center(s, P.norm == 2);
        tm.sum_squares(w);
        const Sums q = tm.join(w, turn, 1, inv);
        const float r = rsqrtf(fmaf(q.sq, inv, P.eps));
        const uint64_t r2 = both(r), off2 = both((w.mean - q.mean) * r);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          V8 up, add;
          mod(0, i, up);
          mod(2, i, add);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = fma2(fma2(s[i][j], r2, off2), up[j], add[j]);
        }
        if (live) put<T, N>(P.y, P.y_b, P.y_t, at, tm, s);
      }
    }
  }
}

// The gradient.  Dynamic shared memory: where a weight's is wanted the teams' dw and dpw,
// [teams of the block][2][C], every column of them one thread's own; then (a team that is a
// block) the ring, [stages][s, dy, dsum, u: those there are][columns of the team].  kMost,
// kPerSm: threads at most, blocks an SM at least; kU: there is a branch's output; kPost: it is
// normed.
template <typename T, int kTeam, int N, int kMost, int kPerSm, bool kU, bool kPost>
__global__ void __launch_bounds__(kMost, kPerSm)
    block_norm_bwd_kernel(const __grid_constant__ NormParams P) {
  __shared__ Box box;
  __shared__ RowRing ring;
  extern __shared__ __align__(16) float wsum[];
  pdl_launch_dependents();
  const Team<kTeam, N, kTeamBlock> tm(P.C, &box);
  float *own = wsum + (kTeam ? (int)threadIdx.x / tm.kLanes : 0) * 2 * P.C;
  uint8_t *rows = reinterpret_cast<uint8_t *>(wsum + (P.wpart ? 2 * P.C : 0));
  // a row's copy, and its place: as many columns as the team's threads read, the last ones 0
  const uint32_t bytes = P.C * sizeof(T), pitch = blockDim.x * 8 * N * sizeof(T);
  const int tensors = (P.norm ? 2 : 0) + (P.dsum ? 1 : 0) + (kU ? 1 : 0);
  if (P.wpart)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (tm.on[i])
#pragma unroll
        for (int j = 0; j < 8; ++j) own[tm.col[i] + j] = own[P.C + tm.col[i] + j] = 0.f;
  if (!kTeam) {
    for (int x = 0; x < P.stages * tensors; ++x)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!tm.on[i]) {
          const float none[8] = {};
          store8(reinterpret_cast<T *>(rows + x * pitch) + tm.col[i], none);
        }
    if (threadIdx.x == 0) {
      for (int i = 0; i < P.stages; ++i) tc::mbar_init(&ring.full[i], 1);
      ring.abort = 0;
      ring.stages = P.stages;
      tc::fence_barrier_init();
    }
    __syncthreads();
  }
  pdl_wait();
  const long first = tm.id * P.L, end = first + P.L < P.T ? first + P.L : P.T;
  Place at{first / P.S, (int)(first % P.S)}, ahead = at;
  const float inv = 1.f / (float)P.C;
  V8 up[N], by[N], acc[3][N];
  long m = first / P.n, left = 0;
  Raw<T> sr[N], ur[N], gr[N], yr[N];
  // A team that is a block: thread 0 asks for `row`, the next one to be loaded.
  int ask = 0, stage = 0;
  uint32_t phase = 0;
  auto request = [&](long row) {
    if (row >= end) return;
    tc::mbar_expect_tx(&ring.full[ask], tensors * bytes);
    uint8_t *to = rows + ask * tensors * pitch;
    auto copy = [&](const void *p, int64_t bst, int64_t tst) {
      tc::bulk_load(to, static_cast<const T *>(p) + ahead.b * bst + ahead.s * tst, bytes,
                    &ring.full[ask]);
      to += pitch;
    };
    if (P.norm) {
      copy(P.x, P.x_b, P.x_t);
      copy(P.dy, P.dy_b, P.dy_t);
    }
    if (P.dsum) copy(P.dsum, P.ds_b, P.ds_t);
    if (kU) copy(P.u, P.u_b, P.u_t);
    ahead.next(P.S);
    if (++ask == P.stages) ask = 0;
  };
  // The next row into registers: from memory, or out of the ring.
  auto load = [&](long row) {
    const bool live = row < end;
    if (kTeam) {
      if (P.norm) {
        fetch<T, N>(P.x, P.x_b, P.x_t, ahead, tm, live, sr);
        fetch<T, N>(P.dy, P.dy_b, P.dy_t, ahead, tm, live, yr);
      }
      if (P.dsum) fetch<T, N>(P.dsum, P.ds_b, P.ds_t, ahead, tm, live, gr);
      if (kU) fetch<T, N>(P.u, P.u_b, P.u_t, ahead, tm, live, ur);
      ahead.next(P.S);
      return;
    }
    if (!tc::mbar_try_wait(&ring.full[stage], phase))
      wait_for_row(&ring.full[stage], phase, &ring, P.status);
    const T *from = reinterpret_cast<const T *>(rows + stage * tensors * pitch);
    auto take = [&](Raw<T> (&r)[N]) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = load_raw(from + tm.col[i], true);
      from += pitch / sizeof(T);
    };
    if (P.norm) {
      take(sr);
      take(yr);
    }
    if (P.dsum) take(gr);
    if (kU) take(ur);
    if (++stage == P.stages) stage = 0, phase ^= 1u;
  };
  // the sums of row m of the modulations, whose tokens up to `upto` this run has seen
  auto finish = [&](long upto) {
    const long g0 = m * P.n;
    const bool whole = g0 >= first && upto == g0 + P.n;
    float *part = P.part ? P.part + ((size_t)tm.id * 2 + (first >= g0 ? 0 : 1)) * 3 * P.C : nullptr;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!tm.on[i]) continue;
      const int c = tm.col[i];
      float t[8], w[8], a[3][8];
#pragma unroll
      for (int k = 0; k < 3; ++k) singles(acc[k][i], a[k]);
      if (P.wpart) {  // what the modulations contribute to the weights' gradients
        load_vec(P.scale.p, P.mdt, m * P.scale.st + c, true, 0.f, t);
        load8(own + c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = fmaf(1.f + t[j], a[0][j], w[j]);
        store8(own + c, w);
        if (kPost) {
          load_vec(P.gate.p, P.mdt, m * P.gate.st + c, true, 1.f, t);
          load8(own + P.C + c, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = fmaf(P.rs * t[j], a[2][j], w[j]);
          store8(own + P.C + c, w);
        }
      }
      if (!P.part) continue;
      if (!whole) {
#pragma unroll
        for (int k = 0; k < 3; ++k) store8(part + k * P.C + c, a[k]);
        continue;
      }
      const int64_t o = m * P.C + c;
      if (P.dscale) {
        load_vec(P.w, P.wdt, c, true, 1.f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = w[j] * a[0][j];
        store_vec(P.dscale, P.mdt, o, t);
      }
      if (P.dshift) store_vec(P.dshift, P.mdt, o, a[1]);
      if (P.dgate) {
        load_vec(P.pw, P.wdt, c, true, 1.f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = P.rs * w[j] * a[2][j];
        store_vec(P.dgate, P.mdt, o, t);
      }
    }
  };
  if (kTeam)
    load(first);
  else if (threadIdx.x == 0)
    for (int i = 0; i < P.stages; ++i) request(first + i);
  int turn = 0;
#pragma unroll 1
  for (long row = first; row < first + P.L; ++row, turn ^= 1) {
    const bool live = row < end;
    if (!kTeam && !live) break;
    if (!kTeam) load(row);
    if (left == 0 && live) {
      if (row != first) {
        finish(row);
        ++m;
      }
      left = (m + 1) * P.n - row;
      load_mods<N>(P, tm, m, up, by);
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[k][i][j] = 0ull;
    }
    --left;
    V8 s[N], ds[N], v[N], d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (P.norm) {
        unpack(sr[i], s[i]);
        unpack(yr[i], d[i]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) ds[i][j] = 0ull;
      if (P.dsum) unpack(gr[i], ds[i]);
      if (kU) unpack(ur[i], v[i]);
    }
    if (kTeam) load(row + 1);
    if (!kTeam && !P.norm) {  // with a norm, the warps meet there
      __syncthreads();
      if (threadIdx.x == 0) request(row + P.stages);
    }
    if (P.norm) {
      V8 g[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) g[i][j] = mul2(d[i][j], up[i][j]);
      Sums w = tm.center(s, P.norm == 2);
      tm.products(g, s, w);
      const Sums q = tm.join(w, turn, 0, inv);
      // every warp has taken the row out of the ring
      if (!kTeam && threadIdx.x == 0) request(row + P.stages);
      const float r = rsqrtf(fmaf(q.sq, inv, P.eps));
      const uint64_t r2 = both(r), off2 = both((w.mean - q.mean) * r);
      const uint64_t mg = both(P.norm == 2 ? -r * q.d * inv : 0.f), mgn = both(-r * r * q.dt * inv);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t n = fma2(s[i][j], r2, off2);
          if (live) {
            acc[0][i][j] = fma2(d[i][j], n, acc[0][i][j]);
            acc[1][i][j] = add2(d[i][j], acc[1][i][j]);
          }
          // dsum + (r g - r mean(g) - n r mean(g n))
          ds[i][j] = add2(ds[i][j], fma2(n, mgn, fma2(g[i][j], r2, mg)));
        }
    }
    if (live && P.dx) put<T, N>(P.dx, P.dx_b, P.dx_t, at, tm, ds);
    if (kU) {
      V8 e[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) e[i][j] = mul2(ds[i][j], by[i][j]);
      if (kPost) {
        Sums w = tm.center(v, P.post == 2);
        tm.products(e, v, w);
        const Sums q = tm.join(w, turn, 1, inv);
        const float r = rsqrtf(fmaf(q.sq, inv, P.eps));
        const uint64_t r2 = both(r), off2 = both((w.mean - q.mean) * r);
        const uint64_t me = both(P.post == 2 ? -r * q.d * inv : 0.f);
        const uint64_t men = both(-r * r * q.dt * inv);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[i][j] = fma2(v[i][j], r2, off2);
            e[i][j] = fma2(v[i][j], men, fma2(e[i][j], r2, me));
          }
      }
      if (live)
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[2][i][j] = fma2(ds[i][j], v[i][j], acc[2][i][j]);
      if (live && P.du) put<T, N>(P.du, P.du_b, P.du_t, at, tm, e);
    } else if (live && P.du) {  // without the branch's output: du alone
      V8 e[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) e[i][j] = mul2(ds[i][j], by[i][j]);
      put<T, N>(P.du, P.du_b, P.du_t, at, tm, e);
    }
    at.next(P.S);
  }
  if (first < end) finish(end);
  if (P.wpart && first < end) {
    float *o = P.wpart + (size_t)tm.id * 2 * P.C;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (tm.on[i])
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const int c = tm.col[i] + j;
          *reinterpret_cast<float4 *>(o + c) = *reinterpret_cast<const float4 *>(own + c);
          *reinterpret_cast<float4 *>(o + P.C + c) =
              *reinterpret_cast<const float4 *>(own + P.C + c);
        }
  }
}

// The sums that no run saw whole: blockIdx.y < ny: of a row of the modulations (there are
// `rows`, and as many as ny of them can lie in more than one run); the last: of the
// weights.  32 columns a block, blockDim / 32 teams at a time.
__global__ void __launch_bounds__(1024)
    block_norm_join_kernel(const __grid_constant__ NormParams P, int teams, int ny, long rows,
                           void *dw, void *dpw) {
  __shared__ float sums[3][32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  const int lanes = blockDim.x >> 5;  // 3 at least
  pdl_launch_dependents();
  pdl_wait();  // in every block, so that whoever waits for this kernel waits for the first
  const bool weights = (int)blockIdx.y == ny;
  long m = blockIdx.y;
  if (!weights && ny < rows) {  // by the runs' borders: the rows that run y + 1 goes on with
    const long at = ((long)blockIdx.y + 1) * P.L;
    m = at / P.n;
    if (at == m * P.n || at - P.L > m * P.n) return;  // begins there; another's
  }
  const long g0 = m * P.n, g1 = g0 + P.n;
  const int t0 = weights ? 0 : (int)(g0 / P.L), t1 = weights ? teams - 1 : (int)((g1 - 1) / P.L);
  if (!weights && t0 == t1) return;  // seen whole
  float a[3] = {0.f, 0.f, 0.f};
  if (c < P.C)
#pragma unroll 4
    for (int t = t0 + ty; t <= t1; t += lanes) {
      const float *p = weights ? P.wpart + (size_t)t * 2 * P.C
                               : P.part + ((size_t)t * 2 + ((long)t * P.L >= g0 ? 0 : 1)) * 3 * P.C;
      a[0] += p[c];
      a[1] += p[P.C + c];
      if (!weights) a[2] += p[2 * P.C + c];
    }
#pragma unroll
  for (int k = 0; k < 3; ++k) sums[k][ty][tx] = a[k];
  __syncthreads();
  if (ty >= 3 || c >= P.C) return;  // a warp for each of the three
  float v = 0.f;
  for (int k = 0; k < lanes; ++k) v += sums[ty][k][tx];
  void *o = weights ? (ty == 0 ? dw : ty == 1 ? dpw : nullptr)
                    : (ty == 0 ? P.dscale : ty == 1 ? P.dshift : P.dgate);
  if (!o) return;
  auto weight = [&](const void *w) {
    return !w ? 1.f
           : P.wdt == NABLA_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c])
                                 : static_cast<const float *>(w)[c];
  };
  if (!weights && ty == 0) v *= weight(P.w);
  if (!weights && ty == 2) v *= P.rs * weight(P.pw);
  const int64_t to = weights ? c : m * P.C + c;
  if ((weights ? P.wdt : P.mdt) == NABLA_BF16)
    static_cast<__nv_bfloat16 *>(o)[to] = __float2bfloat16_rn(v);
  else
    static_cast<float *>(o)[to] = v;
}

// Lanes of a team in a warp (0: a block), vectors a thread, threads of a block.
struct Form {
  int team, vecs, threads;
};
Form bwd_form(int C) {
  if (C <= 64) return {8, 1, kTeamBlock};
  if (C <= 128) return {16, 1, kTeamBlock};
  if (C <= 256) return {32, 1, kTeamBlock};
  if (C <= 4096) return {0, 1, (C + 255) / 256 * 32};
  return {0, 2, (C + 511) / 512 * 32};
}
// bf16: up to 8 vectors a lane, fp32 (twice the registers): 4.  A row of several warps has 6 or 8
// of them, or 4.
Form fwd_form(int C, nabla_dtype dt, bool u) {
  if (C <= 64) return {8, 1, 256};
  if (C <= 128) return {16, 1, 256};
  const int most = dt == NABLA_BF16 ? 8 : 4, warps = (C + most * 256 - 1) / (most * 256);
  int vecs = (C + warps * 256 - 1) / (warps * 256);
  if (vecs > 1) vecs = (vecs + 1) / 2 * 2;  // 1, 2, 4, 6, 8
  const int threads = vecs == 8 && u ? kFwdBlock<8, true> : 256;
  return {warps == 1 ? 32 : 0, vecs, warps == 1 ? threads : warps * 32};
}

// bf16 rows of up to 2560 columns: two blocks of up to 320 threads on an SM, at 96 registers,
// with some of them spilled (16384 rows, norms before and after: 2152 columns 159 us against 183,
// 2560 157 against 182).  In fp32 or with 384 threads more spill (fp32, 2560 242 against 209).
bool bwd_pair(const Form &f, nabla_dtype dt) {
  return dt == NABLA_BF16 && f.vecs == 1 && f.threads > 256 && f.threads <= 320;
}
int bwd_per_sm(const Form &f, nabla_dtype dt) { return bwd_pair(f, dt) ? 2 : 512 / f.threads; }

// Teams and rows of a run of the backward.  Sized for GB300's 152 SMs, so that the workspace
// depends on the shape alone: 512 threads an SM or two blocks.  n: tokens of a row of the modulations.
struct Runs {
  long teams;
  int L;
};
Runs bwd_runs(const NormShape &s, long n, nabla_dtype dt) {
  const Form f = bwd_form(s.C);
  const long T = (long)s.B * s.S;
  const int per = f.team ? f.threads / f.team : 1;  // teams of a block
  const long most = 152L * bwd_per_sm(f, dt) * per;
  long L = (T + most - 1) / most;
  // Whole rows of the modulations where that changes little: nothing to join then.  Teams of
  // a warp or less: up to a run's length (65536 x 256, fp32 modulations, 16 tokens a row: 94 us
  // against 118; 8: 103 against 126), a block a row: to a quarter of it (32768 x 1536, 16
  // tokens: 208 against 221 us, 8: 224 against 231, but 64: 217 against 206).
  if (n * (f.team ? 1 : 4) <= L) L = (L + n - 1) / n * n;
  return {(T + L - 1) / L, (int)L};
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

struct NormLayout {
  size_t part, wpart, total;
};
NormLayout norm_layout(const NormShape &s) {
  const Runs r = bwd_runs(s, s.B * (long)s.S, NABLA_BF16);  // the most runs
  NormLayout w;
  w.part = 0;
  w.wpart = round_up((size_t)r.teams * 6 * s.C * sizeof(float));
  w.total = w.wpart + round_up((size_t)r.teams * 2 * s.C * sizeof(float));
  return w;
}

// Tokens of a row of the modulations from which on it is worth laying out in shared memory
// (8192 rows, 4 tokens each: C 1536 41.5 us against 56.5, C 5120 133 against 156, but C 512
// 20.4 against 17.4; 8 tokens, C 512: 14.1 against 17.4; 2, C 1536: 67 against 58).
constexpr int shared_from(int C) { return C > 512 ? 4 : 8; }

constexpr int kMostColumns = 8192;
// Dynamic shared memory of the backward's blocks on an SM.
constexpr int kBwdRoom = 220 * 1024;

// A kernel's limit of dynamic shared memory is one for all host threads, and calls of several
// widths share a kernel: `limit` is what the kernel may need at any of them, so that no thread's
// call takes from another's, about to be launched.
cudaError_t launch_with_room(void (*kern)(NormParams), int limit, dim3 grid, dim3 block,
                             size_t smem, cudaStream_t st, const NormParams &p) {
  if (smem > 40000) {  // with less (and 48 KB in all) a kernel needs no limit of its own
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, limit);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, grid, block, smem, st, p);
}

template <typename T, int kTeam, int N, int kSpread, bool kU>
cudaError_t launch_fwd_u(NormParams p, const Form &f, cudaStream_t st) {
  const bool shared = !kSpread && p.n >= shared_from(p.C);
  const size_t smem = shared ? (size_t)3 * p.C * sizeof(float) : 0;
  // as many warps an SM as their registers allow, if shared memory holds their modulations
  int per_sm = kSpread ? 2048 / f.threads : kFwdPerSm<N> * kFwdBlock<N, kU> / f.threads;
  while (per_sm > 1 && per_sm * smem > 200 * 1024) --per_sm;
  const long most = 152L * per_sm;
  p.L = (int)((p.T + most - 1) / most);
  const dim3 grid((unsigned)((p.T + p.L - 1) / p.L)), block(f.threads);
  auto kern = shared ? block_norm_kernel<T, kTeam, N, !kSpread, kSpread, kU>
                     : block_norm_kernel<T, kTeam, N, false, kSpread, kU>;
  constexpr int limit = 3 * (kTeam ? kTeam * 8 * N : kMostColumns) * (int)sizeof(float);
  return launch_with_room(kern, limit, grid, block, smem, st, p);
}

template <typename T, int kTeam, int N, int kSpread = 0>
cudaError_t launch_fwd(const NormParams &p, const Form &f, cudaStream_t st) {
  return p.u ? launch_fwd_u<T, kTeam, N, kSpread, true>(p, f, st)
             : launch_fwd_u<T, kTeam, N, kSpread, false>(p, f, st);
}

template <typename T, int kTeam, int N, int kMost, int kPerSm = 1>
cudaError_t launch_bwd(NormParams p, const Form &f, long teams, cudaStream_t st) {
  const int per = kTeam ? f.threads / (kTeam ? kTeam : 1) : 1;
  const dim3 grid((unsigned)((teams + per - 1) / per)), block(f.threads);
  size_t smem = p.wpart ? (size_t)per * 2 * p.C * sizeof(float) : 0;
  if (!kTeam) {  // as many rows as fit the SM's share of shared memory
    const size_t row =
        ((p.norm ? 2 : 0) + (p.dsum ? 1 : 0) + (p.u ? 1 : 0)) * f.threads * 8 * N * sizeof(T);
    const int per_sm = bwd_per_sm(f, sizeof(T) == 2 ? NABLA_BF16 : NABLA_F32);
    const size_t room = (size_t)kBwdRoom / per_sm - 2048;
    p.stages = smem + row < room ? (int)((room - smem) / row) : 1;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    smem += p.stages * row;
  }
  auto kern = p.post ? block_norm_bwd_kernel<T, kTeam, N, kMost, kPerSm, true, true>
              : p.u  ? block_norm_bwd_kernel<T, kTeam, N, kMost, kPerSm, true, false>
                     : block_norm_bwd_kernel<T, kTeam, N, kMost, kPerSm, false, false>;
  return launch_with_room(kern, kBwdRoom, grid, block, smem, st, p);
}

template <typename T>
cudaError_t launch_fwd_form(const NormParams &p, const Form &f, cudaStream_t st) {
  // Few rows: what counts is how long one takes (C 1536: 16 rows 3.0 us against 3.7, 608 3.6
  // against 4.6, 1216 6.8 against 4.8; C 4096: 152 3.5 against 10.7, 608 7.8 against 12.2,
  // 1216 20 against 15; C 5120, two vectors a thread: 304 8.6 against 10.8, 456 11.5 against
  // 10.9).
  if (p.C > 256 && p.T <= (p.C <= 4096 ? 608 : 304)) {
    const int vecs = p.C <= 4096 ? 1 : 2;
    const Form g{0, vecs, (p.C + vecs * 256 - 1) / (vecs * 256) * 32};
    if (vecs == 2) return launch_fwd<T, 0, 2, 512>(p, g, st);
    return g.threads <= 256 ? launch_fwd<T, 0, 1, 256>(p, g, st)
                            : launch_fwd<T, 0, 1, 512>(p, g, st);
  }
  if (f.team == 8) return launch_fwd<T, 8, 1>(p, f, st);
  if (f.team == 16) return launch_fwd<T, 16, 1>(p, f, st);
  constexpr bool kWide = sizeof(T) == 4;
  if (f.team == 32) {
    if (f.vecs == 1) return launch_fwd<T, 32, 1>(p, f, st);
    if (f.vecs == 2) return launch_fwd<T, 32, 2>(p, f, st);
    if (kWide || f.vecs == 4) return launch_fwd<T, 32, 4>(p, f, st);
    if constexpr (!kWide)
      return f.vecs == 6 ? launch_fwd<T, 32, 6>(p, f, st) : launch_fwd<T, 32, 8>(p, f, st);
  }
  if constexpr (kWide)
    return launch_fwd<T, 0, 4>(p, f, st);
  else
    return f.vecs == 6 ? launch_fwd<T, 0, 6>(p, f, st) : launch_fwd<T, 0, 8>(p, f, st);
}

template <typename T>
cudaError_t launch_bwd_form(const NormParams &p, const Form &f, long teams, cudaStream_t st) {
  switch (f.team) {
    case 8: return launch_bwd<T, 8, 1, kTeamBlock>(p, f, teams, st);
    case 16: return launch_bwd<T, 16, 1, kTeamBlock>(p, f, teams, st);
    case 32: return launch_bwd<T, 32, 1, kTeamBlock>(p, f, teams, st);
  }
  if constexpr (sizeof(T) == 2)
    if (bwd_pair(f, NABLA_BF16)) return launch_bwd<T, 0, 1, 320, 2>(p, f, teams, st);
  if (f.vecs == 1) return launch_bwd<T, 0, 1, 512>(p, f, teams, st);
  // two vectors a thread want more than the 128 registers that 512 threads have (16384 x 5120:
  // 341 us against 510)
  return f.threads <= 384 ? launch_bwd<T, 0, 2, 384>(p, f, teams, st)
                          : launch_bwd<T, 0, 2, 512>(p, f, teams, st);
}

}  // namespace

size_t block_norm_bwd_workspace(const NormShape &s) { return norm_layout(s).total; }

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t st) {
  NormParams p{};
  p.x = a.x, p.u = a.u, p.dsum = a.dsum, p.dy = a.dy;
  p.s = a.s, p.y = a.y, p.dx = a.dx, p.du = a.du;
  p.x_b = a.x_st.batch, p.x_t = a.x_st.token, p.u_b = a.u_st.batch, p.u_t = a.u_st.token;
  p.ds_b = a.dsum_st.batch, p.ds_t = a.dsum_st.token;
  p.dy_b = a.dy_st.batch, p.dy_t = a.dy_st.token;
  p.s_b = a.s_st.batch, p.s_t = a.s_st.token, p.y_b = a.y_st.batch, p.y_t = a.y_st.token;
  p.dx_b = a.dx_st.batch, p.dx_t = a.dx_st.token;
  p.du_b = a.du_st.batch, p.du_t = a.du_st.token;
  p.w = a.w, p.pw = a.pw, p.wdt = a.wdt, p.mdt = a.mdt;
  p.gate = Mod{a.gate, a.gate_st}, p.scale = Mod{a.scale, a.scale_st};
  p.shift = Mod{a.shift, a.shift_st};
  p.dgate = a.dgate, p.dscale = a.dscale, p.dshift = a.dshift;
  p.T = (long)a.shape.B * a.shape.S;
  p.n = p.T / a.rows;
  p.S = a.shape.S, p.C = a.shape.C;
  p.norm = a.norm, p.post = a.post;
  p.rs = a.rs, p.eps = a.eps;
  p.status = a.status;
  if (!a.bwd)
    return a.dt == NABLA_BF16 ? launch_fwd_form<__nv_bfloat16>(p, fwd_form(p.C, a.dt, p.u), st)
                              : launch_fwd_form<float>(p, fwd_form(p.C, a.dt, p.u), st);
  const Form f = bwd_form(p.C);
  const Runs r = bwd_runs(a.shape, p.n, a.dt);
  p.L = r.L;
  const NormLayout w = norm_layout(a.shape);
  char *ws = static_cast<char *>(a.workspace);
  if (p.dgate || p.dscale || p.dshift) p.part = reinterpret_cast<float *>(ws + w.part);
  if (a.dw || a.dpw) p.wpart = reinterpret_cast<float *>(ws + w.wpart);
  const cudaError_t e = a.dt == NABLA_BF16
                            ? launch_bwd_form<__nv_bfloat16>(p, f, r.teams, st)
                            : launch_bwd_form<float>(p, f, r.teams, st);
  if (e != cudaSuccess || !(p.part || p.wpart)) return e;
  // rows of the modulations that may lie in several runs: none, all, or one a border
  long ny = !p.part || p.L % p.n == 0 ? 0 : a.rows <= r.teams - 1 ? a.rows : r.teams - 1;
  const unsigned nx = (unsigned)((p.C + 31) / 32);
  auto join = [&](unsigned y, unsigned threads, long borders) {
    return launch_pdl(block_norm_join_kernel, dim3(nx, y), dim3(threads), 0, st, p, (int)r.teams,
                      (int)borders, (long)a.rows, a.dw, a.dpw);
  };
  // a row of them lies in few runs: small blocks (16384 x 1536, 5 runs: 106 us against 120;
  // 4096 x 1536, 18 runs: 41.4 against 39.9)
  if (ny > 0 && p.n <= 10L * p.L) {
    const cudaError_t e2 = join((unsigned)ny, 128, ny);
    if (e2 != cudaSuccess) return e2;
    ny = 0;
  }
  if (ny == 0 && !p.wpart) return e;
  return join((unsigned)ny + (p.wpart ? 1 : 0), 1024, ny);
}

}  // namespace nabla
