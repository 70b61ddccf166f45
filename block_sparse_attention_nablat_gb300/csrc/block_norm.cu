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
// written).  A team of threads holds a row, 8 (or 16) columns a thread, and walks a run
// of rows with the next row's loads under way; the modulations of its columns stay in
// registers until the run comes to another row of them.  A team is a whole block, whose
// warps exchange their sums once a norm, or, up to 256 columns, 8 to 32 lanes.  Variances
// are summed about each warp's own mean and joined exactly, so a large mean costs nothing.
//
// The gradient's sums over tokens: every team adds up its run's, a modulation row at a
// time.  A row whose tokens all lie in the run is finished there, the others' parts (of
// the run's first and last row of modulations) go to the workspace and are added up in
// order by a second kernel, as are the teams' sums for the weights.
#include <cuda_bf16.h>

#include "internal.h"
#include "pdl.cuh"
#include "vec8.cuh"

namespace nabla {
namespace {

constexpr int kTeamBlock = 128;  // threads of a block of several teams

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
  float rs, eps;
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
template <int kTeam, int N>
struct Team {
  static constexpr int kLanes = kTeam ? kTeam : 32;
  long id;
  int size, lane, warps;
  int col[N];
  bool on[N];  // the columns exist
  float own;   // columns of this thread's warp, or of the team in it
  Box *box;

  __device__ __forceinline__ Team(int C, Box *b) : box(b) {
    size = kTeam ? kTeam : (int)blockDim.x;
    warps = kTeam ? 1 : (int)blockDim.x >> 5;
    lane = kTeam ? (int)threadIdx.x % kLanes : (int)threadIdx.x;
    id = kTeam ? (long)blockIdx.x * (kTeamBlock / kLanes) + (int)threadIdx.x / kLanes : blockIdx.x;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      col[i] = (lane + i * size) * 8;
      on[i] = col[i] < C;
      n += __popc(__ballot_sync(0xffffffffu, on[i])) * 8;
    }
    own = kTeam ? (float)C : (float)n;
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
  __device__ __forceinline__ Sums join(const Sums &v, int turn, int which, int C) const {
    if (kTeam || warps == 1) return v;
    Sums *b = box->of[turn][which];
    if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
    __syncthreads();
    Sums r{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < warps; ++i) r.mean = fmaf(b[i].mean, box->cols[i], r.mean);
    r.mean /= (float)C;
    for (int i = 0; i < warps; ++i) {
      const Sums a = b[i];
      const float off = a.mean - r.mean;
      r.sq += fmaf(box->cols[i] * off, off, a.sq);
      r.d += a.d;
      r.dt += fmaf(off, a.d, a.dt);
    }
    return r;
  }

  // This warp's mean and squares about it (columns that do not exist hold 0).
  __device__ __forceinline__ Sums squares(const float (&v)[N][8], bool layer) const {
    Sums r{0.f, 0.f, 0.f, 0.f};
    if (layer) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) r.mean += v[i][j];
      r.mean = sum(r.mean) / own;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i])
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = v[i][j] - r.mean;
          r.sq = fmaf(t, t, r.sq);
        }
    r.sq = sum(r.sq);
    return r;
  }
  // The sums of d and of d (t - mean) of this warp, t = (v - mean) mul.
  __device__ __forceinline__ void products(const float (&d)[N][8], const float (&v)[N][8],
                                           float mean, float mul, Sums &r) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r.d += d[i][j];
        r.dt = fmaf(d[i][j] * mul, v[i][j] - mean, r.dt);
      }
    r.d = sum(r.d);
    r.dt = sum(r.dt);
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
                                    const Tm &tm, const float (&v)[N][8]) {
  T *row = static_cast<T *>(p) + at.b * bst + at.s * tst;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (tm.on[i]) store8(row + tm.col[i], v[i]);
}

// up = w (1 + scale) and by = rs gate pw of the team's columns in row `m` of the modulations.
template <int N, class Tm>
__device__ __forceinline__ void load_mods(const NormParams &P, const Tm &tm, long m,
                                          float (&up)[N][8], float (&by)[N][8]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t[8];
    load_vec(P.w, P.wdt, tm.col[i], tm.on[i], 1.f, up[i]);
    load_vec(P.scale.p, P.mdt, m * P.scale.st + tm.col[i], tm.on[i], 0.f, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) up[i][j] *= 1.f + t[j];
    load_vec(P.pw, P.wdt, tm.col[i], tm.on[i], 1.f, by[i]);
    load_vec(P.gate.p, P.mdt, m * P.gate.st + tm.col[i], tm.on[i], 1.f, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) by[i][j] *= P.rs * t[j];
  }
}

template <typename T, int kTeam, int N>
__global__ void __launch_bounds__(kTeam ? kTeamBlock : 512)
    block_norm_kernel(const __grid_constant__ NormParams P) {
  __shared__ Box box;
  pdl_launch_dependents();
  const Team<kTeam, N> tm(P.C, &box);
  pdl_wait();
  const long first = tm.id * P.L, end = first + P.L < P.T ? first + P.L : P.T;
  Place at{first / P.S, (int)(first % P.S)}, ahead = at;
  const float inv = 1.f / (float)P.C;
  float up[N][8], by[N][8], add[N][8];
  long m = first / P.n, left = 0;  // left: tokens of row m of the modulations still to come
  Raw<T> xr[N], ur[N];
  auto load = [&](long row) {
    fetch<T, N>(P.x, P.x_b, P.x_t, ahead, tm, row < end, xr);
    if (P.u) fetch<T, N>(P.u, P.u_b, P.u_t, ahead, tm, row < end, ur);
    ahead.next(P.S);
  };
  load(first);
  int turn = 0;
#pragma unroll 1
  for (long row = first; row < first + P.L; ++row, turn ^= 1) {
    const bool live = row < end;
    if (!kTeam && !live) break;  // teams in a warp stay together
    if (left == 0 && live) {
      if (row != first) ++m;
      left = (m + 1) * P.n - row;
      load_mods<N>(P, tm, m, up, by);
#pragma unroll
      for (int i = 0; i < N; ++i)
        load_vec(P.shift.p, P.mdt, m * P.shift.st + tm.col[i], tm.on[i], 0.f, add[i]);
    }
    --left;
    float s[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) unpack8(xr[i], s[i]);
    if (P.u) {
      float v[N][8];
#pragma unroll
      for (int i = 0; i < N; ++i) unpack8(ur[i], v[i]);
      load(row + 1);
      float mean = 0.f, r = 1.f;
      if (P.post) {
        const Sums q = tm.join(tm.squares(v, P.post == 2), turn, 0, P.C);
        mean = q.mean;
        r = rsqrtf(fmaf(q.sq, inv, P.eps));
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (tm.on[i]) s[i][j] = fmaf((v[i][j] - mean) * r, by[i][j], s[i][j]);
      if (live) put<T, N>(P.s, P.s_b, P.s_t, at, tm, s);
    } else {
      load(row + 1);
    }
    if (P.norm) {
      const Sums q = tm.join(tm.squares(s, P.norm == 2), turn, 1, P.C);
      const float r = rsqrtf(fmaf(q.sq, inv, P.eps));
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          s[i][j] = fmaf((s[i][j] - q.mean) * r, up[i][j], add[i][j]);
      if (live) put<T, N>(P.y, P.y_b, P.y_t, at, tm, s);
    }
    at.next(P.S);
  }
}

// The gradient; dynamic shared memory (where a weight's is wanted): the teams' dw and dpw,
// [teams of the block][2][C], every column of them one thread's own.
template <typename T, int kTeam, int N>
__global__ void __launch_bounds__(kTeam ? kTeamBlock : 512)
    block_norm_bwd_kernel(const __grid_constant__ NormParams P) {
  __shared__ Box box;
  extern __shared__ __align__(16) float wsum[];
  pdl_launch_dependents();
  const Team<kTeam, N> tm(P.C, &box);
  float *own = wsum + (kTeam ? (int)threadIdx.x / tm.kLanes : 0) * 2 * P.C;
  if (P.wpart)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (tm.on[i])
#pragma unroll
        for (int j = 0; j < 8; ++j) own[tm.col[i] + j] = own[P.C + tm.col[i] + j] = 0.f;
  pdl_wait();
  const long first = tm.id * P.L, end = first + P.L < P.T ? first + P.L : P.T;
  Place at{first / P.S, (int)(first % P.S)}, ahead = at;
  const float inv = 1.f / (float)P.C;
  float up[N][8], by[N][8], acc[3][N][8];
  long m = first / P.n, left = 0;
  Raw<T> sr[N], ur[N], gr[N], yr[N];
  auto load = [&](long row) {
    const bool live = row < end;
    if (P.norm) {
      fetch<T, N>(P.x, P.x_b, P.x_t, ahead, tm, live, sr);
      fetch<T, N>(P.dy, P.dy_b, P.dy_t, ahead, tm, live, yr);
    }
    if (P.dsum) fetch<T, N>(P.dsum, P.ds_b, P.ds_t, ahead, tm, live, gr);
    if (P.u) fetch<T, N>(P.u, P.u_b, P.u_t, ahead, tm, live, ur);
    ahead.next(P.S);
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
      float t[8], w[8];
      if (P.wpart) {  // what the modulations contribute to the weights' gradients
        load_vec(P.scale.p, P.mdt, m * P.scale.st + c, true, 0.f, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) own[c + j] = fmaf(1.f + t[j], acc[0][i][j], own[c + j]);
        load_vec(P.gate.p, P.mdt, m * P.gate.st + c, true, 1.f, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          own[P.C + c + j] = fmaf(P.rs * t[j], acc[2][i][j], own[P.C + c + j]);
      }
      if (!P.part) continue;
      if (!whole) {
#pragma unroll
        for (int k = 0; k < 3; ++k) store8(part + k * P.C + c, acc[k][i]);
        continue;
      }
      const int64_t o = m * P.C + c;
      if (P.dscale) {
        load_vec(P.w, P.wdt, c, true, 1.f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = w[j] * acc[0][i][j];
        store_vec(P.dscale, P.mdt, o, t);
      }
      if (P.dshift) store_vec(P.dshift, P.mdt, o, acc[1][i]);
      if (P.dgate) {
        load_vec(P.pw, P.wdt, c, true, 1.f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = P.rs * w[j] * acc[2][i][j];
        store_vec(P.dgate, P.mdt, o, t);
      }
    }
  };
  load(first);
  int turn = 0;
#pragma unroll 1
  for (long row = first; row < first + P.L; ++row, turn ^= 1) {
    const bool live = row < end;
    if (!kTeam && !live) break;
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
          for (int j = 0; j < 8; ++j) acc[k][i][j] = 0.f;
    }
    --left;
    float s[N][8], ds[N][8], v[N][8], d[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (P.norm) {
        unpack8(sr[i], s[i]);
        unpack8(yr[i], d[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ds[i][j] = 0.f;
      if (P.dsum) unpack8(gr[i], ds[i]);
      if (P.u) unpack8(ur[i], v[i]);
    }
    load(row + 1);
    if (P.norm) {
      float g[N][8];
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = d[i][j] * up[i][j];
      Sums q = tm.squares(s, P.norm == 2);
      tm.products(g, s, q.mean, 1.f, q);
      q = tm.join(q, turn, 0, P.C);
      const float r = rsqrtf(fmaf(q.sq, inv, P.eps));
      const float mg = P.norm == 2 ? q.d * inv : 0.f, mgn = q.dt * r * inv;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = (s[i][j] - q.mean) * r;
          if (live) {
            acc[0][i][j] = fmaf(d[i][j], n, acc[0][i][j]);
            acc[1][i][j] += d[i][j];
          }
          ds[i][j] = fmaf(r, g[i][j] - mg - n * mgn, ds[i][j]);
        }
    }
    if (live && P.dx) put<T, N>(P.dx, P.dx_b, P.dx_t, at, tm, ds);
    if (P.du || P.dgate || P.wpart) {
      float mean = 0.f, r = 1.f, me = 0.f, men = 0.f;
      if (P.post) {
        float e[N][8];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) e[i][j] = tm.on[i] ? ds[i][j] * by[i][j] : 0.f;
        Sums q = tm.squares(v, P.post == 2);
        tm.products(e, v, q.mean, 1.f, q);
        q = tm.join(q, turn, 1, P.C);
        mean = q.mean;
        r = rsqrtf(fmaf(q.sq, inv, P.eps));
        men = q.dt * r * inv;
        if (P.post == 2) me = q.d * inv;
      }
      if (P.u) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float n = (v[i][j] - mean) * r;
            if (live) acc[2][i][j] = fmaf(ds[i][j], n, acc[2][i][j]);
            ds[i][j] *= by[i][j];
            if (P.post) ds[i][j] = r * (ds[i][j] - me - n * men);
          }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) ds[i][j] *= by[i][j];
      }
      if (live && P.du) put<T, N>(P.du, P.du_b, P.du_t, at, tm, ds);
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
// weights.  32 columns a block, 32 teams at a time.
__global__ void __launch_bounds__(1024)
    block_norm_join_kernel(const __grid_constant__ NormParams P, int teams, int ny, long rows,
                           void *dw, void *dpw) {
  __shared__ float sums[3][32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
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
    for (int t = t0 + ty; t <= t1; t += 32) {
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
#pragma unroll
  for (int k = 0; k < 32; ++k) v += sums[ty][k][tx];
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
Form form_of(int C) {
  if (C <= 64) return {8, 1, kTeamBlock};
  if (C <= 128) return {16, 1, kTeamBlock};
  if (C <= 256) return {32, 1, kTeamBlock};
  if (C <= 4096) return {0, 1, (C + 255) / 256 * 32};
  return {0, 2, (C + 511) / 512 * 32};
}

// Teams and rows of a run.  Sized for GB300's 152 SMs, so that the workspace depends on the
// shape alone.
struct Runs {
  long teams;
  int L;
};
Runs runs_of(const NormShape &s, bool bwd) {
  const Form f = form_of(s.C);
  const long T = (long)s.B * s.S;
  const int per = f.team ? f.threads / f.team : 1;  // teams of a block
  const long most = 152L * ((bwd ? 512 : 1024) / f.threads) * per;
  long L = (T + most - 1) / most;
  if (bwd && L < 4) L = 4;  // shorter ones would have more partial sums than rows
  return {(T + L - 1) / L, (int)L};
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

struct NormLayout {
  size_t part, wpart, total;
};
NormLayout norm_layout(const NormShape &s) {
  const Runs r = runs_of(s, true);
  NormLayout w;
  w.part = 0;
  w.wpart = round_up((size_t)r.teams * 6 * s.C * sizeof(float));
  w.total = w.wpart + round_up((size_t)r.teams * 2 * s.C * sizeof(float));
  return w;
}

template <typename T, int kTeam, int N>
cudaError_t launch_typed(const NormParams &p, const Form &f, long teams, bool bwd,
                         cudaStream_t st) {
  const int per = kTeam ? f.threads / (kTeam ? kTeam : 1) : 1;
  const dim3 grid((unsigned)((teams + per - 1) / per)), block(f.threads);
  if (!bwd) return launch_pdl(block_norm_kernel<T, kTeam, N>, grid, block, 0, st, p);
  const size_t smem = p.wpart ? (size_t)per * 2 * p.C * sizeof(float) : 0;
  auto kern = block_norm_bwd_kernel<T, kTeam, N>;
  if (smem > 40000) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, grid, block, smem, st, p);
}

template <typename T>
cudaError_t launch_form(const NormParams &p, const Form &f, long teams, bool bwd,
                        cudaStream_t st) {
  switch (f.team) {
    case 8: return launch_typed<T, 8, 1>(p, f, teams, bwd, st);
    case 16: return launch_typed<T, 16, 1>(p, f, teams, bwd, st);
    case 32: return launch_typed<T, 32, 1>(p, f, teams, bwd, st);
  }
  return f.vecs == 1 ? launch_typed<T, 0, 1>(p, f, teams, bwd, st)
                     : launch_typed<T, 0, 2>(p, f, teams, bwd, st);
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
  const Form f = form_of(p.C);
  const Runs r = runs_of(a.shape, a.bwd);
  p.L = r.L;
  if (a.bwd) {
    const NormLayout w = norm_layout(a.shape);
    char *ws = static_cast<char *>(a.workspace);
    if (p.dgate || p.dscale || p.dshift) p.part = reinterpret_cast<float *>(ws + w.part);
    if (a.dw || a.dpw) p.wpart = reinterpret_cast<float *>(ws + w.wpart);
  }
  cudaError_t e = a.dt == NABLA_BF16 ? launch_form<__nv_bfloat16>(p, f, r.teams, a.bwd, st)
                                     : launch_form<float>(p, f, r.teams, a.bwd, st);
  if (e != cudaSuccess || !(p.part || p.wpart)) return e;
  // rows of the modulations that may lie in several runs: all, or one a border
  const long ny = !p.part ? 0 : a.rows <= r.teams - 1 ? a.rows : r.teams - 1;
  if (ny == 0 && !p.wpart) return e;
  const dim3 grid((unsigned)((p.C + 31) / 32), (unsigned)(ny + (p.wpart ? 1 : 0)));
  return launch_pdl(block_norm_join_kernel, grid, dim3(1024), 0, st, p, (int)r.teams, (int)ny,
                    (long)a.rows, a.dw, a.dpw);
}

}  // namespace nabla
