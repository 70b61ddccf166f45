// K13 -- bf16 differential attention backward on the tcgen05 tensor cores.
//
// With z_m = scale q_m k_m^T over a batch's states, P_m = softmax(z_m) = 2^(z_m log2(e) -
// lse_m), delta_m = dout . o_m and Y = dout v^T:
//   dz_1 = P_1 (Y - delta_1),  dz_2 = -lam P_2 (Y - delta_2),
//   dV = (P_1 - lam P_2)^T dout,  dK_m = scale dz_m^T q_m,  dQ_m = scale dz_m k_m,
//   dlam = -sum P_2 Y
// (the last from the map itself in fp32, rounded nowhere before).
//
// Two kernels, as in the cross attention's backward, their accumulators in TMEM from the
// first step of a unit to the last, and no atomics.  A step is 128 x 64: X_1, X_2 and Y are
// then 64 columns each, which leaves room beside the 256 columns of dK and dV to hand on P
// and dz in buffers of their own, so that a step's scores are formed while the softmax warps
// still work on the step before.
//
//  * dK, dV: unit = a tile of 128 states of one (batch, key head) over a run of subtiles of
//    64 packed query rows.  K and V stay in shared memory as A operands; X_m = K_m Q_m^T,
//    Y = V dO^T, W^T = (P_1 - lam P_2)^T and dz_m^T as bf16 in TMEM, then dV += W^T dO,
//    dK_m += dz_m^T Q_m.  One warp issues X and dV, another Y and dK.
//  * dQ: unit = a tile of 128 packed query rows over the batch's tiles of 64 states, or a
//    run of them: X_m = Q_m K_m^T, Y = dO V^T, dz_m in one of two buffers, dQ_m += dz_m K_m.
//    The rows' sums of P_2 Y are kept beside it.
//
// At D 64 a map's accumulator takes the products with both maps' 64 columns and half of them
// are not looked at: a product of 32 columns takes as long.
//
// Eight softmax warps: thread = TMEM lane, group grp takes columns 32 grp .. + 31.  States
// past kv_len: rows (columns, in dQ) of W and dz are 0 there; in dQ the rows of K that share
// the last 16-row MMA step with them are zeroed in shared memory.  Query rows that are none
// have lse = +inf, so P = 0.
//
// Bound by a step's chain, scores, dz, product with dz (dK / dV 2340 cycles for 128 x 64, of
// which the tensor pipe works 1280; dQ 2100): one set of scores is in work at a time, and a
// second one, 192 columns, would have to share those of dz.  (dK / dV hold all 512 columns at
// D 128, dQ 448.)  32768 tokens, 512 states, 12 heads, D 128: 208 us, tensor pipe active in 45%
// of the cycles, and 177 us, 39%.  Sixteen softmax warps: dK / dV 217 us, dQ 172, and the whole
// backward slower (525 us against 478).
// Every mbarrier wait is bounded (1 s), as in the forward.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "diff_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace nabla {
namespace {

using namespace tc;
using cross::kTile;
using diff::kStates;
using tcattn::add2;
using tcattn::f2;
using tcattn::fma2;
using tcattn::Ring;
using tcattn::unf2;

constexpr int kRowsArrays = 5;  // -lse_1, -lse_2, -delta_1, -delta_2, -lam of the packed rows

template <int D>
struct BCfg {
  static constexpr int kBoxes = D / 64;                          // 64-column swizzle boxes
  static constexpr int kBox = 128 * 128, kSmall = 64 * 128;      // of 128-row and 64-row tiles
  static constexpr int kTileBytes = kBoxes * kBox, kSmallBytes = kBoxes * kSmall;
  static constexpr int kSteps = D / 32;  // 16-column MMA steps of a map's scores
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kThreads = 384;
  static constexpr uint32_t kIdSS = idesc_bf16(128, 64, 0, 0);
  static constexpr uint32_t kIdTS = idesc_bf16(128, 64, 0, 1);   // dK_m, dQ_m
  static constexpr uint32_t kIdV = idesc_bf16(128, D, 0, 1);     // dV
  // B operand of a map's dK or dQ: its box, or (D 64) the one box
  static constexpr int kMapBox = D == 128 ? kSmall : 0;
  // dK / dV: K, V, rings of Q and dO subtiles and of the rows' numbers
  static constexpr int kRing = 4, kNums = kRowsArrays * 256;
  static constexpr int kOffK = 0, kOffV = kTileBytes, kOffQ = 2 * kTileBytes;
  static constexpr int kOffG = kOffQ + kRing * kSmallBytes;
  static constexpr int kOffL = kOffG + kRing * kSmallBytes;
  static constexpr int kOffSync1 = kOffL + kRing * kNums;
  static constexpr uint32_t kDV = 0, kDK = 128, kX1 = 256, kY1 = 384, kW = 448;  // W b: + 32 b
  // dQ: two Q tiles, dO, rings of K and V
  static constexpr int kK = 4, kV = 3;
  static constexpr int kOffG2 = 2 * kTileBytes, kOffK2 = 3 * kTileBytes;
  static constexpr int kOffV2 = kOffK2 + kK * kSmallBytes;
  static constexpr int kOffSync2 = kOffV2 + kV * kSmallBytes;
  static constexpr uint32_t kDQ = 0, kX2 = 128, kY2 = 256, kZ = 320;  // dz buffer b: + 64 b
};

struct KSync {
  uint64_t kv_full, kv_empty, q_full[4], q_empty[4], g_full[4], g_empty[4];
  uint64_t x_full, x_free, y_full, w_full[2], dv_done[2], z_full, dk_done, acc_full, acc_free;
  uint64_t drain;
  uint32_t tmem_slot;
  int abort;
};
struct QSync {
  uint64_t q_full[2], q_empty[2], g_full, g_empty, k_full[4], k_empty[4], k_raw;
  uint64_t v_full[3], v_empty[3];
  uint64_t x_full, y_full, x_free, y_free, z_full[2], acc_full, out_full, drain;
  uint32_t tmem_slot;
  int abort;
};
template <int D, bool kDQ>
constexpr int b_smem_bytes() {
  return kDQ ? BCfg<D>::kOffSync2 + (int)sizeof(QSync) : BCfg<D>::kOffSync1 + (int)sizeof(KSync);
}
static_assert(b_smem_bytes<128, false>() <= 232448, "shared memory budget (dK, dV)");
static_assert(b_smem_bytes<128, true>() <= 232448, "shared memory budget (dQ)");

struct BParams {
  __nv_bfloat16 *dq, *dk, *dv;  // [B, Sq, h, D], [B, Sk, hk, D]
  float *part;                  // dK / dV sums of the runs: [nsplit][2][B, Sk, hk, D]; or dQ's
  const float *rows;            // kRowsArrays x [B, hk, nsub, 64]
  size_t nrows;                 // of each
  float *t2;                    // [nsplit][2 groups][nrows]: sums of P_2 Y
  const int32_t *kv_len;
  int B, Sq, Sk, h, hk, G, tq, nsub, nsteps, nsplit;  // nsub: even; nsteps: subtiles with rows
  uint32_t units;
  cross::WalkStep walk;
  float scale, scale_log2;  // scale_log2 of |scale|, never 0
  uint32_t neg;             // kIdescNegA for a negative scale
  int *status;
};

__device__ __forceinline__ void b_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// A wait of a whole warp that goes on in step.
__device__ __forceinline__ bool b_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                       int *status) {
  return __all_sync(0xffffffffu, cross::thread_wait(bar, parity, abort, status));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair(const uint32_t *r) {
  return f2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ uint64_t ex2_pair(uint64_t v) {
  float a, b;
  unf2(v, a, b);
  return f2(ex2(a), ex2(b));
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
  float a, b;
  unf2(v, a, b);
  return pack_bf16x2(a, b);
}

// D (+)= A B^T over the 16-column steps [k0, k0 + n) of a 128-row tile A and a 64-row tile B.
template <int D, int n>
__device__ __forceinline__ void issue_ss(uint32_t d, uint64_t a, uint64_t b, int k0, uint32_t id) {
#pragma unroll
  for (int x = 0; x < n; ++x)
    mma_ss(d, a + diff::k_step(k0 + x, BCfg<D>::kBox), b + diff::k_step(k0 + x, BCfg<D>::kSmall),
           id, x > 0 ? 1u : 0u);
}

// ---------------------------------------------------------------- dK, dV

struct KUnit {
  int b, j, kt, sp, len, i0, n;  // n subtiles of query rows from i0
};
__device__ __forceinline__ KUnit k_unit(const BParams &P, const cross::Walk &w) {
  KUnit r{w.b, w.j, w.t, w.sp, cross::batch_len(P.kv_len, w.b, P.Sk), 0, 0};
  if (r.kt * kTile >= r.len) return r;  // no states: nothing to walk
  r.i0 = (int)((long)P.nsteps * r.sp / P.nsplit);
  r.n = (int)((long)P.nsteps * (r.sp + 1) / P.nsplit) - r.i0;
  return r;
}

// Warp 0, lane 0: the unit's K and V, then the steps' Q, dO and rows' numbers.
template <int D>
__device__ void k_load(const BParams &P, const CUtensorMap *mq, const CUtensorMap *mk,
                       const CUtensorMap *mv, const CUtensorMap *mg, uint8_t *smem, KSync *sy,
                       volatile int *abort) {
  using C = BCfg<D>;
  Ring<C::kRing> r;
  uint32_t g = 0, gq = 0, ku = 0;  // steps whose dO, whose Q has been asked for
  bool go = true;
  const uint32_t rows = (uint32_t)(P.G * P.tq) * 128 * C::kBoxes;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && go && !*abort;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const KUnit u = k_unit(P, w);
    cross::check_len(P.kv_len, u.b, P.Sk, P.status);
    if (u.n == 0) continue;
    go = cross::thread_wait(&sy->kv_empty, (ku & 1u) ^ 1u, abort, P.status);
    if (!go) break;
    mbar_expect_tx(&sy->kv_full, 2 * C::kTileBytes);
    for (int c = 0; c < C::kBoxes; ++c) {
      tma_load_4d(smem + C::kOffK + c * C::kBox, mk, &sy->kv_full, c * 64, u.j, u.kt * kTile, u.b);
      tma_load_4d(smem + C::kOffV + c * C::kBox, mv, &sy->kv_full, c * 64, u.j, u.kt * kTile, u.b);
    }
    ++ku;
    for (int i = 0; i < u.n && go; ++i, r.next()) {
      go = cross::thread_wait(&sy->q_empty[r.slot], r.phase ^ 1u, abort, P.status);
      if (!go) break;
      const int t0 = (u.i0 + i) * P.tq;
      mbar_expect_tx(&sy->q_full[r.slot], rows);
#pragma unroll
      for (int c = 0; c < C::kBoxes; ++c)
        tma_load_4d(smem + C::kOffQ + r.slot * C::kSmallBytes + c * C::kSmall, mq,
                    &sy->q_full[r.slot], c * 64, u.j * P.G, t0, u.b);
      ++gq;
      go = cross::thread_wait(&sy->g_empty[r.slot], r.phase ^ 1u, abort, P.status);
      if (!go) break;
      mbar_expect_tx(&sy->g_full[r.slot], rows + C::kNums);
      const float *at =
          P.rows + ((size_t)((uint32_t)u.b * P.hk + u.j) * P.nsub + u.i0 + i) * 64;
#pragma unroll 1
      for (int a = 0; a < kRowsArrays; ++a)
        bulk_load(smem + C::kOffL + r.slot * C::kNums + a * 256, at + a * P.nrows, 256,
                  &sy->g_full[r.slot]);
#pragma unroll
      for (int c = 0; c < C::kBoxes; ++c)
        tma_load_4d(smem + C::kOffG + r.slot * C::kSmallBytes + c * C::kSmall, mg,
                    &sy->g_full[r.slot], c * 64, u.j * P.G, t0, u.b);
      ++g;
    }
  }
  if (!go || *abort) {  // let copies in flight land before the CTA exits
    for (uint32_t e = gq > (uint32_t)C::kRing ? gq - C::kRing : 0u; e < gq; ++e)
      cross::thread_wait(&sy->q_full[e % C::kRing], (e / C::kRing) & 1u, nullptr, P.status);
    for (uint32_t e = g > (uint32_t)C::kRing ? g - C::kRing : 0u; e < g; ++e)
      cross::thread_wait(&sy->g_full[e % C::kRing], (e / C::kRing) & 1u, nullptr, P.status);
    if (ku > 0) cross::thread_wait(&sy->kv_full, (ku - 1) & 1u, nullptr, P.status);
  }
}

// Warp 1: X_m = K_m Q_m^T of a step as soon as the softmax warps hold the last one's, and
// dV += W^T dO.
template <int D>
__device__ void k_mma_x(const BParams &P, uint8_t *smem, KSync *sy, uint32_t tmem,
                        volatile int *abort) {
  using C = BCfg<D>;
  const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
  const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
  const uint64_t g_mn = smem_desc_sw128(smem_u32(smem + C::kOffG), C::kSmall, 1024);
  Ring<C::kRing> xr, r;  // of X's step, of dV's
  uint32_t gx = 0, g = 0, ku = 0;
  bool ok = true;
  auto issue_x = [&](bool last) {
    ok = b_wait(&sy->q_full[xr.slot], xr.phase, abort, P.status) &&
         b_wait(&sy->x_free, (gx & 1u) ^ 1u, abort, P.status);
    if (!ok) return;
    tc_fence_after();
    if (elect_one()) {
      const uint64_t qd = q_desc + (uint64_t)((xr.slot * C::kSmallBytes) >> 4);
#pragma unroll
      for (int m = 0; m < 2; ++m)
        issue_ss<D, C::kSteps>(tmem + C::kX1 + m * 64, k_desc, qd, m * C::kSteps,
                               C::kIdSS | P.neg);
      mma_commit(&sy->x_full);
      if (last) mma_commit(&sy->kv_empty);
    }
    __syncwarp();
    xr.next();
    ++gx;
  };
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && ok;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const KUnit u = k_unit(P, w);
    if (u.n == 0) continue;
    ok = b_wait(&sy->kv_full, ku & 1u, abort, P.status);
    if (ok) issue_x(u.n == 1);
    // the last unit's rows of dK and dV have been read
    if (ok && ku > 0) ok = b_wait(&sy->acc_free, (ku - 1) & 1u, abort, P.status);
    for (int i = 0; i < u.n && ok; ++i, ++g, r.next()) {
      if (i + 1 < u.n) issue_x(i + 2 == u.n);
      ok = ok && b_wait(&sy->g_full[r.slot], r.phase, abort, P.status) &&
           b_wait(&sy->w_full[g & 1u], (g >> 1) & 1u, abort, P.status);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t b = g_mn + (uint64_t)((r.slot * C::kSmallBytes) >> 4);
        const uint32_t a = tmem + C::kW + (g & 1u) * 32;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(tmem + C::kDV, a + kk * 8, b + (uint64_t)((kk * 16 * 128) >> 4), C::kIdV,
                 i > 0 || kk > 0 ? 1u : 0u);
        mma_commit(&sy->dv_done[g & 1u]);
        mma_commit(&sy->g_empty[r.slot]);
        if (i + 1 == u.n) mma_commit(&sy->acc_full);
      }
      __syncwarp();
    }
    ++ku;
  }
  if (elect_one()) mma_commit(&sy->drain);  // never exit with MMAs in flight
  __syncwarp();
  cross::thread_wait(&sy->drain, 0, nullptr, P.status);
}

// Warp 2: Y = V dO^T, over the columns whose dz the last step's dK has read, and
// dK_m += dz_m^T Q_m.
template <int D>
__device__ void k_mma_y(const BParams &P, uint8_t *smem, KSync *sy, uint32_t tmem,
                        volatile int *abort) {
  using C = BCfg<D>;
  const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + C::kOffV), 16, 1024);
  const uint64_t g_desc = smem_desc_sw128(smem_u32(smem + C::kOffG), 16, 1024);
  const uint64_t q_mn = smem_desc_sw128(smem_u32(smem + C::kOffQ), C::kSmall, 1024);
  Ring<C::kRing> yr, r;  // of Y's step, of dK's
  uint32_t g = 0, ku = 0;
  bool ok = true;
  auto issue_y = [&](bool last) {  // of step g; dK of step g - 1 is issued
    ok = b_wait(&sy->g_full[yr.slot], yr.phase, abort, P.status) &&
         (g == 0 || b_wait(&sy->dk_done, (g - 1) & 1u, abort, P.status));
    if (!ok) return;
    tc_fence_after();
    if (elect_one()) {
      issue_ss<D, D / 16>(tmem + C::kY1, v_desc,
                          g_desc + (uint64_t)((yr.slot * C::kSmallBytes) >> 4), 0, C::kIdSS);
      mma_commit(&sy->y_full);
      mma_commit(&sy->g_empty[yr.slot]);
      if (last) mma_commit(&sy->kv_empty);
    }
    __syncwarp();
    yr.next();
  };
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && ok;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const KUnit u = k_unit(P, w);
    if (u.n == 0) continue;
    ok = b_wait(&sy->kv_full, ku & 1u, abort, P.status);
    if (ok) issue_y(u.n == 1);
    if (ok && ku > 0) ok = b_wait(&sy->acc_free, (ku - 1) & 1u, abort, P.status);
    for (int i = 0; i < u.n && ok; ++i, r.next()) {
      ok = b_wait(&sy->q_full[r.slot], r.phase, abort, P.status) &&
           b_wait(&sy->z_full, g & 1u, abort, P.status);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t b = q_mn + (uint64_t)((r.slot * C::kSmallBytes) >> 4);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            // dz of a group's 32 query rows: 16 columns a map, from 32 grp on
            mma_ts(tmem + C::kDK + m * 64, tmem + C::kY1 + (kk >> 1) * 32 + m * 16 + (kk & 1) * 8,
                   b + (uint64_t)((m * C::kMapBox + kk * 16 * 128) >> 4), C::kIdTS,
                   i > 0 || kk > 0 ? 1u : 0u);
        mma_commit(&sy->dk_done);
        mma_commit(&sy->q_empty[r.slot]);
        if (i + 1 == u.n) mma_commit(&sy->acc_full);
      }
      __syncwarp();
      ++g;
      if (i + 1 < u.n) issue_y(i + 2 == u.n);
    }
    ++ku;
  }
  if (elect_one()) mma_commit(&sy->drain);
  __syncwarp();
  cross::thread_wait(&sy->drain, 0, nullptr, P.status);
}

// Column of dK's or dQ's accumulator that holds column c of a map's half.
template <int D>
__device__ __forceinline__ uint32_t acc_col(int map, int c) {
  return D == 128 ? (uint32_t)c : (uint32_t)(map * 64 + c);
}

// Nothing for a state that is none, whatever was computed.
__device__ __forceinline__ void none(bool act, uint32_t (&v)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = act ? v[e] : 0u;
}

// Warps 4-11: W^T and dz^T of every step, then the unit's rows of dK and dV.  Thread =
// state, columns = query rows, whose numbers come with dO.
template <int D>
__device__ void k_softmax(const BParams &P, uint8_t *smem, KSync *sy, uint32_t tmem,
                          volatile int *abort) {
  using C = BCfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
  const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16);
  const uint32_t xa = at + C::kX1 + grp * 32, ya = at + C::kY1 + grp * 32;
  const uint64_t sc2 = f2(P.scale_log2, P.scale_log2);
  Ring<C::kRing> r;
  uint32_t g = 0, ku = 0;
  bool live = true;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units; i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const KUnit u = k_unit(P, w);
    const int state = u.kt * kTile + row;
    const bool act = state < u.len, all_act = __all_sync(0xffffffffu, act);
    for (int i = 0; i < u.n; ++i, ++g, r.next()) {
      const bool g_over = diff::is_over(&sy->g_full[r.slot], r.phase);
      const bool x_over = diff::is_over(&sy->x_full, g & 1u);
      // the product of two steps before has read W's buffer
      const bool w_over = diff::is_over(&sy->dv_done[g & 1u], ((g >> 1) & 1u) ^ 1u);
      diff::wait_unless(g_over, live, &sy->g_full[r.slot], r.phase, abort, P.status);
      diff::wait_unless(x_over, live, &sy->x_full, g & 1u, abort, P.status);
      tc_fence_after();
      // per query row, 64 apart: -lse_1, -lse_2, -delta_1, -delta_2, -lam
      const float *num = reinterpret_cast<const float *>(smem + C::kOffL + r.slot * C::kNums) +
                         grp * 32;
      uint32_t x1[32], x2[32];
      tmem_ld32(xa, x1);
      tmem_ld32(xa + 64, x2);
      tmem_wait_ld();
      reg_fence(x1);
      reg_fence(x2);
      tc_fence_before();
      b_arrive(&sy->x_free, lane);
      uint64_t p1[16], p2[16];  // P_1, -lam P_2
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const ulonglong2 l1 = *reinterpret_cast<const ulonglong2 *>(num + e);
        const ulonglong2 l2 = *reinterpret_cast<const ulonglong2 *>(num + 64 + e);
        const ulonglong2 lm = *reinterpret_cast<const ulonglong2 *>(num + 256 + e);
        p1[e / 2] = ex2_pair(fma2(pair(x1 + e), sc2, l1.x));
        p1[e / 2 + 1] = ex2_pair(fma2(pair(x1 + e + 2), sc2, l1.y));
        p2[e / 2] = mul2(ex2_pair(fma2(pair(x2 + e), sc2, l2.x)), lm.x);
        p2[e / 2 + 1] = mul2(ex2_pair(fma2(pair(x2 + e + 2), sc2, l2.y)), lm.y);
        pk[e / 2] = pack_pair(add2(p1[e / 2], p2[e / 2]));
        pk[e / 2 + 1] = pack_pair(add2(p1[e / 2 + 1], p2[e / 2 + 1]));
      }
      if (!all_act) none(act, pk);
      const bool y_over = diff::is_over(&sy->y_full, g & 1u);
      diff::wait_unless(w_over, live, &sy->dv_done[g & 1u], ((g >> 1) & 1u) ^ 1u, abort,
                        P.status);
      tc_fence_after();
      tmem_st16(at + C::kW + (g & 1u) * 32 + grp * 16, pk);
      tmem_wait_st();
      tc_fence_before();
      b_arrive(&sy->w_full[g & 1u], lane);
      diff::wait_unless(y_over, live, &sy->y_full, g & 1u, abort, P.status);
      tc_fence_after();
      tmem_ld32(ya, x1);
      tmem_wait_ld();
      reg_fence(x1);
      uint32_t z2[16];
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const ulonglong2 d1 = *reinterpret_cast<const ulonglong2 *>(num + 128 + e);
        const ulonglong2 d2 = *reinterpret_cast<const ulonglong2 *>(num + 192 + e);
        const uint64_t y0 = pair(x1 + e), y1 = pair(x1 + e + 2);
        pk[e / 2] = pack_pair(mul2(p1[e / 2], add2(y0, d1.x)));
        pk[e / 2 + 1] = pack_pair(mul2(p1[e / 2 + 1], add2(y1, d1.y)));
        z2[e / 2] = pack_pair(mul2(p2[e / 2], add2(y0, d2.x)));
        z2[e / 2 + 1] = pack_pair(mul2(p2[e / 2 + 1], add2(y1, d2.y)));
      }
      if (!all_act) {
        none(act, pk);
        none(act, z2);
      }
      tmem_st16(ya, pk);  // over columns of Y that this thread has read
      tmem_st16(ya + 16, z2);
      tmem_wait_st();
      tc_fence_before();
      b_arrive(&sy->z_full, lane);
      if (lane == 0) mbar_arrive(&sy->g_empty[r.slot]);  // the rows' numbers have been read
    }
    // ---- the unit's rows: dV, dK (scaled), or their sums over this run; 0 past the length
    if (u.n > 0) {
      cross::warp_wait(live, &sy->acc_full, ku & 1u, abort, P.status);
      tc_fence_after();
    }
    if (u.n > 0 || P.nsplit == 1) {
      const size_t orow = (((size_t)u.b * P.Sk + state) * P.hk + u.j) * D;
      const size_t all = (size_t)P.B * P.Sk * P.hk * D;
#pragma unroll 1
      for (int x = 0; x < D / 16; ++x) {  // 16 columns; the first half dK's, the other dV's
        const bool dv = x >= D / 32;
        const int c = grp * (D / 2) + (dv ? x - D / 32 : x) * 16;
        uint32_t t[16];
        if (u.n > 0) {
          tmem_ld16(at + (dv ? C::kDV + c : C::kDK + acc_col<D>(grp, c)), t);
          tmem_wait_ld();
          reg_fence16(t);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) t[e] = 0u;
        }
        if (state >= P.Sk) continue;
        const float m = dv ? 1.f : P.scale;
        if (P.nsplit > 1) {
          float4 *o =
              reinterpret_cast<float4 *>(P.part + ((size_t)u.sp * 2 + dv) * all + orow + c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = make_float4(__uint_as_float(t[4 * e]) * m, __uint_as_float(t[4 * e + 1]) * m,
                               __uint_as_float(t[4 * e + 2]) * m,
                               __uint_as_float(t[4 * e + 3]) * m);
        } else {
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = pack_bf16x2(__uint_as_float(t[2 * e]) * m, __uint_as_float(t[2 * e + 1]) * m);
          uint4 *o = reinterpret_cast<uint4 *>((dv ? P.dv : P.dk) + orow + c);
          o[0] = make_uint4(v[0], v[1], v[2], v[3]);
          o[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
      }
    }
    if (u.n > 0) {
      tc_fence_before();
      b_arrive(&sy->acc_free, lane);
      ++ku;
    }
  }
}

// Rows of `n` 64-row pieces (128 bytes a row) that no box fills (G not dividing 64) as zeros.
__device__ __forceinline__ void zero_gap(uint8_t *tiles, int n, int used) {
  const int per = (64 - used) * 8;
  for (int e = threadIdx.x; e < per * n; e += blockDim.x) {
    const int sub = e / per, to = e - sub * per;
    *reinterpret_cast<uint4 *>(tiles + sub * 64 * 128 + used * 128 + to * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    diff_dkv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg,
                    const __grid_constant__ BParams P) {
  using C = BCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  KSync *sy = reinterpret_cast<KSync *>(smem + C::kOffSync1);
  volatile int *abort = &sy->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles would be misread
    if (threadIdx.x == 0) atomicCAS(P.status, kDevOk, kDevTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&sy->kv_full, 1);
    mbar_init(&sy->kv_empty, 2);  // both chains
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&sy->q_full[i], 1);
      mbar_init(&sy->q_empty[i], 1);  // dK; X is done long before
      mbar_init(&sy->g_full[i], 1);
      mbar_init(&sy->g_empty[i], 2 + 8);  // both chains, the softmax warps
    }
    mbar_init(&sy->x_full, 1);
    mbar_init(&sy->x_free, 8);
    mbar_init(&sy->y_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sy->w_full[i], 8);
      mbar_init(&sy->dv_done[i], 1);
    }
    mbar_init(&sy->z_full, 8);
    mbar_init(&sy->dk_done, 1);
    mbar_init(&sy->acc_full, 2);
    mbar_init(&sy->acc_free, 8);
    mbar_init(&sy->drain, 2);
    sy->abort = 0;
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mg);
    fence_barrier_init();
  }
  zero_gap(smem + C::kOffQ, 2 * C::kRing * C::kBoxes, P.G * P.tq);
  fence_async_smem();
  if (warp == 1) tmem_alloc(&sy->tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sy->tmem_slot;
  pdl_wait();
  if (warp == 0) {
    if (lane == 0) k_load<D>(P, &mq, &mk, &mv, &mg, smem, sy, abort);
    __syncwarp();
  } else if (warp == 1) {
    k_mma_x<D>(P, smem, sy, tmem, abort);
  } else if (warp == 2) {
    k_mma_y<D>(P, smem, sy, tmem, abort);
  } else if (warp >= 4) {
    k_softmax<D>(P, smem, sy, tmem, abort);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- dQ

struct QUnit {
  int b, j, qt, sp, len, t0, n;  // n state tiles from t0
};
__device__ __forceinline__ QUnit q_unit(const BParams &P, const cross::Walk &w) {
  QUnit r{w.b, w.j, w.t, w.sp, cross::batch_len(P.kv_len, w.b, P.Sk), 0, 0};
  const int nt = (r.len + kStates - 1) / kStates;
  r.t0 = (int)((long)nt * r.sp / P.nsplit);
  r.n = (int)((long)nt * (r.sp + 1) / P.nsplit) - r.t0;
  return r;
}

// Warp 0, lane 0: the units' Q (a unit ahead) and dO.
template <int D>
__device__ void q_load(const BParams &P, const CUtensorMap *mq, const CUtensorMap *mg,
                       uint8_t *smem, QSync *sy, volatile int *abort) {
  using C = BCfg<D>;
  uint32_t ku = 0;  // units whose Q and dO have been asked for
  bool go = true;
  const uint32_t rows = (uint32_t)(P.G * P.tq) * 128 * 2 * C::kBoxes;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && go && !*abort;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const QUnit u = q_unit(P, w);
    if (u.n == 0) continue;
#pragma unroll 1
    for (int which = 0; which < 2 && go; ++which) {  // Q, then dO
      uint64_t *full = which ? &sy->g_full : &sy->q_full[ku & 1u];
      go = which ? cross::thread_wait(&sy->g_empty, (ku & 1u) ^ 1u, abort, P.status)
                 : cross::thread_wait(&sy->q_empty[ku & 1u], ((ku >> 1) & 1u) ^ 1u, abort,
                                      P.status);
      if (!go) break;
      uint8_t *tile = smem + (which ? C::kOffG2 : (int)(ku & 1u) * C::kTileBytes);
      mbar_expect_tx(full, rows);
#pragma unroll 1
      for (int x = 0; x < 2 * C::kBoxes; ++x)
        tma_load_4d(tile + (x >> 1) * C::kBox + (x & 1) * 64 * 128, which ? mg : mq, full,
                    (x >> 1) * 64, u.j * P.G, (u.qt * 2 + (x & 1)) * P.tq, u.b);
      ku += which;
    }
  }
  if (!go || *abort) {
    // copies in flight: the last two units' Q and the last dO; where the loop broke between
    // the two, one Q more
    for (uint32_t e = ku > 2u ? ku - 2u : 0u; e < ku; ++e)
      cross::thread_wait(&sy->q_full[e & 1u], (e >> 1) & 1u, nullptr, P.status);
    if (ku > 0) cross::thread_wait(&sy->g_full, (ku - 1) & 1u, nullptr, P.status);
    if (!go) cross::thread_wait(&sy->q_full[ku & 1u], (ku >> 1) & 1u, nullptr, P.status);
  }
}

// Warp 3: K and V of every step.  A K tile whose last 16 rows reach past the length comes
// in on k_raw: the warp zeroes those rows, then hands the tile on.
template <int D>
__device__ void q_load_kv(const BParams &P, const CUtensorMap *mk, const CUtensorMap *mv,
                          uint8_t *smem, QSync *sy, volatile int *abort) {
  using C = BCfg<D>;
  const int lane = threadIdx.x & 31;
  Ring<C::kK> kr;
  Ring<C::kV> vr;
  uint32_t g = 0, raw = 0;
  bool go = true;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && go;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const QUnit u = q_unit(P, w);
    if (lane == 0) cross::check_len(P.kv_len, u.b, P.Sk, P.status);
    for (int t = 0; t < u.n && go; ++t, ++g, kr.next(), vr.next()) {
      const int rows = u.len - (u.t0 + t) * kStates;
      const int end = diff::steps16(u.len, u.t0 + t) * 16;
      const bool mend = rows < end && u.len < P.Sk;  // zero K's rows [rows, end)
      uint8_t *tile = smem + C::kOffK2 + kr.slot * C::kSmallBytes;
      bool ok = true;
      if (lane == 0) {
        ok = !*abort && cross::thread_wait(&sy->k_empty[kr.slot], kr.phase ^ 1u, abort, P.status);
        if (ok) {
          uint64_t *bar = mend ? &sy->k_raw : &sy->k_full[kr.slot];
          mbar_expect_tx(bar, C::kSmallBytes);
          for (int c = 0; c < C::kBoxes; ++c)
            tma_load_4d(tile + c * C::kSmall, mk, bar, c * 64, u.j, (u.t0 + t) * kStates, u.b);
          if (mend) ok = cross::thread_wait(&sy->k_raw, raw & 1u, nullptr, P.status);
        }
      }
      go = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!go) break;
      if (mend) {
        ++raw;
        diff::zero_rows<C::kBoxes>(tile, C::kSmall, rows, end);
        if (lane == 0) mbar_arrive(&sy->k_full[kr.slot]);
      }
      if (lane == 0) {
        ok = cross::thread_wait(&sy->v_empty[vr.slot], vr.phase ^ 1u, abort, P.status);
        if (ok) {
          mbar_expect_tx(&sy->v_full[vr.slot], C::kSmallBytes);
          for (int c = 0; c < C::kBoxes; ++c)
            tma_load_4d(smem + C::kOffV2 + vr.slot * C::kSmallBytes + c * C::kSmall, mv,
                        &sy->v_full[vr.slot], c * 64, u.j, (u.t0 + t) * kStates, u.b);
        } else {  // the K tile of this step is in flight
          cross::thread_wait(&sy->k_full[kr.slot], kr.phase, nullptr, P.status);
        }
      }
      go = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!go) break;
    }
  }
  if (lane == 0 && (!go || *abort)) {
    for (uint32_t e = g > (uint32_t)C::kK ? g - C::kK : 0u; e < g; ++e)
      cross::thread_wait(&sy->k_full[e % C::kK], (e / C::kK) & 1u, nullptr, P.status);
    for (uint32_t e = g > (uint32_t)C::kV ? g - C::kV : 0u; e < g; ++e)
      cross::thread_wait(&sy->v_full[e % C::kV], (e / C::kV) & 1u, nullptr, P.status);
  }
}

// Warp 1, one thread: all products: X_m, Y of every step, each over the last step's once the
// softmax warps hold that, and dQ_m += dz_m K_m of the step before.  A step's X is
// committed after the dQ of two steps before, so x_full also says that the dz buffer is
// free; and dz of a unit's first step comes after the last unit's rows were read, so it
// says that dQ may be written over.  Y of a unit's first step comes after that dQ, since
// it may still wait for dO.
template <int D>
__device__ void q_mma(const BParams &P, uint8_t *smem, QSync *sy, uint32_t tmem,
                      volatile int *abort) {
  using C = BCfg<D>;
  const uint64_t q_desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t g_desc = smem_desc_sw128(smem_u32(smem + C::kOffG2), 16, 1024);
  const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + C::kOffK2), 16, 1024);
  const uint64_t k_mn = smem_desc_sw128(smem_u32(smem + C::kOffK2), C::kSmall, 1024);
  const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + C::kOffV2), 16, 1024);
  Ring<2> q;
  Ring<C::kK> kr, kd;           // of X's step, and of dQ's
  Ring<C::kV> vr;
  uint32_t g = 0, ku = 0;       // steps of X so far
  int left = 0;                 // states from the first of dQ's next tile on
  bool first = true, ok = true;  // dQ's next step begins a unit
  auto issue_dq = [&](bool last) {  // of step g - 1
    ok = cross::thread_wait(&sy->z_full[(g - 1) & 1u], ((g - 1) >> 1) & 1u, abort, P.status);
    if (!ok) return;
    tc_fence_after();
    const uint32_t a = tmem + C::kZ + ((g - 1) & 1u) * 64;
    const uint64_t b = k_mn + (uint64_t)((kd.slot * C::kSmallBytes) >> 4);
    const int k16 = left >= kStates ? 4 : (left + 15) >> 4;  // the last tile: its states only
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint64_t bm = b + (uint64_t)((m * C::kMapBox) >> 4);
      if (k16 == 4) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(tmem + C::kDQ + m * 64, a + m * 32 + kk * 8,
                 bm + (uint64_t)((kk * 16 * 128) >> 4), C::kIdTS, kk > 0 || !first ? 1u : 0u);
      } else {
#pragma unroll 1
        for (int kk = 0; kk < k16; ++kk)
          mma_ts(tmem + C::kDQ + m * 64, a + m * 32 + kk * 8,
                 bm + (uint64_t)((kk * 16 * 128) >> 4), C::kIdTS, kk > 0 || !first ? 1u : 0u);
      }
    }
    mma_commit(&sy->k_empty[kd.slot]);
    if (last) mma_commit(&sy->acc_full);
    kd.next();
    first = last;
  };
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && ok;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const QUnit u = q_unit(P, w);
    if (u.n == 0) continue;
    ok = cross::thread_wait(&sy->q_full[q.slot], q.phase, abort, P.status);
    for (int t = 0; t < u.n && ok; ++t, ++g) {
      ok = cross::thread_wait(&sy->k_full[kr.slot], kr.phase, abort, P.status) &&
           cross::thread_wait(&sy->x_free, (g & 1u) ^ 1u, abort, P.status);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int m = 0; m < 2; ++m)
        issue_ss<D, C::kSteps>(tmem + C::kX2 + m * 64,
                               q_desc + (uint64_t)((q.slot * C::kTileBytes) >> 4),
                               k_desc + (uint64_t)((kr.slot * C::kSmallBytes) >> 4),
                               m * C::kSteps, C::kIdSS | P.neg);
      mma_commit(&sy->x_full);
      kr.next();
      if (t == 0) {
        if (g > 0) issue_dq(true);  // the last unit's last step
        ok = ok && cross::thread_wait(&sy->g_full, ku & 1u, abort, P.status);
      }
      ok = ok && cross::thread_wait(&sy->v_full[vr.slot], vr.phase, abort, P.status) &&
           cross::thread_wait(&sy->y_free, (g & 1u) ^ 1u, abort, P.status);
      if (!ok) break;
      tc_fence_after();
      issue_ss<D, D / 16>(tmem + C::kY2, g_desc,
                          v_desc + (uint64_t)((vr.slot * C::kSmallBytes) >> 4), 0, C::kIdSS);
      mma_commit(&sy->y_full);
      mma_commit(&sy->v_empty[vr.slot]);
      vr.next();
      if (t + 1 == u.n) mma_commit(&sy->g_empty);
      if (t > 0) issue_dq(false);
      left = u.len - (u.t0 + t) * kStates;
    }
    q.next();
    ++ku;
  }
  if (ok && g > 0) issue_dq(true);
  mma_commit(&sy->drain);
  cross::thread_wait(&sy->drain, 0, nullptr, P.status);
}

// Warp 2: hands the units' rows from their Q tiles to the TMA, and the tiles back to the
// loader once they have been read.
template <int D>
__device__ void q_store(const BParams &P, const CUtensorMap *mo, const uint8_t *smem, QSync *sy,
                        volatile int *abort) {
  using C = BCfg<D>;
  uint32_t ku = 0;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units; i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const QUnit u = q_unit(P, w);
    if (u.n == 0) continue;
    if (!cross::thread_wait(&sy->out_full, ku & 1u, abort, P.status)) break;
    const uint8_t *tile = smem + (ku & 1u) * C::kTileBytes;
    if (P.nsplit == 1) {  // (a run's sums do not come this way)
#pragma unroll 1
      for (int x = 0; x < 2 * C::kBoxes; ++x) {
        const int t0 = (u.qt * 2 + (x & 1)) * P.tq;
        if (t0 < P.Sq)
          tma_store_4d(mo, tile + (x >> 1) * C::kBox + (x & 1) * 64 * 128, (x >> 1) * 64,
                       u.j * P.G, t0, u.b);
      }
      bulk_commit();
      bulk_wait_read();
    }
    mbar_arrive(&sy->q_empty[ku & 1u]);
    ++ku;
  }
  bulk_wait_all();
}

// Warps 4-11: dz of every step, and the units' rows of dQ (through the unit's Q tile, which
// no MMA reads any more).  Thread = query row, columns = states.  A unit's rows are written
// in the first step of the next unit, after its exponentials, so that the last dQ product
// runs meanwhile.
template <int D>
__device__ void q_softmax(const BParams &P, uint8_t *smem, QSync *sy, uint32_t tmem,
                          volatile int *abort) {
  using C = BCfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane, r64 = row & 63;
  const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16);
  const uint64_t sc2 = f2(P.scale_log2, P.scale_log2);
  const int tok = r64 / P.G, head = r64 - tok * P.G;
  uint32_t g = 0, ku = 0;
  bool live = true, x_over = false;
  QUnit last{};  // unit ku - 1
  auto write_rows = [&]() {  // of unit ku - 1, over its Q; a run's sums to their part
    cross::warp_wait(live, &sy->acc_full, (ku - 1) & 1u, abort, P.status);
    tc_fence_after();
    uint8_t *tile = smem + ((ku - 1) & 1u) * C::kTileBytes + row * 128;
    const int token = (last.qt * 2 + (row >> 6)) * P.tq + tok, hh = last.j * P.G + head;
    float *part = nullptr;
    if (P.nsplit > 1 && tok < P.tq && token < P.Sq)
      part = P.part + ((((size_t)last.sp * P.B + last.b) * P.Sq + token) * P.h + hh) * D;
#pragma unroll 1
    for (int x = 0; x < D / 64; ++x) {  // 32 columns of this group's D / 2
      const int c = grp * (D / 2) + x * 32;
      uint32_t t[32];
      tmem_ld32(at + C::kDQ + acc_col<D>(grp, c), t);
      tmem_wait_ld();
      reg_fence(t);
      if (P.nsplit > 1) {
        if (part)
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4 *>(part + c + e) =
                make_uint4(t[e], t[e + 1], t[e + 2], t[e + 3]);
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          v[y] = pack_bf16x2(__uint_as_float(t[8 * e + 2 * y]) * P.scale,
                             __uint_as_float(t[8 * e + 2 * y + 1]) * P.scale);
        const int piece = (c >> 3) + e;  // 16-byte piece of the row, swizzled in its box
        *reinterpret_cast<uint4 *>(tile + (piece >> 3) * C::kBox +
                                   (((piece & 7) ^ (row & 7)) << 4)) =
            make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    fence_async_smem();
    b_arrive(&sy->out_full, lane);
  };
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units; i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const QUnit c = q_unit(P, w);
    const size_t prow = ((size_t)((uint32_t)w.b * P.hk + w.j) * P.nsub + w.t * 2) * 64 + row;
    float t2 = 0.f;
    if (c.n > 0) {
      float n[kRowsArrays];
#pragma unroll
      for (int i = 0; i < kRowsArrays; ++i) n[i] = __ldg(P.rows + i * P.nrows + prow);
      const uint64_t l1 = f2(n[0], n[0]), l2 = f2(n[1], n[1]), d1 = f2(n[2], n[2]),
                     d2 = f2(n[3], n[3]), by = f2(n[4], n[4]);
      for (int t = 0; t < c.n; ++t, ++g) {
        const int mine = c.len - (c.t0 + t) * kStates - grp * 32;  // own columns that are states
        diff::wait_unless(x_over, live, &sy->x_full, g & 1u, abort, P.status);
        tc_fence_after();
        uint32_t x1[32], x2[32];
        tmem_ld32(at + C::kX2 + grp * 32, x1);
        tmem_ld32(at + C::kX2 + 64 + grp * 32, x2);
        tmem_wait_ld();
        reg_fence(x1);
        reg_fence(x2);
        tc_fence_before();
        b_arrive(&sy->x_free, lane);
        uint64_t p1[16], p2[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          p1[e] = ex2_pair(fma2(pair(x1 + 2 * e), sc2, l1));
          p2[e] = ex2_pair(fma2(pair(x2 + 2 * e), sc2, l2));
        }
        const bool y_over = diff::is_over(&sy->y_full, g & 1u);
        if (t == 0 && ku > 0) write_rows();
        diff::wait_unless(y_over, live, &sy->y_full, g & 1u, abort, P.status);
        tc_fence_after();
        tmem_ld32(at + C::kY2 + grp * 32, x1);
        tmem_wait_ld();
        reg_fence(x1);
        tc_fence_before();
        b_arrive(&sy->y_free, lane);
        // the next step's scores, asked for ahead of this one's products
        x_over = diff::is_over(&sy->x_full, (g & 1u) ^ 1u);
        if (mine < 32) {  // past the length: nothing, whatever was computed there
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, b, u, v;
            unf2(p1[e], a, b);
            unf2(p2[e], u, v);
            p1[e] = f2(2 * e < mine ? a : 0.f, 2 * e + 1 < mine ? b : 0.f);
            p2[e] = f2(2 * e < mine ? u : 0.f, 2 * e + 1 < mine ? v : 0.f);
            x1[2 * e] = 2 * e < mine ? x1[2 * e] : 0u;
            x1[2 * e + 1] = 2 * e + 1 < mine ? x1[2 * e + 1] : 0u;
          }
        }
        uint32_t z1[16], z2[16];
        uint64_t sum = f2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t y = pair(x1 + 2 * e);
          sum = fma2(p2[e], y, sum);
          z1[e] = pack_pair(mul2(p1[e], add2(y, d1)));
          z2[e] = pack_pair(mul2(mul2(p2[e], by), add2(y, d2)));
        }
        float s0, s1;
        unf2(sum, s0, s1);
        t2 += s0 + s1;
        const uint32_t za = at + C::kZ + (g & 1u) * 64 + grp * 16;
        tmem_st16(za, z1);
        tmem_st16(za + 32, z2);
        tmem_wait_st();
        tc_fence_before();
        b_arrive(&sy->z_full[g & 1u], lane);
      }
      last = c;
      ++ku;
    } else {
      const int token = (c.qt * 2 + (row >> 6)) * P.tq + tok, hh = c.j * P.G + head;
      if (P.nsplit == 1 && tok < P.tq && token < P.Sq) {
        uint4 *o = reinterpret_cast<uint4 *>(
            P.dq + (((size_t)c.b * P.Sq + token) * P.h + hh) * D + grp * (D / 2));
#pragma unroll 1
        for (int e = 0; e < D / 16; ++e) o[e] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    P.t2[(size_t)(c.sp * 2 + grp) * P.nrows + prow] = t2;
  }
  if (ku > 0) write_rows();
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    diff_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg,
                   const __grid_constant__ CUtensorMap mo, const __grid_constant__ BParams P) {
  using C = BCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  QSync *sy = reinterpret_cast<QSync *>(smem + C::kOffSync2);
  volatile int *abort = &sy->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles would be misread
    if (threadIdx.x == 0) atomicCAS(P.status, kDevOk, kDevTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sy->q_full[i], 1);
      mbar_init(&sy->q_empty[i], 1);
      mbar_init(&sy->z_full[i], 8);
    }
    for (int i = 0; i < C::kK; ++i) {
      mbar_init(&sy->k_full[i], 1);
      mbar_init(&sy->k_empty[i], 1);
    }
    mbar_init(&sy->g_full, 1);
    mbar_init(&sy->g_empty, 1);
    mbar_init(&sy->k_raw, 1);
    for (int i = 0; i < C::kV; ++i) {
      mbar_init(&sy->v_full[i], 1);
      mbar_init(&sy->v_empty[i], 1);
    }
    mbar_init(&sy->x_full, 1);
    mbar_init(&sy->y_full, 1);
    mbar_init(&sy->x_free, 8);
    mbar_init(&sy->y_free, 8);
    mbar_init(&sy->acc_full, 1);
    mbar_init(&sy->out_full, 8);
    mbar_init(&sy->drain, 1);
    sy->abort = 0;
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mg);
    tma_prefetch_desc(&mo);
    fence_barrier_init();
  }
  zero_gap(smem, 3 * 2 * C::kBoxes, P.G * P.tq);  // Q tiles and dO
  fence_async_smem();
  if (warp == 1) tmem_alloc(&sy->tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sy->tmem_slot;
  pdl_wait();
  if (warp == 0) {
    if (lane == 0) q_load<D>(P, &mq, &mg, smem, sy, abort);
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) q_mma<D>(P, smem, sy, tmem, abort);
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) q_store<D>(P, &mo, smem, sy, abort);
    __syncwarp();
  } else if (warp == 3) {
    q_load_kv<D>(P, &mk, &mv, smem, sy, abort);
    __syncwarp();
  } else if (warp >= 4) {
    q_softmax<D>(P, smem, sy, tmem, abort);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D>
cudaError_t launch_b(const DiffArgs &a, const DiffRows &r, float *part, int nsplit, float *qpart,
                     int qsplit, cudaStream_t st) {
  using C = BCfg<D>;
  const CrossShape &s = a.x.s;
  cudaError_t err;
  auto enc = tensor_map_encoder(&err);
  if (!enc) return err;
  const cross::Packing pk = cross::packing(s);
  const nabla_strides dq_st{(int64_t)s.Sq * s.h * D, (int64_t)s.h * D, D};
  CUtensorMap mq, mk, mv, mg, mo, mk64, mv64;
  if (!cross::cross_map(enc, &mq, a.x.q, s.B, s.Sq, s.h, D, a.x.q_st, pk.G, pk.tq) ||
      !cross::cross_map(enc, &mk, a.x.k, s.B, s.Sk, s.hk, D, a.x.k_st, 1, kTile) ||
      !cross::cross_map(enc, &mv, a.x.v, s.B, s.Sk, s.hk, D, a.x.v_st, 1, kTile) ||
      !cross::cross_map(enc, &mk64, a.x.k, s.B, s.Sk, s.hk, D, a.x.k_st, 1, kStates) ||
      !cross::cross_map(enc, &mv64, a.x.v, s.B, s.Sk, s.hk, D, a.x.v_st, 1, kStates) ||
      !cross::cross_map(enc, &mg, a.x.dout, s.B, s.Sq, s.h, D, a.x.dout_st, pk.G, pk.tq) ||
      !cross::cross_map(enc, &mo, a.x.dq, s.B, s.Sq, s.h, D, dq_st, pk.G, pk.tq))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
  if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return err;
  BParams p{};
  p.dq = static_cast<__nv_bfloat16 *>(a.x.dq);
  p.dk = static_cast<__nv_bfloat16 *>(a.x.dk);
  p.dv = static_cast<__nv_bfloat16 *>(a.x.dv);
  p.part = part;
  p.rows = r.rows, p.nrows = r.nrows, p.t2 = r.t2;
  p.kv_len = a.x.kv_len;
  p.B = s.B, p.Sq = s.Sq, p.Sk = s.Sk, p.h = s.h, p.hk = s.hk;
  p.G = pk.G, p.tq = pk.tq, p.nsub = r.nsub, p.nsteps = pk.nsub;
  p.nsplit = nsplit;
  p.scale = a.x.scale;
  p.scale_log2 = a.x.scale == 0.f ? 1e-30f : fabsf(a.x.scale) * 1.4426950408889634f;
  p.neg = a.x.scale < 0.f ? kIdescNegA : 0u;
  p.status = a.x.status;
  const int nkt = (s.Sk + kTile - 1) / kTile;
  p.units = (uint32_t)((long)s.B * s.hk * nkt * p.nsplit);
  auto kern = diff_dkv_kernel<D>;
  if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  b_smem_bytes<D, false>())) != cudaSuccess)
    return err;
  unsigned grid = p.units < (unsigned)sms ? p.units : (unsigned)sms;
  p.walk = cross::walk_step(grid, p.nsplit, nkt, s.hk);
  err = launch_pdl(kern, dim3(grid), dim3(C::kThreads), b_smem_bytes<D, false>(), st, mq, mk, mv,
                   mg, p);
  if (err == cudaSuccess && p.nsplit > 1)
    err = launch_cross_dkv_join(a.x, NABLA_BF16, part, p.nsplit, st);
  if (err != cudaSuccess) return err;
  p.nsplit = qsplit;
  p.part = qpart;
  p.units = (uint32_t)((long)s.B * s.hk * (r.nsub / 2) * p.nsplit);
  auto kern2 = diff_dq_kernel<D>;
  if ((err = cudaFuncSetAttribute(kern2, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  b_smem_bytes<D, true>())) != cudaSuccess)
    return err;
  grid = p.units < (unsigned)sms ? p.units : (unsigned)sms;
  p.walk = cross::walk_step(grid, p.nsplit, r.nsub / 2, s.hk);
  err = launch_pdl(kern2, dim3(grid), dim3(C::kThreads), b_smem_bytes<D, true>(), st, mq, mk64,
                   mv64, mg, mo, p);
  if (err != cudaSuccess || p.nsplit == 1) return err;
  return launch_diff_dq_sum(a, NABLA_BF16, qpart, qsplit, st);
}

}  // namespace

cudaError_t launch_diff_bwd_tc(const DiffArgs &a, const DiffRows &r, float *part, int nsplit,
                               float *qpart, int qsplit, cudaStream_t st) {
  return a.x.s.D == 64 ? launch_b<64>(a, r, part, nsplit, qpart, qsplit, st)
                       : launch_b<128>(a, r, part, nsplit, qpart, qsplit, st);
}

}  // namespace nabla
