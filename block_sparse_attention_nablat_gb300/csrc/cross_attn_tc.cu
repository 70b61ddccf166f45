// K9 -- bf16 cross attention forward on the tcgen05 tensor cores: every query row
// attends to the first kv_len[b] of its batch's encoder states.
//
//   o_s = sum_u softmax_u(scale <q_s, k_u>) v_u,  u < kv_len[b]
//
//  * Work unit = 128 packed query rows (two 64-row subtiles, cross_common.cuh) of one
//    (batch, key head), over all of the batch's state tiles or, when there are few
//    units, over one of `nsplit` equal runs of them (cross_combine joins the runs).
//    Persistent CTAs (one per SM) take units round-robin, so the CTAs at work share a
//    few heads' K and V in L2.
//  * A step covers a tile of 128 states: S = Q K^T is one SS MMA (M = 128, N = 128),
//    O += P V a TS MMA with P (bf16) in TMEM over the scores it came from.  The last
//    tile of a batch runs at N = its states rounded up to 16.
//  * TMEM: O in columns [0, D), three score buffers of 128 columns, so S of step g + 2
//    waits only for the PV of step g - 1.  Shared memory: two Q, two K and two V tiles
//    and one for the rows on their way out.
//  * Encoder states are few (a prompt is four tiles), so a unit is short and every role
//    runs ahead into the next unit: warp 0 loads Q and K (TMA), warp 3 V; one thread of
//    warp 1 issues the QK^T, one of warp 2 the PV; eight softmax warps (two threads per
//    row, 64 columns each) do nothing but softmax; four warps take O out of TMEM, scale
//    and store it.
//  * Softmax in base 2 with the scale folded in.  The running maximum is only the
//    exponent's bias: it is the row maximum of a unit's first step, and is raised (O and
//    l rescaled) only for a step whose maximum exceeds it by more than 8.  (A fixed bias
//    would need no maximum, but P next to 1, where the heaviest states are, is rounded
//    with half the average relative error: the rows come out 0.0020 off instead of 0.0023
//    at 140 states, and exact at one.)  P is rounded to bf16 for the tensor cores, l sums
//    the fp32 P.
//  * States past kv_len never enter: their columns get P = 0 whatever K holds there, and
//    the rows of V that share the last 16-row MMA step with them are zeroed in shared
//    memory before it runs, so a NaN behind the length stays there.
//  * The output warps stage a unit's rows as bf16 in shared memory and store them by TMA.
//
// 32768 tokens, 24 heads, D 128: 512 states 161 us, 1280 TFLOP/s; 4096 states 984 us, 1680
// (0.87 of a large library product's rate); 128 states 79 us, 5.1 TB/s of rows in and out.
// A unit costs about 1,500 cycles a step and 1,900 more: at few steps its start and end,
// and the instruction fetches of code that runs once a unit, bound it, so the waits' slow
// paths are out of line and no role's code exists twice.
// At D 64 a step's products take half as long and its softmax as long as at D 128, so the
// kernel does too: 512 states 150 us, 4096 states 1000, of floors of 54 and 433.
// Measured and not kept at 512 states: two or three sets of softmax warps on alternating
// steps 168 to 200, the units walked without divisions (more code) 165.  (Two chains of four
// softmax warps each were 256 beside 238 before the waits' slow paths were out of line; not
// measured since.)
// Every mbarrier wait is bounded (1 s); on expiry the kernel records
// NABLA_ERR_TIMEOUT, the roles stop waiting, copies and MMAs in flight are drained and
// TMEM is released.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "cross_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "softmax_tc.cuh"
#include "tc_ptx.cuh"

namespace nabla {
namespace {

using namespace tc;
using cross::kTile;
using cross::x_exp;
using cross::x_mask;
using cross::x_max;
using tcattn::add2;
using tcattn::f2;
using tcattn::fma2;
using tcattn::max3;
using tcattn::Ring;
using tcattn::unf2;

template <int D>
struct XCfg {
  static constexpr int kBoxes = D / 64;   // 64-column (128-byte) swizzle boxes
  static constexpr int kBox = 128 * 128;  // one box of a 128-row tile
  static constexpr int kTileBytes = kBoxes * kBox;
  static constexpr int kQBufs = 2, kKBufs = 2, kVBufs = 2, kSBufs = 3;
  static_assert(kKBufs < kSBufs, "s_full of step g - kKBufs cannot have moved on");
  static_assert(kVBufs < kSBufs, "pv_done of step g - kVBufs cannot have moved on");
  static constexpr uint32_t kSCol = 128;  // score buffer b at 128 + 128 b
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kThreads = 512;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kQBufs * kTileBytes;
  static constexpr int kOffV = kOffK + kKBufs * kTileBytes;
  static constexpr int kOffO = kOffV + kVBufs * kTileBytes;  // rows on their way out
  static constexpr int kOffL = kOffO + kTileBytes;    // the rows' l: [128]
  static constexpr int kOffM = kOffL + 128 * 4;       // their bias: [128]
  static constexpr int kOffX = kOffM + 128 * 4;       // the halves' maxima, or l: [2][128]
  static constexpr int kOffF = kOffX + 2 * 128 * 4;   // flags: [2 in turn][2 halves][128]
  static constexpr int kOffSync = kOffF + 4 * 128;
};

struct XSync {
  uint64_t q_full[2], q_empty[2], k_full[2], v_full[2], v_raw;
  uint64_t s_full[3], p_full[3], pv_done[3];
  uint64_t o_free, l_full, l_empty, drain;
  uint32_t tmem_slot;
  int abort;
};

// The tiles sit at the 1024-byte aligned start of the dynamic shared memory (the
// kernel checks), so there is no slack for aligning them by hand.
template <int D>
constexpr int x_smem_bytes() {
  return XCfg<D>::kOffSync + (int)sizeof(XSync);
}
static_assert(x_smem_bytes<128>() <= 232448, "shared memory budget");

struct XParams {
  __nv_bfloat16 *o;   // [B, Sq, h, D]
  float *lse;         // [B, h, Sq] or null
  float *po, *plse;   // runs (nsplit > 1): [nsplit, B, h, Sq, D] and [nsplit, B, h, Sq]
  const int32_t *kv_len;
  int B, Sq, Sk, h, hk, G, tq, nqt, nsplit;
  uint32_t units;  // B hk nqt nsplit
  float scale_log2;  // of |scale|, never 0
  uint32_t neg;      // kIdescNegA for a negative scale: the scores come negated
  int *status;
};

struct XUnit {
  int b, j, qt, sp, len, t0, n;  // n state tiles from t0
};
// Unit u: runs of one tile of queries first, then query tiles, key heads, batches.
__device__ __noinline__ XUnit x_unit(const XParams &P, uint32_t u) {
  XUnit r;
  uint32_t v = u;
  r.sp = 0;
  if (P.nsplit > 1) {
    v = u / (uint32_t)P.nsplit;
    r.sp = (int)(u - v * (uint32_t)P.nsplit);
  }
  const uint32_t bj = v / (uint32_t)P.nqt;
  r.qt = (int)(v - bj * (uint32_t)P.nqt);
  r.b = (int)(bj / (uint32_t)P.hk);
  r.j = (int)(bj - (uint32_t)r.b * (uint32_t)P.hk);
  r.len = cross::batch_len(P.kv_len, r.b, P.Sk);
  const int nt = (r.len + kTile - 1) / kTile;
  r.t0 = 0;
  r.n = nt;
  if (P.nsplit > 1) {
    r.t0 = (int)((long)nt * r.sp / P.nsplit);
    r.n = (int)((long)nt * (r.sp + 1) / P.nsplit) - r.t0;
  }
  return r;
}
// 16-state MMA steps of tile t (8, or fewer in the last tile).
__device__ __forceinline__ int x_k16(const XUnit &u, int t) {
  const int left = u.len - t * kTile;
  return left >= kTile ? 8 : (left + 15) >> 4;
}

// Warp 0, lane 0: Q of every unit and K of every step, as far ahead as the rings allow.
template <int D>
__device__ void x_load_qk(const XParams &P, const CUtensorMap *mq, const CUtensorMap *mk,
                          uint8_t *smem, XSync *sy, volatile int *abort) {
  using C = XCfg<D>;
  uint32_t g = 0, kq = 0;
  Ring<C::kQBufs> q;
  bool go = true;
  const uint32_t qbytes = (uint32_t)(P.G * P.tq) * 128 * 2 * C::kBoxes;
  for (uint32_t i = blockIdx.x; i < P.units && go && !*abort; i += gridDim.x) {
    const XUnit u = x_unit(P, i);
    cross::check_len(P.kv_len, u.b, P.Sk, P.status);
    if (u.n == 0) continue;
    go = mbar_wait_small(&sy->q_empty[q.slot], q.phase ^ 1u, abort, P.status, kDevTimeout);
    if (!go) break;
    mbar_expect_tx(&sy->q_full[q.slot], qbytes);
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int c = 0; c < C::kBoxes; ++c)  // tokens past Sq are zero-filled
        tma_load_4d(smem + C::kOffQ + q.slot * C::kTileBytes + c * C::kBox + side * 64 * 128, mq,
                    &sy->q_full[q.slot], c * 64, u.j * P.G, (u.qt * 2 + side) * P.tq, u.b);
    ++kq;
    q.next();
    for (int s = 0; s < u.n && go; ++s, ++g) {
      const uint32_t ks = g % C::kKBufs;
      if (g >= (uint32_t)C::kKBufs) {  // free once the QK^T of step g - 2 is done
        const uint32_t gp = g - C::kKBufs;
        go = mbar_wait_small(&sy->s_full[gp % C::kSBufs], (gp / C::kSBufs) & 1u, abort, P.status,
                             kDevTimeout);
        if (!go) break;
      }
      mbar_expect_tx(&sy->k_full[ks], C::kTileBytes);
#pragma unroll
      for (int c = 0; c < C::kBoxes; ++c)
        tma_load_4d(smem + C::kOffK + ks * C::kTileBytes + c * C::kBox, mk, &sy->k_full[ks],
                    c * 64, u.j, (u.t0 + s) * kTile, u.b);
    }
  }
  if (!go || *abort) {  // let copies in flight land before the CTA exits
    for (uint32_t e = g > (uint32_t)C::kKBufs ? g - C::kKBufs : 0u; e < g; ++e)
      mbar_wait_small(&sy->k_full[e % C::kKBufs], (e / C::kKBufs) & 1u, nullptr, P.status,
                      kDevTimeout);
    for (uint32_t e = kq > (uint32_t)C::kQBufs ? kq - C::kQBufs : 0u; e < kq; ++e)
      mbar_wait_small(&sy->q_full[e % C::kQBufs], (e / C::kQBufs) & 1u, nullptr, P.status,
                      kDevTimeout);
  }
}

// Warp 3: V of every step.  Slot g % 2 is free once the PV of step g - 2 is done.  A
// tile whose last 16-row step reaches past the batch's length comes in on v_raw: the
// warp zeroes those rows, then hands the tile on.
template <int D>
__device__ void x_load_v(const XParams &P, const CUtensorMap *mv, uint8_t *smem, XSync *sy,
                         volatile int *abort) {
  using C = XCfg<D>;
  const int lane = threadIdx.x & 31;
  uint32_t g = 0, raw = 0;
  bool go = true;
  for (uint32_t i = blockIdx.x; i < P.units && go; i += gridDim.x) {
    const XUnit u = x_unit(P, i);
    for (int s = 0; s < u.n && go; ++s, ++g) {
      const uint32_t vs = g % C::kVBufs;
      const int t = u.t0 + s;
      const int rows = u.len - t * kTile, end = x_k16(u, t) * 16;  // zero rows [rows, end)
      const bool mend = rows < end && u.len < P.Sk;
      uint8_t *tile = smem + C::kOffV + vs * C::kTileBytes;
      bool ok = true;
      if (lane == 0) {
        ok = !*abort;
        if (ok && g >= (uint32_t)C::kVBufs) {
          const uint32_t gp = g - C::kVBufs;
          ok = mbar_wait_small(&sy->pv_done[gp % C::kSBufs], (gp / C::kSBufs) & 1u, abort, P.status,
                         kDevTimeout);
        }
        if (ok) {
          uint64_t *bar = mend ? &sy->v_raw : &sy->v_full[vs];
          mbar_expect_tx(bar, C::kTileBytes);
#pragma unroll
          for (int c = 0; c < C::kBoxes; ++c)
            tma_load_4d(tile + c * C::kBox, mv, bar, c * 64, u.j, t * kTile, u.b);
          if (mend) ok = mbar_wait_small(&sy->v_raw, raw & 1u, nullptr, P.status, kDevTimeout);
        }
      }
      go = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!go) break;
      if (mend) {
        ++raw;
        const int n16 = (end - rows) * 8;  // 16-byte pieces per box; a row is 128 bytes of it
        for (int c = 0; c < C::kBoxes; ++c)
          for (int e = lane; e < n16; e += 32)
            *reinterpret_cast<uint4 *>(tile + c * C::kBox + rows * 128 + e * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sy->v_full[vs]);
      }
    }
  }
  if (lane == 0 && (!go || *abort))
    for (uint32_t e = g > (uint32_t)C::kVBufs ? g - C::kVBufs : 0u; e < g; ++e)
      mbar_wait_small(&sy->v_full[e % C::kVBufs], (e / C::kVBufs) & 1u, nullptr, P.status,
                      kDevTimeout);
}

// Warp 1: S of step g into score buffer g % 3, once the PV of step g - 3 (its last
// reader) is done.
template <int D>
__device__ void x_qk(const XParams &P, uint8_t *smem, XSync *sy, uint32_t tmem,
                     volatile int *abort) {
  using C = XCfg<D>;
  const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
  const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
  Ring<C::kSBufs> sb;
  Ring<C::kKBufs> ks;
  Ring<C::kQBufs> q;
  bool ok = true;
  for (uint32_t i = blockIdx.x; i < P.units && ok; i += gridDim.x) {
    const XUnit u = x_unit(P, i);
    if (u.n == 0) continue;
    ok = cross::thread_wait(&sy->q_full[q.slot], q.phase, abort, P.status);
    const uint64_t qd = q_desc + (uint64_t)((q.slot * C::kTileBytes) >> 4);
    for (int s = 0; s < u.n && ok; ++s) {
      ok = cross::thread_wait(&sy->pv_done[sb.slot], sb.phase ^ 1u, abort, P.status) &&
           cross::thread_wait(&sy->k_full[ks.slot], ks.phase, abort, P.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + C::kSCol + sb.slot * 128;
      const uint64_t kd = k_desc + (uint64_t)((ks.slot * C::kTileBytes) >> 4);
      const uint32_t id = idesc_bf16(128, x_k16(u, u.t0 + s) * 16, 0, 0) | P.neg;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        // 16 columns: 32 bytes inside a 128-byte swizzle row, every 4 the next box
        const uint64_t at = (uint64_t)(((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4);
        mma_ss(d, qd + at, kd + at, id, kk > 0 ? 1u : 0u);
      }
      mma_commit(&sy->s_full[sb.slot]);  // also frees the K slot
      if (s + 1 == u.n) mma_commit(&sy->q_empty[q.slot]);
      sb.next();
      ks.next();
    }
    q.next();
  }
  mma_commit(&sy->drain);  // never exit with MMAs in flight
  mbar_wait_small(&sy->drain, 0, nullptr, P.status, kDevTimeout);
}

// Warp 2: O += P V once the softmax warps have written the step's P.
template <int D>
__device__ void x_pv(const XParams &P, uint8_t *smem, XSync *sy, uint32_t tmem,
                     volatile int *abort) {
  using C = XCfg<D>;
  const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + C::kOffV), C::kBox, 1024);
  constexpr uint32_t id = idesc_bf16(128, D, 0, 1);
  Ring<C::kSBufs> sb;
  Ring<C::kVBufs> vs;
  uint32_t kq = 0;
  bool ok = true;
  for (uint32_t i = blockIdx.x; i < P.units && ok; i += gridDim.x) {
    const XUnit u = x_unit(P, i);
    if (u.n == 0) continue;
    // the previous unit's O must have been read before the first PV overwrites it
    if (kq > 0) ok = cross::thread_wait(&sy->o_free, (kq - 1) & 1u, abort, P.status);
    for (int s = 0; s < u.n && ok; ++s) {
      ok = cross::thread_wait(&sy->v_full[vs.slot], vs.phase, abort, P.status) &&
           cross::thread_wait(&sy->p_full[sb.slot], sb.phase, abort, P.status);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = v_desc + (uint64_t)((vs.slot * C::kTileBytes) >> 4);
      const uint32_t a = tmem + C::kSCol + sb.slot * 128;
      const int k16 = x_k16(u, u.t0 + s);
      // 16 states a MMA: 8 columns of P, the right half's from 64; all eight without a
      // branch between them but in a batch's last tile
      if (k16 == 8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem, a + (kk >> 2) * 64 + (kk & 3) * 8,
                 vd + (uint64_t)((kk * 16 * 128) >> 4), id, (s > 0 || kk > 0) ? 1u : 0u);
      } else {
#pragma unroll 1
        for (int kk = 0; kk < k16; ++kk)
          mma_ts(tmem, a + (kk >> 2) * 64 + (kk & 3) * 8,
                 vd + (uint64_t)((kk * 16 * 128) >> 4), id, (s > 0 || kk > 0) ? 1u : 0u);
      }
      mma_commit(&sy->pv_done[sb.slot]);  // frees the score buffer and the V slot
      sb.next();
      vs.next();
    }
    ++kq;
  }
  mma_commit(&sy->drain);
  mbar_wait_small(&sy->drain, 0, nullptr, P.status, kDevTimeout);
}

__device__ __forceinline__ void x_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// The two softmax warps that hold the same rows (q4) meet.
__device__ __forceinline__ void x_pair_sync(int q4) {
  asm volatile("bar.sync %0, 64;" ::"r"(1 + q4) : "memory");
}

// A later step's maximum may exceed the bias by this much (base 2) before O is rescaled.
constexpr float kXSlack = 8.f;

// Warps 4-11: P of every step; thread = row, group grp takes columns 64 grp .. + 63.  The
// two threads of a row exchange the maxima of a unit's first step, the row's bias.  In
// later steps the first exponentials go ahead with it while the two tell each other, by a
// flag, whether it will do; only where it will not do they exchange maxima again, rescale
// and start anew.
template <int D>
__device__ void x_softmax(const XParams &P, uint8_t *smem, XSync *sy, uint32_t tmem,
                          volatile int *abort) {
  using C = XCfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
  const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16);
  float *xl = reinterpret_cast<float *>(smem + C::kOffL) + row;
  float *xm = reinterpret_cast<float *>(smem + C::kOffM) + row;
  volatile float *xx = reinterpret_cast<volatile float *>(smem + C::kOffX) + row;
  const float sl2 = P.scale_log2;
  Ring<C::kSBufs> sb;
  uint32_t g = 0, kq = 0;
  bool live = true;  // false after a wait gave up: keep meeting the barriers, do no work
  for (uint32_t i = blockIdx.x; i < P.units; i += gridDim.x) {
    const XUnit u = x_unit(P, i);
    if (u.n == 0) continue;
    float m_run = 0.f, l_run = 0.f;
    for (int s = 0; s < u.n; ++s, ++g, sb.next()) {
      const int mine = u.len - (u.t0 + s) * kTile - grp * 64;  // own columns that are states
      cross::warp_wait(live, &sy->s_full[sb.slot], sb.phase, abort, P.status);
      tc_fence_after();
      const uint32_t own = at + C::kSCol + sb.slot * 128 + grp * 64;
      uint32_t r0[32], r1[32];
      tmem_ld32(own, r0);
      tmem_ld32(own + 32, r1);
      tmem_wait_ld();
      reg_fence(r0);
      reg_fence(r1);
      if (mine < 64) {
        x_mask(mine, r0);
        x_mask(mine - 32, r1);
      }
      float a0 = -INFINITY, a1 = -INFINITY;
      x_max(r0, a0, a1);
      x_max(r1, a0, a1);
      const float mh = fmaxf(a0, a1) * sl2;
      volatile uint8_t *f = smem + C::kOffF + (g & 1u) * 256 + row;
      if (s == 0) {
        xx[grp * 128] = mh;
        x_pair_sync(q4);
        m_run = fmaxf(mh, xx[(grp ^ 1) * 128]);
      } else {
        f[grp * 128] = mh > m_run + kXSlack ? 1 : 0;
      }
      uint32_t pk[16];
      uint64_t sc2 = f2(sl2, sl2), nm2, acc0, acc1;
#pragma unroll 1
      for (bool again = s == 0;; again = true) {
        nm2 = f2(-m_run, -m_run);
        acc0 = acc1 = f2(0.f, 0.f);
        x_exp(r0, sc2, nm2, acc0, acc1, pk);
        if (again) break;
        x_pair_sync(q4);
        const bool need = (f[0] | f[128]) != 0;
        if (!__any_sync(0xffffffffu, need)) break;  // the same in both warps
        xx[grp * 128] = mh;
        x_pair_sync(q4);
        const float m_new = need ? fmaxf(mh, xx[(grp ^ 1) * 128]) : m_run;
        // O must hold every PV up to the previous step before it is rescaled; each half
        // takes half of its columns
        const uint32_t gp = g - 1;
        const float alpha = ex2(m_run - m_new);
        cross::warp_wait(live, &sy->pv_done[gp % C::kSBufs], (gp / C::kSBufs) & 1u, abort,
                         P.status);
        tc_fence_after();
#pragma unroll 1
        for (int x = 0; x < D / 32; ++x) {
          const uint32_t ta = at + grp * (D / 2) + x * 16;
          uint32_t t[16];
          tmem_ld16(ta, t);
          tmem_wait_ld();
          reg_fence16(t);
#pragma unroll
          for (int e = 0; e < 16; ++e) t[e] = __float_as_uint(__uint_as_float(t[e]) * alpha);
          tmem_st16(ta, t);
        }
        tmem_wait_st();
        l_run *= alpha;
        m_run = m_new;
      }
      tmem_st16(own, pk);
      x_exp(r1, sc2, nm2, acc0, acc1, pk);
      tmem_st16(own + 16, pk);
      float s0, s1, s2, s3;
      unf2(acc0, s0, s1);
      unf2(acc1, s2, s3);
      l_run += (s0 + s1) + (s2 + s3);
      tmem_wait_st();
      tc_fence_before();
      x_arrive(&sy->p_full[sb.slot], lane);
    }
    if (grp == 1) xx[0] = l_run;
    x_pair_sync(q4);
    if (grp == 0) {
      // the output warps have read the last unit's l and bias
      cross::warp_wait(live, &sy->l_empty, (kq & 1u) ^ 1u, abort, P.status);
      *xl = l_run + xx[0];
      *xm = m_run;
      x_arrive(&sy->l_full, lane);
    }
    ++kq;
  }
}

// The four output warps.
__device__ __forceinline__ void x_out_sync() { asm volatile("bar.sync 13, 128;" ::: "memory"); }

// Warps 12-15: the units' rows; thread = row.
template <int D>
__device__ void x_output(const XParams &P, const CUtensorMap *mo, uint8_t *smem, XSync *sy,
                         uint32_t tmem, volatile int *abort) {
  using C = XCfg<D>;
  const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
  const int row = q4 * 32 + lane, r64 = row & 63;
  const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16);
  const float *xl = reinterpret_cast<const float *>(smem + C::kOffL);
  const float *xm = reinterpret_cast<const float *>(smem + C::kOffM);
  uint8_t *tile = smem + C::kOffO;
  const int tok = r64 / P.G, head = r64 - tok * P.G;  // of this row, in its subtile
  uint32_t gs = 0, kq = 0;  // steps and units (with states) so far
  bool live = true;         // false after a wait gave up: keep meeting the barrier, do no work
  for (uint32_t i = blockIdx.x; i < P.units; i += gridDim.x) {
    const XUnit u = x_unit(P, i);
    const int token = (u.qt * 2 + (row >> 6)) * P.tq + tok, hh = u.j * P.G + head;
    const bool row_ok = tok < P.tq && token < P.Sq;
    const size_t lrow = ((size_t)u.b * P.h + hh) * P.Sq + token;
    float l = 0.f, m = 0.f;
    if (u.n > 0) {
      const uint32_t gl = gs + u.n - 1;
      cross::warp_wait(live, &sy->l_full, kq & 1u, abort, P.status);
      l = xl[row];
      m = xm[row];
      x_arrive(&sy->l_empty, lane);
      // the last unit's store has read the tile (long ago)
      if (q4 == 0 && lane == 0) bulk_wait_read();
      x_out_sync();
      cross::warp_wait(live, &sy->pv_done[gl % C::kSBufs], (gl / C::kSBufs) & 1u, abort, P.status);
      tc_fence_after();
      gs += u.n;
      ++kq;
    }
    const float inv = l > 0.f ? 1.0f / l : l;  // 0 for no states; NaN stays
    float *run = P.po + ((size_t)u.sp * P.B * P.h * P.Sq + lrow) * D;
    if (u.n > 0) {
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        uint32_t t[32];
        tmem_ld32(at + x * 32, t);
        tmem_wait_ld();
        reg_fence(t);
        if (x + 1 == D / 32) {
          tc_fence_before();
          x_arrive(&sy->o_free, lane);
        }
        if (P.nsplit > 1) {
          if (row_ok && live)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(run + x * 32 + e) = make_float4(
                  __uint_as_float(t[e]) * inv, __uint_as_float(t[e + 1]) * inv,
                  __uint_as_float(t[e + 2]) * inv, __uint_as_float(t[e + 3]) * inv);
          continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            w[y] = pack_bf16x2(__uint_as_float(t[8 * e + 2 * y]) * inv,
                               __uint_as_float(t[8 * e + 2 * y + 1]) * inv);
          // 16-byte piece of the row's 128 bytes in box x / 2, swizzled by the row
          const int piece = (x & 1) * 4 + e;
          *reinterpret_cast<uint4 *>(tile + (x >> 1) * C::kBox + row * 128 +
                                     ((piece ^ (row & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_async_smem();
      x_out_sync();
      if (q4 == 0 && lane == 0 && live && P.nsplit == 1) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const int t0 = (u.qt * 2 + side) * P.tq;
          if (t0 >= P.Sq) break;
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
            tma_store_4d(mo, tile + x * C::kBox + side * 64 * 128, x * 64, u.j * P.G, t0, u.b);
        }
        bulk_commit();
      }
    } else if (P.nsplit == 1 && row_ok) {  // o = 0 (joining runs leaves one without states out)
      uint4 *dst = reinterpret_cast<uint4 *>(P.o + (((size_t)u.b * P.Sq + token) * P.h + hh) * D);
#pragma unroll 1
      for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (row_ok && live) {
      const float lse = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
      if (P.nsplit > 1)
        P.plse[(size_t)u.sp * P.B * P.h * P.Sq + lrow] = lse;
      else if (P.lse)
        P.lse[lrow] = lse;
    }
  }
  if (q4 == 0 && lane == 0) bulk_wait_all();
}

template <int D>
__global__ void __launch_bounds__(512, 1)
    cross_attn_tc_kernel(const __grid_constant__ CUtensorMap mq,
                         const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv,
                         const __grid_constant__ CUtensorMap mo,
                         const __grid_constant__ XParams P) {
  using C = XCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  XSync *sy = reinterpret_cast<XSync *>(smem + C::kOffSync);
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
      mbar_init(&sy->k_full[i], 1);
      mbar_init(&sy->v_full[i], 1);
    }
    mbar_init(&sy->v_raw, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sy->s_full[i], 1);
      mbar_init(&sy->p_full[i], 8);  // softmax warps
      mbar_init(&sy->pv_done[i], 1);
    }
    mbar_init(&sy->o_free, 4);  // output warps
    mbar_init(&sy->l_full, 4);
    mbar_init(&sy->l_empty, 4);
    mbar_init(&sy->drain, 2);  // one commit per MMA-issuing thread
    sy->abort = 0;
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mo);
    fence_barrier_init();
  }
  // rows of the Q tiles that no box fills (G not dividing 64)
  const int used = P.G * P.tq;
  for (int e = threadIdx.x; e < (64 - used) * 8 * 2 * C::kBoxes * C::kQBufs; e += C::kThreads) {
    const int per = (64 - used) * 8, sub = e / per, to = e - sub * per;
    *reinterpret_cast<uint4 *>(smem + C::kOffQ + sub * 64 * 128 + used * 128 + to * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_async_smem();
  if (warp == 1) tmem_alloc(&sy->tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sy->tmem_slot;
  pdl_wait();  // the inputs are written; no earlier kernel still reads o

  if (warp < 4) {
    if (warp == 0) {
      if (lane == 0) x_load_qk<D>(P, &mq, &mk, smem, sy, abort);
    } else if (warp == 1) {
      if (elect_one()) x_qk<D>(P, smem, sy, tmem, abort);
    } else if (warp == 2) {
      if (elect_one()) x_pv<D>(P, smem, sy, tmem, abort);
    } else {
      x_load_v<D>(P, &mv, smem, sy, abort);
    }
    __syncwarp();
  } else if (warp < 12) {
    x_softmax<D>(P, smem, sy, tmem, abort);
  } else {
    x_output<D>(P, &mo, smem, sy, tmem, abort);
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
cudaError_t launch_x(const CrossArgs &a, cudaStream_t st) {
  using C = XCfg<D>;
  const CrossShape &s = a.s;
  cudaError_t err;
  auto enc = tensor_map_encoder(&err);
  if (!enc) return err;
  const cross::Packing pk = cross::packing(s);
  const nabla_strides o_st{(int64_t)s.Sq * s.h * D, (int64_t)s.h * D, D};
  CUtensorMap mq, mk, mv, mo;
  if (!cross::cross_map(enc, &mq, a.q, s.B, s.Sq, s.h, D, a.q_st, pk.G, pk.tq) ||
      !cross::cross_map(enc, &mk, a.k, s.B, s.Sk, s.hk, D, a.k_st, 1, kTile) ||
      !cross::cross_map(enc, &mv, a.v, s.B, s.Sk, s.hk, D, a.v_st, 1, kTile) ||
      !cross::cross_map(enc, &mo, a.o, s.B, s.Sq, s.h, D, o_st, pk.G, pk.tq))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
  if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return err;
  auto kern = cross_attn_tc_kernel<D>;
  if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  x_smem_bytes<D>())) != cudaSuccess)
    return err;
  XParams p{};
  p.o = static_cast<__nv_bfloat16 *>(a.o);
  p.lse = a.lse;
  p.kv_len = a.kv_len;
  p.B = s.B, p.Sq = s.Sq, p.Sk = s.Sk, p.h = s.h, p.hk = s.hk;
  p.G = pk.G, p.tq = pk.tq;
  p.nqt = (pk.nsub + 1) / 2, p.nsplit = cross_fwd_splits(s, NABLA_BF16);
  // a scale of 0 weighs all states alike, as one too small to tell scores apart does
  p.scale_log2 = a.scale == 0.f ? 1e-30f : fabsf(a.scale) * 1.4426950408889634f;
  p.neg = a.scale < 0.f ? kIdescNegA : 0u;
  p.status = a.status;
  const CrossRuns runs = cross_runs(a, p.nsplit);
  p.po = runs.po, p.plse = runs.plse;
  p.units = (uint32_t)((long)s.B * s.hk * p.nqt * p.nsplit);
  const unsigned grid = p.units < (unsigned)sms ? p.units : (unsigned)sms;
  err = launch_pdl(kern, dim3(grid), dim3(C::kThreads), x_smem_bytes<D>(), st, mq, mk, mv, mo,
                   p);
  if (err != cudaSuccess || p.nsplit == 1) return err;
  return launch_cross_combine(a, NABLA_BF16, p.nsplit, st);
}

}  // namespace

cudaError_t launch_cross_attn_tc(const CrossArgs &a, cudaStream_t st) {
  return a.s.D == 64 ? launch_x<64>(a, st) : launch_x<128>(a, st);
}

}  // namespace nabla
