// K12 -- bf16 differential attention forward on the tcgen05 tensor cores: the difference of
// two softmax maps over the first kv_len[b] of a batch's states, with a learned weight.
//
//   o = o1 - lam o2,   o_m = softmax(scale q_m k_m^T) v
//
//  * Work unit = 128 packed query rows (two 64-row subtiles, cross_common.cuh) of one
//    (batch, key head) over the batch's state tiles, or a part of them: persistent CTAs (one
//    per SM) take units in turn and, in the end, equal shares of the rest (diff_common.cuh;
//    diff_stream_join joins the parts).
//  * A step covers 64 states.  For each map m: S_m = Q_m K_m^T is one SS MMA (M = 128,
//    N = 64, depth D / 2), O_m += P_m V a TS MMA with P_m (bf16) over the scores.  The maps
//    share K's tile (each its half of the columns) and V's.
//  * TMEM: O_1, O_2 (D columns each, 128 apart) and two 64-column score buffers a map: all 512
//    columns at D 128, while 64 beside each O stay unused at D 64.  The maps could only be
//    subtracted before the product with V if their sums were known, so the forward takes two
//    products where the definition has one.
//  * Each map has four softmax warps, thread = row: a row's maximum and sum never leave its
//    thread, and the two maps' chains (S, softmax, P V) fill each other's gaps, as do the
//    two buffers of a chain.
//  * Softmax in base 2 with the scale folded in.  The running maximum is only the exponents'
//    bias: the row maximum of a unit's first step, raised (O and l rescaled) only where a later
//    step's P add up to more than 2^8.
//  * Four output warps take O_1 and O_2 out of TMEM, scale and subtract in fp32, round once
//    and store rows by TMA; likewise o_2, which the backward needs, where it is wanted.
//  * V's rows that share the last 16-row MMA step with states past the length are zeroed in
//    shared memory, scores past it are -inf.
//
// Bound by the chain of a map's step, score product, softmax, product with V: 1250 cycles for
// 128 x 64 scores of both maps, where the tensor pipe needs 900 and a softmax warp 830 (110 to
// read the scores, 650 for maximum and exponentials, 55 to write P).  12 heads, D 128: 8192
// tokens and states 455 us, 0.91 PFLOP/s of the definition's two products (times 1.5 as they
// are run); 8192 x 1024: the tensor pipe active in 54% of the cycles, exponentials 36%.  A
// buffer of scores and two of P a map, so that its next scores need not wait for P V, in place
// of two that both share: 520 us against 473.  Four K and V tiles in place of three: the same.
// Every mbarrier wait is bounded (1 s), as in the cross attention.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <cfloat>

#include "attn_common.cuh"
#include "diff_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "softmax_tc.cuh"
#include "tc_ptx.cuh"

namespace nabla {
namespace {

using namespace tc;
using diff::kStates;
using tcattn::add2;
using tcattn::f2;
using tcattn::fma2;
using tcattn::Ring;
using tcattn::unf2;

template <int D>
struct FCfg {
  static constexpr int kBoxes = D / 64;  // 64-column (128-byte) swizzle boxes
  static constexpr int kQBox = 128 * 128, kSBox = kStates * 128;  // of Q's tiles, of K's and V's
  static constexpr int kQTile = kBoxes * kQBox, kSTile = kBoxes * kSBox;
  static constexpr int kSteps = D / 32;  // 16-column MMA steps of a map's scores
  static constexpr int kKBufs = 3, kVBufs = 3;
  static constexpr uint32_t kOCol = 128, kSCol = 256;  // O_m at 128 m; scores 256 + 128 m + 64 b
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kThreads = 512;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kQTile;
  static constexpr int kOffV = kOffK + kKBufs * kSTile;
  static constexpr int kOffO = kOffV + kVBufs * kSTile;  // rows on their way out: o, o2
  static constexpr int kOffL = kOffO + 2 * kQTile;       // l and bias of the rows: [2 maps][2][128]
  static constexpr int kOffSync = kOffL + 4 * 128 * 4;
};

// n state tiles of unit (b, j, qt) from t0 on; `part`: the CTA's place for the results of a
// part, or -1: all of the unit; `more` 0: there are no more units.
struct alignas(16) FUnit {
  int b, j, qt, len, t0, n, part, more;
};
constexpr int kUnits = 4;  // of the ring

struct FSync {
  FUnit units[kUnits];
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  uint64_t q_full[2], q_empty[2], k_full[3], k_empty[3], v_full[3], v_empty[3], v_raw;
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [map][buffer]
  uint64_t o_free, l_full, l_empty, drain;
  uint32_t tmem_slot;
  int abort;
};

template <int D>
constexpr int f_smem_bytes() {
  return FCfg<D>::kOffSync + (int)sizeof(FSync);
}
static_assert(f_smem_bytes<128>() <= 232448, "shared memory budget");

struct FParams {
  __nv_bfloat16 *o, *o2;  // [B, Sq, h, D]; o2 or null
  float *lse;             // [B, h, 2, Sq] or null
  float *po, *plse;       // parts: [kCtas, 2 places, 2 maps, D / 4, 128, 4], [.., 128]
  const float *lam;
  const int32_t *kv_len;
  int lam_step;  // 1: a weight for each head; 0: one
  int B, Sq, Sk, h, hk, G, tq, nqt;
  uint32_t whole;  // units that go round; those from there on are cut
  bool cut;        // there are such
  float scale_log2;  // of |scale|, never 0
  uint32_t neg;      // kIdescNegA for a negative scale: the scores come negated
  int *status;
};

// The CTA's way through its units: the thread that runs furthest ahead (Q's and K's loader)
// finds the next one and leaves it in a ring for the other roles, whose registers and
// instructions are scarce (as a function that each of them calls the kernel took 489 us
// against 473 for 8192 x 8192 states, 12 heads).
struct FWalk {
  uint32_t i;      // of the units that go round
  int b, unit, t;  // of the piece
  long left;
  int seen;        // parts of the piece so far
};
__device__ __forceinline__ FUnit f_next(const FParams &P, FWalk &w) {
  FUnit r;
  if (w.i < P.whole) {
    const uint32_t bj = w.i / (uint32_t)P.nqt;
    r.qt = (int)(w.i - bj * (uint32_t)P.nqt);
    r.b = (int)(bj / (uint32_t)P.hk);
    r.j = (int)(bj - (uint32_t)r.b * (uint32_t)P.hk);
    r.len = cross::batch_len(P.kv_len, r.b, P.Sk);
    r.t0 = 0;
    r.n = (r.len + kStates - 1) / kStates;
    r.part = -1;
    r.more = 1;
    w.i += gridDim.x;
    return r;
  }
  r.more = w.left > 0;
  if (!r.more) return r;
  r.len = cross::batch_len(P.kv_len, w.b, P.Sk);
  const int tiles = (r.len + kStates - 1) / kStates, all = tiles > 0 ? tiles : 1;
  const int n = w.left < all - w.t ? (int)w.left : all - w.t;
  r.b = w.b;
  r.j = w.unit / P.nqt;
  r.qt = w.unit - r.j * P.nqt;
  r.t0 = w.t;
  r.n = tiles > 0 ? n : 0;
  r.part = n == all ? -1 : w.seen > 0;
  ++w.seen;
  w.left -= n;
  w.t = 0;
  if (++w.unit == P.nqt * P.hk) w.unit = 0, ++w.b;
  return r;
}
// The next unit, for one thread (kWarp false) or a whole warp; false at the end, or when the
// wait gave up.
template <bool kWarp>
__device__ __forceinline__ bool f_get(const FParams &P, FSync *sy, Ring<kUnits> &r, FUnit &u,
                                      volatile int *abort) {
  bool ok = cross::thread_wait(&sy->unit_full[r.slot], r.phase, abort, P.status);
  if (kWarp) ok = __all_sync(0xffffffffu, ok);
  if (!ok) return false;
  u = sy->units[r.slot];
  if (kWarp) __syncwarp();
  if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(&sy->unit_empty[r.slot]);
  r.next();
  return u.more != 0;
}

// Warp 0, lane 0: Q of every unit and K of every step, as far ahead as the rings allow.
template <int D>
__device__ void f_load_qk(const FParams &P, const CUtensorMap *mq, const CUtensorMap *mk,
                          uint8_t *smem, FSync *sy, FWalk w, volatile int *abort) {
  using C = FCfg<D>;
  Ring<2> q;
  Ring<C::kKBufs> k;
  uint32_t g = 0, kq = 0;
  bool go = true;
  const uint32_t qbytes = (uint32_t)(P.G * P.tq) * 128 * 2 * C::kBoxes;
  Ring<kUnits> ur;
  while (go && !*abort) {
    const FUnit u = f_next(P, w);
    go = cross::thread_wait(&sy->unit_empty[ur.slot], ur.phase ^ 1u, abort, P.status);
    if (!go) break;
    sy->units[ur.slot] = u;
    mbar_arrive(&sy->unit_full[ur.slot]);
    ur.next();
    if (!u.more) break;
    cross::check_len(P.kv_len, u.b, P.Sk, P.status);
    if (u.n == 0) continue;
    go = cross::thread_wait(&sy->q_empty[q.slot], q.phase ^ 1u, abort, P.status);
    if (!go) break;
    mbar_expect_tx(&sy->q_full[q.slot], qbytes);
#pragma unroll 1
    for (int x = 0; x < 2 * C::kBoxes; ++x)  // box x / 2, subtile x & 1; past Sq: zeros
      tma_load_4d(smem + C::kOffQ + q.slot * C::kQTile + (x >> 1) * C::kQBox + (x & 1) * 64 * 128,
                  mq, &sy->q_full[q.slot], (x >> 1) * 64, u.j * P.G, (u.qt * 2 + (x & 1)) * P.tq,
                  u.b);
    ++kq;
    q.next();
    for (int s = 0; s < u.n && go; ++s) {
      go = cross::thread_wait(&sy->k_empty[k.slot], k.phase ^ 1u, abort, P.status);
      if (!go) break;
      mbar_expect_tx(&sy->k_full[k.slot], C::kSTile);
#pragma unroll
      for (int c = 0; c < C::kBoxes; ++c)
        tma_load_4d(smem + C::kOffK + k.slot * C::kSTile + c * C::kSBox, mk, &sy->k_full[k.slot],
                    c * 64, u.j, (u.t0 + s) * kStates, u.b);
      ++g;
      k.next();
    }
  }
  if (!go || *abort) {  // let copies in flight land before the CTA exits
    for (uint32_t e = g > (uint32_t)C::kKBufs ? g - C::kKBufs : 0u; e < g; ++e)
      cross::thread_wait(&sy->k_full[e % C::kKBufs], (e / C::kKBufs) & 1u, nullptr, P.status);
    for (uint32_t e = kq > 2u ? kq - 2u : 0u; e < kq; ++e)
      cross::thread_wait(&sy->q_full[e % 2], (e / 2) & 1u, nullptr, P.status);
  }
}

// Warp 3: V of every step.  A tile whose last 16-row step reaches past the batch's length
// comes in on v_raw: the warp zeroes those rows, then hands the tile on.
template <int D>
__device__ void f_load_v(const FParams &P, const CUtensorMap *mv, uint8_t *smem, FSync *sy,
                         volatile int *abort) {
  using C = FCfg<D>;
  const int lane = threadIdx.x & 31;
  Ring<C::kVBufs> v;
  uint32_t g = 0, raw = 0;
  bool go = true;
  Ring<kUnits> ur;
  for (FUnit u; go && f_get<true>(P, sy, ur, u, abort);) {
    for (int s = 0; s < u.n && go; ++s, ++g, v.next()) {
      const int t = u.t0 + s;
      const int rows = u.len - t * kStates, end = diff::steps16(u.len, t) * 16;
      const bool mend = rows < end && u.len < P.Sk;  // rows [rows, end) hold other things
      uint8_t *tile = smem + C::kOffV + v.slot * C::kSTile;
      bool ok = true;
      if (lane == 0) {
        ok = !*abort && cross::thread_wait(&sy->v_empty[v.slot], v.phase ^ 1u, abort, P.status);
        if (ok) {
          uint64_t *bar = mend ? &sy->v_raw : &sy->v_full[v.slot];
          mbar_expect_tx(bar, C::kSTile);
#pragma unroll
          for (int c = 0; c < C::kBoxes; ++c)
            tma_load_4d(tile + c * C::kSBox, mv, bar, c * 64, u.j, t * kStates, u.b);
          if (mend) ok = cross::thread_wait(&sy->v_raw, raw & 1u, nullptr, P.status);
        }
      }
      go = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!go) break;
      if (mend) {
        ++raw;
        diff::zero_rows<C::kBoxes>(tile, C::kSBox, rows, end);
        if (lane == 0) mbar_arrive(&sy->v_full[v.slot]);
      }
    }
  }
  if (lane == 0 && (!go || *abort))
    for (uint32_t e = g > (uint32_t)C::kVBufs ? g - C::kVBufs : 0u; e < g; ++e)
      cross::thread_wait(&sy->v_full[e % C::kVBufs], (e / C::kVBufs) & 1u, nullptr, P.status);
}

// Warp 1, one thread: S_m of step g into its buffer g & 1, once the P V of step g - 2 (its
// last reader) is done.
template <int D>
__device__ void f_qk(const FParams &P, uint8_t *smem, FSync *sy, uint32_t tmem,
                     volatile int *abort) {
  using C = FCfg<D>;
  const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
  const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
  Ring<2> sb, q;
  Ring<C::kKBufs> k;
  bool ok = true;
  Ring<kUnits> ur;
  for (FUnit u; ok && f_get<false>(P, sy, ur, u, abort);) {
    if (u.n == 0) continue;
    ok = cross::thread_wait(&sy->q_full[q.slot], q.phase, abort, P.status);
    const uint64_t qd = q_desc + (uint64_t)((q.slot * C::kQTile) >> 4);
    for (int s = 0; s < u.n && ok; ++s) {
      ok = cross::thread_wait(&sy->k_full[k.slot], k.phase, abort, P.status);
      const uint64_t kd = k_desc + (uint64_t)((k.slot * C::kSTile) >> 4);
      const uint32_t id = idesc_bf16(128, diff::steps16(u.len, u.t0 + s) * 16, 0, 0) | P.neg;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (ok) ok = cross::thread_wait(&sy->pv_done[m][sb.slot], sb.phase ^ 1u, abort, P.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + C::kSCol + m * 128 + sb.slot * 64;
#pragma unroll
        for (int x = 0; x < C::kSteps; ++x)
          mma_ss(d, qd + diff::k_step(m * C::kSteps + x, C::kQBox),
                 kd + diff::k_step(m * C::kSteps + x, C::kSBox), id, x > 0 ? 1u : 0u);
        mma_commit(&sy->s_full[m][sb.slot]);
      }
      if (!ok) break;
      mma_commit(&sy->k_empty[k.slot]);
      if (s + 1 == u.n) mma_commit(&sy->q_empty[q.slot]);
      sb.next();
      k.next();
    }
    q.next();
  }
  mma_commit(&sy->drain);  // never exit with MMAs in flight
  cross::thread_wait(&sy->drain, 0, nullptr, P.status);
}

// Warp 2, one thread: O_m += P_m V once the softmax warps have written the step's P_m.
template <int D>
__device__ void f_pv(const FParams &P, uint8_t *smem, FSync *sy, uint32_t tmem,
                     volatile int *abort) {
  using C = FCfg<D>;
  const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + C::kOffV), C::kSBox, 1024);
  constexpr uint32_t id = idesc_bf16(128, D, 0, 1);
  Ring<2> sb;
  Ring<C::kVBufs> v;
  uint32_t kq = 0;
  bool ok = true;
  Ring<kUnits> ur;
  for (FUnit u; ok && f_get<false>(P, sy, ur, u, abort);) {
    if (u.n == 0) continue;
    // the previous unit's O must have been read before the first product overwrites it
    if (kq > 0) ok = cross::thread_wait(&sy->o_free, (kq - 1) & 1u, abort, P.status);
    for (int s = 0; s < u.n && ok; ++s) {
      ok = cross::thread_wait(&sy->v_full[v.slot], v.phase, abort, P.status);
      const uint64_t vd = v_desc + (uint64_t)((v.slot * C::kSTile) >> 4);
      const int k16 = diff::steps16(u.len, u.t0 + s);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (ok) ok = cross::thread_wait(&sy->p_full[m][sb.slot], sb.phase, abort, P.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = tmem + C::kSCol + m * 128 + sb.slot * 64, d = tmem + m * C::kOCol;
        if (k16 == 4) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(d, a + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), id,
                   (s > 0 || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll 1
          for (int kk = 0; kk < k16; ++kk)
            mma_ts(d, a + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), id,
                   (s > 0 || kk > 0) ? 1u : 0u);
        }
        mma_commit(&sy->pv_done[m][sb.slot]);  // frees the score buffer
      }
      if (!ok) break;
      mma_commit(&sy->v_empty[v.slot]);
      sb.next();
      v.next();
    }
    ++kq;
  }
  mma_commit(&sy->drain);
  cross::thread_wait(&sy->drain, 0, nullptr, P.status);
}

__device__ __forceinline__ void f_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// A row's P of a later step may add up to this much before O is rescaled: P is at most 2^8,
// or the bias is raised to the step's maximum.
constexpr float kFMost = 256.f;

__device__ __forceinline__ float f_max(const uint32_t (&r0)[32], const uint32_t (&r1)[32]) {
  float a = -INFINITY, b = -INFINITY, c = -INFINITY, d = -INFINITY;  // four short chains
  cross::x_max(r0, a, b);
  cross::x_max(r1, c, d);
  return fmaxf(fmaxf(a, b), fmaxf(c, d));
}

// Warps 4-7 (map 0) and 8-11 (map 1): P of every step; thread = row.
template <int D>
__device__ void f_softmax(const FParams &P, uint8_t *smem, FSync *sy, uint32_t tmem,
                          volatile int *abort) {
  using C = FCfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int map = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
  const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16);
  const uint32_t oc = at + map * C::kOCol;
  float *xl = reinterpret_cast<float *>(smem + C::kOffL) + map * 256 + row;
  const float sl2 = P.scale_log2;
  const uint64_t sc2 = f2(sl2, sl2);
  Ring<2> sb;
  uint32_t kq = 0;
  bool live = true;  // false after a wait gave up: keep meeting the barriers, do no work
  Ring<kUnits> ur;
  for (FUnit u; f_get<true>(P, sy, ur, u, abort);) {
    if (u.n == 0) continue;
    float m_run = 0.f, l_run = 0.f;
    for (int s = 0; s < u.n; ++s, sb.next()) {
      const int mine = u.len - (u.t0 + s) * kStates;  // columns that are states
      cross::warp_wait(live, &sy->s_full[map][sb.slot], sb.phase, abort, P.status);
      tc_fence_after();
      const uint32_t own = at + C::kSCol + map * 128 + sb.slot * 64;
      uint32_t pk0[16], pk1[16];
      float sum;
      // Once, or twice where the bias is raised: the sum of a later step's P says whether it
      // will do, and the scores are read again rather than kept (which took 160 bytes of
      // spills: 677 us against 503 for 8192 x 8192 states, 12 heads).
#pragma unroll 1
      for (bool again = false;; again = true) {
        uint32_t r0[32], r1[32];
        tmem_ld32(own, r0);
        tmem_ld32(own + 32, r1);
        tmem_wait_ld();
        reg_fence(r0);
        reg_fence(r1);
        if (mine < kStates) {
          cross::x_mask(mine, r0);
          cross::x_mask(mine - 32, r1);
        }
        if (s == 0) {
          // (finite even if no score is: a later step's can still raise it)
          m_run = fmaxf(f_max(r0, r1) * sl2, -FLT_MAX);
        } else if (again) {
          const float mh = f_max(r0, r1) * sl2;
          const float m_new = sum > kFMost ? fmaxf(m_run, mh) : m_run, alpha = ex2(m_run - m_new);
          // O must hold the product of the step before when it is rescaled
          cross::warp_wait(live, &sy->pv_done[map][sb.slot ^ 1u],
                           sb.slot ? sb.phase : sb.phase ^ 1u, abort, P.status);
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < D / 16; ++x) {
            uint32_t t[16];
            tmem_ld16(oc + x * 16, t);
            tmem_wait_ld();
            reg_fence16(t);
#pragma unroll
            for (int e = 0; e < 16; ++e) t[e] = __float_as_uint(__uint_as_float(t[e]) * alpha);
            tmem_st16(oc + x * 16, t);
          }
          tmem_wait_st();
          l_run *= alpha;
          m_run = m_new;
        }
        const uint64_t nm2 = f2(-m_run, -m_run);
        uint64_t acc0 = f2(0.f, 0.f), acc1 = acc0;
        cross::x_exp(r0, sc2, nm2, acc0, acc1, pk0);
        cross::x_exp(r1, sc2, nm2, acc0, acc1, pk1);
        float s0, s1;
        unf2(add2(acc0, acc1), s0, s1);
        sum = s0 + s1;
        if (s == 0 || again || !__any_sync(0xffffffffu, sum > kFMost)) break;
      }
      tmem_st16(own, pk0);
      tmem_st16(own + 16, pk1);
      l_run += sum;
      tmem_wait_st();
      tc_fence_before();
      f_arrive(&sy->p_full[map][sb.slot], lane);
    }
    // the output warps have read the last unit's l and bias
    cross::warp_wait(live, &sy->l_empty, (kq & 1u) ^ 1u, abort, P.status);
    xl[0] = l_run;
    xl[128] = m_run;
    f_arrive(&sy->l_full, lane);
    ++kq;
  }
}

// The four output warps.
__device__ __forceinline__ void f_out_sync() { asm volatile("bar.sync 13, 128;" ::: "memory"); }
__device__ __forceinline__ bool f_out_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 13, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float f_lse(float l, float m) {
  return l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
}
__device__ __forceinline__ float f_inv(float l) {
  return l > 0.f ? 1.0f / l : l;  // 0 for no states; NaN stays
}

// Warps 12-15: the units' rows; thread = row.
template <int D>
__device__ void f_output(const FParams &P, const CUtensorMap *mo, const CUtensorMap *mo2,
                         uint8_t *smem, FSync *sy, uint32_t tmem, volatile int *abort) {
  using C = FCfg<D>;
  const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
  const int row = q4 * 32 + lane, r64 = row & 63;
  const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16);
  const float *xl = reinterpret_cast<const float *>(smem + C::kOffL) + row;
  uint8_t *tile = smem + C::kOffO;
  const int tok = r64 / P.G, head = r64 - tok * P.G;  // of this row, in its subtile
  Ring<2> sb;   // of the next step
  uint32_t kq = 0;
  bool live = true;  // false after a wait gave up: keep meeting the barrier, do no work
  Ring<kUnits> ur;
  // the four warps meet at barriers, so they go on together or not at all
  for (FUnit u; f_out_all(f_get<true>(P, sy, ur, u, abort));) {
    const int token = (u.qt * 2 + (row >> 6)) * P.tq + tok, hh = u.j * P.G + head;
    const bool row_ok = tok < P.tq && token < P.Sq;
    const bool split = u.part >= 0;
    const size_t place = (size_t)blockIdx.x * 2 + (split ? u.part : 0);  // of a part
    float l1 = 0.f, m1 = 0.f, l2 = 0.f, m2 = 0.f;
    const float lam = row_ok ? __ldg(P.lam + hh * P.lam_step) : 0.f;
    if (u.n > 0) {
      cross::warp_wait(live, &sy->l_full, kq & 1u, abort, P.status);
      l1 = xl[0], m1 = xl[128], l2 = xl[256], m2 = xl[384];
      f_arrive(&sy->l_empty, lane);
      // the last unit's stores have read the tiles (long ago)
      if (q4 == 0 && lane == 0) bulk_wait_read();
      f_out_sync();
      const uint32_t last = (sb.slot + (uint32_t)u.n - 1u) & 1u;  // the last step's buffer
      const uint32_t turn = sb.phase ^ (((sb.slot + (uint32_t)u.n - 1u) >> 1) & 1u);
#pragma unroll
      for (int m = 0; m < 2; ++m)
        cross::warp_wait(live, &sy->pv_done[m][last], turn, abort, P.status);
      tc_fence_after();
      sb.phase ^= ((sb.slot + (uint32_t)u.n) >> 1) & 1u;
      sb.slot = (sb.slot + (uint32_t)u.n) & 1u;
      ++kq;
      const float inv1 = f_inv(l1), inv2 = f_inv(l2), by2 = -lam * inv2;
      const uint64_t i1 = f2(inv1, inv1), i2 = f2(inv2, inv2), b2 = f2(by2, by2);
      // a part's rows lie side by side, four columns at a time: 512 bytes a warp and store
      float4 *run = reinterpret_cast<float4 *>(P.po) + place * 2 * (D / 4) * 128 + row;
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        uint32_t a[32], c[32];
        tmem_ld32(at + x * 32, a);
        tmem_ld32(at + C::kOCol + x * 32, c);
        tmem_wait_ld();
        reg_fence(a);
        reg_fence(c);
        if (x + 1 == D / 32) {
          tc_fence_before();
          f_arrive(&sy->o_free, lane);
        }
        if (split) {
          if (row_ok && live)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float4 *to = run + (x * 8 + e / 4) * 128;
              *to = make_float4(__uint_as_float(a[e]) * inv1, __uint_as_float(a[e + 1]) * inv1,
                                __uint_as_float(a[e + 2]) * inv1,
                                __uint_as_float(a[e + 3]) * inv1);
              to[D / 4 * 128] =
                  make_float4(__uint_as_float(c[e]) * inv2, __uint_as_float(c[e + 1]) * inv2,
                              __uint_as_float(c[e + 2]) * inv2, __uint_as_float(c[e + 3]) * inv2);
            }
          continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // 16-byte piece of the row's 128 bytes in box x / 2, swizzled by the row
          const int piece = (x & 1) * 4 + e;
          uint8_t *to = tile + (x >> 1) * C::kQBox + row * 128 + ((piece ^ (row & 7)) << 4);
          uint32_t v1[4], v2[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int at2 = 8 * e + 2 * y;
            const uint64_t c2 = f2(__uint_as_float(c[at2]), __uint_as_float(c[at2 + 1]));
            float x0, x1;
            unf2(fma2(f2(__uint_as_float(a[at2]), __uint_as_float(a[at2 + 1])), i1, mul2(c2, b2)),
                 x0, x1);
            v1[y] = pack_bf16x2(x0, x1);
            unf2(mul2(c2, i2), x0, x1);
            v2[y] = pack_bf16x2(x0, x1);
          }
          *reinterpret_cast<uint4 *>(to) = make_uint4(v1[0], v1[1], v1[2], v1[3]);
          if (P.o2)
            *reinterpret_cast<uint4 *>(to + C::kQTile) = make_uint4(v2[0], v2[1], v2[2], v2[3]);
        }
      }
      fence_async_smem();
      f_out_sync();
      if (q4 == 0 && lane == 0 && live && !split) {
#pragma unroll 1
        for (int x = 0; x < 2 * C::kBoxes; ++x) {
          const int t0 = (u.qt * 2 + (x & 1)) * P.tq;
          if (t0 >= P.Sq) continue;
          const uint8_t *from = tile + (x >> 1) * C::kQBox + (x & 1) * 64 * 128;
          tma_store_4d(mo, from, (x >> 1) * 64, u.j * P.G, t0, u.b);
          if (P.o2) tma_store_4d(mo2, from + C::kQTile, (x >> 1) * 64, u.j * P.G, t0, u.b);
        }
        bulk_commit();
      }
    } else if (!split && row_ok) {  // o = o2 = 0 (joining runs leaves one without states out)
      const size_t to = (((size_t)u.b * P.Sq + token) * P.h + hh) * D;
#pragma unroll 1
      for (int e = 0; e < D / 8; ++e) {
        reinterpret_cast<uint4 *>(P.o + to)[e] = make_uint4(0u, 0u, 0u, 0u);
        if (P.o2) reinterpret_cast<uint4 *>(P.o2 + to)[e] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (row_ok && live) {
      if (split) {
        float *to = P.plse + place * 256 + row;
        to[0] = f_lse(l1, m1);
        to[128] = f_lse(l2, m2);
      } else if (P.lse) {
        float *to = P.lse + ((size_t)u.b * P.h + hh) * 2 * P.Sq + token;
        to[0] = f_lse(l1, m1);
        to[P.Sq] = f_lse(l2, m2);
      }
    }
  }
  if (q4 == 0 && lane == 0) bulk_wait_all();
}

template <int D>
__global__ void __launch_bounds__(512, 1)
    diff_attn_tc_kernel(const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv,
                        const __grid_constant__ CUtensorMap mo,
                        const __grid_constant__ CUtensorMap mo2,
                        const __grid_constant__ FParams P) {
  using C = FCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  FSync *sy = reinterpret_cast<FSync *>(smem + C::kOffSync);
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
      for (int m = 0; m < 2; ++m) {
        mbar_init(&sy->s_full[m][i], 1);
        mbar_init(&sy->p_full[m][i], 4);  // the map's softmax warps
        mbar_init(&sy->pv_done[m][i], 1);
      }
    }
    for (int i = 0; i < C::kKBufs; ++i) {
      mbar_init(&sy->k_full[i], 1);
      mbar_init(&sy->k_empty[i], 1);
    }
    for (int i = 0; i < C::kVBufs; ++i) {
      mbar_init(&sy->v_full[i], 1);
      mbar_init(&sy->v_empty[i], 1);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&sy->unit_full[i], 1);
      mbar_init(&sy->unit_empty[i], 3 + 8 + 4);  // V's loader, the products', softmax, output
    }
    mbar_init(&sy->v_raw, 1);
    mbar_init(&sy->o_free, 4);  // output warps
    mbar_init(&sy->l_full, 8);  // softmax warps
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
  const int used = P.G * P.tq, per = (64 - used) * 8;
  for (int e = threadIdx.x; e < per * 4 * C::kBoxes; e += C::kThreads) {
    const int sub = e / per, to = e - sub * per;
    *reinterpret_cast<uint4 *>(smem + C::kOffQ + sub * 64 * 128 + used * 128 + to * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_async_smem();
  if (warp == 1) tmem_alloc(&sy->tmem_slot, C::kTmemCols);
  pdl_wait();  // the inputs are written; no earlier kernel still reads o
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sy->tmem_slot;

  if (warp < 4) {
    if (warp == 0) {
      FWalk w{blockIdx.x, 0, 0, 0, 0, 0};
      if (P.cut) {  // the CTA's piece
        const int per = P.nqt * P.hk;
        const long p0 = diff::span_of_unit(P.kv_len, P.Sk, per, P.whole);
        const long n = diff::span_total(P.kv_len, P.B, P.Sk, per) - p0;
        const long from = diff::piece(p0, n, blockIdx.x);
        w.left = diff::piece(p0, n, blockIdx.x + 1) - from;
        if (w.left > 0) {
          const diff::Span at = diff::span_find(P.kv_len, P.B, P.Sk, per, from);
          w.b = at.b, w.unit = at.unit, w.t = at.t;
        }
      }
      if (lane == 0) f_load_qk<D>(P, &mq, &mk, smem, sy, w, abort);
      __syncwarp();
    } else if (warp == 1) {
      if (elect_one()) f_qk<D>(P, smem, sy, tmem, abort);
      __syncwarp();
    } else if (warp == 2) {
      if (elect_one()) f_pv<D>(P, smem, sy, tmem, abort);
      __syncwarp();
    } else if (warp == 3) {
      f_load_v<D>(P, &mv, smem, sy, abort);
      __syncwarp();
    }
  } else if (warp < 12) {
    f_softmax<D>(P, smem, sy, tmem, abort);
  } else {
    f_output<D>(P, &mo, &mo2, smem, sy, tmem, abort);
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
cudaError_t launch_f(const DiffArgs &a, cudaStream_t st) {
  using C = FCfg<D>;
  const CrossShape &s = a.x.s;
  cudaError_t err;
  auto enc = tensor_map_encoder(&err);
  if (!enc) return err;
  const cross::Packing pk = cross::packing(s);
  const nabla_strides o_st{(int64_t)s.Sq * s.h * D, (int64_t)s.h * D, D};
  CUtensorMap mq, mk, mv, mo, mo2;
  if (!cross::cross_map(enc, &mq, a.x.q, s.B, s.Sq, s.h, D, a.x.q_st, pk.G, pk.tq) ||
      !cross::cross_map(enc, &mk, a.x.k, s.B, s.Sk, s.hk, D, a.x.k_st, 1, kStates) ||
      !cross::cross_map(enc, &mv, a.x.v, s.B, s.Sk, s.hk, D, a.x.v_st, 1, kStates) ||
      !cross::cross_map(enc, &mo, a.x.o, s.B, s.Sq, s.h, D, o_st, pk.G, pk.tq) ||
      !cross::cross_map(enc, &mo2, a.o2 ? a.o2 : a.x.o, s.B, s.Sq, s.h, D, o_st, pk.G, pk.tq))
    return cudaErrorInvalidValue;
  auto kern = diff_attn_tc_kernel<D>;
  if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  f_smem_bytes<D>())) != cudaSuccess)
    return err;
  FParams p{};
  p.o = static_cast<__nv_bfloat16 *>(a.x.o);
  p.o2 = static_cast<__nv_bfloat16 *>(a.o2);
  p.lse = a.x.lse;
  p.lam = a.lam, p.lam_step = a.lam_n > 1 ? 1 : 0;
  p.kv_len = a.x.kv_len;
  p.B = s.B, p.Sq = s.Sq, p.Sk = s.Sk, p.h = s.h, p.hk = s.hk;
  p.G = pk.G, p.tq = pk.tq;
  p.nqt = (pk.nsub + 1) / 2;
  // a scale of 0 weighs all states alike, as one too small to tell scores apart does
  p.scale_log2 = a.x.scale == 0.f ? 1e-30f : fabsf(a.x.scale) * 1.4426950408889634f;
  p.neg = a.x.scale < 0.f ? kIdescNegA : 0u;
  p.status = a.x.status;
  const DiffPlan plan = diff_fwd_plan(s, NABLA_BF16, a.x.kv_len != nullptr);
  p.whole = (uint32_t)plan.whole, p.cut = plan.cut;
  const DiffRuns parts = diff_runs(a, NABLA_BF16);
  p.po = parts.po, p.plse = parts.plse;
  const unsigned grid =
      plan.cut || plan.whole > diff::kCtas ? (unsigned)diff::kCtas : (unsigned)plan.whole;
  err = launch_pdl(kern, dim3(grid), dim3(C::kThreads), f_smem_bytes<D>(), st, mq, mk, mv, mo,
                   mo2, p);
  if (err != cudaSuccess || !plan.cut) return err;
  return launch_diff_stream_join(a, parts, st);
}

}  // namespace

cudaError_t launch_diff_attn_tc(const DiffArgs &a, cudaStream_t st) {
  return a.x.s.D == 64 ? launch_f<64>(a, st) : launch_f<128>(a, st);
}

}  // namespace nabla
