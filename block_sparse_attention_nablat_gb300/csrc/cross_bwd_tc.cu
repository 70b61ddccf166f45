// K10 -- bf16 cross attention backward on the tcgen05 tensor cores.
//
// With z = scale q k^T over a batch's states, P = softmax(z) = 2^(z log2(e) - lse),
// delta_s = dout_s . o_s and dz = P (dout v^T - delta):
//   dV = P^T dout,  dK = scale dz^T q,  dQ = scale dz k,
// dK and dV summed over the heads that share a key head (their rows are packed into one
// tile, cross_common.cuh, so the sum is the product's own).
//
// Few states and many queries, so two kernels, each with its accumulators in TMEM from
// the first step of a unit to the last, and no atomics:
//
//  * dK, dV: unit = a tile of 128 states of one (batch, key head) over a run of the
//    query tiles.  Its K and V rows stay in shared memory as A operands; a step takes a
//    tile of 128 packed query rows: X = K Q^T, Y = V dO^T (SS MMAs, M = N = 128),
//    P^T = 2^(X - lse), dz^T = P^T (Y - delta) as bf16 over X and Y in TMEM, then
//    dV += P^T dO, dK += dz^T Q (TS MMAs).  TMEM holds dK, dV, X and Y: 4 x 128 columns.
//    One warp issues dV and X (which goes over P), another dK and Y: two chains that fill
//    each other's gaps.  (One warp for all four, in the best order, leaves the tensor pipe
//    to drain at every wait: 3500 cycles a step where two take 2900, of 2048 in the pipe.)
//    Where there are few state tiles the query tiles are split over several units whose
//    fp32 sums cross_dkv_join adds up in a fixed order.
//  * dQ: unit = a tile of 128 packed query rows over the batch's state tiles.  X = Q K^T,
//    Y = dO V^T, dz as bf16 in one of two buffers, dQ += dz K.  X and Y are free for the
//    next step as soon as the softmax warps have them in registers.
//    Few units are split over runs of the states (cross_dq_splits), whose fp32 sums
//    cross_dq_sum adds up in order.
//
// Eight softmax warps: thread = TMEM lane, group grp takes columns 64 grp .. + 63; P stays
// in fp32 registers between the two phases.  States past kv_len: dK/dV rows of P and dz
// are 0 there; in dQ their columns are 0 and the rows of K that share the last 16-row MMA
// step with them are zeroed in shared memory.  Query rows that are none (a tile's end)
// have lse = +inf, so P = 0.
//
// 32768 tokens, 24 heads, D 128, 512 states: 589 us in all, 875 TFLOP/s of the five
// products (0.45 of a large library product's rate): rows' lse and delta 72, dK and dV 281
// (tensor pipe 63% active), their sum 11, dQ 218 (59%).  4096 states: 3.8 to 4.0 ms, 1040 to
// 1080.  Of the 319 us above the five products' 270, X and Y formed a second time are 108, the
// pass before them 72, the sum 11, and what the two kernels take beyond their seven products'
// time about 125: a step of dK / dV waits for the chain X, P, dV, next X (X goes over P: TMEM
// is full), one of dQ for V's tile, which is loaded when the last Y is done, and for the
// products' own chain.  At D 64 the products take half the time and the softmax as long: 433 us
// at 512 states, 2.81 ms at 4096.
// Measured and not kept: dO as dQ's TMEM operand, which makes room for a second V tile,
// but starts a unit later: 4096 states 3.80 ms, 512 584 us, 256 416 against 399; dQ started
// on the SMs that dK / dV leave: 600 against 595 at 512 states, 313 against 321 at 128.
// Every mbarrier wait is bounded (1 s), as in the forward.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "cross_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace nabla {
namespace {

using namespace tc;
using cross::kTile;
using tcattn::add2;
using tcattn::f2;
using tcattn::fma2;
using tcattn::Ring;
using tcattn::unf2;

template <int D>
struct YCfg {
  static constexpr int kBoxes = D / 64;   // 64-column (128-byte) swizzle boxes
  static constexpr int kBox = 128 * 128;  // one box of a 128-row tile
  static constexpr int kTileBytes = kBoxes * kBox;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kThreads = 384;
  static constexpr uint32_t kIdSS = idesc_bf16(128, 128, 0, 0);
  static constexpr uint32_t kIdTS = idesc_bf16(128, D, 0, 1);
  // dK / dV: K, V, three Q tiles, two dO tiles, two sets of a step's lse and delta
  static constexpr int kQ = 3, kG = 2;
  static constexpr int kOffK = 0, kOffV = kTileBytes, kOffQ = 2 * kTileBytes;
  static constexpr int kOffG = kOffQ + kQ * kTileBytes;
  static constexpr int kOffL = kOffG + kG * kTileBytes;
  static constexpr int kOffSync1 = kOffL + kG * 1024;
  static constexpr uint32_t kDK = 0, kDV = 128, kX1 = 256, kY1 = 384;
  // dQ: two Q tiles, dO, three K tiles, V (two tiles where there is room: with one, its
  // loads bound a step)
  static constexpr int kK = 3, kV = D == 64 ? 2 : 1;
  static constexpr int kOffG2 = 2 * kTileBytes, kOffK2 = 3 * kTileBytes;
  static constexpr int kOffV2 = kOffK2 + kK * kTileBytes;
  static constexpr int kOffSync2 = kOffV2 + kV * kTileBytes;
  static constexpr uint32_t kDQ = 0, kX2 = 128, kY2 = 256, kZ = 384;  // dz buffer b: + 64 b
};

struct KSync {
  uint64_t kv_full, kv_empty, q_full[3], q_empty[3], g_full[2], g_empty[2];
  uint64_t x_full, y_full, p_full[2], z_full[2], dv_done, dk_done, acc_full, acc_free, drain;
  uint32_t tmem_slot;
  int abort;
};
struct QSync {
  uint64_t q_full[2], q_empty[2], g_full, g_empty, k_full[3], k_empty[3], k_raw;
  uint64_t v_full[2], v_empty[2];
  uint64_t x_full, y_full, x_free, y_free, z_full[2], acc_full, out_full, drain;
  uint32_t tmem_slot;
  int abort;
};
template <int D, bool kDQ>
constexpr int y_smem_bytes() {
  return kDQ ? YCfg<D>::kOffSync2 + (int)sizeof(QSync) : YCfg<D>::kOffSync1 + (int)sizeof(KSync);
}
static_assert(y_smem_bytes<128, false>() <= 232448, "shared memory budget (dK, dV)");
static_assert(y_smem_bytes<128, true>() <= 232448, "shared memory budget (dQ)");

struct YParams {
  __nv_bfloat16 *dq, *dk, *dv;  // [B, Sq, h, D], [B, Sk, hk, D]
  float *part;                  // dK / dV sums of the runs: [nsplit][2][B, Sk, hk, D]
  const float *nlse, *ndelta;   // -lse, -delta of the packed rows: [B, hk, 2 nq, 64]
  const int32_t *kv_len;
  int B, Sq, Sk, h, hk, G, tq, nq, nkt, nsplit;  // nq: tiles of 128 packed rows
  uint32_t units;
  cross::WalkStep walk;
  float scale, scale_log2;  // scale_log2 of |scale|, never 0
  uint32_t neg;             // kIdescNegA for a negative scale
  int *status;
};

__device__ __forceinline__ void y_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// D (+)= A B^T over D columns, both operands K-major 128-row tiles (one thread).
template <int D>
__device__ __forceinline__ void issue_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t at = (uint64_t)(((kk >> 2) * YCfg<D>::kBox + (kk & 3) * 32) >> 4);
    mma_ss(d, a + at, b + at, id, kk > 0 ? 1u : 0u);
  }
}
// The half of such a product: 16-row steps 2 half, 2 half + 1 of each side (the first 32
// of every 64 columns of A, or the others).
template <int D>
__device__ __forceinline__ void issue_ts_half(uint32_t d, uint32_t a, uint32_t right, uint64_t b,
                                              int half, bool first) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int kk = (x >> 1) * 4 + half * 2 + (x & 1);
    mma_ts(d, a + (kk >> 2) * right + (kk & 3) * 8, b + (uint64_t)((kk * 16 * 128) >> 4),
           YCfg<D>::kIdTS, x > 0 || half > 0 || !first ? 1u : 0u);
  }
}
// D += A B, A 128 columns of bf16 in TMEM from `a` on (columns 64.. at `a` + right),
// B an MN-major 128-row tile.
template <int D>
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint32_t right, uint64_t b,
                                         bool first) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(d, a + (kk >> 2) * right + (kk & 3) * 8, b + (uint64_t)((kk * 16 * 128) >> 4),
           YCfg<D>::kIdTS, kk > 0 || !first ? 1u : 0u);
}

// ---------------------------------------------------------------- dK, dV

struct KUnit {
  int b, j, kt, sp, len, i0, n;  // n query tiles from i0
};
__device__ __forceinline__ KUnit k_unit(const YParams &P, const cross::Walk &w) {
  KUnit r{w.b, w.j, w.t, w.sp, cross::batch_len(P.kv_len, w.b, P.Sk), 0, 0};
  if (r.kt * kTile >= r.len) return r;  // no states: nothing to walk
  r.i0 = (int)((long)P.nq * r.sp / P.nsplit);
  r.n = (int)((long)P.nq * (r.sp + 1) / P.nsplit) - r.i0;
  return r;
}

// Warp 0, lane 0: the unit's K and V, then the steps' Q, dO, lse and delta.
template <int D>
__device__ void k_load(const YParams &P, const CUtensorMap *mq, const CUtensorMap *mk,
                       const CUtensorMap *mv, const CUtensorMap *mg, uint8_t *smem, KSync *sy,
                       volatile int *abort) {
  using C = YCfg<D>;
  Ring<C::kQ> q;
  Ring<C::kG> gr;
  uint32_t g = 0, ku = 0;
  bool go = true;
  const uint32_t rows = (uint32_t)(P.G * P.tq) * 128 * 2 * C::kBoxes;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && go && !*abort;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const KUnit u = k_unit(P, w);
    cross::check_len(P.kv_len, u.b, P.Sk, P.status);
    if (u.n == 0) continue;
    go = mbar_wait_small(&sy->kv_empty, (ku & 1u) ^ 1u, abort, P.status, kDevTimeout);
    if (!go) break;
    mbar_expect_tx(&sy->kv_full, 2 * C::kTileBytes);
    for (int c = 0; c < C::kBoxes; ++c) {
      tma_load_4d(smem + C::kOffK + c * C::kBox, mk, &sy->kv_full, c * 64, u.j, u.kt * kTile, u.b);
      tma_load_4d(smem + C::kOffV + c * C::kBox, mv, &sy->kv_full, c * 64, u.j, u.kt * kTile, u.b);
    }
    ++ku;
    for (int i = 0; i < u.n && go; ++i, ++g) {
      go = mbar_wait_small(&sy->q_empty[q.slot], q.phase ^ 1u, abort, P.status, kDevTimeout);
      if (!go) break;
      const int t0 = (u.i0 + i) * 2 * P.tq;
      mbar_expect_tx(&sy->q_full[q.slot], rows);
#pragma unroll 1
      for (int x = 0; x < 2 * C::kBoxes; ++x)  // box x / 2, subtile x & 1
        tma_load_4d(smem + C::kOffQ + q.slot * C::kTileBytes + (x >> 1) * C::kBox +
                        (x & 1) * 64 * 128,
                    mq, &sy->q_full[q.slot], (x >> 1) * 64, u.j * P.G, t0 + (x & 1) * P.tq, u.b);
      q.next();
      go = mbar_wait_small(&sy->g_empty[gr.slot], gr.phase ^ 1u, abort, P.status, kDevTimeout);
      if (!go) break;
      mbar_expect_tx(&sy->g_full[gr.slot], rows + 1024);
      const size_t at = ((size_t)((uint32_t)u.b * P.hk + u.j) * P.nq + u.i0 + i) * 128;
      bulk_load(smem + C::kOffL + gr.slot * 1024, P.nlse + at, 512, &sy->g_full[gr.slot]);
      bulk_load(smem + C::kOffL + gr.slot * 1024 + 512, P.ndelta + at, 512, &sy->g_full[gr.slot]);
#pragma unroll 1
      for (int x = 0; x < 2 * C::kBoxes; ++x)
        tma_load_4d(smem + C::kOffG + gr.slot * C::kTileBytes + (x >> 1) * C::kBox +
                        (x & 1) * 64 * 128,
                    mg, &sy->g_full[gr.slot], (x >> 1) * 64, u.j * P.G, t0 + (x & 1) * P.tq, u.b);
      gr.next();
    }
  }
  if (!go || *abort) {  // let copies in flight land before the CTA exits (Q may be one ahead)
    for (uint32_t s = 0; s < (uint32_t)C::kQ; ++s) {
      const uint32_t used = q.slot > s ? 1u : 0u;  // the slot's last use has this ring phase
      if (g > 0 || used)
        mbar_wait_small(&sy->q_full[s], used ? q.phase : q.phase ^ 1u, nullptr, P.status,
                        kDevTimeout);
    }
    for (uint32_t s = 0; s < (uint32_t)C::kG && g > 0; ++s)
      mbar_wait_small(&sy->g_full[s], gr.slot > s ? gr.phase : gr.phase ^ 1u, nullptr, P.status,
                      kDevTimeout);
    if (ku > 0)
      mbar_wait_small(&sy->kv_full, (ku - 1) & 1u, nullptr, P.status, kDevTimeout);
  }
}

// A wait of a whole warp that goes on in step.
__device__ __forceinline__ bool k_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                       int *status) {
  return __all_sync(0xffffffffu, cross::thread_wait(bar, parity, abort, status));
}

// Warp 1 (kV): dV += P^T dO and X = K Q^T.  Warp 2: dK += dz^T Q and Y = V dO^T.  Each
// chain's SS product of a step goes over the columns its TS product of the step before
// has read; the TS product starts on the first half of P or dz.  (As single threads, the form of
// the other kernels, the two chains are 4% slower: 288 against 280 us at 32768 x 512,
// 2286 against 2203 at 32768 x 4096, 24 heads, D 128.)
template <int D, bool kV>
__device__ void k_mma(const YParams &P, uint8_t *smem, KSync *sy, uint32_t tmem,
                      volatile int *abort) {
  using C = YCfg<D>;
  const uint64_t a_desc = smem_desc_sw128(smem_u32(smem + (kV ? C::kOffK : C::kOffV)), 16, 1024);
  const uint64_t b_desc = smem_desc_sw128(smem_u32(smem + (kV ? C::kOffQ : C::kOffG)), 16, 1024);
  const uint64_t t_desc =
      smem_desc_sw128(smem_u32(smem + (kV ? C::kOffG : C::kOffQ)), C::kBox, 1024);
  const uint32_t xy = tmem + (kV ? C::kX1 : C::kY1), acc = tmem + (kV ? C::kDV : C::kDK);
  uint64_t *b_full = kV ? sy->q_full : sy->g_full, *t_full = kV ? sy->g_full : sy->q_full;
  uint64_t *ss_full = kV ? &sy->x_full : &sy->y_full;  // X or Y of a step is there
  uint64_t *a_full = kV ? sy->p_full : sy->z_full;     // the halves of its P or dz are there
  uint64_t *ts_done = kV ? &sy->dv_done : &sy->dk_done;
  Ring<kV ? C::kQ : C::kG> br;  // of the SS product's tile, and of the TS product's
  Ring<kV ? C::kG : C::kQ> tr;
  uint32_t g = 0, ku = 0;
  bool ok = true;
  auto issue = [&](bool last) {  // the SS product of the next step
    tc_fence_after();
    if (elect_one()) {
      issue_ss<D>(xy, a_desc, b_desc + (uint64_t)((br.slot * C::kTileBytes) >> 4),
                  kV ? C::kIdSS | P.neg : C::kIdSS);
      mma_commit(ss_full);
      if (!kV) mma_commit(&sy->g_empty[br.slot]);
      if (last) mma_commit(&sy->kv_empty);
    }
    __syncwarp();
    br.next();
  };
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && ok;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const KUnit u = k_unit(P, w);
    if (u.n == 0) continue;
    ok = k_wait(&sy->kv_full, ku & 1u, abort, P.status) &&
         k_wait(&b_full[br.slot], br.phase, abort, P.status) &&
         (g == 0 || k_wait(ts_done, (g - 1) & 1u, abort, P.status));
    if (!ok) break;
    issue(u.n == 1);
    // the last unit's rows of dK and dV have been read
    if (ku > 0) ok = k_wait(&sy->acc_free, (ku - 1) & 1u, abort, P.status);
    for (int i = 0; i < u.n && ok; ++i, ++g) {
      const bool more = i + 1 < u.n;
      ok = k_wait(&t_full[tr.slot], tr.phase, abort, P.status);
      const uint64_t b = t_desc + (uint64_t)((tr.slot * C::kTileBytes) >> 4);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (ok) ok = k_wait(&a_full[half], g & 1u, abort, P.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ts_half<D>(acc, xy, 64, b, half, i == 0);
          if (half) {
            mma_commit(ts_done);
            mma_commit(kV ? &sy->g_empty[tr.slot] : &sy->q_empty[tr.slot]);
            if (!more) mma_commit(&sy->acc_full);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      tr.next();
      if (more) {
        ok = k_wait(&b_full[br.slot], br.phase, abort, P.status) &&
             k_wait(ts_done, g & 1u, abort, P.status);
        if (ok) issue(i + 2 == u.n);
      }
    }
    ++ku;
  }
  if (elect_one()) mma_commit(&sy->drain);  // never exit with MMAs in flight
  __syncwarp();
  mbar_wait_small(&sy->drain, 0, nullptr, P.status, kDevTimeout);
}

// Warps 4-11: P^T and dz^T of every step, then the unit's rows of dK and dV.  Thread =
// state, columns = query rows, whose lse and delta come with dO.  Each half (32 of a
// group's 64 columns) is handed on as it is written.
template <int D>
__device__ void k_softmax(const YParams &P, uint8_t *smem, KSync *sy, uint32_t tmem,
                          volatile int *abort) {
  using C = YCfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
  const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16);
  const uint32_t xa = at + C::kX1 + grp * 64, ya = at + C::kY1 + grp * 64;
  const uint64_t sc2 = f2(P.scale_log2, P.scale_log2);
  Ring<C::kG> gr;
  uint32_t g = 0, ku = 0;
  bool live = true;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const KUnit u = k_unit(P, w);
    const int state = u.kt * kTile + row;
    const bool act = state < u.len;
    for (int i = 0; i < u.n; ++i, ++g, gr.next()) {
      cross::warp_wait(live, &sy->g_full[gr.slot], gr.phase, abort, P.status);
      cross::warp_wait(live, &sy->x_full, g & 1u, abort, P.status);
      tc_fence_after();
      const float *ld = reinterpret_cast<const float *>(smem + C::kOffL + gr.slot * 1024) +
                        grp * 64;
      float p[64];
      uint32_t r[2][32], pk[16];
      tmem_ld32(xa, r[0]);
      tmem_ld32(xa + 32, r[1]);
      tmem_wait_ld();
      reg_fence(r[0]);
      reg_fence(r[1]);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float *ph = p + half * 32;
        const uint32_t *rh = r[half];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const ulonglong2 nl = *reinterpret_cast<const ulonglong2 *>(ld + half * 32 + e);
          unf2(fma2(f2(__uint_as_float(rh[e]), __uint_as_float(rh[e + 1])), sc2, nl.x), ph[e],
               ph[e + 1]);
          unf2(fma2(f2(__uint_as_float(rh[e + 2]), __uint_as_float(rh[e + 3])), sc2, nl.y),
               ph[e + 2], ph[e + 3]);
#pragma unroll
          for (int y = 0; y < 4; ++y) ph[e + y] = ex2(ph[e + y]);
          pk[e >> 1] = act ? pack_bf16x2(ph[e], ph[e + 1]) : 0u;
          pk[(e >> 1) + 1] = act ? pack_bf16x2(ph[e + 2], ph[e + 3]) : 0u;
        }
        tmem_st16(xa + half * 16, pk);  // over scores this thread has read
        tmem_wait_st();
        tc_fence_before();
        y_arrive(&sy->p_full[half], lane);
      }
      cross::warp_wait(live, &sy->y_full, g & 1u, abort, P.status);
      tc_fence_after();
      tmem_ld32(ya, r[0]);
      tmem_ld32(ya + 32, r[1]);
      tmem_wait_ld();
      reg_fence(r[0]);
      reg_fence(r[1]);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float *ph = p + half * 32;
        const uint32_t *rh = r[half];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const ulonglong2 nd = *reinterpret_cast<const ulonglong2 *>(ld + 128 + half * 32 + e);
          float a, b, c, d;
          unf2(mul2(f2(ph[e], ph[e + 1]),
                    add2(f2(__uint_as_float(rh[e]), __uint_as_float(rh[e + 1])), nd.x)), a, b);
          unf2(mul2(f2(ph[e + 2], ph[e + 3]),
                    add2(f2(__uint_as_float(rh[e + 2]), __uint_as_float(rh[e + 3])), nd.y)), c,
               d);
          pk[e >> 1] = act ? pack_bf16x2(a, b) : 0u;
          pk[(e >> 1) + 1] = act ? pack_bf16x2(c, d) : 0u;
        }
        tmem_st16(ya + half * 16, pk);
        tmem_wait_st();
        tc_fence_before();
        y_arrive(&sy->z_full[half], lane);
      }
      if (lane == 0) mbar_arrive(&sy->g_empty[gr.slot]);  // lse and delta have been read
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
          tmem_ld16(at + (dv ? C::kDV : C::kDK) + c, t);
          tmem_wait_ld();
          reg_fence16(t);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) t[e] = 0u;
        }
        if (state >= P.Sk) continue;
        const float m = dv ? 1.f : P.scale;
        if (P.nsplit > 1) {
          float4 *o = reinterpret_cast<float4 *>(P.part + ((size_t)u.sp * 2 + dv) * all + orow +
                                                 c);
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
      y_arrive(&sy->acc_free, lane);
      ++ku;
    }
  }
}

// Rows of the ring's query tiles that no box fills (G not dividing 64) as zeros.
template <int D>
__device__ void zero_gap(uint8_t *tiles, int ntiles, int used) {
  const int per = (64 - used) * 8;
  for (int e = threadIdx.x; e < per * 2 * YCfg<D>::kBoxes * ntiles; e += YCfg<D>::kThreads) {
    const int sub = e / per, to = e - sub * per;
    *reinterpret_cast<uint4 *>(tiles + sub * 64 * 128 + used * 128 + to * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    cross_dkv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg,
                     const __grid_constant__ YParams P) {
  using C = YCfg<D>;
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
    for (int i = 0; i < C::kQ; ++i) {
      mbar_init(&sy->q_full[i], 1);
      mbar_init(&sy->q_empty[i], 1);
    }
    for (int i = 0; i < C::kG; ++i) {
      mbar_init(&sy->g_full[i], 1);
      mbar_init(&sy->g_empty[i], 2 + 8);  // both chains, the softmax warps
    }
    mbar_init(&sy->x_full, 1);
    mbar_init(&sy->y_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sy->p_full[i], 8);
      mbar_init(&sy->z_full[i], 8);
    }
    mbar_init(&sy->dv_done, 1);
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
  zero_gap<D>(smem + C::kOffQ, C::kQ + C::kG, P.G * P.tq);
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
    k_mma<D, true>(P, smem, sy, tmem, abort);
  } else if (warp == 2) {
    k_mma<D, false>(P, smem, sy, tmem, abort);
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
__device__ __forceinline__ QUnit q_unit(const YParams &P, const cross::Walk &w) {
  QUnit r{w.b, w.j, w.t, w.sp, cross::batch_len(P.kv_len, w.b, P.Sk), 0, 0};
  r.n = (r.len + kTile - 1) / kTile;
  if (P.nsplit > 1) {  // a run of them
    r.t0 = (int)((long)r.n * r.sp / P.nsplit);
    r.n = (int)((long)r.n * (r.sp + 1) / P.nsplit) - r.t0;
  }
  return r;
}

// Warp 0, lane 0: the units' Q (a unit ahead) and dO.
template <int D>
__device__ void q_load(const YParams &P, const CUtensorMap *mq, const CUtensorMap *mg,
                       uint8_t *smem, QSync *sy, volatile int *abort) {
  using C = YCfg<D>;
  Ring<2> q;
  uint32_t ku = 0;
  bool go = true;
  const uint32_t rows = (uint32_t)(P.G * P.tq) * 128 * 2 * C::kBoxes;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units && go && !*abort;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
    const QUnit u = q_unit(P, w);
    if (u.n == 0) continue;
#pragma unroll 1
    for (int which = 0; which < 2 && go; ++which) {  // Q, then dO
      uint64_t *full = which ? &sy->g_full : &sy->q_full[q.slot];
      go = mbar_wait_small(which ? &sy->g_empty : &sy->q_empty[q.slot],
                           (which ? ku & 1u : q.phase) ^ 1u, abort, P.status, kDevTimeout);
      if (!go) break;
      uint8_t *tile = smem + (which ? C::kOffG2 : (int)q.slot * C::kTileBytes);
      mbar_expect_tx(full, rows);
#pragma unroll 1
      for (int x = 0; x < 2 * C::kBoxes; ++x)
        tma_load_4d(tile + (x >> 1) * C::kBox + (x & 1) * 64 * 128, which ? mg : mq, full,
                    (x >> 1) * 64, u.j * P.G, (u.qt * 2 + (x & 1)) * P.tq, u.b);
    }
    if (!go) break;
    q.next();
    ++ku;
  }
  if (!go || *abort) {
    // at most the last unit's copies and, where the loop broke between the two, one Q more
    for (uint32_t s = 0; s < 2; ++s)
      if (ku > s)
        mbar_wait_small(&sy->q_full[s], q.slot > s ? q.phase : q.phase ^ 1u, nullptr, P.status,
                        kDevTimeout);
    if (ku > 0) mbar_wait_small(&sy->g_full, (ku - 1) & 1u, nullptr, P.status, kDevTimeout);
    if (!go) mbar_wait_small(&sy->q_full[q.slot], q.phase, nullptr, P.status, kDevTimeout);
  }
}

// Warp 3: K and V of every step.  A K tile whose last 16 rows reach past the length comes
// in on k_raw: the warp zeroes those rows, then hands the tile on.
template <int D>
__device__ void q_load_kv(const YParams &P, const CUtensorMap *mk, const CUtensorMap *mv,
                          uint8_t *smem, QSync *sy, volatile int *abort) {
  using C = YCfg<D>;
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
      const int rows = u.len - (u.t0 + t) * kTile, end = rows >= kTile ? kTile : (rows + 15) & ~15;
      const bool mend = rows < end && u.len < P.Sk;  // zero K's rows [rows, end)
      uint8_t *tile = smem + C::kOffK2 + kr.slot * C::kTileBytes;
      bool ok = true;
      if (lane == 0) {
        ok = !*abort && mbar_wait_small(&sy->k_empty[kr.slot], kr.phase ^ 1u, abort, P.status,
                                        kDevTimeout);
        if (ok) {
          uint64_t *bar = mend ? &sy->k_raw : &sy->k_full[kr.slot];
          mbar_expect_tx(bar, C::kTileBytes);
          for (int c = 0; c < C::kBoxes; ++c)
            tma_load_4d(tile + c * C::kBox, mk, bar, c * 64, u.j, (u.t0 + t) * kTile, u.b);
          if (mend) ok = mbar_wait_small(&sy->k_raw, raw & 1u, nullptr, P.status, kDevTimeout);
        }
      }
      go = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!go) break;
      if (mend) {
        ++raw;
        const int n16 = (end - rows) * 8;
        for (int c = 0; c < C::kBoxes; ++c)
          for (int e = lane; e < n16; e += 32)
            *reinterpret_cast<uint4 *>(tile + c * C::kBox + rows * 128 + e * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sy->k_full[kr.slot]);
      }
      if (lane == 0) {
        ok = cross::thread_wait(&sy->v_empty[vr.slot], vr.phase ^ 1u, abort, P.status);
        if (ok) {
          mbar_expect_tx(&sy->v_full[vr.slot], C::kTileBytes);
          for (int c = 0; c < C::kBoxes; ++c)
            tma_load_4d(smem + C::kOffV2 + vr.slot * C::kTileBytes + c * C::kBox, mv,
                        &sy->v_full[vr.slot], c * 64, u.j, (u.t0 + t) * kTile, u.b);
        } else {  // the K tile of this step is in flight
          mbar_wait_small(&sy->k_full[kr.slot], kr.phase, nullptr, P.status, kDevTimeout);
        }
      }
      go = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!go) break;
    }
  }
  if (lane == 0 && (!go || *abort)) {
    for (uint32_t e = g > (uint32_t)C::kK ? g - C::kK : 0u; e < g; ++e)
      mbar_wait_small(&sy->k_full[e % C::kK], (e / C::kK) & 1u, nullptr, P.status, kDevTimeout);
    for (uint32_t e = g > (uint32_t)C::kV ? g - C::kV : 0u; e < g; ++e)
      mbar_wait_small(&sy->v_full[e % C::kV], (e / C::kV) & 1u, nullptr, P.status, kDevTimeout);
  }
}

// Warp 1: all products: X = Q K^T, Y = dO V^T of every step, each over the last step's
// once the softmax warps hold that, and dQ += dz K of the step before.  A step's X is
// committed after the dQ of two steps before, so x_full also says that the dz buffer is
// free; and dz of a unit's first step comes after the last unit's rows were read, so it
// says that dQ may be written over.  Y of a unit's first step comes after that dQ, since
// it may still wait for dO.
template <int D>
__device__ void q_mma(const YParams &P, uint8_t *smem, QSync *sy, uint32_t tmem,
                      volatile int *abort) {
  using C = YCfg<D>;
  const uint64_t q_desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t g_desc = smem_desc_sw128(smem_u32(smem + C::kOffG2), 16, 1024);
  const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + C::kOffK2), 16, 1024);
  const uint64_t k_mn = smem_desc_sw128(smem_u32(smem + C::kOffK2), C::kBox, 1024);
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
    const uint64_t b = k_mn + (uint64_t)((kd.slot * C::kTileBytes) >> 4);
    if (left > kTile - 16) {
      issue_ts<D>(tmem + C::kDQ, a, 32, b, first);
    } else {  // the batch's last tile: its 16-state steps only
#pragma unroll 1
      for (int kk = 0; kk * 16 < left; ++kk)
        mma_ts(tmem + C::kDQ, a + kk * 8, b + (uint64_t)((kk * 16 * 128) >> 4), C::kIdTS,
               kk > 0 || !first ? 1u : 0u);
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
      issue_ss<D>(tmem + C::kX2, q_desc + (uint64_t)((q.slot * C::kTileBytes) >> 4),
                  k_desc + (uint64_t)((kr.slot * C::kTileBytes) >> 4), C::kIdSS | P.neg);
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
      issue_ss<D>(tmem + C::kY2, g_desc, v_desc + (uint64_t)((vr.slot * C::kTileBytes) >> 4),
                  C::kIdSS);
      mma_commit(&sy->y_full);
      mma_commit(&sy->v_empty[vr.slot]);
      vr.next();
      if (t + 1 == u.n) mma_commit(&sy->g_empty);
      if (t > 0) issue_dq(false);
      left = u.len - (u.t0 + t) * kTile;
    }
    q.next();
    ++ku;
  }
  if (ok && g > 0) issue_dq(true);
  mma_commit(&sy->drain);
  mbar_wait_small(&sy->drain, 0, nullptr, P.status, kDevTimeout);
}

// Warp 2: hands the units' rows from their Q tiles to the TMA, and the tiles back to the
// loader once they have been read.
template <int D>
__device__ void q_store(const YParams &P, const CUtensorMap *mo, const uint8_t *smem, QSync *sy,
                        volatile int *abort) {
  using C = YCfg<D>;
  uint32_t ku = 0;
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  for (uint32_t i0 = blockIdx.x; i0 < P.units;
       i0 += gridDim.x, cross::walk_next(P.walk, w)) {
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

// Warps 4-11: dz of every step, and the units' rows of dQ (through the unit's Q tile,
// which no MMA reads any more).  Thread = query row, columns = states.  A
// unit's rows are written in the first step of the next unit, after its exponentials, so
// that the last dQ product runs meanwhile.
template <int D>
__device__ void q_softmax(const YParams &P, uint8_t *smem, QSync *sy, uint32_t tmem,
                          volatile int *abort) {
  using C = YCfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane, r64 = row & 63;
  const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16);
  const uint64_t sc2 = f2(P.scale_log2, P.scale_log2);
  const int tok = r64 / P.G, head = r64 - tok * P.G;
  uint32_t g = 0, ku = 0;
  bool live = true;
  QUnit last{};              // unit ku - 1
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
      tmem_ld32(at + C::kDQ + c, t);
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
    y_arrive(&sy->out_full, lane);
  };
  auto rows_at = [&](const cross::Walk &w) {
    return ((size_t)((uint32_t)w.b * P.hk + w.j) * P.nq + w.t) * 128 + row;
  };
  cross::Walk w = cross::walk_start(P.walk, blockIdx.x);
  float nl_next = 0.f, nd_next = 0.f;
  if (blockIdx.x < P.units) {
    const size_t r = rows_at(w);
    nl_next = __ldg(P.nlse + r);
    nd_next = __ldg(P.ndelta + r);
  }
  for (uint32_t i0 = blockIdx.x; i0 < P.units; i0 += gridDim.x) {
    const QUnit c = q_unit(P, w);
    const float nl = nl_next, nd = nd_next;
    cross::walk_next(P.walk, w);
    if (i0 + gridDim.x < P.units) {  // the next unit's rows, long before they are needed
      const size_t r = rows_at(w);
      nl_next = __ldg(P.nlse + r);
      nd_next = __ldg(P.ndelta + r);
    }
    if (c.n == 0) {
      const int token = (c.qt * 2 + (row >> 6)) * P.tq + tok, hh = c.j * P.G + head;
      if (P.nsplit == 1 && tok < P.tq && token < P.Sq) {
        uint4 *o = reinterpret_cast<uint4 *>(
            P.dq + (((size_t)c.b * P.Sq + token) * P.h + hh) * D + grp * (D / 2));
#pragma unroll 1
        for (int e = 0; e < D / 16; ++e) o[e] = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    const uint64_t nl2 = f2(nl, nl), nd2 = f2(nd, nd);
    for (int t = 0; t < c.n; ++t, ++g) {
      const int mine = c.len - (c.t0 + t) * kTile - grp * 64;  // own columns that are states
      cross::warp_wait(live, &sy->x_full, g & 1u, abort, P.status);
      tc_fence_after();
      uint32_t x0[32], x1[32];
      tmem_ld32(at + C::kX2 + grp * 64, x0);
      tmem_ld32(at + C::kX2 + grp * 64 + 32, x1);
      tmem_wait_ld();
      reg_fence(x0);
      reg_fence(x1);
      tc_fence_before();
      y_arrive(&sy->x_free, lane);
      float p[64];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        unf2(fma2(f2(__uint_as_float(x0[e]), __uint_as_float(x0[e + 1])), sc2, nl2), p[e],
             p[e + 1]);
        unf2(fma2(f2(__uint_as_float(x1[e]), __uint_as_float(x1[e + 1])), sc2, nl2), p[32 + e],
             p[33 + e]);
        p[e] = ex2(p[e]);
        p[e + 1] = ex2(p[e + 1]);
        p[32 + e] = ex2(p[32 + e]);
        p[33 + e] = ex2(p[33 + e]);
      }
      if (t == 0 && ku > 0) write_rows();
      cross::warp_wait(live, &sy->y_full, g & 1u, abort, P.status);
      tc_fence_after();
      tmem_ld32(at + C::kY2 + grp * 64, x0);
      tmem_ld32(at + C::kY2 + grp * 64 + 32, x1);
      tmem_wait_ld();
      reg_fence(x0);
      reg_fence(x1);
      tc_fence_before();
      y_arrive(&sy->y_free, lane);
      uint32_t pk[16];
      const uint32_t za = at + C::kZ + (g & 1u) * 64 + grp * 32;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint32_t ya = half ? x1[e] : x0[e], yb = half ? x1[e + 1] : x0[e + 1];
          float a, b;
          unf2(mul2(f2(p[half * 32 + e], p[half * 32 + e + 1]),
                    add2(f2(__uint_as_float(ya), __uint_as_float(yb)), nd2)),
               a, b);
          pk[e >> 1] = pack_bf16x2(a, b);
        }
        if (mine < 64) {  // past the length: 0, whatever was computed there
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int col = half * 32 + 2 * e;
            pk[e] = col + 1 < mine ? pk[e] : col < mine ? pk[e] & 0xffffu : 0u;
          }
        }
        tmem_st16(za + half * 16, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      y_arrive(&sy->z_full[g & 1u], lane);
    }
    last = c;
    ++ku;
  }
  if (ku > 0) write_rows();
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg,
                    const __grid_constant__ CUtensorMap mo, const __grid_constant__ YParams P) {
  using C = YCfg<D>;
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
  zero_gap<D>(smem, 3, P.G * P.tq);  // Q tiles and dO
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

// dQ of runs: their sums added up in order, scaled and rounded.  A thread per four columns.
__global__ void __launch_bounds__(256)
    cross_dq_sum_kernel(const __grid_constant__ YParams P, long n4, int row) {
  pdl_launch_dependents();
  pdl_wait();
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const long e = i * 4;
  const int b = (int)(e / row / P.Sq);
  const int tiles = (cross::batch_len(P.kv_len, b, P.Sk) + kTile - 1) / kTile;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int sp = 0; sp < P.nsplit; ++sp) {
    if ((long)tiles * sp / P.nsplit == (long)tiles * (sp + 1) / P.nsplit) continue;  // no states
    const float4 x = *reinterpret_cast<const float4 *>(P.part + (size_t)sp * n4 * 4 + e);
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
  }
  *reinterpret_cast<uint2 *>(P.dq + e) = make_uint2(pack_bf16x2(s.x * P.scale, s.y * P.scale),
                                                    pack_bf16x2(s.z * P.scale, s.w * P.scale));
}

template <int D>
cudaError_t launch_y(const CrossArgs &a, const float *nlse, const float *ndelta, float *part,
                     float *qpart, cudaStream_t st) {
  using C = YCfg<D>;
  const CrossShape &s = a.s;
  cudaError_t err;
  auto enc = tensor_map_encoder(&err);
  if (!enc) return err;
  const cross::Packing pk = cross::packing(s);
  const nabla_strides dq_st{(int64_t)s.Sq * s.h * D, (int64_t)s.h * D, D};
  CUtensorMap mq, mk, mv, mg, mo;
  if (!cross::cross_map(enc, &mq, a.q, s.B, s.Sq, s.h, D, a.q_st, pk.G, pk.tq) ||
      !cross::cross_map(enc, &mk, a.k, s.B, s.Sk, s.hk, D, a.k_st, 1, kTile) ||
      !cross::cross_map(enc, &mv, a.v, s.B, s.Sk, s.hk, D, a.v_st, 1, kTile) ||
      !cross::cross_map(enc, &mg, a.dout, s.B, s.Sq, s.h, D, a.dout_st, pk.G, pk.tq) ||
      !cross::cross_map(enc, &mo, a.dq, s.B, s.Sq, s.h, D, dq_st, pk.G, pk.tq))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
  if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return err;
  YParams p{};
  p.dq = static_cast<__nv_bfloat16 *>(a.dq);
  p.dk = static_cast<__nv_bfloat16 *>(a.dk);
  p.dv = static_cast<__nv_bfloat16 *>(a.dv);
  p.part = part;
  p.nlse = nlse;
  p.ndelta = ndelta;
  p.kv_len = a.kv_len;
  p.B = s.B, p.Sq = s.Sq, p.Sk = s.Sk, p.h = s.h, p.hk = s.hk;
  p.G = pk.G, p.tq = pk.tq, p.nq = (pk.nsub + 1) / 2, p.nkt = (s.Sk + kTile - 1) / kTile;
  p.nsplit = cross_dkv_splits(s, NABLA_BF16);
  p.scale = a.scale;
  p.scale_log2 = a.scale == 0.f ? 1e-30f : fabsf(a.scale) * 1.4426950408889634f;
  p.neg = a.scale < 0.f ? kIdescNegA : 0u;
  p.status = a.status;
  p.units = (uint32_t)((long)s.B * s.hk * p.nkt * p.nsplit);
  auto kern = cross_dkv_kernel<D>;
  if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  y_smem_bytes<D, false>())) != cudaSuccess)
    return err;
  unsigned grid = p.units < (unsigned)sms ? p.units : (unsigned)sms;
  p.walk = cross::walk_step(grid, p.nsplit, p.nkt, s.hk);
  err = launch_pdl(kern, dim3(grid), dim3(C::kThreads), y_smem_bytes<D, false>(), st, mq, mk, mv,
                   mg, p);
  if (err == cudaSuccess && p.nsplit > 1)
    err = launch_cross_dkv_join(a, NABLA_BF16, part, p.nsplit, st);
  if (err != cudaSuccess) return err;
  p.nsplit = cross_dq_splits(s);
  p.part = qpart;
  p.units = (uint32_t)((long)s.B * s.hk * p.nq * p.nsplit);
  auto kern2 = cross_dq_kernel<D>;
  if ((err = cudaFuncSetAttribute(kern2, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  y_smem_bytes<D, true>())) != cudaSuccess)
    return err;
  grid = p.units < (unsigned)sms ? p.units : (unsigned)sms;
  p.walk = cross::walk_step(grid, p.nsplit, p.nq, s.hk);
  err = launch_pdl(kern2, dim3(grid), dim3(C::kThreads), y_smem_bytes<D, true>(), st, mq, mk, mv,
                   mg, mo, p);
  if (err != cudaSuccess || p.nsplit == 1) return err;
  const long n4 = (long)s.B * s.Sq * s.h * (D / 4);
  return launch_pdl(cross_dq_sum_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, st, p,
                    n4, s.h * D);
}

}  // namespace

cudaError_t launch_cross_bwd_tc(const CrossArgs &a, const float *nlse, const float *ndelta,
                                float *part, float *qpart, cudaStream_t st) {
  return a.s.D == 64 ? launch_y<64>(a, nlse, ndelta, part, qpart, st)
                     : launch_y<128>(a, nlse, ndelta, part, qpart, st);
}

}  // namespace nabla
