// C ABI of the NABLA hot path: argument checks, workspace layout, dispatch.
// The operations and their sources are documented in include/nabla.h.
#include <cmath>
#include <cstdint>
#include <utility>

#include "internal.h"

namespace nabla {

namespace {

constexpr int kMaxBlocks = 2048;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool valid_shape(int B, int S, int h, int D) {
  if (B < 1 || h < 1 || S < 64 || S % 64 != 0) return false;
  if (D != 64 && D != 128) return false;
  if (S / 64 > kMaxBlocks) return false;
  // element counts must fit the kernels' index arithmetic
  const double elems = (double)B * S * h * D;
  if (elems > 4.0e12) return false;
  if ((double)B * h * (S / 64) > 2.0e9) return false;
  return true;
}

bool valid_dtype(nabla_dtype dt) { return dt == NABLA_F32 || dt == NABLA_BF16; }

nabla_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NABLA_OK : NABLA_ERR_CUDA; }

// ---- tensors given by strides (nabla_strides)

// A [B, S, h, D] tensor's rows: the caller's strides, or the dense ones.
struct Rows {
  const void *p;
  nabla_strides st;
  int h;
};

Rows rows_of(const void *p, const nabla_strides *st, int B, int S, int h, int D) {
  Rows r{p, {(int64_t)S * h * D, (int64_t)h * D, D}, h};
  if (st) {
    if (B > 1) r.st.batch = st->batch;
    if (S > 1) r.st.token = st->token;
    if (h > 1) r.st.head = st->head;
  }
  return r;
}

bool valid_rows(const Rows &r, int B, int S, int D, size_t esz) {
  if (!r.p || !aligned(r.p, 16)) return false;
  int64_t st[3] = {r.st.head, r.st.token, r.st.batch}, n[3] = {r.h, S, B};
  for (int i = 0; i < 2; ++i)  // the smallest stride first
    for (int j = 0; j < 2 - i; ++j)
      if (st[j] > st[j + 1]) {
        std::swap(st[j], st[j + 1]);
        std::swap(n[j], n[j + 1]);
      }
  int64_t span = D;  // elements from the first to behind the last, dimension by dimension
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (st[i] < span || st[i] > (int64_t)1 << 38 || st[i] * esz % 16 != 0) return false;
    span += st[i] * (n[i] - 1);
  }
  return true;
}

// Bytes from the tensor's first element to behind its last.
uintptr_t extent(const Rows &r, int B, int S, int D, size_t esz) {
  return (uintptr_t)((B - 1) * r.st.batch + (S - 1) * r.st.token + (r.h - 1) * r.st.head + D) *
         esz;
}

bool ranges_meet(const void *a, uintptr_t an, const void *b, uintptr_t bn) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bn && b0 < a0 + an;
}

struct Range {
  const void *p;
  uintptr_t n;
};

// A tensor's dimensions larger than 1, the largest stride first; each stride is at least
// what the dimensions after it span (valid_rows).
struct Dim {
  int64_t st, n;
};
struct Nest {
  Dim d[3];
  int k;
};

Nest nest_of(const Rows &r, int B, int S) {
  const Dim all[3] = {{r.st.batch, B}, {r.st.token, S}, {r.st.head, r.h}};
  Nest v{};
  for (const Dim &d : all) {
    if (d.n == 1) continue;
    int at = v.k++;
    for (; at > 0 && v.d[at - 1].st < d.st; --at) v.d[at] = v.d[at - 1];
    v.d[at] = d;
  }
  return v;
}

int64_t nest_span(const Dim *d, int k, int D) {
  int64_t n = D;
  for (int i = 0; i < k; ++i) n += d[i].st * (d[i].n - 1);
  return n;
}

// Whether two tensors of rows of D elements share one, b's first element lying `off` behind
// a's.  The larger stride st is peeled off: step i of a and j of b lie off + (j - i) st
// apart, and what is inside a step spans at most st, so at most two values of j - i bring
// the insides together.  Exact where both have the same strides; where the inside of one
// spans more than the other's stride, they count as sharing.
bool nests_meet(const Dim *a, int ka, const Dim *b, int kb, int64_t off, int D) {
  if (off >= nest_span(a, ka, D) || -off >= nest_span(b, kb, D)) return false;
  if (ka == 0 && kb == 0) return true;
  const bool of_a = ka > 0 && (kb == 0 || a[0].st >= b[0].st);
  const bool of_b = kb > 0 && (ka == 0 || b[0].st >= a[0].st);
  const int64_t st = of_a ? a[0].st : b[0].st, na = of_a ? a[0].n : 1, nb = of_b ? b[0].n : 1;
  if (of_a) ++a, --ka;
  if (of_b) ++b, --kb;
  if (nest_span(a, ka, D) > st || nest_span(b, kb, D) > st) return true;
  const int64_t d = (off % st + st) % st;
  for (int64_t x : {d, d - st}) {
    const int64_t m = (x - off) / st;  // j - i
    if (m > -na && m < nb && nests_meet(a, ka, b, kb, x, D)) return true;
  }
  return false;
}

// Whether two [B, S, heads, D] tensors share elements.
bool rows_meet(const Rows &a, const Rows &b, int B, int S, int D, size_t esz) {
  const Nest x = nest_of(a, B, S), y = nest_of(b, B, S);
  const int64_t off = (int64_t)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p)) /
                      (int64_t)esz;
  return nests_meet(x.d, x.k, y.d, y.k, off, D);
}

}  // namespace

MaskWorkspace mask_workspace_layout(const Shape &s) {
  MaskWorkspace w{};
  w.mean_bytes = round_up((size_t)s.B * s.h * s.s1 * s.D * sizeof(float), 256);
  const size_t logits = (size_t)s.B * s.h * s.s1 * s.s1 * sizeof(float);
  w.qa_hi = 0;
  w.qa_lo = w.mean_bytes;
  w.ka_hi = 2 * w.mean_bytes;
  w.ka_lo = 3 * w.mean_bytes;
  w.logits = 4 * w.mean_bytes;
  w.total = round_up(w.logits + logits, 256);
  return w;
}

}  // namespace nabla

using nabla::Shape;

extern "C" {

int nabla_abi_version(void) { return 1; }

const char *nabla_status_string(nabla_status s) {
  switch (s) {
    case NABLA_OK: return "NABLA_OK";
    case NABLA_ERR_INVALID_ARG: return "NABLA_ERR_INVALID_ARG";
    case NABLA_ERR_UNSUPPORTED: return "NABLA_ERR_UNSUPPORTED";
    case NABLA_ERR_CUDA: return "NABLA_ERR_CUDA";
    case NABLA_ERR_TIMEOUT: return "NABLA_ERR_TIMEOUT";
    case NABLA_ERR_BAD_INDEX: return "NABLA_ERR_BAD_INDEX";
  }
  return "NABLA_ERR_UNKNOWN";
}

size_t nabla_build_mask_workspace_bytes(int B, int S, int h, int D) {
  if (!nabla::valid_shape(B, S, h, D)) return 0;
  return nabla::mask_workspace_layout(Shape{B, S, h, D, S / 64}).total;
}

nabla_status nabla_build_mask(const void *q, const void *k, nabla_dtype dt, int B, int S, int h,
                              int D, const uint8_t *sta, double thr, int32_t *kv_nb,
                              int32_t *kv_inds, void *workspace, size_t ws_bytes,
                              nabla_stream_t stream) {
  using namespace nabla;
  if (!valid_shape(B, S, h, D) || !valid_dtype(dt)) return NABLA_ERR_INVALID_ARG;
  if (!(thr > 0.0 && thr <= 1.0)) return NABLA_ERR_INVALID_ARG;  // also rejects NaN
  if (!q || !k || !sta || !kv_nb || !kv_inds || !workspace) return NABLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(workspace, 256) || !aligned(kv_nb, 4) ||
      !aligned(kv_inds, 4))
    return NABLA_ERR_INVALID_ARG;
  const Shape s{B, S, h, D, S / 64};
  const MaskWorkspace w = mask_workspace_layout(s);
  if (ws_bytes < w.total) return NABLA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  float *qa_hi = reinterpret_cast<float *>(ws + w.qa_hi);
  float *qa_lo = reinterpret_cast<float *>(ws + w.qa_lo);
  float *ka_hi = reinterpret_cast<float *>(ws + w.ka_hi);
  float *ka_lo = reinterpret_cast<float *>(ws + w.ka_lo);
  float *L = reinterpret_cast<float *>(ws + w.logits);
  const float t = (float)(1.0 - thr);  // cut level, formed in fp64 then rounded once
  const size_t lo_off = w.mean_bytes / sizeof(float);
  cudaError_t e;
  int *status = device_status_ptr(&e);
  if (!status) return NABLA_ERR_CUDA;
  e = launch_pool(q, k, dt, s, 0, h, qa_hi, ka_hi, lo_off, st);
  if (e == cudaSuccess) e = launch_pooled_map(qa_hi, qa_lo, ka_hi, ka_lo, s, 0, h, L, status, st);
  if (e == cudaSuccess) e = launch_select(L, s, 0, h, sta, t, kv_nb, kv_inds, st);
  return from_cuda(e);
}

nabla_status nabla_build_mask_topk(const void *q, const void *k, nabla_dtype dt, int B, int S,
                                   int h, int D, double topk_ratio, int32_t *kv_nb,
                                   int32_t *kv_inds, void *workspace, size_t ws_bytes,
                                   nabla_stream_t stream) {
  using namespace nabla;
  if (!valid_shape(B, S, h, D) || !valid_dtype(dt)) return NABLA_ERR_INVALID_ARG;
  if (!(topk_ratio >= 0.0) || !std::isfinite(topk_ratio)) return NABLA_ERR_INVALID_ARG;
  if (!q || !k || !kv_nb || !kv_inds || !workspace) return NABLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(workspace, 256) || !aligned(kv_nb, 4) ||
      !aligned(kv_inds, 4))
    return NABLA_ERR_INVALID_ARG;
  const Shape s{B, S, h, D, S / 64};
  const MaskWorkspace w = mask_workspace_layout(s);
  if (ws_bytes < w.total) return NABLA_ERR_INVALID_ARG;
  // topk = min(s1, floor(ratio * s1)), the product formed in fp64
  const double prod = topk_ratio * (double)s.s1;
  const int topk = prod >= (double)s.s1 ? s.s1 : (int)std::floor(prod);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (topk == 0)
    return from_cuda(cudaMemsetAsync(kv_nb, 0, (size_t)B * h * s.s1 * sizeof(int32_t), st));
  char *ws = static_cast<char *>(workspace);
  float *qa_hi = reinterpret_cast<float *>(ws + w.qa_hi);
  float *qa_lo = reinterpret_cast<float *>(ws + w.qa_lo);
  float *ka_hi = reinterpret_cast<float *>(ws + w.ka_hi);
  float *ka_lo = reinterpret_cast<float *>(ws + w.ka_lo);
  float *L = reinterpret_cast<float *>(ws + w.logits);
  const size_t lo_off = w.mean_bytes / sizeof(float);
  cudaError_t e;
  int *status = device_status_ptr(&e);
  if (!status) return NABLA_ERR_CUDA;
  e = launch_pool(q, k, dt, s, 0, h, qa_hi, ka_hi, lo_off, st);
  if (e == cudaSuccess) e = launch_pooled_map(qa_hi, qa_lo, ka_hi, ka_lo, s, 0, h, L, status, st);
  if (e == cudaSuccess) e = launch_select_topk(L, s, 0, h, topk, kv_nb, kv_inds, st);
  return from_cuda(e);
}

static nabla_status attn_fwd_call(const void *q, const void *k, const void *v, nabla_dtype dt,
                                  int B, int S, int h, int D, const int32_t *kv_nb,
                                  const int32_t *kv_inds, float scale, void *o, float *lse,
                                  nabla_stream_t stream) {
  using namespace nabla;
  if (!valid_shape(B, S, h, D) || !valid_dtype(dt)) return NABLA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return NABLA_ERR_INVALID_ARG;
  if (!q || !k || !v || !o || !kv_nb || !kv_inds) return NABLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(kv_nb, 4) || !aligned(kv_inds, 4) || !aligned(lse, 4))
    return NABLA_ERR_INVALID_ARG;
  const Shape s{B, S, h, D, S / 64};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  int *status = device_status_ptr(&e);
  if (!status) return NABLA_ERR_CUDA;
  if (dt == NABLA_BF16)
    e = launch_attn_tc(q, k, v, s, kv_nb, kv_inds, scale, o, lse, status, st);
  else
    e = launch_attn_simt(q, k, v, dt, s, kv_nb, kv_inds, scale, o, lse, status, st);
  return from_cuda(e);
}

nabla_status nabla_attn_fwd(const void *q, const void *k, const void *v, nabla_dtype dt, int B,
                            int S, int h, int D, const int32_t *kv_nb, const int32_t *kv_inds,
                            float scale, void *o, nabla_stream_t stream) {
  return attn_fwd_call(q, k, v, dt, B, S, h, D, kv_nb, kv_inds, scale, o, nullptr, stream);
}

nabla_status nabla_attn_fwd_lse(const void *q, const void *k, const void *v, nabla_dtype dt,
                                int B, int S, int h, int D, const int32_t *kv_nb,
                                const int32_t *kv_inds, float scale, void *o, float *lse,
                                nabla_stream_t stream) {
  if (!lse) return NABLA_ERR_INVALID_ARG;
  return attn_fwd_call(q, k, v, dt, B, S, h, D, kv_nb, kv_inds, scale, o, lse, stream);
}

size_t nabla_attn_bwd_workspace_bytes(int B, int S, int h, int D) {
  if (!nabla::valid_shape(B, S, h, D)) return 0;
  return nabla::bwd_workspace_layout(Shape{B, S, h, D, S / 64}).total;
}

nabla_status nabla_attn_bwd(const void *q, const void *k, const void *v, const void *o,
                            const float *lse, const void *dout, nabla_dtype dt, int B, int S,
                            int h, int D,
                            const int32_t *kv_nb, const int32_t *kv_inds, float scale, void *dq,
                            void *dk, void *dv, void *workspace, size_t ws_bytes,
                            nabla_stream_t stream) {
  using namespace nabla;
  if (!valid_shape(B, S, h, D) || !valid_dtype(dt)) return NABLA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return NABLA_ERR_INVALID_ARG;
  const void *in[] = {q, k, v, o, dout};
  void *out[] = {dq, dk, dv};
  for (const void *p : in)
    if (!p || !aligned(p, 16)) return NABLA_ERR_INVALID_ARG;
  for (void *p : out)
    if (!p || !aligned(p, 16)) return NABLA_ERR_INVALID_ARG;
  if (!kv_nb || !kv_inds || !workspace || !aligned(kv_nb, 4) || !aligned(kv_inds, 4) ||
      !aligned(workspace, 256) || !aligned(lse, 16))
    return NABLA_ERR_INVALID_ARG;
  const Shape s{B, S, h, D, S / 64};
  if (ws_bytes < bwd_workspace_layout(s).total) return NABLA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  int *status = device_status_ptr(&e);
  if (!status) return NABLA_ERR_CUDA;
  return from_cuda(launch_attn_bwd(q, k, v, o, lse, dout, dt, s, kv_nb, kv_inds, scale, dq, dk,
                                   dv, workspace, status, st));
}

static nabla_status fractal_call(const void *src, void *dst, bool flatten, nabla_dtype dt, int B,
                                 int T, int H, int W, int h, int D, int P,
                                 nabla_stream_t stream) {
  using namespace nabla;
  if (!valid_dtype(dt)) return NABLA_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || H < 1 || W < 1 || h < 1 || D < 1 || P < 1) return NABLA_ERR_INVALID_ARG;
  if (H % P != 0 || W % P != 0) return NABLA_ERR_INVALID_ARG;
  const double tokens = (double)B * T * H * W;
  const size_t esz = dt == NABLA_BF16 ? 2 : 4;
  const size_t row_bytes = (size_t)h * D * esz;
  if (row_bytes % 16 != 0 || tokens * (double)row_bytes > 1.0e13 || tokens > 4.0e12)
    return NABLA_ERR_INVALID_ARG;
  if (!src || !dst || !aligned(src, 16) || !aligned(dst, 16)) return NABLA_ERR_INVALID_ARG;
  const size_t bytes = (size_t)tokens * row_bytes;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(src), b0 = reinterpret_cast<uintptr_t>(dst);
  if (a0 < b0 + bytes && b0 < a0 + bytes) return NABLA_ERR_INVALID_ARG;  // overlapping buffers
  return from_cuda(launch_fractal(src, dst, flatten, B, T, H, W, P, row_bytes,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

nabla_status nabla_fractal_flatten(const void *x, nabla_dtype dt, int B, int T, int H, int W,
                                   int h, int D, int P, void *y, nabla_stream_t stream) {
  return fractal_call(x, y, true, dt, B, T, H, W, h, D, P, stream);
}

nabla_status nabla_fractal_unflatten(const void *y, nabla_dtype dt, int B, int T, int H, int W,
                                     int h, int D, int P, void *x, nabla_stream_t stream) {
  return fractal_call(y, x, false, dt, B, T, H, W, h, D, P, stream);
}

nabla_status nabla_sta_mask(int T, int H, int W, int wt, int wh, int ww, uint8_t *sta,
                            nabla_stream_t stream) {
  if (T < 1 || H < 1 || W < 1 || wt < 0 || wh < 0 || ww < 0 || !sta) return NABLA_ERR_INVALID_ARG;
  if ((long)T * H * W > nabla::kMaxBlocks) return NABLA_ERR_INVALID_ARG;
  return nabla::from_cuda(
      nabla::launch_sta(T, H, W, wt, wh, ww, sta, reinterpret_cast<cudaStream_t>(stream)));
}

// Checks and call of nabla_qk_norm_rope (dz all null) and its backward.
static nabla_status qk_norm_call(const void *const (&x)[2], const nabla_strides *const (&x_st)[2],
                                 const void *const (&dz)[2], const nabla_strides *const (&dz_st)[2],
                                 void *const (&out)[2], const nabla_strides *const (&out_st)[2],
                                 bool bwd, nabla_dtype dt, int B, int S, int hq, int hk, int D,
                                 const void *const (&w)[2], void *const (&dw)[2], nabla_dtype wdt,
                                 const float *cos_t, const float *sin_t, int rope_rows, int R,
                                 int interleaved, const int32_t *pos, float eps, void *workspace,
                                 size_t ws_bytes, nabla_stream_t stream) {
  using namespace nabla;
  if (!valid_dtype(dt) || !valid_dtype(wdt)) return NABLA_ERR_INVALID_ARG;
  if (B < 1 || S < 1 || hq < 1 || hk < 0 || (D != 64 && D != 128)) return NABLA_ERR_INVALID_ARG;
  if ((hk == 0) != (x[1] == nullptr)) return NABLA_ERR_INVALID_ARG;
  if ((double)B * S * ((double)hq + hk) * D > 4.0e12) return NABLA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return NABLA_ERR_INVALID_ARG;
  if (R < 0 || R > D || R % 16 != 0) return NABLA_ERR_INVALID_ARG;
  if (R > 0) {
    if (!cos_t || !sin_t || !aligned(cos_t, 16) || !aligned(sin_t, 16) || rope_rows < 1)
      return NABLA_ERR_INVALID_ARG;
    if (pos ? !aligned(pos, 4) : rope_rows < S) return NABLA_ERR_INVALID_ARG;
  }
  const size_t esz = dt == NABLA_BF16 ? 2 : 4, wsz = wdt == NABLA_BF16 ? 2 : 4;
  const int h[2] = {hq, hk}, sides = hk > 0 ? 2 : 1;
  QkNormArgs a{};
  Rows rx[2], rz[2], ro[2];
  for (int i = 0; i < sides; ++i) {
    rx[i] = rows_of(x[i], x_st[i], B, S, h[i], D);
    ro[i] = rows_of(out[i], out_st[i], B, S, h[i], D);
    if (!valid_rows(rx[i], B, S, D, esz) || !valid_rows(ro[i], B, S, D, esz))
      return NABLA_ERR_INVALID_ARG;
    if (bwd) {
      rz[i] = rows_of(dz[i], dz_st[i], B, S, h[i], D);
      if (!valid_rows(rz[i], B, S, D, esz)) return NABLA_ERR_INVALID_ARG;
    }
    if (!aligned(w[i], 16) || !aligned(dw[i], wsz)) return NABLA_ERR_INVALID_ARG;
    a.x[i] = x[i];
    a.dz[i] = dz[i];
    a.w[i] = w[i];
    a.out[i] = out[i];
    a.dw[i] = dw[i];
    a.x_st[i] = rx[i].st;
    a.out_st[i] = ro[i].st;
    if (bwd) a.dz_st[i] = rz[i].st;
    a.h[i] = h[i];
  }
  for (int i = 0; i < sides; ++i) {  // what is written overlaps nothing else
    const uintptr_t n = extent(ro[i], B, S, D, esz);
    for (int j = 0; j < sides; ++j) {
      if (rows_meet(ro[i], rx[j], B, S, D, esz) || (bwd && rows_meet(ro[i], rz[j], B, S, D, esz)))
        return NABLA_ERR_INVALID_ARG;
      const size_t row = (size_t)D * wsz;
      if (w[j] && (ranges_meet(ro[i].p, n, w[j], row) ||
                   (dw[i] && ranges_meet(dw[i], row, w[j], row))))
        return NABLA_ERR_INVALID_ARG;
      if (dw[j] && ranges_meet(ro[i].p, n, dw[j], row)) return NABLA_ERR_INVALID_ARG;
    }
  }
  if (sides == 2 && rows_meet(ro[0], ro[1], B, S, D, esz)) return NABLA_ERR_INVALID_ARG;
  if (bwd && (dw[0] || dw[1])) {
    if (dw[0] && dw[1] && ranges_meet(dw[0], (size_t)D * wsz, dw[1], (size_t)D * wsz))
      return NABLA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || ws_bytes < qk_norm_bwd_workspace(D))
      return NABLA_ERR_INVALID_ARG;
  }
  a.dt = dt;
  a.wdt = wdt;
  a.B = B;
  a.S = S;
  a.D = D;
  a.R = R;
  a.rope_rows = rope_rows;
  a.interleaved = interleaved != 0;
  a.cos_t = cos_t;
  a.sin_t = sin_t;
  a.pos = R > 0 ? pos : nullptr;
  a.eps = eps;
  a.workspace = workspace;
  cudaError_t e;
  a.status = device_status_ptr(&e);
  if (!a.status) return NABLA_ERR_CUDA;
  return from_cuda(launch_qk_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

nabla_status nabla_qk_norm_rope(const void *q, const nabla_strides *q_st, const void *k,
                                const nabla_strides *k_st, nabla_dtype dt, int B, int S, int hq,
                                int hk, int D, const void *wq, const void *wk, nabla_dtype wdt,
                                const float *cos_t, const float *sin_t, int rope_rows, int R,
                                int interleaved, const int32_t *pos, float eps, void *q_out,
                                const nabla_strides *qo_st, void *k_out,
                                const nabla_strides *ko_st, nabla_stream_t stream) {
  const void *x[2] = {q, k}, *none[2] = {}, *w[2] = {wq, wk};
  const nabla_strides *x_st[2] = {q_st, k_st}, *no_st[2] = {}, *out_st[2] = {qo_st, ko_st};
  void *out[2] = {q_out, k_out}, *dw[2] = {};
  return qk_norm_call(x, x_st, none, no_st, out, out_st, false, dt, B, S, hq, hk, D, w, dw, wdt,
                      cos_t, sin_t, rope_rows, R, interleaved, pos, eps, nullptr, 0, stream);
}

size_t nabla_qk_norm_rope_bwd_workspace_bytes(int D) {
  return D == 64 || D == 128 ? nabla::qk_norm_bwd_workspace(D) : 0;
}

nabla_status nabla_qk_norm_rope_bwd(
    const void *q, const nabla_strides *q_st, const void *k, const nabla_strides *k_st,
    nabla_dtype dt, int B, int S, int hq, int hk, int D, const void *wq, const void *wk,
    nabla_dtype wdt, const float *cos_t, const float *sin_t, int rope_rows, int R,
    int interleaved, const int32_t *pos, float eps, const void *dq_out,
    const nabla_strides *dqo_st, const void *dk_out, const nabla_strides *dko_st, void *dq,
    const nabla_strides *dq_st, void *dk, const nabla_strides *dk_st, void *dwq, void *dwk,
    void *workspace, size_t ws_bytes, nabla_stream_t stream) {
  const void *x[2] = {q, k}, *dz[2] = {dq_out, dk_out}, *w[2] = {wq, wk};
  const nabla_strides *x_st[2] = {q_st, k_st}, *dz_st[2] = {dqo_st, dko_st},
                      *out_st[2] = {dq_st, dk_st};
  void *out[2] = {dq, dk}, *dw[2] = {dwq, dwk};
  return qk_norm_call(x, x_st, dz, dz_st, out, out_st, true, dt, B, S, hq, hk, D, w, dw, wdt,
                      cos_t, sin_t, rope_rows, R, interleaved, pos, eps, workspace, ws_bytes,
                      stream);
}

namespace nabla {
namespace {

bool valid_cross_shape(const CrossShape &s) {
  if (s.B < 1 || s.Sq < 1 || s.Sk < 1 || s.h < 1 || s.hk < 1) return false;
  if (s.D != 64 && s.D != 128) return false;
  if (s.h % s.hk != 0 || s.h / s.hk > 64) return false;
  if (s.Sq > (1 << 30) || s.Sk > (1 << 30)) return false;
  // element counts and the grids' block counts must fit the kernels' arithmetic
  if ((double)s.B * s.Sq * s.h * s.D > 4.0e12 || (double)s.B * s.Sk * s.hk * s.D > 4.0e12)
    return false;
  return (double)s.B * s.h * s.Sq <= 2.0e9 && (double)s.B * s.h * s.Sk <= 2.0e9;
}

// Checks of q, k, v (and their strides, filled in) and kv_len; the rows' extents.
struct CrossRows {
  Rows q, k, v;
  uintptr_t qn, kn, vn;
};
bool valid_cross_inputs(CrossArgs &a, const nabla_strides *q_st, const nabla_strides *k_st,
                        const nabla_strides *v_st, size_t esz, CrossRows &r) {
  const CrossShape &s = a.s;
  if (!std::isfinite(a.scale) || !aligned(a.kv_len, 4)) return false;
  r.q = rows_of(a.q, q_st, s.B, s.Sq, s.h, s.D);
  r.k = rows_of(a.k, k_st, s.B, s.Sk, s.hk, s.D);
  r.v = rows_of(a.v, v_st, s.B, s.Sk, s.hk, s.D);
  if (!valid_rows(r.q, s.B, s.Sq, s.D, esz) || !valid_rows(r.k, s.B, s.Sk, s.D, esz) ||
      !valid_rows(r.v, s.B, s.Sk, s.D, esz))
    return false;
  a.q_st = r.q.st;
  a.k_st = r.k.st;
  a.v_st = r.v.st;
  r.qn = extent(r.q, s.B, s.Sq, s.D, esz);
  r.kn = extent(r.k, s.B, s.Sk, s.D, esz);
  r.vn = extent(r.v, s.B, s.Sk, s.D, esz);
  return true;
}
// Whether what is written (n bytes at p) meets an input.
bool meets_inputs(const void *p, uintptr_t n, const CrossArgs &a, const CrossRows &r) {
  return ranges_meet(p, n, r.q.p, r.qn) || ranges_meet(p, n, r.k.p, r.kn) ||
         ranges_meet(p, n, r.v.p, r.vn) ||
         (a.kv_len && ranges_meet(p, n, a.kv_len, (uintptr_t)a.s.B * 4));
}

}  // namespace
}  // namespace nabla

size_t nabla_cross_attn_fwd_workspace_bytes(nabla_dtype dt, int B, int Sq, int Sk, int h, int hk,
                                            int D) {
  const nabla::CrossShape s{B, Sq, Sk, h, hk, D};
  if (!nabla::valid_dtype(dt) || !nabla::valid_cross_shape(s)) return 0;
  return nabla::cross_fwd_workspace(s, dt);
}

nabla_status nabla_cross_attn_fwd(const void *q, const nabla_strides *q_st, const void *k,
                                  const nabla_strides *k_st, const void *v,
                                  const nabla_strides *v_st, nabla_dtype dt, int B, int Sq, int Sk,
                                  int h, int hk, int D, const int32_t *kv_len, float scale,
                                  void *o, float *lse, void *workspace, size_t ws_bytes,
                                  nabla_stream_t stream) {
  using namespace nabla;
  CrossArgs a{};
  a.s = CrossShape{B, Sq, Sk, h, hk, D};
  if (!valid_dtype(dt) || !valid_cross_shape(a.s)) return NABLA_ERR_INVALID_ARG;
  const size_t esz = dt == NABLA_BF16 ? 2 : 4;
  a.q = q;
  a.k = k;
  a.v = v;
  a.kv_len = kv_len;
  a.scale = scale;
  CrossRows r;
  if (!valid_cross_inputs(a, q_st, k_st, v_st, esz, r)) return NABLA_ERR_INVALID_ARG;
  const uintptr_t rows = (uintptr_t)B * Sq * h, on = rows * D * esz;
  if (!o || !aligned(o, 16) || !aligned(lse, 4) || meets_inputs(o, on, a, r) ||
      (lse && (meets_inputs(lse, rows * 4, a, r) || ranges_meet(o, on, lse, rows * 4))))
    return NABLA_ERR_INVALID_ARG;
  const size_t need = cross_fwd_workspace(a.s, dt);
  if (need && (!workspace || !aligned(workspace, 256) || ws_bytes < need))
    return NABLA_ERR_INVALID_ARG;
  a.o = o;
  a.lse = lse;
  a.workspace = workspace;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  a.status = device_status_ptr(&e);
  if (!a.status) return NABLA_ERR_CUDA;
  return from_cuda(dt == NABLA_BF16 ? launch_cross_attn_tc(a, st) : launch_cross_attn_simt(a, st));
}

size_t nabla_cross_attn_bwd_workspace_bytes(nabla_dtype dt, int B, int Sq, int Sk, int h, int hk,
                                            int D) {
  const nabla::CrossShape s{B, Sq, Sk, h, hk, D};
  if (!nabla::valid_dtype(dt) || !nabla::valid_cross_shape(s)) return 0;
  return nabla::cross_bwd_workspace(s, dt);
}

nabla_status nabla_cross_attn_bwd(const void *q, const nabla_strides *q_st, const void *k,
                                  const nabla_strides *k_st, const void *v,
                                  const nabla_strides *v_st, const void *o,
                                  const nabla_strides *o_st, const float *lse, const void *dout,
                                  const nabla_strides *dout_st, nabla_dtype dt, int B, int Sq,
                                  int Sk, int h, int hk, int D, const int32_t *kv_len, float scale,
                                  void *dq, void *dk, void *dv, void *workspace, size_t ws_bytes,
                                  nabla_stream_t stream) {
  using namespace nabla;
  CrossArgs a{};
  a.s = CrossShape{B, Sq, Sk, h, hk, D};
  if (!valid_dtype(dt) || !valid_cross_shape(a.s)) return NABLA_ERR_INVALID_ARG;
  const size_t esz = dt == NABLA_BF16 ? 2 : 4;
  a.q = q;
  a.k = k;
  a.v = v;
  a.kv_len = kv_len;
  a.scale = scale;
  CrossRows r;
  if (!valid_cross_inputs(a, q_st, k_st, v_st, esz, r)) return NABLA_ERR_INVALID_ARG;
  if (!lse || !dq || !dk || !dv || !workspace) return NABLA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(workspace, 256)) return NABLA_ERR_INVALID_ARG;
  const Rows ro = rows_of(o, o_st, B, Sq, h, D), rg = rows_of(dout, dout_st, B, Sq, h, D);
  if (!valid_rows(ro, B, Sq, D, esz) || !valid_rows(rg, B, Sq, D, esz))
    return NABLA_ERR_INVALID_ARG;
  a.o_st = ro.st;
  a.dout_st = rg.st;
  const uintptr_t rows = (uintptr_t)B * Sq * h, qn = rows * D * esz;
  const uintptr_t kn = (uintptr_t)B * Sk * hk * D * esz;
  void *const out[3] = {dq, dk, dv};
  const uintptr_t on[3] = {qn, kn, kn};
  for (int i = 0; i < 3; ++i) {
    if (!aligned(out[i], 16) || meets_inputs(out[i], on[i], a, r) ||
        ranges_meet(out[i], on[i], o, extent(ro, B, Sq, D, esz)) ||
        ranges_meet(out[i], on[i], dout, extent(rg, B, Sq, D, esz)) ||
        ranges_meet(out[i], on[i], lse, rows * 4))
      return NABLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (ranges_meet(out[i], on[i], out[j], on[j])) return NABLA_ERR_INVALID_ARG;
  }
  if (ws_bytes < cross_bwd_workspace(a.s, dt)) return NABLA_ERR_INVALID_ARG;
  a.of = o;
  a.lse = const_cast<float *>(lse);
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.workspace = workspace;
  cudaError_t e;
  a.status = device_status_ptr(&e);
  if (!a.status) return NABLA_ERR_CUDA;
  return from_cuda(launch_cross_bwd(a, dt, reinterpret_cast<cudaStream_t>(stream)));
}

namespace nabla {
namespace {

bool valid_norm_shape(const NormShape &s) {
  if (s.B < 1 || s.S < 1 || s.C < 8 || s.C > 8192 || s.C % 8 != 0) return false;
  return (double)s.B * s.S <= 2.0e9 && (double)s.B * s.S * s.C <= 4.0e12;
}

// What both directions of the block norm check: shape, norms, weights, modulations and
// scalars; collects the arrays that outputs must keep clear of.
struct NormCheck {
  NormArgs &a;
  size_t esz, wsz, msz;
  Range arrays[8];
  int count = 0;

  explicit NormCheck(NormArgs &args)
      : a(args),
        esz(args.dt == NABLA_BF16 ? 2 : 4),
        wsz(args.wdt == NABLA_BF16 ? 2 : 4),
        msz(args.mdt == NABLA_BF16 ? 2 : 4) {}

  bool array(const void *p, uintptr_t n) {
    if (!p) return true;
    if (!aligned(p, 16)) return false;
    arrays[count++] = Range{p, n};
    return true;
  }
  bool mod(const void *p, int64_t &st) {
    if (!p) return true;
    if (a.rows == 1) st = a.shape.C;
    if (st < a.shape.C || st > (int64_t)1 << 38 || st * msz % 16 != 0) return false;
    if ((double)(a.rows - 1) * (double)st > 4.0e12) return false;  // nor do its bytes wrap
    return array(p, (uintptr_t)((a.rows - 1) * st + a.shape.C) * msz);
  }
  bool common() {
    if (!valid_dtype(a.dt) || !valid_dtype(a.wdt) || !valid_dtype(a.mdt)) return false;
    if (!valid_norm_shape(a.shape)) return false;
    if (a.norm < 0 || a.norm > 2 || a.post < 0 || a.post > 2) return false;
    if (a.rows < 1 || (long)a.shape.B * a.shape.S % a.rows != 0) return false;
    if (!std::isfinite(a.rs) || !(a.eps >= 0.f) || !std::isfinite(a.eps)) return false;
    if (a.norm == 0 && (a.w || a.scale || a.shift)) return false;
    if (a.post == 0 && a.pw) return false;
    return array(a.w, a.shape.C * wsz) && array(a.pw, a.shape.C * wsz) &&
           mod(a.gate, a.gate_st) && mod(a.scale, a.scale_st) && mod(a.shift, a.shift_st);
  }
  // A [B, S, C] tensor that may be absent; its strides filled in.
  bool rows(const void *p, const nabla_strides *st, nabla_strides &to, Rows &r) {
    r = rows_of(p, st, a.shape.B, a.shape.S, 1, a.shape.C);
    to = r.st;
    return !p || valid_rows(r, a.shape.B, a.shape.S, a.shape.C, esz);
  }
  bool apart(const Rows &o, const Rows &in) const {
    return !o.p || !in.p || !rows_meet(o, in, a.shape.B, a.shape.S, a.shape.C, esz);
  }
  // `o` keeps clear of `in` or is it, row by row.
  bool apart_or_same(const Rows &o, const Rows &in) const {
    return apart(o, in) || (o.p == in.p && (a.shape.B == 1 || o.st.batch == in.st.batch) &&
                            (a.shape.S == 1 || o.st.token == in.st.token));
  }
  bool clear_of_arrays(const Rows &o) const {
    const uintptr_t n = o.p ? extent(o, a.shape.B, a.shape.S, a.shape.C, esz) : 0;
    for (int i = 0; i < count && o.p; ++i)
      if (ranges_meet(o.p, n, arrays[i].p, arrays[i].n)) return false;
    return true;
  }
};

}  // namespace
}  // namespace nabla

nabla_status nabla_block_norm(const void *x, const nabla_strides *x_st, const void *u,
                              const nabla_strides *u_st, nabla_dtype dt, int B, int S, int C,
                              nabla_norm norm, nabla_norm post, const void *weight,
                              const void *post_weight, nabla_dtype wdt, const void *gate,
                              int64_t gate_st, const void *scale, int64_t scale_st,
                              const void *shift, int64_t shift_st, nabla_dtype mdt, int rows,
                              float residual_scale, float eps, void *x_out,
                              const nabla_strides *xo_st, void *y, const nabla_strides *y_st,
                              nabla_stream_t stream) {
  using namespace nabla;
  NormArgs a{};
  a.shape = NormShape{B, S, C};
  a.x = x, a.u = u, a.s = x_out, a.y = y;
  a.w = weight, a.pw = post_weight, a.gate = gate, a.scale = scale, a.shift = shift;
  a.gate_st = gate_st, a.scale_st = scale_st, a.shift_st = shift_st;
  a.dt = dt, a.wdt = wdt, a.mdt = mdt;
  a.rows = rows, a.norm = norm, a.post = post, a.rs = residual_scale, a.eps = eps;
  NormCheck c(a);
  if (!x || !c.common()) return NABLA_ERR_INVALID_ARG;
  if ((u == nullptr) != (x_out == nullptr) || (norm == 0) != (y == nullptr) || (!u && !y))
    return NABLA_ERR_INVALID_ARG;
  if (!u && (gate || post != 0)) return NABLA_ERR_INVALID_ARG;
  Rows rx, ru, rs, ry;
  if (!c.rows(x, x_st, a.x_st, rx) || !c.rows(u, u_st, a.u_st, ru) ||
      !c.rows(x_out, xo_st, a.s_st, rs) || !c.rows(y, y_st, a.y_st, ry))
    return NABLA_ERR_INVALID_ARG;
  if (!c.apart_or_same(rs, rx) || !c.apart(rs, ru) || !c.apart(ry, rx) || !c.apart(ry, ru) ||
      !c.apart(ry, rs) || !c.clear_of_arrays(rs) || !c.clear_of_arrays(ry))
    return NABLA_ERR_INVALID_ARG;
  cudaError_t e;
  a.status = device_status_ptr(&e);
  if (!a.status) return NABLA_ERR_CUDA;
  return from_cuda(launch_block_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t nabla_block_norm_bwd_workspace_bytes(int B, int S, int C) {
  const nabla::NormShape s{B, S, C};
  return nabla::valid_norm_shape(s) ? nabla::block_norm_bwd_workspace(s) : 0;
}

nabla_status nabla_block_norm_bwd(
    const void *s, const nabla_strides *s_st, const void *u, const nabla_strides *u_st,
    const void *dsum, const nabla_strides *dsum_st, const void *dy, const nabla_strides *dy_st,
    nabla_dtype dt, int B, int S, int C, nabla_norm norm, nabla_norm post, const void *weight,
    const void *post_weight, nabla_dtype wdt, const void *gate, int64_t gate_st,
    const void *scale, int64_t scale_st, nabla_dtype mdt, int rows, float residual_scale,
    float eps, void *dx, const nabla_strides *dx_st, void *du, const nabla_strides *du_st,
    void *dgate, void *dscale, void *dshift, void *dweight, void *dpost_weight, void *workspace,
    size_t ws_bytes, nabla_stream_t stream) {
  using namespace nabla;
  NormArgs a{};
  a.shape = NormShape{B, S, C};
  a.x = s, a.u = u, a.dsum = dsum, a.dy = dy, a.dx = dx, a.du = du;
  a.w = weight, a.pw = post_weight, a.gate = gate, a.scale = scale;
  a.gate_st = gate_st, a.scale_st = scale_st;
  a.dw = dweight, a.dpw = dpost_weight, a.dgate = dgate, a.dscale = dscale, a.dshift = dshift;
  a.dt = dt, a.wdt = wdt, a.mdt = mdt;
  a.rows = rows, a.norm = norm, a.post = post, a.rs = residual_scale, a.eps = eps;
  a.bwd = true;
  NormCheck c(a);
  if (!c.common()) return NABLA_ERR_INVALID_ARG;
  if ((norm == 0) != (s == nullptr) || (norm == 0) != (dy == nullptr)) return NABLA_ERR_INVALID_ARG;
  if (norm == 0 && (dscale || dshift || dweight)) return NABLA_ERR_INVALID_ARG;
  if (!u && (post != 0 || dgate || dpost_weight)) return NABLA_ERR_INVALID_ARG;
  if (post == 0 && dpost_weight) return NABLA_ERR_INVALID_ARG;
  if ((!dsum && !dy) || (!dx && !du && !dgate && !dscale && !dshift && !dweight && !dpost_weight))
    return NABLA_ERR_INVALID_ARG;
  Rows r[4], o[2];
  if (!c.rows(s, s_st, a.x_st, r[0]) || !c.rows(u, u_st, a.u_st, r[1]) ||
      !c.rows(dsum, dsum_st, a.dsum_st, r[2]) || !c.rows(dy, dy_st, a.dy_st, r[3]) ||
      !c.rows(dx, dx_st, a.dx_st, o[0]) || !c.rows(du, du_st, a.du_st, o[1]))
    return NABLA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i) {
    for (int j = 0; j < 4; ++j)
      if (i == 0 && j == 2 ? !c.apart_or_same(o[i], r[j]) : !c.apart(o[i], r[j]))
        return NABLA_ERR_INVALID_ARG;
    if (!c.clear_of_arrays(o[i])) return NABLA_ERR_INVALID_ARG;
  }
  if (!c.apart(o[0], o[1])) return NABLA_ERR_INVALID_ARG;
  // the small gradients keep clear of everything else, too
  const uintptr_t mn = (uintptr_t)rows * C * c.msz, wn = (uintptr_t)C * c.wsz;
  const Range small[5] = {{dgate, mn}, {dscale, mn}, {dshift, mn}, {dweight, wn},
                          {dpost_weight, wn}};
  bool any = false;
  for (int i = 0; i < 5; ++i) {
    const Range &g = small[i];
    if (!g.p) continue;
    any = true;
    if (!aligned(g.p, 16)) return NABLA_ERR_INVALID_ARG;
    for (int j = 0; j < c.count; ++j)
      if (ranges_meet(g.p, g.n, c.arrays[j].p, c.arrays[j].n)) return NABLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (small[j].p && ranges_meet(g.p, g.n, small[j].p, small[j].n)) return NABLA_ERR_INVALID_ARG;
    for (const Rows *t : {&r[0], &r[1], &r[2], &r[3], &o[0], &o[1]})
      if (t->p && ranges_meet(g.p, g.n, t->p, extent(*t, B, S, C, c.esz)))
        return NABLA_ERR_INVALID_ARG;
  }
  if (any && (!workspace || !aligned(workspace, 256) ||
              ws_bytes < block_norm_bwd_workspace(a.shape)))
    return NABLA_ERR_INVALID_ARG;
  a.workspace = workspace;
  cudaError_t e;
  a.status = device_status_ptr(&e);
  if (!a.status) return NABLA_ERR_CUDA;
  return from_cuda(launch_block_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

namespace nabla {
namespace {

// lam: [1] or [h] fp32, kept clear of what is written.
bool valid_lam(const float *lam, int n, int h) {
  return lam && aligned(lam, 4) && (n == 1 || n == h);
}

}  // namespace
}  // namespace nabla

size_t nabla_diff_attn_fwd_workspace_bytes(nabla_dtype dt, int B, int Sq, int Sk, int h, int hk,
                                           int D) {
  const nabla::CrossShape s{B, Sq, Sk, h, hk, D};
  if (!nabla::valid_dtype(dt) || !nabla::valid_cross_shape(s)) return 0;
  return nabla::diff_fwd_workspace(s, dt);
}

nabla_status nabla_diff_attn_fwd(const void *q, const nabla_strides *q_st, const void *k,
                                 const nabla_strides *k_st, const void *v,
                                 const nabla_strides *v_st, nabla_dtype dt, int B, int Sq, int Sk,
                                 int h, int hk, int D, const float *lam, int lam_n,
                                 const int32_t *kv_len, float scale, void *o, void *o2, float *lse,
                                 void *workspace, size_t ws_bytes, nabla_stream_t stream) {
  using namespace nabla;
  DiffArgs a{};
  a.x.s = CrossShape{B, Sq, Sk, h, hk, D};
  if (!valid_dtype(dt) || !valid_cross_shape(a.x.s) || !valid_lam(lam, lam_n, h))
    return NABLA_ERR_INVALID_ARG;
  const size_t esz = dt == NABLA_BF16 ? 2 : 4;
  a.x.q = q, a.x.k = k, a.x.v = v;
  a.x.kv_len = kv_len;
  a.x.scale = scale;
  CrossRows r;
  if (!valid_cross_inputs(a.x, q_st, k_st, v_st, esz, r)) return NABLA_ERR_INVALID_ARG;
  const uintptr_t rows = (uintptr_t)B * Sq * h, on = rows * D * esz;
  if (!o || !aligned(o, 16) || !aligned(o2, 16) || !aligned(lse, 4)) return NABLA_ERR_INVALID_ARG;
  const Range out[3] = {{o, on}, {o2, on}, {lse, rows * 8}};
  for (int i = 0; i < 3; ++i) {
    if (!out[i].p) continue;
    if (meets_inputs(out[i].p, out[i].n, a.x, r) ||
        ranges_meet(out[i].p, out[i].n, lam, (uintptr_t)lam_n * 4))
      return NABLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (out[j].p && ranges_meet(out[i].p, out[i].n, out[j].p, out[j].n))
        return NABLA_ERR_INVALID_ARG;
  }
  const size_t need = diff_fwd_workspace(a.x.s, dt);
  if (need && (!workspace || !aligned(workspace, 256) || ws_bytes < need))
    return NABLA_ERR_INVALID_ARG;
  a.x.o = o, a.o2 = o2, a.x.lse = lse;
  a.lam = lam, a.lam_n = lam_n;
  a.x.workspace = workspace;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  a.x.status = device_status_ptr(&e);
  if (!a.x.status) return NABLA_ERR_CUDA;
  if (diff_few_rows(a.x.s, dt)) return from_cuda(launch_diff_few(a, dt, st));
  return from_cuda(dt == NABLA_BF16 ? launch_diff_attn_tc(a, st) : launch_diff_attn_simt(a, st));
}

size_t nabla_diff_attn_bwd_workspace_bytes(nabla_dtype dt, int B, int Sq, int Sk, int h, int hk,
                                           int D) {
  const nabla::CrossShape s{B, Sq, Sk, h, hk, D};
  if (!nabla::valid_dtype(dt) || !nabla::valid_cross_shape(s)) return 0;
  return nabla::diff_bwd_workspace(s, dt);
}

nabla_status nabla_diff_attn_bwd(const void *q, const nabla_strides *q_st, const void *k,
                                 const nabla_strides *k_st, const void *v,
                                 const nabla_strides *v_st, const void *o,
                                 const nabla_strides *o_st, const void *o2,
                                 const nabla_strides *o2_st, const float *lse, const void *dout,
                                 const nabla_strides *dout_st, nabla_dtype dt, int B, int Sq,
                                 int Sk, int h, int hk, int D, const float *lam, int lam_n,
                                 const int32_t *kv_len, float scale, void *dq, void *dk, void *dv,
                                 float *dlam, void *workspace, size_t ws_bytes,
                                 nabla_stream_t stream) {
  using namespace nabla;
  DiffArgs a{};
  a.x.s = CrossShape{B, Sq, Sk, h, hk, D};
  if (!valid_dtype(dt) || !valid_cross_shape(a.x.s) || !valid_lam(lam, lam_n, h))
    return NABLA_ERR_INVALID_ARG;
  const size_t esz = dt == NABLA_BF16 ? 2 : 4;
  a.x.q = q, a.x.k = k, a.x.v = v;
  a.x.kv_len = kv_len;
  a.x.scale = scale;
  CrossRows r;
  if (!valid_cross_inputs(a.x, q_st, k_st, v_st, esz, r)) return NABLA_ERR_INVALID_ARG;
  if (!lse || !dq || !dk || !dv || !dlam || !workspace) return NABLA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(dlam, 4) || !aligned(workspace, 256))
    return NABLA_ERR_INVALID_ARG;
  const Rows in[3] = {rows_of(o, o_st, B, Sq, h, D), rows_of(o2, o2_st, B, Sq, h, D),
                      rows_of(dout, dout_st, B, Sq, h, D)};
  for (const Rows &t : in)
    if (!valid_rows(t, B, Sq, D, esz)) return NABLA_ERR_INVALID_ARG;
  a.x.o_st = in[0].st, a.o2_st = in[1].st, a.x.dout_st = in[2].st;
  const uintptr_t rows = (uintptr_t)B * Sq * h, kn = (uintptr_t)B * Sk * hk * D * esz;
  const Range out[4] = {{dq, rows * D * esz}, {dk, kn}, {dv, kn}, {dlam, (uintptr_t)lam_n * 4}};
  for (int i = 0; i < 4; ++i) {
    if ((i < 3 && !aligned(out[i].p, 16)) || meets_inputs(out[i].p, out[i].n, a.x, r) ||
        ranges_meet(out[i].p, out[i].n, lse, rows * 8) ||
        ranges_meet(out[i].p, out[i].n, lam, (uintptr_t)lam_n * 4))
      return NABLA_ERR_INVALID_ARG;
    for (const Rows &t : in)
      if (ranges_meet(out[i].p, out[i].n, t.p, extent(t, B, Sq, D, esz)))
        return NABLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (ranges_meet(out[i].p, out[i].n, out[j].p, out[j].n)) return NABLA_ERR_INVALID_ARG;
  }
  if (ws_bytes < diff_bwd_workspace(a.x.s, dt)) return NABLA_ERR_INVALID_ARG;
  a.x.of = o, a.o2f = o2;
  a.x.lse = const_cast<float *>(lse);
  a.x.dout = dout;
  a.x.dq = dq, a.x.dk = dk, a.x.dv = dv;
  a.lam = lam, a.lam_n = lam_n, a.dlam = dlam;
  a.x.workspace = workspace;
  cudaError_t e;
  a.x.status = device_status_ptr(&e);
  if (!a.x.status) return NABLA_ERR_CUDA;
  return from_cuda(launch_diff_bwd(a, dt, reinterpret_cast<cudaStream_t>(stream)));
}

nabla_status nabla_selftest_bounded_wait(nabla_stream_t stream) {
  return nabla::from_cuda(nabla::launch_bounded_wait_probe(reinterpret_cast<cudaStream_t>(stream)));
}

nabla_status nabla_get_last_device_status(nabla_stream_t stream) {
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return NABLA_ERR_CUDA;
  int *status = nabla::device_status_ptr(&e);
  if (!status) return NABLA_ERR_CUDA;
  int host = 0;
  e = cudaMemcpy(&host, status, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return NABLA_ERR_CUDA;
  if (host != 0) {
    const int zero = 0;
    e = cudaMemcpy(status, &zero, sizeof(int), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return NABLA_ERR_CUDA;
  }
  return static_cast<nabla_status>(host);
}

}  // extern "C"
