// C entry points of the layer-computation operators: argument checks and
// kernel parameters.  Every rejected call returns before any launch.
#include <math.h>
#include <nvtx3/nvToolsExt.h>

#include "zero_ops.h"

namespace {

using zk::mat;

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

#define ZERO_TRY(x)               \
  do {                            \
    const int _s = (x);           \
    if (_s != ZERO_OK) return _s; \
  } while (0)

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return ZERO_OK;
  zk::record_cuda_error((int)e);
  return ZERO_ECUDA;
}

constexpr int64_t kMost = (int64_t)1 << 31;   // row distances stay below,
constexpr int64_t kMostSize = kMost - 1024;  // sizes so far below that tiles rounded up do too

int check_sizes(int64_t a, int64_t b, int64_t c = 0) {
  if (a < 0 || b < 0 || c < 0) return ZERO_EINVAL;
  return a < kMostSize && b < kMostSize && c < kMostSize ? ZERO_OK : ZERO_ERANGE;
}

int check_dtype(int d) { return d == ZERO_F32 || d == ZERO_BF16 ? ZERO_OK : ZERO_EDTYPE; }

int check_aligned(const void* p, int dtype) {
  return ((uintptr_t)p & (dtype == ZERO_F32 ? 3u : 1u)) == 0 ? ZERO_OK : ZERO_EALIGN;
}

// A required matrix of rows x cols (it may be NULL where it has no element).
int check_mat(const void* p, int64_t ld, int dtype, int64_t rows, int64_t cols) {
  ZERO_TRY(check_dtype(dtype));
  if (ld < cols) return ZERO_EINVAL;
  if (ld >= kMost) return ZERO_ERANGE;
  if (!p && rows > 0 && cols > 0) return ZERO_EINVAL;
  return check_aligned(p, dtype);
}
int check_opt_mat(const void* p, int64_t ld, int dtype, int64_t rows, int64_t cols) {
  return p ? check_mat(p, ld, dtype, rows, cols) : ZERO_OK;
}
int check_opt_vec(const void* p, int dtype) {
  if (!p) return ZERO_OK;
  ZERO_TRY(check_dtype(dtype));
  return check_aligned(p, dtype);
}

bool same(const void* a, const void* b) { return a && a == b; }

int check_act(int act) {
  return act >= ZERO_ACT_NONE && act <= ZERO_ACT_SILU ? ZERO_OK : ZERO_EINVAL;
}
int check_layout(int l) { return l == ZERO_W_NK || l == ZERO_W_KN ? ZERO_OK : ZERO_EINVAL; }

int drop_k(const zero_dropout_t* r, zk::DropK* out) {
  if (!r || !(r->p >= 0.0f && r->p <= 1.0f) || r->reserved != 0) return ZERO_EINVAL;
  if (((uintptr_t)r->d_offset & 7u) != 0) return ZERO_EALIGN;
  const double least = floor((double)r->p * 4294967296.0);
  out->on = 1;
  out->all = least >= 4294967296.0;
  out->least = out->all ? 0xFFFFFFFFu : (uint32_t)least;
  out->scale = out->all ? 0.0f : 1.0f / (1.0f - r->p);
  for (uint32_t i = 0; i < 10; ++i) {  // the Weyl sequences of the key's words
    out->keys[2 * i] = (uint32_t)r->seed + i * 0x9E3779B9u;
    out->keys[2 * i + 1] = (uint32_t)(r->seed >> 32) + i * 0xBB67AE85u;
  }
  out->offset = r->offset;
  out->d_offset = r->d_offset;
  return ZERO_OK;
}

}  // namespace

extern "C" int zero_linear(const void* x, int64_t ldx, const void* w, int64_t ldw,
                           int32_t w_layout, int64_t m, int64_t n, int64_t k,
                           const zero_linear_epilogue_t* ep, void* y, int64_t ldy,
                           zero_dtype_t ydtype, zero_stream_t stream) {
  NvtxRange nvtx("zero_linear");
  ZERO_TRY(check_layout(w_layout));
  ZERO_TRY(check_sizes(m, n, k));
  const bool nk = w_layout == ZERO_W_NK;
  ZERO_TRY(check_mat(x, ldx, ZERO_BF16, m, k));
  ZERO_TRY(check_mat(w, ldw, ZERO_BF16, nk ? n : k, nk ? k : n));
  ZERO_TRY(check_mat(y, ldy, ydtype, m, n));
  if (same(y, x) || same(y, w)) return ZERO_EINVAL;
  zk::ProductK p;
  p.epi.out = mat(y, ldy, ydtype);
  if (ep) {
    ZERO_TRY(check_act(ep->act));
    if (ep->reserved != 0) return ZERO_EINVAL;
    ZERO_TRY(check_opt_vec(ep->bias, ep->bias_dtype));
    ZERO_TRY(check_opt_mat(ep->pre, ep->ldpre, ZERO_BF16, m, n));
    ZERO_TRY(check_opt_mat(ep->gate, ep->ldgate, ZERO_BF16, m, n));
    ZERO_TRY(check_opt_mat(ep->residual, ep->ldres, ep->res_dtype, m, n));
    if (same(ep->pre, x) || same(ep->pre, w) || same(ep->pre, y) || same(ep->pre, ep->gate) ||
        same(ep->pre, ep->residual) || same(ep->gate, y) || same(ep->bias, y) ||
        same(ep->bias, ep->pre))
      return ZERO_EINVAL;
    if (same(ep->residual, y) && (ep->ldres != ldy || ep->res_dtype != (int32_t)ydtype))
      return ZERO_EINVAL;
    if (ep->dropout) ZERO_TRY(drop_k(ep->dropout, &p.epi.drop));
    p.epi.act = ep->act;
    if (ep->bias) p.epi.bias = mat(ep->bias, 0, ep->bias_dtype);
    if (ep->pre) p.epi.pre = mat(ep->pre, ep->ldpre, ZERO_BF16);
    if (ep->gate) p.epi.gate = mat(ep->gate, ep->ldgate, ZERO_BF16);
    if (ep->residual) p.epi.residual = mat(ep->residual, ep->ldres, ep->res_dtype);
  }
  p.a = mat(x, ldx, ZERO_BF16);
  p.b = mat(w, ldw, ZERO_BF16);
  p.a_c = 1;
  p.b_c = nk;
  p.rows = m;
  p.cols = n;
  p.depth = k;
  return cuda_status(zk::launch_product(p, zk::LIN_FORWARD, (cudaStream_t)stream));
}

extern "C" int zero_linear_dinput(const void* dy, int64_t lddy, const void* w, int64_t ldw,
                                  int32_t w_layout, int64_t m, int64_t n, int64_t k,
                                  const zero_act_grad_t* ag, void* dx, int64_t lddx,
                                  zero_dtype_t dxdtype, zero_stream_t stream) {
  NvtxRange nvtx("zero_linear_dinput");
  ZERO_TRY(check_layout(w_layout));
  ZERO_TRY(check_sizes(m, n, k));
  const bool nk = w_layout == ZERO_W_NK;
  ZERO_TRY(check_mat(dy, lddy, ZERO_BF16, m, n));
  ZERO_TRY(check_mat(w, ldw, ZERO_BF16, nk ? n : k, nk ? k : n));
  ZERO_TRY(check_mat(dx, lddx, dxdtype, m, k));
  if (same(dx, dy) || same(dx, w)) return ZERO_EINVAL;
  zk::ProductK p;
  p.epi.out = mat(dx, lddx, dxdtype);
  if (ag) {
    ZERO_TRY(check_act(ag->act));
    if (ag->reserved != 0) return ZERO_EINVAL;
    ZERO_TRY(check_mat(ag->pre, ag->ldpre, ZERO_BF16, m, k));
    ZERO_TRY(check_opt_mat(ag->gate, ag->ldgate, ZERO_BF16, m, k));
    ZERO_TRY(check_opt_mat(ag->dgate, ag->lddgate, ZERO_BF16, m, k));
    if (ag->dgate && !ag->gate) return ZERO_EINVAL;
    if (same(ag->dgate, dx) || same(ag->dgate, dy) || same(ag->dgate, w) ||
        same(ag->dgate, ag->pre) || same(ag->dgate, ag->gate) || same(ag->pre, dx) ||
        same(ag->gate, dx))
      return ZERO_EINVAL;
    p.epi.act = ag->act;
    p.epi.pre = mat(ag->pre, ag->ldpre, ZERO_BF16);
    if (ag->gate) p.epi.gate = mat(ag->gate, ag->ldgate, ZERO_BF16);
    if (ag->dgate) p.epi.dgate = mat(ag->dgate, ag->lddgate, ZERO_BF16);
  }
  p.a = mat(dy, lddy, ZERO_BF16);
  p.b = mat(w, ldw, ZERO_BF16);
  p.a_c = 1;
  p.b_c = !nk;
  p.rows = m;
  p.cols = k;
  p.depth = n;
  return cuda_status(zk::launch_product(p, zk::LIN_DINPUT, (cudaStream_t)stream));
}

extern "C" int zero_linear_dweight(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                   int64_t m, int64_t n, int64_t k, int32_t w_layout, void* dw,
                                   int64_t lddw, zero_dtype_t dwdtype, void* dbias,
                                   zero_dtype_t dbdtype, int32_t accumulate,
                                   zero_stream_t stream) {
  NvtxRange nvtx("zero_linear_dweight");
  ZERO_TRY(check_layout(w_layout));
  ZERO_TRY(check_sizes(m, n, k));
  const bool nk = w_layout == ZERO_W_NK;
  ZERO_TRY(check_mat(dy, lddy, ZERO_BF16, m, n));
  ZERO_TRY(check_mat(x, ldx, ZERO_BF16, m, k));
  ZERO_TRY(check_mat(dw, lddw, dwdtype, nk ? n : k, nk ? k : n));
  ZERO_TRY(check_opt_vec(dbias, dbdtype));
  if (same(dw, dy) || same(dw, x) || same(dbias, dw) || same(dbias, dy) || same(dbias, x))
    return ZERO_EINVAL;
  zk::ProductK p;
  p.epi.out = mat(dw, lddw, dwdtype);
  p.epi.accumulate = accumulate != 0;
  if (dbias) p.dbias = mat(dbias, 0, dbdtype);
  // rows of dw are the product's rows in either layout
  const zk::Mat d = mat(dy, lddy, ZERO_BF16), in = mat(x, ldx, ZERO_BF16);
  p.a = nk ? d : in;
  p.b = nk ? in : d;
  p.a_c = 0;
  p.b_c = 0;
  p.rows = nk ? n : k;
  p.cols = nk ? k : n;
  p.bias_b = !nk;
  p.depth = m;
  return cuda_status(zk::launch_product(p, zk::LIN_DWEIGHT, (cudaStream_t)stream));
}

extern "C" int zero_dropout(const void* x, int64_t ldx, zero_dtype_t xdtype,
                            const void* residual, int64_t ldres, zero_dtype_t res_dtype,
                            int64_t m, int64_t n, const zero_dropout_t* rng, void* y,
                            int64_t ldy, zero_dtype_t ydtype, zero_stream_t stream) {
  NvtxRange nvtx("zero_dropout");
  ZERO_TRY(check_sizes(m, n));
  ZERO_TRY(check_mat(x, ldx, xdtype, m, n));
  ZERO_TRY(check_opt_mat(residual, ldres, res_dtype, m, n));
  ZERO_TRY(check_mat(y, ldy, ydtype, m, n));
  if (same(y, x) && (ldy != ldx || ydtype != xdtype)) return ZERO_EINVAL;
  if (same(y, residual) && (ldy != ldres || ydtype != res_dtype)) return ZERO_EINVAL;
  zk::DropK d;
  ZERO_TRY(drop_k(rng, &d));
  return cuda_status(zk::launch_dropout(mat(x, ldx, xdtype), mat(residual, ldres, res_dtype),
                                        mat(y, ldy, ydtype), m, n, d, (cudaStream_t)stream));
}

namespace {

int check_norm(int kind, const void* mean, const void* rstd) {
  if (kind != ZERO_NORM_LAYER && kind != ZERO_NORM_RMS) return ZERO_EINVAL;
  if (mean && kind == ZERO_NORM_RMS) return ZERO_EINVAL;
  ZERO_TRY(check_aligned(mean, ZERO_F32));
  return check_aligned(rstd, ZERO_F32);
}

}  // namespace

extern "C" int zero_layer_norm(const void* x, int64_t ldx, zero_dtype_t xdtype,
                               const void* weight, const void* bias, zero_dtype_t pdtype,
                               int64_t m, int64_t n, int32_t kind, float eps, void* y,
                               int64_t ldy, zero_dtype_t ydtype, float* mean, float* rstd,
                               zero_stream_t stream) {
  NvtxRange nvtx("zero_layer_norm");
  ZERO_TRY(check_sizes(m, n));
  ZERO_TRY(check_norm(kind, mean, rstd));
  if (!isfinite(eps) || eps < 0.0f) return ZERO_EINVAL;
  ZERO_TRY(check_mat(x, ldx, xdtype, m, n));
  ZERO_TRY(check_mat(y, ldy, ydtype, m, n));
  ZERO_TRY(check_mat(weight, n, pdtype, 1, n));
  ZERO_TRY(check_opt_vec(bias, pdtype));
  if (same(y, x) && (ldy != ldx || ydtype != xdtype)) return ZERO_EINVAL;
  if (same(y, weight) || same(y, bias) || same(mean, rstd) || same(mean, y) || same(rstd, y) ||
      same(mean, x) || same(rstd, x))
    return ZERO_EINVAL;
  zk::NormK k;
  k.x = mat(x, ldx, xdtype);
  k.y = mat(y, ldy, ydtype);
  k.w = mat(weight, 0, pdtype);
  k.b = mat(bias, 0, pdtype);
  k.m = m;
  k.n = n;
  k.rms = kind == ZERO_NORM_RMS;
  k.eps = eps;
  k.mean = mean;
  k.rstd = rstd;
  return cuda_status(zk::launch_layer_norm(k, (cudaStream_t)stream));
}

extern "C" int zero_layer_norm_workspace(int64_t m, int64_t n, int64_t* bytes) {
  if (!bytes) return ZERO_EINVAL;
  ZERO_TRY(check_sizes(m, n));
  *bytes = zk::norm_partials(m) * 2 * n * (int64_t)sizeof(float);
  return ZERO_OK;
}

extern "C" int zero_layer_norm_backward(
    const void* dy, int64_t lddy, zero_dtype_t dydtype, const void* x, int64_t ldx,
    zero_dtype_t xdtype, const void* weight, zero_dtype_t pdtype, const float* mean,
    const float* rstd, int64_t m, int64_t n, int32_t kind, const void* dres, int64_t lddres,
    void* dx, int64_t lddx, zero_dtype_t dxdtype, void* dweight, void* dbias,
    zero_dtype_t gdtype, int32_t accumulate, void* workspace, int64_t workspace_bytes,
    zero_stream_t stream) {
  NvtxRange nvtx("zero_layer_norm_backward");
  ZERO_TRY(check_sizes(m, n));
  ZERO_TRY(check_norm(kind, mean, rstd));
  if (m > 0 && n > 0 && (!rstd || (kind == ZERO_NORM_LAYER && !mean))) return ZERO_EINVAL;
  ZERO_TRY(check_mat(dy, lddy, dydtype, m, n));
  ZERO_TRY(check_mat(x, ldx, xdtype, m, n));
  ZERO_TRY(check_mat(dx, lddx, dxdtype, m, n));
  ZERO_TRY(check_mat(weight, n, pdtype, 1, n));
  ZERO_TRY(check_mat(dweight, n, gdtype, 1, n));
  ZERO_TRY(check_opt_vec(dbias, gdtype));
  ZERO_TRY(check_opt_mat(dres, lddres, dxdtype, m, n));
  if (same(dx, dy) || same(dx, x) || same(dx, weight) || same(dweight, dbias) ||
      same(dweight, weight) || same(dbias, weight) || same(dweight, dx) || same(dbias, dx))
    return ZERO_EINVAL;
  if (same(dx, dres) && lddx != lddres) return ZERO_EINVAL;
  int64_t need = 0;
  ZERO_TRY(zero_layer_norm_workspace(m, n, &need));
  if (workspace_bytes < need || (need > 0 && !workspace)) return ZERO_EINVAL;
  if (((uintptr_t)workspace & 15u) != 0) return ZERO_EALIGN;
  zk::NormGradK k;
  k.dy = mat(dy, lddy, dydtype);
  k.x = mat(x, ldx, xdtype);
  k.w = mat(weight, 0, pdtype);
  k.dres = mat(dres, lddres, dxdtype);
  k.dx = mat(dx, lddx, dxdtype);
  k.dw = mat(dweight, 0, gdtype);
  k.db = mat(dbias, 0, gdtype);
  k.m = m;
  k.n = n;
  k.rms = kind == ZERO_NORM_RMS;
  k.accumulate = accumulate != 0;
  k.mean = mean;
  k.rstd = rstd;
  k.partials = static_cast<float*>(workspace);
  return cuda_status(zk::launch_layer_norm_grad(k, (cudaStream_t)stream));
}
