// C entry points of the layer-computation operators: argument checks and
// kernel parameters.  Every rejected call returns before any launch.
#include <math.h>

#include <initializer_list>

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

// The checked epilogue of a forward product of x and w into y.
int epilogue_k(const zero_linear_epilogue_t* ep, const void* x, const void* w, int64_t m,
               int64_t n, const void* y, int64_t ldy, int32_t ydtype, zk::EpiK* out) {
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
  if (ep->dropout) ZERO_TRY(drop_k(ep->dropout, &out->drop));
  out->act = ep->act;
  if (ep->bias) out->bias = mat(ep->bias, 0, ep->bias_dtype);
  if (ep->pre) out->pre = mat(ep->pre, ep->ldpre, ZERO_BF16);
  if (ep->gate) out->gate = mat(ep->gate, ep->ldgate, ZERO_BF16);
  if (ep->residual) out->residual = mat(ep->residual, ep->ldres, ep->res_dtype);
  return ZERO_OK;
}
// The checked activation gradient behind an input gradient of dy and w into dx.
int act_grad_k(const zero_act_grad_t* ag, const void* dy, const void* w, int64_t m, int64_t k,
               const void* dx, zk::EpiK* out) {
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
  out->act = ag->act;
  out->pre = mat(ag->pre, ag->ldpre, ZERO_BF16);
  if (ag->gate) out->gate = mat(ag->gate, ag->ldgate, ZERO_BF16);
  if (ag->dgate) out->dgate = mat(ag->dgate, ag->lddgate, ZERO_BF16);
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
  if (ep) ZERO_TRY(epilogue_k(ep, x, w, m, n, y, ldy, ydtype, &p.epi));
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
  if (ag) ZERO_TRY(act_grad_k(ag, dy, w, m, k, dx, &p.epi));
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

namespace {

int check_format(int32_t format) {
  return format == ZERO_FP4_MX || format == ZERO_FP4_NV ? ZERO_OK : ZERO_EINVAL;
}

// A 4-bit matrix of rows x cols.
int fp4_k(const zero_fp4_t* q, int32_t format, int64_t rows, int64_t cols, zk::Fp4Mat* out) {
  if (!q) return ZERO_EINVAL;
  ZERO_TRY(zero_fp4_size(rows, cols, format, &out->line_bytes, &out->scale_bytes));
  if (q->ld < out->line_bytes) return ZERO_EINVAL;
  if (q->ld >= kMost) return ZERO_ERANGE;
  if (rows > 0 && cols > 0 && (!q->codes || !q->scales)) return ZERO_EINVAL;
  if (format == ZERO_FP4_MX && q->tensor_scale) return ZERO_EINVAL;
  if ((((uintptr_t)q->codes | (uintptr_t)q->scales | (uintptr_t)q->ld) & 15u) != 0 ||
      ((uintptr_t)q->tensor_scale & 3u) != 0)
    return ZERO_EALIGN;
  if (same(q->codes, q->scales) || same(q->codes, q->tensor_scale) ||
      same(q->scales, q->tensor_scale))
    return ZERO_EINVAL;
  out->codes = static_cast<unsigned char*>(q->codes);
  out->ld = q->ld;
  out->scales = static_cast<unsigned char*>(q->scales);
  const int64_t size = format == ZERO_FP4_NV ? 16 : 32, blocks = (cols + size - 1) / size;
  out->scale_tiles = (blocks + 3) / 4;
  return ZERO_OK;
}

// Whether p is one of q's buffers.
bool within(const void* p, const zero_fp4_t* q) {
  return q && (same(p, q->codes) || same(p, q->scales) || same(p, q->tensor_scale));
}

// a [rows, depth] times b [cols, depth] transposed.
int fp4_product(const zero_fp4_t* a, const zero_fp4_t* b, int32_t format, int64_t rows,
                int64_t cols, int64_t depth, zk::ProductK* p) {
  zk::Fp4Mat qa, qb;
  ZERO_TRY(fp4_k(a, format, rows, depth, &qa));
  ZERO_TRY(fp4_k(b, format, cols, depth, &qb));
  p->a = mat(qa.codes, qa.ld / 2, ZERO_BF16);
  p->b = mat(qb.codes, qb.ld / 2, ZERO_BF16);
  p->rows = rows;
  p->cols = cols;
  p->depth = qa.line_bytes / 2;
  p->scales_a = qa.scales;
  p->scales_b = qb.scales;
  p->whole_a = a->tensor_scale;
  p->whole_b = b->tensor_scale;
  p->blocks_of = format == ZERO_FP4_NV ? 16 : 32;
  p->scale_tiles = qa.scale_tiles;
  return ZERO_OK;
}

}  // namespace

extern "C" int zero_fp4_size(int64_t rows, int64_t cols, int32_t format, int64_t* row_bytes,
                             int64_t* scale_bytes) {
  if (!row_bytes || !scale_bytes) return ZERO_EINVAL;
  ZERO_TRY(check_format(format));
  ZERO_TRY(check_sizes(rows, cols));
  const int64_t size = format == ZERO_FP4_NV ? 16 : 32, blocks = (cols + size - 1) / size;
  *row_bytes = (cols + 31) / 32 * 16;
  *scale_bytes = (rows + 127) / 128 * ((blocks + 3) / 4) * 512;
  return ZERO_OK;
}

extern "C" int zero_fp4_tensor_scale(const void* x, int64_t ldx, zero_dtype_t xdtype,
                                     int64_t rows, int64_t cols, float* tensor_scale,
                                     void* workspace, int64_t workspace_bytes,
                                     zero_stream_t stream) {
  NvtxRange nvtx("zero_fp4_tensor_scale");
  ZERO_TRY(check_sizes(rows, cols));
  ZERO_TRY(check_mat(x, ldx, xdtype, rows, cols));
  if (!tensor_scale || !workspace || workspace_bytes < ZERO_FP4_WORKSPACE) return ZERO_EINVAL;
  if (((uintptr_t)tensor_scale & 3u) != 0 || ((uintptr_t)workspace & 15u) != 0)
    return ZERO_EALIGN;
  if (same(tensor_scale, x) || same(workspace, x) || same(workspace, tensor_scale))
    return ZERO_EINVAL;
  zk::MaxK k;
  k.x = mat(x, ldx, xdtype);
  k.rows = rows;
  k.cols = cols;
  k.maxima = static_cast<float*>(workspace);
  return cuda_status(zk::launch_tensor_scale(k, tensor_scale, (cudaStream_t)stream));
}

extern "C" int zero_fp4_quantize(const void* x, int64_t ldx, zero_dtype_t xdtype, int64_t rows,
                                 int64_t cols, int32_t format, const zero_fp4_t* q,
                                 const zero_fp4_t* qt, zero_stream_t stream) {
  NvtxRange nvtx("zero_fp4_quantize");
  ZERO_TRY(check_format(format));
  ZERO_TRY(check_sizes(rows, cols));
  ZERO_TRY(check_mat(x, ldx, xdtype, rows, cols));
  if (!q && !qt) return ZERO_EINVAL;
  zk::QuantK k;
  if (q) ZERO_TRY(fp4_k(q, format, rows, cols, &k.q));
  if (qt) ZERO_TRY(fp4_k(qt, format, cols, rows, &k.qt));
  if (q && qt &&
      (q->tensor_scale != qt->tensor_scale || within(q->codes, qt) || within(q->scales, qt)))
    return ZERO_EINVAL;
  if (within(x, q) || within(x, qt)) return ZERO_EINVAL;
  k.x = mat(x, ldx, xdtype);
  k.rows = rows;
  k.cols = cols;
  k.g = (q ? q : qt)->tensor_scale;
  k.nv = format == ZERO_FP4_NV;
  return cuda_status(zk::launch_quantize(k, (cudaStream_t)stream));
}

extern "C" int zero_fp4_dequantize(const zero_fp4_t* q, int64_t rows, int64_t cols,
                                   int32_t format, void* y, int64_t ldy, zero_dtype_t ydtype,
                                   zero_stream_t stream) {
  NvtxRange nvtx("zero_fp4_dequantize");
  ZERO_TRY(check_format(format));
  ZERO_TRY(check_sizes(rows, cols));
  zk::DequantK k;
  ZERO_TRY(fp4_k(q, format, rows, cols, &k.q));
  ZERO_TRY(check_mat(y, ldy, ydtype, rows, cols));
  if (within(y, q)) return ZERO_EINVAL;
  k.g = q->tensor_scale;
  k.nv = format == ZERO_FP4_NV;
  k.rows = rows;
  k.cols = cols;
  k.y = mat(y, ldy, ydtype);
  return cuda_status(zk::launch_dequantize(k, (cudaStream_t)stream));
}

extern "C" int zero_fp4_linear(const zero_fp4_t* x, const zero_fp4_t* w, int32_t format,
                               int64_t m, int64_t n, int64_t k,
                               const zero_linear_epilogue_t* ep, void* y, int64_t ldy,
                               zero_dtype_t ydtype, zero_stream_t stream) {
  NvtxRange nvtx("zero_fp4_linear");
  ZERO_TRY(check_format(format));
  ZERO_TRY(check_sizes(m, n, k));
  zk::ProductK p;
  ZERO_TRY(fp4_product(x, w, format, m, n, k, &p));
  ZERO_TRY(check_mat(y, ldy, ydtype, m, n));
  if (within(y, x) || within(y, w)) return ZERO_EINVAL;
  p.epi.out = mat(y, ldy, ydtype);
  if (ep) {
    if (within(ep->pre, x) || within(ep->pre, w)) return ZERO_EINVAL;
    ZERO_TRY(epilogue_k(ep, nullptr, nullptr, m, n, y, ldy, ydtype, &p.epi));
  }
  return cuda_status(zk::launch_fp4_product(p, zk::LIN_FORWARD, (cudaStream_t)stream));
}

extern "C" int zero_fp4_linear_dinput(const zero_fp4_t* dy, const zero_fp4_t* w, int32_t format,
                                      int64_t m, int64_t n, int64_t k, const zero_act_grad_t* ag,
                                      void* dx, int64_t lddx, zero_dtype_t dxdtype,
                                      zero_stream_t stream) {
  NvtxRange nvtx("zero_fp4_linear_dinput");
  ZERO_TRY(check_format(format));
  ZERO_TRY(check_sizes(m, n, k));
  zk::ProductK p;
  ZERO_TRY(fp4_product(dy, w, format, m, k, n, &p));
  ZERO_TRY(check_mat(dx, lddx, dxdtype, m, k));
  if (within(dx, dy) || within(dx, w)) return ZERO_EINVAL;
  p.epi.out = mat(dx, lddx, dxdtype);
  if (ag) {
    if (within(ag->dgate, dy) || within(ag->dgate, w)) return ZERO_EINVAL;
    ZERO_TRY(act_grad_k(ag, nullptr, nullptr, m, k, dx, &p.epi));
  }
  return cuda_status(zk::launch_fp4_product(p, zk::LIN_DINPUT, (cudaStream_t)stream));
}

extern "C" int zero_fp4_linear_dweight(const zero_fp4_t* dy, const zero_fp4_t* x, int32_t format,
                                       int64_t m, int64_t n, int64_t k, void* dw, int64_t lddw,
                                       zero_dtype_t dwdtype, int32_t accumulate,
                                       zero_stream_t stream) {
  NvtxRange nvtx("zero_fp4_linear_dweight");
  ZERO_TRY(check_format(format));
  ZERO_TRY(check_sizes(m, n, k));
  zk::ProductK p;
  ZERO_TRY(fp4_product(dy, x, format, n, k, m, &p));
  ZERO_TRY(check_mat(dw, lddw, dwdtype, n, k));
  if (within(dw, dy) || within(dw, x)) return ZERO_EINVAL;
  p.epi.out = mat(dw, lddw, dwdtype);
  if (accumulate) p.epi.residual = p.epi.out;
  return cuda_status(zk::launch_fp4_product(p, zk::LIN_FORWARD, (cudaStream_t)stream));
}

namespace {

int check_ns(const zero_newton_schulz_t* ns) {
  if (!ns || ns->steps < 0 || ns->steps > ZERO_NS_MOST) return ZERO_EINVAL;
  if (!isfinite(ns->eps) || ns->eps < 0.0f) return ZERO_EINVAL;
  for (int i = 0; i < ns->steps; ++i)
    for (float c : ns->coef[i])
      if (!isfinite(c)) return ZERO_EINVAL;
  return ZERO_OK;
}
void put_ns(const zero_newton_schulz_t* ns, zk::OrthoCall* c) {
  c->steps = ns->steps;
  c->source.eps = ns->eps;
  for (int i = 0; i < ns->steps; ++i)
    for (int q = 0; q < 3; ++q) c->coef[i][q] = ns->coef[i][q];
}

int check_batch(int64_t m, int64_t n, int64_t batch) {
  ZERO_TRY(check_sizes(m, n, batch));
  return zk::ortho_fits(m, n, batch) ? ZERO_OK : ZERO_ERANGE;
}

int check_scratch(const void* workspace, int64_t bytes, int64_t m, int64_t n, int64_t batch) {
  const int64_t need = m > 0 && n > 0 && batch > 0 ? zk::ortho_space(m, n, batch).bytes : 0;
  if (bytes < need || (need > 0 && !workspace)) return ZERO_EINVAL;
  return ((uintptr_t)workspace & 15u) == 0 ? ZERO_OK : ZERO_EALIGN;
}

// Matrices of a batch: none begins inside the one before.
int check_stride(int64_t stride, int64_t ld, int64_t m, int64_t n, int64_t batch) {
  if (batch <= 1 || m == 0 || n == 0) return ZERO_OK;
  if (stride < (m - 1) * ld + n) return ZERO_EINVAL;
  return stride < ((int64_t)1 << 62) / batch ? ZERO_OK : ZERO_ERANGE;
}

int check_flat(const void* p) {
  if (!p) return ZERO_EINVAL;
  return ((uintptr_t)p & 15u) == 0 ? ZERO_OK : ZERO_EALIGN;
}

}  // namespace

extern "C" int zero_orthogonalize_workspace(int64_t m, int64_t n, int64_t batch,
                                            int64_t* bytes) {
  if (!bytes) return ZERO_EINVAL;
  ZERO_TRY(check_batch(m, n, batch));
  *bytes = m > 0 && n > 0 && batch > 0 ? zk::ortho_space(m, n, batch).bytes : 0;
  return ZERO_OK;
}

extern "C" int zero_orthogonalize(const void* x, int64_t ldx, int64_t stride_x,
                                  zero_dtype_t xdtype, int64_t m, int64_t n, int64_t batch,
                                  const zero_newton_schulz_t* ns, void* y, int64_t ldy,
                                  int64_t stride_y, void* workspace, int64_t workspace_bytes,
                                  zero_stream_t stream) {
  NvtxRange nvtx("zero_orthogonalize");
  ZERO_TRY(check_batch(m, n, batch));
  ZERO_TRY(check_ns(ns));
  ZERO_TRY(check_mat(x, ldx, xdtype, batch ? m : 0, n));
  ZERO_TRY(check_mat(y, ldy, ZERO_BF16, batch ? m : 0, n));
  ZERO_TRY(check_stride(stride_x, ldx, m, n, batch));
  ZERO_TRY(check_stride(stride_y, ldy, m, n, batch));
  if (same(y, x) && (xdtype != ZERO_BF16 || ldy != ldx || (batch > 1 && stride_y != stride_x)))
    return ZERO_EINVAL;
  ZERO_TRY(check_scratch(workspace, workspace_bytes, m, n, batch));
  if (same(workspace, x) || same(workspace, y)) return ZERO_EINVAL;
  zk::OrthoCall c;
  put_ns(ns, &c);
  c.source.x = mat(x, ldx, xdtype);
  c.source.places.stride = stride_x;
  c.source.m = m;
  c.source.n = n;
  c.finish.y = mat(y, ldy, ZERO_BF16);
  c.finish.places.stride = stride_y;
  c.batch = batch;
  c.workspace = workspace;
  return cuda_status(zk::launch_orthogonalize(c, (cudaStream_t)stream));
}

extern "C" int zero_muon_workspace(int64_t rows, int64_t cols, int32_t count, int64_t* bytes) {
  if (count < 0) return ZERO_EINVAL;
  if (count > ZERO_MUON_MOST) return ZERO_ERANGE;
  return zero_orthogonalize_workspace(rows, cols, count, bytes);
}

extern "C" int zero_muon_step(const zero_plan_t* plan, const int64_t* tensors, int32_t count,
                              int64_t rows, int64_t cols, float* master, float* momentum,
                              const float* reduced, const zero_muon_t* hp, const float* d_coef,
                              void* out, zero_dtype_t out_dtype, void* workspace,
                              int64_t workspace_bytes, zero_stream_t stream) {
  NvtxRange nvtx("zero_muon_step");
  if (!plan || count < 0 || (count > 0 && !tensors)) return ZERO_EINVAL;
  if (count > ZERO_MUON_MOST) return ZERO_ERANGE;
  ZERO_TRY(check_batch(rows, cols, count));
  if (!hp || hp->reserved != 0) return ZERO_EINVAL;
  for (float v : {hp->lr, hp->momentum, hp->weight_decay, hp->grad_scale, hp->scale})
    if (!isfinite(v)) return ZERO_EINVAL;
  if (!(hp->momentum >= 0.0f && hp->momentum < 1.0f)) return ZERO_EINVAL;
  ZERO_TRY(check_ns(&hp->ns));
  ZERO_TRY(check_flat(master));
  ZERO_TRY(check_flat(momentum));
  ZERO_TRY(check_flat(reduced));
  if (out) {
    ZERO_TRY(check_dtype(out_dtype));
    ZERO_TRY(check_flat(out));
  }
  if (((uintptr_t)d_coef & 3u) != 0) return ZERO_EALIGN;
  if (same(master, momentum) || same(master, reduced) || same(momentum, reduced) ||
      same(out, master) || same(out, momentum) || same(out, reduced))
    return ZERO_EINVAL;
  zk::OrthoCall c;
  for (int32_t i = 0; i < count; ++i) {
    ZERO_TRY(zero_plan_tensor(plan, tensors[i], &c.source.places.offset[i], nullptr, nullptr));
    if (plan->numels[tensors[i]] != rows * cols) return ZERO_EINVAL;
    for (int32_t j = 0; j < i; ++j)
      if (tensors[j] == tensors[i]) return ZERO_EINVAL;
  }
  ZERO_TRY(check_scratch(workspace, workspace_bytes, rows, cols, count));
  if (same(workspace, master) || same(workspace, momentum) || same(workspace, reduced) ||
      same(workspace, out))
    return ZERO_EINVAL;
  put_ns(&hp->ns, &c);
  c.source.places.listed = 1;
  c.source.x = mat(reduced, cols, ZERO_F32);
  c.source.momentum = mat(momentum, cols, ZERO_F32);
  c.source.m = rows;
  c.source.n = cols;
  c.source.muon = 1;
  c.source.nesterov = hp->nesterov != 0;
  c.source.mu = hp->momentum;
  c.source.grad_scale = hp->grad_scale;
  c.source.coef = d_coef;
  c.finish.places = c.source.places;
  c.finish.y = mat(master, cols, ZERO_F32);
  if (out) c.finish.out = mat(out, cols, out_dtype);
  c.finish.update = 1;
  c.finish.rate = hp->lr * hp->scale;
  c.finish.decay = hp->lr * hp->weight_decay;
  c.batch = count;
  c.workspace = workspace;
  return cuda_status(zk::launch_orthogonalize(c, (cudaStream_t)stream));
}
