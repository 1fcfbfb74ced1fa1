// Private declarations of the layer-computation operators (linear, dropout,
// layer norm): kernel parameters prepared by zero_ops_api.cpp and launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zk {

// A matrix as the kernels see it; p == nullptr where an operand is absent.
struct Mat {
  void* p = nullptr;
  int64_t ld = 0;  // elements between rows
  int dtype = ZERO_BF16;
  int vec = 0;     // 8 columns starting at a multiple of 8 lie on 16-byte boundaries
};
inline Mat mat(const void* p, int64_t ld, int dtype) {
  Mat m;
  m.p = const_cast<void*>(p);
  m.ld = ld;
  m.dtype = dtype;
  const int es = dtype == ZERO_F32 ? 4 : 2;
  m.vec = ((uintptr_t)p & 15u) == 0 && (ld * es) % 16 == 0;
  return m;
}

// Dropout as the kernels see it (zero_dropout_t).
struct DropK {
  int on = 0;
  uint32_t all = 0;  // p = 1: every element dropped
  uint32_t least = 0;  // keep a word >= least
  float scale = 1.0f;
  uint64_t offset = 0;
  const uint64_t* d_offset = nullptr;
  uint32_t keys[20] = {};  // Philox's key of each of the ten rounds, two words
};

enum LinearMode : int { LIN_FORWARD = 0, LIN_DINPUT = 1, LIN_DWEIGHT = 2 };

// What follows a product's fp32 result v at (row, col) of the output.
struct EpiK {
  Mat out;
  Mat bias;      // forward: [n]
  Mat pre;       // forward: output z; dinput: input z
  Mat gate;
  Mat dgate;     // dinput
  Mat residual;  // forward
  DropK drop;    // forward
  int act = ZERO_ACT_NONE;
  int vec = 1;         // every matrix of the output's shape present has its vec
  int accumulate = 0;  // dweight
};

// D[i][j] = sum over c of A(i, c) B(j, c), i < rows, j < cols, c < depth.
// a_c / b_c: the operand's contraction index is the contiguous one.
// out_t: element (i, j) is stored (and the epilogue addressed) at (j, i).
struct ProductK {
  Mat a, b;
  int a_c = 1, b_c = 1, out_t = 0;
  int bias_b = 0;  // dbias sums B's rows (else A's)
  int64_t rows = 0, cols = 0, depth = 0;
  EpiK epi;
  Mat dbias;  // dweight: sums over c of the rows of A or B
  // 4-bit operands (then a and b hold four codes per 16-bit element of theirs):
  // scale tiles of 128 rows and four blocks, scale_tiles of them along the
  // contraction; what the whole operands are scaled by, or nullptr
  const void *scales_a = nullptr, *scales_b = nullptr;
  const float *whole_a = nullptr, *whole_b = nullptr;
  int blocks_of = 0;  // 16 or 32 codes
  int64_t scale_tiles = 0;
};

cudaError_t launch_product(const ProductK& k, int mode, cudaStream_t st);
// Forward products and input gradients of up to kFewRows rows.
constexpr int kFewRows = 8;
cudaError_t launch_rows(const ProductK& k, int mode, cudaStream_t st);

cudaError_t launch_dropout(const Mat& x, const Mat& residual, const Mat& y, int64_t m, int64_t n,
                           const DropK& d, cudaStream_t st);

struct NormK {
  Mat x, y, w, b;
  int64_t m, n;
  int rms;
  float eps;
  float *mean, *rstd;
};
cudaError_t launch_layer_norm(const NormK& k, cudaStream_t st);

struct NormGradK {
  Mat dy, x, w, dres, dx, dw, db;
  int64_t m, n;
  int rms, accumulate;
  const float *mean, *rstd;
  float* partials;
};
// Row groups whose parameter-gradient sums are kept apart in the workspace.
int64_t norm_partials(int64_t m);
cudaError_t launch_layer_norm_grad(const NormGradK& k, cudaStream_t st);

// A matrix in 4-bit codes and its scales as the kernels see it (zero_fp4_t).
struct Fp4Mat {
  unsigned char* codes = nullptr;
  int64_t ld = 0, line_bytes = 0;  // bytes between rows, and that a row fills
  unsigned char* scales = nullptr;
  int64_t scale_tiles = 0, scale_bytes = 0;  // tiles along a row; all of them
};
struct QuantK {
  Mat x;
  int64_t rows = 0, cols = 0, tiles = 0;
  Fp4Mat q, qt;  // codes nullptr: direction not asked for
  const float* g = nullptr;
  int nv = 0;
};
cudaError_t launch_quantize(const QuantK& k, cudaStream_t st);
struct DequantK {
  Fp4Mat q;
  const float* g = nullptr;
  int nv = 0;
  int64_t rows = 0, cols = 0;
  Mat y;
};
cudaError_t launch_dequantize(const DequantK& k, cudaStream_t st);
constexpr int kMaxima = ZERO_FP4_WORKSPACE / (int)sizeof(float);
struct MaxK {
  Mat x;
  int64_t rows = 0, cols = 0;
  float* maxima = nullptr;  // kMaxima
};
cudaError_t launch_tensor_scale(const MaxK& k, float* g, cudaStream_t st);
cudaError_t launch_fp4_product(const ProductK& k, int mode, cudaStream_t st);
// Of up to kFewRows rows of 4-bit operands.
cudaError_t launch_fp4_rows(const ProductK& k, int mode, cudaStream_t st);

// Matrices of a batch: `stride` elements apart, or (listed) from these elements on.
struct OrthoPlaces {
  int listed = 0;
  int64_t stride = 0;
  int64_t offset[ZERO_MUON_MOST] = {};
};
// What is orthogonalised: x, or the gradients and momenta of tensors.
struct OrthoSource {
  OrthoPlaces places;
  Mat x;         // muon: the reduced gradient
  Mat momentum;  // muon
  int64_t m = 0, n = 0;
  int muon = 0, nesterov = 0;
  float mu = 0.0f, grad_scale = 1.0f, eps = 0.0f;
  const float* coef = nullptr;
  // the workspace's (see ortho_space)
  int64_t rows = 0, ld = 0;
  int blocks = 0;
  double* partials = nullptr;
  uint32_t* done = nullptr;  // finished tiles of each matrix
  uint16_t *hi = nullptr, *lo = nullptr;
};
struct OrthoFinish {
  OrthoPlaces places;
  Mat y;    // the result, or master weights
  Mat out;  // update: the gathered parameters, or absent
  int update = 0;
  float rate = 0.0f, decay = 0.0f;
  int64_t m = 0, n = 0, rows = 0, ld = 0;
  const uint16_t* x = nullptr;
};
struct OrthoCall {
  OrthoSource source;
  OrthoFinish finish;
  int64_t batch = 0;
  int steps = 0;
  float coef[ZERO_NS_MOST][3] = {};
  void* workspace = nullptr;
};
// Byte offsets of a call's workspace.  X is stored in rows of ld columns, `rows`
// of them a matrix (whole tiles, zeros around it); G and P in `side` of `side`.
struct OrthoSpace {
  int64_t rows, ld, side, blocks;
  bool fine;  // see zero_ortho.cu: lo and poly twice
  int64_t hi[2], lo[2], gram, poly, poly_lo, diag_gram, diag_poly, done, partials, bytes;
};
// Whether the kernels' counters hold such a batch.
bool ortho_fits(int64_t m, int64_t n, int64_t batch);
OrthoSpace ortho_space(int64_t m, int64_t n, int64_t batch);
cudaError_t launch_orthogonalize(const OrthoCall& c, cudaStream_t st);

// Bounded waits that gave up / out-of-extent records of these units.
cudaError_t timeouts_linear(unsigned long long* out, bool reset);
cudaError_t timeouts_fp4(unsigned long long* out, bool reset);
cudaError_t timeouts_ortho(unsigned long long* out, bool reset);
cudaError_t bounds_linear(BoundsRec* out, bool reset);
cudaError_t bounds_dropout(BoundsRec* out, bool reset);
cudaError_t bounds_lnorm(BoundsRec* out, bool reset);
cudaError_t bounds_rows(BoundsRec* out, bool reset);
cudaError_t bounds_fp4(BoundsRec* out, bool reset);
cudaError_t bounds_fp4_rows(BoundsRec* out, bool reset);
cudaError_t bounds_ortho(BoundsRec* out, bool reset);

}  // namespace zk
