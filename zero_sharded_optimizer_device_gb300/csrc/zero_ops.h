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

// Bounded waits that gave up / out-of-extent records of these units.
cudaError_t ops_timeouts(unsigned long long* out, bool reset);
cudaError_t bounds_linear(BoundsRec* out, bool reset);
cudaError_t bounds_dropout(BoundsRec* out, bool reset);
cudaError_t bounds_lnorm(BoundsRec* out, bool reset);
cudaError_t bounds_rows(BoundsRec* out, bool reset);

}  // namespace zk
