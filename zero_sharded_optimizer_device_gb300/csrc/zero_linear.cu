// Products of bf16 matrices with what follows them fused in (see zero_linear*,
// include/zero.h): the kernel of zero_product.cuh, or zero_rows.cu's for few rows.
#include "zero_product.cuh"

namespace zk {

// Whether a few rows are quicker without tensor cores, by the times of both in
// us, w being millions of weights and m the rows (1, 2, 4 or 8): the weight is
// read by 4 outputs a warp or 32 a block (zero_rows.cu), or in tiles of 256
// outputs whose steps of 64 follow one another.  (Measured, few rows / tiles, m =
// 1, 4, 8: 4096 x 1024 [n, k] 3.6, 5.4, 8.2 / 7.4; 4096 x 4096 [n, k] 5.4, 9.1,
// 16.7 / 12.5, [k, n] 10.3, 14.3, 23.3 / 12.7; 11008 x 4096 [n, k] 18.3, 25.7,
// 50 / 19.4; off 16-byte boundaries 4096 x 4096 11, 17, 28 / 24 and 383 x 6850
// 5.8, 7.8, 12 / 33.)
static bool few_rows_win(const ProductK& k) {
  if (k.rows > kFewRows) return false;
  const double m = k.rows <= 2 ? (double)k.rows : k.rows <= 4 ? 4 : 8;
  const double w = 1e-6 * (double)k.cols * (double)k.depth;
  const bool off = off_words(k.a, k.rows) || off_words(k.b, k.b_c ? k.cols : k.depth);
  const double along = off ? 0.4 + 0.14 * m : (m > 2 ? 0.1 + 0.1 * m : 0.3);
  const double across = off ? 0.5 + 0.16 * m : 0.3 + 0.1 * m;
  const double rows_us = k.b_c ? 2.3 + w * along : 4 + w * across;
  const int64_t pairs = sm_count() / 2, tiles = (k.cols + 255) / 256;
  const int64_t steps = (k.depth + kDeep - 1) / kDeep;
  const int64_t parts = tiles * 2 <= pairs && steps >= 4 ? 2 : 1;
  const double waves = (double)((tiles * parts + pairs - 1) / pairs);
  const double tiles_us = 6 + waves * (double)steps / (double)parts * (off ? 0.5 : 0.24);
  return rows_us <= tiles_us;
}

cudaError_t launch_product(const ProductK& k, int mode, cudaStream_t st) {
  const int64_t sums = !k.dbias.p ? 0 : k.bias_b ? k.cols : k.rows;
  if ((k.rows <= 0 || k.cols <= 0) && sums <= 0) return cudaSuccess;
  if (mode != LIN_DWEIGHT && few_rows_win(k)) return launch_rows(k, mode, st);
  if (mode == LIN_FORWARD) return launch_mode<LIN_FORWARD, OF_BF16>(k, st);
  if (mode == LIN_DINPUT) return launch_mode<LIN_DINPUT, OF_BF16>(k, st);
  return launch_mode<LIN_DWEIGHT, OF_BF16>(k, st);
}

cudaError_t timeouts_linear(unsigned long long* out, bool reset) {
  return unit_timeouts(out, reset);
}

cudaError_t bounds_linear(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
