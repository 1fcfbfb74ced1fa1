// Products of bf16 matrices with what follows them fused in: the forward
// product, its input's and its weight's gradients (see zero_linear*,
// include/zero.h).
#include "zero_ops_device.cuh"

namespace zk {

// ---------------------------------------------------------------------------
// Plain tiles: 64 x 64 outputs per block, 4 x 4 fp32 sums per thread, operands
// staged 16 deep through shared memory.
// ---------------------------------------------------------------------------
constexpr int kTile = 64, kDepth = 16;

__device__ __forceinline__ float operand(const Mat& a, bool contig, int64_t i, int64_t c,
                                         int64_t rows, int64_t depth) {
  if (i >= rows || c >= depth) return 0.0f;
  const int64_t at = contig ? i * a.ld + c : c * a.ld + i;
  const int64_t last = contig ? (rows - 1) * a.ld + depth : (depth - 1) * a.ld + rows;
  if (!in_extent(at, at + 1, 0, last, ZERO_SITE_LINEAR_IN)) return 0.0f;
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.p)[at] << 16);
}

template <int MODE>
__global__ void __launch_bounds__(256) product_plain_kernel(ProductK k) {
  __shared__ float a[kDepth][kTile + 4], b[kDepth][kTile + 4];
  __shared__ float d[kTile][kTile + 4];
  const int t = threadIdx.x, ti = (t / 16) * 4, tj = (t % 16) * 4;
  const int64_t i0 = (int64_t)blockIdx.y * kTile, j0 = (int64_t)blockIdx.x * kTile;
  float s[4][4] = {};
  for (int64_t c0 = 0; c0 < k.depth; c0 += kDepth) {
    for (int q = t; q < kTile * kDepth; q += 256) {
      const int ai = k.a_c ? q / kDepth : q % kTile, ac = k.a_c ? q % kDepth : q / kTile;
      a[ac][ai] = operand(k.a, k.a_c, i0 + ai, c0 + ac, k.rows, k.depth);
      const int bi = k.b_c ? q / kDepth : q % kTile, bc = k.b_c ? q % kDepth : q / kTile;
      b[bc][bi] = operand(k.b, k.b_c, j0 + bi, c0 + bc, k.cols, k.depth);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kDepth; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] += a[c][ti + i] * b[c][tj + j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k.out_t)
        d[tj + j][ti + i] = s[i][j];
      else
        d[ti + i][tj + j] = s[i][j];
    }
  __syncthreads();
  const int64_t r0 = k.out_t ? j0 : i0, c0 = k.out_t ? i0 : j0;
  const Extent e{k.out_t ? k.cols : k.rows, k.out_t ? k.rows : k.cols};
  const uint64_t offset = MODE == LIN_FORWARD && k.epi.drop.on ? drop_offset(k.epi.drop) : 0;
  for (int q = t; q < kTile * kTile / 8; q += 256) {
    const int r = q / 8, c = (q % 8) * 8;
    if (r0 + r >= e.rows || c0 + c >= e.cols) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = d[r][c + j];
    epilogue8<MODE>(k.epi, offset, r0 + r, c0 + c,
                    e.cols - c0 - c < 8 ? (int)(e.cols - c0 - c) : 8, v, e);
  }
}

// Sums over the contraction of A (k.a_c == 0): 32 of its rows per block.
__global__ void __launch_bounds__(256) column_sum_kernel(ProductK k) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  for (int64_t c = warp; c < k.depth; c += 8) s += operand(k.a, false, i, c, k.rows, k.depth);
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < k.rows && in_extent(i, i + 1, 0, k.rows, ZERO_SITE_LINEAR_OUT)) {
    s = 0.0f;
    for (int w = 0; w < 8; ++w) s += sum[w][lane];
    if (k.epi.accumulate) s += load1(k.dbias, i);
    store1(k.dbias, i, s);
  }
}

template <int MODE>
static cudaError_t launch_plain(const ProductK& k, cudaStream_t st) {
  // rows run along grid.y (65535 blocks at most): longer products in slices
  constexpr int64_t most = 65535 * (int64_t)kTile;
  if (k.rows > most) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((k.cols + kTile - 1) / kTile),
                  (unsigned)((k.rows + kTile - 1) / kTile));
  product_plain_kernel<MODE><<<grid, 256, 0, st>>>(k);
  return cudaGetLastError();
}

cudaError_t launch_product(const ProductK& k, int mode, cudaStream_t st) {
  if (k.rows <= 0) return cudaSuccess;
  if (k.dbias.p) {
    column_sum_kernel<<<(unsigned)((k.rows + 31) / 32), 256, 0, st>>>(k);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (k.cols <= 0) return cudaSuccess;
  if (mode == LIN_FORWARD) return launch_plain<LIN_FORWARD>(k, st);
  if (mode == LIN_DINPUT) return launch_plain<LIN_DINPUT>(k, st);
  return launch_plain<LIN_DWEIGHT>(k, st);
}

cudaError_t ops_timeouts(unsigned long long* out, bool) {
  *out = 0;  // no bounded wait in these kernels
  return cudaSuccess;
}

cudaError_t bounds_linear(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
