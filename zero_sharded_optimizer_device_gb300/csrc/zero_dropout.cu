// Dropout with a residual: y = residual + keep(x) / (1 - p).
//
// One pass over memory, the mask recomputed from its counter instead of
// stored (a stored mask would add a byte per element each way).  A thread
// takes 8 consecutive columns, 16 bytes of bf16: two Philox blocks, whose
// ~140 integer instructions stay below what the memory traffic costs.
#include "zero_ops_device.cuh"

namespace zk {

// q / d for q < 2^31 by one multiplication: m = ceil(2^(31 + s) / d) with
// s = ceil(log2 d) [Granlund and Montgomery 1994].
struct Div31 {
  uint32_t m, s, d;
};
static Div31 div31(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return Div31{(uint32_t)(((1ull << (31 + s)) + d - 1) / d), s, d};
}
__device__ __forceinline__ uint32_t divide(uint32_t q, const Div31& v) {
  return (uint32_t)(((uint64_t)q * v.m) >> 31 >> v.s);
}

__global__ void __launch_bounds__(kThreads)
    dropout_kernel(Mat x, Mat residual, Mat y, int64_t row0, Extent e, uint32_t items, Div31 per,
                   DropK d) {
  const uint32_t q = blockIdx.x * kThreads + threadIdx.x;
  if (q >= items) return;
  const uint32_t r = divide(q, per);
  const int64_t row = row0 + r, col = (int64_t)(q - r * per.d) * 8;
  const int valid = e.cols - col < 8 ? (int)(e.cols - col) : 8;
  float v[8], f[8];
  load8(x, row, col, valid, v, e, ZERO_SITE_DROPOUT);
  if (residual.p) load8(residual, row, col, valid, f, e, ZERO_SITE_DROPOUT);
  drop8(d, drop_offset(d), (uint32_t)row, col, v);
  if (residual.p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += f[j];
  }
  store8(y, row, col, valid, v, e, ZERO_SITE_DROPOUT);
}

cudaError_t launch_dropout(const Mat& x, const Mat& residual, const Mat& y, int64_t m, int64_t n,
                           const DropK& d, cudaStream_t st) {
  if (m <= 0 || n <= 0) return cudaSuccess;
  const int64_t per = (n + 7) / 8;
  // a launch counts its vectors in 31 bits: longer inputs take several
  const int64_t most = 0x7FFFFFFFll / per;
  for (int64_t r = 0; r < m; r += most) {
    const int64_t items = per * (m - r < most ? m - r : most);
    dropout_kernel<<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        x, residual, y, r, Extent{m, n}, (uint32_t)items, div31((uint32_t)per), d);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t bounds_dropout(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
