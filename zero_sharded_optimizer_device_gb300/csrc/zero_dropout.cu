// Dropout with a residual: y = residual + keep(x) / (1 - p).
//
// One pass over memory, the mask recomputed from its counter instead of
// stored (a stored mask would add a byte per element each way).  A thread
// takes 8 consecutive columns, 16 bytes of bf16, and two Philox blocks: 40
// widening multiplications at 4 cycles per warp, about half of what the memory
// traffic costs, so the loads are issued first and the masks drawn while they
// are in flight.  16384 x 1024 bf16 with a residual: 20.7 us, 4.9 TB/s.
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

constexpr int kBlocksPerSm = 8;

// 8 elements from index i on, of a matrix without gaps.
__device__ __forceinline__ Raw8 flat8(const Mat& m, int64_t i, int64_t size) {
  Raw8 r{};
  if (!in_extent(i, i + 8, 0, size, ZERO_SITE_DROPOUT)) return r;
  if (m.dtype == ZERO_F32) {
    r.a = ld16(static_cast<const float*>(m.p) + i);
    r.b = ld16(static_cast<const float*>(m.p) + i + 4);
  } else {
    r.a = ld16(static_cast<const uint16_t*>(m.p) + i);
  }
  return r;
}

// FLAT: every matrix is gapless, on 16-byte boundaries, with rows a multiple
// of 8: vector q then lies at element 8 q, and row and column are wanted for
// the counter alone.  The kernel is bound by instructions, and addresses,
// bounds and formats took two of three (16384 x 1024 bf16 with a residual: 24
// us for the general form).
template <bool RES, bool FLAT>
__global__ void __launch_bounds__(kThreads)
    dropout_kernel(Mat x, Mat residual, Mat y, int64_t row0, Extent e, uint32_t items, Div31 per,
                   const __grid_constant__ DropK d) {
  after_previous_kernel();
  const uint64_t offset = drop_offset(d);
  const uint32_t lo = (uint32_t)offset, hi = (uint32_t)(offset >> 32);
  const int64_t base = row0 * e.cols, size = e.rows * e.cols;
  const uint32_t step = gridDim.x * kThreads;
  // the next vector's operands are on their way while this one's mask is drawn
  Raw8 a, b;
  auto fetch = [&](uint32_t q) {
    if (FLAT) {
      a = flat8(x, base + (int64_t)q * 8, size);
      if (RES) b = flat8(residual, base + (int64_t)q * 8, size);
    } else {
      const uint32_t r = divide(q, per);
      const int64_t row = row0 + r, col = (int64_t)(q - r * per.d) * 8;
      const int valid = e.cols - col >= 8 ? 8 : (int)(e.cols - col);
      a = raw8(x, row, col, valid, e, ZERO_SITE_DROPOUT);
      if (RES) b = raw8(residual, row, col, valid, e, ZERO_SITE_DROPOUT);
    }
  };
  uint32_t q = blockIdx.x * kThreads + threadIdx.x;
  if (q < items) fetch(q);
  for (; q < items; q += step) {
    const Raw8 a0 = a, b0 = b;
    if (q + step < items) fetch(q + step);
    const uint32_t r = divide(q, per), c8 = q - r * per.d;
    const int64_t row = row0 + r, col = (int64_t)c8 * 8, i = base + (int64_t)q * 8;
    const uint4 w0 = philox(make_uint4(2 * c8, (uint32_t)row, lo, hi), d);
    const uint4 w1 = philox(make_uint4(2 * c8 + 1, (uint32_t)row, lo, hi), d);
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float v[8], f[8];
    from_raw(x, a0, v);
    if (RES) from_raw(residual, b0, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = w[j] >= d.least && !d.all ? v[j] * d.scale : 0.0f;
      if (RES) v[j] += f[j];
    }
    if (!FLAT) {
      store8(y, row, col, e.cols - col >= 8 ? 8 : (int)(e.cols - col), v, e, ZERO_SITE_DROPOUT);
    } else if (in_extent(i, i + 8, 0, size, ZERO_SITE_DROPOUT)) {
      if (y.dtype == ZERO_F32) {
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(y.p) + i);
        to[0] = make_float4(v[0], v[1], v[2], v[3]);
        to[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y.p) + i) = pack8(v);
      }
    }
  }
}

cudaError_t launch_dropout(const Mat& x, const Mat& residual, const Mat& y, int64_t m, int64_t n,
                           const DropK& d, cudaStream_t st) {
  if (m <= 0 || n <= 0) return cudaSuccess;
  const int64_t per = (n + 7) / 8;
  const int64_t wave = (int64_t)sm_count() * kBlocksPerSm;
  // a launch counts its vectors in 31 bits (and steps on by a wave of them in
  // 32): longer inputs take several
  const int64_t most = 0x7FFFFFFFll / per;
  bool flat = n % 8 == 0;
  for (const Mat* a : {&x, &residual, &y}) flat = flat && (!a->p || (a->vec && a->ld == n));
  const auto kernel = residual.p ? (flat ? dropout_kernel<true, true> : dropout_kernel<true, false>)
                                 : (flat ? dropout_kernel<false, true> : dropout_kernel<false, false>);
  for (int64_t r = 0; r < m; r += most) {
    const int64_t items = per * (m - r < most ? m - r : most);
    const int64_t blocks = (items + kThreads - 1) / kThreads;
    const cudaError_t e =
        launch_next(kernel, dim3((unsigned)(blocks < wave ? blocks : wave)), dim3(kThreads), st, x,
                    residual, y, r, Extent{m, n}, (uint32_t)items, div31((uint32_t)per), d);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t bounds_dropout(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
