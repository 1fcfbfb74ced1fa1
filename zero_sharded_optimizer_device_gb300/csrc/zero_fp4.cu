// Matrices in microscaled 4-bit numbers (zero_fp4_*, include/zero.h): to E2M1
// codes with a scale per block and back, and their products on the tensor
// cores' block-scaled instructions (the kernel of zero_product.cuh).
#include "zero_product.cuh"

namespace zk {

// ------------------------------------------------------------- conversions --
// Eight values to codes, the first in the lowest four bits (nearest, ties to
// the even code, beyond 6 to 6).
__device__ __forceinline__ uint32_t to_codes8(const float v[8]) {
  uint32_t r;
  asm("{ .reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d}; }"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ void from_codes8(uint32_t codes, float v[8]) {
  uint32_t h[4];
  asm("{ .reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(h[i]));
}
// E4M3, nearest, beyond 448 to 448; and back.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t byte) {
  uint32_t h;
  float f;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo; }" : "=f"(f) : "r"(h));
  return f;
}

// A block's scale byte and the factor that brings its values to codes, from
// the largest magnitude's bits (NaN and infinity are the largest as integers).
// A block that holds either has scale NaN and codes 0.
constexpr uint32_t kInfBits = 0x7F800000u;
template <bool NV>
__device__ __forceinline__ uint32_t block_scale(uint32_t top, float six_g, float g,
                                                float& factor) {
  factor = 0.0f;
  if (NV) {
    if (top >= kInfBits) return 0x7Fu;
    const uint32_t byte = to_e4m3(__fdiv_rn(__uint_as_float(top), six_g));
    const float d = __fmul_rn(from_e4m3(byte), g);
    if (d > 0.0f) factor = __fdiv_rn(1.0f, d);
    return byte;
  }
  if (top >= kInfBits) return 0xFFu;
  // 2^(floor(log2 top) - 2) as E8M0, at least 2^-127
  const int exponent = (int)(top >> 23);
  const uint32_t byte = exponent > 2 ? (uint32_t)(exponent - 2) : 0u;
  factor = __uint_as_float((254u - byte) << 23);
  return byte;
}
// What a scale byte stands for, times g.
template <bool NV>
__device__ __forceinline__ float scale_value(uint32_t byte, float g) {
  if (NV) return byte == 0x7Fu ? __uint_as_float(0x7FC00000u) : __fmul_rn(from_e4m3(byte), g);
  if (byte == 0xFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

__device__ __forceinline__ uint32_t top8(const float v[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    top = b > top ? b : top;
  }
  return top;
}
// Codes of eight values of a block whose factor is known.
__device__ __forceinline__ uint32_t codes8(const float v[8], float factor) {
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = __fmul_rn(v[j], factor);
  return to_codes8(s);
}

// ----------------------------------------------------------------- quantise --
// A block of 256 threads takes 128 x 128 values: their codes and scales are
// whole scale tiles in both directions, so that every byte of those (padding
// included) has one writer.  Rows straight from the loads, a lane having 8
// columns; columns through shared memory, a thread having one block of one.
constexpr int kQuantTile = 128, kQuantThreads = 256;

template <bool NV, bool WIDE>
struct QuantShared {
  static constexpr int kElem = WIDE ? 4 : 2, kLine = kQuantTile * kElem + 16;
  unsigned char tile[kQuantTile * kLine];
  unsigned char codes[kQuantTile * 80];  // of the columns: 64 bytes each
  unsigned char scales[2][1024];         // rows', columns'
};

template <bool NV>
__device__ __forceinline__ int scale_at(int line, int block) {  // in a 128-line tile's scales
  return (block >> 2) * kScaleTile + (line & 31) * 16 + (line >> 5) * 4 + (block & 3);
}

// One direction's scale tiles to memory: tile (line_tile, t) for the t of this
// 128-wide piece that exist.
__device__ __forceinline__ void store_scales(const Fp4Mat& o, const unsigned char* from,
                                             int64_t line_tile, int64_t tile0, int tiles) {
  const int unit = threadIdx.x;  // 16 bytes
  const int64_t t = tile0 + unit / 32;
  if (unit >= tiles * 32 || t >= o.scale_tiles) return;
  const int64_t at = (line_tile * o.scale_tiles + t) * kScaleTile + unit % 32 * 16;
  if (!in_extent(at, at + 16, 0, o.scale_bytes, ZERO_SITE_FP4)) return;
  *reinterpret_cast<uint4*>(o.scales + at) = *reinterpret_cast<const uint4*>(from + unit * 16);
}

template <bool NV, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const __grid_constant__ QuantK k) {
  extern __shared__ __align__(16) unsigned char quant_smem[];
  using Shared = QuantShared<NV, WIDE>;
  Shared& sh = *reinterpret_cast<Shared*>(quant_smem);
  constexpr int kSize = NV ? 16 : 32, kTiles = NV ? 2 : 1;
  after_previous_kernel();
  const float g = NV && k.g ? *(volatile const float*)k.g : 1.0f;
  const float six_g = __fmul_rn(6.0f, g);
  const int64_t row0 = (int64_t)(blockIdx.x / k.tiles_j) * kQuantTile;
  const int64_t col0 = (int64_t)(blockIdx.x % k.tiles_j) * kQuantTile;
  const int t = threadIdx.x, line = t >> 4, unit = t & 15;
  const Extent e{k.rows, k.cols};
  const int64_t col = col0 + unit * 8;
  const int valid = col >= k.cols ? 0 : k.cols - col < 8 ? (int)(k.cols - col) : 8;
  const bool rows = k.q.codes != nullptr, columns = k.qt.codes != nullptr;
#pragma unroll 4
  for (int p = 0; p < 8; ++p) {
    const int r = p * 16 + line;
    const int64_t row = row0 + r;
    float v[8] = {};
    if (row < k.rows && valid) {
      const Raw8 raw = raw8(k.x, row, col, valid, e, ZERO_SITE_FP4);
      from_raw(k.x, raw, v);
    }
    if (columns) {
      unsigned char* at = sh.tile + r * Shared::kLine + unit * 8 * Shared::kElem;
      if (WIDE) {
        reinterpret_cast<float4*>(at)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(at)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(at) = pack8(v);
      }
    }
    if (rows) {
      uint32_t top = top8(v);
#pragma unroll
      for (int m = 1; m < kSize / 8; m *= 2) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, top, m);
        top = other > top ? other : top;
      }
      float factor;
      const uint32_t byte = block_scale<NV>(top, six_g, g, factor);
      const uint32_t codes = top >= kInfBits ? 0u : codes8(v, factor);
      const int64_t at = row * k.q.ld + col / 2;
      if (row < k.rows && col / 2 < k.q.line_bytes &&
          in_extent(at, at + 4, row * k.q.ld, row * k.q.ld + k.q.line_bytes, ZERO_SITE_FP4))
        *reinterpret_cast<uint32_t*>(k.q.codes + at) = codes;
      if (unit % (kSize / 8) == 0) sh.scales[0][scale_at<NV>(r, unit * 8 / kSize)] = byte;
    }
  }
  __syncthreads();
  if (rows) store_scales(k.q, sh.scales[0], row0 / kQuantTile, col0 / (4 * kSize), kTiles);
  if (!columns) return;
  constexpr int kBlocks = kQuantTile / kSize;
  for (int u = t; u < kQuantTile * kBlocks; u += kQuantThreads) {
    const int c = u % kQuantTile, b = u / kQuantTile;
    float v[kSize];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kSize; ++i) {
      const unsigned char* at = sh.tile + (b * kSize + i) * Shared::kLine + c * Shared::kElem;
      v[i] = WIDE ? *reinterpret_cast<const float*>(at)
                  : __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(at) << 16);
      const uint32_t bits = __float_as_uint(v[i]) & 0x7FFFFFFFu;
      top = bits > top ? bits : top;
    }
    float factor;
    sh.scales[1][scale_at<NV>(c, b)] = (unsigned char)block_scale<NV>(top, six_g, g, factor);
    uint32_t* out = reinterpret_cast<uint32_t*>(sh.codes + c * 80 + b * (kSize / 2));
#pragma unroll
    for (int i = 0; i < kSize / 8; ++i) out[i] = top >= kInfBits ? 0u : codes8(v + 8 * i, factor);
  }
  __syncthreads();
  for (int u = t; u < kQuantTile * 4; u += kQuantThreads) {
    const int c = u >> 2;
    const int64_t to = col0 + c, byte = row0 / 2 + (u & 3) * 16, at = to * k.qt.ld + byte;
    if (to < k.cols && byte < k.qt.line_bytes &&
        in_extent(at, at + 16, to * k.qt.ld, to * k.qt.ld + k.qt.line_bytes, ZERO_SITE_FP4))
      *reinterpret_cast<uint4*>(k.qt.codes + at) =
          *reinterpret_cast<const uint4*>(sh.codes + c * 80 + (u & 3) * 16);
  }
  store_scales(k.qt, sh.scales[1], col0 / kQuantTile, row0 / (4 * kSize), kTiles);
}

template <bool NV, bool WIDE>
static cudaError_t launch_quantize_as(const QuantK& k, int64_t blocks, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  constexpr int bytes = (int)sizeof(QuantShared<NV, WIDE>);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(quantize_kernel<NV, WIDE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  return launch_next_with(bytes, quantize_kernel<NV, WIDE>, dim3((unsigned)blocks),
                          dim3(kQuantThreads), st, k);
}

cudaError_t launch_quantize(const QuantK& in, cudaStream_t st) {
  QuantK k = in;
  k.tiles_j = (k.cols + kQuantTile - 1) / kQuantTile;
  const int64_t blocks = (k.rows + kQuantTile - 1) / kQuantTile * k.tiles_j;
  if (blocks == 0) return cudaSuccess;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  const bool wide = k.x.dtype == ZERO_F32;
  if (k.nv) return wide ? launch_quantize_as<true, true>(k, blocks, st)
                        : launch_quantize_as<true, false>(k, blocks, st);
  return wide ? launch_quantize_as<false, true>(k, blocks, st)
              : launch_quantize_as<false, false>(k, blocks, st);
}

// --------------------------------------------------------------- dequantise --
// A thread takes 8 columns of a row: 4 bytes of codes, one scale.
template <bool NV>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ DequantK k) {
  after_previous_kernel();
  const float g = NV && k.g ? *(volatile const float*)k.g : 1.0f;
  const Extent e{k.rows, k.cols};
  const int64_t units = (k.cols + 7) / 8, total = units * k.rows;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < total;
       u += (int64_t)gridDim.x * kThreads) {
    const int64_t row = u / units, col = u % units * 8;
    const int64_t at = row * k.q.ld + col / 2, block = col / (NV ? 16 : 32);
    const int64_t scale = (row / 128 * k.q.scale_tiles + block / 4) * kScaleTile + row % 32 * 16 +
                          row % 128 / 32 * 4 + block % 4;
    if (!in_extent(at, at + 4, row * k.q.ld, row * k.q.ld + k.q.line_bytes, ZERO_SITE_FP4) ||
        !in_extent(scale, scale + 1, 0, k.q.scale_bytes, ZERO_SITE_FP4))
      continue;
    float v[8];
    from_codes8(*reinterpret_cast<const uint32_t*>(k.q.codes + at), v);
    const float d = scale_value<NV>(k.q.scales[scale], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], d);
    store8(k.y, row, col, k.cols - col < 8 ? (int)(k.cols - col) : 8, v, e, ZERO_SITE_FP4);
  }
}

cudaError_t launch_dequantize(const DequantK& k, cudaStream_t st) {
  const int64_t total = (k.cols + 7) / 8 * k.rows;
  if (total == 0) return cudaSuccess;
  const int64_t most = (int64_t)sm_count() * 8, blocks = (total + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  return k.nv ? launch_next(dequantize_kernel<true>, grid, dim3(kThreads), st, k)
              : launch_next(dequantize_kernel<false>, grid, dim3(kThreads), st, k);
}

// ------------------------------------------------------- the whole's scale --
// g = the largest finite magnitude / 2688 (6 x 448: the largest block's scale
// is then E4M3's largest), 1 where there is none.  Maxima of blocks, then one
// block over those; a maximum does not depend on the order.
__device__ __forceinline__ float block_max(float v) {
  __shared__ float part[32];
#pragma unroll
  for (int m = 16; m; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = threadIdx.x < blockDim.x / 32 ? part[threadIdx.x] : 0.0f;
#pragma unroll
  for (int m = 16; m; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
  return v;
}
__global__ void __launch_bounds__(kThreads) maxima_kernel(const __grid_constant__ MaxK k) {
  after_previous_kernel();
  const Extent e{k.rows, k.cols};
  const int64_t units = (k.cols + 7) / 8, total = units * k.rows;
  float top = 0.0f;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < total;
       u += (int64_t)gridDim.x * kThreads) {
    const int64_t row = u / units, col = u % units * 8;
    float v[8];
    load8(k.x, row, col, k.cols - col < 8 ? (int)(k.cols - col) : 8, v, e, ZERO_SITE_FP4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(v[j]);
      top = a < __uint_as_float(kInfBits) ? fmaxf(top, a) : top;
    }
  }
  top = block_max(top);
  if (threadIdx.x == 0 && in_extent(blockIdx.x, blockIdx.x + 1, 0, kMaxima, ZERO_SITE_FP4))
    k.maxima[blockIdx.x] = top;
}
__global__ void __launch_bounds__(kMaxima) maximum_kernel(const float* maxima, int n, float* g) {
  after_previous_kernel();
  float top = (int)threadIdx.x < n ? maxima[threadIdx.x] : 0.0f;
  top = block_max(top);
  if (threadIdx.x == 0) *g = top > 0.0f ? __fdiv_rn(top, 2688.0f) : 1.0f;
}

cudaError_t launch_tensor_scale(const MaxK& k, float* g, cudaStream_t st) {
  const int64_t total = (k.cols + 7) / 8 * k.rows;
  const int64_t most = (int64_t)sm_count() * 4 < kMaxima ? (int64_t)sm_count() * 4 : kMaxima;
  const int64_t blocks = (total + kThreads - 1) / kThreads;
  const int n = (int)(blocks < most ? blocks : most);
  if (n > 0) {
    cudaError_t e = launch_next(maxima_kernel, dim3(n), dim3(kThreads), st, k);
    if (e != cudaSuccess) return e;
  }
  return launch_next(maximum_kernel, dim3(1), dim3(kMaxima), st, k.maxima, n, g);
}

cudaError_t launch_fp4_product(const ProductK& k, int mode, cudaStream_t st) {
  if (k.rows <= 0 || k.cols <= 0) return cudaSuccess;
  return mode == LIN_FORWARD ? launch_mode<LIN_FORWARD, OF_FP4>(k, st)
                             : launch_mode<LIN_DINPUT, OF_FP4>(k, st);
}

cudaError_t timeouts_fp4(unsigned long long* out, bool reset) { return unit_timeouts(out, reset); }
cudaError_t bounds_fp4(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
