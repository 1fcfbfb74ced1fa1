// Matrices in microscaled 4-bit numbers (zero_fp4_*, include/zero.h): to E2M1
// codes with a scale per block and back, and their products on the tensor
// cores' block-scaled instructions (the kernel of zero_product.cuh).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "zero_fp4.cuh"
#include "zero_product.cuh"
#include "zero_walk.cuh"

namespace zk {

// A block's scale byte and the factor that brings its values to codes, from
// the largest magnitude's bits (NaN and infinity are the largest as integers).
// A block that holds either has scale NaN and codes 0.
// NV: E4M3 of the quotient by 6 g.  Its product with the reciprocal is within
// 2^-22 of it; where 2^-21 more and less round to one byte, so does the quotient.
// Only else is it divided.
constexpr uint32_t kInfBits = 0x7F800000u;
struct Whole {
  float g, six_g, by_six_g;  // 1 / (6 g)
};
template <bool NV>
__device__ __forceinline__ Whole whole_of(const float* at) {
  Whole w;
  w.g = NV && at ? *(volatile const float*)at : 1.0f;
  w.six_g = __fmul_rn(6.0f, w.g);
  // finite whatever g is, so that a block of zeros gets the scale 0
  w.by_six_g = fminf(__frcp_rn(w.six_g), 3.4028234e38f);
  return w;
}
template <bool NV>
__device__ __forceinline__ uint32_t block_scale(uint32_t top, const Whole& w, float& factor) {
  factor = 0.0f;
  if (NV) {
    if (top >= kInfBits) return 0x7Fu;
    const float most = __uint_as_float(top), t = most * w.by_six_g;
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(two)
        : "f"(t + t * 0x1p-21f), "f"(t - t * 0x1p-21f));
    uint32_t byte = two & 0xFFu;
    if (byte != two >> 8) byte = to_e4m3(__fdiv_rn(most, w.six_g));
    const float d = __fmul_rn(from_e4m3(byte), w.g);
    if (d > 0.0f) factor = __frcp_rn(d);
    return byte;
  }
  if (top >= kInfBits) return 0xFFu;
  // 2^(floor(log2 top) - 2) as E8M0, at least 2^-127
  const int exponent = (int)(top >> 23);
  const uint32_t byte = exponent > 2 ? (uint32_t)(exponent - 2) : 0u;
  factor = __uint_as_float((254u - byte) << 23);
  return byte;
}

// Codes of eight values of a block whose factor is known.
__device__ __forceinline__ uint32_t codes8(const float v[8], float factor) {
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = __fmul_rn(v[j], factor);
  return to_codes8(s);
}

// ----------------------------------------------------------------- quantise --
// Along the rows, along the columns, and both by a kernel each.  A block of 256
// threads takes whole scale tiles, or halves of them that no other block has, so
// that every byte of codes and scales, padding included, has one writer.  Bound by
// instructions, about 13 a value of each direction, 68 % of the issue slots.  (us,
// NV, alone along rows, along columns / by the kernel for both, both: 8192 x 4096
// bf16 19.0, 21.1 / 21.3, 21.8, 31.5 (105 MB); fp32 27.3, 32.8 / 40.4, 41.0, 52.8;
// 1024 x 1024 bf16 2.8, 2.9 / 3.6, 3.6, 5.0.  Blocks of 256 columns along the rows,
// a thread having eight rows instead of two, take 17.7 at 8192 x 4096, but at 8192 x
// 1024 8.2 instead of 7.3 and at 1024 x 1024 4.1 instead of 2.8.)
constexpr int kQuantRows = 128, kQuantThreads = 256;

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
// The larger magnitude of two bf16 in each half; NaN where there is one.
__device__ __forceinline__ uint32_t larger2(uint32_t top, uint32_t w) {
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w & 0x7FFF7FFFu));
  return top;
}
__device__ __forceinline__ int scale_at(int line, int block) {  // in a tile of 128 lines
  return (line & 31) * 16 + (line >> 5) * 4 + block;
}

// Along the rows: 128 rows by the columns of one scale tile, a thread having 16
// columns of every 64th (NV) or 32nd row: a block, or half of one.
template <bool NV, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_kernel(const __grid_constant__ QuantK k) {
  __shared__ __align__(16) unsigned char scales[kScaleTile];
  constexpr int kSize = NV ? 16 : 32, kAcross = kSize / 4, kDown = kQuantThreads / kAcross;
  constexpr int kAhead = 2;
  after_previous_kernel();
  const Whole whole = whole_of<NV>(k.g);
  const int64_t line_tile = blockIdx.x / k.tiles, tile = blockIdx.x % k.tiles;
  const int64_t row0 = line_tile * kQuantRows;
  const int unit = threadIdx.x % kAcross, line = threadIdx.x / kAcross;
  const int64_t col = tile * (4 * kSize) + unit * 16;
  const Extent e{k.rows, k.cols};
  auto valid = [&](int64_t c) {
    return c >= k.cols ? 0 : k.cols - c < 8 ? (int)(k.cols - c) : 8;
  };
  const bool kept = col / 2 < k.q.line_bytes;
#pragma unroll
  for (int p0 = 0; p0 < kQuantRows / kDown; p0 += kAhead) {
    Raw8 raw[2][kAhead];
    const int64_t first = row0 + p0 * kDown + line;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (first < k.rows) {
        Down<WIDE, ZERO_SITE_FP4>(k.x, first, kDown, col + 8 * h, valid(col + 8 * h))
            .template get<kAhead>(raw[h], k.rows, e);
      } else {
#pragma unroll
        for (int p = 0; p < kAhead; ++p) raw[h][p].a = raw[h][p].b = make_uint4(0, 0, 0, 0);
      }
    }
    unsigned char* to = k.q.codes + first * k.q.ld + col / 2;
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      const int64_t row = first + p * kDown;
      uint32_t top = 0;
      float v[16];
      values8<WIDE>(raw[0][p], v);
      values8<WIDE>(raw[1][p], v + 8);
      if (WIDE) {
#pragma unroll
        for (int j = 0; j < 16; ++j) top = larger(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      } else {
        uint32_t two = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          two = larger2(larger2(larger2(larger2(two, raw[h][p].a.x), raw[h][p].a.y),
                                raw[h][p].a.z),
                        raw[h][p].a.w);
        top = larger(two << 16, two & 0xFFFF0000u);
      }
      if (!NV) top = larger(top, __shfl_xor_sync(0xffffffffu, top, 1));
      float factor;
      const uint32_t byte = block_scale<NV>(top, whole, factor);
      uint2 codes = make_uint2(codes8(v, factor), codes8(v + 8, factor));
      if (top >= kInfBits) codes = make_uint2(0u, 0u);
      if (row < k.rows && kept && in_extent(row, row + 1, 0, k.rows, ZERO_SITE_FP4) &&
          in_extent(col / 2, col / 2 + 8, 0, k.q.line_bytes, ZERO_SITE_FP4))
        *reinterpret_cast<uint2*>(to + p * kDown * k.q.ld) = codes;
      if (NV || unit % 2 == 0)
        scales[scale_at(p0 * kDown + p * kDown + line, NV ? unit : unit / 2)] =
            (unsigned char)byte;
    }
  }
  __syncthreads();
  const int64_t at = (line_tile * k.q.scale_tiles + tile) * kScaleTile + threadIdx.x * 16;
  if (threadIdx.x < kScaleTile / 16 && in_extent(at, at + 16, 0, k.q.scale_bytes, ZERO_SITE_FP4))
    *reinterpret_cast<uint4*>(k.q.scales + at) =
        *reinterpret_cast<const uint4*>(scales + threadIdx.x * 16);
}

// Along the columns: 128 rows by 64 columns cross shared memory.  A thread has
// a block of one column, or (bf16, NV) of two side by side, one 32-bit word of
// each row.  Codes go out through shared memory, 64 bytes of each line; of a
// scale tile's 16-byte rows the 64 columns fill half.
constexpr int kQuantCols = 64, kCodeLine = 80;

template <bool NV, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_cols_kernel(const __grid_constant__ QuantK k) {
  constexpr int kElem = WIDE ? 4 : 2, kLine = kQuantCols * kElem + 16;
  constexpr int kSize = NV ? 16 : 32, kBlocks = kQuantRows / kSize, kTiles = NV ? 2 : 1;
  constexpr int kSide = NV && !WIDE ? 2 : 1;  // columns of a thread
  __shared__ __align__(16) unsigned char tile[kQuantRows * kLine];
  __shared__ __align__(16) unsigned char codes[kQuantCols * kCodeLine];
  __shared__ __align__(16) unsigned char scales[kTiles][32 * 8];
  after_previous_kernel();
  const Whole whole = whole_of<NV>(k.g);
  const int64_t row_tile = blockIdx.x / k.tiles, col0 = blockIdx.x % k.tiles * kQuantCols;
  const int64_t row0 = row_tile * kQuantRows;
  const Extent e{k.rows, k.cols};
  {
    constexpr int kAcross = kQuantCols / 8, kDown = kQuantThreads / kAcross;  // 4 rows a thread
    const int unit = threadIdx.x % kAcross, line = threadIdx.x / kAcross;
    const int64_t col = col0 + unit * 8;
    const int valid = col >= k.cols ? 0 : k.cols - col < 8 ? (int)(k.cols - col) : 8;
    Raw8 raw[kQuantRows / kDown];
#pragma unroll
    for (int p = 0; p < kQuantRows / kDown; ++p) raw[p].a = raw[p].b = make_uint4(0, 0, 0, 0);
    if (row0 + line < k.rows)
      Down<WIDE, ZERO_SITE_FP4>(k.x, row0 + line, kDown, col, valid)
          .template get<kQuantRows / kDown>(raw, k.rows, e);
#pragma unroll
    for (int p = 0; p < kQuantRows / kDown; ++p) {
      uint4* at =
          reinterpret_cast<uint4*>(tile + (p * kDown + line) * kLine + unit * 8 * kElem);
      at[0] = raw[p].a;
      if (WIDE) at[1] = raw[p].b;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int u = threadIdx.x; u < kQuantCols / kSide * kBlocks; u += kQuantThreads) {
    const int c = u % (kQuantCols / kSide) * kSide, b = u / (kQuantCols / kSide);
    const unsigned char* at = tile + b * kSize * kLine + c * kElem;
    uint32_t raw[kSize], top[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kSize; ++i)
      raw[i] = WIDE || kSide == 2 ? *reinterpret_cast<const uint32_t*>(at + i * kLine)
                                  : *reinterpret_cast<const uint16_t*>(at + i * kLine);
    if (WIDE) {
#pragma unroll
      for (int i = 0; i < kSize; ++i) top[0] = larger(top[0], raw[i] & 0x7FFFFFFFu);
    } else {
      uint32_t two = 0;
#pragma unroll
      for (int i = 0; i < kSize; ++i) two = larger2(two, raw[i]);
      top[0] = two << 16;
      top[1] = two & 0xFFFF0000u;
    }
#pragma unroll
    for (int h = 0; h < kSide; ++h) {
      float factor;
      const uint32_t byte = block_scale<NV>(top[h], whole, factor);
      scales[b >> 2][((c + h) & 31) * 8 + ((c + h) >> 5) * 4 + (b & 3)] = (unsigned char)byte;
      uint32_t* out = reinterpret_cast<uint32_t*>(codes + (c + h) * kCodeLine + b * (kSize / 2));
#pragma unroll
      for (int i = 0; i < kSize / 8; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = raw[8 * i + j];
          v[j] = WIDE ? __uint_as_float(w) : h ? bf16_hi(w) : bf16_lo(w);
        }
        out[i] = top[h] >= kInfBits ? 0u : codes8(v, factor);
      }
    }
  }
  __syncthreads();
  {
    const int c = threadIdx.x >> 2;
    const int64_t line = col0 + c, byte = row0 / 2 + (threadIdx.x & 3) * 16;
    if (line < k.cols && byte < k.qt.line_bytes &&
        in_extent(line, line + 1, 0, k.cols, ZERO_SITE_FP4) &&
        in_extent(byte, byte + 16, 0, k.qt.line_bytes, ZERO_SITE_FP4))
      *reinterpret_cast<uint4*>(k.qt.codes + line * k.qt.ld + byte) =
          *reinterpret_cast<const uint4*>(codes + c * kCodeLine + (threadIdx.x & 3) * 16);
  }
  const int64_t t = row_tile * kTiles + threadIdx.x / 32;
  const int64_t at = (col0 / 128 * k.qt.scale_tiles + t) * kScaleTile + threadIdx.x % 32 * 16 +
                     col0 % 128 / 8;
  if (threadIdx.x < kTiles * 32 && t < k.qt.scale_tiles &&
      in_extent(at, at + 8, 0, k.qt.scale_bytes, ZERO_SITE_FP4))
    *reinterpret_cast<uint2*>(k.qt.scales + at) =
        *reinterpret_cast<const uint2*>(scales[threadIdx.x / 32] + threadIdx.x % 32 * 8);
}

// In both directions: 128 x 128 values cross shared memory, where they are whole
// scale tiles either way.  A thread takes one block of a row after another, then
// blocks of two columns side by side (bf16: one 32-bit word) or of one.
template <bool WIDE>
struct QuantShared {
  static constexpr int kElem = WIDE ? 4 : 2, kLine = kQuantRows * kElem + 16;
  unsigned char tile[kQuantRows * kLine];
  unsigned char codes[kQuantRows * kCodeLine];  // of one direction, 64 bytes a line
  unsigned char scales[2][1024];                // rows', columns'
};

// One direction's codes and scale tiles to memory.  line0: its first line;
// byte0: of the lines' codes; tiles (line0 / 128, tile0 + t), t < tiles.
__device__ __forceinline__ void store_quantized(const Fp4Mat& o, const unsigned char* codes,
                                                const unsigned char* scales, int64_t line0,
                                                int64_t lines, int64_t byte0, int64_t tile0,
                                                int tiles) {
#pragma unroll
  for (int p = 0; p < kQuantRows * 4 / kQuantThreads; ++p) {
    const int u = p * kQuantThreads + threadIdx.x, c = u >> 2;
    const int64_t line = line0 + c, byte = byte0 + (u & 3) * 16, at = line * o.ld + byte;
    if (line < lines && byte < o.line_bytes &&
        in_extent(at, at + 16, line * o.ld, line * o.ld + o.line_bytes, ZERO_SITE_FP4))
      *reinterpret_cast<uint4*>(o.codes + at) =
          *reinterpret_cast<const uint4*>(codes + c * kCodeLine + (u & 3) * 16);
  }
  const int unit = threadIdx.x;  // 16 bytes
  const int64_t t = tile0 + unit / 32;
  if (unit >= tiles * 32 || t >= o.scale_tiles) return;
  const int64_t at = (line0 / kQuantRows * o.scale_tiles + t) * kScaleTile + unit % 32 * 16;
  if (!in_extent(at, at + 16, 0, o.scale_bytes, ZERO_SITE_FP4)) return;
  *reinterpret_cast<uint4*>(o.scales + at) = *reinterpret_cast<const uint4*>(scales + unit * 16);
}

template <bool NV, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads, WIDE ? 2 : 4)
    quantize_both_kernel(const __grid_constant__ QuantK k) {
  extern __shared__ __align__(16) unsigned char quant_smem[];
  using Shared = QuantShared<WIDE>;
  Shared& sh = *reinterpret_cast<Shared*>(quant_smem);
  constexpr int kSize = NV ? 16 : 32, kTiles = NV ? 2 : 1, kBlocks = kQuantRows / kSize;
  after_previous_kernel();
  const Whole whole = whole_of<NV>(k.g);
  const int64_t row_tile = blockIdx.x / (uint32_t)k.tiles, row0 = row_tile * kQuantRows;
  const int64_t col0 = (blockIdx.x - row_tile * k.tiles) * kQuantRows;
  const int t = threadIdx.x;
  {
    const int line = t >> 4, unit = t & 15;
    const Extent e{k.rows, k.cols};
    const int64_t col = col0 + unit * 8;
    const int valid = col >= k.cols ? 0 : k.cols - col < 8 ? (int)(k.cols - col) : 8;
    Raw8 raw[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) raw[p].a = raw[p].b = make_uint4(0, 0, 0, 0);
    if (row0 + line < k.rows)
      Down<WIDE, ZERO_SITE_FP4>(k.x, row0 + line, 16, col, valid)
          .template get<8>(raw, k.rows, e);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint4* at = reinterpret_cast<uint4*>(sh.tile + (p * 16 + line) * Shared::kLine +
                                           unit * 8 * Shared::kElem);
      at[0] = raw[p].a;
      if (WIDE) at[1] = raw[p].b;
    }
  }
  __syncthreads();
  for (int u = t; u < kQuantRows * kBlocks; u += kQuantThreads) {
    const int r = u % kQuantRows, b = u / kQuantRows;
    const unsigned char* at = sh.tile + r * Shared::kLine + b * kSize * Shared::kElem;
    constexpr int kWords = kSize * Shared::kElem / 16;
    uint4 raw[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) raw[i] = reinterpret_cast<const uint4*>(at)[i];
    uint32_t top = 0;
    if (WIDE) {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        top = larger(larger(top, larger(raw[i].x & 0x7FFFFFFFu, raw[i].y & 0x7FFFFFFFu)),
                     larger(raw[i].z & 0x7FFFFFFFu, raw[i].w & 0x7FFFFFFFu));
    } else {
      uint32_t two = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        two = larger2(larger2(larger2(larger2(two, raw[i].x), raw[i].y), raw[i].z), raw[i].w);
      top = larger(two << 16, two & 0xFFFF0000u);
    }
    float factor;
    sh.scales[0][(b >> 2) * kScaleTile + scale_at(r, b & 3)] =
        (unsigned char)block_scale<NV>(top, whole, factor);
    uint32_t* out = reinterpret_cast<uint32_t*>(sh.codes + r * kCodeLine + b * (kSize / 2));
#pragma unroll
    for (int i = 0; i < kSize / 8; ++i) {
      float v[8];
      if (WIDE) {
        const uint4 x = raw[(2 * i) % kWords], y = raw[(2 * i + 1) % kWords];
        v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
        v[4] = __uint_as_float(y.x); v[5] = __uint_as_float(y.y);
        v[6] = __uint_as_float(y.z); v[7] = __uint_as_float(y.w);
      } else {
        from_bf16(raw[i % kWords], v);
      }
      out[i] = top >= kInfBits ? 0u : codes8(v, factor);
    }
  }
  __syncthreads();
  store_quantized(k.q, sh.codes, sh.scales[0], row0, k.rows, col0 / 2, col0 / (4 * kSize), kTiles);
  __syncthreads();  // the codes are read
  constexpr int kSide = WIDE ? 1 : 2;  // columns of a thread
  for (int u = t; u < kQuantRows / kSide * kBlocks; u += kQuantThreads) {
    const int c = u % (kQuantRows / kSide) * kSide, b = u / (kQuantRows / kSide);
    const unsigned char* at = sh.tile + b * kSize * Shared::kLine + c * Shared::kElem;
    uint32_t raw[kSize], top[kSide];
#pragma unroll
    for (int i = 0; i < kSize; ++i)
      raw[i] = *reinterpret_cast<const uint32_t*>(at + i * Shared::kLine);
    if (WIDE) {
      top[0] = 0;
#pragma unroll
      for (int i = 0; i < kSize; ++i) top[0] = larger(top[0], raw[i] & 0x7FFFFFFFu);
    } else {
      uint32_t two = 0;
#pragma unroll
      for (int i = 0; i < kSize; ++i) two = larger2(two, raw[i]);
      top[0] = two << 16;
      top[kSide - 1] = two & 0xFFFF0000u;
    }
#pragma unroll
    for (int h = 0; h < kSide; ++h) {
      float factor;
      const uint32_t most = !WIDE && h == 0 ? top[0] : top[kSide - 1];
      sh.scales[1][(b >> 2) * kScaleTile + scale_at(c + h, b & 3)] =
          (unsigned char)block_scale<NV>(most, whole, factor);
      uint32_t* out =
          reinterpret_cast<uint32_t*>(sh.codes + (c + h) * kCodeLine + b * (kSize / 2));
#pragma unroll
      for (int i = 0; i < kSize / 8; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = raw[8 * i + j];
          v[j] = WIDE ? __uint_as_float(w) : h ? bf16_hi(w) : bf16_lo(w);
        }
        out[i] = most >= kInfBits ? 0u : codes8(v, factor);
      }
    }
  }
  __syncthreads();
  store_quantized(k.qt, sh.codes, sh.scales[1], col0, k.cols, row0 / 2, row0 / (4 * kSize), kTiles);
}

template <bool NV, bool WIDE>
static cudaError_t launch_quantize_both(const QuantK& k, int64_t blocks, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  constexpr int bytes = (int)sizeof(QuantShared<WIDE>);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(quantize_both_kernel<NV, WIDE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  return launch_next_with(bytes, quantize_both_kernel<NV, WIDE>, dim3((unsigned)blocks),
                          dim3(kQuantThreads), st, k);
}
template <bool NV, bool WIDE>
static cudaError_t launch_quantize_as(QuantK k, cudaStream_t st) {
  const int64_t row_tiles = (k.rows + kQuantRows - 1) / kQuantRows;
  const bool both = k.q.codes && k.qt.codes;
  // (along the columns the last half too: its scales are padding)
  k.tiles = both ? (k.cols + kQuantRows - 1) / kQuantRows
            : k.q.codes ? k.q.scale_tiles : (k.cols + 127) / 128 * 2;
  const int64_t blocks = row_tiles * k.tiles;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  if (both) return launch_quantize_both<NV, WIDE>(k, blocks, st);
  return launch_next(k.q.codes ? quantize_rows_kernel<NV, WIDE> : quantize_cols_kernel<NV, WIDE>,
                     dim3((unsigned)blocks), dim3(kQuantThreads), st, k);
}

cudaError_t launch_quantize(const QuantK& k, cudaStream_t st) {
  if (k.rows == 0 || k.cols == 0) return cudaSuccess;
  const bool wide = k.x.dtype == ZERO_F32;
  if (k.nv) return wide ? launch_quantize_as<true, true>(k, st)
                        : launch_quantize_as<true, false>(k, st);
  return wide ? launch_quantize_as<false, true>(k, st) : launch_quantize_as<false, false>(k, st);
}

// --------------------------------------------------------------- dequantise --
// A warp takes 256 columns of every 8th row of a block's, PASSES of them, a lane 8
// columns: 4 bytes of codes and one scale of each.  Bound by memory, mostly by the
// stores: 8192 x 4096 to bf16 (86 MB) 16.5 us.  (Walking down the rows four at a
// time with every address from the walk's took 19.3, 11 instructions a value.)
constexpr int kDequantCols = 256, kDequantDown = 8;
template <bool NV, bool WIDE, int PASSES>
__global__ void __launch_bounds__(kQuantThreads)
    dequantize_kernel(const __grid_constant__ DequantK k, int tiles) {
  constexpr int kElem = WIDE ? 4 : 2, kRows = kDequantDown * PASSES;
  after_previous_kernel();
  const float g = NV && k.g ? *(volatile const float*)k.g : 1.0f;
  const int64_t part = blockIdx.x / (uint32_t)tiles;
  const int64_t col = (blockIdx.x - part * tiles) * kDequantCols + threadIdx.x % 32 * 8;
  const int64_t row0 = part * kRows + threadIdx.x / 32;
  if (col >= k.cols || row0 >= k.rows) return;
  const Extent e{k.rows, k.cols};
  const int there =
      (int)min((k.rows - row0 + kDequantDown - 1) / kDequantDown, (int64_t)PASSES);
  const int64_t last = row0 + (there - 1) * kDequantDown;
  const bool in = in_extent(col / 2, col / 2 + 4, 0, k.q.line_bytes, ZERO_SITE_FP4) &&
                  in_extent(last, last + 1, 0, k.rows, ZERO_SITE_FP4);
  // (a block's rows lie in one tile of scales)
  const int64_t block = col / (NV ? 16 : 32);
  const int64_t tile = ((row0 >> 7) * k.q.scale_tiles + block / 4) * kScaleTile;
  const unsigned char* scales = k.q.scales + tile + (block & 3);
  const unsigned char* from = k.q.codes + row0 * k.q.ld + col / 2;
  uint32_t codes[PASSES], scale[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = ((int)row0 & 127) + p * kDequantDown, at = (r & 31) * 16 + (r >> 5) * 4;
    codes[p] = scale[p] = 0;
    if (p < there && in && in_extent(tile + at, tile + at + 4, 0, k.q.scale_bytes, ZERO_SITE_FP4)) {
      codes[p] = *reinterpret_cast<const uint32_t*>(from);
      scale[p] = scales[at];
    }
    from += kDequantDown * k.q.ld;
  }
  const int valid = k.cols - col < 8 ? (int)(k.cols - col) : 8;
  const bool fast = k.y.vec && valid == 8;
  char* to = static_cast<char*>(k.y.p) + (row0 * k.y.ld + col) * kElem;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    if (p >= there) break;
    const float d = scale_value<NV>(scale[p], g);
    float v[8];
    from_codes8(codes[p], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], d);
    if (fast && in) {
      if (WIDE) {
        reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(to) = pack8(v);
      }
    } else {
      store8(k.y, row0 + p * kDequantDown, col, valid, v, e, ZERO_SITE_FP4);
    }
    to += kDequantDown * k.y.ld * kElem;
  }
}

template <int PASSES>
static cudaError_t launch_dequantize_as(const DequantK& k, int64_t tiles, cudaStream_t st) {
  const int64_t parts = (k.rows + kDequantDown * PASSES - 1) / (kDequantDown * PASSES);
  if (parts * tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  const bool wide = k.y.dtype == ZERO_F32;
  return launch_next(
      k.nv ? (wide ? dequantize_kernel<true, true, PASSES> : dequantize_kernel<true, false, PASSES>)
      : wide ? dequantize_kernel<false, true, PASSES>
             : dequantize_kernel<false, false, PASSES>,
      dim3((unsigned)(parts * tiles)), dim3(kQuantThreads), st, k, (int)tiles);
}
cudaError_t launch_dequantize(const DequantK& k, cudaStream_t st) {
  if (k.rows == 0 || k.cols == 0) return cudaSuccess;
  const int64_t tiles = (k.cols + kDequantCols - 1) / kDequantCols;
  // Eight rows a thread where that leaves four blocks for each SM; two else, and
  // from MX to fp32, where the stores alone count and shorter blocks keep more of
  // them in flight.  (us with eight / two: 8192 x 4096 NV to fp32 38.2 / 43.1, MX to
  // fp32 37.8 / 33.5; 6001 x 2048 NV 16.0 / 17.1, MX 17.1 / 14.0.)
  const bool few_bytes = k.nv || k.y.dtype != ZERO_F32;
  return few_bytes && (k.rows + 63) / 64 * tiles >= 4 * (int64_t)sm_count()
             ? launch_dequantize_as<8>(k, tiles, st)
             : launch_dequantize_as<2>(k, tiles, st);
}

// ------------------------------------------------------- the whole's scale --
// g = the largest finite magnitude / 2688 (6 x 448: the largest block's scale
// is then E4M3's largest), 1 where there is none.  Not below kLeastWhole, from
// which on the least scale's product with g, 2^-9 g, and the reciprocals of that
// and of 6 g are normal numbers: below 2^-130 or so they are infinite, and values
// times them NaN.  What this loses is blocks of values up to 3.5e-38 (6 2^-127).
// Maxima of blocks, then one block over those; a maximum does not depend on the
// order.  Bound by memory: 8192 x 4096 bf16 (67 MB) 14.3 us, and 2 to 4 for the
// second kernel.
constexpr float kLeastWhole = 0x1p-117f;
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
// NaN loses every comparison; a thread that met an infinity goes over its
// values once more and leaves what is not finite out.
template <bool WIDE>
__device__ __forceinline__ float unit_top(float top, const Raw8& raw, bool finite) {
  const uint32_t w[8] = {raw.a.x, raw.a.y, raw.a.z, raw.a.w, raw.b.x, raw.b.y, raw.b.z, raw.b.w};
  if (WIDE || finite) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a =
          fabsf(WIDE ? __uint_as_float(w[j]) : j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]));
      top = finite && !(a < __uint_as_float(kInfBits)) ? top : fmaxf(top, a);
    }
    return top;
  }
  uint32_t two = w[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int j = 1; j < 4; ++j)
    asm("max.bf16x2 %0, %0, %1;" : "+r"(two) : "r"(w[j] & 0x7FFF7FFFu));
  return fmaxf(top, fmaxf(bf16_lo(two), bf16_hi(two)));
}
template <bool WIDE>
__global__ void __launch_bounds__(kThreads)
    maxima_kernel(const __grid_constant__ MaxK k, int log2_across) {
  after_previous_kernel();
  constexpr int kAhead = WIDE ? 4 : 8;  // rows whose loads are in flight together
  const Extent e{k.rows, k.cols};
  const int across = 1 << log2_across, down = kThreads >> log2_across;
  const int64_t step = (int64_t)gridDim.y * down;
  auto over = [&](bool finite) {
    float top = 0.0f;
    for (int64_t col = ((int64_t)blockIdx.x * across + (threadIdx.x & (across - 1))) * 8;
         col < k.cols; col += (int64_t)gridDim.x * across * 8) {
      const int valid = k.cols - col < 8 ? (int)(k.cols - col) : 8;
      const int64_t first = (int64_t)blockIdx.y * down + (threadIdx.x >> log2_across);
      Down<WIDE, ZERO_SITE_FP4> x(k.x, first, step, col, valid);
      for (; x.row < k.rows; x.on(kAhead)) {
        Raw8 raw[kAhead];
        x.template get<kAhead>(raw, k.rows, e);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) top = unit_top<WIDE>(top, raw[i], finite);
      }
    }
    return top;
  };
  float top = over(false);
  if (top >= __uint_as_float(kInfBits)) top = over(true);
  top = block_max(top);
  const int at = (int)(blockIdx.y * gridDim.x + blockIdx.x);
  if (threadIdx.x == 0 && in_extent(at, at + 1, 0, kMaxima, ZERO_SITE_FP4)) k.maxima[at] = top;
}
__global__ void __launch_bounds__(kMaxima) maximum_kernel(const float* maxima, int n, float* g) {
  after_previous_kernel();
  float top = (int)threadIdx.x < n ? *(volatile const float*)(maxima + threadIdx.x) : 0.0f;
  top = block_max(top);
  if (threadIdx.x == 0) *g = top > 0.0f ? fmaxf(__fdiv_rn(top, 2688.0f), kLeastWhole) : 1.0f;
}

cudaError_t launch_tensor_scale(const MaxK& k, float* g, cudaStream_t st) {
  int n = 0;
  if (k.rows > 0 && k.cols > 0) {
    Walk w = walk_over(k.rows, k.cols, (int64_t)sm_count() * 8);
    if (w.grid.x > kMaxima) w.grid.x = kMaxima;
    if (w.grid.x * w.grid.y > kMaxima) w.grid.y = kMaxima / w.grid.x;
    n = (int)(w.grid.x * w.grid.y);
    cudaError_t e = launch_next(k.x.dtype == ZERO_F32 ? maxima_kernel<true> : maxima_kernel<false>,
                                w.grid, dim3(kThreads), st, k, w.log2_across);
    if (e != cudaSuccess) return e;
  }
  return launch_next(maximum_kernel, dim3(1), dim3(kMaxima), st, k.maxima, n, g);
}

// Whether a few rows are quicker by zero_fp4_rows.cu, by the times of both in us:
// blocks of 16 outputs that share an SM's instruction slots, each taking 2048
// codes at a time; or tiles of 256 outputs whose steps of 256 codes follow one
// another.  Neither depends much on the rows, 1 to 8.  (Measured, NV, 8 rows, few
// rows / tiles, [n, k]: 1024 x 256 2.3 / 4.5, 1024 x 4096 4.7 / 7.2, 4096 x 4096 5.8
// / 7.7, 4096 x 8192 9.2 / 9.4, 4096 x 11008 11.2 / 10.8, 8192 x 1024 5.7 / 5.8, 8192 x
// 2048 7.2 / 6.6, 11008 x 2048 9.2 / 7.1, 11008 x 4096 12.6 / 9.0, 16384 x 512 8.4 /
// 5.8, 50257 x 768 22 / 9.2, 256 x 16384 8.6 / 11.0.)
static bool few_rows_win(const ProductK& k) {
  if (k.rows > kFewRows) return false;
  const double codes = 4.0 * (double)k.depth, n = (double)k.cols;
  const double turns = std::max(0.5, codes / 2048), steps = std::ceil(codes / 256);
  const double blocks = std::ceil(n / 16 / sm_count()), tiles = std::ceil(n / 256);
  const double rows_us = 1.7 + blocks * (0.5 + 0.83 * turns);
  const double tiles_us = 4.7 + 0.115 * steps + 0.02 * tiles + 2.2e-8 * n * codes;
  return rows_us <= tiles_us;
}

cudaError_t launch_fp4_product(const ProductK& k, int mode, cudaStream_t st) {
  if (k.rows <= 0 || k.cols <= 0) return cudaSuccess;
  if (few_rows_win(k)) return launch_fp4_rows(k, mode, st);
  return mode == LIN_FORWARD ? launch_mode<LIN_FORWARD, OF_FP4>(k, st)
                             : launch_mode<LIN_DINPUT, OF_FP4>(k, st);
}

cudaError_t timeouts_fp4(unsigned long long* out, bool reset) { return unit_timeouts(out, reset); }
cudaError_t bounds_fp4(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
