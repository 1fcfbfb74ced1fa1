// Matrices in microscaled 4-bit numbers (zero_fp4_*, include/zero.h): to E2M1
// codes with a scale per block and back, and their products on the tensor
// cores' block-scaled instructions (the kernel of zero_product.cuh).
#include "zero_fp4.cuh"
#include "zero_product.cuh"

namespace zk {

// A block's scale byte and the factor that brings its values to codes, from
// the largest magnitude's bits (NaN and infinity are the largest as integers).
// A block that holds either has scale NaN and codes 0.
// NV: the quotient by 6 g first by its reciprocal, half a unit of E4M3's
// sixteenths from it at most where both neighbours at 2^-21 give the same byte;
// else divided (an IEEE division for each block: __DIV__).
constexpr uint32_t kInfBits = 0x7F800000u;
struct Whole {
  float g, six_g, by_six_g;  // 1 / (6 g)
};
template <bool NV>
__device__ __forceinline__ Whole whole_of(const float* at) {
  Whole w;
  w.g = NV && at ? *(volatile const float*)at : 1.0f;
  w.six_g = __fmul_rn(6.0f, w.g);
  w.by_six_g = __frcp_rn(w.six_g);
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

// Eight columns of rows some distance apart, as they lie in memory: one or two
// 16-byte accesses where the matrix and the columns allow it, decided once.
template <bool WIDE>
struct Down {
  const Mat& m;
  char* p;
  int64_t step, row, col, rows_apart;
  int valid;
  bool fast;
  __device__ __forceinline__ Down(const Mat& mat, int64_t row0, int64_t apart, int64_t column,
                                  int count)
      : m(mat), row(row0), col(column), rows_apart(apart), valid(count) {
    constexpr int es = WIDE ? 4 : 2;
    p = static_cast<char*>(m.p) + (row0 * m.ld + column) * es;
    step = apart * m.ld * es;
    fast = m.vec && count == 8;
  }
  // N rows, zeros from row `rows` on.  One test for all: conditions between the
  // loads would keep them from being in flight together (maxima of 8192 x 4096
  // bf16: 31 us so, __MAX__ with one).
  template <int N>
  __device__ __forceinline__ void get(Raw8 r[N], int64_t rows, const Extent& e) const {
    if (fast && in_extent(row, row + 1, 0, e.rows, ZERO_SITE_FP4) &&
        in_extent(col, col + 8, 0, e.cols, ZERO_SITE_FP4)) {
      const char* at = p;
      int64_t here = row;
#pragma unroll
      for (int i = 0; i < N; ++i) {  // past the last row the one before again
        r[i].a = ld16(at);
        r[i].b = WIDE ? ld16(at + 16) : make_uint4(0, 0, 0, 0);
        here += rows_apart;
        at += here < rows ? step : 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        r[i].a = r[i].b = make_uint4(0, 0, 0, 0);
        if (row + i * rows_apart < rows && valid > 0)
          r[i] = raw8(m, row + i * rows_apart, col, valid, e, ZERO_SITE_FP4);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (row + i * rows_apart >= rows) r[i].a = r[i].b = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void put(int i, const float v[8], const Extent& e) const {
    const int64_t at = row + i * rows_apart;
    if (fast && in_extent(at, at + 1, 0, e.rows, ZERO_SITE_FP4) &&
        in_extent(col, col + 8, 0, e.cols, ZERO_SITE_FP4)) {
      if (WIDE) {
        float4* to = reinterpret_cast<float4*>(p + i * step);
        to[0] = make_float4(v[0], v[1], v[2], v[3]);
        to[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(p + i * step) = pack8(v);
      }
      return;
    }
    store8(m, at, col, valid, v, e, ZERO_SITE_FP4);
  }
  __device__ __forceinline__ void on(int steps) {
    p += steps * step;
    row += steps * rows_apart;
  }
};

// Codes of eight values of a block whose factor is known.
__device__ __forceinline__ uint32_t codes8(const float v[8], float factor) {
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = __fmul_rn(v[j], factor);
  return to_codes8(s);
}

// ----------------------------------------------------------------- quantise --
// A block of 256 threads takes 128 x 128 values into shared memory: their codes
// and scales are whole scale tiles in both directions, so that every byte of
// those (padding included) has one writer.  Then a thread takes one block of a
// row after another, and in the other direction the blocks of two columns side
// by side (bf16: one 32-bit word); largest magnitudes of bf16 are found two at
// a time, fp32's as integers, which order NaN and infinity above all numbers.
// Codes go out through shared memory, 64 bytes of each line.
constexpr int kQuantTile = 128, kQuantThreads = 256, kCodeLine = 80;

template <bool WIDE>
struct QuantShared {
  static constexpr int kElem = WIDE ? 4 : 2, kLine = kQuantTile * kElem + 16;
  unsigned char tile[kQuantTile * kLine];
  unsigned char codes[kQuantTile * kCodeLine];  // of one direction, 64 bytes a line
  unsigned char scales[2][1024];                // rows', columns'
};

__device__ __forceinline__ int scale_at(int line, int block) {  // in a 128-line tile's scales
  return (block >> 2) * kScaleTile + (line & 31) * 16 + (line >> 5) * 4 + (block & 3);
}

// One direction's codes and scale tiles to memory.  line0: its first line;
// byte0: of the lines' codes; tiles (line0 / 128, tile0 + t), t < tiles.
__device__ __forceinline__ void store_quantized(const Fp4Mat& o, const unsigned char* codes,
                                                const unsigned char* scales, int64_t line0,
                                                int64_t lines, int64_t byte0, int64_t tile0,
                                                int tiles) {
#pragma unroll
  for (int p = 0; p < kQuantTile * 4 / kQuantThreads; ++p) {
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
  const int64_t at = (line0 / kQuantTile * o.scale_tiles + t) * kScaleTile + unit % 32 * 16;
  if (!in_extent(at, at + 16, 0, o.scale_bytes, ZERO_SITE_FP4)) return;
  *reinterpret_cast<uint4*>(o.scales + at) = *reinterpret_cast<const uint4*>(scales + unit * 16);
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
// The larger magnitude of two bf16 in each half; NaN where there is one.
__device__ __forceinline__ uint32_t larger2(uint32_t top, uint32_t w) {
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w & 0x7FFF7FFFu));
  return top;
}

template <bool NV, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads, WIDE ? 2 : 4)
    quantize_kernel(const __grid_constant__ QuantK k) {
  extern __shared__ __align__(16) unsigned char quant_smem[];
  using Shared = QuantShared<WIDE>;
  Shared& sh = *reinterpret_cast<Shared*>(quant_smem);
  constexpr int kSize = NV ? 16 : 32, kTiles = NV ? 2 : 1, kBlocks = kQuantTile / kSize;
  after_previous_kernel();
  const Whole whole = whole_of<NV>(k.g);
  const int64_t row0 = (int64_t)(blockIdx.x / k.tiles_j) * kQuantTile;
  const int64_t col0 = (int64_t)(blockIdx.x % k.tiles_j) * kQuantTile;
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
      Down<WIDE>(k.x, row0 + line, 16, col, valid).template get<8>(raw, k.rows, e);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint4* at = reinterpret_cast<uint4*>(sh.tile + (p * 16 + line) * Shared::kLine +
                                           unit * 8 * Shared::kElem);
      at[0] = raw[p].a;
      if (WIDE) at[1] = raw[p].b;
    }
  }
  __syncthreads();
  const bool rows = k.q.codes != nullptr, columns = k.qt.codes != nullptr;
  if (rows) {
    for (int u = t; u < kQuantTile * kBlocks; u += kQuantThreads) {
      const int r = u % kQuantTile, b = u / kQuantTile;
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
      sh.scales[0][scale_at(r, b)] = (unsigned char)block_scale<NV>(top, whole, factor);
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
    store_quantized(k.q, sh.codes, sh.scales[0], row0, k.rows, col0 / 2, col0 / (4 * kSize),
                    kTiles);
  }
  if (!columns) return;
  if (rows) __syncthreads();  // the codes are read
  constexpr int kSide = WIDE ? 1 : 2;  // columns of a thread
  for (int u = t; u < kQuantTile / kSide * kBlocks; u += kQuantThreads) {
    const int c = u % (kQuantTile / kSide) * kSide, b = u / (kQuantTile / kSide);
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
      sh.scales[1][scale_at(c + h, b)] = (unsigned char)block_scale<NV>(most, whole, factor);
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
static cudaError_t launch_quantize_as(const QuantK& k, int64_t blocks, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  constexpr int bytes = (int)sizeof(QuantShared<WIDE>);
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

// ------------------------------------------------------- walks over a matrix --
// Units of 8 columns: a block of 256 threads covers `across` units (a power of
// two, up to 32) of 256 / across rows, and goes on down the rows: no division.
struct Walk {
  int log2_across;
  dim3 grid;
};
static Walk walk_over(int64_t rows, int64_t cols) {
  const int64_t units = (cols + 7) / 8;
  Walk w;
  w.log2_across = 0;
  while (w.log2_across < 5 && (1ll << w.log2_across) < units) ++w.log2_across;
  const int64_t x = (units + (1 << w.log2_across) - 1) >> w.log2_across;
  const int64_t each = kThreads >> w.log2_across;
  int64_t y = (rows + each - 1) / each, most = (int64_t)sm_count() * 8 / (x < 1 ? 1 : x) + 1;
  if (most > 65535) most = 65535;
  if (y > most) y = most;
  w.grid = dim3((unsigned)x, (unsigned)y);
  return w;
}

// --------------------------------------------------------------- dequantise --
// A thread takes 8 columns of four rows at a time: 4 bytes of codes, one scale.
template <bool NV, bool WIDE>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const __grid_constant__ DequantK k, int log2_across) {
  after_previous_kernel();
  const float g = NV && k.g ? *(volatile const float*)k.g : 1.0f;
  const Extent e{k.rows, k.cols};
  const int across = 1 << log2_across, down = kThreads >> log2_across;
  const int64_t col = ((int64_t)blockIdx.x * across + (threadIdx.x & (across - 1))) * 8;
  if (col >= k.cols) return;
  const int valid = k.cols - col < 8 ? (int)(k.cols - col) : 8;
  const int64_t block = col / (NV ? 16 : 32), per_tile = k.q.scale_tiles * kScaleTile;
  const unsigned char* scales = k.q.scales + block / 4 * kScaleTile + block % 4;
  const int64_t step = (int64_t)gridDim.y * down;
  Down<WIDE> y(k.y, (int64_t)blockIdx.y * down + (threadIdx.x >> log2_across), step, col, valid);
  const unsigned char* from = k.q.codes + y.row * k.q.ld + col / 2;
  const int64_t down_bytes = step * k.q.ld;
  for (; y.row < k.rows; y.on(4), from += 4 * down_bytes) {
    uint32_t codes[4], scale[4];
    int64_t row = y.row;
    const unsigned char* at = from;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // past the last row the one before again
      const uint32_t low = (uint32_t)row;
      const int64_t s = (row >> 7) * per_tile + ((low & 31) << 4 | (low >> 3 & 12));
      codes[i] = scale[i] = 0;
      if (in_extent(row, row + 1, 0, k.rows, ZERO_SITE_FP4) &&
          in_extent(col / 2, col / 2 + 4, 0, k.q.line_bytes, ZERO_SITE_FP4) &&
          in_extent(s, s + 1, 0, k.q.scale_bytes, ZERO_SITE_FP4)) {
        codes[i] = *reinterpret_cast<const uint32_t*>(at);
        scale[i] = scales[s];
      }
      const bool more = row + step < k.rows;
      row += more ? step : 0;
      at += more ? down_bytes : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
      from_codes8(codes[i], v);
      const float d = scale_value<NV>(scale[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], d);
      if (y.row + i * step < k.rows) y.put(i, v, e);
    }
  }
}

template <bool NV>
static cudaError_t launch_dequantize_as(const DequantK& k, cudaStream_t st) {
  const Walk w = walk_over(k.rows, k.cols);
  return k.y.dtype == ZERO_F32
             ? launch_next(dequantize_kernel<NV, true>, w.grid, dim3(kThreads), st, k,
                           w.log2_across)
             : launch_next(dequantize_kernel<NV, false>, w.grid, dim3(kThreads), st, k,
                           w.log2_across);
}
cudaError_t launch_dequantize(const DequantK& k, cudaStream_t st) {
  if (k.rows == 0 || k.cols == 0) return cudaSuccess;
  return k.nv ? launch_dequantize_as<true>(k, st) : launch_dequantize_as<false>(k, st);
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
      Down<WIDE> x(k.x, (int64_t)blockIdx.y * down + (threadIdx.x >> log2_across), step, col,
                   valid);
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
  if (threadIdx.x == 0) *g = top > 0.0f ? __fdiv_rn(top, 2688.0f) : 1.0f;
}

cudaError_t launch_tensor_scale(const MaxK& k, float* g, cudaStream_t st) {
  int n = 0;
  if (k.rows > 0 && k.cols > 0) {
    Walk w = walk_over(k.rows, k.cols);
    if (w.grid.x > kMaxima) w.grid.x = kMaxima;
    if (w.grid.x * w.grid.y > kMaxima) w.grid.y = kMaxima / w.grid.x;
    n = (int)(w.grid.x * w.grid.y);
    cudaError_t e = launch_next(k.x.dtype == ZERO_F32 ? maxima_kernel<true> : maxima_kernel<false>,
                                w.grid, dim3(kThreads), st, k, w.log2_across);
    if (e != cudaSuccess) return e;
  }
  return launch_next(maximum_kernel, dim3(1), dim3(kMaxima), st, k.maxima, n, g);
}

cudaError_t launch_fp4_product(const ProductK& k, int mode, cudaStream_t st) {
  if (k.rows <= 0 || k.cols <= 0) return cudaSuccess;
  if (k.rows <= kFewRows) return launch_fp4_rows(k, mode, st);
  return mode == LIN_FORWARD ? launch_mode<LIN_FORWARD, OF_FP4>(k, st)
                             : launch_mode<LIN_DINPUT, OF_FP4>(k, st);
}

cudaError_t timeouts_fp4(unsigned long long* out, bool reset) { return unit_timeouts(out, reset); }
cudaError_t bounds_fp4(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
