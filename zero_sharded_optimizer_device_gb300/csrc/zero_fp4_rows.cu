// Products of few rows of 4-bit operands, tokens being generated: D[i][j] = sum
// over c of A(i, c) B(j, c) for up to 8 rows i of A, and what follows them (see
// zero_fp4_linear and zero_fp4_linear_dinput, include/zero.h).
//
// The weight is read once and the rest is small: bound by memory and by how soon
// and widely its loads start.  A warp takes 16 of its rows by 256 codes at a
// time, copied to shared memory three pieces ahead, and has the eight tokens'
// codes of the same 256 in registers: mma.sync m16n8k16 on fp16 has just this
// shape (tcgen05's least tile is 64 rows, through descriptors and barriers that
// cost more than such a product).  Which of a block's codes stand at which place
// of the instruction is free as long as both operands agree, so that a lane
// reads 8 codes in a row of each.
//   NV  a code times its scale is exact in fp16 (2 + 4 bits, 2^-10 to 2688), so
//       both operands are scaled before the product.
//   MX  a block's product is exact in fp32, a multiple of 1/4 up to 1152, and so is
//       that times the smaller of its two scales; then it is scaled by the larger
//       and added.  Which comes first matters only where the weight's scale alone
//       takes a product out of fp32's range: a warp applies that first and, where
//       an infinity or NaN comes out, sums once more in order.  (4096 x 4096, 1
//       token 5.0 us, 4.9 without any of it, 5.3 with both scales compared at every product,
//       and 256 x 16384 7.2, 7.2 and 8.1; 7.7 with large scales looked for beforehand.)
// The eight warps of a block split the contraction and are joined in order.
// Bound by latencies: at 4096 codes a warp has two pieces for a ring that runs three
// ahead, and a large weight's blocks take turns, two an SM, each with the way of its
// first bytes, a join and a start; 39 % of the issue slots are used, 4 instructions a
// code (of 32 lanes).  4096 x 4096 (9.4 MB) 5.4 us for 1 token and 5.9 for 8 (NV), 1024 x
// 1024 2.4, of which 2 are the launch and the first bytes' way.  (With dp4a on codes as bytes and the
// tokens decoded for every four outputs 6.8 and 19.5 us; two groups of 16 outputs
// a warp, which halve the tokens' decoding but leave the SMs 8 warps, 7.8; the
// tokens' codes in shared memory 5.6 and 6.9.)
#include <atomic>

#include "zero_fp4.cuh"

namespace zk {

constexpr int kFewWarps = 8, kFewLines = 16, kFewDeep = 128;  // bytes of a line in a piece
constexpr int kFewPitch = kFewDeep + 16;
constexpr int kFewScales = 256;  // 4 tiles' (NV; MX: 2) 16 lines of 4 blocks
constexpr int kFewStage = kFewLines * kFewPitch + kFewScales, kFewStages = 4;
constexpr int kFewSmem = kFewWarps * kFewStages * kFewStage;

// 16 bytes from memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(some ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint32_t lds4(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
// Eight codes as fp16 pairs.
__device__ __forceinline__ void pairs8(uint32_t codes, uint32_t h[4]) {
  asm("{ .reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}
__device__ __forceinline__ void times8(uint32_t h[4], uint32_t by) {
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(by));
}
// A word of NV scales: of its two pairs of 16 codes, this lane's (t / 2) in each,
// as fp16 twice.
__device__ __forceinline__ void nv_scales(uint32_t word, int t, uint32_t s[2]) {
  const uint32_t two = __byte_perm(word, 0, t >> 1 ? 0x31 : 0x20);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  s[0] = __byte_perm(h, 0, 0x1010);
  s[1] = __byte_perm(h, 0, 0x3232);
}
// A word of MX scales.
__device__ __forceinline__ void mx_scales(uint32_t word, float s[4]) {
  uint32_t lo, hi;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)word));
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(word >> 16)));
  s[0] = bf16_lo(lo);
  s[1] = bf16_hi(lo);
  s[2] = bf16_lo(hi);
  s[3] = bf16_hi(hi);
}
__device__ __forceinline__ void mma16(float d[4], const uint32_t lo[2], const uint32_t hi[2],
                                      const uint32_t b[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(lo[0]), "r"(hi[0]), "r"(lo[1]), "r"(hi[1]), "r"(b[0]), "r"(b[1]));
}

// Outputs of a group: 16 that lie 32 apart four at a time, whose scales are 64
// bytes of a scale tile.
__device__ __forceinline__ int64_t few_output(int64_t group, int line) {
  return (group >> 3) * 128 + (group & 7) * 4 + (line & 3) + (line >> 2) * 32;
}

// MX: this warp's sums with the smaller scale of two applied first, straight from
// memory.
static __device__ __noinline__ float4 mx_sum_ordered(const ProductK& k, int64_t group) {
  constexpr int kIn = ZERO_SITE_LINEAR_IN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t rows = k.rows, cols = k.cols, bytes = 2 * k.depth, tiles = k.scale_tiles;
  auto codes = [&](const Mat& m, int64_t lines, int64_t line, int64_t block) {
    const int64_t at = line * 2 * m.ld + block * 16 + 4 * t;
    if (line >= lines || !in_extent(at, at + 4, 0, (lines - 1) * 2 * m.ld + bytes, kIn)) return 0u;
    return *reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(m.p) + at);
  };
  auto scale = [&](const void* s, int64_t lines, int64_t line, int64_t block) {
    const int64_t at = (line / 128 * tiles + block / 4) * kScaleTile + line % 32 * 16 +
                       line % 128 / 32 * 4 + block % 4;
    if (line >= lines || !in_extent(at, at + 1, 0, (lines + 127) / 128 * tiles * kScaleTile, kIn))
      return 0.0f;
    return scale_value<false>(static_cast<const unsigned char*>(s)[at], 1.0f);
  };
  const int64_t line[2] = {few_output(group, g), few_output(group, g + 8)};
  float acc[4] = {};
  for (int64_t chunk = warp; chunk * kFewDeep < bytes; chunk += kFewWarps)
    for (int64_t block = chunk * 8; block < chunk * 8 + 8 && block * 16 < bytes; ++block) {
      uint32_t lo[4], hi[4], b[4];
      pairs8(codes(k.b, cols, line[0], block), lo);
      pairs8(codes(k.b, cols, line[1], block), hi);
      pairs8(codes(k.a, rows, g, block), b);
      float d[4] = {};
      mma16(d, lo, hi, b);
      mma16(d, lo + 2, hi + 2, b + 2);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float sw = scale(k.scales_b, cols, line[q >> 1], block);
        const float sx = scale(k.scales_a, rows, 2 * t + (q & 1), block);
        float least, most;  // NaN stays NaN
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(least) : "f"(sw), "f"(sx));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(most) : "f"(sw), "f"(sx));
        acc[q] += d[q] * least * most;
      }
    }
  return make_float4(acc[0], acc[1], acc[2], acc[3]);
}

template <int MODE, bool NV>
__global__ void __launch_bounds__(kFewWarps * 32, 2)
    fp4_rows_kernel(const __grid_constant__ ProductK k) {
  extern __shared__ __align__(16) unsigned char few_smem[];
  __shared__ float red[kFewWarps][kFewLines][kFewRows];
  constexpr int kIn = ZERO_SITE_LINEAR_IN;
  constexpr int kTiles = NV ? 4 : 2;  // scale tiles of a piece
  after_previous_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t group = blockIdx.x;
  const int64_t rows = k.rows, cols = k.cols, bytes = 2 * k.depth;
  const int64_t ldw = 2 * k.b.ld, ldx = 2 * k.a.ld, tiles = k.scale_tiles;
  const unsigned char* w = static_cast<const unsigned char*>(k.b.p);
  const unsigned char* x = static_cast<const unsigned char*>(k.a.p);
  const unsigned char* ws = static_cast<const unsigned char*>(k.scales_b);
  const unsigned char* xs = static_cast<const unsigned char*>(k.scales_a);
  const int64_t w_scales = (cols + 127) / 128 * tiles * kScaleTile;
  const int64_t x_scales = (rows + 127) / 128 * tiles * kScaleTile;
  const uint64_t offset = MODE == LIN_FORWARD && k.epi.drop.on ? drop_offset(k.epi.drop) : 0;
  const uint32_t ring =
      (uint32_t)__cvta_generic_to_shared(few_smem) + warp * (kFewStages * kFewStage);

  // Every eighth chunk of 256 codes is this warp's.
  const int chunks = (int)((bytes + kFewDeep - 1) / kFewDeep);
  const int mine = warp < chunks ? (chunks - warp + kFewWarps - 1) / kFewWarps : 0;
  // What this lane copies of each: of one of four lines 16 bytes (their next, how
  // many of the lines there are and how many of the chunks have them), and of
  // the scales another 16.
  auto left_of = [](int64_t n, int64_t step) {
    return n > 0 ? (int)((n + step - 1) / step) : 0;
  };
  const int unit = lane & 7;
  const int with_codes = left_of(bytes - warp * kFewDeep - unit * 16, kFewWarps * kFewDeep);
  const int with_scales =
      lane < 4 * kTiles ? left_of(tiles - warp * kTiles - (lane >> 2), kFewWarps * kTiles) : 0;
  const int64_t first = few_output(group, lane >> 3);
  const int lines = min(4, left_of(cols - first, 32));
  const unsigned char* codes_at = w + first * ldw + warp * kFewDeep + unit * 16;
  const int64_t tile0 = (group >> 3) * tiles + warp * kTiles + (lane >> 2);
  const unsigned char* scales_at =
      ws + tile0 * kScaleTile + (group & 7) * 64 + (lane & 3) * 16;
  auto issue = [&](int i) {  // in order
    const uint32_t to = ring + i % kFewStages * kFewStage;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const unsigned char* from = codes_at + u * 32 * ldw;
      const bool some = u < lines && i < with_codes &&
                        in_extent(from - w, from - w + 16, 0, (cols - 1) * ldw + bytes, kIn);
      copy16(to + (4 * u + (lane >> 3)) * kFewPitch + unit * 16, some ? from : w, some);
    }
    if (lane < 4 * kTiles) {
      const bool some = i < with_scales &&
                        in_extent(scales_at - ws, scales_at - ws + 16, 0, w_scales, kIn);
      copy16(to + kFewLines * kFewPitch + lane * 16, some ? scales_at : ws, some);
    }
    codes_at += kFewWarps * kFewDeep;
    scales_at += kFewWarps * kTiles * kScaleTile;
  };
  // The tokens' codes of the next chunk, token g's, and its scales: NV token
  // g's, MX those of tokens 2 t and 2 t + 1.
  uint32_t next_codes[8], next_scales[4];
  int64_t x_chunk = warp;
  auto fetch = [&]() {
    const unsigned char* from = x + g * ldx + x_chunk * kFewDeep + 4 * t;
    const int some = g < rows ? (int)min((int64_t)8, (bytes - x_chunk * kFewDeep) / 16) : 0;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      next_codes[s] = 0;
      if (s < some && in_extent(from - x, from - x + s * 16 + 4, 0, (rows - 1) * ldx + bytes, kIn))
        next_codes[s] = *reinterpret_cast<const uint32_t*>(from + s * 16);
    }
    const int64_t at = x_chunk * kTiles * kScaleTile + (NV ? g : 2 * t) * 16;
    const int left = (int)min((int64_t)4, tiles - x_chunk * kTiles);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int token = NV ? g : 2 * t + (q & 1), tile = NV ? q : q >> 1;
      const int64_t of = at + tile * kScaleTile + (NV ? 0 : (q & 1) * 16);
      next_scales[q] = 0;
      if (tile < left && token < rows && in_extent(of, of + 4, 0, x_scales, kIn))
        next_scales[q] = *reinterpret_cast<const uint32_t*>(xs + of);
    }
    x_chunk += kFewWarps;
  };

  float acc[4] = {};
#pragma unroll
  for (int i = 0; i < kFewStages - 1; ++i) {
    if (i < mine) issue(i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  if (mine) fetch();
  for (int i = 0; i < mine; ++i) {
    uint32_t b[8][4];
    float sx[2][8];  // MX
#pragma unroll
    for (int s = 0; s < 8; ++s) pairs8(next_codes[s], b[s]);
    if (NV) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t by[2];
        nv_scales(next_scales[q], t, by);
        times8(b[2 * q], by[0]);
        times8(b[2 * q + 1], by[1]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) mx_scales(next_scales[q], sx[q & 1] + 4 * (q >> 1));
    }
    if (i + 1 < mine) fetch();
    asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 2) : "memory");
    __syncwarp();
    // (into the place of the chunk before this one, which every lane is done with)
    if (i + kFewStages - 1 < mine) issue(i + kFewStages - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const uint32_t at = ring + i % kFewStages * kFewStage;
    const uint32_t codes = at + g * kFewPitch + 4 * t;
    const uint32_t scales = at + kFewLines * kFewPitch + (g & 3) * 16 + (g >> 2) * 4;
    float sw[2][4];     // MX: lines g and g + 8, the blocks of a tile
    uint32_t by[2][2];  // NV
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (NV && s % 2 == 0) {
        nv_scales(lds4(scales + s / 2 * 64), t, by[0]);
        nv_scales(lds4(scales + s / 2 * 64 + 8), t, by[1]);
      }
      if (!NV && s % 4 == 0) {
        mx_scales(lds4(scales + s / 4 * 64), sw[0]);
        mx_scales(lds4(scales + s / 4 * 64 + 8), sw[1]);
      }
      uint32_t lo[4], hi[4];
      pairs8(lds4(codes + s * 16), lo);
      pairs8(lds4(codes + s * 16 + 8 * kFewPitch), hi);
      if (NV) {
        times8(lo, by[0][s & 1]);
        times8(hi, by[1][s & 1]);
        mma16(acc, lo, hi, b[s]);
        mma16(acc, lo + 2, hi + 2, b[s] + 2);
      } else {
        float d[4] = {};
        mma16(d, lo, hi, b[s]);
        mma16(d, lo + 2, hi + 2, b[s] + 2);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] += d[q] * sw[q >> 1][s & 3] * sx[q & 1][s];
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!NV) {
    bool lost = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) lost |= !(fabsf(acc[q]) < INFINITY);
    if (__any_sync(0xffffffffu, lost)) {
      const float4 v = mx_sum_ordered(k, group);
      acc[0] = v.x; acc[1] = v.y; acc[2] = v.z; acc[3] = v.w;
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) red[warp][g + 8 * (q >> 1)][2 * t + (q & 1)] = acc[q];
  __syncthreads();
  const int line = threadIdx.x % kFewLines, row = threadIdx.x / kFewLines;
  const int64_t col = few_output(group, line);
  if (row >= rows || col >= cols) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < kFewWarps; ++i) v += red[i][line][row];
  v *= (k.whole_a ? *(volatile const float*)k.whole_a : 1.0f) *
       (k.whole_b ? *(volatile const float*)k.whole_b : 1.0f);
  finish1<MODE>(k.epi, row, col, v, Extent{rows, cols}, offset);
}

template <int MODE, bool NV>
static cudaError_t launch_few(const ProductK& k, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(fp4_rows_kernel<MODE, NV>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  // groups of 16 outputs; the last tile of 128 may lack the higher ones
  const int64_t left = k.cols % 128, last = left < 32 ? (left + 3) / 4 : 8;
  const int64_t groups = k.cols / 128 * 8 + last;
  if (groups >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch_next_with(kFewSmem, fp4_rows_kernel<MODE, NV>, dim3((unsigned)groups),
                          dim3(kFewWarps * 32), st, k);
}

cudaError_t launch_fp4_rows(const ProductK& k, int mode, cudaStream_t st) {
  if (mode == LIN_FORWARD)
    return k.blocks_of == 16 ? launch_few<LIN_FORWARD, true>(k, st)
                             : launch_few<LIN_FORWARD, false>(k, st);
  return k.blocks_of == 16 ? launch_few<LIN_DINPUT, true>(k, st)
                           : launch_few<LIN_DINPUT, false>(k, st);
}

cudaError_t bounds_fp4_rows(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
