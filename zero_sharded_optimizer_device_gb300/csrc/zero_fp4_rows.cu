// Products of few rows of 4-bit operands, tokens being generated: D[i][j] = sum
// over c of A(i, c) B(j, c) for up to 8 rows i of A, and what follows them (see
// zero_fp4_linear and zero_fp4_linear_dinput, include/zero.h).
//
// The weight's codes are read once and the rest is small: bound by memory and
// by how soon and widely its loads start.  A warp takes the four outputs whose
// scales lie in one 16-byte word (32 rows apart in a scale tile) and 1024 codes
// of each at a time, a lane 32.  Codes become twice their value in 8 bits by
// byte permutations (a table of eight bytes and its negative), and four
// products are one dp4a: a block's sum is exact in 32 bits.  It is scaled and
// added in fp32; lanes and warps join in a fixed order.
#include "zero_fp4.cuh"

namespace zk {

constexpr int kFewWarps = 8, kFewOutputs = 4;

// Eight codes as twice their values, a byte each, in the codes' order.
__device__ __forceinline__ void doubled8(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  const uint32_t mag = codes & 0x77777777u, sign = (codes >> 3) & 0x11111111u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t at = mag >> (16 * h), neg = __byte_perm(0x0000FF00u, 0, sign >> (16 * h));
    const uint32_t a = __byte_perm(0x03020100u, 0x0C080604u, at);
    const uint32_t b = __byte_perm(0xFDFEFF00u, 0xF4F8FAFCu, at);
    (h ? hi : lo) = (a & ~neg) | (b & neg);
  }
}
__device__ __forceinline__ void doubled32(const uint4& codes, uint32_t v[8]) {
  doubled8(codes.x, v[0], v[1]);
  doubled8(codes.y, v[2], v[3]);
  doubled8(codes.z, v[4], v[5]);
  doubled8(codes.w, v[6], v[7]);
}

// 32 codes of each of a warp's outputs, and the word with their scales.
struct FewWeights {
  uint4 codes[kFewOutputs], scales;
};

template <int MODE, int M, bool NV>
__global__ void __launch_bounds__(kFewWarps * 32, M <= 2 ? 2 : 1)
    fp4_rows_kernel(const __grid_constant__ ProductK k, int share) {
  __shared__ float red[kFewWarps][M * kFewOutputs];
  after_previous_kernel();
  constexpr int kIn = ZERO_SITE_LINEAR_IN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % share, groups = kFewWarps / share;
  const int64_t group = (int64_t)blockIdx.x * groups + warp / share;
  const int64_t tile = group >> 5, r = group & 31, j0 = tile * 128 + r;  // outputs j0 + 32 q
  const int64_t rows = k.rows, cols = k.cols, bytes = 2 * k.depth;
  const int64_t ldw = 2 * k.b.ld, ldx = 2 * k.a.ld, tiles = k.scale_tiles;
  const unsigned char* w = static_cast<const unsigned char*>(k.b.p);
  const unsigned char* x = static_cast<const unsigned char*>(k.a.p);
  const unsigned char* ws = static_cast<const unsigned char*>(k.scales_b);
  const unsigned char* xs = static_cast<const unsigned char*>(k.scales_a);
  const int64_t w_scales = (cols + 127) / 128 * tiles * kScaleTile;
  const int64_t x_scales = (rows + 127) / 128 * tiles * kScaleTile;
  const uint64_t offset = MODE == LIN_FORWARD && k.epi.drop.on ? drop_offset(k.epi.drop) : 0;

  // (outputs past the last read the first one's codes again)
  auto load = [&](FewWeights& f, int64_t c) {
#pragma unroll
    for (int q = 0; q < kFewOutputs; ++q) {
      const int64_t j = j0 + 32 * q < cols ? j0 + 32 * q : j0;
      f.codes[q] = make_uint4(0, 0, 0, 0);
      if (in_extent(c, c + 16, 0, bytes, kIn) && in_extent(j, j + 1, 0, cols, kIn))
        f.codes[q] = *reinterpret_cast<const uint4*>(w + j * ldw + c);
    }
    const int64_t block = c / (NV ? 8 : 16), at = (tile * tiles + block / 4) * kScaleTile + r * 16;
    f.scales = make_uint4(0, 0, 0, 0);
    if (in_extent(at, at + 16, 0, w_scales, kIn))
      f.scales = *reinterpret_cast<const uint4*>(ws + at);
  };
  float acc[M][kFewOutputs] = {};
  auto add = [&](const FewWeights& f, int64_t c) {
    const int64_t block = c / (NV ? 8 : 16);
    const int byte = (int)(block & 3) * 8;
    uint32_t xv[M][8];
    float xa[M], xb[M];  // the scales of a row's first and (NV) second 16 codes
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int64_t row = i < rows ? i : 0, at = block / 4 * kScaleTile + row * 16;
      uint4 codes = make_uint4(0, 0, 0, 0);
      uint32_t word = 0;
      if (in_extent(c, c + 16, 0, bytes, kIn) && in_extent(at, at + 4, 0, x_scales, kIn)) {
        codes = *reinterpret_cast<const uint4*>(x + row * ldx + c);
        word = *reinterpret_cast<const uint32_t*>(xs + at) >> byte;
      }
      doubled32(codes, xv[i]);
      xa[i] = scale_value<NV>(word & 0xFFu, 1.0f);
      xb[i] = NV ? scale_value<NV>((word >> 8) & 0xFFu, 1.0f) : 0.0f;
    }
    const uint32_t words[kFewOutputs] = {f.scales.x, f.scales.y, f.scales.z, f.scales.w};
#pragma unroll
    for (int q = 0; q < kFewOutputs; ++q) {
      uint32_t wv[8];
      doubled32(f.codes[q], wv);
      const uint32_t word = words[q] >> byte;
      const float wa = scale_value<NV>(word & 0xFFu, 1.0f);
      const float wb = NV ? scale_value<NV>((word >> 8) & 0xFFu, 1.0f) : 0.0f;
#pragma unroll
      for (int i = 0; i < M; ++i) {
        int a = 0, b = 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) a = __dp4a((int)wv[v], (int)xv[i][v], a);
#pragma unroll
        for (int v = 4; v < 8; ++v) {
          if (NV)
            b = __dp4a((int)wv[v], (int)xv[i][v], b);
          else
            a = __dp4a((int)wv[v], (int)xv[i][v], a);
        }
        acc[i][q] += (float)a * wa * xa[i];
        if (NV) acc[i][q] += (float)b * wb * xb[i];
      }
    }
  };
  if (j0 < cols) {
    constexpr int kAhead = 2;  // pieces whose weights are fetched together
    const int64_t step = (int64_t)share * 512;
    int64_t c = (int64_t)(part * 32 + lane) * 16;
    for (; c + (kAhead - 1) * step < bytes; c += kAhead * step) {
      FewWeights f[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load(f[u], c + u * step);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) add(f[u], c + u * step);
    }
    for (; c < bytes; c += step) {
      FewWeights f;
      load(f, c);
      add(f, c);
    }
  }
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int q = 0; q < kFewOutputs; ++q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[i][q] += __shfl_xor_sync(0xffffffffu, acc[i][q], o);
      if (lane == 0) red[warp][i * kFewOutputs + q] = acc[i][q];
    }
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= groups * M * kFewOutputs) return;
  const int which = t / (M * kFewOutputs), at = t % (M * kFewOutputs);
  float v = 0.0f;
  for (int s = 0; s < share; ++s) v += red[which * share + s][at];
  // (both operands' codes were doubled)
  v *= 0.25f;
  v *= (k.whole_a ? *(volatile const float*)k.whole_a : 1.0f) *
       (k.whole_b ? *(volatile const float*)k.whole_b : 1.0f);
  const int64_t mine = (int64_t)blockIdx.x * groups + which;
  const int64_t row = at / kFewOutputs;
  const int64_t col = (mine >> 5) * 128 + (mine & 31) + 32 * (at % kFewOutputs);
  if (row < rows && col < cols) finish1<MODE>(k.epi, row, col, v, Extent{rows, cols}, offset);
}

template <int MODE, int M>
static cudaError_t launch_few(const ProductK& k, cudaStream_t st) {
  // groups of four outputs; the last tile of 128 may lack the higher ones
  const int64_t whole = k.cols / 128 * 32, left = k.cols % 128;
  const int64_t groups = whole + (left < 32 ? left : 32);
  // warps share a contraction while they would not fill the GPU otherwise
  int share = 1;
  while (share < kFewWarps && groups * share < 16 * sm_count() &&
         2 * k.depth > (int64_t)share * 512)
    share *= 2;
  const int64_t per = kFewWarps / share;
  const dim3 grid((unsigned)((groups + per - 1) / per)), block(kFewWarps * 32);
  return k.blocks_of == 16
             ? launch_next(fp4_rows_kernel<MODE, M, true>, grid, block, st, k, share)
             : launch_next(fp4_rows_kernel<MODE, M, false>, grid, block, st, k, share);
}
template <int MODE>
static cudaError_t launch_few_mode(const ProductK& k, cudaStream_t st) {
  if (k.rows <= 1) return launch_few<MODE, 1>(k, st);
  if (k.rows <= 2) return launch_few<MODE, 2>(k, st);
  if (k.rows <= 4) return launch_few<MODE, 4>(k, st);
  return launch_few<MODE, 8>(k, st);
}

cudaError_t launch_fp4_rows(const ProductK& k, int mode, cudaStream_t st) {
  return mode == LIN_FORWARD ? launch_few_mode<LIN_FORWARD>(k, st)
                             : launch_few_mode<LIN_DINPUT>(k, st);
}

cudaError_t bounds_fp4_rows(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
