// Products of few rows, tokens being generated: D[i][j] = sum over c of A(i, c)
// B(j, c) for up to 8 rows i of A, and what follows them (see zero_linear and
// zero_linear_dinput, include/zero.h).
//
// The weight B is read once and the rest is small, so the kernels are bound by
// memory and, at sizes of one layer, by how soon and how widely its loads
// start: no tensor maps, no tensor memory, no cluster where the weight's lines
// run along the contraction.  Products and sums are fp32 on the CUDA cores, a
// sum being split over lanes, warps and (lines across the contraction) CTAs of
// a cluster and joined in a fixed order.
//   along:  a warp takes 4 outputs and 256 of the contraction at a time, its
//           lanes 8 each; the block's warps share the contraction or, where it
//           is short, the outputs
//   across: a block takes 32 outputs, 8 a lane, and 64 of the contraction at a
//           time; rows of A wait in shared memory
// Lines off 16-byte boundaries are read a value a lane, 32 in a row.
// One row (4096 outputs of 4096, bf16 weights): along 5.3 us, 6.3 TB/s; across
// 9.8; in tiles on the tensor cores 12.5.  A lane's loads of several steps are
// issued together and without conditions between them: across 4096 x 11008 one
// by one took 50 us, so 24.
#include "zero_ops_device.cuh"

namespace zk {

constexpr int kIn = ZERO_SITE_LINEAR_IN, kOut = ZERO_SITE_LINEAR_OUT;
constexpr int kWarps = 8, kOutputs = 4, kAcross = 32;

// What follows the product at one element.
template <int MODE>
__device__ __forceinline__ void finish1(const EpiK& k, int64_t row, int64_t col, float v,
                                        const Extent& e, uint64_t offset) {
  auto in = [&](const Mat& m) {
    const int64_t at = row * m.ld;
    return in_extent(at + col, at + col + 1, at, at + e.cols, kOut) &&
           in_extent(row, row + 1, 0, e.rows, kOut);
  };
  auto get = [&](const Mat& m) { return in(m) ? load1(m, row * m.ld + col) : 0.0f; };
  auto put = [&](const Mat& m, float x) {
    if (in(m)) store1(m, row * m.ld + col, x);
  };
  if constexpr (MODE == LIN_FORWARD) {
    const float residual = k.residual.p ? get(k.residual) : 0.0f;
    const float gate = k.gate.p ? get(k.gate) : 1.0f;
    if (k.bias.p && in_extent(col, col + 1, 0, e.cols, kIn)) v += load1(k.bias, col);
    if (k.pre.p) put(k.pre, v);
    float z[1] = {v};
    activate<1>(z, k.act);
    v = z[0];
    if (k.gate.p) v *= gate;
    if (k.drop.on) {
      const uint4 w = philox(make_uint4((uint32_t)(col >> 2), (uint32_t)row, (uint32_t)offset,
                                        (uint32_t)(offset >> 32)),
                             k.drop);
      const uint32_t word = col & 2 ? (col & 1 ? w.w : w.z) : (col & 1 ? w.y : w.x);
      v = word >= k.drop.least && !k.drop.all ? v * k.drop.scale : 0.0f;
    }
    if (k.residual.p) v += residual;
  } else {
    if (k.pre.p) {
      float value[1] = {get(k.pre)}, slope[1];
      activate_grad<1>(value, slope, k.act);
      if (k.gate.p) {
        if (k.dgate.p) put(k.dgate, value[0] * v);
        slope[0] *= get(k.gate);
      }
      v *= slope[0];
    }
  }
  put(k.out, v);
}

// V = 8 or 1 consecutive values of a line as they lie in memory.
template <int V>
struct Word;
template <>
struct Word<8> {
  uint4 u;
};
template <>
struct Word<1> {
  uint16_t u;
};
template <int V>
__device__ __forceinline__ Word<V> word_at(const Mat& m, int64_t line, int64_t at, int64_t lines,
                                           int64_t length) {
  Word<V> w{};
  if (!in_extent(at, at + V, 0, length, kIn) || !in_extent(line, line + 1, 0, lines, kIn)) return w;
  const uint16_t* p = static_cast<const uint16_t*>(m.p) + line * m.ld + at;
  if constexpr (V == 8)
    w.u = *reinterpret_cast<const uint4*>(p);
  else
    w.u = *p;
  return w;
}
__device__ __forceinline__ float value_of(const Word<1>& w) {
  return __uint_as_float((uint32_t)w.u << 16);
}

// Two fp32 products and sums in one instruction, each rounded as an fmaf.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ void fma2(uint64_t& sum, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(a), "l"(b));
}
__device__ __forceinline__ float2 halves(uint64_t p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ void pairs_of(const Word<8>& w, uint64_t p[4]) {
  p[0] = pair(bf16_lo(w.u.x), bf16_hi(w.u.x));
  p[1] = pair(bf16_lo(w.u.y), bf16_hi(w.u.y));
  p[2] = pair(bf16_lo(w.u.z), bf16_hi(w.u.z));
  p[3] = pair(bf16_lo(w.u.w), bf16_hi(w.u.w));
}

template <int MODE, int M, int VEC>
__global__ void __launch_bounds__(kWarps * 32, 2)
    along_kernel(const __grid_constant__ ProductK k, int share) {
  __shared__ float red[kWarps][M * kOutputs];
  after_previous_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % share, groups = kWarps / share;
  const int64_t j0 = ((int64_t)blockIdx.x * groups + warp / share) * kOutputs;
  const int64_t rows = k.rows, cols = k.cols, depth = k.depth;
  const uint64_t offset = MODE == LIN_FORWARD && k.epi.drop.on ? drop_offset(k.epi.drop) : 0;
  // past the outputs and rows, the last one again
  auto load = [&](auto& w, int64_t c) {
#pragma unroll
    for (int q = 0; q < kOutputs; ++q)
      w[q] = word_at<sizeof(w[0]) / 2>(k.b, j0 + q < cols ? j0 + q : cols - 1, c, cols, depth);
  };
  float acc[M][kOutputs] = {};
  uint64_t both[M][kOutputs] = {};  // sums of even and of odd contraction indexes
  auto add = [&](const auto& w, int64_t c) {
    constexpr int V = sizeof(w[0]) / 2;
    uint64_t wp[kOutputs][4];
    if constexpr (V == 8)
#pragma unroll
      for (int q = 0; q < kOutputs; ++q) pairs_of(w[q], wp[q]);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const Word<V> x = word_at<V>(k.a, i < rows ? i : rows - 1, c, rows, depth);
      if constexpr (V == 8) {
        uint64_t xp[4];
        pairs_of(x, xp);
#pragma unroll
        for (int q = 0; q < kOutputs; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) fma2(both[i][q], xp[v], wp[q][v]);
      } else {
#pragma unroll
        for (int q = 0; q < kOutputs; ++q) acc[i][q] += value_of(x) * value_of(w[q]);
      }
    }
  };
  if (j0 < cols) {
    constexpr int kAhead = VEC == 8 ? 2 : 4;  // steps whose weights are fetched together
    const int64_t step = (int64_t)share * 32 * VEC;
    int64_t c = (part * 32 + lane) * VEC;
    for (; c + (kAhead - 1) * step + VEC <= depth; c += kAhead * step) {
      Word<VEC> w[kAhead][kOutputs];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load(w[u], c + u * step);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) add(w[u], c + u * step);
    }
    for (; c + VEC <= depth; c += step) {
      Word<VEC> w[kOutputs];
      load(w, c);
      add(w, c);
    }
    if (VEC == 8 && part == 0 && lane < (int)(depth & 7)) {
      Word<1> w[kOutputs];
      load(w, (depth & ~7ll) + lane);
      add(w, (depth & ~7ll) + lane);
    }
  }
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int q = 0; q < kOutputs; ++q) {
      const float2 f = halves(both[i][q]);
      acc[i][q] += f.x + f.y;
    }
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int q = 0; q < kOutputs; ++q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[i][q] += __shfl_xor_sync(0xffffffffu, acc[i][q], o);
      if (lane == 0) red[warp][i * kOutputs + q] = acc[i][q];
    }
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= groups * M * kOutputs) return;
  const int group = t / (M * kOutputs), at = t % (M * kOutputs);
  float v = 0.0f;
  for (int p = 0; p < share; ++p) v += red[group * share + p][at];
  const int64_t row = at / kOutputs;
  const int64_t col = ((int64_t)blockIdx.x * groups + group) * kOutputs + at % kOutputs;
  if (row < rows && col < cols) finish1<MODE>(k.epi, row, col, v, Extent{rows, cols}, offset);
}

// The CTAs of a cluster of `parts` share the contraction of their 32 outputs.
template <int MODE, int M, int VEC, int W>
__global__ void __launch_bounds__(W * 32, W == kWarps ? 2 : 1)
    across_kernel(const __grid_constant__ ProductK k, int parts) {
  constexpr int kLanes = kAcross / VEC, kLines = 32 / kLanes;  // of a warp
  constexpr int kDepth = M < 4 ? 1024 : 512, kAhead = VEC == 8 ? 4 : 16;
  __shared__ __align__(16) uint64_t xs[kDepth][M];  // each value twice
  __shared__ float red[W][M * kAcross], sum[M * kAcross];
  after_previous_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (int)(blockIdx.x % parts);
  const int64_t j0 = (int64_t)(blockIdx.x / parts) * kAcross;
  const int64_t rows = k.rows, cols = k.cols, depth = k.depth;
  const int64_t first = depth * part / parts, last = depth * (part + 1) / parts;
  const uint64_t offset = MODE == LIN_FORWARD && k.epi.drop.on ? drop_offset(k.epi.drop) : 0;
  const int64_t col = j0 + (lane % kLanes) * VEC;
  const bool whole = col + VEC <= cols;
  constexpr int kPairs = VEC == 8 ? 4 : 1;
  uint64_t both[M][kPairs] = {};
  auto ragged = [&](int64_t line) {  // the lane in which the outputs end
    uint32_t e[8];
#pragma unroll
    for (int v = 0; v < 8; ++v)
      e[v] = col + v < cols ? word_at<1>(k.b, line, col + v, depth, cols).u : 0;
    Word<8> w;
    w.u = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    return w;
  };
  auto add = [&](const Word<VEC>& w, int r) {
    uint64_t wp[kPairs];
    if constexpr (VEC == 8)
      pairs_of(w, wp);
    else
      wp[0] = pair(value_of(w), 0.0f);
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int v = 0; v < kPairs; ++v) fma2(both[i][v], xs[r][i], wp[v]);
  };
  for (int64_t base = first; base < last; base += kDepth) {
    const int n = (int)(last - base < kDepth ? last - base : kDepth);
    constexpr int kStep = W * kLines;
    int r = warp * kLines + lane / kLanes;
    // the first batch of weights is on its way while A's rows are
    const bool ahead = VEC == 8 && whole && r + (kAhead - 1) * kStep < n;
    Word<VEC> w0[kAhead];
    if (ahead)
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        w0[u] = word_at<VEC>(k.b, base + r + u * kStep, col, depth, cols);
    if (base > first) __syncthreads();
    for (int r = threadIdx.x; r < n; r += W * 32)
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const float x =
            value_of(word_at<1>(k.a, i < rows ? i : rows - 1, base + r, rows, depth));
        xs[r][i] = pair(x, x);
      }
    __syncthreads();
    if (ahead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) add(w0[u], r + u * kStep);
      r += kAhead * kStep;
    }
    if (whole) {  // (no condition around a load: a batch is in flight at once)
      for (; r + (kAhead - 1) * kStep < n; r += kAhead * kStep) {
        Word<VEC> w[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          w[u] = word_at<VEC>(k.b, base + r + u * kStep, col, depth, cols);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) add(w[u], r + u * kStep);
      }
      for (; r < n; r += kStep) add(word_at<VEC>(k.b, base + r, col, depth, cols), r);
    } else if (VEC == 8 && col < cols) {
      if constexpr (VEC == 8)
        for (; r < n; r += kStep) add(ragged(base + r), r);
    }
  }
  float acc[M][VEC];
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int v = 0; v < VEC; v += 2) {
      const float2 f = halves(both[i][v / 2]);
      acc[i][v] = f.x;
      if constexpr (VEC == 8) acc[i][v + 1] = f.y;
    }
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) acc[i][v] += __shfl_xor_sync(0xffffffffu, acc[i][v], o);
      if (lane < kLanes) red[warp][i * kAcross + lane * VEC + v] = acc[i][v];
    }
  __syncthreads();
  const int t = threadIdx.x;
  float v = 0.0f;
  if (t < M * kAcross) {
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[w][t];
    sum[t] = v;
  }
  if (parts > 1) {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    if (part == 0 && t < M * kAcross)
      for (int p = 1; p < parts; ++p) {
        uint32_t there;
        float other;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(there)
                     : "r"((uint32_t)__cvta_generic_to_shared(sum + t)), "r"(p));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other) : "r"(there) : "memory");
        v += other;
      }
    // nobody leaves while its sums are read
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
  }
  const int64_t row = t / kAcross, at = j0 + t % kAcross;
  if (part == 0 && t < M * kAcross && row < rows && at < cols)
    finish1<MODE>(k.epi, row, at, v, Extent{rows, cols}, offset);
}

template <int MODE, int M, int VEC>
static cudaError_t launch_vec(const ProductK& k, cudaStream_t st) {
  if (k.b_c) {
    // warps share a contraction while they would not fill the GPU otherwise and
    // each keeps 256 of it (32 by single values)
    const int64_t groups = (k.cols + kOutputs - 1) / kOutputs;
    int share = 1;
    while (share < kWarps && groups * share < 24 * sm_count() &&
           k.depth > (int64_t)share * 32 * VEC)
      share *= 2;
    const int64_t per = kWarps / share * kOutputs;
    return launch_next(along_kernel<MODE, M, VEC>, dim3((unsigned)((k.cols + per - 1) / per)),
                       dim3(kWarps * 32), st, k, share);
  }
  const int64_t blocks = (k.cols + kAcross - 1) / kAcross;
  // one row: 32 warps instead of a cluster while one CTA's share of loads is
  // small.  (us with 32 warps / in clusters: 4096 outputs of 520 to 1016 3.6 to
  // 3.9 / 6.7 to 7.2, of 1024 3.9 / 6.4; 1024 outputs of 520 to 1024 3.5 to 3.8 /
  // 3.8 to 4.0; 264 outputs of 520 to 1024 3.6 to 3.9 / 3.6 to 3.8.  Past 1024
  // A's row takes shared memory twice: 768 outputs of 1536 4.9 / 4.2.)
  constexpr int kMany = M == 1 && VEC == 8 ? 32 : kWarps;
  const bool many =
      kMany > kWarps && k.depth > 512 && k.depth <= 1024 && blocks <= sm_count();
  int parts = 1;
  while (!many && parts < 8 && blocks * parts < 3 * sm_count() &&
         k.depth >= (int64_t)parts * 256)
    parts *= 2;
  const auto kernel =
      many ? across_kernel<MODE, M, VEC, kMany> : across_kernel<MODE, M, VEC, kWarps>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * parts));
  cfg.blockDim = dim3((many ? kMany : kWarps) * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, k, parts);
}
template <int MODE, int M>
static cudaError_t launch_few(const ProductK& k, cudaStream_t st) {
  const bool vec = k.b.vec && (!k.b_c || k.a.vec || (k.rows == 1 && ((uintptr_t)k.a.p & 15) == 0));
  return vec ? launch_vec<MODE, M, 8>(k, st) : launch_vec<MODE, M, 1>(k, st);
}
template <int MODE>
static cudaError_t launch_mode(const ProductK& k, cudaStream_t st) {
  if (k.rows <= 1) return launch_few<MODE, 1>(k, st);
  if (k.rows <= 2) return launch_few<MODE, 2>(k, st);
  if (k.rows <= 4) return launch_few<MODE, 4>(k, st);
  return launch_few<MODE, 8>(k, st);
}

cudaError_t launch_rows(const ProductK& k, int mode, cudaStream_t st) {
  return mode == LIN_FORWARD ? launch_mode<LIN_FORWARD>(k, st) : launch_mode<LIN_DINPUT>(k, st);
}

cudaError_t bounds_rows(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
