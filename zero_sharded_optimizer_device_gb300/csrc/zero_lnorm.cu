// Layer norm and RMS norm over the rows of a matrix, and their gradients.
//
// Both are bound by memory.  A row is read once into registers by the T
// threads that share it (8 or 16 columns each, one to 32 warps), its sums run
// over warp shuffles and one exchange through shared memory, and the result
// is written from the registers.  The launch is one wave of blocks walking
// the rows, and a row's loads are issued a row ahead, so that memory is busy
// while the sums wait for one another.  The variance is the mean of squared
// distances from the mean already found (two sweeps over registers), not a
// difference of moments, which loses the digits of rows whose mean is large.
#include "zero_ops_device.cuh"

namespace zk {

constexpr int kSite = ZERO_SITE_LNORM;
// Most blocks of the backward pass: 3 on each of this GPU's 152 SMs.  Fixed, so
// that a workspace's size depends on its matrix alone.
constexpr int64_t kNormPartials = 456;

int64_t norm_partials(int64_t m) { return m < kNormPartials ? m : kNormPartials; }

// Sum of v (N values) over the T threads sharing a row (group `group` of the
// block's); every one of them gets the sum.  red: two buffers of 32 N floats,
// used in turn, so that one barrier per sum is enough: nobody writes a buffer
// again before everyone has passed the barrier of the sum between.
template <int T, int N>
__device__ __forceinline__ void row_sum(float v[N], float* red, int& turn, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (T > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* buf = red + turn * 32 * N;
    turn ^= 1;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) buf[warp * N + i] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(T) : "memory");
    constexpr int W = T / 32;
    const int w0 = group * W;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // lane w holds warp w's part; a shuffle tree adds them in a fixed order
      float a = lane < W ? buf[(w0 + lane) * N + i] : 0.0f;
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      v[i] = __shfl_sync(0xffffffffu, a, 0);
    }
  }
}

__device__ __forceinline__ int valid_of(int64_t col, int64_t n) {
  return col >= n ? 0 : (n - col < 8 ? (int)(n - col) : 8);
}

// Rows off 16-byte boundaries: the 8 columns of a thread's vector lie S = T
// apart instead of side by side, so that each of its single loads and stores is
// one of consecutive columns over the T threads (8192 x 4097 RMS norm: 50 us,
// 154 with 8 columns side by side; 6760 x 2568 fp32 28 and 73).  Columns from `valid` on lie outside.
template <int S>
__device__ __forceinline__ int valid_columns(int64_t col, int64_t n) {
  if (S == 1) return valid_of(col, n);
  if (col >= n) return 0;
  const int64_t count = (n - col + S - 1) / S;
  return count < 8 ? (int)count : 8;
}
// Such a vector as its values lie in memory, 0 outside; whole ones without a
// condition per load.
template <int S, typename T>
__device__ __forceinline__ void singles(const T* p, int valid, uint32_t u[8]) {
  if (valid == 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = p[j * S];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = j < valid ? p[j * S] : 0;
  }
}
template <int S>
__device__ __forceinline__ void load_columns(const Mat& m, int64_t row, int64_t col, int valid,
                                             const Extent& e, uint32_t u[8]) {
  const int64_t i = row * m.ld + col;
  if (!valid || !in_extent(col, col + (valid - 1) * S + 1, 0, e.cols, kSite) ||
      !in_extent(row, row + 1, 0, e.rows, kSite)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = 0;
  } else if (m.dtype == ZERO_F32) {
    singles<S>(static_cast<const uint32_t*>(m.p) + i, valid, u);
  } else {
    singles<S>(static_cast<const uint16_t*>(m.p) + i, valid, u);
  }
}
template <int S, typename T>
__device__ __forceinline__ void put_singles(T* p, int valid, const T v[8]) {
  if (valid == 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j * S] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) p[j * S] = v[j];
  }
}
template <int S>
__device__ __forceinline__ void store_columns(const Mat& m, int64_t row, int64_t col, int valid,
                                              const float f[8], const Extent& e) {
  if constexpr (S == 1) {
    store8(m, row, col, valid, f, e, kSite);
  } else {
    const int64_t i = row * m.ld + col;
    if (!valid || !in_extent(col, col + (valid - 1) * S + 1, 0, e.cols, kSite) ||
        !in_extent(row, row + 1, 0, e.rows, kSite))
      return;
    if (m.dtype == ZERO_F32) {
      put_singles<S>(static_cast<float*>(m.p) + i, valid, f);
    } else {
      uint16_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = to_bf16(f[j]);
      put_singles<S>(static_cast<uint16_t*>(m.p) + i, valid, h);
    }
  }
}

// A row's vectors as they lie in memory, in registers: 4 of them per 8 bf16
// values, 8 per 8 fp32 ones (WIDE: the matrices may be either) or single ones.
template <bool WIDE, int S>
struct RowVec {
  uint32_t u[8];
  __device__ __forceinline__ void load(const Mat& m, int64_t row, int64_t col, int valid,
                                       const Extent& e) {
    load_columns<S>(m, row, col, valid, e, u);
  }
  __device__ __forceinline__ void get(const Mat& m, float f[8]) const {
    const int up = WIDE && m.dtype == ZERO_F32 ? 0 : 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(u[j] << up);
  }
};
template <>
struct RowVec<false, 1> {
  uint4 a;
  __device__ __forceinline__ void load(const Mat& m, int64_t row, int64_t col, int valid,
                                       const Extent& e) {
    a = raw8_bf16(m, row, col, valid, e, kSite);
  }
  __device__ __forceinline__ void get(const Mat&, float f[8]) const { from_bf16(a, f); }
};
template <>
struct RowVec<true, 1> {
  Raw8 r;
  __device__ __forceinline__ void load(const Mat& m, int64_t row, int64_t col, int valid,
                                       const Extent& e) {
    r = raw8(m, row, col, valid, e, kSite);
  }
  __device__ __forceinline__ void get(const Mat& m, float f[8]) const { from_raw(m, r, f); }
};

__device__ __forceinline__ uint4 param16(const void* p) {
  uint4 u;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}
// 8 parameters, kept in registers for all rows.  Coherent loads: a gather may
// write them while this kernel is already resident, waiting for it.  (Read
// again for every row, from L1, fp32 rows of 4096 take 75 us instead of 65.)
template <int S>
__device__ __forceinline__ void param8(const Mat& p, int64_t col, int valid, int64_t n,
                                       float f[8]) {
  if constexpr (S > 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t c = col + j * S;
      f[j] = j < valid && in_extent(c, c + 1, 0, n, kSite) ? load1(p, c) : 0.0f;
    }
    return;
  }
  if (!in_extent(col, col + valid, 0, n, kSite)) valid = 0;
  if (p.vec && valid == 8) {
    if (p.dtype == ZERO_F32) {
      const float* q = static_cast<const float*>(p.p) + col;
      Raw8 r;
      r.a = param16(q);
      r.b = param16(q + 4);
      from_raw(p, r, f);
    } else {
      from_bf16(param16(static_cast<const uint16_t*>(p.p) + col), f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < valid ? load1(p, col + j) : 0.0f;
  }
}

// T threads per row, V vectors of 8 columns each (8 T V >= n).
template <int T, int V, bool WIDE, int S>
__global__ void __launch_bounds__(T < 256 ? 256 : T) lnorm_kernel(NormK k) {
  __shared__ float red[2 * 32];
  after_previous_kernel();
  constexpr int R = T < 256 ? 256 / T : 1;  // rows a block works on at a time
  const int t = threadIdx.x % T, group = threadIdx.x / T;
  const Extent e{k.m, k.n};
  const int64_t m = k.m, n = k.n, step = (int64_t)gridDim.x * R;
  const float inv_n = 1.0f / (float)n;
  const bool rms = k.rms, has_bias = k.b.p;
  int turn = 0;
  // this thread's columns, and their parameters for all its rows
  int64_t col[V];
  int valid[V];
  float w[V][8], b[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = S == 1 ? (int64_t)(v * T + t) * 8 : (int64_t)v * T * 8 + t;
    valid[v] = valid_columns<S>(col[v], n);
    if (!valid[v]) col[v] = 0;
    param8<S>(k.w, col[v], valid[v], n, w[v]);
    if (has_bias) param8<S>(k.b, col[v], valid[v], n, b[v]);
  }
  RowVec<WIDE, S> next[V];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < V; ++v) next[v].load(k.x, row, col[v], valid[v], e);
  };
  int64_t row = (int64_t)blockIdx.x * R + group;
  if (row < m) fetch(row);
  for (; row < m; row += step) {  // the same rows for all T threads
    float x[V][8], mean = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) next[v].get(k.x, x[v]);
    if (row + step < m) fetch(row + step);
    if (!rms) {
      float s[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += x[v][j];
      row_sum<T, 1>(s, red, turn, group);
      mean = s[0] * inv_n;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (valid[v] == 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[v][j] -= mean;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[v][j] = j < valid[v] ? x[v][j] - mean : 0.0f;
        }
      }
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) q[0] += x[v][j] * x[v][j];
    row_sum<T, 1>(q, red, turn, group);
    const float rstd = 1.0f / sqrtf(q[0] * inv_n + k.eps);
    if (t == 0) {
      if (k.mean && in_extent(row, row + 1, 0, m, kSite)) k.mean[row] = mean;
      if (k.rstd && in_extent(row, row + 1, 0, m, kSite)) k.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!valid[v]) continue;
      if (has_bias) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] = x[v][j] * rstd * w[v][j] + b[v][j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] = x[v][j] * rstd * w[v][j];
      }
      store_columns<S>(k.y, row, col[v], valid[v], x[v], e);
    }
  }
}

// Rows too long for the registers of one block: three sweeps over memory.
constexpr int kLong = 1024;
__global__ void __launch_bounds__(kLong) lnorm_long_kernel(NormK k) {
  __shared__ float red[2 * 32];
  after_previous_kernel();
  int turn = 0;
  const Extent e{k.m, k.n}, pe{1, k.n};
  const int64_t row = blockIdx.x;
  float x[8], s[1] = {0.0f}, q[1] = {0.0f};
  float mean = 0.0f;
  if (!k.rms) {
    for (int64_t col = threadIdx.x * 8; col < k.n; col += kLong * 8) {
      load8(k.x, row, col, valid_of(col, k.n), x, e, kSite);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += x[j];
    }
    row_sum<kLong, 1>(s, red, turn, 0);
    mean = s[0] / (float)k.n;
  }
  for (int64_t col = threadIdx.x * 8; col < k.n; col += kLong * 8) {
    const int valid = valid_of(col, k.n);
    load8(k.x, row, col, valid, x, e, kSite);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) q[0] += (x[j] - mean) * (x[j] - mean);
  }
  row_sum<kLong, 1>(q, red, turn, 0);
  const float rstd = 1.0f / sqrtf(q[0] / (float)k.n + k.eps);
  if (threadIdx.x == 0) {
    if (k.mean && in_extent(row, row + 1, 0, k.m, kSite)) k.mean[row] = mean;
    if (k.rstd && in_extent(row, row + 1, 0, k.m, kSite)) k.rstd[row] = rstd;
  }
  for (int64_t col = threadIdx.x * 8; col < k.n; col += kLong * 8) {
    const int valid = valid_of(col, k.n);
    float w[8], b[8];
    load8(k.x, row, col, valid, x, e, kSite);
    load8(k.w, 0, col, valid, w, pe, kSite);
    if (k.b.p) load8(k.b, 0, col, valid, b, pe, kSite);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = (x[j] - mean) * rstd * w[j];
      if (k.b.p) x[j] += b[j];
    }
    store8(k.y, row, col, valid, x, e, kSite);
  }
}

// One wave of blocks, or fewer where there are fewer rows.
template <int T, int V, bool WIDE, int S>
static cudaError_t launch_step(const NormK& k, cudaStream_t st) {
  constexpr int threads = T < 256 ? 256 : T, R = threads / T;
  const auto kernel = lnorm_kernel<T, V, WIDE, S>;
  const int64_t wave =
      (int64_t)sm_count() * occupancy_of(reinterpret_cast<const void*>(kernel), threads);
  const int64_t blocks = (k.m + R - 1) / R;
  return launch_next(kernel, dim3((unsigned)(blocks < wave ? blocks : wave)), dim3(threads), st,
                     k);
}
template <int T, int V, bool WIDE>
static cudaError_t launch_wave(const NormK& k, cudaStream_t st) {
  return k.x.vec && k.y.vec ? launch_step<T, V, WIDE, 1>(k, st)
                            : launch_step<T, V, WIDE, T>(k, st);
}
// 16 columns per thread in bf16, 8 in fp32 (which takes twice the registers)
// while 1024 threads can hold the row so.
static cudaError_t launch_rows_bf16(const NormK& k, cudaStream_t st) {
  if (k.n <= 512) return launch_wave<32, 2, false>(k, st);
  if (k.n <= 1024) return launch_wave<64, 2, false>(k, st);
  if (k.n <= 2048) return launch_wave<128, 2, false>(k, st);
  if (k.n <= 4096) return launch_wave<256, 2, false>(k, st);
  if (k.n <= 8192) return launch_wave<512, 2, false>(k, st);
  if (k.n <= 16384) return launch_wave<1024, 2, false>(k, st);
  return launch_next(lnorm_long_kernel, dim3((unsigned)k.m), dim3(kLong), st, k);
}
static cudaError_t launch_rows_f32(const NormK& k, cudaStream_t st) {
  if (k.n <= 256) return launch_wave<32, 1, true>(k, st);
  if (k.n <= 512) return launch_wave<64, 1, true>(k, st);
  if (k.n <= 1024) return launch_wave<128, 1, true>(k, st);
  if (k.n <= 2048) return launch_wave<256, 1, true>(k, st);
  if (k.n <= 4096) return launch_wave<512, 1, true>(k, st);
  if (k.n <= 8192) return launch_wave<1024, 1, true>(k, st);
  return launch_next(lnorm_long_kernel, dim3((unsigned)k.m), dim3(kLong), st, k);
}

cudaError_t launch_layer_norm(const NormK& k, cudaStream_t st) {
  if (k.m <= 0 || k.n <= 0) return cudaSuccess;
  return k.x.dtype == ZERO_F32 ? launch_rows_f32(k, st) : launch_rows_bf16(k, st);
}

// ---------------------------------------------------------------------------
// Backward.  With h = (x - mean) rstd and g = dy w, one sweep over a row gives
// its two sums (g, g h), the second the row's dx from registers.  The
// parameters' gradients are sums over rows: block p keeps its columns' sums
// of dy h and dy in registers over rows p, p + P, ... and leaves them in
// partials[p]; a second launch adds the P partials in order.
// ---------------------------------------------------------------------------
template <int T, int V, bool WIDE, int S>
__global__ void __launch_bounds__(T < 256 ? 256 : T) lnorm_grad_kernel(NormGradK k) {
  __shared__ float red[2 * 64];
  after_previous_kernel();
  constexpr int R = T < 256 ? 256 / T : 1;
  const int t = threadIdx.x % T, group = threadIdx.x / T;
  int turn = 0;
  const Extent e{k.m, k.n};
  const int64_t n = k.n, step = (int64_t)gridDim.x * R;
  const bool has_res = k.dres.p;
  int64_t col[V];
  int valid[V];
  float w[V][8], dw[V][8], db[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = S == 1 ? (int64_t)(v * T + t) * 8 : (int64_t)v * T * 8 + t;
    valid[v] = valid_columns<S>(col[v], n);
    if (!valid[v]) col[v] = 0;
    param8<S>(k.w, col[v], valid[v], n, w[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = db[v][j] = 0.0f;
  }
  const float inv_n = 1.0f / (float)n;
  // the next row's operands are on their way while this row is worked on
  RowVec<WIDE, S> g0[V], x0[V], r0[V];
  float mean0 = 0.0f, rstd0 = 0.0f;
  auto fetch = [&](int64_t row) {
    mean0 = k.mean ? k.mean[row] : 0.0f;
    rstd0 = k.rstd[row];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      g0[v].load(k.dy, row, col[v], valid[v], e);
      x0[v].load(k.x, row, col[v], valid[v], e);
      if (has_res) r0[v].load(k.dres, row, col[v], valid[v], e);
    }
  };
  int64_t row = (int64_t)blockIdx.x * R + group;
  if (row < k.m) fetch(row);
  for (; row < k.m; row += step) {
    const float mean = mean0, rstd = rstd0;
    float g[V][8], h[V][8], s[2] = {0.0f, 0.0f};
    RowVec<WIDE, S> res[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // beyond the row dy, and so every sum, is 0
      g0[v].get(k.dy, g[v]);
      x0[v].get(k.x, h[v]);
      res[v] = r0[v];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[v][j] = (h[v][j] - mean) * rstd;
        db[v][j] += g[v][j];
        dw[v][j] += g[v][j] * h[v][j];
        g[v][j] *= w[v][j];
        s[0] += g[v][j];
        s[1] += g[v][j] * h[v][j];
      }
    }
    if (row + step < k.m) fetch(row + step);
    row_sum<T, 2>(s, red, turn, group);
    const float mg = k.rms ? 0.0f : s[0] * inv_n, mgh = s[1] * inv_n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!valid[v]) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[v][j] = (g[v][j] - mg - h[v][j] * mgh) * rstd;
      if (has_res) {
        float r[8];
        res[v].get(k.dres, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[v][j] += r[j];
      }
      store_columns<S>(k.dx, row, col[v], valid[v], g[v], e);
    }
  }
  float* out = k.partials + (int64_t)blockIdx.x * 2 * k.n;
  if constexpr (R > 1) {  // the block's groups in order, 2 KiB of columns at a time
    __shared__ float sum[256 * 8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sum[group * (T * 8) + (S == 1 ? t * 8 + j : j * T + t)] = which ? db[v][j] : dw[v][j];
        __syncthreads();
        for (int c = threadIdx.x; c < T * 8; c += 256) {
          const int64_t col = (int64_t)v * T * 8 + c;
          float a = 0.0f;
#pragma unroll
          for (int r = 0; r < R; ++r) a += sum[r * (T * 8) + c];
          if (col < n) out[which * n + col] = a;
        }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t c = (S == 1 ? (int64_t)(v * T + t) * 8 : (int64_t)v * T * 8 + t) + j * S;
        if (c < n) {
          out[c] = dw[v][j];
          out[n + c] = db[v][j];
        }
      }
  }
}

// Long rows: dx alone, re-reading the row, ...
__global__ void __launch_bounds__(kLong) lnorm_grad_long_kernel(NormGradK k) {
  __shared__ float red[2 * 64];
  after_previous_kernel();
  int turn = 0;
  const Extent e{k.m, k.n}, pe{1, k.n};
  const int64_t row = blockIdx.x;
  const float mean = k.mean ? k.mean[row] : 0.0f, rstd = k.rstd[row];
  float g[8], h[8], w[8], s[2] = {0.0f, 0.0f};
  for (int64_t col = threadIdx.x * 8; col < k.n; col += kLong * 8) {
    const int valid = valid_of(col, k.n);
    load8(k.dy, row, col, valid, g, e, kSite);
    load8(k.x, row, col, valid, h, e, kSite);
    load8(k.w, 0, col, valid, w, pe, kSite);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] *= w[j];
      s[0] += g[j];
      if (j < valid) s[1] += g[j] * (h[j] - mean) * rstd;
    }
  }
  row_sum<kLong, 2>(s, red, turn, 0);
  const float inv_n = 1.0f / (float)k.n;
  const float mg = k.rms ? 0.0f : s[0] * inv_n, mgh = s[1] * inv_n;
  for (int64_t col = threadIdx.x * 8; col < k.n; col += kLong * 8) {
    const int valid = valid_of(col, k.n);
    float r[8];
    load8(k.dy, row, col, valid, g, e, kSite);
    load8(k.x, row, col, valid, h, e, kSite);
    load8(k.w, 0, col, valid, w, pe, kSite);
    if (k.dres.p) load8(k.dres, row, col, valid, r, e, kSite);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = (g[j] * w[j] - mg - (h[j] - mean) * rstd * mgh) * rstd;
      if (k.dres.p) g[j] += r[j];
    }
    store8(k.dx, row, col, valid, g, e, kSite);
  }
}

// ... and the parameters' sums by columns: block (column block, p).
__global__ void __launch_bounds__(256) lnorm_columns_kernel(NormGradK k, int64_t parts) {
  __shared__ float sum[2][8][32];
  after_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float dw = 0.0f, db = 0.0f;
  if (col < k.n)
    for (int64_t row = blockIdx.y + (int64_t)warp * parts; row < k.m; row += 8 * parts) {
      const float mean = k.mean ? k.mean[row] : 0.0f;
      if (!in_extent(row, row + 1, 0, k.m, kSite)) continue;
      const float d = load1(k.dy, row * k.dy.ld + col);
      db += d;
      dw += d * (load1(k.x, row * k.x.ld + col) - mean) * k.rstd[row];
    }
  sum[0][warp][lane] = dw;
  sum[1][warp][lane] = db;
  __syncthreads();
  if (warp < 2 && col < k.n) {
    float a = 0.0f;
    for (int w = 0; w < 8; ++w) a += sum[warp][w][lane];
    k.partials[((int64_t)blockIdx.y * 2 + warp) * k.n + col] = a;
  }
}

// dw (blockIdx.y = 0) or db (1): the parts' sums of 32 columns in a fixed
// order, 32 warps taking every 32nd part.
__global__ void __launch_bounds__(1024) lnorm_finish_kernel(NormGradK k, int64_t parts) {
  __shared__ float sum[32][33];
  after_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
  const Mat& out = which ? k.db : k.dw;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float a = 0.0f;
  if (col < k.n) {
#pragma unroll 4
    for (int64_t p = warp; p < parts; p += 32) a += k.partials[(p * 2 + which) * k.n + col];
  }
  sum[warp][lane] = a;
  __syncthreads();
  a = sum[lane][warp];  // column `warp` of the block, one part per lane
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  const int64_t c = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && c < k.n && in_extent(c, c + 1, 0, k.n, kSite)) {
    if (k.accumulate) a += load1(out, c);
    store1(out, c, a);
  }
}

template <int T, int V, bool WIDE, int S>
static cudaError_t launch_grad_step(const NormGradK& k, int64_t& parts, cudaStream_t st) {
  constexpr int threads = T < 256 ? 256 : T;
  constexpr int R = T < 256 ? 256 / T : 1;
  const auto kernel = lnorm_grad_kernel<T, V, WIDE, S>;
  // one wave of blocks, each with a part of its own
  const int64_t wave =
      (int64_t)sm_count() * occupancy_of(reinterpret_cast<const void*>(kernel), threads);
  const int64_t blocks = (k.m + R - 1) / R;
  if (blocks < parts) parts = blocks;
  if (wave < parts) parts = wave;
  return launch_next(kernel, dim3((unsigned)parts), dim3(threads), st, k);
}
template <int T, int V, bool WIDE>
static cudaError_t launch_grad(const NormGradK& k, int64_t& parts, cudaStream_t st) {
  return k.dy.vec && k.x.vec && k.dx.vec && (!k.dres.p || k.dres.vec)
             ? launch_grad_step<T, V, WIDE, 1>(k, parts, st)
             : launch_grad_step<T, V, WIDE, T>(k, parts, st);
}
template <bool WIDE>
static cudaError_t launch_grad_rows(const NormGradK& k, int64_t& parts, cudaStream_t st) {
  if (k.n <= 256) return launch_grad<32, 1, WIDE>(k, parts, st);
  if (k.n <= 512) return launch_grad<64, 1, WIDE>(k, parts, st);
  if (k.n <= 1024) return launch_grad<128, 1, WIDE>(k, parts, st);
  if (k.n <= 2048) return launch_grad<256, 1, WIDE>(k, parts, st);
  if (k.n <= 4096) return launch_grad<512, 1, WIDE>(k, parts, st);
  return launch_grad<512, 2, WIDE>(k, parts, st);
}

cudaError_t launch_layer_norm_grad(const NormGradK& k, cudaStream_t st) {
  if (k.n <= 0) return cudaSuccess;
  int64_t parts = norm_partials(k.m);
  cudaError_t e = cudaSuccess;
  if (k.m > 0) {
    const bool wide = k.dy.dtype == ZERO_F32 || k.x.dtype == ZERO_F32 ||
                      (k.dres.p && k.dres.dtype == ZERO_F32);
    if (k.n <= 8192) {
      e = wide ? launch_grad_rows<true>(k, parts, st) : launch_grad_rows<false>(k, parts, st);
    } else {
      e = launch_next(lnorm_grad_long_kernel, dim3((unsigned)k.m), dim3(kLong), st, k);
      if (e != cudaSuccess) return e;
      if (parts > 32) parts = 32;  // long rows already give many column blocks
      e = launch_next(lnorm_columns_kernel, dim3((unsigned)((k.n + 31) / 32), (unsigned)parts),
                      dim3(256), st, k, parts);
    }
    if (e != cudaSuccess) return e;
  }
  return launch_next(lnorm_finish_kernel, dim3((unsigned)((k.n + 31) / 32), k.db.p ? 2 : 1),
                     dim3(1024), st, k, parts);
}

cudaError_t bounds_lnorm(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
