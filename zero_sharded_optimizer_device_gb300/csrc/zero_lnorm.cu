// Layer norm and RMS norm over the rows of a matrix, and their gradients.
//
// Both are bound by memory: a row is read once into registers by the T
// threads that share it (a warp, a block of 256, or more for long rows), its
// sums run over warp shuffles and, for a block, one exchange through shared
// memory, and the result is written from the registers.  The variance is the
// mean of squared distances from the mean already found (two sweeps over
// registers), not a difference of moments, which loses the digits of rows
// whose mean is large.
#include "zero_ops_device.cuh"

namespace zk {

constexpr int kSite = ZERO_SITE_LNORM;
constexpr int64_t kNormPartials = 304;  // row groups of the backward pass: 2 per SM

int64_t norm_partials(int64_t m) { return m < kNormPartials ? m : kNormPartials; }

// Sum of v (N values) over the T threads sharing a row; every one of them
// gets the sum.  red: 32 * N floats per block.
template <int T, int N>
__device__ __forceinline__ void row_sum(float v[N], float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (T > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // the last use of red is over
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[warp * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = 0; w < T / 32; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += red[w * N + i];
  }
}

__device__ __forceinline__ int valid_of(int64_t col, int64_t n) {
  return col >= n ? 0 : (n - col < 8 ? (int)(n - col) : 8);
}

// T threads per row, V vectors of 8 columns each (8 T V >= n).
template <int T, int V>
__global__ void __launch_bounds__(T < 256 ? 256 : T) lnorm_kernel(NormK k) {
  __shared__ float red[32];
  constexpr int R = T < 256 ? 256 / T : 1;  // rows per block
  const int t = threadIdx.x % T;
  const int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / T;
  if (row >= k.m) return;  // whole warps where T = 32, never where T > 32
  const Extent e{k.m, k.n}, pe{1, k.n};
  float x[V][8], s[1] = {0.0f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t col = (int64_t)(v * T + t) * 8;
    const int valid = valid_of(col, k.n);
    load8(k.x, row, valid ? col : 0, valid, x[v], e, kSite);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] += x[v][j];
  }
  float mean = 0.0f;
  if (!k.rms) {
    row_sum<T, 1>(s, red);
    mean = s[0] / (float)k.n;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int valid = valid_of((int64_t)(v * T + t) * 8, k.n);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[v][j] -= mean;
      if (j < valid) q[0] += x[v][j] * x[v][j];
    }
  }
  row_sum<T, 1>(q, red);
  const float rstd = 1.0f / sqrtf(q[0] / (float)k.n + k.eps);
  if (t == 0) {
    if (k.mean && in_extent(row, row + 1, 0, k.m, kSite)) k.mean[row] = mean;
    if (k.rstd && in_extent(row, row + 1, 0, k.m, kSite)) k.rstd[row] = rstd;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t col = (int64_t)(v * T + t) * 8;
    const int valid = valid_of(col, k.n);
    if (!valid) continue;
    float w[8], b[8];
    load8(k.w, 0, col, valid, w, pe, kSite);
    if (k.b.p) load8(k.b, 0, col, valid, b, pe, kSite);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[v][j] = x[v][j] * rstd * w[j];
      if (k.b.p) x[v][j] += b[j];
    }
    store8(k.y, row, col, valid, x[v], e, kSite);
  }
}

// Rows too long for the registers of one block: three sweeps over memory.
constexpr int kLong = 1024;
__global__ void __launch_bounds__(kLong) lnorm_long_kernel(NormK k) {
  __shared__ float red[32];
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
    row_sum<kLong, 1>(s, red);
    mean = s[0] / (float)k.n;
  }
  for (int64_t col = threadIdx.x * 8; col < k.n; col += kLong * 8) {
    const int valid = valid_of(col, k.n);
    load8(k.x, row, col, valid, x, e, kSite);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) q[0] += (x[j] - mean) * (x[j] - mean);
  }
  row_sum<kLong, 1>(q, red);
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

cudaError_t launch_layer_norm(const NormK& k, cudaStream_t st) {
  if (k.m <= 0 || k.n <= 0) return cudaSuccess;
  const unsigned m = (unsigned)k.m, m8 = (unsigned)((k.m + 7) / 8);
  if (k.n <= 256) lnorm_kernel<32, 1><<<m8, 256, 0, st>>>(k);
  else if (k.n <= 512) lnorm_kernel<32, 2><<<m8, 256, 0, st>>>(k);
  else if (k.n <= 1024) lnorm_kernel<32, 4><<<m8, 256, 0, st>>>(k);
  else if (k.n <= 2048) lnorm_kernel<256, 1><<<m, 256, 0, st>>>(k);
  else if (k.n <= 4096) lnorm_kernel<256, 2><<<m, 256, 0, st>>>(k);
  else if (k.n <= 8192) lnorm_kernel<256, 4><<<m, 256, 0, st>>>(k);
  else if (k.n <= 16384) lnorm_kernel<512, 4><<<m, 512, 0, st>>>(k);
  else lnorm_long_kernel<<<m, kLong, 0, st>>>(k);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Backward.  With h = (x - mean) rstd and g = dy w, one sweep over a row gives
// its two sums (g, g h), the second the row's dx from registers.  The
// parameters' gradients are sums over rows: block p keeps its columns' sums
// of dy h and dy in registers over rows p, p + P, ... and leaves them in
// partials[p]; a second launch adds the P partials in order.
// ---------------------------------------------------------------------------
template <int T, int V>
__global__ void __launch_bounds__(T < 256 ? 256 : T) lnorm_grad_kernel(NormGradK k) {
  __shared__ float red[64];
  constexpr int R = T < 256 ? 256 / T : 1;
  const int t = threadIdx.x % T;
  const Extent e{k.m, k.n}, pe{1, k.n};
  float dw[V][8], db[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = db[v][j] = 0.0f;
  const float inv_n = 1.0f / (float)k.n;
  for (int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / T; row < k.m;
       row += (int64_t)gridDim.x * R) {
    const float mean = k.mean ? k.mean[row] : 0.0f, rstd = k.rstd[row];
    float g[V][8], h[V][8], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t col = (int64_t)(v * T + t) * 8;
      const int valid = valid_of(col, k.n);
      float w[8];
      load8(k.dy, row, valid ? col : 0, valid, g[v], e, kSite);
      load8(k.x, row, valid ? col : 0, valid, h[v], e, kSite);
      load8(k.w, 0, valid ? col : 0, valid, w, pe, kSite);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[v][j] = j < valid ? (h[v][j] - mean) * rstd : 0.0f;
        db[v][j] += g[v][j];
        dw[v][j] += g[v][j] * h[v][j];
        g[v][j] *= w[j];
        s[0] += g[v][j];
        s[1] += g[v][j] * h[v][j];
      }
    }
    row_sum<T, 2>(s, red);
    const float mg = k.rms ? 0.0f : s[0] * inv_n, mgh = s[1] * inv_n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t col = (int64_t)(v * T + t) * 8;
      const int valid = valid_of(col, k.n);
      if (!valid) continue;
      float r[8];
      if (k.dres.p) load8(k.dres, row, col, valid, r, e, kSite);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[v][j] = (g[v][j] - mg - h[v][j] * mgh) * rstd;
        if (k.dres.p) g[v][j] += r[j];
      }
      store8(k.dx, row, col, valid, g[v], e, kSite);
    }
  }
  float* out = k.partials + (int64_t)blockIdx.x * 2 * k.n;
  if constexpr (R > 1) {  // the block's rows in warp order
    __shared__ float sum[256 * 8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sum[(threadIdx.x / T) * (T * 8) + t * 8 + j] = which ? db[v][j] : dw[v][j];
        __syncthreads();
        const int c = threadIdx.x;  // T * 8 = 256 columns, one per thread
        const int64_t col = (int64_t)v * T * 8 + c;
        float a = 0.0f;
        for (int r = 0; r < R; ++r) a += sum[r * (T * 8) + c];
        if (col < k.n) out[which * k.n + col] = a;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t col = (int64_t)(v * T + t) * 8 + j;
        if (col < k.n) {
          out[col] = dw[v][j];
          out[k.n + col] = db[v][j];
        }
      }
  }
}

// Long rows: dx alone, re-reading the row, ...
__global__ void __launch_bounds__(kLong) lnorm_grad_long_kernel(NormGradK k) {
  __shared__ float red[64];
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
  row_sum<kLong, 2>(s, red);
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

// dw (blockIdx.y = 0) or db (1): the parts' sums of 32 columns in order, 8
// warps taking every eighth part.
__global__ void __launch_bounds__(256) lnorm_finish_kernel(NormGradK k, int64_t parts) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
  const Mat& out = which ? k.db : k.dw;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float a = 0.0f;
  if (col < k.n)
    for (int64_t p = warp; p < parts; p += 8) a += k.partials[(p * 2 + which) * k.n + col];
  sum[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && col < k.n && in_extent(col, col + 1, 0, k.n, kSite)) {
    a = 0.0f;
    for (int w = 0; w < 8; ++w) a += sum[w][lane];
    if (k.accumulate) a += load1(out, col);
    store1(out, col, a);
  }
}

cudaError_t launch_layer_norm_grad(const NormGradK& k, cudaStream_t st) {
  if (k.n <= 0) return cudaSuccess;
  int64_t parts = norm_partials(k.m);
  if (k.m > 0) {
    if (k.n <= 1024) {
      const int64_t blocks = (k.m + 7) / 8;
      if (blocks < parts) parts = blocks;
      const unsigned p = (unsigned)parts;
      if (k.n <= 256) lnorm_grad_kernel<32, 1><<<p, 256, 0, st>>>(k);
      else if (k.n <= 512) lnorm_grad_kernel<32, 2><<<p, 256, 0, st>>>(k);
      else lnorm_grad_kernel<32, 4><<<p, 256, 0, st>>>(k);
    } else if (k.n <= 16384) {
      const unsigned p = (unsigned)parts;
      if (k.n <= 2048) lnorm_grad_kernel<256, 1><<<p, 256, 0, st>>>(k);
      else if (k.n <= 4096) lnorm_grad_kernel<256, 2><<<p, 256, 0, st>>>(k);
      else if (k.n <= 8192) lnorm_grad_kernel<256, 4><<<p, 256, 0, st>>>(k);
      else lnorm_grad_kernel<512, 4><<<p, 512, 0, st>>>(k);
    } else {
      lnorm_grad_long_kernel<<<(unsigned)k.m, kLong, 0, st>>>(k);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      if (parts > 32) parts = 32;  // long rows already give many column blocks
      lnorm_columns_kernel<<<dim3((unsigned)((k.n + 31) / 32), (unsigned)parts), 256, 0, st>>>(
          k, parts);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  lnorm_finish_kernel<<<dim3((unsigned)((k.n + 31) / 32), k.db.p ? 2 : 1), 256, 0, st>>>(k,
                                                                                        parts);
  return cudaGetLastError();
}

cudaError_t bounds_lnorm(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
