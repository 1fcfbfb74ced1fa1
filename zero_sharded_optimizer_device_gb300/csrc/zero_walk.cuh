// Walks over a matrix 8 columns at a time, down its rows.
#pragma once

#include "zero_ops_device.cuh"

namespace zk {

// Eight columns of rows some distance apart, as they lie in memory: one or two
// 16-byte accesses where the matrix and the columns allow it, decided once.
template <bool WIDE, int SITE>
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
  __device__ __forceinline__ bool inside(int64_t at, const Extent& e) const {
    return in_extent(at, at + 1, 0, e.rows, SITE) && in_extent(col, col + 8, 0, e.cols, SITE);
  }
  // N rows, zeros from row `rows` on; the first one exists.  No conditions
  // between the loads: they would keep them from being in flight together
  // (maxima of 8192 x 4096 bf16: 31 us so, 15.5 without).
  template <int N>
  __device__ __forceinline__ void get(Raw8 r[N], int64_t rows, const Extent& e) const {
    if (fast && row + (N - 1) * rows_apart < rows && inside(row, e)) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        r[i].a = ld16(p + i * step);
        r[i].b = WIDE ? ld16(p + i * step + 16) : make_uint4(0, 0, 0, 0);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t at = row + i * rows_apart;
      r[i].a = r[i].b = make_uint4(0, 0, 0, 0);
      if (at >= rows || valid <= 0) continue;
      if (fast && inside(at, e)) {
        r[i].a = ld16(p + i * step);
        if (WIDE) r[i].b = ld16(p + i * step + 16);
      } else {
        r[i] = raw8(m, at, col, valid, e, SITE);
      }
    }
  }
  __device__ __forceinline__ void put(int i, const float v[8], const Extent& e) const {
    const int64_t at = row + i * rows_apart;
    if (fast && inside(at, e)) {
      if (WIDE) {
        float4* to = reinterpret_cast<float4*>(p + i * step);
        to[0] = make_float4(v[0], v[1], v[2], v[3]);
        to[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(p + i * step) = pack8(v);
      }
      return;
    }
    store8(m, at, col, valid, v, e, SITE);
  }
  __device__ __forceinline__ void on(int steps) {
    p += steps * step;
    row += steps * rows_apart;
  }
};
template <bool WIDE>
__device__ __forceinline__ void values8(const Raw8& r, float v[8]) {
  if (!WIDE) {
    from_bf16(r.a, v);
    return;
  }
  v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
  v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
  v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
  v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
}

// Units of 8 columns: a block of 256 threads covers `across` units (a power of
// two, up to 32) of 256 / across rows, and goes on down the rows: no division.
// `blocks`: about how many the GPU should get.
struct Walk {
  int log2_across;
  dim3 grid;
};
static inline Walk walk_over(int64_t rows, int64_t cols, int64_t blocks) {
  const int64_t units = (cols + 7) / 8;
  Walk w;
  w.log2_across = 0;
  while (w.log2_across < 5 && (1ll << w.log2_across) < units) ++w.log2_across;
  const int64_t x = (units + (1 << w.log2_across) - 1) >> w.log2_across;
  const int64_t each = kThreads >> w.log2_across;
  int64_t y = (rows + each - 1) / each, most = blocks / (x < 1 ? 1 : x) + 1;
  if (most > 65535) most = 65535;
  if (y > most) y = most;
  w.grid = dim3((unsigned)x, (unsigned)y);
  return w;
}

}  // namespace zk
