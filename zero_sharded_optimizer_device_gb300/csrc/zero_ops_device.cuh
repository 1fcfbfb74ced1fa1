// Device helpers of the layer-computation operators: vectors of 8 values in
// either dtype, activations and their slopes, dropout's random words.
#pragma once

#include "zero_device.cuh"
#include "zero_ops.h"

namespace zk {

// ------------------------------------------------------------------------
// 8 consecutive columns of a matrix row as fp32, in one or two 16-byte
// accesses where the matrix allows it (vec) and all 8 exist, singly
// otherwise; columns from `valid` on read as 0 and are not written.  The
// checked build tests every access against the matrix's extent: rows rows of
// cols columns.
// ------------------------------------------------------------------------
struct Extent {
  int64_t rows, cols;
};

__device__ __forceinline__ void load8(const Mat& a, int64_t row, int64_t col, int valid,
                                      float f[8], const Extent& e, int site) {
  const int64_t i = row * a.ld + col;
  if (!in_extent(i, i + valid, row * a.ld, row * a.ld + e.cols, site) ||
      !in_extent(row, row + 1, 0, e.rows, site)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    return;
  }
  if (a.dtype == ZERO_F32) {
    const float* p = static_cast<const float*>(a.p) + i;
    if (a.vec && valid == 8) {
      const float4 u = ld_state(p), v = ld_state(p + 4);
      f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
      f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = j < valid ? p[j] : 0.0f;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.p) + i;
    if (a.vec && valid == 8) {
      uint4 u;
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                   : "l"(p));
      f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x);
      f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
      f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z);
      f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = j < valid ? __uint_as_float((uint32_t)p[j] << 16) : 0.0f;
    }
  }
}

__device__ __forceinline__ uint4 pack8(const float f[8]) {
  uint4 u;
  u.x = pack_bf16x2(f[0], f[1]);
  u.y = pack_bf16x2(f[2], f[3]);
  u.z = pack_bf16x2(f[4], f[5]);
  u.w = pack_bf16x2(f[6], f[7]);
  return u;
}

__device__ __forceinline__ void store8(const Mat& a, int64_t row, int64_t col, int valid,
                                       const float f[8], const Extent& e, int site) {
  const int64_t i = row * a.ld + col;
  if (!in_extent(i, i + valid, row * a.ld, row * a.ld + e.cols, site) ||
      !in_extent(row, row + 1, 0, e.rows, site))
    return;
  if (a.dtype == ZERO_F32) {
    float* p = static_cast<float*>(a.p) + i;
    if (a.vec && valid == 8) {
      *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) p[j] = f[j];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(a.p) + i;
    if (a.vec && valid == 8) {
      *reinterpret_cast<uint4*>(p) = pack8(f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) p[j] = to_bf16(f[j]);
    }
  }
}

__device__ __forceinline__ float load1(const Mat& a, int64_t i) {
  return a.dtype == ZERO_F32
             ? static_cast<const float*>(a.p)[i]
             : __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.p)[i] << 16);
}
__device__ __forceinline__ void store1(const Mat& a, int64_t i, float v) {
  if (a.dtype == ZERO_F32)
    static_cast<float*>(a.p)[i] = v;
  else
    static_cast<uint16_t*>(a.p)[i] = to_bf16(v);
}

// ------------------------------------------------------------------------
// Activations.  Both GELU forms and SiLU are z times a distribution function
// s(z); the tanh form's (1 + tanh u) / 2 is the logistic function of 2u, so
// it costs one exponential and one division, as SiLU does.
// ------------------------------------------------------------------------
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;
constexpr float kRsqrt2 = 0.70710678118654752f;
constexpr float kRsqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case ZERO_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    case ZERO_ACT_GELU: return 0.5f * z * (1.0f + erff(z * kRsqrt2));
    case ZERO_ACT_GELU_TANH: return z * logistic(kGeluA * (z + kGeluB * z * z * z));
    case ZERO_ACT_SILU: return z * logistic(z);
    default: return z;
  }
}

// act(z) and d act / dz.
__device__ __forceinline__ void activate_grad(float z, int act, float& value, float& slope) {
  switch (act) {
    case ZERO_ACT_RELU:
      value = z < 0.0f ? 0.0f : z;
      slope = z > 0.0f ? 1.0f : 0.0f;
      break;
    case ZERO_ACT_GELU: {
      const float s = 0.5f * (1.0f + erff(z * kRsqrt2));
      value = z * s;
      slope = s + z * kRsqrt2Pi * __expf(-0.5f * z * z);
      break;
    }
    case ZERO_ACT_GELU_TANH: {
      const float s = logistic(kGeluA * (z + kGeluB * z * z * z));
      value = z * s;
      slope = s + value * (1.0f - s) * (kGeluA * (1.0f + 3.0f * kGeluB * z * z));
      break;
    }
    case ZERO_ACT_SILU: {
      const float s = logistic(z);
      value = z * s;
      slope = s + value * (1.0f - s);
      break;
    }
    default:
      value = z;
      slope = 1.0f;
  }
}

// ------------------------------------------------------------------------
// Philox4x32-10 [Salmon et al. 2011, "Parallel random numbers: as easy as 1,
// 2, 3"]: ten rounds of two 32x32 -> 64 multiplications and the Weyl key
// sequence, integers throughout, so every build draws the same words.
// ------------------------------------------------------------------------
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)c.x * 0xD2511F53u, q = (uint64_t)c.z * 0xCD9E8D57u;
    c = make_uint4((uint32_t)(q >> 32) ^ c.y ^ k0, (uint32_t)q, (uint32_t)(p >> 32) ^ c.w ^ k1,
                   (uint32_t)p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// Drops in place among 8 consecutive columns starting at col (a multiple of
// 8) of a row; `offset` as drop_offset() gives it.
__device__ __forceinline__ uint64_t drop_offset(const DropK& d) {
  return d.offset + (d.d_offset ? *d.d_offset : 0ull);
}
__device__ __forceinline__ void drop8(const DropK& d, uint64_t offset, uint32_t row, int64_t col,
                                      float f[8]) {
  const uint32_t k0 = (uint32_t)d.seed, k1 = (uint32_t)(d.seed >> 32);
  const uint32_t g = (uint32_t)(col >> 2), lo = (uint32_t)offset, hi = (uint32_t)(offset >> 32);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 w = philox(make_uint4(g + h, row, lo, hi), k0, k1);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[4 * h + j] = (u[j] >= d.least && !d.all) ? f[4 * h + j] * d.scale : 0.0f;
  }
}

// ------------------------------------------------------------------------
// What follows a product: 8 consecutive columns of output row `row` (of an
// output of e.rows x e.cols), v holding the fp32 sums on entry.
// ------------------------------------------------------------------------
template <int MODE>
__device__ __forceinline__ void epilogue8(const EpiK& k, uint64_t offset, int64_t row,
                                          int64_t col, int valid, float v[8], const Extent& e) {
  constexpr int site = ZERO_SITE_LINEAR_OUT;
  float f[8];
  if constexpr (MODE == LIN_FORWARD) {
    if (k.bias.p) {
      load8(k.bias, 0, col, valid, f, Extent{1, e.cols}, site);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
    if (k.pre.p) store8(k.pre, row, col, valid, v, e, site);
    if (k.act != ZERO_ACT_NONE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = activate(v[j], k.act);
    }
    if (k.gate.p) {
      load8(k.gate, row, col, valid, f, e, site);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f[j];
    }
    if (k.drop.on) drop8(k.drop, offset, (uint32_t)row, col, v);
    if (k.residual.p) {
      load8(k.residual, row, col, valid, f, e, site);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
  } else if constexpr (MODE == LIN_DINPUT) {
    if (k.pre.p) {
      float value[8], slope[8];
      load8(k.pre, row, col, valid, f, e, site);
#pragma unroll
      for (int j = 0; j < 8; ++j) activate_grad(f[j], k.act, value[j], slope[j]);
      if (k.gate.p) {
        load8(k.gate, row, col, valid, f, e, site);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          value[j] *= v[j];
          slope[j] *= f[j];
        }
        if (k.dgate.p) store8(k.dgate, row, col, valid, value, e, site);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= slope[j];
    }
  } else {
    if (k.accumulate) {
      load8(k.out, row, col, valid, f, e, site);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
  }
  store8(k.out, row, col, valid, v, e, site);
}

}  // namespace zk
