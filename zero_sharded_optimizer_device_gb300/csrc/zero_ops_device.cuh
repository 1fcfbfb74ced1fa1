// Device helpers of the layer-computation operators: vectors of 8 values in
// either dtype, activations and their slopes, dropout's random words.
#pragma once

#include "zero_device.cuh"
#include "zero_ops.h"

namespace zk {

// Launches a kernel that may set up while the one before it on the stream is
// still running (it executes griddepcontrol.wait before it touches memory).
template <typename... P, typename... A>
static cudaError_t launch_next(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t st,
                               A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

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

// 8 columns as they lie in memory (bf16 fills `a` alone), so that a load can
// be in flight while other work goes on.
struct Raw8 {
  uint4 a, b;
};
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}
__device__ __forceinline__ uint4 raw8_bf16(const Mat& a, int64_t row, int64_t col, int valid,
                                           const Extent& e, int site) {
  const int64_t i = row * a.ld + col;
  if (!in_extent(i, i + valid, row * a.ld, row * a.ld + e.cols, site) ||
      !in_extent(row, row + 1, 0, e.rows, site))
    return make_uint4(0, 0, 0, 0);
  const uint16_t* p = static_cast<const uint16_t*>(a.p) + i;
  if (a.vec && valid == 8) return ld16(p);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) w[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ Raw8 raw8(const Mat& a, int64_t row, int64_t col, int valid,
                                     const Extent& e, int site) {
  Raw8 r;
  if (a.dtype != ZERO_F32) {
    r.a = raw8_bf16(a, row, col, valid, e, site);
    r.b = make_uint4(0, 0, 0, 0);
    return r;
  }
  float f[8];
  load8(a, row, col, valid, f, e, site);
  r.a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
  r.b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                   __float_as_uint(f[7]));
  return r;
}
__device__ __forceinline__ void from_bf16(const uint4& u, float f[8]) {
  f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x);
  f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
  f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z);
  f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void from_raw(const Mat& a, const Raw8& r, float f[8]) {
  if (a.dtype != ZERO_F32) {
    from_bf16(r.a, f);
  } else {
    f[0] = __uint_as_float(r.a.x); f[1] = __uint_as_float(r.a.y);
    f[2] = __uint_as_float(r.a.z); f[3] = __uint_as_float(r.a.w);
    f[4] = __uint_as_float(r.b.x); f[5] = __uint_as_float(r.b.y);
    f[6] = __uint_as_float(r.b.z); f[7] = __uint_as_float(r.b.w);
  }
}

// ------------------------------------------------------------------------
// Activations.  Both GELU forms and SiLU are z times a distribution function
// s(z); the tanh form's (1 + tanh u) / 2 is the logistic function of 2u, so
// it costs one exponential and one division, as SiLU does.
// ------------------------------------------------------------------------
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;
constexpr float kRsqrt2Pi = 0.39894228040143268f;

// The normal distribution's mass below z, and e = exp(-z^2 / 2).  With x = |z| /
// sqrt 2 the mass beyond |z| is erfc(x) / 2 = t Q(t) e for t = 1 / (1 + 0.33 x),
// the form of Hastings' approximations (1955).  Q has degree 7 and was fitted
// here, by weighted least squares, to erfc(x) exp(x^2) for x up to 9.6 with
// relative error 8e-8: the mass keeps small *relative* error in the negative
// tail, where GELU is z times it.  In fp32 12 + z^2 ulps at most by the steps'
// own bounds; measured 4 near 0, 13 down to -8, 27 down to -12.5, where half an
// ulp of z alone is z^2 / 2 of them.  (Five terms took 60 us instead of 65 for
// 8192 x 1024 to 4096 with bias and kept z, and were 5e-4 off at -4.)
// No branch, and the exponential serves the slope too.
__device__ __forceinline__ float normal_mass(float z, float& e) {
  const float t = __fdividef(1.0f, 1.0f + 0.233345238f * fabsf(z));
  e = __expf(-0.5f * z * z);
  float q = -0.0679643974f;
  q = q * t + 0.231344119f;
  q = q * t - 0.177719474f;
  q = q * t + 0.206270799f;
  q = q * t + 0.0225053225f;
  q = q * t + 0.100961916f;
  q = q * t + 0.0914186239f;
  q = q * t + 0.0931830555f;
  const float tail = q * t * e;
  return z < 0.0f ? tail : 1.0f - tail;
}

// N values through an activation, in place.
template <int N>
__device__ __forceinline__ void activate(float z[N], int act) {
  switch (act) {
    case ZERO_ACT_RELU:
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = z[j] < 0.0f ? 0.0f : z[j];  // NaN stays NaN
      break;
    case ZERO_ACT_GELU:
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float e;
        z[j] = z[j] * normal_mass(z[j], e);
      }
      break;
    case ZERO_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < N; ++j)
        z[j] = z[j] * logistic(z[j] * (kGeluA + kGeluA * kGeluB * z[j] * z[j]));
      break;
    case ZERO_ACT_SILU:
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = z[j] * logistic(z[j]);
      break;
    default:
      break;
  }
}

// act(z) in the place of N values z, and d act / dz.
template <int N>
__device__ __forceinline__ void activate_grad(float value[N], float slope[N], int act) {
  switch (act) {
    case ZERO_ACT_RELU:
#pragma unroll
      for (int j = 0; j < N; ++j) {
        slope[j] = value[j] > 0.0f ? 1.0f : 0.0f;
        value[j] = value[j] < 0.0f ? 0.0f : value[j];
      }
      break;
    case ZERO_ACT_GELU:
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float e;
        const float z = value[j], s = normal_mass(z, e);
        value[j] = z * s;
        slope[j] = s + z * kRsqrt2Pi * e;
      }
      break;
    case ZERO_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // s is 0 or 1 long before the cap, under which the factor of its slope
        // stays finite
        const float z = value[j], q = fminf(z * z, 1e30f);
        const float s = logistic(z * (kGeluA + kGeluA * kGeluB * q));
        value[j] = z * s;
        slope[j] = s + value[j] * (1.0f - s) * (kGeluA + 3.0f * kGeluA * kGeluB * q);
      }
      break;
    case ZERO_ACT_SILU:
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float z = value[j], s = logistic(z);
        value[j] = z * s;
        slope[j] = s + value[j] * (1.0f - s);
      }
      break;
    default:
#pragma unroll
      for (int j = 0; j < N; ++j) slope[j] = 1.0f;
  }
}

// ------------------------------------------------------------------------
// Philox4x32-10 [Salmon et al. 2011, "Parallel random numbers: as easy as 1,
// 2, 3"]: ten rounds of two 32x32 -> 64 multiplications and the Weyl key
// sequence, integers throughout, so every build draws the same words.
// ------------------------------------------------------------------------
__device__ __forceinline__ uint4 philox(uint4 c, const DropK& d) {
  // the multipliers from registers: two blocks take 137 cycles per warp, with
  // immediate operands 172; the rounds' keys straight from the parameters
  uint32_t m0, m1;
  asm volatile("mov.u32 %0, 0xD2511F53;" : "=r"(m0));
  asm volatile("mov.u32 %0, 0xCD9E8D57;" : "=r"(m1));
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)c.x * m0, q = (uint64_t)c.z * m1;
    c = make_uint4((uint32_t)(q >> 32) ^ c.y ^ d.keys[2 * r], (uint32_t)q,
                   (uint32_t)(p >> 32) ^ c.w ^ d.keys[2 * r + 1], (uint32_t)p);
  }
  return c;
}

// The counter's offset: the host's plus the device's.
__device__ __forceinline__ uint64_t drop_offset(const DropK& d) {
  return d.offset + (d.d_offset ? *d.d_offset : 0ull);
}

// bits = 2 * bits + (w >= least), for below = 2^32 - least: the carry of w +
// below, two adds instead of a comparison, a selection and a shift.
__device__ __forceinline__ void push_keep(uint32_t& bits, uint32_t w, uint32_t below) {
  asm("{ .reg .u32 t; add.cc.u32 t, %1, %2; addc.u32 %0, %0, %0; }"
      : "+r"(bits)
      : "r"(w), "r"(below));
}

// The mask of 4 G elements as G groups of 4 columns, PER groups in each of
// G / PER rows `row_step` apart; the first element is the highest bit.  A loop
// of two blocks, not G copies: an epilogue runs this a few times per kernel
// and has to fetch the code as well.
template <int G, int PER>
__device__ __forceinline__ uint32_t keep_mask(const DropK& d, uint64_t offset, uint32_t row,
                                              uint32_t row_step, int64_t col) {
  const uint32_t lo = (uint32_t)offset, hi = (uint32_t)(offset >> 32), below = 0u - d.least;
  const uint32_t group = (uint32_t)(col >> 2);
  uint32_t keep = 0;
#pragma unroll 1
  for (uint32_t g = 0; g < G; g += 2) {
    uint4 w[2];
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h)
      w[h] = philox(make_uint4(group + (g + h) % PER, row + row_step * ((g + h) / PER), lo, hi),
                    d);
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h) {
      push_keep(keep, w[h].x, below);
      push_keep(keep, w[h].y, below);
      push_keep(keep, w[h].z, below);
      push_keep(keep, w[h].w, below);
    }
  }
  keep <<= 32 - 4 * G;
  return d.all ? 0u : d.least == 0 ? 0xFFFFFFFFu : keep;
}

// N values whose mask bits are the highest of `keep`.
template <int N>
__device__ __forceinline__ void apply_keep(uint32_t keep, float scale, float v[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    v[j] = (int32_t)keep < 0 ? v[j] * scale : 0.0f;
    keep += keep;
  }
}

}  // namespace zk
