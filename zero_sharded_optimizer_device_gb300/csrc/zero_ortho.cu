// Orthogonalised updates (zero_orthogonalize, zero_muon_step in
// include/zero.h): Newton-Schulz steps on a batch of matrices,
//   G = X X^T (of the shorter side),  P = b G + c G^2,  X <- a X + P X,
// three products a step on the tensor cores.
//
// Number formats.  A step takes near-equal terms apart (at a singular value of
// 1: 3.44 - 4.78 + 2.03 = 0.70), so roundings are multiplied by 14, and small
// singular values grow 3.44 times a step with the roundings of the large ones
// beside them.  Operands of products are fp16 (three bits more than bf16 at
// the same rate), scaled by powers of two into its range.  X itself is held in
// two fp16 numbers, the operand and what its rounding left: the term a X then
// loses nothing.  The diagonals of G and P, their largest elements, are held
// apart in fp32, the operands having zeros there, and enter by
//   G^2 = O^2 + (d_i + d_j) O + d^2,   P X = O_P X + d_P X.
// Five steps are off by 5e-4 to 7e-4 in 2-norm (random or of any steep
// spectrum); with operands alone in fp16, 1.3e-3 on random matrices and 4e-2
// at rank 16; in bf16 1e-2 and 0.3.
#include "zero_tile.cuh"

#include <cuda_fp16.h>

namespace zk {

// Powers of two that operands are stored times: X, O of G, O of P.
constexpr float kScaleX = 4096.0f, kScaleG = 256.0f, kScaleP = 64.0f;

constexpr int kBoxChunks = 2;                    // chunks in flight, two boxes each
constexpr int kBox = 16384;                      // 128 rows of 64 fp16 columns
constexpr int kSideBytes = 2 * kBoxChunks * kBox;
constexpr int kStagesMost = 8;
constexpr int kEpi0 = 4, kEpis = 16;             // epilogue warps
constexpr int kOrthoThreads = 32 * (kEpi0 + kEpis);

// ------------------------------------------------------------- the product --
enum OrthoStep : int { GRAM = 0, POLY = 1, GROW = 2 };

// D = A B over the contraction, with 256 x bn tiles of one matrix of the batch.
struct OrthoK {
  int kblocks, stages, bn, bn_log2;
  int tiles, tiles_each;    // all, of one matrix
  int tiles_j;              // GROW: across
  int cols;                 // GROW: columns of X as stored
  int a_c, b_c;             // the operand's contraction index is the contiguous one
  int rows_a, rows_b, rows_out;  // rows of the batch's matrices, one below the other
  int by_column;            // GROW: P's diagonal goes by column
  int last;                 // GROW: the remainder is not needed any more
  float a, b, c;
  const float* diag_in;     // POLY: of G; GROW: of P
  float* diag_out;          // GRAM, POLY
  int diag_rows;            // of each matrix
};
struct OrthoMaps {
  CUtensorMap in0, in1;     // POLY: G; GROW: X's two parts
  CUtensorMap out0, out1;   // GRAM, POLY: result, and in boxes of 64 x 64; GROW: X's two parts
};

struct OrthoTile {
  int b, i0, j0, chunks;    // matrix, first row and column, 64-column pieces
};
// Tiles of symmetric results are those of the lower triangle, row by row: row i
// of 256 has i + 1 squares of 256, each of 256 / bn tiles.
template <int STEP>
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoK& k, int t) {
  OrthoTile o;
  o.b = t / k.tiles_each;
  t -= o.b * k.tiles_each;
  if (STEP == GROW) {
    const int i = t / k.tiles_j;
    o.i0 = i * 256;
    o.j0 = (t - i * k.tiles_j) << k.bn_log2;
    const int left = k.cols - o.j0;
    o.chunks = (left < k.bn ? left : k.bn) / 64;
  } else {
    const int s = 8 - k.bn_log2, square = t >> s;
    int i = (int)((sqrtf(8.0f * (float)square + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > square) --i;
    while ((i + 1) * (i + 2) / 2 <= square) ++i;
    o.i0 = i * 256;
    o.j0 = (square - i * (i + 1) / 2) * 256 + ((t & ((1 << s) - 1)) << k.bn_log2);
    o.chunks = k.bn / 64;
  }
  return o;
}
// Whether the result's transpose has to be stored too.
template <int STEP>
__device__ __forceinline__ bool mirrored(const OrthoK& k, const OrthoTile& o) {
  return STEP != GROW && o.j0 + k.bn <= o.i0;
}

__device__ __forceinline__ uint32_t box_at(int row, int unit) {  // 16-byte units, 128-byte swizzle
  return (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4));
}
__device__ __forceinline__ void halves8(const uint4& u, float f[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 to_halves8(const float f[8]) {
  return make_uint4(half2_of(f[0], f[1]), half2_of(f[2], f[3]), half2_of(f[4], f[5]),
                    half2_of(f[6], f[7]));
}
// hi = v rounded; v becomes what that left.
__device__ __forceinline__ uint4 split_halves8(float v[8]) {
  const uint4 hi = to_halves8(v);
  float f[8];
  halves8(hi, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] -= f[j];
  return hi;
}

// Warp 3: brings the operands of the epilogue's chunks and stores its results.
template <int STEP>
__device__ __forceinline__ void ortho_traffic(const OrthoMaps& maps, const OrthoK& k,
                                              uint32_t boxes, uint32_t efull, uint32_t edone,
                                              int first, int step, int half, volatile int* dead) {
  constexpr uint32_t bytes = STEP == GRAM ? 0 : STEP == POLY ? kBox : 2 * kBox;
  OrthoTile in{}, out{};
  int in_t = first, out_t = first, in_c = 0, out_c = 0;
  if (first < k.tiles) in = out = ortho_tile<STEP>(k, first);
  uint32_t ahead = 0, lb = 0, sb = 0, sph = 0;
  bool live = true;
  while (out_t < k.tiles) {
    while (in_t < k.tiles && ahead < kBoxChunks) {
      const uint32_t at = boxes + lb * 2 * kBox, bar = efull + 8 * lb;
      const int x = in.j0 + 64 * in_c, y = in.b * k.rows_out + in.i0 + half * kRowsCta;
      if (elect() && live) {
        bar_expect(bar, bytes);
        if (STEP != GRAM) box_load(&maps.in0, at, x, y, bar);
        if (STEP == GROW) box_load(&maps.in1, at + kBox, x, y, bar);
      }
      __syncwarp();
      ++ahead;
      if (++lb == kBoxChunks) lb = 0;
      if (++in_c == in.chunks) {
        in_c = 0;
        in_t += step;
        if (in_t < k.tiles) in = ortho_tile<STEP>(k, in_t);
      }
    }
    live = live && bar_wait(edone + 8 * sb, sph, dead);
    live = __all_sync(0xffffffffu, live);  // the lanes leave together
    if (!live) break;
    const uint32_t at = boxes + sb * 2 * kBox;
    const int x = out.j0 + 64 * out_c, row = out.i0 + half * kRowsCta;
    if (elect()) {
      box_store(&maps.out0, at, x, out.b * k.rows_out + row);
      if (STEP == GROW) {
        if (!k.last) box_store(&maps.out1, at + kBox, x, out.b * k.rows_out + row);
      } else if (mirrored<STEP>(k, out)) {
        box_store(&maps.out1, at + kBox, row, out.b * k.rows_out + x);
        box_store(&maps.out1, at + kBox + kBox / 2, row + 64, out.b * k.rows_out + x);
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    __syncwarp();
    --ahead;
    if (++sb == kBoxChunks) {
      sb = 0;
      sph ^= 1;
    }
    if (++out_c == out.chunks) {
      out_c = 0;
      out_t += step;
      if (out_t < k.tiles) out = ortho_tile<STEP>(k, out_t);
    }
  }
  // after a wait that gave up: the boxes in flight land before the CTA returns
  for (; !live && ahead > 0; --ahead) {
    const long long t0 = clock64();
    while (!bar_try(efull + 8 * sb, sph) && clock64() - t0 < kWaitCycles / 8) {
    }
    if (++sb == kBoxChunks) {
      sb = 0;
      sph ^= 1;
    }
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// 16 sums v of row `row` of the box (row `i` of the matrix), columns j.. of the
// matrix from 16-byte unit `unit` of the box on.
template <int STEP>
__device__ __forceinline__ void ortho_piece(const OrthoK& k, const float* diag_in, float diag_row,
                                            float* diag_out, bool mirror, uint32_t at, int row,
                                            int i, int j, int unit, float v[16]) {
  float d[16];
  if (STEP == POLY || (STEP == GROW && k.by_column)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 x = ld_state(diag_in + j + 4 * q);
      d[4 * q] = x.x; d[4 * q + 1] = x.y; d[4 * q + 2] = x.z; d[4 * q + 3] = x.w;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t p0 = at + box_at(row, unit + h), p1 = p0 + kBox;
    float* w = v + 8 * h;
    const int on_diag = i - (j + 8 * h);  // which of the eight, if any
    if (STEP == GRAM) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (on_diag == q) {
          diag_out[i] = w[q] * (1.0f / (kScaleX * kScaleX));
          w[q] = 0.0f;
        }
        w[q] *= kScaleG / (kScaleX * kScaleX);
      }
      sts16(p0, to_halves8(w));
    } else if (STEP == POLY) {
      float o[8];
      halves8(lds16(p0), o);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float s = w[q] * (1.0f / (kScaleG * kScaleG)), g = o[q] * (1.0f / kScaleG);
        float r = k.b * g + k.c * (s + (diag_row + d[8 * h + q]) * g);
        if (on_diag == q) {
          diag_out[i] = k.b * diag_row + k.c * (s + diag_row * diag_row);
          r = 0.0f;
        }
        w[q] = r * kScaleP;
      }
      sts16(p0, to_halves8(w));
    } else {
      float x[8], y[8];
      halves8(lds16(p0), x);
      halves8(lds16(p1), y);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float f = k.a + (k.by_column ? d[8 * h + q] : diag_row);
        w[q] = f * x[q] + (f * y[q] + w[q] * (1.0f / kScaleP));
      }
      sts16(p0, split_halves8(w));
      sts16(p1, to_halves8(w));
    }
  }
  if (STEP != GROW && mirror) {
    // element (row, c) of the box to row c, column row of two boxes of 64 x 64
    const uint32_t to = at + kBox + (uint32_t)(row >> 6) * (kBox / 2) + (uint32_t)(row & 7) * 2;
    const int u = (row & 63) >> 3;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const __half x = __float2half_rn(v[q]);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + box_at(unit * 8 + q, u)),
                   "h"(*reinterpret_cast<const uint16_t*>(&x)));
    }
  }
}

template <int STEP>
__global__ void __launch_bounds__(kOrthoThreads, 1)
    ortho_kernel(const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ CUtensorMap map_b, const __grid_constant__ OrthoMaps maps,
                 const __grid_constant__ OrthoK k) {
  extern __shared__ __align__(1024) unsigned char ortho_smem[];
  __shared__ __align__(8) uint64_t bars[2 * kStagesMost + 5 + 2 * kBoxChunks];
  __shared__ uint32_t tmem_at;
  __shared__ int dead;
  const uint32_t rank = cluster_rank(), half = rank & 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = kBytesA + k.bn * kDeep;
  const uint32_t ring = smem_u32(ortho_smem), boxes = ring + k.stages * stage_bytes;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStagesMost;
  const uint32_t tfull = empty + 8 * kStagesMost, tempty = tfull + 16, ready = tempty + 16;
  const uint32_t efull = ready + 8, edone = efull + 8 * kBoxChunks;

  if (warp == 0 && elect()) {
    dead = 0;
    for (int s = 0; s < k.stages; ++s) {
      bar_init(full + 8 * s, 1);
      bar_init(empty + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      bar_init(tfull + 8 * a, 1);
      bar_init(tempty + 8 * a, 2 * kEpis);
    }
    bar_init(ready, 2);
    for (int b = 0; b < kBoxChunks; ++b) {
      bar_init(efull + 8 * b, 1);
      bar_init(edone + 8 * b, kEpis);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  cluster_arrive();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 1 && elect()) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_a) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_b) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.out0) : "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_at)),
                 "r"(2 * k.bn)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  const int clusters = (int)(gridDim.x >> 1), first = (int)(blockIdx.x >> 1);
  cluster_wait();
  if (warp == 2) {
    if (elect()) bar_arrive_cluster(remote(ready, 0));
    __syncwarp();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint32_t tmem = 0;
  if (warp == 1 || warp == 2 || warp >= kEpi0) {
    asm volatile("bar.sync 1, %0;" ::"n"((kEpis + 2) * 32) : "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem = *(volatile uint32_t*)&tmem_at;
  }
  const bool early = warp == 3;  // only moves this CTA's own boxes from here on
  if (early) cluster_arrive();

  if (warp == 0) {
    const uint32_t full_lead = remote(full, 0), stages = k.stages, b_bytes = k.bn * kDeep;
    const bool a_c = k.a_c, b_c = k.b_c;
    uint32_t s = 0, ph = 0, end_s = 0, end_ph = 0;  // end: where a wait gave up
    bool live = true;
    for (int t = first; t < k.tiles; t += clusters) {
      const OrthoTile o = ortho_tile<STEP>(k, t);
      const int i0 = o.i0 + (int)half * kRowsCta, j0 = o.j0 + (int)half * (k.bn / 2);
      const int ya = o.b * k.rows_a, yb = o.b * k.rows_b;
      for (int kb = 0; kb < k.kblocks; ++kb) {
        if (live) {
          live = bar_wait(empty + 8 * s, ph ^ 1, &dead);
          end_s = s;
          end_ph = ph;
        }
        const uint32_t a_at = ring + s * stage_bytes, b_at = a_at + kBytesA;
        const uint32_t bar = full_lead + 8 * s;
        const int c = kb * kDeep;
        if (elect() && live) {
          if (half == 0) bar_expect(full + 8 * s, 2 * (kBytesA + b_bytes));
          if (a_c) {
            tma_load(&map_a, a_at, c, ya + i0, bar);
          } else {
            tma_load(&map_a, a_at, i0, ya + c, bar);
            tma_load(&map_a, a_at + 8192, i0 + 64, ya + c, bar);
          }
          if (b_c) {
            tma_load(&map_b, b_at, c, yb + j0, bar);
          } else {
            tma_load(&map_b, b_at, j0, yb + c, bar);
            if (k.bn > 128) tma_load(&map_b, b_at + 8192, j0 + 64, yb + c, bar);
          }
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // a wait gave up: let the loads in flight land before the CTAs return
    if (!live && half == 0)
      for (uint32_t q = 0; q < stages; ++q) {
        const uint32_t parity = q < end_s ? end_ph : end_ph ^ 1;
        const long long t0 = clock64();
        while (!bar_try(full + 8 * q, parity) && clock64() - t0 < kWaitCycles / 8) {
        }
      }
    __syncwarp();
  } else if (warp == 1) {
    if (half == 0) {
      const uint16_t mask = 3;
      const bool a_c = k.a_c, b_c = k.b_c;
      // fp32 sums of fp16 values, M = 256, N = bn
      const uint32_t idesc = (1u << 4) | ((a_c ? 0u : 1u) << 15) | ((b_c ? 0u : 1u) << 16) |
                             ((uint32_t)(k.bn >> 3) << 17) | (16u << 24);
      const uint32_t step_a = a_c ? 2 : 128, step_b = b_c ? 2 : 128;
      const uint32_t stages = k.stages;
      uint32_t s = 0, ph = 0, acc = 0, aph = 0;
      bool live = bar_wait(ready, 0, &dead);
      for (int t = first; t < k.tiles; t += clusters) {
        live = live && bar_wait(tempty + 8 * acc, aph ^ 1, &dead);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + acc * k.bn;
        for (int kb = 0; kb < k.kblocks; ++kb) {
          live = live && bar_wait(full + 8 * s, ph, &dead);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t a_at = ring + s * stage_bytes;
          const uint64_t da = operand_desc(a_at, a_c), db = operand_desc(a_at + kBytesA, b_c);
          if (elect() && live) {
#pragma unroll
            for (int q = 0; q < kDeep / 16; ++q)
              mma_pair(d, da + q * step_a, db + q * step_b, idesc, kb > 0 || q > 0);
            commit_pair(empty + 8 * s, mask);
          }
          __syncwarp();
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (elect() && live) commit_pair(tfull + 8 * acc, mask);
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          aph ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    ortho_traffic<STEP>(maps, k, boxes, efull, edone, first, clusters, (int)half, &dead);
    __syncwarp();
  } else if (warp >= kEpi0) {
    const int w = (warp - kEpi0) & 3, set = (warp - kEpi0) >> 2;
    const int row = w * 32 + lane;
    const uint32_t tempty_lead = remote(tempty, 0);
    uint32_t acc = 0, aph = 0, eb = 0, eph = 0;
    bool ok = true;
    for (int t = first; t < k.tiles && ok; t += clusters) {
      const OrthoTile o = ortho_tile<STEP>(k, t);
      const int i = o.i0 + (int)half * kRowsCta + row;
      const float* diag_in = STEP == GRAM ? nullptr : k.diag_in + (int64_t)o.b * k.diag_rows;
      float* diag_out = STEP == GROW ? nullptr : k.diag_out + (int64_t)o.b * k.diag_rows;
      const float diag_row =
          STEP == POLY || (STEP == GROW && !k.by_column) ? *(volatile const float*)(diag_in + i)
                                                         : 0.0f;
      const bool mirror = mirrored<STEP>(k, o);
      ok = bar_wait(tfull + 8 * acc, aph, &dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tmem + ((uint32_t)(w * 32) << 16) + acc * k.bn + set * 16;
      for (int cc = 0; cc < o.chunks; ++cc) {
        const uint32_t b = eb;
        ok = bar_wait(efull + 8 * b, eph, &dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (++eb == kBoxChunks) {
          eb = 0;
          eph ^= 1;
        }
        uint32_t r[16];
        tmem_load16(d + cc * 64, r);
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = __uint_as_float(r[q]);
        ortho_piece<STEP>(k, diag_in, diag_row, diag_out, mirror, boxes + b * 2 * kBox, row, i,
                          o.j0 + cc * 64 + set * 16, set * 2, v);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(edone + 8 * b);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive_fenced(tempty_lead + 8 * acc);
      if (++acc == 2) {
        acc = 0;
        aph ^= 1;
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  if (!early) cluster_arrive();
  cluster_wait();
  if (warp == 2) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(2 * k.bn));
  }
}

// ------------------------------------------------- what comes before and after --
// Where the matrices come from: the call's x, or reduced gradients and momenta
// of tensors of the flat arrays.
__device__ __forceinline__ Mat source_mat(const OrthoPlaces& s, const Mat& base, int b) {
  Mat m = base;
  const int64_t off = s.listed ? s.offset[b] : b * s.stride;
  m.p = static_cast<char*>(base.p) + off * (base.dtype == ZERO_F32 ? 4 : 2);
  m.vec = ((uintptr_t)m.p & 15) == 0 && base.ld * (base.dtype == ZERO_F32 ? 4 : 2) % 16 == 0;
  return m;
}
__device__ __forceinline__ float muon_grad(const OrthoSource& s, float reduced, float coef) {
  return __fmul_rn(__fmul_rn(reduced, s.grad_scale), coef);
}

// Sums of squares of values whose square may leave fp32's range: as they are,
// times 2^-80 and times 2^100 before squaring.
struct Squares {
  float mid = 0.0f, big = 0.0f, small = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float b = v * 0x1p-80f, s = v * 0x1p100f;
    mid += v * v;
    big += b * b;
    small += s * s;
  }
};

// One block's share of a matrix: its new momentum (muon), and its squares.
__global__ void __launch_bounds__(kThreads) ortho_squares(const __grid_constant__ OrthoSource s) {
  after_previous_kernel();
  const int b = blockIdx.y;
  const Extent e{s.m, s.n};
  const int64_t units = (s.n + 7) / 8, total = units * s.m;
  Squares q;
  const Mat x = source_mat(s.places, s.x, b);
  Mat mom;
  float coef = 1.0f;
  if (s.muon) {
    mom = source_mat(s.places, s.momentum, b);
    if (s.coef) coef = *(volatile const float*)s.coef;
  }
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < total;
       u += (int64_t)gridDim.x * kThreads) {
    const int64_t row = u / units, col = u % units * 8;
    const int valid = s.n - col < 8 ? (int)(s.n - col) : 8;
    float v[8];
    load8(x, row, col, valid, v, e, ZERO_SITE_ORTHO);
    if (s.muon) {
      float m[8];
      load8(mom, row, col, valid, m, e, ZERO_SITE_ORTHO);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = muon_grad(s, v[j], coef);
        m[j] = __fadd_rn(__fmul_rn(s.mu, m[j]), g);
        v[j] = s.nesterov ? __fadd_rn(g, __fmul_rn(s.mu, m[j])) : m[j];
      }
      store8(mom, row, col, valid, m, e, ZERO_SITE_ORTHO);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) q.add(v[j]);
  }
  __shared__ double part[3][kThreads / 32];
  double sum[3] = {q.mid, q.big, q.small};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
#pragma unroll
    for (int m = 16; m; m >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], m);
    if ((threadIdx.x & 31) == 0) part[i][threadIdx.x >> 5] = sum[i];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    double t = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) t += part[threadIdx.x][w];
    s.partials[((int64_t)b * gridDim.x + blockIdx.x) * 3 + threadIdx.x] = t;
  }
}

// X0 = x / (|x| + eps) in two fp16 numbers, zeros around it.
__global__ void __launch_bounds__(kThreads) ortho_scale(const __grid_constant__ OrthoSource s) {
  __shared__ float factor_at;
  after_previous_kernel();
  const int b = blockIdx.y;
  if (threadIdx.x < 32) {
    double sum[3] = {};
    for (int i = threadIdx.x; i < s.blocks; i += 32)
      for (int q = 0; q < 3; ++q) sum[q] += s.partials[((int64_t)b * s.blocks + i) * 3 + q];
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int m = 16; m; m >>= 1) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], m);
    if (threadIdx.x == 0) {
      // (the plain sum holds unless it is this large or small; NaN stays)
      double square = sum[0];
      if (sum[0] > 1e30) square = sum[1] * 0x1p160;
      else if (sum[0] < 1e-30) square = sum[2] * 0x1p-200;
      const double size = sqrt(square) + (double)s.eps;
      // applied twice: its square may lie outside fp32
      float f = size > 0.0 ? (float)sqrt((double)kScaleX / size) : 0.0f;
      if (!(square < (double)INFINITY)) f = __uint_as_float(0x7FC00000u);
      factor_at = f;
    }
  }
  __syncthreads();
  const float f = factor_at;
  const Extent e{s.m, s.n};
  const Mat x = source_mat(s.places, s.x, b);
  Mat mom;
  float coef = 1.0f;
  if (s.muon) {
    mom = source_mat(s.places, s.momentum, b);
    if (s.coef) coef = *(volatile const float*)s.coef;
  }
  const int64_t units = s.ld / 8, total = units * s.rows;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < total;
       u += (int64_t)gridDim.x * kThreads) {
    const int64_t row = u / units, col = u % units * 8;
    float v[8] = {};
    if (row < s.m && col < s.n) {
      const int valid = s.n - col < 8 ? (int)(s.n - col) : 8;
      load8(x, row, col, valid, v, e, ZERO_SITE_ORTHO);
      if (s.muon) {
        float m[8];
        load8(mom, row, col, valid, m, e, ZERO_SITE_ORTHO);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = s.nesterov ? __fadd_rn(muon_grad(s, v[j], coef), __fmul_rn(s.mu, m[j])) : m[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < valid ? v[j] * f * f : 0.0f;
    }
    const int64_t at = ((int64_t)b * s.rows + row) * s.ld + col;
    *reinterpret_cast<uint4*>(s.hi + at) = split_halves8(v);
    *reinterpret_cast<uint4*>(s.lo + at) = to_halves8(v);
  }
}

// y = X, or the update of the master weights by it.
__global__ void __launch_bounds__(kThreads) ortho_finish(const __grid_constant__ OrthoFinish s) {
  after_previous_kernel();
  const int b = blockIdx.y;
  const Extent e{s.m, s.n};
  const int64_t units = (e.cols + 7) / 8, total = units * e.rows;
  const Mat y = source_mat(s.places, s.y, b);
  Mat out;
  if (s.update && s.out.p) out = source_mat(s.places, s.out, b);
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < total;
       u += (int64_t)gridDim.x * kThreads) {
    const int64_t row = u / units, col = u % units * 8;
    const int valid = e.cols - col < 8 ? (int)(e.cols - col) : 8;
    float v[8];
    halves8(ld16(s.x + ((int64_t)b * s.rows + row) * s.ld + col), v);
    if (s.update) {
      float w[8];
      load8(y, row, col, valid, w, e, ZERO_SITE_ORTHO);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (s.decay != 0.0f) w[j] = __fsub_rn(w[j], __fmul_rn(s.decay, w[j]));
        v[j] = __fsub_rn(w[j], __fmul_rn(s.rate, v[j] * (1.0f / kScaleX)));
      }
      if (out.p) store8(out, row, col, valid, v, e, ZERO_SITE_ORTHO);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= 1.0f / kScaleX;
    }
    store8(y, row, col, valid, v, e, ZERO_SITE_ORTHO);
  }
}

// ------------------------------------------------------------------- host --
static int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

bool ortho_fits(int64_t m, int64_t n, int64_t batch) {
  // rows one below the other, tiles and grids in 32 bits; sizes far from 64
  const int64_t k = up(m < n ? m : n, 256), rows = up(m, 256), cols = up(n, 128);
  return batch < 65536 && rows * batch < (1ll << 31) && k * batch < (1ll << 31) &&
         rows / 256 * (cols / 128) < (1ll << 30) / (batch + 1) &&
         k / 256 * (k / 256 + 1) < (1ll << 30) / (batch + 1);
}

OrthoSpace ortho_space(int64_t m, int64_t n, int64_t batch) {
  OrthoSpace w;
  const int64_t k = m < n ? m : n;
  w.rows = up(m, 256);
  w.ld = up(n, 64);
  w.side = up(k, 256);
  // blocks of a matrix's norm: about four of 256 threads per SM for the batch
  const int64_t units = (n + 7) / 8 * m, want = (int64_t)152 * 4 / (batch > 0 ? batch : 1);
  w.blocks = (units + kThreads - 1) / kThreads;
  if (w.blocks > want) w.blocks = want;
  if (w.blocks < 1) w.blocks = 1;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = up(at + bytes, 1024);
    return here;
  };
  const int64_t x = batch * w.rows * w.ld * 2, g = batch * w.side * w.side * 2;
  w.hi[0] = take(x);
  w.hi[1] = take(x);
  w.lo = take(x);
  w.gram = take(g);
  w.poly = take(g);
  w.diag_gram = take(batch * w.side * 4);
  w.diag_poly = take(batch * w.side * 4);
  w.partials = take(batch * w.blocks * 3 * 8);
  w.bytes = at;
  return w;
}

// A matrix of fp16 in boxes of box_x columns x box_y rows.
static bool half_map(CUtensorMap* map, void* p, int64_t cols, int64_t rows, int box_y) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_y}, one[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p, dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int STEP>
static cudaError_t launch_ortho(const CUtensorMap& a, const CUtensorMap& b, const OrthoMaps& maps,
                                OrthoK& k, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  constexpr int most = kSmemMost - 1024;  // the rest is the kernel's static shared memory
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(ortho_kernel<STEP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             most);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  const int stage = kBytesA + k.bn * kDeep;
  k.stages = (most - kSideBytes) / stage;
  if (k.stages > kStagesMost) k.stages = kStagesMost;
  const int pairs = sm_count() / 2, clusters = k.tiles < pairs ? k.tiles : pairs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)clusters * 2);
  cfg.blockDim = dim3(kOrthoThreads);
  cfg.dynamicSmemBytes = (size_t)k.stages * stage + kSideBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ortho_kernel<STEP>, a, b, maps, k);
}

// Tile width: waves of tiles times a tile's steps (see zero_product.cuh's
// measurements of a step at 256 and at 128 columns) and its epilogue.
static int tile_width(int64_t tiles256, int64_t tiles128, int64_t kblocks) {
  const int64_t pairs = sm_count() / 2;
  const double wide = (double)((tiles256 + pairs - 1) / pairs) * (520.0 * kblocks) + 25 * 256;
  const double narrow = (double)((tiles128 + pairs - 1) / pairs) * (430.0 * kblocks) + 25 * 128;
  return wide <= narrow ? 256 : 128;
}

cudaError_t launch_orthogonalize(const OrthoCall& c, cudaStream_t st) {
  const int64_t m = c.source.m, n = c.source.n, batch = c.batch;
  if (m == 0 || n == 0 || batch == 0) return cudaSuccess;
  const OrthoSpace w = ortho_space(m, n, batch);
  char* base = static_cast<char*>(c.workspace);
  const bool tall = m > n;
  const int64_t k = tall ? n : m, far = tall ? m : n;
  const int64_t squares = w.side / 256 * (w.side / 256 + 1) / 2, rows = w.rows / 256;
  OrthoSource s = c.source;
  s.rows = w.rows;
  s.ld = w.ld;
  s.blocks = (int)w.blocks;
  s.partials = reinterpret_cast<double*>(base + w.partials);
  s.hi = reinterpret_cast<uint16_t*>(base + w.hi[0]);
  s.lo = reinterpret_cast<uint16_t*>(base + w.lo);
  cudaError_t e = launch_next(ortho_squares, dim3((unsigned)w.blocks, (unsigned)batch),
                              dim3(kThreads), st, s);
  if (e != cudaSuccess) return e;
  const int64_t each = (w.rows * w.ld / 8 + kThreads - 1) / kThreads;
  const int64_t share = (int64_t)sm_count() * 8 / batch + 1;
  const dim3 grid((unsigned)(each < share ? each : share), (unsigned)batch);
  e = launch_next(ortho_scale, grid, dim3(kThreads), st, s);
  if (e != cudaSuccess) return e;

  void* hi[2] = {base + w.hi[0], base + w.hi[1]};
  void *gram = base + w.gram, *poly = base + w.poly, *lo = base + w.lo;
  const int64_t all = batch * w.rows, sides = batch * w.side;
  const int64_t kb_far = (far + kDeep - 1) / kDeep, kb_k = (k + kDeep - 1) / kDeep;
  const int bn_gram = tile_width(batch * squares, batch * squares * 2, kb_far);
  const int bn_poly = tile_width(batch * squares, batch * squares * 2, kb_k);
  const int bn_grow = tile_width(batch * rows * (up(w.ld, 256) / 256),
                                 batch * rows * (up(w.ld, 128) / 128), kb_k);
  // Operands by rows (boxes of 128 rows, or half a tile's width of them) or, where
  // the contraction runs down the rows, in boxes of 64 of them.
  CUtensorMap x_a[2], x_b[2], gram_a, gram_b, poly_a, poly_b;
  OrthoMaps g{}, p{}, x[2];
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    // in the Gram product, and in the last product of a step
    ok = ok && half_map(&x_a[i], hi[i], w.ld, all, tall ? 64 : kRowsCta) &&
         half_map(&x_b[i], hi[i], w.ld, all, tall ? 64 : bn_gram / 2);
    x[i] = OrthoMaps{};
    ok = ok && half_map(&x[i].in0, hi[i], w.ld, all, kRowsCta) &&
         half_map(&x[i].in1, lo, w.ld, all, kRowsCta) &&
         half_map(&x[i].out0, hi[1 - i], w.ld, all, kRowsCta) &&
         half_map(&x[i].out1, lo, w.ld, all, kRowsCta);
  }
  CUtensorMap grow_x[2];
  for (int i = 0; i < 2; ++i)
    ok = ok && half_map(&grow_x[i], hi[i], w.ld, all, tall ? kRowsCta : 64);
  ok = ok && half_map(&gram_a, gram, w.side, sides, kRowsCta) &&
       half_map(&gram_b, gram, w.side, sides, bn_poly / 2) &&
       half_map(&poly_a, poly, w.side, sides, kRowsCta) &&
       half_map(&poly_b, poly, w.side, sides, bn_grow / 2) &&
       half_map(&g.out0, gram, w.side, sides, kRowsCta) &&
       half_map(&g.out1, gram, w.side, sides, 64) &&
       half_map(&p.in0, gram, w.side, sides, kRowsCta) &&
       half_map(&p.out0, poly, w.side, sides, kRowsCta) &&
       half_map(&p.out1, poly, w.side, sides, 64);
  if (!ok) return cudaErrorInvalidValue;

  auto log2_of = [](int bn) { return bn == 256 ? 8 : 7; };
  OrthoK kg{}, kp{}, kx{};
  kg.kblocks = (int)kb_far;
  kg.bn = bn_gram;
  kg.a_c = kg.b_c = !tall;
  kg.rows_a = kg.rows_b = (int)w.rows;
  kg.rows_out = (int)w.side;
  kg.diag_out = reinterpret_cast<float*>(base + w.diag_gram);
  kp.kblocks = (int)kb_k;
  kp.bn = bn_poly;
  kp.a_c = kp.b_c = 1;
  kp.rows_a = kp.rows_b = kp.rows_out = (int)w.side;
  kp.diag_in = kg.diag_out;
  kp.diag_out = reinterpret_cast<float*>(base + w.diag_poly);
  kx.kblocks = (int)kb_k;
  kx.bn = bn_grow;
  kx.a_c = 1;
  kx.b_c = tall;
  kx.rows_a = (int)(tall ? w.rows : w.side);
  kx.rows_b = (int)(tall ? w.side : w.rows);
  kx.rows_out = (int)w.rows;
  kx.by_column = tall;
  kx.cols = (int)w.ld;
  kx.tiles_j = (int)(up(w.ld, bn_grow) / bn_grow);
  kx.tiles_each = (int)(rows * kx.tiles_j);
  kx.diag_in = kp.diag_out;
  for (OrthoK* q : {&kg, &kp, &kx}) {
    q->bn_log2 = log2_of(q->bn);
    q->diag_rows = (int)w.side;
    if (q != &kx) q->tiles_each = (int)(squares * (256 / q->bn));
    q->tiles = (int)(batch * q->tiles_each);
  }
  int now = 0;
  for (int step = 0; step < c.steps; ++step, now ^= 1) {
    kp.b = c.coef[step][1];
    kp.c = c.coef[step][2];
    kx.a = c.coef[step][0];
    kx.last = step + 1 == c.steps;
    e = launch_ortho<GRAM>(x_a[now], x_b[now], g, kg, st);
    if (e == cudaSuccess) e = launch_ortho<POLY>(gram_a, gram_b, p, kp, st);
    if (e == cudaSuccess)
      e = launch_ortho<GROW>(tall ? grow_x[now] : poly_a, tall ? poly_b : grow_x[now], x[now], kx,
                             st);
    if (e != cudaSuccess) return e;
  }
  OrthoFinish f = c.finish;
  f.m = m;
  f.n = n;
  f.rows = w.rows;
  f.ld = w.ld;
  f.x = reinterpret_cast<const uint16_t*>(hi[now]);
  const int64_t units = ((n + 7) / 8 * m + kThreads - 1) / kThreads;
  return launch_next(ortho_finish, dim3((unsigned)(units < share ? units : share), (unsigned)batch),
                     dim3(kThreads), st, f);
}

cudaError_t timeouts_ortho(unsigned long long* out, bool reset) {
  return unit_timeouts(out, reset);
}
cudaError_t bounds_ortho(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
