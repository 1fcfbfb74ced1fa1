// Products of bf16 matrices with what follows them fused in: the forward
// product, its input's and its weight's gradients (see zero_linear*,
// include/zero.h).
//
// D[i][j] = sum over c of A(i, c) B(j, c) on the 5th-generation tensor cores.
// A pair of CTAs (a cluster of two SMs) computes a tile of 256 x BN: each CTA
// keeps 128 rows of A and BN / 2 rows of B in shared memory and 128 x BN fp32
// sums in its tensor memory, so every operand byte is read from shared memory
// by both halves of the tile but stored once.  Warp roles per CTA:
//   warp 0        loads operand tiles 64 deep by TMA into a ring of stages
//   warp 1        (first CTA of the pair) issues the tensor-core instructions
//   warp 2        allocates and frees tensor memory
//   warp 3        (boxes) loads the side operands' boxes by TMA ahead of the
//                 epilogue and stores the finished ones
//   warps 4-      epilogue, in one of two forms:
//                 boxes (16 warps): a thread keeps its row of sums as tensor
//                 memory gives it, reads the side operands from the boxes warp
//                 3 brought and writes its results in their place; addresses,
//                 bounds and coalescing are TMA's
//                 patches (8 warps): 32 x 32 sums cross a patch of shared
//                 memory, and a thread goes on with 8 consecutive columns by
//                 plain loads and stores; for transposed outputs and rows off
//                 16-byte boundaries
//   warps 12-19   (gen) shift operands whose base or rows lie off 16-byte
//                 boundaries into place; warps 2 (A's) and 3 (B's) bring
//                 them to raw buffers
// Tiles are walked persistently with two sets of sums, so one tile's epilogue
// runs under the next one's products.  Where there are too few tiles to fill
// the GPU the contraction is split over the S pairs of a larger cluster, whose
// sums meet in shared memory in a fixed order (no atomics, no workspace).
//
// Operands are bf16, or E2M1 codes with a scale for each block of 16 or 32 of
// them (OF_FP4): then a step's 128 bytes of a row are 256 codes, four
// block-scaled products of 64, and the scales of the step's rows, which lie in
// memory as tensor memory wants them, are copied there before its products.
#pragma once

#include "zero_fp4.cuh"
#include "zero_tile.cuh"

namespace zk {

constexpr int kEpiWarp0 = 4, kPatchWarps = 8, kBoxWarps = 16, kGenWarp0 = 12, kGenWarps = 8;
constexpr int kPatch = 32 * 36;        // floats of a 32 x 32 patch, rows 36 apart
constexpr int kMaxStages = 9;
constexpr int kMostRaw = 4;            // raw buffers
constexpr int kRound = 12;             // 64-deep steps of a round (see launch_mode)
constexpr int kOnesBytes = 2048;
constexpr int kSlot = 16384;           // a box of 128 rows of 128 bytes
constexpr int kMostBoxes = 3;          // chunks of boxes in the ring
constexpr uint32_t kScaleColumn = 384; // where they lie in tensor memory, behind the sums

// What the operands hold.
enum Operands : int { OF_BF16 = 0, OF_FP4 = 1 };

// Forms of the kernel: how operands come in and results go out.
enum Form : int {
  PATCH = 0,      // operands by TMA, results over patches
  PATCH_GEN = 1,  // an operand off 16-byte boundaries, results over patches
  BOX_BF16 = 2,   // operands by TMA, results in boxes of 64 bf16 columns
  BOX_F32 = 3     // operands by TMA, results in boxes of 32 fp32 columns
};

constexpr int threads_of(int form) {
  return 32 * (form == PATCH_GEN ? kGenWarp0 + kGenWarps
                                 : kEpiWarp0 + (form == PATCH ? kPatchWarps : kBoxWarps));
}

// How a launch walks its product (host-made).
struct TileK {
  int tiles_i, tiles_j;
  int bias_tiles;  // that many more sum one operand's rows alone, or
  int bias_fused;  // the first tile of every row (column) sums them beside its products
  int bias_b;      // rows of B (else of A)
  int kblocks, splits, bn, stages;
  int split_log2, clusters;          // splits = 1 << split_log2; clusters launched
  int by_i, by_j;                    // from a cluster's tile to its next (see TileWalk)
  int round;                         // steps whose sums the tensor cores keep (see launch_mode)
  int acc_sets;                      // sets of sums in tensor memory used in turn
  int i_fast;                        // consecutive tiles differ in i (else in j)
  int gen_a, gen_b;                  // operand off 16-byte boundaries
  int raws;                          // raw buffers: a GEN warp's bytes
  int raw_a, raw_b;                  // of either operand in each
  int boxes;                         // ring of box chunks (box forms)
  int two_slots;                     // a chunk holds two slots
  uint32_t tmem_cols;
  int bias_in;                       // bytes of staged forward biases
  int scale_deep, scale_chunks;      // OF_FP4: scale tiles along a step, and over B's rows
  int scale_bytes;                   // of a stage
};

// Box forms: the side operands and outputs (see box_chunk).
struct BoxMaps {
  CUtensorMap out, pre, gate, extra;  // extra: forward residual, dinput dgate
};
// PATCH_GEN: the operands' lines r, r + 8, ... for r = 0..7 (see gen_load).
struct GenMaps {
  CUtensorMap a[8], b[8];
};
// OF_FP4: the operands' scale tiles too.
struct Fp4Maps : BoxMaps {
  CUtensorMap scale_a, scale_b;
};
template <int FORM, int KIND>
struct MapsOf {
  using type = BoxMaps;
};
template <>
struct MapsOf<PATCH_GEN, OF_BF16> {
  using type = GenMaps;
};
template <int FORM>
struct MapsOf<FORM, OF_FP4> {
  using type = Fp4Maps;
};

// ---------------------------------------------------------------------------
// Operands off 16-byte boundaries.  A line of a tile is 64 consecutive
// elements: a row's contraction, or 64 rows at one depth.  Lines 8 apart are
// 16 ld bytes apart, a multiple of 16 whatever ld is, so that the lines r, r +
// 8, ... of a matrix, each begun at the 16-byte word it begins in, make a
// matrix that TMA can read; all of them begin equally far into that word.
// Eight such maps cover an operand.  A warp brings nine words of each line of a
// tile to a raw buffer some steps ahead; a GEN warp writes the lines of one
// map, shifted by their one distance, to the operand's swizzled tile.  Lines
// and elements outside the matrix arrive as zeros.  (3873 x 1614 by 9592 x 1614,
// odd rows: 195 us; by 16-byte asynchronous copies, a line's words in one
// thread, 536; by plain loads into registers 877; by 2-byte loads 2181.)
// ---------------------------------------------------------------------------
constexpr int kRawLine = 9 * 16;
// A tile's lines by one thread: those of rows i0.. (contiguous contraction), or
// of depths c.. and blocks of 64 rows from i0 on; `all` lines exist.
__device__ __forceinline__ void gen_load(const CUtensorMap* maps, bool contig, int64_t all, int i0,
                                         int c, int lines, uint32_t raw, uint32_t raw_warp,
                                         uint32_t bar) {
  constexpr int kNone = 1 << 30;  // a coordinate past every matrix: zeros
  const int x = contig ? c : i0, y = contig ? i0 >> 3 : c >> 3;
  const bool two = !contig && lines > 8;
#pragma unroll
  for (int r = 0; r < kGenWarps; ++r, raw += raw_warp) {
    const int at = all > r ? y : kNone;
    box_load(maps + r, raw, x, at, bar);
    if (two) box_load(maps + r, raw + 8 * kRawLine, x + 64, at, bar);
  }
}
// `lines` lines from the raw buffer to line r, r + 8, ... of the tile: a lane
// has unit lane % 8 (8 elements) of every fourth, N of them at a time.  The
// result begins `bits` into word FIRST of a unit's eight.
template <int FIRST, int N>
__device__ __forceinline__ void gen_units(uint32_t from, uint32_t to, int lines, uint32_t bits) {
  uint4 a[N], b[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    a[q] = b[q] = make_uint4(0, 0, 0, 0);
    if (4 * q < lines) {
      a[q] = lds16(from + 4 * q * kRawLine);
      b[q] = lds16(from + 4 * q * kRawLine + 16);
    }
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const uint32_t x[8] = {a[q].x, a[q].y, a[q].z, a[q].w, b[q].x, b[q].y, b[q].z, b[q].w};
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __funnelshift_r(x[FIRST + i], x[FIRST + i + 1], bits);
    if (4 * q < lines) sts16(to + 4096 * q, make_uint4(u[0], u[1], u[2], u[3]));
  }
}
__device__ __forceinline__ void gen_shift(uint32_t raw, uint32_t tile, int lines, int r,
                                          uint32_t distance, int lane) {
  const int unit = lane & 7, line = lane >> 3;
  const uint32_t from = raw + (uint32_t)(line * kRawLine + unit * 16);
  const uint32_t to = tile + (uint32_t)(line * 1024 + r * 128 + ((unit ^ r) << 4));
  const uint32_t bits = (distance & 2) * 8;
  switch (distance >> 2) {
    case 0: gen_units<0, 4>(from, to, lines - line, bits); break;
    case 1: gen_units<1, 4>(from, to, lines - line, bits); break;
    case 2: gen_units<2, 4>(from, to, lines - line, bits); break;
    default: gen_units<3, 4>(from, to, lines - line, bits);
  }
}
// How far into its 16-byte word line r begins.
__device__ __forceinline__ uint32_t gen_distance(const Mat& a, int r) {
  return ((uint32_t)(uintptr_t)a.p + 2 * (uint32_t)r * (uint32_t)a.ld) & 15;
}

// The tile of index t: its row and column, or the bias column (j < 0).
__device__ __forceinline__ void tile_at(const TileK& g, int t, int& i, int& j) {
  const int main = g.tiles_i * g.tiles_j;
  if (t >= main) {
    i = t - main;
    j = -1;
  } else if (g.i_fast) {
    i = t % g.tiles_i;
    j = t / g.tiles_i;
  } else {
    j = t % g.tiles_j;
    i = t / g.tiles_j;
  }
}

// A walk over a cluster's tiles: the next one without a division (two of them
// for each tile of 4-bit products took a third of a plain epilogue's time), and how
// far it lies from the host (divided out in each warp, 509 x 768 to 50257 fp32 took
// 46.7 us instead of 45.6, 4-bit 1024 x 1024 x 1024 6.6 instead of 6.2).
struct TileWalk {
  int t, ti, tj;
  __device__ __forceinline__ TileWalk(const TileK& g, int first) : t(first) {
    tile_at(g, first, ti, tj);
  }
  __device__ __forceinline__ void next(const TileK& g, int step) {
    t += step;
    const int main = g.tiles_i * g.tiles_j;
    if (t >= main) {
      ti = t - main;
      tj = -1;
      return;
    }
    ti += g.by_i;
    tj += g.by_j;
    if (g.i_fast ? ti >= g.tiles_i : tj >= g.tiles_j) {
      ti += g.i_fast ? -g.tiles_i : 1;
      tj += g.i_fast ? 1 : -g.tiles_j;
    }
  }
};

// Where the sums for the bias lie in tensor memory beside the products of set
// acc: one tile per cluster leaves the second set free, else behind both sets.
__device__ __forceinline__ uint32_t bias_column(const TileK& g, uint32_t acc) {
  if (g.round) return (uint32_t)(3 * g.bn) + 32 * acc;
  return (uint32_t)(g.tiles_i * g.tiles_j <= g.clusters ? g.bn : 2 * g.bn) + 32 * acc;
}
// Rounds of a contraction (see launch_mode), and the column of the sum of the
// rounds before the last.
__device__ __forceinline__ int rounds_of(const TileK& g, int steps) {
  return g.round && steps > 0 ? (steps + g.round - 1) / g.round : 1;
}
__device__ __forceinline__ uint32_t sum_column(const TileK& g) {
  return (uint32_t)(g.acc_sets * g.bn);
}

// A warp finishes a 32 x 32 block of the output (rows row0.., columns col0..)
// as four steps of 8 rows, a lane taking 8 consecutive columns of one row in
// each: 16-byte accesses of bf16, 64 consecutive bytes per row.
struct Block {
  int64_t row, col;  // this lane's in step 0; step it adds 8 it rows
  int valid;         // its columns inside the output
};
__device__ __forceinline__ Block block_of(int64_t row0, int64_t col0, const Extent& e, int lane) {
  Block b;
  b.row = row0 + (lane >> 2);
  b.col = col0 + (lane & 3) * 8;
  b.valid = b.col >= e.cols ? 0 : (e.cols - b.col < 8 ? (int)(e.cols - b.col) : 8);
  return b;
}

// The side operands of a block, read before the sums are at hand.
template <int MODE>
struct Sides {
  uint4 p[4];  // forward: gate; dinput: pre
  Raw8 q[4];   // forward: residual; dinput: gate; dweight: what dw holds
};
template <int MODE>
__device__ __forceinline__ void load_sides(const EpiK& k, const Block& b, const Extent& e,
                                           Sides<MODE>& s) {
  constexpr int site = ZERO_SITE_LINEAR_OUT;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int64_t row = b.row + it * 8;
    if (row >= e.rows || !b.valid) continue;
    if constexpr (MODE == LIN_FORWARD) {
      if (k.gate.p) s.p[it] = raw8_bf16(k.gate, row, b.col, b.valid, e, site);
      if (k.residual.p) s.q[it] = raw8(k.residual, row, b.col, b.valid, e, site);
    } else if constexpr (MODE == LIN_DINPUT) {
      if (k.pre.p) s.p[it] = raw8_bf16(k.pre, row, b.col, b.valid, e, site);
      if (k.gate.p) s.q[it].a = raw8_bf16(k.gate, row, b.col, b.valid, e, site);
    } else {
      if (k.accumulate) s.q[it] = raw8(k.out, row, b.col, b.valid, e, site);
    }
  }
}

// What follows the product for 8 columns of row `row`, v holding their sums.
template <int MODE>
__device__ __forceinline__ void finish8(const EpiK& k, int64_t row,
                                        const Block& b, const Extent& e, const float bias[8],
                                        const uint4& p, const Raw8& q, uint32_t keep,
                                        float v[8]) {
  constexpr int site = ZERO_SITE_LINEAR_OUT;
  float f[8];
  if constexpr (MODE == LIN_FORWARD) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += bias[j];
    if (k.pre.p) store8(k.pre, row, b.col, b.valid, v, e, site);
    activate<8>(v, k.act);
    if (k.gate.p) {
      from_bf16(p, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f[j];
    }
    if (k.drop.on) apply_keep<8>(keep, k.drop.scale, v);
    if (k.residual.p) {
      from_raw(k.residual, q, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
  } else if constexpr (MODE == LIN_DINPUT) {
    if (k.pre.p) {
      float value[8], slope[8];
      from_bf16(p, f);
      #pragma unroll
      for (int j = 0; j < 8; ++j) value[j] = f[j];
      activate_grad<8>(value, slope, k.act);
      if (k.gate.p) {
        from_bf16(q.a, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          value[j] *= v[j];
          slope[j] *= f[j];
        }
        if (k.dgate.p) store8(k.dgate, row, b.col, b.valid, value, e, site);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= slope[j];
    }
  } else {
    if (k.accumulate) {
      from_raw(k.out, q, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
  }
  store8(k.out, row, b.col, b.valid, v, e, site);
}

// The block's sums, lying in the patch in the output's orientation (row r of
// the patch is output row row0 + r).
template <int MODE>
__device__ __forceinline__ void finish_block(const EpiK& k, uint32_t keep, uint32_t patch,
                                             uint32_t biases, const Block& b, const Extent& e,
                                             const Sides<MODE>& s, int lane) {
  float4 b0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b1 = b0;
  if (MODE == LIN_FORWARD && k.bias.p) {
    b0 = ld_shared4(biases + (uint32_t)(lane & 3) * 32);
    b1 = ld_shared4(biases + (uint32_t)(lane & 3) * 32 + 16);
  }
  const float bias[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const uint32_t at = patch + (uint32_t)((it * 8 + (lane >> 2)) * 36 + (lane & 3) * 8) * 4;
    const float4 x = ld_shared4(at), y = ld_shared4(at + 16);
    float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    const int64_t row = b.row + it * 8;
    if (row < e.rows && b.valid)
      finish8<MODE>(k, row, b, e, bias, s.p[it], s.q[it], keep << (8 * it), v);
  }
}

// ---------------------------------------------------------------------------
// Box forms.  A chunk is 64 bf16 or 32 fp32 columns of the tile's 128 rows,
// one or two slots of 16 KiB in which results take the place of operands:
//   forward, bf16: slot 0 gate -> pre, slot 1 residual -> y
//   forward, fp32: the same, slot 0 rows being 64 bytes
//   dinput,  bf16: slot 0 pre -> dx, slot 1 gate -> dgate
//   dinput,  fp32: slot 0 dx, slot 1 pre (first half) and gate -> dgate
//   dweight:       slot 0 what dw holds -> dw
// (forward without gate and pre keeps slot 1 alone, at the chunk's start).
// Rows of 128 bytes are swizzled in 16-byte units by row mod 8, rows of 64 by
// row / 2 mod 4, so that a warp's threads, a row each, meet no bank twice.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t at128(int row, int unit) {
  return (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint32_t at64(int row, int unit) {
  return (uint32_t)(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ void lds_f32(uint32_t base, int row, int i, float f[8]) {
  const uint4 a = lds16(base + at128(row, 2 * i)), b = lds16(base + at128(row, 2 * i + 1));
  f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
  f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
  f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
  f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
}
__device__ __forceinline__ void sts_f32(uint32_t base, int row, int i, const float f[8]) {
  sts16(base + at128(row, 2 * i),
        make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3])));
  sts16(base + at128(row, 2 * i + 1),
        make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                   __float_as_uint(f[7])));
}

// What the box form asks of the epilogue's parameters, read once per kernel.
struct BoxEpi {
  bool bias, gate, pre, residual, dgate, old, drop;
  int act;
  float scale;
};
template <int MODE>
__device__ __forceinline__ BoxEpi box_epi(const EpiK& k) {
  BoxEpi e;
  e.bias = MODE == LIN_FORWARD && k.bias.p;
  e.gate = MODE != LIN_DWEIGHT && k.gate.p;
  e.pre = MODE != LIN_DWEIGHT && k.pre.p;
  e.residual = MODE == LIN_FORWARD && k.residual.p;
  e.dgate = MODE == LIN_DINPUT && k.dgate.p;
  e.old = MODE == LIN_DWEIGHT && k.accumulate;
  e.act = k.act;
  e.drop = MODE == LIN_FORWARD && k.drop.on;
  e.scale = k.drop.scale;
  return e;
}

// 16 sums v of a thread's row `row` of the tile through the epilogue; unit:
// their first 16-byte unit in a bf16 row of the chunk's boxes; bias: where
// their columns' biases lie.  Each step runs over all 16 before the next: a
// branch per step, not per value.
template <int MODE, int FORM>
__device__ __forceinline__ void box_piece(const BoxEpi& k, uint32_t keep, uint32_t chunk,
                                         uint32_t second, int row, int unit, uint32_t bias,
                                         float v[16]) {
  constexpr bool wide = FORM == BOX_F32;
  const uint32_t slot1 = chunk + second;
  float f[8];
  // the two bf16 units of a box, and groups of 8 in the output's dtype
  auto bf16_at = [&](uint32_t base, int i) {
    return base + (wide ? at64(row, unit + i) : at128(row, unit + i));
  };
  auto old8 = [&](uint32_t base, int i) {
    if constexpr (wide)
      lds_f32(base, row, unit + i, f);
    else
      from_bf16(lds16(base + at128(row, unit + i)), f);
  };
  auto put8 = [&](uint32_t base, int i) {
    if constexpr (wide)
      sts_f32(base, row, unit + i, v + 8 * i);
    else
      sts16(base + at128(row, unit + i), pack8(v + 8 * i));
  };
  if constexpr (MODE == LIN_FORWARD) {
    if (k.bias) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 b = ld_shared4(bias + 16 * i);
        v[4 * i] += b.x;
        v[4 * i + 1] += b.y;
        v[4 * i + 2] += b.z;
        v[4 * i + 3] += b.w;
      }
    }
    uint4 gate[2];
    if (k.gate) {
      gate[0] = lds16(bf16_at(chunk, 0));
      gate[1] = lds16(bf16_at(chunk, 1));
    }
    if (k.pre) {
      sts16(bf16_at(chunk, 0), pack8(v));
      sts16(bf16_at(chunk, 1), pack8(v + 8));
    }
    activate<16>(v, k.act);
    if (k.gate) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        from_bf16(gate[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] *= f[j];
      }
    }
    if (k.drop) apply_keep<16>(keep, k.scale, v);
    if (k.residual) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        old8(slot1, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] += f[j];
      }
    }
    put8(slot1, 0);
    put8(slot1, 1);
  } else if constexpr (MODE == LIN_DINPUT) {
    const uint32_t pre_box = wide ? slot1 : chunk, gate_box = wide ? slot1 + kSlot / 2 : slot1;
    if (k.pre) {
      float value[16], slope[16];
      from_bf16(lds16(bf16_at(pre_box, 0)), value);
      from_bf16(lds16(bf16_at(pre_box, 1)), value + 8);
      activate_grad<16>(value, slope, k.act);
      if (k.gate) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t at = bf16_at(gate_box, i);
          from_bf16(lds16(at), f);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            value[8 * i + j] *= v[8 * i + j];
            slope[8 * i + j] *= f[j];
          }
          if (k.dgate) sts16(at, pack8(value + 8 * i));
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] *= slope[j];
    }
    put8(chunk, 0);
    put8(chunk, 1);
  } else {
    if (k.old) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        old8(chunk, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] += f[j];
      }
    }
    put8(chunk, 0);
    put8(chunk, 1);
  }
}

// The chunks of a tile that this CTA has: from cc to count.
template <int WIDTH>
__device__ __forceinline__ void tile_chunks(const TileK& g, int64_t cols, int split, int tj,
                                            int& cc, int& count) {
  const int64_t left = cols - (int64_t)tj * g.bn;
  cc = 0;
  count = tj < 0 ? 0 : ((int)(left < g.bn ? left : g.bn) + WIDTH - 1) / WIDTH;
  if (g.splits > 1) {  // half of the tile's columns
    const int half = g.bn / WIDTH / 2;
    cc = split * half;
    if (count > cc + half) count = cc + half;
  }
}
// A walk over the chunks of this CTA's tiles, in order.
template <int WIDTH>
struct ChunkWalk {
  TileWalk w;
  int cc, count;
  __device__ __forceinline__ ChunkWalk(const TileK& g, int64_t cols, int split, int first,
                                       int tiles, int step)
      : w(g, first), cc(0), count(0) {
    if (first >= tiles) return;
    tile_chunks<WIDTH>(g, cols, split, w.tj, cc, count);
    --cc;
    next(g, cols, split, tiles, step);
  }
  __device__ __forceinline__ void next(const TileK& g, int64_t cols, int split, int tiles,
                                       int step) {
    ++cc;
    while (cc >= count) {
      w.next(g, step);
      if (w.t >= tiles) return;
      tile_chunks<WIDTH>(g, cols, split, w.tj, cc, count);
    }
  }
};

// Warp 3: brings the side operands of up to g.boxes chunks ahead and stores
// each chunk when the epilogue is done with it.
template <int MODE, int FORM>
__device__ __forceinline__ void box_traffic(const BoxMaps& maps, const ProductK& k,
                                            const TileK& g, uint32_t boxes, uint32_t efull,
                                            uint32_t edone, int first, int tiles, int step,
                                            uint32_t half, int split, volatile int* dead) {
  constexpr bool wide = FORM == BOX_F32;
  constexpr int W = wide ? 32 : 64;
  const uint32_t ring = g.boxes, second = g.two_slots ? kSlot : 0, chunk_bytes = kSlot + second;
  constexpr uint32_t narrow = wide ? kSlot / 2 : kSlot;  // a bf16 box
  const BoxEpi e = box_epi<MODE>(k.epi);
  const uint32_t bytes = (e.gate ? narrow : 0) + (e.residual || e.old ? kSlot : 0) +
                         (MODE == LIN_DINPUT && e.pre ? narrow : 0);
  const int64_t rows = k.rows, cols = k.cols;
  const int bn = g.bn;
  ChunkWalk<W> in(g, cols, split, first, tiles, step), out = in;
  uint32_t ahead = 0, lb = 0, sb = 0, sph = 0;  // ahead: chunks whose memory is in use
  int64_t stored = 0;
  const bool lag = bytes == 0 && ring > 2;
  bool live = true;
  while (out.w.t < tiles) {
    while (in.w.t < tiles && ahead < ring) {
      const uint32_t at = boxes + lb * chunk_bytes, slot1 = at + second;
      const uint32_t bar = efull + 8 * lb;
      const int x = in.w.tj * bn + in.cc * W, y = in.w.ti * 256 + (int)half * kRowsCta;
      if (elect() && live) {
        bar_expect(bar, bytes);
        if constexpr (MODE == LIN_FORWARD) {
          if (e.gate) box_load(&maps.gate, at, x, y, bar);
          if (e.residual) box_load(&maps.extra, slot1, x, y, bar);
        } else if constexpr (MODE == LIN_DINPUT) {
          if (e.pre) box_load(&maps.pre, wide ? slot1 : at, x, y, bar);
          if (e.gate) box_load(&maps.gate, wide ? slot1 + kSlot / 2 : slot1, x, y, bar);
        } else {
          if (e.old) box_load(&maps.out, at, x, y, bar);
        }
      }
      __syncwarp();
      ++ahead;
      if (++lb == ring) lb = 0;
      in.next(g, cols, split, tiles, step);
    }
    live = live && bar_wait(edone + 8 * sb, sph, dead);
    live = __all_sync(0xffffffffu, live);  // the lanes leave together
    const uint32_t at = boxes + sb * chunk_bytes, slot1 = at + second;
    const int x = out.w.tj * bn + out.cc * W, y = out.w.ti * 256 + (int)half * kRowsCta;
    if (elect() && live) {
      if (y < rows) {
        if constexpr (MODE == LIN_FORWARD) {
          if (e.pre) box_store(&maps.pre, at, x, y);
          box_store(&maps.out, slot1, x, y);
        } else if constexpr (MODE == LIN_DINPUT) {
          if (e.dgate) box_store(&maps.extra, wide ? slot1 + kSlot / 2 : slot1, x, y);
          box_store(&maps.out, at, x, y);
        } else {
          box_store(&maps.out, at, x, y);
        }
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      // with nothing to load the next chunk may wait: then the one stored
      // before this is free, else this one
      if (lag)
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      else
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    __syncwarp();
    if (!live) break;
    if (!lag || stored > 0) --ahead;
    ++stored;
    if (++sb == ring) {
      sb = 0;
      sph ^= 1;
    }
    out.next(g, cols, split, tiles, step);
  }
  // after a wait that gave up: the boxes in flight land before the CTA returns
  for (; !live && ahead > 0; --ahead) {
    const long long t0 = clock64();
    while (!bar_try(efull + 8 * sb, sph) && clock64() - t0 < kWaitCycles / 8) {
    }
    if (++sb == ring) {
      sb = 0;
      sph ^= 1;
    }
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// OF_FP4: a warp each for bringing and for storing (a tile's products are a
// quarter of bf16's there, and its boxes have to keep up), with a barrier for
// slots that have been read out.
template <int MODE, int FORM>
__device__ __forceinline__ void box_bring(const BoxMaps& maps, const ProductK& k, const TileK& g,
                                          uint32_t boxes, uint32_t efull, uint32_t bfree,
                                          int first, int tiles, int step, uint32_t half,
                                          int split, volatile int* dead) {
  constexpr bool wide = FORM == BOX_F32;
  constexpr int W = wide ? 32 : 64;
  const uint32_t ring = g.boxes, second = g.two_slots ? kSlot : 0, chunk_bytes = kSlot + second;
  constexpr uint32_t narrow = wide ? kSlot / 2 : kSlot;  // a bf16 box
  const BoxEpi e = box_epi<MODE>(k.epi);
  const uint32_t bytes = (e.gate ? narrow : 0) + (e.residual || e.old ? kSlot : 0) +
                         (MODE == LIN_DINPUT && e.pre ? narrow : 0);
  const int64_t cols = k.cols;
  ChunkWalk<W> in(g, cols, split, first, tiles, step);
  uint32_t lb = 0, lph = 1, issued = 0;
  bool live = true;
  while (in.w.t < tiles) {
    live = bar_wait(bfree + 8 * lb, lph, dead);
    live = __all_sync(0xffffffffu, live);
    if (!live) break;
    const uint32_t at = boxes + lb * chunk_bytes, slot1 = at + second, bar = efull + 8 * lb;
    const int x = in.w.tj * g.bn + in.cc * W, y = in.w.ti * 256 + (int)half * kRowsCta;
    if (elect()) {
      bar_expect(bar, bytes);
      if constexpr (MODE == LIN_FORWARD) {
        if (e.gate) box_load(&maps.gate, at, x, y, bar);
        if (e.residual) box_load(&maps.extra, slot1, x, y, bar);
      } else {
        if (e.pre) box_load(&maps.pre, wide ? slot1 : at, x, y, bar);
        if (e.gate) box_load(&maps.gate, wide ? slot1 + kSlot / 2 : slot1, x, y, bar);
      }
    }
    __syncwarp();
    ++issued;
    if (++lb == ring) {
      lb = 0;
      lph ^= 1;
    }
    in.next(g, cols, split, tiles, step);
  }
  // after a wait that gave up: the boxes in flight land before the CTA returns
  for (uint32_t q = issued > ring ? issued - ring : 0; !live && q < issued; ++q) {
    const long long t0 = clock64();
    while (!bar_try(efull + 8 * (q % ring), (q / ring) & 1) && clock64() - t0 < kWaitCycles / 8) {
    }
  }
}
template <int MODE, int FORM>
__device__ __forceinline__ void box_put(const BoxMaps& maps, const ProductK& k, const TileK& g,
                                        uint32_t boxes, uint32_t edone, uint32_t bfree, int first,
                                        int tiles, int step, uint32_t half, int split,
                                        volatile int* dead) {
  constexpr bool wide = FORM == BOX_F32;
  constexpr int W = wide ? 32 : 64;
  const uint32_t ring = g.boxes, second = g.two_slots ? kSlot : 0, chunk_bytes = kSlot + second;
  const BoxEpi e = box_epi<MODE>(k.epi);
  const int64_t rows = k.rows, cols = k.cols;
  ChunkWalk<W> out(g, cols, split, first, tiles, step);
  uint32_t sb = 0, sph = 0;
  while (out.w.t < tiles) {
    bool live = bar_wait(edone + 8 * sb, sph, dead);
    live = __all_sync(0xffffffffu, live);  // the lanes leave together
    if (!live) break;
    const uint32_t at = boxes + sb * chunk_bytes, slot1 = at + second;
    const int x = out.w.tj * g.bn + out.cc * W, y = out.w.ti * 256 + (int)half * kRowsCta;
    if (elect()) {
      if (y < rows) {
        if constexpr (MODE == LIN_FORWARD) {
          if (e.pre) box_store(&maps.pre, at, x, y);
          box_store(&maps.out, slot1, x, y);
        } else {
          if (e.dgate) box_store(&maps.extra, wide ? slot1 + kSlot / 2 : slot1, x, y);
          box_store(&maps.out, at, x, y);
        }
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      bar_arrive(bfree + 8 * sb);
    }
    __syncwarp();
    if (++sb == ring) {
      sb = 0;
      sph ^= 1;
    }
    out.next(g, cols, split, tiles, step);
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// The same for rows off 16-byte boundaries: a lane takes one column and its 32
// rows, so that a warp's accesses of a row are consecutive whatever its
// alignment.
struct Column {
  int64_t row, col;
  int count;  // rows this lane has: 0 outside the columns
};
__device__ __forceinline__ bool column_in(const Mat& m, const Column& c, int i, const Extent& e) {
  const int64_t at = (c.row + i) * m.ld;
  return in_extent(at + c.col, at + c.col + 1, at, at + e.cols, ZERO_SITE_LINEAR_OUT) &&
         in_extent(c.row + i, c.row + i + 1, 0, e.rows, ZERO_SITE_LINEAR_OUT);
}
// Past its rows a lane reads the last one again: loads without a condition
// each are all in flight together (7615 x 80 by 4624 with SiLU, a gate and its
// input kept, odd rows: 242 us, 289 with conditions).
template <int R, typename T>
__device__ __forceinline__ void column_words(const T* p, const Mat& m, const Column& c, int i0,
                                             const Extent& e, T u[R]) {
  const int last = c.count - 1;
  int i = i0 < last ? i0 : last;
  p += (c.row + i) * m.ld + c.col;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    u[j] = column_in(m, c, i, e) ? *p : T(0);
    const bool on = i < last;
    p += on ? m.ld : 0;
    i += on;
  }
}
template <int R>
__device__ __forceinline__ void column_load(const Mat& m, const Column& c, int i0,
                                            const Extent& e, float f[R]) {
  if (c.count <= 0) return;
  if (m.dtype == ZERO_F32) {
    column_words<R>(static_cast<const float*>(m.p), m, c, i0, e, f);
  } else {
    uint16_t u[R];
    column_words<R>(static_cast<const uint16_t*>(m.p), m, c, i0, e, u);
#pragma unroll
    for (int j = 0; j < R; ++j) f[j] = __uint_as_float((uint32_t)u[j] << 16);
  }
}
template <int R>
__device__ __forceinline__ void column_store(const Mat& m, const Column& c, int i0,
                                             const Extent& e, const float f[R]) {
  const int64_t at = (c.row + i0) * m.ld + c.col;
  if (m.dtype == ZERO_F32) {
    float* p = static_cast<float*>(m.p) + at;
#pragma unroll
    for (int j = 0; j < R; ++j, p += m.ld)
      if (i0 + j < c.count && column_in(m, c, i0 + j, e)) *p = f[j];
  } else {
    uint16_t* p = static_cast<uint16_t*>(m.p) + at;
#pragma unroll
    for (int j = 0; j < R; ++j, p += m.ld)
      if (i0 + j < c.count && column_in(m, c, i0 + j, e)) *p = to_bf16(f[j]);
  }
}

// R rows at a time.  `keep` holds the mask as finish_block would use it.
template <int MODE, int R, bool SIDES>
__device__ __forceinline__ void finish_columns(const EpiK& k, uint32_t keep, uint32_t patch,
                                               uint32_t biases, int64_t row0, int64_t col0,
                                               const Extent& e, int lane) {
  Column c;
  c.row = row0;
  c.col = col0 + lane;
  c.count = c.col >= e.cols ? 0 : (int)(e.rows - row0 < 32 ? e.rows - row0 : 32);
  float bias = 0.0f;
  if (MODE == LIN_FORWARD && k.bias.p)
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(bias) : "r"(biases + (uint32_t)lane * 4));
#pragma unroll 1
  for (int i0 = 0; i0 < 32 && row0 + i0 < e.rows; i0 += R) {
    float v[R], f[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(v[i])
                   : "r"(patch + ((i0 + i) * 36 + lane) * 4));
    if constexpr (MODE == LIN_FORWARD) {
#pragma unroll
      for (int i = 0; i < R; ++i) v[i] += bias;
      if (SIDES && k.pre.p) column_store<R>(k.pre, c, i0, e, v);
      activate<R>(v, k.act);
      if (SIDES && k.gate.p) {
        column_load<R>(k.gate, c, i0, e, f);
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] *= f[i];
      }
      if (k.drop.on) {
#pragma unroll
        for (int i = 0; i < R; ++i) {  // the lane and bit that hold this element
          const uint32_t m = __shfl_sync(0xffffffffu, keep, (i & 7) << 2 | lane >> 3);
          v[i] = m >> (31 - ((i0 + i) >> 3) * 8 - (lane & 7)) & 1 ? v[i] * k.drop.scale : 0.0f;
        }
      }
      if (SIDES && k.residual.p) {
        column_load<R>(k.residual, c, i0, e, f);
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] += f[i];
      }
    } else if constexpr (MODE == LIN_DINPUT) {
      if (SIDES && k.pre.p) {
        column_load<R>(k.pre, c, i0, e, f);
        float slope[R];
        activate_grad<R>(f, slope, k.act);
        if (SIDES && k.gate.p) {
          if (k.dgate.p) {
#pragma unroll
            for (int i = 0; i < R; ++i) f[i] *= v[i];
            column_store<R>(k.dgate, c, i0, e, f);
          }
          column_load<R>(k.gate, c, i0, e, f);
#pragma unroll
          for (int i = 0; i < R; ++i) slope[i] *= f[i];
        }
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] *= slope[i];
      }
    } else {
      if (SIDES && k.accumulate) {
        column_load<R>(k.out, c, i0, e, f);
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] += f[i];
      }
    }
    column_store<R>(k.out, c, i0, e, v);
  }
}

// Without side operands 32 rows in one go (768 to 50257 fp32: 45 us, 49 by 16
// rows); with them 16, as 32 leave too few registers (gradient of 4868 x 1134
// inputs through 192 outputs and a gated GELU: 50.5 us, 53.7 by 32 rows).
template <int MODE>
__device__ __forceinline__ void finish_any_columns(const EpiK& k, uint32_t keep, uint32_t patch,
                                                   uint32_t biases, int64_t row0, int64_t col0,
                                                   const Extent& e, int lane) {
  const bool sides = MODE == LIN_FORWARD  ? k.pre.p || k.gate.p || k.residual.p
                     : MODE == LIN_DINPUT ? k.pre.p != nullptr
                                          : k.accumulate != 0;
  if (sides)
    finish_columns<MODE, 16, true>(k, keep, patch, biases, row0, col0, e, lane);
  else
    finish_columns<MODE, 32, false>(k, keep, patch, biases, row0, col0, e, lane);
}

// Dropout's masks of a thread's share of a tile, 32 elements each: drawn while
// the tile's products are still running, on warps that otherwise wait.
struct Masks {
  uint32_t m0, m1, m2, m3;  // highest bit first
  __device__ __forceinline__ uint32_t at(int q) const {
    return q < 2 ? (q == 0 ? m0 : m1) : (q == 2 ? m2 : m3);
  }
  __device__ __forceinline__ void set(int q, uint32_t m) {
    if (q == 0) m0 = m;
    if (q == 1) m1 = m;
    if (q == 2) m2 = m;
    if (q == 3) m3 = m;
  }
};

// ---------------------------------------------------------------------------
// A contraction split in two: both pairs of a cluster hold sums of the whole
// tile.  Each pair finishes half of its pieces; it writes the sums of the
// other half into the memory of the partner's CTA with the same rows (the
// operand ring, free by then) and adds what it finds in its own.  Two addends:
// the same result whichever pair adds.  A warp's piece of N columns takes
// 128 N bytes, 16-byte units of consecutive threads side by side.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool owns_piece(int split, int piece, int pieces, int w) {
  return (pieces == 1 ? (w & 1) : (int)(piece >= pieces / 2)) == split;
}
// Where the owner of a piece finds the other's sums: its own pieces in order,
// then those of the bias (piece == pieces): at most 80 KiB of the ring, which
// has 96 at least.
template <int N>
__device__ __forceinline__ uint32_t part_at(uint32_t ring, int piece, int pieces, int w,
                                            int lane) {
  const int half = pieces > 1 ? pieces / 2 : 1;
  const int at = piece == pieces ? half : piece % half;
  return ring + (uint32_t)((at * 4 + w) * (N * 128) + lane * 16);
}
template <int N>
__device__ __forceinline__ void push_part(uint32_t there, const uint32_t r[N]) {
#pragma unroll
  for (int u = 0; u < N / 4; ++u) st_cluster4(there + u * 512, r + 4 * u);
}
template <int N>
__device__ __forceinline__ void add_part(uint32_t here, uint32_t r[N]) {
#pragma unroll
  for (int u = 0; u < N / 4; ++u) {
    const float4 x = ld_shared4(here + u * 512);
    r[4 * u] = __float_as_uint(__uint_as_float(r[4 * u]) + x.x);
    r[4 * u + 1] = __float_as_uint(__uint_as_float(r[4 * u + 1]) + x.y);
    r[4 * u + 2] = __float_as_uint(__uint_as_float(r[4 * u + 2]) + x.z);
    r[4 * u + 3] = __float_as_uint(__uint_as_float(r[4 * u + 3]) + x.w);
  }
}

// The gradient of bias element i.
__device__ __forceinline__ void store_bias(const ProductK& k, const TileK& g, int64_t i,
                                           float v) {
  const int64_t n = g.bias_b ? k.cols : k.rows;
  if (i >= n || !in_extent(i, i + 1, 0, n, ZERO_SITE_LINEAR_OUT)) return;
  if (k.epi.accumulate) v += load1(k.dbias, i);
  store1(k.dbias, i, v);
}

// Scale tiles from `column`'s tiles on, `rows_tile` down, of a step's depth.
__device__ __forceinline__ void scales_load(const CUtensorMap* map, uint32_t dst, int column,
                                            int rows_tile, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(column), "r"(rows_tile), "r"(cluster_bar)
      : "memory");
}
// One scale tile of both CTAs from shared memory to four columns of tensor
// memory: row r of the tile in lane r % 32, column r / 32, for each of the four
// groups of 32 lanes.  Runs in order with the products issued before and after.
__device__ __forceinline__ void scales_copy(uint32_t column, uint32_t tile) {
  const uint64_t desc = (uint64_t)((tile & 0x3FFFF) >> 4) | (1ull << 16) | (8ull << 32) |
                        (1ull << 46);  // 8-row groups 128 bytes apart, no swizzle
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(column), "l"(desc)
               : "memory");
}
// 64 codes of every row: four scales each (blocks of 16), or two (32).
template <bool NV>
__device__ __forceinline__ void mma_pair_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t scale_a, uint32_t scale_b, uint32_t add) {
  if constexpr (NV)
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X "
        "[%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"(add)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"(add)
        : "memory");
}
// The products of a stage, 256 deep.  The scales of 128 (MX) or 64 (NV) codes
// of 128 rows make a tile; CHUNKS tiles over B's columns, which begin `shift`
// rows of 32 into theirs.  Straight code: what issues these instructions is
// the bottleneck otherwise (a step of 256 x 192, NV: 1184 cycles with a loop
// over the chunks, 596 without, 470 in a loop that one thread runs alone).
template <bool NV, int CHUNKS>
__device__ __forceinline__ void mma_stage_fp4(uint32_t d, uint32_t tmem, uint64_t da, uint64_t db,
                                              uint32_t scales, uint32_t shift, uint32_t bn,
                                              bool first) {
  constexpr uint32_t deep = NV ? 4 : 2;
  const uint32_t sa = tmem + kScaleColumn, sb = sa + 4 * deep;
#pragma unroll
  for (uint32_t t = 0; t < deep; ++t) {
    scales_copy(sa + 4 * t, scales + t * kScaleTile);
    scales_copy(sb + 8 * t, scales + (deep + t) * kScaleTile);
    if (CHUNKS > 1) scales_copy(sb + 8 * t + 4, scales + (2 * deep + t) * kScaleTile);
  }
  // E2M1 both, M = 256; MX: scales E8M0, of which a product takes the first or
  // second two of a tile's four
  const uint32_t idesc = (1u << 7) | (1u << 10) | ((bn >> 3) << 17) | ((NV ? 0u : 1u) << 23) |
                         (2u << 27);
#pragma unroll
  for (uint32_t q = 0; q < 4; ++q) {
    const uint32_t t = NV ? q : q / 2, half = NV ? 0u : 2u * (q & 1);
    mma_pair_fp4<NV>(d, da + 2 * q, db + 2 * q, idesc | (half << 4) | (half << 29), sa + 4 * t,
                     sb + 8 * t + shift, !first || q > 0);
  }
}

// The operands' ring as one thread loads or multiplies it: a stage and its phase.
struct RingFp4 {
  uint32_t at, full, empty, stages, stage_bytes;
  uint32_t s = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == stages) {
      s = 0;
      ph ^= 1;
    }
  }
};
// All of a CTA's copies by one thread: its rows of A and of B, its scales of A and
// the pair's of B.  (A warp whose lanes met at every step, one of them issuing,
// bounded steps: 8192 x 11008 x 4096 152 us, now 124, 2048 x 2048 x 8192 24.7 and 20.8.)
static __device__ __forceinline__ void load_fp4(RingFp4 r, const CUtensorMap& map_a,
                                                const CUtensorMap& map_b,
                                                const CUtensorMap& map_sa,
                                                const CUtensorMap& map_sb, const TileK& g,
                                                int first, int clusters, int tiles, int kb0,
                                                int kb1, int half, uint32_t full_lead,
                                                volatile int* dead) {
  const int bn = g.bn, deep = g.scale_deep;
  const uint32_t b_bytes = (uint32_t)bn * kDeep;
  const uint32_t bytes = 2 * (kBytesA + b_bytes + g.scale_bytes);
  bool live = true;
  for (TileWalk walk(g, first); live && walk.t < tiles; walk.next(g, clusters)) {
    const int i0 = walk.ti * 256 + half * kRowsCta, j0 = walk.tj * bn + half * (bn / 2);
    const int rows = walk.ti * 2 + half, cols = walk.tj * bn / kRowsCta;
    for (int kb = kb0; kb < kb1; ++kb) {
      live = bar_wait(r.empty + 8 * r.s, r.ph ^ 1, dead);
      if (!live) break;
      const uint32_t a_at = r.at + r.s * r.stage_bytes, b_at = a_at + kBytesA;
      const uint32_t bar = full_lead + 8 * r.s, scales = b_at + b_bytes;
      if (half == 0) bar_expect(r.full + 8 * r.s, bytes);
      tma_load(&map_a, a_at, kb * kDeep, i0, bar);
      tma_load(&map_b, b_at, kb * kDeep, j0, bar);
      scales_load(&map_sa, scales, kb * deep, rows, bar);
      scales_load(&map_sb, scales + deep * kScaleTile, kb * deep, cols, bar);
      r.next();
    }
  }
  // a wait gave up: let the loads in flight land before the CTAs return (stages
  // before this one hold its phase, the others the one before)
  if (!live && half == 0)
    for (uint32_t q = 0; q < r.stages; ++q) {
      const long long t0 = clock64();
      while (!bar_try(r.full + 8 * q, q < r.s ? r.ph : r.ph ^ 1) &&
             clock64() - t0 < kWaitCycles / 8) {
      }
    }
}
// All of a pair's products, by one thread.
template <bool NV, int CHUNKS>
__device__ __forceinline__ void multiply_fp4(RingFp4 r, const TileK& g, int first, int clusters,
                                             int tiles, int kb0, int kb1, uint32_t tmem,
                                             uint32_t tfull, uint32_t tempty, uint16_t mask,
                                             volatile int* dead) {
  const uint32_t bn = g.bn, sets = g.acc_sets, step = r.stage_bytes >> 4;
  const int round = g.round, rounds = rounds_of(g, kb1 - kb0);
  const uint64_t a0 = operand_desc(r.at, true), b0 = operand_desc(r.at + kBytesA, true);
  uint32_t acc = 0, aph = 0;
  for (TileWalk walk(g, first); walk.t < tiles; walk.next(g, clusters)) {
    const uint32_t shift = (uint32_t)walk.tj * bn % kRowsCta / 32;
    int kb = kb0;
    for (int q = 0; q < rounds; ++q) {
      if (!bar_wait(tempty + 8 * acc, aph ^ 1, dead)) return;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int start = kb, end = q + 1 < rounds ? kb + round : kb1;
      for (; kb < end; ++kb) {
        if (!bar_wait(r.full + 8 * r.s, r.ph, dead)) return;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t stage = (uint64_t)(r.s * step);  // descriptors count 16 bytes
        mma_stage_fp4<NV, CHUNKS>(tmem + acc * bn, tmem, a0 + stage, b0 + stage,
                                  r.at + r.s * r.stage_bytes + kBytesA + bn * kDeep, shift, bn,
                                  kb == start);
        commit_pair(r.empty + 8 * r.s, mask);
        r.next();
      }
      commit_pair(tfull + 8 * acc, mask);
      if (++acc == sets) {
        acc = 0;
        aph ^= 1;
      }
    }
  }
}

template <int MODE, int FORM, int KIND>
__global__ void __launch_bounds__(threads_of(FORM), 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ typename MapsOf<FORM, KIND>::type maps,
                   const __grid_constant__ ProductK k,
                   const __grid_constant__ TileK g) {
  constexpr bool GEN = FORM == PATCH_GEN, BOX = FORM == BOX_BF16 || FORM == BOX_F32;
  constexpr bool FP4 = KIND == OF_FP4;
  constexpr int kOwn = 1 + MODE * 8 + FORM * 2 + KIND;  // a slow wait of its own (see bar_wait)
  constexpr int kWidth = FORM == BOX_F32 ? 32 : 64;  // columns of a chunk
  // The epilogue's warps in sets of four (one per 32 rows); a set takes every
  // kSets-th piece of kPiece columns of a tile.  Boxes want twice the warps,
  // as half of their time is latency (8192 x 1024 x 4096 with a GELU gradient:
  // 63 us with 8, 51 with 16); patches want the registers (509 x 768 to 50257
  // fp32: 45 us with 8, 53 with 16).
  constexpr int kEpiWarps = BOX ? kBoxWarps : kPatchWarps;
  constexpr int kPiece = BOX ? 16 : 32, kSets = kEpiWarps / 4;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5 + (FP4 ? 3 : 2) * kMostBoxes];
  __shared__ __align__(8) uint64_t raw_bars[GEN ? 2 * kMostRaw : 1];
  __shared__ uint32_t tmem_at;
  __shared__ int dead;
  const uint32_t rank = cluster_rank(), half = rank & 1, leader = rank & ~1u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = (int)(rank >> 1), S = g.splits;
  const uint32_t stage_bytes =
      kBytesA + g.bn * kDeep + (FP4 ? g.scale_bytes : 0);  // bn / 2 rows of 128 bytes
  const uint32_t ring = smem_u32(smem);
  const uint32_t patches = ring + g.stages * stage_bytes;
  const uint32_t ones = patches + (BOX ? g.boxes * kSlot * (g.two_slots ? 2 : 1)
                                       : kPatchWarps * kPatch * 4);
  const uint32_t bias_smem = ones + (g.bias_tiles || g.bias_fused ? kOnesBytes : 0);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxStages;
  const uint32_t tfull = empty + 8 * kMaxStages, tempty = tfull + 16, ready = tempty + 16;
  const uint32_t efull = ready + 8, edone = efull + 8 * kMostBoxes;
  const uint32_t bfree = edone + 8 * kMostBoxes;  // OF_FP4
  const uint32_t landed = smem_u32(raw_bars), used = landed + 8 * kMostRaw;  // raw buffers

  if (warp == 0 && elect()) {
    dead = 0;
    for (int s = 0; s < g.stages; ++s) {
      bar_init(full + 8 * s, GEN ? 1 + 2 * kGenWarps : 1);
      bar_init(empty + 8 * s, 1);
    }
    if (GEN)
      for (int q = 0; q < g.raws; ++q) {
        bar_init(landed + 8 * q, 2);
        bar_init(used + 8 * q, kGenWarps);
      }
    for (int a = 0; a < 2; ++a) {
      bar_init(tfull + 8 * a, 1);
      bar_init(tempty + 8 * a, 2 * kEpiWarps);
    }
    bar_init(ready, 2);  // tensor memory of both CTAs
    if (BOX)
      for (int b = 0; b < g.boxes; ++b) {
        bar_init(efull + 8 * b, 1);
        bar_init(edone + 8 * b, kEpiWarps);
        if (FP4) bar_init(bfree + 8 * b, 1);
      }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (MODE == LIN_DWEIGHT && (g.bias_tiles || g.bias_fused) && warp == 3) {
    for (int q = lane; q < kOnesBytes / 16; q += 32)  // bf16 1.0 twice
      asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(ones + q * 16),
                   "r"(0x3F803F80u)
                   : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncwarp();
  cluster_arrive();  // this CTA's barriers are ready; what follows needs no other CTA
  // the next kernel on the stream may set up while this one runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 1 && elect()) {
    // (an operand off 16-byte boundaries, or an empty one, has no such map)
    if (!g.gen_a && g.kblocks > 0 && k.rows > 0)
      asm volatile("prefetch.tensormap [%0];" ::"l"(&map_a) : "memory");
    if (!g.gen_b && g.kblocks > 0 && k.cols > 0)
      asm volatile("prefetch.tensormap [%0];" ::"l"(&map_b) : "memory");
    if constexpr (BOX) asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.out) : "memory");
    if constexpr (FP4) {
      if (g.kblocks > 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.scale_a) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.scale_b) : "memory");
      }
    }
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_at)),
                 "r"(g.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  // this cluster's tiles, and this pair's share of the contraction
  const int clusters = g.clusters, first = (int)(blockIdx.x >> (1 + g.split_log2));
  const int tiles = g.tiles_i * g.tiles_j + g.bias_tiles;
  const int kb0 = (int)(((int64_t)g.kblocks * split) >> g.split_log2);
  const int kb1 = (int)(((int64_t)g.kblocks * (split + 1)) >> g.split_log2);
  const bool a_c = k.a_c, b_c = k.b_c;
  // fetched before the wait, not when first used after it
  asm volatile("" ::"r"(clusters), "r"(first), "r"(tiles), "r"(kb0), "r"(kb1), "r"((int)a_c),
               "r"((int)b_c), "r"(g.stages), "r"(g.gen_a), "r"(g.gen_b), "r"(g.i_fast));
  cluster_wait();
  if (warp == 2) {
    if (elect()) bar_arrive_cluster(remote(ready, leader));
    __syncwarp();
  }
  // what ran before this on the stream is done and its writes are visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint32_t tmem = 0;
  if (warp == 1 || warp == 2 || (warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps)) {
    asm volatile("bar.sync 1, %0;" ::"n"((kEpiWarps + 2) * 32) : "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem = *(volatile uint32_t*)&tmem_at;
  }
  // The last barrier of the cluster, at which nobody signals another CTA or
  // reads its memory any more: warp 3 only moves this CTA's own boxes.
  const bool early = BOX && warp == 3 && S == 1;
  if (early) cluster_arrive();
  int barriers = 0;  // of a split's two, passed so far

  if (FP4 && warp == 0) {
    if constexpr (FP4)
      if (elect())
        load_fp4(RingFp4{ring, full, empty, (uint32_t)g.stages, stage_bytes}, map_a, map_b,
                 maps.scale_a, maps.scale_b, g, first, clusters, tiles, kb0, kb1, (int)half,
                 remote(full, leader), &dead);
    __syncwarp();
  } else if (FP4 && warp == 1) {
    if constexpr (FP4) {
      if (half == 0) {
        const uint16_t mask = (uint16_t)(3u << leader);
        const RingFp4 r{ring, full, empty, (uint32_t)g.stages, stage_bytes};
        const bool live = bar_wait<kOwn>(ready, 0, &dead);
        const bool nv = g.scale_deep == 4, two = g.scale_chunks == 2;
        if (elect() && live) {
          if (nv && two)
            multiply_fp4<true, 2>(r, g, first, clusters, tiles, kb0, kb1, tmem, tfull, tempty,
                                  mask, &dead);
          else if (nv)
            multiply_fp4<true, 1>(r, g, first, clusters, tiles, kb0, kb1, tmem, tfull, tempty,
                                  mask, &dead);
          else if (two)
            multiply_fp4<false, 2>(r, g, first, clusters, tiles, kb0, kb1, tmem, tfull, tempty,
                                   mask, &dead);
          else
            multiply_fp4<false, 1>(r, g, first, clusters, tiles, kb0, kb1, tmem, tfull, tempty,
                                   mask, &dead);
        }
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    const uint32_t full_lead = remote(full, leader);
    const uint32_t stages = g.stages, b_bytes = (uint32_t)g.bn * kDeep;
    const int bn = g.bn, blocks_b = bn / 128;
    const bool tma_a = g.gen_a == 0, tma_b = g.gen_b == 0, bias_b = g.bias_b;
    uint32_t s = 0, ph = 0, end_s = 0, end_ph = 0;  // end: where a wait gave up
    bool live = true;
    for (TileWalk walk(g, first); walk.t < tiles; walk.next(g, clusters)) {
      const int ti = walk.ti, tj = walk.tj;
      const int i0 = ti * 256 + (int)half * kRowsCta;
      const int j0 = tj * bn + (int)half * (bn / 2);
      const bool load_a = tj < 0 && bias_b ? tma_b : tma_a;
      const bool load_b = tma_b && tj >= 0;
      // The second CTA's warp stops where it has nothing to load (and so
      // nothing in the tiles after it): no stage waits for it there, so it
      // could fall two phases behind and wait for one that never comes.
      if (half != 0 && !load_a && !load_b) break;
      const CUtensorMap* map_i = tj < 0 && bias_b ? &map_b : &map_a;
      const uint32_t bytes = 2 * ((load_a ? kBytesA : 0) + (load_b ? b_bytes : 0));
      for (int kb = kb0; kb < kb1; ++kb) {
        if (live) {
          live = bar_wait<kOwn>(empty + 8 * s, ph ^ 1, &dead);
          end_s = s;
          end_ph = ph;
        }
        const uint32_t a_at = ring + s * stage_bytes, b_at = a_at + kBytesA;
        const uint32_t bar = full_lead + 8 * s;
        const int c = kb * kDeep;
        if (elect() && live) {
          if (half == 0) bar_expect(full + 8 * s, bytes);
          if (load_a) {
            if (a_c) {
              tma_load(map_i, a_at, c, i0, bar);
            } else {
              tma_load(map_i, a_at, i0, c, bar);
              tma_load(map_i, a_at + 8192, i0 + 64, c, bar);
            }
          }
          if (load_b) {
            if (b_c) {
              tma_load(&map_b, b_at, c, j0, bar);
            } else {
              tma_load(&map_b, b_at, j0, c, bar);
              if (blocks_b > 1) tma_load(&map_b, b_at + 8192, j0 + 64, c, bar);
            }
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
    // (a ring slot holds at most one load, those from end_s on the lap before's;
    // waits are again limited)
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
      const uint16_t mask = (uint16_t)(3u << leader);
      // fp32 sums of bf16 values, M = 256; N = bn, or 32 columns of ones
      const uint32_t base = (1u << 4) | (1u << 7) | (1u << 10) | ((a_c ? 0u : 1u) << 15) |
                            (16u << 24);
      const uint32_t idesc_n = base | ((b_c ? 0u : 1u) << 16) | ((uint32_t)(g.bn >> 3) << 17);
      const uint32_t idesc_1 = base | (4u << 17);
      const uint32_t step_a = a_c ? 2 : 128, step_b = b_c ? 2 : 128;  // 16 deep, in 16 bytes
      const uint32_t stages = g.stages, bn = g.bn, sets = g.acc_sets;
      const int round = g.round, rounds = rounds_of(g, kb1 - kb0);
      const bool fused = MODE == LIN_DWEIGHT && g.bias_fused, bias_b = g.bias_b;
      uint32_t s = 0, ph = 0, acc = 0, aph = 0;
      bool live = bar_wait<kOwn>(ready, 0, &dead);
      for (TileWalk walk(g, first); walk.t < tiles; walk.next(g, clusters)) {
        const int ti = walk.ti, tj = walk.tj;
        const bool sums = fused && (bias_b ? ti : tj) == 0;
        const uint32_t idesc = tj >= 0 ? idesc_n : idesc_1, sb = tj >= 0 ? step_b : 0;
        int kb = kb0;
        for (int r = 0; r < rounds; ++r) {
          live = live && bar_wait<kOwn>(tempty + 8 * acc, aph ^ 1, &dead);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t d = tmem + acc * bn, d_bias = tmem + bias_column(g, acc);
          const int start = kb, end = r + 1 < rounds ? kb + round : kb1;
          for (; kb < end; ++kb) {
            live = live && bar_wait<kOwn>(full + 8 * s, ph, &dead);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t a_at = ring + s * stage_bytes;
            const uint64_t da = operand_desc(a_at, a_c);
            const uint64_t db = tj >= 0 ? operand_desc(a_at + kBytesA, b_c)
                                        : operand_desc(ones, true);
            if (elect() && live) {
#pragma unroll
              for (int q = 0; q < kDeep / 16; ++q)
                mma_pair(d, da + q * step_a, db + q * sb, idesc, kb > start || q > 0);
              if (MODE == LIN_DWEIGHT && sums) {
                const uint64_t dr = operand_desc(bias_b ? a_at + kBytesA : a_at, a_c);
                const uint64_t d1 = operand_desc(ones, true);
#pragma unroll
                for (int q = 0; q < kDeep / 16; ++q)
                  mma_pair(d_bias, dr + q * step_a, d1, idesc_1, kb > start || q > 0);
              }
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
          if (++acc == sets) {
            acc = 0;
            aph ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (BOX && (warp == 3 || (FP4 && warp == 2))) {
    for (; S > 1 && barriers < 2; ++barriers) {  // its boxes come after the exchange
      cluster_arrive();
      cluster_wait();
    }
    if constexpr (BOX && FP4) {
      if (warp == 2)
        box_bring<MODE, FORM>(maps, k, g, patches, efull, bfree, first, tiles, clusters, half,
                              split, &dead);
      else
        box_put<MODE, FORM>(maps, k, g, patches, edone, bfree, first, tiles, clusters, half, split,
                            &dead);
    } else if constexpr (BOX) {
      box_traffic<MODE, FORM>(maps, k, g, patches, efull, edone, first, tiles, clusters, half,
                              split, &dead);
    }
    __syncwarp();
  } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps) {
    const int w = (warp - kEpiWarp0) & 3, set = (warp - kEpiWarp0) >> 2;  // lanes 32 w...
    const uint32_t tempty_lead = remote(tempty, leader);
    const Extent e{k.out_t ? k.cols : k.rows, k.out_t ? k.rows : k.cols};
    const uint64_t offset =
        MODE == LIN_FORWARD && k.epi.drop.on ? drop_offset(k.epi.drop) : 0ull;
    const uint32_t mine = patches + (uint32_t)(warp - kEpiWarp0) * kPatch * 4;
    const BoxEpi be = box_epi<MODE>(k.epi);
    // this warp's biases of a tile, those of its pieces in a row
    const uint32_t biases = bias_smem + (uint32_t)(warp - kEpiWarp0) * (kPiece * 16);
    const DropK& drop = k.epi.drop;
    const bool empty_sum = kb1 == kb0, out_t = k.out_t;
    const uint32_t boxes = g.boxes, boxes0 = patches, second = g.two_slots ? kSlot : 0,
                   chunk_bytes = kSlot + second;
    const int bn = g.bn, rounds = rounds_of(g, kb1 - kb0);
    const uint32_t sets = g.acc_sets;
    const int64_t cols = k.cols, rows = k.rows;
    // what both operands' tensors are scaled by
    const float whole = FP4 ? (k.whole_a ? *(volatile const float*)k.whole_a : 1.0f) *
                                  (k.whole_b ? *(volatile const float*)k.whole_b : 1.0f)
                            : 1.0f;
    uint32_t acc = 0, aph = 0, eb = 0, eph = 0;
    bool ok = true;
    for (TileWalk walk(g, first); walk.t < tiles && ok; walk.next(g, clusters)) {
      const int ti = walk.ti, tj = walk.tj;
      const int64_t i0 = (int64_t)ti * 256 + half * kRowsCta + w * 32;
      const int pieces = tj >= 0 ? bn / kPiece : 1;
      // While the products run: the biases and dropout masks of this warp's
      // pieces, the q-th being piece kSets q + set.
      if (MODE == LIN_FORWARD && be.bias) {
        for (int q = 0; kSets * q + set < pieces; ++q) {
          const int64_t c =
              (out_t ? i0 : (int64_t)tj * bn + (kSets * q + set) * kPiece) + lane;
          const bool in = c < e.cols && lane < kPiece &&
                          in_extent(c, c + 1, 0, e.cols, ZERO_SITE_LINEAR_IN);
          const float b = in ? load1(k.epi.bias, c) : 0.0f;
          if (lane < kPiece)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(biases + (uint32_t)(q * kPiece + lane) * 4),
                         "f"(b));
        }
        __syncwarp();
      }
      Masks masks{};
      if (MODE == LIN_FORWARD && drop.on) {
#pragma unroll 1
        for (int q = 0; kSets * q + set < pieces; ++q) {
          const int piece = kSets * q + set;
          const int64_t j0 = (int64_t)tj * bn + piece * kPiece;
          if (i0 >= rows || j0 >= cols) break;
          if (S > 1 && !owns_piece(split, piece, pieces, w)) continue;
          if (BOX) {
            masks.set(q, keep_mask<4, 4>(drop, offset, (uint32_t)(i0 + lane), 0, j0));
          } else {
            const Block b = block_of(out_t ? j0 : i0, out_t ? i0 : j0, e, lane);
            masks.set(q, keep_mask<8, 2>(drop, offset, (uint32_t)b.row, 8, b.col));
          }
        }
      }
      const bool sums =
          MODE == LIN_DWEIGHT && g.bias_fused && (g.bias_b ? ti : tj) == 0 && set == 0;
      const uint32_t lanes = tmem + ((uint32_t)(w * 32) << 16);
      const uint32_t summed = lanes + sum_column(g);
      float bias_sum = 0.0f;
      // rounds before the last: their sums leave the tensor cores' set, which
      // a later round writes again, for a set of their own
      for (int r = 1; r < rounds && ok; ++r) {
        ok = bar_wait<kOwn>(tfull + 8 * acc, aph, &dead);
        ok = __all_sync(0xffffffffu, ok);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int piece = set; piece < pieces; piece += kSets) {
          uint32_t v[kPiece];
          tmem_load<kPiece>(lanes + acc * bn + piece * kPiece, v);
          if (r > 1) tmem_add<kPiece>(summed + piece * kPiece, v);
          tmem_store<kPiece>(summed + piece * kPiece, v);
        }
        if (sums) {
          uint32_t v[16];
          tmem_load16(lanes + bias_column(g, acc), v);
          bias_sum += __uint_as_float(v[0]);
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive_fenced(tempty_lead + 8 * acc);
        if (++acc == sets) {
          acc = 0;
          aph ^= 1;
        }
      }
      if (!ok) break;
      ok = bar_wait<kOwn>(tfull + 8 * acc, aph, &dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = lanes + acc * bn;
      if (sums) {
        uint32_t v[16];
        tmem_load16(lanes + bias_column(g, acc), v);
        bias_sum += __uint_as_float(v[0]);
      }
      if (S > 1) {
        cluster_arrive();
        cluster_wait();  // both pairs' products are done: the rings are free
        for (int piece = set; piece < pieces; piece += kSets) {
          if (tj < 0 ? split == 0 : owns_piece(split, piece, pieces, w)) continue;
          uint32_t r[kPiece];
          tmem_load<kPiece>(d + piece * kPiece, r);
          if (rounds > 1) tmem_add<kPiece>(summed + piece * kPiece, r);
          push_part<kPiece>(remote(part_at<kPiece>(ring, piece, pieces, w, lane), rank ^ 2), r);
        }
        if (sums && split == 1)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                           remote(part_at<kPiece>(ring, pieces, pieces, w, lane), rank ^ 2)),
                       "f"(bias_sum));
        cluster_arrive();
        cluster_wait();
        barriers = 2;
      }
      // The sums of a piece: this round's, the rounds' before, the partner's.
      auto piece_sums = [&](int piece, float v[kPiece]) {
        uint32_t r[kPiece];
        tmem_load<kPiece>(d + piece * kPiece, r);
        if (rounds > 1) tmem_add<kPiece>(summed + piece * kPiece, r);
        if (S > 1) add_part<kPiece>(part_at<kPiece>(ring, piece, pieces, w, lane), r);
        if (empty_sum) {
#pragma unroll
          for (int q = 0; q < kPiece; ++q) v[q] = 0.0f;
          return;
        }
#pragma unroll
        for (int q = 0; q < kPiece; ++q)
          v[q] = FP4 ? __uint_as_float(r[q]) * whole : __uint_as_float(r[q]);
      };
      if (tj < 0) {  // a tile of bias sums: its first column
        if (set == 0 && (S == 1 || split == 0)) {
          float v[kPiece];
          piece_sums(0, v);
          store_bias(k, g, i0 + lane, v[0]);
        }
      } else if constexpr (BOX) {
        int cc, count;
        tile_chunks<kWidth>(g, cols, split, tj, cc, count);
        for (; cc < count; ++cc) {
          const uint32_t b = eb, bph = eph;
          if (++eb == boxes) {
            eb = 0;
            eph ^= 1;
          }
          // 64 columns are shared by all sets of epilogue warps, 32 by half.  The
          // other half passes the chunk's phases too: a wait names its phase
          // by parity alone, and one who skipped a phase of a slot would take
          // the phase before it for the one after.
          ok = bar_wait<kOwn>(efull + 8 * b, bph, &dead);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (kWidth == 32 && (cc & 1) != set >> 1) {
            if (lane == 0) bar_arrive(edone + 8 * b);
            continue;
          }
          const int piece = kWidth == 64 ? 4 * cc + set : 2 * cc + (set & 1);
          const int unit = kWidth == 64 ? 2 * set : 2 * (set & 1);  // of a bf16 row
          float v[kPiece];
          piece_sums(piece, v);
          box_piece<MODE, FORM>(be, masks.at(piece >> 2), boxes0 + b * chunk_bytes, second,
                               w * 32 + lane, unit, biases + (uint32_t)(piece >> 2) * (kPiece * 4),
                               v);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) bar_arrive(edone + 8 * b);
        }
      } else {
        for (int piece = set; piece < pieces; piece += kSets) {
          const int64_t j0 = (int64_t)tj * bn + piece * kPiece;
          if (i0 >= rows || j0 >= cols) continue;
          if (S > 1 && !owns_piece(split, piece, pieces, w)) continue;
          const Block b = block_of(out_t ? j0 : i0, out_t ? i0 : j0, e, lane);
          const uint32_t bias = biases + (uint32_t)(piece >> 1) * (kPiece * 4);
          Sides<MODE> sides;
          if (k.epi.vec) load_sides<MODE>(k.epi, b, e, sides);
          // (half a piece at a time: the side operands take many registers)
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
            uint32_t r[16];
            tmem_load16(d + piece * 32 + h, r);
            if (rounds > 1) tmem_add<16>(summed + piece * 32 + h, r);
            if (S > 1) add_part<16>(part_at<32>(ring, piece, pieces, w, lane) + h / 4 * 512, r);
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              v[q] = empty_sum ? 0.0f : __uint_as_float(r[q]);
              if (FP4) v[q] *= whole;
            }
            if (out_t) {
#pragma unroll
              for (int q = 0; q < 16; ++q)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + ((h + q) * 36 + lane) * 4),
                             "f"(v[q]));
            } else {
#pragma unroll
              for (int q = 0; q < 16; q += 4)
                st_shared4(mine + (lane * 36 + h + q) * 4, v[q], v[q + 1], v[q + 2], v[q + 3]);
            }
          }
          __syncwarp();
          if (k.epi.vec)
            finish_block<MODE>(k.epi, masks.at(piece >> 1), mine, bias, b, e, sides, lane);
          else
            finish_any_columns<MODE>(k.epi, masks.at(piece >> 1), mine, bias, out_t ? j0 : i0,
                                     out_t ? i0 : j0, e, lane);
          __syncwarp();
        }
      }
      if (sums && split == 0) {
        if (S > 1) {
          float other;
          asm volatile("ld.shared.f32 %0, [%1];"
                       : "=f"(other)
                       : "r"(part_at<kPiece>(ring, pieces, pieces, w, lane)));
          bias_sum += other;
        }
        store_bias(k, g, (int64_t)(g.bias_b ? tj : ti) * 256 + half * kRowsCta + w * 32 + lane,
                   empty_sum ? 0.0f : bias_sum);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive_fenced(tempty_lead + 8 * acc);
      if (++acc == sets) {
        acc = 0;
        aph ^= 1;
      }
    }
  } else if (GEN && warp >= kGenWarp0) {
    const int r = warp - kGenWarp0, bn = g.bn, stages = g.stages, raws = g.raws;
    const bool gen_a = g.gen_a, gen_b = g.gen_b, bias_b = g.bias_b;
    const int lines_b = bn / 16;
    const uint32_t full_lead = remote(full, leader);
    const uint32_t by_a = gen_distance(k.a, r), by_b = gen_distance(k.b, r);
    const uint32_t raw_a = g.raw_a, raw0 = bias_smem + g.bias_in + (uint32_t)r * (raw_a + g.raw_b),
                   raw_step = (uint32_t)kGenWarps * (raw_a + g.raw_b);
    uint32_t s = 0, ph = 0, rb = 0, rph = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += clusters) {
      int ti, tj;
      tile_at(g, t, ti, tj);
      // for a tile of B's bias sums, B is in A's place
      const bool swap = tj < 0 && bias_b, a = swap ? gen_b : gen_a, b = tj >= 0 && gen_b;
      const uint32_t by = swap ? by_b : by_a;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = bar_wait<kOwn>(landed + 8 * rb, rph, &dead) &&
             bar_wait<kOwn>(empty + 8 * s, ph ^ 1, &dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t a_at = ring + s * stage_bytes, raw = raw0 + rb * raw_step;
        if (a) gen_shift(raw, a_at, kRowsCta / 8, r, by, lane);
        if (b) gen_shift(raw + raw_a, a_at + kBytesA, lines_b, r, by_b, lane);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();  // the raw lines are read, the tile's are written
        if (lane == 0) {
          release_shared();
          bar_arrive_fenced(full_lead + 8 * s);
          bar_arrive(used + 8 * rb);
        }
        if (++s == (uint32_t)stages) {
          s = 0;
          ph ^= 1;
        }
        if (++rb == (uint32_t)raws) {
          rb = 0;
          rph ^= 1;
        }
      }
    }
  } else if (GEN && (warp == 2 || warp == 3)) {
    if constexpr (GEN) {
      const bool for_a = warp == 2, bias_b = g.bias_b;
      const int bn = g.bn, lines = for_a ? kRowsCta / 8 : bn / 16;
      const uint32_t raw_warp = g.raw_a + g.raw_b, raws = g.raws;
      const uint32_t raw0 = bias_smem + g.bias_in + (for_a ? 0 : g.raw_a);
      uint32_t issued = 0, wb = 0, wph = 0;
      bool live = true;
      for (int t = first; t < tiles; t += clusters) {
        int ti, tj;
        tile_at(g, t, ti, tj);
        // for a tile of B's bias sums, B is in A's place
        const bool b = !for_a || (tj < 0 && bias_b), contig = b ? b_c : a_c;
        const bool on = (b ? g.gen_b : g.gen_a) && (for_a || tj >= 0);
        const int64_t all = b ? (b_c ? k.cols : k.depth) : (a_c ? k.rows : k.depth);
        const CUtensorMap* of = b ? maps.b : maps.a;
        const int i0 = for_a ? ti * 256 + (int)half * kRowsCta : tj * bn + (int)half * (bn / 2);
        const uint32_t bytes = on ? (uint32_t)lines * (kRawLine * kGenWarps) : 0;
        for (int kb = kb0; kb < kb1; ++kb) {
          live = live && bar_wait<kOwn>(used + 8 * wb, wph ^ 1, &dead);
          if (elect() && live) {
            const uint32_t bar = landed + 8 * wb;
            bar_expect(bar, bytes);
            if (on)
              gen_load(of, contig, all, i0, kb * kDeep, lines, raw0 + wb * kGenWarps * raw_warp,
                       raw_warp, bar);
          }
          __syncwarp();
          issued += live;
          if (++wb == raws) {
            wb = 0;
            wph ^= 1;
          }
        }
      }
      // after a wait that gave up: what is in flight lands before the CTA returns
      for (uint32_t q = issued > raws ? issued - raws : 0; !live && q < issued; ++q) {
        const long long t0 = clock64();
        while (!bar_try(landed + 8 * (q % raws), (q / raws) & 1) &&
               clock64() - t0 < kWaitCycles / 8) {
        }
      }
    }
  }
  __syncwarp();

  // The exchange of a split contraction passes two barriers of the cluster:
  // so do the warps that have no part in it.
  for (int q = barriers; S > 1 && q < 2; ++q) {
    cluster_arrive();
    cluster_wait();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  if (!early) cluster_arrive();
  cluster_wait();
  if (warp == 2) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(g.tmem_cols));
  }
}

// ------------------------------------------------------------------- host --
// Whether an operand lies off 16-byte boundaries: its base or its rows (where
// there are several).
static bool off_words(const Mat& a, int64_t lines) {
  return ((uintptr_t)a.p & 15) != 0 || (lines > 1 && a.ld % 8 != 0);
}

// An operand's tiles: 64 deep x box_rows, or blocks of 64 rows x 64 deep.
static bool operand_map(CUtensorMap* map, const Mat& a, bool contig, int64_t rows, int64_t depth,
                        int box_rows) {
  return contig ? encode(map, false, a.p, depth, rows, a.ld, kDeep, box_rows,
                         CU_TENSOR_MAP_SWIZZLE_128B)
                : encode(map, false, a.p, rows, depth, a.ld, 64, kDeep,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

// The eight maps of such an operand: lines r, r + 8, ... of `lines` lines of
// `inner` elements, each from the 16-byte word it begins in (which for the
// first may begin before the matrix; what lies there is shifted out).
static bool gen_maps(CUtensorMap map[8], const Mat& a, int64_t lines, int64_t inner, int box_y) {
  for (int r = 0; r < 8; ++r) {
    const int64_t at = r < lines ? r : 0;  // (no such line: any map will do)
    char* p = static_cast<char*>(a.p) + 2 * at * a.ld;
    const int into = (int)((uintptr_t)p & 15);
    if (!encode(&map[r], false, p - into, inner + into / 2, (lines - at + 7) / 8, 8 * a.ld,
                kRawLine / 2, box_y, CU_TENSOR_MAP_SWIZZLE_NONE))
      return false;
  }
  return true;
}

// An operand's scale tiles: `deep` along the contraction, `chunks` down the rows.
static bool scale_map(CUtensorMap* map, const void* scales, int64_t rows, int64_t tiles, int deep,
                      int chunks) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  constexpr int units = kScaleTile / 2;
  const cuuint64_t dims[3] = {(cuuint64_t)units, (cuuint64_t)tiles,
                              (cuuint64_t)((rows + kRowsCta - 1) / kRowsCta)};
  const cuuint64_t strides[2] = {(cuuint64_t)kScaleTile, (cuuint64_t)(tiles * kScaleTile)};
  const cuuint32_t box[3] = {(cuuint32_t)units, (cuuint32_t)deep, (cuuint32_t)chunks};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(scales), dims, strides, box,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A side operand's or output's boxes of `width` columns x 128 rows.
static bool box_map(CUtensorMap* map, const Mat& a, int64_t rows, int64_t cols, int width) {
  if (!a.p) return true;
  const bool f32 = a.dtype == ZERO_F32;
  return encode(map, f32, a.p, cols, rows, a.ld, width, kRowsCta,
                width * (f32 ? 4 : 2) == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                             : CU_TENSOR_MAP_SWIZZLE_64B);
}

// Shared memory beside the operand ring, and the ring's stages in what is left.
static int side_bytes(const TileK& g, int form) {
  return (g.bias_tiles || g.bias_fused ? kOnesBytes : 0) + g.bias_in +
         (form == PATCH_GEN ? g.raws * kGenWarps * (g.raw_a + g.raw_b) : 0) +
         (form >= BOX_BF16 ? g.boxes * kSlot * (g.two_slots ? 2 : 1) : kPatchWarps * kPatch * 4);
}
static int stages_for(const TileK& g, int form) {
  const int n =
      (kSmemMost - 1024 - side_bytes(g, form)) / (kBytesA + g.bn * kDeep + g.scale_bytes);
  return n < kMaxStages ? n : kMaxStages;
}

template <int MODE, int FORM, int KIND>
static cudaError_t launch_tiles(const CUtensorMap& ma, const CUtensorMap& mb,
                                const typename MapsOf<FORM, KIND>::type& maps, const ProductK& k,
                                TileK& g,
                                cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  constexpr int most = kSmemMost - 1024;  // the rest is the kernel's static shared memory
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(product_kernel<MODE, FORM, KIND>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  g.stages = stages_for(g, FORM);
  const int64_t tiles = (int64_t)g.tiles_i * g.tiles_j + g.bias_tiles;
  const int64_t pairs = sm_count() / 2;
  const int64_t clusters = g.splits > 1 || tiles < pairs ? tiles : pairs;
  g.clusters = (int)clusters;
  const int fast = g.i_fast ? g.tiles_i : g.tiles_j;
  const int whole = fast > 0 ? g.clusters / fast : 0, rest = fast > 0 ? g.clusters % fast : 0;
  g.by_i = g.i_fast ? rest : whole;
  g.by_j = g.i_fast ? whole : rest;
  g.split_log2 = g.splits - 1;  // 1 or 2 parts
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * 2 * g.splits));
  cfg.blockDim = dim3(threads_of(FORM));
  cfg.dynamicSmemBytes =
      (size_t)g.stages * (kBytesA + g.bn * kDeep + g.scale_bytes) + side_bytes(g, FORM);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * g.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, product_kernel<MODE, FORM, KIND>, ma, mb, maps, k, g);
}

// Whether a side matrix can move in boxes: absent, or on 16-byte boundaries.
// A store writes whole 16-byte units, so an output's rows must end with one.
static bool boxable(const Mat& a, int64_t rows) {
  return !a.p || a.vec || (rows == 1 && ((uintptr_t)a.p & 15) == 0);
}
static bool box_output(const Mat& a, int64_t rows, int64_t cols) {
  return boxable(a, rows) && (!a.p || (cols * (a.dtype == ZERO_F32 ? 4 : 2)) % 16 == 0);
}

template <int MODE, int KIND>
static cudaError_t launch_mode(const ProductK& in, cudaStream_t st) {
  constexpr bool FP4 = KIND == OF_FP4;
  ProductK k = in;
  // Few rows (tokens): the weight's side fills the 256 rows of a tile and the
  // tokens are its columns; the output is written transposed.
  if (MODE != LIN_DWEIGHT && k.rows <= 128) {
    const Mat a = k.a;
    k.a = in.b;
    k.b = a;
    k.a_c = in.b_c;
    k.b_c = in.a_c;
    std::swap(k.scales_a, k.scales_b);
    std::swap(k.whole_a, k.whole_b);
    k.rows = in.cols;
    k.cols = in.rows;
    k.out_t = !in.out_t;
  }
  for (const Mat* m : {&k.epi.out, &k.epi.pre, &k.epi.gate, &k.epi.dgate, &k.epi.residual})
    if (m->p && !m->vec) k.epi.vec = 0;
  TileK g{};
  const int64_t kblocks = (k.depth + kDeep - 1) / kDeep;
  const int64_t tiles_i = (k.rows + 255) / 256;
  const int64_t pairs = sm_count() / 2;
  // Width and split by a cost model: waves of tiles times the cycles of one.
  // A 64-deep step takes 520 cycles at BN = 256 (the tensor cores' own time)
  // and 430 at 128 and below, where loading A's rows decides; the last tile's
  // epilogue 25 per column; joining two halves of a contraction 2500 and 15
  // per column, and a further wave of those its start as well.  (Measured, us,
  // one part / two: 1 x 4096 x 4096 17.4 / 11.9, 1024 x 1024 x 4096 at BN = 128
  // 18.4 / 14.1, 2048 x 1024 x 4096 at BN = 256 23.4 / 18.0, 1024 x 2304 x 768
  // at 128 8.8 / 16.6; four parts, clusters of 8, always lost.)  Lines off
  // 16-byte boundaries bound a step by shifting them: 870 cycles for 144 of
  // them, 1040 for 192, 1430 for 256.  4 bits: a step is 256 codes, 400 cycles at
  // BN = 128 and below, 470 (NV) and 445 (MX) at 192.  (us at 128 / 192, NV: 1024
  // x 11008 x 4096 26.8 / 25.4, 1024 x 4096 x 11008 26.1 / 31.2, 4096 x 4096 x 4096
  // 34.5 / 31.5, 8192 x 11008 x 4096 145 / 124, 1024 x 1024 x 1024 6.8 / 7.2; in
  // two parts at 128 256 x 4096 x 11008 16.4 / 14.5, 1024 x 1024 x 1024 6.8 / 9.0.)
  // The tensor cores add to their fp32 sums without rounding to nearest, so a
  // long contraction loses digits: 7e-7 of the result after 768 terms, 7e-6
  // after 6000 (in 2-norms).  fp32 results therefore take the sums out every
  // `round` steps and add them to nearest, in a third set of tensor memory,
  // where three fit (BN = 128) while the products go on.  Rounds of 12 steps
  // keep any fp32 result at about 7e-7, which sums to nearest throughout reach
  // at 6000 terms (2e-7 at 768).  (Rounds of 4, 8, 12, 16, 24 steps: weight
  // gradient 2048 x 2048 of 6001 rows 57, 42, 39, 38, 36.5 us and 2.5, 4.7,
  // 7.2, 9.8, 15e-7; 2048 x 1024 to 4096 28, 24, 24, 19, 19 us and 2.3, 4.7,
  // 6.4, 10, 10e-7; 2048 x 640 to 4096, one round from 12 on, 22.5, 20, 17.5
  // us and 2.1, 4.3, 6.0e-7.)  bf16 results take them out only where the loss
  // would come near their own rounding, beyond 32768 terms: 3e-5 (8e-5 where all
  // terms have one sign) against 2e-3.  What counts is additions: with 4 bits one
  // takes 64 terms instead of 16, so that a round of 48 additions is four times as
  // long and the limit of bf16 results 131072 terms, where they are off by 2e-5
  // with terms of one sign; fp32 results are off by 1.5e-7 at 4096 to 262144 terms
  // of one sign.
  const bool f32 = k.epi.out.dtype == ZERO_F32 || (k.dbias.p && k.dbias.dtype == ZERO_F32);
  const bool exact = f32 ? kblocks > kRound : kblocks > 512;
  g.bias_b = k.dbias.p && k.bias_b;
  const int64_t bias_rows = !k.dbias.p ? 0 : g.bias_b ? k.cols : k.rows;
  // The bias's sums ride on the first tiles' products (an eighth more work on
  // those) where tensor memory has room for them; else they are tiles of
  // their own, which cost a row of loads and, past a full wave, a wave.
  auto fuses_bias = [&](int bn, int S, int64_t tiles_j) {
    const int64_t main = tiles_i * tiles_j;
    return bias_rows > 0 && main > 0 && (!g.bias_b || bn == 256) &&
           (exact ? bn == 128 : S > 1 || main <= pairs || bn == 128);
  };
  const bool gen_a = k.depth > 0 && k.rows > 0 && off_words(k.a, k.a_c ? k.rows : k.depth);
  const bool gen_b = k.depth > 0 && k.cols > 0 && off_words(k.b, k.b_c ? k.cols : k.depth);
  double best = 0;
  for (int width = 32; width <= 256; width *= 2) {
    // (4 bits: two sets of 256 columns would leave tensor memory no room for
    // the scales)
    const int bn = FP4 && width == 256 ? 192 : width;
    if (!k.b_c && bn < 128) continue;       // blocks of 64 rows per CTA
    if (bn < 128 && k.cols > bn) continue;  // narrow tiles only where one is enough
    const int64_t tiles_j = (k.cols + bn - 1) / bn;
    for (int S = 1; S <= 2; ++S) {
      if (S > 1 && (kblocks < 2 * S || bn == 192)) break;
      const bool fused = fuses_bias(bn, S, tiles_j);
      const int64_t tiles = tiles_i * tiles_j + (fused ? 0 : (bias_rows + 255) / 256);
      const double waves = (double)((tiles * S + pairs - 1) / pairs);
      const double whole = FP4 ? (bn <= 128 ? 400 : k.blocks_of == 16 ? 470 : 445)
                               : (bn <= 128 ? 430 : 520);
      double step = bn > 128 && exact ? whole + 1500.0 / kRound : whole;
      const double shift = 300 + 4.2 * ((gen_a ? kRowsCta : 0) + (gen_b ? bn / 2 : 0));
      if ((gen_a || gen_b) && step < shift) step = shift;
      const double cost =
          waves * ((double)kblocks / S * step + (S > 1 ? 2500 + 15 * bn : 0)) +
          (S > 1 || (exact && bn > 128) ? (waves - 1) * 8000 : 0) + 25 * bn;
      if (best == 0 || cost < best) {
        best = cost;
        g.bn = bn;
        g.splits = S;
        g.tiles_j = (int)tiles_j;
      }
    }
  }
  if (tiles_i * (g.tiles_j + 1) >= (1ll << 28) || kblocks >= (1ll << 30))
    return cudaErrorInvalidValue;
  g.bias_in = k.epi.bias.p ? 4096 : 0;  // 8 warps of 32 columns 4 times, or 16 of 16
  g.tiles_i = (int)tiles_i;
  g.kblocks = (int)kblocks;
  g.round = exact ? kRound : 0;
  g.acc_sets = exact && g.bn > 128 ? 1 : 2;
  g.bias_fused = fuses_bias(g.bn, g.splits, g.tiles_j);
  g.bias_tiles = g.bias_fused ? 0 : (int)((bias_rows + 255) / 256);
  g.i_fast = k.rows <= k.cols;
  g.tmem_cols = FP4 || (g.bn >= 128 && (exact || g.bias_fused)) ? 512 : (exact ? 4 : 2) * g.bn;
  CUtensorMap ma{}, mb{};
  typename MapsOf<PATCH, KIND>::type maps{};
  if constexpr (FP4) {
    g.scale_deep = k.blocks_of == 16 ? 4 : 2;
    g.scale_chunks = g.bn > kRowsCta ? 2 : 1;
    g.scale_bytes = (1 + g.scale_chunks) * g.scale_deep * kScaleTile;
    if (kblocks > 0 &&
        (!scale_map(&maps.scale_a, k.scales_a, k.rows, k.scale_tiles, g.scale_deep, 1) ||
         !scale_map(&maps.scale_b, k.scales_b, k.cols, k.scale_tiles, g.scale_deep,
                    g.scale_chunks)))
      return cudaErrorInvalidValue;
  }
  if (k.depth > 0) {
    g.gen_a = gen_a;
    g.gen_b = gen_b;
    if (!g.gen_a && k.rows > 0 &&
        !operand_map(&ma, k.a, k.a_c, k.rows, k.depth, kRowsCta))
      return cudaErrorInvalidValue;
    if (!g.gen_b && k.cols > 0 &&
        !operand_map(&mb, k.b, k.b_c, k.cols, k.depth, g.bn / 2))
      return cudaErrorInvalidValue;
  }
  if constexpr (!FP4) if (g.gen_a || g.gen_b) {
    GenMaps gen{};
    if (g.gen_a && !gen_maps(gen.a, k.a, k.a_c ? k.rows : k.depth, k.a_c ? k.depth : k.rows,
                             k.a_c ? kRowsCta / 8 : 8))
      return cudaErrorInvalidValue;
    if (g.gen_b && !gen_maps(gen.b, k.b, k.b_c ? k.cols : k.depth, k.b_c ? k.depth : k.cols,
                             k.b_c ? g.bn / 16 : 8))
      return cudaErrorInvalidValue;
    // (TMA writes to 128-byte boundaries)
    g.raw_a = g.gen_a || (g.bias_tiles && g.bias_b) ? kRowsCta / 8 * kRawLine : 0;
    g.raw_b = g.gen_b ? (g.bn / 16 * kRawLine + 127) / 128 * 128 : 0;
    for (g.raws = kMostRaw; g.raws > 2 && stages_for(g, PATCH_GEN) < 4; --g.raws) {
    }
    return launch_tiles<MODE, PATCH_GEN, KIND>(ma, mb, gen, k, g, st);
  }
  const EpiK& o = k.epi;
  const bool pre_ok = MODE == LIN_FORWARD ? box_output(o.pre, k.rows, k.cols)
                                          : boxable(o.pre, k.rows);
  // (each half of a split contraction stores whole boxes)
  const int width = o.out.dtype == ZERO_F32 ? 32 : 64;
  if (k.out_t || g.bn < width * g.splits || k.rows <= 0 || k.cols <= 0 || !pre_ok ||
      !box_output(o.out, k.rows, k.cols) || !boxable(o.gate, k.rows) ||
      !box_output(o.dgate, k.rows, k.cols) ||
      !boxable(o.residual, k.rows) || (o.residual.p && o.residual.dtype != o.out.dtype))
    return launch_tiles<MODE, PATCH, KIND>(ma, mb, maps, k, g, st);
  const bool wide = o.out.dtype == ZERO_F32;
  const Mat& extra = MODE == LIN_FORWARD ? o.residual : o.dgate;
  if (!box_map(&maps.out, o.out, k.rows, k.cols, width) ||
      !box_map(&maps.pre, o.pre, k.rows, k.cols, width) ||
      !box_map(&maps.gate, o.gate, k.rows, k.cols, width) ||
      !box_map(&maps.extra, extra, k.rows, k.cols, width))
    return cudaErrorInvalidValue;
  g.two_slots = MODE == LIN_FORWARD ? o.gate.p || o.pre.p
                : MODE == LIN_DINPUT ? o.gate.p || (wide && o.pre.p)
                                     : 0;
  // Two chunks in flight where they are two boxes each: at BN = 256 the
  // operands' ring then keeps 5 stages (gate 4096-11008: 225 us against 252 at
  // 3 and 4), or 4 beside the biases' 4 KiB (8192 x 1024 to 4096 with GELU and
  // kept z: 56.3 us with a bias, 52.5 without).
  g.boxes = g.two_slots ? 2 : kMostBoxes;
  if (wide) return launch_tiles<MODE, BOX_F32, KIND>(ma, mb, maps, k, g, st);
  return launch_tiles<MODE, BOX_BF16, KIND>(ma, mb, maps, k, g, st);
}

}  // namespace zk
