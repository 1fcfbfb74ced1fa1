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
// Five steps are off by 3e-4 to 1e-3 in 2-norm on matrices of full rank; with
// operands alone in fp16, 1.3e-3 on random matrices and 4e-2 at rank 16; in bf16
// 1e-2 and 0.3.  Directions that x lacks are lifted a-fold by each step, and what
// the roundings of P X put there with them, the more the shorter the smaller side
// k: 1e-3 at 768 (ranks of 96 to 384), 2e-3 at 256, but 2.6e-2 at 16 (rank 1).  So where
// k is 256 or less (`fine`), P is held in two numbers as well and P X is three
// products, P's first part by both of X's and its second by X's first: 5e-4 to 1e-3
// at every rank.  There a product over k is short, and no box of P has a transpose
// to be stored, whose place the second part takes.
#include "zero_tile.cuh"
#include "zero_walk.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

namespace zk {

// Powers of two that operands are stored times: X, O of G, O of P.
constexpr float kScaleX = 4096.0f, kScaleG = 256.0f, kScaleP = 64.0f;

// Chunks of 64 columns (two boxes each) in flight, beside five operand stages
// of 32 KiB: with three chunks and four stages 11008 x 4096 takes 2270 us
// instead of 2126, 24 x 1024 x 1024 546 instead of 530.
constexpr int kBoxChunks = 2;
constexpr int kBox = 16384;                      // 128 rows of 64 fp16 columns
constexpr int kSideBytes = 2 * kBoxChunks * kBox;
// What the epilogue has to know of a tile: the task, and the diagonal of its
// rows (128 of this CTA) and of its columns (256).
constexpr int kNoteInts = 8, kNoteBytes = 2048;
// Tasks on their way from the warp that looks them up to those that load,
// multiply, bring and store.
constexpr int kTaskSlots = 4, kTaskAt = 4 * kNoteInts + 3 * 512;
static_assert(kTaskAt + kTaskSlots * 4 * kNoteInts <= kNoteBytes, "notes");
// A load is 1100 cycles on its way and a stage some 900 more in use, so that the
// ring's length bounds a step where tiles are few: where none is wider than 128
// columns stages take 24 KiB and are six.  (Five steps of 768 x 768 with four, five
// and six 92.8, 88.8 and 86.5 us, 257 x 8192 215, 191 and 181; eight beside one
// chunk 90.7 and 179.)
constexpr int kRingBytes = kSmemMost - 1024 - kSideBytes - kNoteBytes;
constexpr int kMostOrthoStages = 6;
// The tensor cores add to their fp32 sums without rounding to nearest, and the
// diagonals of G and G^2 are sums of terms of one sign: after 8192, 16384, 32768 and
// 524288 terms they are 5e-5, 1e-4, 2e-4 and 3e-3 too small.  So sums leave the tensor
// cores every 256 steps of 64 and are added to nearest.
constexpr int kOrthoRound = 256;
constexpr int kEpi0 = 4, kEpis = 16;             // epilogue warps
constexpr int kTaskWarp = kEpi0 + kEpis;         // looks tasks up
constexpr int kOrthoThreads = 32 * (kTaskWarp + 1);

// ------------------------------------------------------------ the products --
// One launch runs every product of every step.  A task is a tile of 256 x bn of
// one product of one matrix; pairs of CTAs take tasks in turn, in the order
// step, product, matrix, tile.  A task waits until its matrix has all tiles of
// the products before, which a counter of finished tiles tells: with several
// matrices in a batch nobody waits, and no wave of tiles ends in idle pairs.
// Tasks only wait for tasks before them and every pair is resident (a
// cooperative launch), so that the first unfinished task can always go on.
enum OrthoProduct : int { GRAM = 0, POLY = 1, GROW = 2 };

struct OrthoK {
  int kblocks, bn, bn_log2;
  int passes, steps;        // over the contraction (GROW: parts of P and X); of them all
  int tiles;                // of one matrix
  int before;               // of a step's products before this one
  int tiles_j;              // GROW: across
  int a_c, b_c;             // the operand's contraction index is the contiguous one
  int rows_a, rows_b, rows_out;  // rows of the batch's matrices, one below the other
};
struct OrthoMaps {
  CUtensorMap x_a[2], x_b[2];  // GRAM's operands
  CUtensorMap gram_a, gram_b;  // POLY's
  CUtensorMap poly, x[2];      // GROW's
  CUtensorMap poly_lo, x_lo[2];
  // boxes; _t of 64 x 64
  CUtensorMap hi[2], lo[2], gram, gram_t, poly_out, poly_lo_out, poly_t;
};
struct OrthoSteps {
  OrthoMaps maps;
  OrthoK k[3];
  int steps, batch, tiles_step;  // tiles of a matrix's step
  int cols;                 // of X as stored
  int tall;                 // P's diagonal goes by column
  int side;                 // elements of a diagonal
  int fine;                 // P too is held in two numbers, and all of X multiplied
  int stages, stage_bytes;  // of the operands' ring
  float *diag_gram, *diag_poly;
  uint32_t* done;           // finished tiles of each matrix, both CTAs'
  float coef[ZERO_NS_MOST][3];
};

struct OrthoTask {
  int step, product, b;
  int i0, j0, chunks;       // first row and column, 64-column pieces
  uint32_t needs;           // finished tiles of matrix b
  bool mirror;              // the result's transpose has to be stored too
};
// Tiles of symmetric results are those of the lower triangle, row by row: row i
// of 256 has i + 1 squares of 256, each of 256 / bn tiles.
__device__ __forceinline__ OrthoTask ortho_task(const OrthoSteps& s, int t) {
  OrthoTask o;
  const int each = s.batch * s.tiles_step;
  o.step = t / each;
  t -= o.step * each;
  o.product = t < s.batch * s.k[POLY].before ? GRAM : t < s.batch * s.k[GROW].before ? POLY : GROW;
  const OrthoK& k = s.k[o.product];
  t -= s.batch * k.before;
  o.b = t / k.tiles;
  t -= o.b * k.tiles;
  o.needs = 2u * (uint32_t)(o.step * s.tiles_step + k.before);
  if (o.product == GROW) {
    const int i = t / k.tiles_j;
    o.i0 = i * 256;
    o.j0 = (t - i * k.tiles_j) << k.bn_log2;
    const int rest = s.cols - o.j0;
    o.chunks = (rest < k.bn ? rest : k.bn) / 64;
    o.mirror = false;
  } else {
    const int sub = 8 - k.bn_log2, square = t >> sub;
    int i = (int)((sqrtf(8.0f * (float)square + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > square) --i;
    while ((i + 1) * (i + 2) / 2 <= square) ++i;
    o.i0 = i * 256;
    o.j0 = (square - i * (i + 1) / 2) * 256 + ((t & ((1 << sub) - 1)) << k.bn_log2);
    o.chunks = k.bn / 64;
    o.mirror = o.j0 + k.bn <= o.i0;
  }
  return o;
}
// Until matrix o.b has the tiles that the task needs.  Limited as the other
// waits are; the whole warp calls it.
__device__ __forceinline__ bool ortho_wait(const OrthoSteps& s, const OrthoTask& o,
                                           volatile int* dead) {
  const long long t0 = clock64();
  while (true) {
    uint32_t have;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];"
                 : "=r"(have)
                 : "l"(s.done + o.b)
                 : "memory");
    if (__all_sync(0xffffffffu, have >= o.needs)) return true;
    int stop = *dead;
    if (!stop && clock64() - t0 > kWaitCycles) {
      stop = 1;
      if (elect()) {
        *dead = 1;
        atomicAdd(&g_ops_timeouts, 1ull);
      }
    }
    if (__any_sync(0xffffffffu, stop)) return false;
  }
}
// What other CTAs' tensor copies stored before a wait is in place for copies
// behind it, and the other way round.
__device__ __forceinline__ void fence_copies() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

// A task as the looking-up warp hands it on.
struct OrthoNote {
  int product, step, b, i0, j0, chunks;
  bool mirror;
};
__device__ __forceinline__ uint4 note_low(const OrthoTask& o) {
  return make_uint4((uint32_t)o.product, (uint32_t)o.step, (uint32_t)o.b, (uint32_t)o.i0);
}
__device__ __forceinline__ uint4 note_high(const OrthoTask& o) {
  return make_uint4((uint32_t)o.j0, (uint32_t)o.chunks, (uint32_t)o.mirror, 0u);
}
__device__ __forceinline__ OrthoNote note_of(const uint4& lo, const uint4& hi) {
  OrthoNote n;
  n.product = (int)lo.x;
  n.step = (int)lo.y;
  n.b = (int)lo.z;
  n.i0 = (int)lo.w;
  n.j0 = (int)hi.x;
  n.chunks = (int)hi.y;
  n.mirror = hi.z != 0;
  return n;
}
// Looks a pair's tasks up and waits for what they need: ~500 cycles of
// arithmetic, as many for the counter and 1400 for the fence where copies are in
// flight, which the loading warp would miss (24 x 1024 x 1024: 508 us for the products so, 457
// with this warp).
template <bool CAREFUL>
__device__ __forceinline__ void ortho_tasks(const OrthoSteps& s, uint32_t at, uint32_t sfull,
                                            uint32_t sempty, int first, int tasks, int step,
                                            volatile int* dead) {
  uint32_t slot = 0, phase = 1;
  bool live = true;
  for (int t = first; t < tasks && live; t += step) {
    const OrthoTask o = ortho_task(s, t);
    live = ortho_wait(s, o, dead) && bar_wait<CAREFUL>(sempty + 8 * slot, phase, dead);
    live = __all_sync(0xffffffffu, live);
    if (!live) break;
    fence_copies();
    if (elect()) {
      sts16(at + slot * 4 * kNoteInts, note_low(o));
      sts16(at + slot * 4 * kNoteInts + 16, note_high(o));
      bar_arrive(sfull + 8 * slot);
    }
    __syncwarp();
    if (++slot == kTaskSlots) {
      slot = 0;
      phase ^= 1;
    }
  }
}
// One reader's place in that ring.  False: a wait gave up.
struct OrthoTasks {
  uint32_t at, sfull, sempty, slot = 0, phase = 0;
  OrthoNote o{};
  template <bool CAREFUL>
  __device__ __forceinline__ bool next(volatile int* dead) {
    bool live = bar_wait<CAREFUL>(sfull + 8 * slot, phase, dead);
    live = __all_sync(0xffffffffu, live);
    if (!live) return false;
    o = note_of(lds16(at + slot * 4 * kNoteInts), lds16(at + slot * 4 * kNoteInts + 16));
    __syncwarp();
    if (elect()) bar_arrive(sempty + 8 * slot);
    __syncwarp();
    if (++slot == kTaskSlots) {
      slot = 0;
      phase ^= 1;
    }
    return true;
  }
};

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

// The chunk ring's slots.
struct OrthoSlot {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kBoxChunks) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// Warp 2: brings the operands of the epilogue's chunks, and before a tile's
// first the note of the tile, once the epilogue has read the one before
// (noted).  The epilogue takes it behind that chunk's barrier.
template <bool CAREFUL>
__device__ __forceinline__ void ortho_bring(const OrthoSteps& s, OrthoTasks in, uint32_t boxes,
                                            uint32_t note, uint32_t efull, uint32_t bfree,
                                            uint32_t noted, int first, int tasks, int step,
                                            int half, int lane, volatile int* dead) {
  OrthoSlot r;
  bool live = true;
  uint32_t issued = 0, note_phase = 1;
  for (int t = first; t < tasks && live; t += step) {
    live = in.next<CAREFUL>(dead) && bar_wait<CAREFUL>(noted, note_phase, dead);
    live = __all_sync(0xffffffffu, live);
    if (!live) break;
    note_phase ^= 1;
    const OrthoNote& o = in.o;
    if (lane < 2) {
      OrthoTask whole{};
      whole.product = o.product; whole.step = o.step; whole.b = o.b; whole.i0 = o.i0;
      whole.j0 = o.j0; whole.chunks = o.chunks; whole.mirror = o.mirror;
      sts16(note + 16 * lane, lane ? note_high(whole) : note_low(whole));
    }
    if (o.product != GRAM) {
      const float* diag = (o.product == POLY ? s.diag_gram : s.diag_poly) + (int64_t)o.b * s.side;
      const bool by_row = o.product == POLY || !s.tall, by_column = o.product == POLY || s.tall;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f), c[2] = {v, v};
      if (by_row) v = ld_state(diag + o.i0 + half * kRowsCta + 4 * lane);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (by_column && q * 128 + 4 * lane < o.chunks * 64)
          c[q] = ld_state(diag + o.j0 + q * 128 + 4 * lane);
      const uint32_t at = note + 4 * kNoteInts + 16 * lane;
      st_shared4(at, v.x, v.y, v.z, v.w);
#pragma unroll
      for (int q = 0; q < 2; ++q) st_shared4(at + 512 * (q + 1), c[q].x, c[q].y, c[q].z, c[q].w);
    }
    __syncwarp();  // the note is written when the lane below arrives
    const int y = o.b * s.k[o.product].rows_out + o.i0 + half * kRowsCta;
    for (int c = 0; c < o.chunks; ++c) {
      live = bar_wait<CAREFUL>(bfree + 8 * r.slot, r.phase ^ 1, dead);
      live = __all_sync(0xffffffffu, live);
      if (!live) break;
      const uint32_t at = boxes + r.slot * 2 * kBox, bar = efull + 8 * r.slot;
      const int x = o.j0 + 64 * c;
      if (elect()) {
        bar_expect(bar, o.product * kBox);
        if (o.product == POLY) box_load(&s.maps.gram, at, x, y, bar);
        if (o.product == GROW) {
          box_load(&s.maps.hi[o.step & 1], at, x, y, bar);
          box_load(&s.maps.lo[o.step & 1], at + kBox, x, y, bar);
        }
      }
      __syncwarp();
      ++issued;
      r.next();
    }
  }
  // after a wait that gave up: the boxes in flight land before the CTA returns
  for (uint32_t q = issued > kBoxChunks ? issued - kBoxChunks : 0; !live && q < issued; ++q) {
    const long long t0 = clock64();
    while (!bar_try(efull + 8 * (q % kBoxChunks), (q / kBoxChunks) & 1) &&
           clock64() - t0 < kWaitCycles / 8) {
    }
  }
}

// Warp 3: stores the finished chunks and counts finished tiles.
template <bool CAREFUL>
__device__ __forceinline__ void ortho_store(const OrthoSteps& s, OrthoTasks in, uint32_t boxes,
                                            uint32_t edone, uint32_t bfree, int first, int tasks,
                                            int step, int half, volatile int* dead) {
  OrthoSlot r;
  bool live = true;
  for (int t = first; t < tasks && live; t += step) {
    live = in.next<CAREFUL>(dead);
    if (!live) break;
    const OrthoNote& o = in.o;
    const int row = o.i0 + half * kRowsCta, y = o.b * s.k[o.product].rows_out;
    for (int c = 0; c < o.chunks; ++c) {
      live = bar_wait<CAREFUL>(edone + 8 * r.slot, r.phase, dead);
      live = __all_sync(0xffffffffu, live);  // the lanes leave together
      if (!live) break;
      const uint32_t at = boxes + r.slot * 2 * kBox;
      const int x = o.j0 + 64 * c;
      if (elect()) {
        if (o.product == GROW) {
          box_store(&s.maps.hi[~o.step & 1], at, x, y + row);
          if (o.step + 1 < s.steps) box_store(&s.maps.lo[~o.step & 1], at + kBox, x, y + row);
        } else {
          box_store(o.product == GRAM ? &s.maps.gram : &s.maps.poly_out, at, x, y + row);
          if (CAREFUL && s.fine && o.product == POLY)
            box_store(&s.maps.poly_lo_out, at + kBox, x, y + row);
          if (o.mirror) {
            const CUtensorMap* m = o.product == GRAM ? &s.maps.gram_t : &s.maps.poly_t;
            box_store(m, at + kBox, row, y + x);
            box_store(m, at + kBox + kBox / 2, row + 64, y + x);
          }
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        bar_arrive(bfree + 8 * r.slot);
        if (c + 1 == o.chunks) {
          asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
          fence_copies();
          // behind this tile's boxes and (through the chunks' barriers) diagonals
          asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(s.done + o.b) : "memory");
        }
      }
      __syncwarp();
      r.next();
    }
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// 16 sums v of row `row` of the box (row `i` of the matrix), columns j.. of the
// matrix from 16-byte unit `unit` of the box on.
template <int PRODUCT>
__device__ __forceinline__ void ortho_piece(float ca, float cb, float cc, bool by_column, bool fine,
                                            const float d[16], float diag_row, float* diag_out,
                                            bool mirror, uint32_t at, int row, int i, int j,
                                            int unit, float v[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t p0 = at + box_at(row, unit + h), p1 = p0 + kBox;
    float* w = v + 8 * h;
    const int on_diag = i - (j + 8 * h);  // which of the eight, if any
    if (PRODUCT == GRAM) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (on_diag == q) {
          diag_out[i] = w[q] * (1.0f / (kScaleX * kScaleX));
          w[q] = 0.0f;
        }
        w[q] *= kScaleG / (kScaleX * kScaleX);
      }
      sts16(p0, to_halves8(w));
    } else if (PRODUCT == POLY) {
      float o[8];
      halves8(lds16(p0), o);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float sq = w[q] * (1.0f / (kScaleG * kScaleG)), g = o[q] * (1.0f / kScaleG);
        float r = cb * g + cc * (sq + (diag_row + d[8 * h + q]) * g);
        if (on_diag == q) {
          diag_out[i] = cb * diag_row + cc * (sq + diag_row * diag_row);
          r = 0.0f;
        }
        w[q] = r * kScaleP;
      }
      if (fine) {  // (one square of 256: nothing is mirrored)
        sts16(p0, split_halves8(w));
        sts16(p1, to_halves8(w));
      } else {
        sts16(p0, to_halves8(w));
      }
    } else {
      float x[8], y[8];
      halves8(lds16(p0), x);
      halves8(lds16(p1), y);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float f = ca + (by_column ? d[8 * h + q] : diag_row);
        w[q] = f * x[q] + (f * y[q] + w[q] * (1.0f / kScaleP));
      }
      sts16(p0, split_halves8(w));
      sts16(p1, to_halves8(w));
    }
  }
  if (PRODUCT != GROW && mirror) {
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

// The operands' ring as one thread loads or multiplies it: a stage and its phase.
struct OrthoRing {
  uint32_t at, full, empty, stages, stage_bytes;
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
  }
};
// A tile's operands, by one thread in a loop of its layout, as are the products:
// with the layouts asked for in each step, and the warps' lanes kept together, either
// warp took 430 cycles a step of any width (768 x 768 96.3 us, now 86.5; 96 x 8192
// 196 and 155).  A_C, B_C: boxes along the contraction, else across it, 64 columns
// each.
template <bool A_C, bool B_C, bool CAREFUL>
__device__ __forceinline__ bool ortho_load(OrthoRing& r, const CUtensorMap* map_a,
                                           const CUtensorMap* map_b, int xa, int ya, int xb,
                                           int yb, int kblocks, bool lead, uint32_t full_lead,
                                           uint32_t bytes, bool wide, volatile int* dead) {
  int c = 0;
  for (int kb = 0; kb < kblocks; ++kb, c += kDeep) {
    if (!bar_wait<CAREFUL>(r.empty + 8 * r.st, r.ph ^ 1, dead)) return false;
    const uint32_t a_at = r.at + r.st * r.stage_bytes, b_at = a_at + kBytesA;
    const uint32_t bar = full_lead + 8 * r.st;
    if (lead) bar_expect(r.full + 8 * r.st, bytes);
    if (A_C) {
      tma_load(map_a, a_at, c, ya, bar);
    } else {
      tma_load(map_a, a_at, xa, ya + c, bar);
      tma_load(map_a, a_at + 8192, xa + 64, ya + c, bar);
    }
    if (B_C) {
      tma_load(map_b, b_at, c, yb, bar);
    } else {
      tma_load(map_b, b_at, xb, yb + c, bar);
      if (wide) tma_load(map_b, b_at + 8192, xb + 64, yb + c, bar);
    }
    r.next();
  }
  return true;
}
// A tile's products, by one thread.
template <bool A_C, bool B_C, bool CAREFUL>
__device__ __forceinline__ bool ortho_multiply(OrthoRing& r, uint32_t d, uint32_t idesc,
                                               int kblocks, volatile int* dead) {
  constexpr uint32_t step_a = A_C ? 2 : 128, step_b = B_C ? 2 : 128;
  const uint64_t a0 = operand_desc(r.at, A_C), b0 = operand_desc(r.at + kBytesA, B_C);
  for (int kb = 0; kb < kblocks; ++kb) {
    if (!bar_wait<CAREFUL>(r.full + 8 * r.st, r.ph, dead)) return false;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint64_t stage = (uint64_t)(r.st * (r.stage_bytes >> 4));  // descriptors count 16 bytes
#pragma unroll
    for (int q = 0; q < kDeep / 16; ++q)
      mma_pair(d, a0 + stage + q * step_a, b0 + stage + q * step_b, idesc, kb > 0 || q > 0);
    commit_pair(r.empty + 8 * r.st, 3);
    r.next();
  }
  return true;
}

// The sums at `to` += those at `from`: this warp's 16 of every 64 columns.
static __device__ __noinline__ void ortho_join(uint32_t to, uint32_t from, int columns) {
  for (int c = 0; c < columns; c += 64, to += 64, from += 64) {
    uint32_t r[16];
    tmem_load16(to, r);
    tmem_add<16>(from, r);
    tmem_store16(to, r);
  }
}

// CAREFUL: a product has more than kOrthoRound steps, or the call is `fine`.  (One
// kernel for all takes 768 x 768 in 109.9 us instead of 108.5.)
template <bool CAREFUL>
__global__ void __launch_bounds__(kOrthoThreads, 1)
    ortho_kernel(const __grid_constant__ OrthoSteps s, int tasks) {
  extern __shared__ __align__(1024) unsigned char ortho_smem[];
  __shared__ __align__(8) uint64_t bars[2 * kMostOrthoStages + 6 + 3 * kBoxChunks + 2 * kTaskSlots];
  __shared__ uint32_t tmem_at;
  __shared__ int dead;
  const uint32_t stages = s.stages, stage_bytes = s.stage_bytes;
  const uint32_t rank = cluster_rank(), half = rank & 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(ortho_smem), boxes = ring + kRingBytes;
  const uint32_t full = smem_u32(bars), empty = full + 8 * stages;
  const uint32_t tfull = empty + 8 * stages, tempty = tfull + 16, ready = tempty + 16;
  const uint32_t efull = ready + 8, edone = efull + 8 * kBoxChunks;
  const uint32_t bfree = edone + 8 * kBoxChunks, noted = bfree + 8 * kBoxChunks;
  const uint32_t sfull = noted + 8, sempty = sfull + 8 * kTaskSlots;
  const uint32_t note = boxes + kSideBytes;

  if (warp == 0 && elect()) {
    dead = 0;
    for (uint32_t q = 0; q < stages; ++q) {
      bar_init(full + 8 * q, 1);
      bar_init(empty + 8 * q, 1);
    }
    for (int a = 0; a < 2; ++a) {
      bar_init(tfull + 8 * a, 1);
      bar_init(tempty + 8 * a, 2 * kEpis);
    }
    bar_init(ready, 2);
    bar_init(noted, kEpis);
    for (int q = 0; q < kTaskSlots; ++q) {
      bar_init(sfull + 8 * q, 1);
      bar_init(sempty + 8 * q, half == 0 ? 4 : 3);  // the second CTA issues no products
    }
    for (int b = 0; b < kBoxChunks; ++b) {
      bar_init(efull + 8 * b, 1);
      bar_init(edone + 8 * b, kEpis);
      bar_init(bfree + 8 * b, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  cluster_arrive();
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_at)),
                 "r"(512)
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
  uint32_t tmem = 0;
  if (warp == 1 || warp == 2 || (warp >= kEpi0 && warp < kTaskWarp)) {
    asm volatile("bar.sync 1, %0;" ::"n"((kEpis + 2) * 32) : "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem = *(volatile uint32_t*)&tmem_at;
  }
  const bool early = warp == 3 || warp == kTaskWarp;  // only this CTA's own memory from here on
  if (early) cluster_arrive();
  OrthoTasks tasks_in;
  tasks_in.at = note + kTaskAt;
  tasks_in.sfull = sfull;
  tasks_in.sempty = sempty;

  if (warp == 0) {
    const uint32_t full_lead = remote(full, 0);
    OrthoRing r{ring, full, empty, stages, stage_bytes};
    bool live = true;
    const bool one = elect();  // issues all of this warp's copies
    for (int t = first; t < tasks; t += clusters) {
      live = tasks_in.next<CAREFUL>(&dead);
      if (!live) break;
      const OrthoNote& o = tasks_in.o;
      const OrthoK& k = s.k[o.product];
      const int i0 = o.i0 + (int)half * kRowsCta, j0 = o.j0 + (int)half * (k.bn / 2);
      const int ya = o.b * k.rows_a, yb = o.b * k.rows_b, kblocks = k.kblocks;
      const uint32_t b_bytes = k.bn * kDeep;
      const bool a_c = k.a_c, b_c = k.b_c, wide = k.bn > 128;
      const int now = o.step & 1;
      const CUtensorMap* x = &s.maps.x[now];
      const CUtensorMap* map_a = o.product == GRAM   ? &s.maps.x_a[now]
                                 : o.product == POLY ? &s.maps.gram_a
                                 : s.tall            ? x
                                                     : &s.maps.poly;
      const CUtensorMap* map_b = o.product == GRAM   ? &s.maps.x_b[now]
                                 : o.product == POLY ? &s.maps.gram_b
                                 : s.tall            ? &s.maps.poly
                                                     : x;
      if (one) {
        const int xa = i0, xb = j0, row_a = a_c ? ya + i0 : ya, row_b = b_c ? yb + j0 : yb;
        const uint32_t bytes = 2 * (kBytesA + b_bytes);
        const bool lead = half == 0;
        const int passes = CAREFUL ? k.passes : 1;
        for (int pass = 0; pass < passes && live; ++pass) {
          if (CAREFUL && pass > 0) {  // GROW: P's second part by X's first, and the other way round
            const CUtensorMap* poly = pass == 1 ? &s.maps.poly_lo : &s.maps.poly;
            x = pass == 1 ? &s.maps.x[now] : &s.maps.x_lo[now];
            map_a = s.tall ? x : poly;
            map_b = s.tall ? poly : x;
          }
          if (a_c && b_c)
            live = ortho_load<true, true, CAREFUL>(r, map_a, map_b, xa, row_a, xb, row_b, kblocks,
                                                   lead, full_lead, bytes, wide, &dead);
          else if (a_c)
            live = ortho_load<true, false, CAREFUL>(r, map_a, map_b, xa, row_a, xb, row_b, kblocks,
                                                    lead, full_lead, bytes, wide, &dead);
          else
            live = ortho_load<false, false, CAREFUL>(r, map_a, map_b, xa, row_a, xb, row_b,
                                                     kblocks, lead, full_lead, bytes, wide, &dead);
        }
      }
      live = __all_sync(0xffffffffu, live);
      if (!live) break;
    }
    // a wait gave up: let the loads in flight land before the CTAs return (stages
    // before st hold phase ph, the others the one before)
    if (!live && half == 0 && one)
      for (uint32_t q = 0; q < stages; ++q) {
        const uint32_t parity = q < r.st ? r.ph : r.ph ^ 1;
        const long long t0 = clock64();
        while (!bar_try(full + 8 * q, parity) && clock64() - t0 < kWaitCycles / 8) {
        }
      }
    __syncwarp();
  } else if (warp == 1) {
    if (half == 0) {
      OrthoRing r{ring, full, empty, stages, stage_bytes};
      uint32_t acc = 0, aph = 0;
      bool live = bar_wait<CAREFUL>(ready, 0, &dead);
      live = __all_sync(0xffffffffu, live);
      const bool one = elect();  // issues all of the pair's products
      for (int t = first; t < tasks && live; t += clusters) {
        live = tasks_in.next<CAREFUL>(&dead);
        if (!live) break;
        const OrthoK& k = s.k[tasks_in.o.product];
        const bool a_c = k.a_c, b_c = k.b_c;
        const int kblocks = CAREFUL ? k.steps : k.kblocks;
        // fp32 sums of fp16 values, M = 256, N = bn
        const uint32_t idesc = (1u << 4) | ((a_c ? 0u : 1u) << 15) | ((b_c ? 0u : 1u) << 16) |
                               ((uint32_t)(k.bn >> 3) << 17) | (16u << 24);
        int left = kblocks;
        do {
          const int steps = CAREFUL && left > kOrthoRound ? kOrthoRound : left;
          if (one) {
            live = bar_wait<CAREFUL>(tempty + 8 * acc, aph ^ 1, &dead);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + acc * 256;
            if (live)
              live = a_c && b_c ? ortho_multiply<true, true, CAREFUL>(r, d, idesc, steps, &dead)
                     : a_c ? ortho_multiply<true, false, CAREFUL>(r, d, idesc, steps, &dead)
                           : ortho_multiply<false, false, CAREFUL>(r, d, idesc, steps, &dead);
            if (live) commit_pair(tfull + 8 * acc, 3);
          }
          live = __all_sync(0xffffffffu, live);
          if (++acc == 2) {
            acc = 0;
            aph ^= 1;
          }
          left -= steps;
        } while (CAREFUL && live && left > 0);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    ortho_bring<CAREFUL>(s, tasks_in, boxes, note, efull, bfree, noted, first, tasks, clusters,
                        (int)half, lane, &dead);
    __syncwarp();
  } else if (warp == 3) {
    ortho_store<CAREFUL>(s, tasks_in, boxes, edone, bfree, first, tasks, clusters, (int)half,
                         &dead);
    __syncwarp();
  } else if (warp == kTaskWarp) {
    ortho_tasks<CAREFUL>(s, note + kTaskAt, sfull, sempty, first, tasks, clusters, &dead);
    __syncwarp();
  } else if (warp >= kEpi0) {
    const int w = (warp - kEpi0) & 3, set = (warp - kEpi0) >> 2;
    const int row = w * 32 + lane;
    const uint32_t tempty_lead = remote(tempty, 0);
    const uint32_t lanes = tmem + ((uint32_t)(w * 32) << 16) + set * 16;
    const bool tall = s.tall;
    uint32_t acc = 0, aph = 0, eb = 0, eph = 0;
    bool ok = true;
    for (int t = first; t < tasks && ok; t += clusters) {
      // the first chunk's operands, and with them the tile's note
      ok = bar_wait<CAREFUL>(efull + 8 * eb, eph, &dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // Rounds: a round's set takes up the sums of the set before, which the round
      // after it fills.  (Ahead of all that has to be kept in registers else.)
      for (int left = CAREFUL ? s.k[lds16(note).x].steps - kOrthoRound : 0; left > 0;
           left -= kOrthoRound) {
        const uint32_t before = acc;
        ok = bar_wait<CAREFUL>(tfull + 8 * acc, aph, &dead);
        if (++acc == 2) {
          acc = 0;
          aph ^= 1;
        }
        ok = ok && bar_wait<CAREFUL>(tfull + 8 * acc, aph, &dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        ortho_join(lanes + acc * 256, lanes + before * 256, s.k[lds16(note).x].bn);
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive_fenced(tempty_lead + 8 * before);
      }
      if (!ok) break;
      const OrthoNote o = note_of(lds16(note), lds16(note + 16));
      const int product = o.product, step = o.step, i0 = o.i0, j0 = o.j0, chunks = o.chunks;
      const bool mirror = o.mirror;
      const int i = i0 + (int)half * kRowsCta + row;
      float* diag_out =
          (product == GRAM ? s.diag_gram : s.diag_poly) + (int64_t)o.b * s.side;
      const float ca = s.coef[step][0], cb = s.coef[step][1], cc = s.coef[step][2];
      // The diagonal of this thread's row, and of this warp's 16 columns of
      // each chunk (two chunks across a register's lanes).
      const bool by_column = product == POLY || (product == GROW && tall);
      float diag_row, diag_col[2];
      const uint32_t diag_at = note + 4 * kNoteInts;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(diag_row) : "r"(diag_at + 4 * row));
#pragma unroll
      for (int q = 0; q < 2; ++q)
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(diag_col[q])
                     : "r"(diag_at + 512 + 4 * ((2 * q + (lane >> 4)) * 64 + set * 16 +
                                                (lane & 15))));
      __syncwarp();
      if (lane == 0) bar_arrive(noted);
      ok = bar_wait<CAREFUL>(tfull + 8 * acc, aph, &dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = lanes + acc * 256;
      for (int c = 0; c < chunks; ++c) {
        const uint32_t b = eb;
        uint32_t r[16];
        tmem_load16(d + c * 64, r);
        float v[16], dc[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = __uint_as_float(r[q]);
        if (by_column)
#pragma unroll
          for (int q = 0; q < 16; ++q)
            dc[q] = __shfl_sync(0xffffffffu, c < 2 ? diag_col[0] : diag_col[1],
                                (c & 1) * 16 + q);
        ok = bar_wait<CAREFUL>(efull + 8 * b, eph, &dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (++eb == kBoxChunks) {
          eb = 0;
          eph ^= 1;
        }
        const uint32_t at = boxes + b * 2 * kBox;
        const int j = j0 + c * 64 + set * 16;
        if (product == GRAM)
          ortho_piece<GRAM>(ca, cb, cc, tall, false, dc, diag_row, diag_out, mirror, at, row, i,
                            j, set * 2, v);
        else if (product == POLY)
          ortho_piece<POLY>(ca, cb, cc, tall, CAREFUL && s.fine, dc, diag_row, diag_out, mirror,
                            at, row, i, j, set * 2, v);
        else
          ortho_piece<GROW>(ca, cb, cc, tall, false, dc, diag_row, diag_out, mirror, at, row, i,
                            j, set * 2, v);
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
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
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

// The eight columns of this thread, the row it begins with, and from that row
// to its next.
struct OrthoAt {
  int64_t col, row, step;
};
__device__ __forceinline__ OrthoAt ortho_at(int log2_across) {
  const int across = 1 << log2_across, down = kThreads >> log2_across;
  OrthoAt a;
  a.col = ((int64_t)blockIdx.x * across + (threadIdx.x & (across - 1))) * 8;
  a.row = (int64_t)blockIdx.y * down + (threadIdx.x >> log2_across);
  a.step = (int64_t)gridDim.y * down;
  return a;
}
__device__ __forceinline__ int valid8(int64_t col, int64_t cols) {
  return col >= cols ? 0 : cols - col < 8 ? (int)(cols - col) : 8;
}
constexpr int kOrthoAhead = 2;  // rows whose loads are in flight together

// One block's share of a matrix: its new momentum (muon), and its squares.
template <bool WIDE, bool MUON>
__global__ void __launch_bounds__(kThreads)
    ortho_squares(const __grid_constant__ OrthoSource s, int log2_across) {
  after_previous_kernel();
  const int b = blockIdx.z;
  const Extent e{s.m, s.n};
  const OrthoAt at = ortho_at(log2_across);
  const int valid = valid8(at.col, s.n);
  Squares q;
  const Mat xm = source_mat(s.places, s.x, b);
  const Mat mm = MUON ? source_mat(s.places, s.momentum, b) : xm;
  const float coef = MUON && s.coef ? *(volatile const float*)s.coef : 1.0f;
  if (valid > 0) {
    Down<WIDE, ZERO_SITE_ORTHO> x(xm, at.row, at.step, at.col, valid);
    Down<WIDE, ZERO_SITE_ORTHO> mom(mm, at.row, at.step, at.col, valid);
    for (; x.row < s.m; x.on(kOrthoAhead), mom.on(kOrthoAhead)) {
      Raw8 rx[kOrthoAhead], rm[kOrthoAhead];
      x.template get<kOrthoAhead>(rx, s.m, e);
      if (MUON) mom.template get<kOrthoAhead>(rm, s.m, e);
#pragma unroll
      for (int i = 0; i < kOrthoAhead; ++i) {
        if (x.row + i * at.step >= s.m) break;
        float v[8];
        values8<WIDE>(rx[i], v);
        if (MUON) {
          float m[8];
          values8<WIDE>(rm[i], m);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float g = muon_grad(s, v[j], coef);
            m[j] = __fadd_rn(__fmul_rn(s.mu, m[j]), g);
            v[j] = s.nesterov ? __fadd_rn(g, __fmul_rn(s.mu, m[j])) : m[j];
          }
          mom.put(i, m, e);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) q.add(v[j]);  // (0 past the columns)
      }
    }
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
    const int64_t block = ((int64_t)b * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    s.partials[block * 3 + threadIdx.x] = t;
  }
}

// X0 = x / (|x| + eps) in two fp16 numbers, zeros around it.
template <bool WIDE, bool MUON>
__global__ void __launch_bounds__(kThreads)
    ortho_scale(const __grid_constant__ OrthoSource s, int log2_across) {
  __shared__ double part[3][kThreads / 32];
  __shared__ float factor_at;
  after_previous_kernel();
  const int b = blockIdx.z;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) s.done[b] = 0;
  {
    double sum[3] = {};
    const double* from = s.partials + (int64_t)b * s.blocks * 3;
    for (int i = threadIdx.x; i < s.blocks; i += kThreads)
#pragma unroll
      for (int q = 0; q < 3; ++q) sum[q] += *(volatile const double*)(from + 3 * i + q);
#pragma unroll
    for (int q = 0; q < 3; ++q) {
#pragma unroll
      for (int m = 16; m; m >>= 1) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], m);
      if ((threadIdx.x & 31) == 0) part[q][threadIdx.x >> 5] = sum[q];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        sum[q] = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) sum[q] += part[q][w];
      }
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
  const OrthoAt at = ortho_at(log2_across);
  if (at.col >= s.ld) return;
  const int valid = valid8(at.col, s.n);
  const Mat xm = source_mat(s.places, s.x, b);
  const Mat mm = MUON ? source_mat(s.places, s.momentum, b) : xm;
  const float coef = MUON && s.coef ? *(volatile const float*)s.coef : 1.0f;
  Down<WIDE, ZERO_SITE_ORTHO> x(xm, at.row, at.step, at.col, valid);
  Down<WIDE, ZERO_SITE_ORTHO> mom(mm, at.row, at.step, at.col, valid);
  for (; x.row < s.rows; x.on(kOrthoAhead), mom.on(kOrthoAhead)) {
    Raw8 rx[kOrthoAhead], rm[kOrthoAhead];
    x.template get<kOrthoAhead>(rx, s.m, e);  // zeros past the matrix
    if (MUON) mom.template get<kOrthoAhead>(rm, s.m, e);
#pragma unroll
    for (int i = 0; i < kOrthoAhead; ++i) {
      const int64_t row = x.row + i * at.step;
      if (row >= s.rows) break;
      float v[8];
      values8<WIDE>(rx[i], v);
      if (MUON) {
        float m[8];
        values8<WIDE>(rm[i], m);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = s.nesterov ? __fadd_rn(muon_grad(s, v[j], coef), __fmul_rn(s.mu, m[j])) : m[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < valid && row < s.m ? v[j] * f * f : 0.0f;
      const int64_t to = ((int64_t)b * s.rows + row) * s.ld + at.col;
      *reinterpret_cast<uint4*>(s.hi + to) = split_halves8(v);
      *reinterpret_cast<uint4*>(s.lo + to) = to_halves8(v);
    }
  }
}

// y = X, or the update of the master weights by it.
template <bool UPDATE>
__global__ void __launch_bounds__(kThreads)
    ortho_finish(const __grid_constant__ OrthoFinish s, int log2_across) {
  after_previous_kernel();
  const int b = blockIdx.z;
  const Extent e{s.m, s.n};
  const OrthoAt at = ortho_at(log2_across);
  const int valid = valid8(at.col, s.n);
  if (valid <= 0) return;
  const Mat ym = source_mat(s.places, s.y, b);
  Mat om;
  if (UPDATE && s.out.p) om = source_mat(s.places, s.out, b);
  Down<UPDATE, ZERO_SITE_ORTHO> y(ym, at.row, at.step, at.col, valid);  // fp32 or bf16
  for (; y.row < s.m; y.on(kOrthoAhead)) {
    Raw8 rw[kOrthoAhead];
    uint4 rx[kOrthoAhead];
    if (UPDATE) y.template get<kOrthoAhead>(rw, s.m, e);
#pragma unroll
    for (int i = 0; i < kOrthoAhead; ++i) {  // (rows of whole tiles: they exist)
      const int64_t row = y.row + i * at.step < s.m ? y.row + i * at.step : y.row;
      rx[i] = ld16(s.x + ((int64_t)b * s.rows + row) * s.ld + at.col);
    }
#pragma unroll
    for (int i = 0; i < kOrthoAhead; ++i) {
      const int64_t row = y.row + i * at.step;
      if (row >= s.m) break;
      float v[8];
      halves8(rx[i], v);
      if (UPDATE) {
        float w[8];
        values8<true>(rw[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (s.decay != 0.0f) w[j] = __fsub_rn(w[j], __fmul_rn(s.decay, w[j]));
          v[j] = __fsub_rn(w[j], __fmul_rn(s.rate, v[j] * (1.0f / kScaleX)));
        }
        if (om.p) store8(om, row, at.col, valid, v, e, ZERO_SITE_ORTHO);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= 1.0f / kScaleX;
      }
      y.put(i, v, e);
    }
  }
}

// ------------------------------------------------------------------- host --
static int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

constexpr int64_t kMostSide = 1ll << 28;
bool ortho_fits(int64_t m, int64_t n, int64_t batch) {
  // rows one below the other, tiles and grids in 32 bits; sizes far from 64.  A Gram
  // tile of 2^28 columns takes 4.2 million steps of some 400 cycles, less than half of
  // what its waiters' limit allows.
  const int64_t k = up(m < n ? m : n, 256), rows = up(m, 256), cols = up(n, 128);
  return batch < 65536 && (m > n ? m : n) <= kMostSide && rows * batch < (1ll << 31) &&
         k * batch < (1ll << 31) && rows / 256 * (cols / 128) < (1ll << 25) / (batch + 1) &&
         k / 256 * (k / 256 + 1) < (1ll << 25) / (batch + 1);
}

// Walks before and after the products: about eight blocks of 256 threads for
// each of 152 SMs, from the sizes alone (the workspace has a place for each).
static Walk ortho_walk(int64_t rows, int64_t cols, int64_t batch) {
  return walk_over(rows, cols, 152 * 8 / (batch > 0 ? batch : 1));
}

OrthoSpace ortho_space(int64_t m, int64_t n, int64_t batch) {
  OrthoSpace w;
  const int64_t k = m < n ? m : n;
  w.rows = up(m, 256);
  w.ld = up(n, 64);
  w.side = up(k, 256);
  w.fine = w.side == 256;
  // blocks of a matrix's norm
  const Walk walk = ortho_walk(m, n, batch);
  w.blocks = (int64_t)walk.grid.x * walk.grid.y;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = up(at + bytes, 1024);
    return here;
  };
  const int64_t x = batch * w.rows * w.ld * 2, g = batch * w.side * w.side * 2;
  w.hi[0] = take(x);
  w.hi[1] = take(x);
  w.lo[0] = take(x);
  w.lo[1] = w.fine ? take(x) : w.lo[0];
  w.gram = take(g);
  w.poly = take(g);
  w.poly_lo = w.fine ? take(g) : w.poly;
  w.diag_gram = take(batch * w.side * 4);
  w.diag_poly = take(batch * w.side * 4);
  w.done = take(batch * 4);
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

// Pairs of CTAs that are resident together: what a cooperative launch may have.
template <bool CAREFUL>
static cudaError_t ortho_pairs(cudaLaunchConfig_t& cfg, int* pairs) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = known[dev & 63].load();
  if (n == 0) {
    e = cudaFuncSetAttribute(ortho_kernel<CAREFUL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)cfg.dynamicSmemBytes);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, ortho_kernel<CAREFUL>, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    known[dev & 63].store(n);
  }
  *pairs = n;
  return cudaSuccess;
}
template <bool CAREFUL>
static cudaError_t launch_ortho(const OrthoSteps& s, int64_t tasks, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
  cfg.blockDim = dim3(kOrthoThreads);
  cfg.dynamicSmemBytes = (size_t)kRingBytes + kSideBytes + kNoteBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs = 0;
  cudaError_t e = ortho_pairs<CAREFUL>(cfg, &pairs);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(2 * (tasks < pairs ? tasks : pairs)));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ortho_kernel<CAREFUL>, s, (int)tasks);
}

// Tile width: waves of tiles times a tile's steps (see zero_product.cuh's
// measurements of a step at 256 and at 128 columns; at 64 a step is the loads of
// A's rows) and its epilogue.  64 columns only where the contraction lies
// along B's rows, as a box of them holds 64 along its own.  (us of five steps with
// 64 and with 128 at least: 768 x 768, 6 squares of 256 twelve deep, 86.5 and 97.0;
// 1024 x 4096 163 and 179; 257 x 8192 181 and 193; 24 x 1024 x 1024, 240 squares,
// takes 256: 441, and 773 with 128.)
static int tile_width(int64_t squares, int64_t kblocks, bool narrow) {
  const double pairs = (double)(sm_count() / 2), deep = (double)kblocks;
  double best = 0;
  int width = 0;
  for (int bn = 256; bn >= (narrow ? 64 : 128); bn /= 2) {
    const double step = bn == 256 ? 520 : bn == 128 ? 430 : 380;
    const double waves = std::ceil((double)(squares * (256 / bn)) / pairs);
    const double cost = waves * step * deep + 25 * bn;
    if (width && cost >= best) continue;
    best = cost;
    width = bn;
  }
  return width;
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
  s.done = reinterpret_cast<uint32_t*>(base + w.done);
  s.partials = reinterpret_cast<double*>(base + w.partials);
  s.hi = reinterpret_cast<uint16_t*>(base + w.hi[0]);
  s.lo = reinterpret_cast<uint16_t*>(base + w.lo[0]);
  const bool wide = s.x.dtype == ZERO_F32;
  auto grid = [&](const Walk& walk) {
    return dim3(walk.grid.x, walk.grid.y, (unsigned)batch);
  };
  const Walk over = ortho_walk(m, n, batch), padded = ortho_walk(w.rows, w.ld, batch);
  cudaError_t e = launch_next(s.muon ? ortho_squares<true, true>
                              : wide ? ortho_squares<true, false>
                                     : ortho_squares<false, false>,
                              grid(over), dim3(kThreads), st, s, over.log2_across);
  if (e != cudaSuccess) return e;
  e = launch_next(s.muon ? ortho_scale<true, true>
                  : wide ? ortho_scale<true, false>
                         : ortho_scale<false, false>,
                  grid(padded), dim3(kThreads), st, s, padded.log2_across);
  if (e != cudaSuccess) return e;

  if (c.steps > 0) {
    OrthoSteps p{};
    const int64_t sq = batch * squares, kb_far = (far + kDeep - 1) / kDeep,
                  kb_k = (k + kDeep - 1) / kDeep;
    const int bn_gram = tile_width(sq, kb_far, !tall), bn_poly = tile_width(sq, kb_k, true);
    const int passes = w.fine ? 3 : 1;
    const int bn_grow = tile_width(batch * rows * (up(w.ld, 256) / 256), passes * kb_k, tall);
    // Operands by rows (boxes of 128 rows, or half a tile's width of them) or,
    // where the contraction runs down the rows, in boxes of 64 of them.
    const int64_t all = batch * w.rows, sides = batch * w.side;
    void *gram = base + w.gram, *poly = base + w.poly, *poly_lo = base + w.poly_lo;
    OrthoMaps& m = p.maps;
    bool ok = true;
    for (int i = 0; i < 2; ++i) {
      void *hi = base + w.hi[i], *lo = base + w.lo[i];
      ok = ok && half_map(&m.x_a[i], hi, w.ld, all, tall ? 64 : kRowsCta) &&
           half_map(&m.x_b[i], hi, w.ld, all, tall ? 64 : bn_gram / 2) &&
           half_map(&m.x[i], hi, w.ld, all, tall ? kRowsCta : 64) &&
           (!w.fine || half_map(&m.x_lo[i], lo, w.ld, all, tall ? kRowsCta : 64)) &&
           half_map(&m.hi[i], hi, w.ld, all, kRowsCta) &&
           half_map(&m.lo[i], lo, w.ld, all, kRowsCta);
    }
    ok = ok && half_map(&m.gram_a, gram, w.side, sides, kRowsCta) &&
         half_map(&m.gram_b, gram, w.side, sides, bn_poly / 2) &&
         half_map(&m.poly, poly, w.side, sides, tall ? bn_grow / 2 : kRowsCta) &&
         half_map(&m.gram, gram, w.side, sides, kRowsCta) &&
         half_map(&m.gram_t, gram, w.side, sides, 64) &&
         half_map(&m.poly_out, poly, w.side, sides, kRowsCta) &&
         half_map(&m.poly_t, poly, w.side, sides, 64);
    if (w.fine)
      ok = ok && half_map(&m.poly_lo, poly_lo, w.side, sides, tall ? bn_grow / 2 : kRowsCta) &&
           half_map(&m.poly_lo_out, poly_lo, w.side, sides, kRowsCta);
    if (!ok) return cudaErrorInvalidValue;
    OrthoK &g = p.k[GRAM], &q = p.k[POLY], &x = p.k[GROW];
    g.kblocks = (int)kb_far;
    g.bn = bn_gram;
    g.a_c = g.b_c = !tall;
    g.rows_a = g.rows_b = (int)w.rows;
    g.rows_out = (int)w.side;
    g.tiles = (int)(squares * (256 / g.bn));
    q.kblocks = (int)kb_k;
    q.bn = bn_poly;
    q.a_c = q.b_c = 1;
    q.rows_a = q.rows_b = q.rows_out = (int)w.side;
    q.tiles = (int)(squares * (256 / q.bn));
    q.before = g.tiles;
    x.kblocks = (int)kb_k;
    x.bn = bn_grow;
    x.a_c = 1;
    x.b_c = tall;
    x.rows_a = (int)(tall ? w.rows : w.side);
    x.rows_b = (int)(tall ? w.side : w.rows);
    x.rows_out = (int)w.rows;
    x.tiles_j = (int)(up(w.ld, x.bn) / x.bn);
    x.tiles = (int)(rows * x.tiles_j);
    x.before = q.before + q.tiles;
    x.passes = passes;
    g.passes = q.passes = 1;
    for (OrthoK* o : {&g, &q, &x}) {
      o->bn_log2 = o->bn == 256 ? 8 : o->bn == 128 ? 7 : 6;
      o->steps = o->passes * o->kblocks;
    }
    p.steps = c.steps;
    p.batch = (int)batch;
    p.tiles_step = x.before + x.tiles;
    p.cols = (int)w.ld;
    p.tall = tall;
    p.side = (int)w.side;
    p.fine = w.fine;
    const int widest = std::max(g.bn, std::max(q.bn, x.bn));
    p.stage_bytes = kBytesA + widest * kDeep;
    p.stages = std::min(kRingBytes / p.stage_bytes, kMostOrthoStages);
    p.diag_gram = reinterpret_cast<float*>(base + w.diag_gram);
    p.diag_poly = reinterpret_cast<float*>(base + w.diag_poly);
    p.done = s.done;
    for (int i = 0; i < c.steps; ++i)
      for (int j = 0; j < 3; ++j) p.coef[i][j] = c.coef[i][j];
    const int64_t tasks = (int64_t)p.tiles_step * batch * c.steps;
    e = w.fine || kb_far > kOrthoRound ? launch_ortho<true>(p, tasks, st)
                                       : launch_ortho<false>(p, tasks, st);
    if (e != cudaSuccess) return e;
  }
  OrthoFinish f = c.finish;
  f.m = m;
  f.n = n;
  f.rows = w.rows;
  f.ld = w.ld;
  f.x = reinterpret_cast<const uint16_t*>(base + w.hi[c.steps & 1]);
  return launch_next(f.update ? ortho_finish<true> : ortho_finish<false>, grid(over),
                     dim3(kThreads), st, f, over.log2_across);
}

cudaError_t timeouts_ortho(unsigned long long* out, bool reset) {
  return unit_timeouts(out, reset);
}
cudaError_t bounds_ortho(BoundsRec* out, bool reset) { return bounds_record(out, reset); }

}  // namespace zk
