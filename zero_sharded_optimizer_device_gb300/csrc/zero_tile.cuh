// What kernels on the 5th-generation tensor cores share: TMA, mbarriers with
// bounded waits, tensor memory and the products' instructions, cluster pairs.
#pragma once

#include <cuda.h>

#include <atomic>
#include <utility>

#include "zero_ops_device.cuh"

namespace zk {

constexpr int kRowsCta = 128;          // rows of A per CTA (tensor-memory lanes)
constexpr int kDeep = 64;              // contraction per stage: 128 bytes, one swizzle row
constexpr int kBytesA = kRowsCta * kDeep * 2;
constexpr int kSmemMost = 232448;      // shared memory one CTA may have
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s; bounds every wait

static __device__ unsigned long long g_ops_timeouts;  // one per translation unit

// ------------------------------------------------------------ PTX wrappers --
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// One lane of a converged warp, always the same.  Roles that issue from one lane
// run their loops on the whole warp, where addresses and counters live in uniform
// registers, from which TMA and the tensor cores take their operands (a loop of
// many forms inside `if (lane == 0)` took ~650 cycles per stage); or that lane runs
// a loop of one form alone, made for it (4-bit steps 400 to 470 cycles instead of
// 510 to 600, Newton-Schulz steps 300 instead of 430).
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile(
      "{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// Acquires at cluster scope (no measurable cost): the arrivals waited for may
// be the other CTAs'.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; "
      "selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done;
}
// Wait for the phase of this parity.  Gives up after kWaitCycles, or once another
// role of the CTA has (*dead), counts the first giving up and returns false:
// the role then goes through the rest of its loop without waiting or issuing
// anything, and the kernel returns.
// COPY: kernels that call one copy of it also share what it does to their registers
// (two Newton-Schulz kernels with one: 768 x 768 110.4 us, with one each 108.5; 12
// products with one: 64 x 4096 to 4096 14.3 us, 1000 x 777 from 1030, odd, 20.2; with one
// each 14.2 and 19.6).
template <int COPY = 0>
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity,
                                                  volatile int* dead) {
  const long long t0 = clock64();
  while (!bar_try(bar, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > kWaitCycles) {
      *dead = 1;
      atomicAdd(&g_ops_timeouts, 1ull);
      return false;
    }
  }
  return true;
}
template <int COPY = 0>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
  if (bar_try(bar, parity)) return true;
  return bar_wait_slow<COPY>(bar, parity, dead);
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// One arrival on a barrier of any CTA of the cluster, behind everything this
// thread has written or seen written.
__device__ __forceinline__ void bar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
// The same where a fence already orders what is handed over: writes, one of the
// cluster's scope before it; tensor memory, the tcgen05 fences on both sides.
// (A release would wait for an epilogue's stores: 509 x 768 to 50257 fp32
// takes 55 us with it, 48 without.)
__device__ __forceinline__ void bar_arrive_fenced(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
// What this thread has written to, or seen written to, its CTA's shared memory
// is in place for whoever in the cluster acquires its next arrival.  (Weight
// gradient 4593 x 6451 x 1184 fp32, shifted operands: 96 us; a warp of the
// second CTA that forwards arrivals with a full release 149, one full fence for
// all stages at hand 121.)
__device__ __forceinline__ void release_shared() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
// A box of a matrix into this CTA's shared memory, counted on the barrier of
// the pair's first CTA.  x is a multiple of 64 elements.
__device__ __forceinline__ void tma_load(const CUtensorMap* map, uint32_t dst, int x, int y,
                                         uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}
// Boxes of side operands and results: this CTA's own barrier and memory.
__device__ __forceinline__ void box_load(const CUtensorMap* map, uint32_t dst, int x, int y,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void box_store(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::
                   "l"(map),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Tensor-core arrivals: when every instruction issued so far is done, one
// arrival on this barrier of both CTAs of the pair.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t r[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t r[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t r[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t r[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t r[N]) {
  if constexpr (N == 32)
    tmem_load32(addr, r);
  else
    tmem_load16(addr, r);
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t r[N]) {
  if constexpr (N == 32)
    tmem_store32(addr, r);
  else
    tmem_store16(addr, r);
}
// r += the N columns at addr.
template <int N>
__device__ __forceinline__ void tmem_add(uint32_t addr, uint32_t r[N]) {
  uint32_t q[N];
  tmem_load<N>(addr, q);
#pragma unroll
  for (int i = 0; i < N; ++i)
    r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(q[i]));
}
__device__ __forceinline__ void st_shared4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(a), "f"(b), "f"(c),
               "f"(d));
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, const uint32_t r[4]) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]));
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(addr));
  return u;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 u) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(u.x), "r"(u.y), "r"(u.z),
               "r"(u.w));
}
// Reads and writes of shared memory above are volatile, hence kept in order,
// but do not clobber memory: a clobber makes the compiler fetch every kernel
// parameter again at its next use, ~70 cycles each in a row.

// Shared-memory descriptor of an operand tile in 128-byte swizzle rows.
// Contiguous contraction: rows of 64 values, 8-row groups 1024 bytes apart.
// Contiguous rows: blocks of 64 rows x 64 deep (8192 bytes apart: the leading
// offset), 8-deep groups 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool contig) {
  const uint64_t lead = contig ? 1 : (8192 >> 4), stride = 1024 >> 4;
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (lead << 16) | (stride << 32) | (1ull << 46) |
         (2ull << 61);
}

__device__ __forceinline__ float4 ld_shared4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// ------------------------------------------------------------------- host --
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load();
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f);
  }
  return reinterpret_cast<EncodeFn>(f);
}

static bool encode(CUtensorMap* map, bool f32, void* p, int64_t inner, int64_t outer, int64_t ld,
                   int box_x, int box_y, CUtensorMapSwizzle swizzle) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const int es = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  // a single line has no distance to the next: any multiple of 16 bytes will do
  const cuuint64_t strides[1] = {
      (cuuint64_t)(outer > 1 ? ld * es : (inner * es + 15) / 16 * 16)};
  const cuuint32_t box[2] = {(cuuint32_t)box_x, (cuuint32_t)box_y};
  const cuuint32_t one[2] = {1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p,
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// This unit's bounded waits that gave up.
static cudaError_t unit_timeouts(unsigned long long* out, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_ops_timeouts, sizeof(unsigned long long));
  if (e == cudaSuccess && reset) {
    const unsigned long long zero = 0;
    e = cudaMemcpyToSymbol(g_ops_timeouts, &zero, sizeof(zero));
  }
  return e;
}

}  // namespace zk
