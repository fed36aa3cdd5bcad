// kda_latent_tc.cuh -- what the latent-attention tensor-core kernels share: bounded waits,
// the election of an issuing thread, conversions, tensor maps. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <string.h>

#include "kda_latent.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace latent {

using namespace sm100;

// One thread of a converged warp, the same one each time. It runs an issuing role by itself:
// under a branch on it tcgen05.mma goes out every ~30 clocks, under one on `lane == 0` every ~97
// (measured, M = 128, N = 32, 512 in a row), which is more than the instruction takes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(p));
  return p != 0;
}

// Bounded waits. `bail` is a shared word of the CTA: the first wait that runs out (about a
// second) sets it, every later wait returns at once, no further copy is issued, and all loops
// run to their ends (so no named barrier is left short); the CTA then reports kDevWaitTimeout and
// frees its tensor memory. The loading thread always waits (again with a limit) for its last
// copies before it is done, and each issuing thread for its last products, whatever became of
// the others: a wait that runs out after an issuing thread has looked at `bail` must not free
// tensor memory that a product still writes.
#ifndef KDA_LATENT_WAIT_CYCLES  // (the test-only library gives up almost at once)
#define KDA_LATENT_WAIT_CYCLES 2000000000LL
#endif
constexpr long long kWaitCycles = KDA_LATENT_WAIT_CYCLES, kDrainCycles = 100000000LL;
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* bail) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*bail) return;
    if (clock64() - t0 > kWaitCycles) {
      *bail = 1;
      return;
    }
  }
}

// The wait for a unit's last products, behind which results are read. (A test-only library gives
// it up at once: the latest that a wait can run out.)
__device__ __forceinline__ void wait_for_results(uint64_t* bar, uint32_t parity, volatile int* bail) {
#ifdef KDA_LATENT_RESULTS_GIVEN_UP
  *bail = 1;
#else
  wait_for(bar, parity, bail);
#endif
}

__device__ __forceinline__ bool bailed(volatile int* bail) {  // the same answer for a whole warp
  return __any_sync(0xffffffffu, *bail != 0);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two values as bf16 (round to nearest even), `lo` in the lower half
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// pairs of fp32 values, one instruction for both
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r, x, y, z;
  memcpy(&x, &a, 8);
  memcpy(&y, &b, 8);
  memcpy(&z, &c, 8);
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 o;
  memcpy(&o, &r, 8);
  return o;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r, x, y;
  memcpy(&x, &a, 8);
  memcpy(&y, &b, 8);
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  memcpy(&o, &r, 8);
  return o;
}
__device__ __forceinline__ float2 mul2f(float2 a, float2 b) {
  unsigned long long r, x, y;
  memcpy(&x, &a, 8);
  memcpy(&y, &b, 8);
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  memcpy(&o, &r, 8);
  return o;
}
// 3-D tiled bulk copy global -> shared (x innermost, x * sizeof(elem) 16-byte aligned)
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Rows of a staged tile ([128 rows, 128 bytes] swizzled column groups, kRowAtom bytes each) to
// global memory, whole 128-byte lines a quarter warp; `rows` are copied, by `warps` warps.
constexpr uint32_t kRowAtom = 128 * 128;
template <int kGroupsOut>
__device__ __forceinline__ void copy_rows(const unsigned char* tile, unsigned char* dst,
                                          int64_t row_bytes, int row0, int rows, int warp,
                                          int warps, int lane) {
  for (int e = warp * 4 + lane / 8; e < rows * kGroupsOut; e += warps * 4) {
    const int row = row0 + e / kGroupsOut, at = e % kGroupsOut, c = lane % 8;
    *reinterpret_cast<uint4*>(dst + (e / kGroupsOut) * row_bytes + at * 128 + c * 16) =
        *reinterpret_cast<const uint4*>(tile + sw128_chunk(row, at * 8 + c, kRowAtom));
  }
}

// Head and block of place x in the order of a launch: the heads of a group vary fastest, then the
// blocks, then the groups. The CTAs that run at a time then walk few heads' keys, which stay in
// the L2, and a group's heavy blocks still come before its light ones (8K x 32-head prompt 604 us
// with groups of 8, 613 of 16, 605 of 4, 626 with all heads, 638 head by head).
__device__ __forceinline__ void place_of(int x, int H, int blocks, int group, int& h, int& block) {
  const int g = x / (group * blocks), in = x % (group * blocks), width = min(group, H - g * group);
  h = g * group + in % width;
  block = in / width;
}

// Tiled bf16 tensor map of `rank` dimensions (the innermost one contiguous, strides in bytes
// of the others), whose boxes land in the 128-byte-swizzled operand layout.
bool make_tensor_map(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box);

// Map of a [rows, heads, channels] tensor (strides in elements) in boxes of 64 channels of one
// head and `box_rows` rows; rows < 1 makes a map no copy may use.
bool make_head_map(CUtensorMap* m, const void* ptr, int channels, int64_t heads, int64_t head,
                   int64_t rows, int64_t token, uint32_t box_rows);

// Launches a kernel that may be scheduled while what is before it on the stream finishes (once
// every CTA there has triggered or ended); it calls griddep_wait() before it reads or writes
// anything another kernel touches.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// The device's SM count (148 on B200): the width of the persistent grids.
int sm_count();

}  // namespace latent
}  // namespace kda
