// kda_latent_cache.cu -- the paged latent cache: tokens written into it, in bf16 or with the
// latent in 8 bits, and read back.
//
// An 8-bit row holds, for each 128-channel group of the latent, the e4m3 codes of x / 2^e
// with e the smallest integer for which the group's largest finite magnitude is at most
// 448 * 2^e: with amax = m 2^k, 1 <= m < 2, and 448 = 1.75 * 2^8, e = k - 8 + (m > 1.75). A
// power of two makes x / 2^e exact, so the code's is the only rounding (half a step: 2^-4
// relative for normal codes), and every stored value, 4 significant bits times 2^e, is a
// bf16 number: reading back rounds nothing.
//
// Bound by memory: 1152 bytes in and 644 out a token (or the reverse). One warp kTokens tokens,
// 16 channels a lane, so a group is 8 lanes and its maximum three shuffles. A warp's loads are
// all issued before anything is looked at (rows of tokens that turn out to be skipped
// included): the kernels are short chains of memory latencies (with the slot and the page
// waited for first, a write and a read of 61 K tokens took 53 us).
#include <cuda_fp8.h>

#include "kda_latent_tc.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 2;  // (1: 46.6 us, 2: 45.7, 4: 49.4 for a write and a read of 61 K tokens)

// e4m3 codes of two values already divided by their scale; not finite -> NaN
__device__ __forceinline__ uint32_t codes2(float x, float y) {
  uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
  if (!isfinite(x)) c |= 0x7f;
  if (!isfinite(y)) c |= 0x7f00;
  return c;
}

__device__ __forceinline__ float2 unpack(uint32_t b) {
  return make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}

template <bool F8>
__global__ void __launch_bounds__(kWarps * 32)
    cache_write_kernel(const __nv_bfloat16* c, int64_t c_token, const __nv_bfloat16* pe,
                       int64_t pe_token, const int64_t* slots, int64_t T, CacheArgs cache,
                       int32_t* status) {
  const int lane = threadIdx.x % 32;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32) * kTokens;
  griddep_launch_dependents();
  griddep_wait();
  if (t0 >= T) return;
  uint4 v[kTokens][2], p[kTokens];
  int64_t slot[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int64_t t = t0 + i < T ? t0 + i : T - 1;
    const uint4* src = reinterpret_cast<const uint4*>(c + t * c_token);
    slot[i] = t0 + i < T ? slots[t] : -1;
    v[i][0] = __ldcs(src + (F8 ? 2 * lane : lane));
    v[i][1] = __ldcs(src + (F8 ? 2 * lane + 1 : lane + 32));
    if (lane < 8) p[i] = __ldcs(reinterpret_cast<const uint4*>(pe + t * pe_token) + lane);
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    if (slot[i] < 0) continue;
    if (slot[i] >= cache.n_pages * cache.page_size) {
      if (lane == 0) report(status, kDevBadPage);
      continue;
    }
    unsigned char* row = const_cast<unsigned char*>(cache.cache) + slot[i] * (F8 ? kRow8 : DX * 2);
    if constexpr (!F8) {
      uint4* dst = reinterpret_cast<uint4*>(row);
      dst[lane] = v[i][0];
      dst[lane + 32] = v[i][1];
      if (lane < 8) dst[64 + lane] = p[i];
    } else {
      const uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w,
                             v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
      uint32_t amax = 0;  // the largest finite magnitude's bits (bf16 order = integer order)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t lo = w[k] & 0x7fffu, hi = w[k] >> 16 & 0x7fffu;
        if (lo < 0x7f80u && lo > amax) amax = lo;
        if (hi < 0x7f80u && hi > amax) amax = hi;
      }
#pragma unroll
      for (int off = 4; off > 0; off >>= 1)
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      int e = static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 0x7fu) > 0x60u);
      e = max(-120, min(120, e));
      const float inv = __int_as_float((127 - e) << 23);
      uint32_t code[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = unpack(w[2 * k]), y = unpack(w[2 * k + 1]);
        code[k] = codes2(x.x * inv, x.y * inv) | codes2(y.x * inv, y.y * inv) << 16;
      }
      reinterpret_cast<uint4*>(row)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
      uint32_t exps = 0;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        exps |= static_cast<uint32_t>(__shfl_sync(0xffffffffu, e, 8 * g) + 127) << (8 * g);
      if (lane < 8) reinterpret_cast<uint4*>(row + kPe8)[lane] = p[i];
      if (lane == 8) *reinterpret_cast<uint4*>(row + kExp8) = make_uint4(exps, 0, 0, 0);
    }
  }
}

// Two bf16 values of two e4m3 codes times 2^e (exact)
__device__ __forceinline__ uint32_t values2(uint32_t codes, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * scale, f.y * scale);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <bool F8>
__global__ void __launch_bounds__(kWarps * 32)
    cache_read_kernel(CacheArgs cache, const int32_t* table, int64_t table_pages,
                      const int32_t* cu, const int32_t* starts, int n_seqs, int64_t T,
                      __nv_bfloat16* out, int32_t* status) {
  const int lane = threadIdx.x % 32;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32) * kTokens;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t end = min(T, static_cast<int64_t>(cu[n_seqs]));
  if (t0 >= end) return;
  int lo = 0, hi = n_seqs;  // the last s in [0, n_seqs) with cu[s] <= t0
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= t0) lo = mid; else hi = mid;
  }
  const int shift = 31 - __clz(cache.page_size);
  int64_t slot[kTokens];  // -1: past the end, -2: a page out of range
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int64_t t = t0 + i;
    while (lo + 1 < n_seqs && cu[lo + 1] <= t) ++lo;
    slot[i] = -1;
    if (t >= end) continue;
    const int64_t first = cu[lo], pos = t - first + (starts != nullptr ? starts[lo] : 0);
    int64_t page = -1;
    if (t >= first && pos >= 0 && (pos >> shift) < table_pages)
      page = table[static_cast<int64_t>(lo) * table_pages + (pos >> shift)];
    slot[i] = page < 0 || page >= cache.n_pages ? -2 : (page << shift) + (pos & (cache.page_size - 1));
  }
  uint4 v[kTokens][2], p[kTokens];
  uint32_t exps[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    if (slot[i] < 0) continue;
    const unsigned char* row = cache.cache + slot[i] * (F8 ? kRow8 : DX * 2);
    const uint4* src = reinterpret_cast<const uint4*>(row);
    v[i][0] = __ldcs(src + lane);
    if constexpr (F8) {
      exps[i] = *reinterpret_cast<const uint32_t*>(row + kExp8);
      if (lane < 8) p[i] = __ldcs(reinterpret_cast<const uint4*>(row + kPe8) + lane);
    } else {
      v[i][1] = __ldcs(src + lane + 32);
      if (lane < 8) p[i] = __ldcs(src + 64 + lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    if (slot[i] == -1) continue;
    uint4* dst = reinterpret_cast<uint4*>(out + (t0 + i) * DX);
    if (slot[i] == -2) {
      if (lane == 0) report(status, kDevBadPage);
      const uint4 nan = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      dst[lane] = nan;
      dst[lane + 32] = nan;
      if (lane < 8) dst[64 + lane] = nan;
      continue;
    }
    if constexpr (F8) {
      const uint32_t e = exps[i] >> (8 * (lane / 8)) & 0xffu;
      const float scale = __uint_as_float(max(e << 23, 0x00400000u));  // (2^-127: a subnormal)
      const uint32_t w[4] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w};
      uint32_t r[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        r[2 * k] = values2(w[k] & 0xffffu, scale);
        r[2 * k + 1] = values2(w[k] >> 16, scale);
      }
      dst[2 * lane] = make_uint4(r[0], r[1], r[2], r[3]);
      dst[2 * lane + 1] = make_uint4(r[4], r[5], r[6], r[7]);
    } else {
      dst[lane] = v[i][0];
      dst[lane + 32] = v[i][1];
    }
    if (lane < 8) dst[64 + lane] = p[i];
  }
}

unsigned grid_of(int64_t T) {
  return static_cast<unsigned>((T + kWarps * kTokens - 1) / (kWarps * kTokens));
}

}  // namespace

cudaError_t launch_cache_write(const __nv_bfloat16* c, int64_t c_token, const __nv_bfloat16* pe,
                               int64_t pe_token, const int64_t* slots, int64_t T,
                               const CacheArgs& cache, int32_t* status, cudaStream_t st) {
  auto kern = cache.format == KDA_CACHE_E4M3 ? cache_write_kernel<true> : cache_write_kernel<false>;
  return launch_early(kern, dim3(grid_of(T)), kWarps * 32, 0, st, c, c_token, pe, pe_token, slots, T,
                      cache, status);
}

cudaError_t launch_cache_read(const CacheArgs& cache, const int32_t* table, int64_t table_pages,
                              const int32_t* cu, const int32_t* starts, int n_seqs, int64_t T,
                              __nv_bfloat16* out, int32_t* status, cudaStream_t st) {
  auto kern = cache.format == KDA_CACHE_E4M3 ? cache_read_kernel<true> : cache_read_kernel<false>;
  return launch_early(kern, dim3(grid_of(T)), kWarps * 32, 0, st, cache, table, table_pages, cu, starts,
                      n_seqs, T, out, status);
}

cudaError_t take_cache_status(cudaStream_t st, int32_t* code) { return take_status(st, code); }

}  // namespace latent
}  // namespace kda
