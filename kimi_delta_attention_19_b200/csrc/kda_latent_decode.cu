// kda_latent_decode.cu -- absorbed latent attention over the paged cache: one warp a row.
#include <cuda_fp8.h>

#include "kda_latent.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

__device__ __forceinline__ void ld_row(const CacheArgs& c, int64_t slot, int lane, float (&x)[18]) {
  const __nv_bfloat16* pe;
  if (c.format == KDA_CACHE_BF16) {
    const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(c.cache + slot * DX * 2);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __bfloat162float(row[16 * lane + i]);
    pe = row + DC;
  } else {
    const unsigned char* row = c.cache + slot * kRow8;
    const float e = __uint_as_float(static_cast<uint32_t>(row[kExp8 + lane / 8]) << 23);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw(row[16 * lane + i], __NV_E4M3);
      x[i] = __half2float(__half(h)) * e;
    }
    pe = reinterpret_cast<const __nv_bfloat16*>(row + kPe8);
  }
  x[16] = __bfloat162float(pe[2 * lane]);
  x[17] = __bfloat162float(pe[2 * lane + 1]);
}

__global__ void __launch_bounds__(kWarps * 32) decode_kernel(DecodeLatentArgs a) {
  const int lane = threadIdx.x % 32, rows = a.L * a.H;
  const int row = blockIdx.x * kWarps + threadIdx.x / 32, n = blockIdx.y;
  if (row >= rows) return;
  const int i = row / a.H;
  const int64_t at = static_cast<int64_t>(n) * rows + row;
  const int64_t len = a.lens[n];
  __nv_bfloat16* o = a.out + at * DC + 16 * lane;
  bool bad = len < 0 || len > a.table_pages * a.c.page_size;
  float q[18], acc[16] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int x = 0; x < 16; ++x) q[x] = __bfloat162float(a.q[at * DX + 16 * lane + x]);
  q[16] = __bfloat162float(a.q[at * DX + DC + 2 * lane]);
  q[17] = __bfloat162float(a.q[at * DX + DC + 2 * lane + 1]);
  const int64_t first = len - a.L;  // position of the first query token
  const uint64_t word = a.mask != nullptr ? static_cast<uint64_t>(a.mask[n * a.L + i])
                                          : (2ull << i) - 1;
  for (int64_t j = 0; j < len && !bad; ++j) {
    const int64_t page = a.table[n * a.table_pages + j / a.c.page_size];
    if (page < 0 || page >= a.c.n_pages) {
      bad = true;
      break;
    }
    if (j >= first && !(word >> (j - first) & 1)) continue;
    float x[18], s = 0.f;
    ld_row(a.c, page * a.c.page_size + j % a.c.page_size, lane, x);
#pragma unroll
    for (int k = 0; k < 18; ++k) s += q[k] * x[k];
    s = a.scale * warp_sum(s);
    const float m2 = fmaxf(m, s), ms = m2 == -INFINITY ? 0.f : m2;
    const float c = __expf(m - ms), p = __expf(s - ms);
    l = l * c + p;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = acc[k] * c + p * x[k];
    m = m2;
  }
  if (bad) {
    if (lane == 0 && a.status != nullptr) atomicExch(a.status, kDevBadPage);
    l = NAN;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) st_out(o + k, bad ? NAN : l == 0.f ? 0.f : acc[k] / l);
  if (lane == 0 && a.lse != nullptr) a.lse[at] = bad ? NAN : l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + logf(l);
}

}  // namespace

size_t decode_workspace(int N, int L, int H) { return 256; }

cudaError_t launch_latent_decode(const DecodeLatentArgs& a, cudaStream_t st) {
  decode_kernel<<<dim3((a.L * a.H + kWarps - 1) / kWarps, a.N), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace latent
}  // namespace kda
