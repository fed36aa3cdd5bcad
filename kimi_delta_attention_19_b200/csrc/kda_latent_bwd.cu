// kda_latent_bwd.cu -- expanded latent attention, backward: one warp a row.
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

// lane's channels of a row: 4 of k_nope / v (at 4 lane), 2 of k_pe (at 2 lane)
__device__ __forceinline__ void ld4(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xffff0000u);
  x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void ld2(const __nv_bfloat16* p, float (&x)[2]) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  x[0] = __uint_as_float(w << 16); x[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ float dot4(const float (&a)[4], const float (&b)[4]) {
  return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}

// First key query i does not see.
__device__ __forceinline__ int key_end(const AttnArgs& a, const SeqRange& r, int i) {
  return a.causal ? max(0, min(r.lk, i + 1 + r.lk - r.lq)) : r.lk;
}

__global__ void __launch_bounds__(kWarps * 32) dq_kernel(AttnArgs a) {
  const int lane = threadIdx.x % 32, h = blockIdx.y;
  SeqRange r;
  if (!seq_range(a, blockIdx.z, r)) return;
  const int i = blockIdx.x * kWarps + threadIdx.x / 32;
  if (i >= r.lq) return;
  const int64_t t = r.q0 + i, row = t * a.H + h;
  float qn[4], qp[2], g[4], o[4], dn[4] = {0.f, 0.f, 0.f, 0.f}, dp[2] = {0.f, 0.f};
  ld4(a.q + t * a.qt + h * a.qh + 4 * lane, qn);
  ld2(a.q + t * a.qt + h * a.qh + DN + 2 * lane, qp);
  ld4(a.dout + row * DV + 4 * lane, g);
  ld4(a.o + row * DV + 4 * lane, o);
  const float delta = warp_sum(dot4(g, o)), lse = a.lse_in[row];
  if (lane == 0) a.delta[row] = delta;
  const int end = key_end(a, r, i);
  for (int j = 0; j < end; ++j) {
    float kn[4], kp[2], v[4];
    ld4(a.kn + (r.k0 + j) * a.kt + h * a.kh + 4 * lane, kn);
    ld2(a.kp + (r.k0 + j) * a.pt + 2 * lane, kp);
    ld4(a.v + (r.k0 + j) * a.vt + h * a.vh + 4 * lane, v);
    const float s = a.scale * warp_sum(dot4(qn, kn) + qp[0] * kp[0] + qp[1] * kp[1]);
    const float ds = a.scale * __expf(s - lse) * (warp_sum(dot4(g, v)) - delta);
#pragma unroll
    for (int x = 0; x < 4; ++x) dn[x] += ds * kn[x];
#pragma unroll
    for (int x = 0; x < 2; ++x) dp[x] += ds * kp[x];
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) st_out(a.dq + row * DQK + 4 * lane + x, dn[x]);
#pragma unroll
  for (int x = 0; x < 2; ++x) st_out(a.dq + row * DQK + DN + 2 * lane + x, dp[x]);
}

__global__ void __launch_bounds__(kWarps * 32) dkv_kernel(AttnArgs a, int64_t tk_total) {
  const int lane = threadIdx.x % 32, h = blockIdx.y;
  SeqRange r;
  if (!seq_range(a, blockIdx.z, r)) return;
  const int j = blockIdx.x * kWarps + threadIdx.x / 32;
  if (j >= r.lk) return;
  const int64_t t = r.k0 + j, row = t * a.H + h;
  float kn[4], kp[2], v[4], dn[4] = {0.f, 0.f, 0.f, 0.f}, dp[2] = {0.f, 0.f}, dv[4] = {0.f, 0.f, 0.f, 0.f};
  ld4(a.kn + t * a.kt + h * a.kh + 4 * lane, kn);
  ld2(a.kp + t * a.pt + 2 * lane, kp);
  ld4(a.v + t * a.vt + h * a.vh + 4 * lane, v);
  for (int i = a.causal ? max(0, j - (r.lk - r.lq)) : 0; i < r.lq; ++i) {
    const int64_t qr = (r.q0 + i) * a.H + h;
    float qn[4], qp[2], g[4];
    ld4(a.q + (r.q0 + i) * a.qt + h * a.qh + 4 * lane, qn);
    ld2(a.q + (r.q0 + i) * a.qt + h * a.qh + DN + 2 * lane, qp);
    ld4(a.dout + qr * DV + 4 * lane, g);
    const float s = a.scale * warp_sum(dot4(qn, kn) + qp[0] * kp[0] + qp[1] * kp[1]);
    const float p = __expf(s - a.lse_in[qr]);
    const float ds = a.scale * p * (warp_sum(dot4(g, v)) - a.delta[qr]);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      dn[x] += ds * qn[x];
      dv[x] += p * g[x];
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) dp[x] += ds * qp[x];
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    st_out(a.dkn + row * DN + 4 * lane + x, dn[x]);
    st_out(a.dv + row * DV + 4 * lane + x, dv[x]);
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) a.dpe_part[(h * tk_total + t) * DP + 2 * lane + x] = dp[x];
}

// dk_pe = the heads' parts, summed in the heads' order
__global__ void dpe_kernel(AttnArgs a, int64_t tk_total) {
  SeqRange r;
  if (!seq_range(a, blockIdx.z, r)) return;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (e >= static_cast<int64_t>(r.lk) * DP) return;
  const int64_t at = r.k0 * DP + e;
  float s = 0.f;
  for (int h = 0; h < a.H; ++h) s += a.dpe_part[h * tk_total * DP + at];
  st_out(a.dkp + at, s);
}

unsigned blocks(int64_t n, int per) { return static_cast<unsigned>((n + per - 1) / per); }

}  // namespace

cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t st) {
  const int64_t tk_total = a.cu_k != nullptr ? a.Tk : a.Tk * a.n_seqs;
  if (a.max_q > 0) dq_kernel<<<dim3(blocks(a.max_q, kWarps), a.H, a.n_seqs), kWarps * 32, 0, st>>>(a);
  if (a.max_k > 0) {
    dkv_kernel<<<dim3(blocks(a.max_k, kWarps), a.H, a.n_seqs), kWarps * 32, 0, st>>>(a, tk_total);
    dpe_kernel<<<dim3(blocks(a.max_k * DP, 256), 1, a.n_seqs), 256, 0, st>>>(a, tk_total);
  }
  return cudaGetLastError();
}

}  // namespace latent
}  // namespace kda
