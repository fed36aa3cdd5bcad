// kda_latent.cuh -- declarations shared by the latent-attention translation units.
// Not part of the public ABI (that is include/kda.h).
#pragma once

#include <math.h>

#include "kda_internal.cuh"

namespace kda {
namespace latent {

constexpr int DN = 128, DP = 64, DV = 128;  // expanded head: k_nope, shared k_pe, v
constexpr int DQK = DN + DP;
constexpr int DC = 512;                     // latent
constexpr int DX = DC + DP;                 // a cached vector
constexpr int kRow8 = KDA_CACHE_E4M3_ROW_BYTES;
constexpr int kPe8 = DC, kExp8 = DC + 2 * DP;  // byte offsets of k_pe and the exponents
constexpr int kMaxDraft = 64;
constexpr int32_t kDevBadPage = kDevBadSlot;

// Where calls without a status word of their own report: a word of the source file on the device
// (one each, as a file's kernels cannot name another's variables, and a call need not look an
// address up), and what take_status read there last.
[[maybe_unused]] static __device__ int32_t g_word, g_taken;

__device__ __forceinline__ void report(int32_t* status, int32_t code) {
  atomicExch(status != nullptr ? status : &g_word, code);
}

[[maybe_unused]] static __global__ void take_kernel() { g_taken = atomicExch(&g_word, kDevOk); }

// Reads and clears this file's word on the current device, behind the work on `st`, which it
// synchronises. One call at a time (g_taken).
[[maybe_unused]] static cudaError_t take_status(cudaStream_t st, int32_t* code) {
  take_kernel<<<1, 1, 0, st>>>();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(code, g_taken, sizeof *code, 0, cudaMemcpyDeviceToHost, st);
  return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}
cudaError_t take_fwd_status(cudaStream_t st, int32_t* code);
cudaError_t take_bwd_status(cudaStream_t st, int32_t* code);
cudaError_t take_decode_status(cudaStream_t st, int32_t* code);
cudaError_t take_cache_status(cudaStream_t st, int32_t* code);

// Expanded form, resolved on the host.
struct AttnArgs {
  const __nv_bfloat16 *q, *kn, *kp, *v;
  const int32_t *cu_q, *cu_k;  // both or neither
  __nv_bfloat16* out;
  float* lse;                  // or null (forward only)
  int64_t Tq, Tk;              // rows of one sequence (no cu) or of the packed tensors
  int64_t max_q, max_k;
  int64_t qt, qh, kt, kh, pt, vt, vh;
  int n_seqs, H, causal;
  float scale;
  int32_t* status;
  // backward
  const __nv_bfloat16 *o, *dout;
  const float* lse_in;
  float2* stat;                // workspace: (lse log2 e, D) [H, Tq_total]
  float* dpe_part;             // workspace: [H, Tk_total, DP]
  __nv_bfloat16 *dq, *dkn, *dkp, *dv;
};

// Rows [t0, t0 + len) of a sequence's queries and keys.
struct SeqRange {
  int64_t q0, k0;
  int lq, lk;
};

// False when the sequence is malformed or longer than its bound (reported): skip it.
__device__ __forceinline__ bool seq_range(const AttnArgs& a, int s, SeqRange& r) {
  if (a.cu_q == nullptr) {
    r.q0 = s * a.Tq;
    r.k0 = s * a.Tk;
    r.lq = static_cast<int>(a.Tq);
    r.lk = static_cast<int>(a.Tk);
    return true;
  }
  const int64_t q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.Tq && k0 >= 0 && k1 >= k0 && k1 <= a.Tk &&
                  (s != 0 || (q0 == 0 && k0 == 0)) && q1 - q0 <= a.max_q && k1 - k0 <= a.max_k;
  if (!ok) {
    report(a.status, kDevBadSeqlens);
    return false;
  }
  r.q0 = q0;
  r.k0 = k0;
  r.lq = static_cast<int>(q1 - q0);
  r.lk = static_cast<int>(k1 - k0);
  return true;
}

struct CacheArgs {
  const unsigned char* cache;
  int64_t n_pages;
  int page_size, format;
};

struct DecodeLatentArgs {
  CacheArgs c;
  const __nv_bfloat16* q;
  const int32_t *table, *lens;
  const int64_t* mask;
  __nv_bfloat16* out;
  float* lse;
  int64_t table_pages;
  int N, L, H;
  float scale;
  unsigned char* ws;
  int32_t* status;
};

cudaError_t launch_attn_fwd(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t st);
size_t decode_workspace(int L, int H);
cudaError_t launch_latent_decode(const DecodeLatentArgs& a, cudaStream_t st);
cudaError_t launch_cache_write(const __nv_bfloat16* c, int64_t c_token, const __nv_bfloat16* pe,
                               int64_t pe_token, const int64_t* slots, int64_t T,
                               const CacheArgs& cache, int32_t* status, cudaStream_t st);
cudaError_t launch_cache_read(const CacheArgs& cache, const int32_t* table, int64_t table_pages,
                              const int32_t* cu, const int32_t* starts, int n_seqs, int64_t T,
                              __nv_bfloat16* out, int32_t* status, cudaStream_t st);

}  // namespace latent
}  // namespace kda
