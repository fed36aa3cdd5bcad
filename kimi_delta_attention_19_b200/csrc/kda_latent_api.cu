// kda_latent_api.cu -- the latent-attention part of the C ABI (include/kda.h): argument
// checks, workspace layout and dispatch. Nothing here allocates or synchronises.
#include <mutex>

#include "kda_latent.cuh"

namespace kda {
namespace latent {
namespace {

bool misaligned(const void* p, uintptr_t a = 15u) {
  return (reinterpret_cast<uintptr_t>(p) & a) != 0;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

constexpr int64_t kMaxTokens = 0x7fffffff;

bool stride_ok(int64_t s, int64_t at_least) { return s >= at_least && s % 8 == 0 && s < (1LL << 36); }

kda_status check_attn(const kda_latent_shape* s) {
  if (s == nullptr) return KDA_ERR_INVALID_ARG;
  if (s->dtype != KDA_F32 && s->dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (s->H <= 0 || s->B <= 0 || s->Tq < 0 || s->Tk < 0 || s->n_seqs < 0 || s->max_q < 0 ||
      s->max_k < 0)
    return KDA_ERR_INVALID_ARG;
  if (s->n_seqs > 0 && s->B != 1) return KDA_ERR_INVALID_ARG;
  if (s->causal != 0 && s->causal != 1) return KDA_ERR_INVALID_ARG;
  if (!(s->scale >= 0.f) || !isfinite(s->scale)) return KDA_ERR_INVALID_ARG;
  if (s->dtype != KDA_BF16 || s->d_nope != DN || s->d_pe != DP || s->d_v != DV)
    return KDA_ERR_UNSUPPORTED;
  if (!stride_ok(s->q_head, DQK) || !stride_ok(s->q_token, DQK) || !stride_ok(s->k_head, DN) ||
      !stride_ok(s->k_token, DN) || !stride_ok(s->pe_token, DP) || !stride_ok(s->v_head, DV) ||
      !stride_ok(s->v_token, DV))
    return KDA_ERR_INVALID_ARG;
  // token counts and grid dimensions
  if (s->H > 65535 || s->B > 65535 || s->n_seqs > 65535 || s->Tq > kMaxTokens ||
      s->Tk > kMaxTokens || s->Tq * s->B > kMaxTokens || s->Tk * s->B > kMaxTokens)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

void fill(AttnArgs& a, const void* q, const void* kn, const void* kp, const void* v,
          const int32_t* cu_q, const int32_t* cu_k, const kda_latent_shape& s, int32_t* status) {
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.kn = static_cast<const __nv_bfloat16*>(kn);
  a.kp = static_cast<const __nv_bfloat16*>(kp);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.Tq = s.Tq;
  a.Tk = s.Tk;
  const bool packed = s.n_seqs > 0;
  a.n_seqs = packed ? s.n_seqs : s.B;
  a.max_q = packed && s.max_q > 0 && s.max_q < s.Tq ? s.max_q : s.Tq;
  a.max_k = packed && s.max_k > 0 && s.max_k < s.Tk ? s.max_k : s.Tk;
  a.qt = s.q_token; a.qh = s.q_head;
  a.kt = s.k_token; a.kh = s.k_head;
  a.pt = s.pe_token;
  a.vt = s.v_token; a.vh = s.v_head;
  a.H = s.H;
  a.causal = s.causal;
  a.scale = s.scale > 0.f ? s.scale : 1.0f / sqrtf(static_cast<float>(DQK));
  a.status = status;
}

// Pointers every call of the expanded form takes.
bool bad_inputs(const void* q, const void* kn, const void* kp, const void* v,
                const int32_t* cu_q, const int32_t* cu_k, const kda_latent_shape& s,
                const int32_t* status) {
  if ((cu_q != nullptr) != (s.n_seqs > 0) || (cu_k != nullptr) != (s.n_seqs > 0)) return true;
  if (misaligned(cu_q, 3) || misaligned(cu_k, 3) || misaligned(status, 3)) return true;
  if (misaligned(q) || misaligned(kn) || misaligned(kp) || misaligned(v)) return true;
  if (s.Tq > 0 && q == nullptr) return true;
  return s.Tk > 0 && (kn == nullptr || kp == nullptr || v == nullptr);
}

struct BwdLayout {
  size_t stat, dpe, total;
};

BwdLayout bwd_layout(const kda_latent_shape& s) {
  BwdLayout l;
  const size_t tq = static_cast<size_t>(s.Tq) * s.B, tk = static_cast<size_t>(s.Tk) * s.B;
  l.stat = 0;
  l.dpe = align_up(tq * s.H * 8, 256);
  l.total = align_up(l.dpe + tk * s.H * DP * 4, 256);
  if (l.total == 0) l.total = 256;
  return l;
}

kda_status check_cache(const kda_latent_cache* c) {
  if (c == nullptr || c->n_pages < 0) return KDA_ERR_INVALID_ARG;
  if (c->format != KDA_CACHE_BF16 && c->format != KDA_CACHE_E4M3) return KDA_ERR_INVALID_ARG;
  if (c->page_size <= 0) return KDA_ERR_INVALID_ARG;
  if (c->d_c != DC || c->d_pe != DP) return KDA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return KDA_ERR_UNSUPPORTED;
  if (c->n_pages > kMaxTokens / c->page_size) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

CacheArgs cache_args(const void* cache, const kda_latent_cache& c) {
  return CacheArgs{static_cast<const unsigned char*>(cache), c.n_pages, c.page_size, c.format};
}

kda_status check_decode(const kda_latent_decode_shape* s) {
  if (s == nullptr || s->N <= 0 || s->L <= 0 || s->H <= 0 || s->table_pages < 0)
    return KDA_ERR_INVALID_ARG;
  if (s->dtype != KDA_F32 && s->dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (!(s->scale >= 0.f) || !isfinite(s->scale)) return KDA_ERR_INVALID_ARG;
  if (s->dtype != KDA_BF16 || s->L > kMaxDraft || s->H > 1024 || s->N > 65535)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace
}  // namespace latent
}  // namespace kda

using namespace kda::latent;

extern "C" {

kda_status kda_latent_attn_fwd(const void* q, const void* k_nope, const void* k_pe,
                               const void* v, const int32_t* cu_seqlens_q,
                               const int32_t* cu_seqlens_k, void* out, float* lse,
                               const kda_latent_shape* shape, int32_t* status,
                               kda_stream_t stream) {
  const kda_status st = check_attn(shape);
  if (st != KDA_OK) return st;
  if (bad_inputs(q, k_nope, k_pe, v, cu_seqlens_q, cu_seqlens_k, *shape, status) ||
      misaligned(out) || misaligned(lse, 3) || (shape->Tq > 0 && out == nullptr))
    return KDA_ERR_INVALID_ARG;
  AttnArgs a{};
  fill(a, q, k_nope, k_pe, v, cu_seqlens_q, cu_seqlens_k, *shape, status);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  if (a.max_q == 0) return KDA_OK;
  return of(launch_attn_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_latent_attn_bwd_workspace_size(const kda_latent_shape* shape) {
  return check_attn(shape) == KDA_OK ? bwd_layout(*shape).total : 0;
}

kda_status kda_latent_attn_bwd(const void* q, const void* k_nope, const void* k_pe,
                               const void* v, const void* out, const float* lse,
                               const void* d_out, const int32_t* cu_seqlens_q,
                               const int32_t* cu_seqlens_k, void* dq, void* dk_nope,
                               void* dk_pe, void* dv, const kda_latent_shape* shape,
                               void* workspace, size_t workspace_bytes, int32_t* status,
                               kda_stream_t stream) {
  const kda_status st = check_attn(shape);
  if (st != KDA_OK) return st;
  if (bad_inputs(q, k_nope, k_pe, v, cu_seqlens_q, cu_seqlens_k, *shape, status) ||
      misaligned(out) || misaligned(lse, 3) || misaligned(d_out) || misaligned(dq) ||
      misaligned(dk_nope) || misaligned(dk_pe) || misaligned(dv))
    return KDA_ERR_INVALID_ARG;
  if (shape->Tq > 0 && (out == nullptr || lse == nullptr || d_out == nullptr || dq == nullptr))
    return KDA_ERR_INVALID_ARG;
  if (shape->Tk > 0 && (dk_nope == nullptr || dk_pe == nullptr || dv == nullptr))
    return KDA_ERR_INVALID_ARG;
  const BwdLayout l = bwd_layout(*shape);
  if (workspace == nullptr || workspace_bytes < l.total || misaligned(workspace, 255))
    return KDA_ERR_INVALID_ARG;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  AttnArgs a{};
  fill(a, q, k_nope, k_pe, v, cu_seqlens_q, cu_seqlens_k, *shape, status);
  a.o = static_cast<const __nv_bfloat16*>(out);
  a.lse_in = lse;
  a.dout = static_cast<const __nv_bfloat16*>(d_out);
  a.stat = reinterpret_cast<float2*>(ws + l.stat);
  a.dpe_part = reinterpret_cast<float*>(ws + l.dpe);
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dkn = static_cast<__nv_bfloat16*>(dk_nope);
  a.dkp = static_cast<__nv_bfloat16*>(dk_pe);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  if (a.max_q == 0 && a.max_k == 0) return KDA_OK;
  return of(launch_attn_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_latent_cache_write(const void* latent, int64_t latent_token, const void* k_pe,
                                  int64_t pe_token, const int64_t* slots, int64_t T,
                                  void* cache, const kda_latent_cache* cache_shape,
                                  int32_t* status, kda_stream_t stream) {
  const kda_status st = check_cache(cache_shape);
  if (st != KDA_OK) return st;
  if (T < 0 || !stride_ok(latent_token, DC) || !stride_ok(pe_token, DP))
    return KDA_ERR_INVALID_ARG;
  if (T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
  if (misaligned(latent) || misaligned(k_pe) || misaligned(slots, 7) || misaligned(cache) ||
      misaligned(status, 3))
    return KDA_ERR_INVALID_ARG;
  if (T == 0) return KDA_OK;
  if (latent == nullptr || k_pe == nullptr || slots == nullptr ||
      (cache == nullptr && cache_shape->n_pages > 0))
    return KDA_ERR_INVALID_ARG;
  return of(launch_cache_write(static_cast<const __nv_bfloat16*>(latent), latent_token,
                               static_cast<const __nv_bfloat16*>(k_pe), pe_token, slots, T,
                               cache_args(cache, *cache_shape), status,
                               reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_latent_cache_read(const void* cache, const int32_t* block_table,
                                 int64_t table_pages, const int32_t* cu_seqlens,
                                 const int32_t* starts, int32_t n_seqs, int64_t T, void* out,
                                 const kda_latent_cache* cache_shape, int32_t* status,
                                 kda_stream_t stream) {
  const kda_status st = check_cache(cache_shape);
  if (st != KDA_OK) return st;
  if (T < 0 || table_pages < 0 || n_seqs <= 0) return KDA_ERR_INVALID_ARG;
  if (T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
  if (misaligned(cache) || misaligned(block_table, 3) || misaligned(cu_seqlens, 3) ||
      misaligned(starts, 3) || misaligned(out) || misaligned(status, 3))
    return KDA_ERR_INVALID_ARG;
  if (T == 0) return KDA_OK;
  if (cu_seqlens == nullptr || out == nullptr || (block_table == nullptr && table_pages > 0) ||
      (cache == nullptr && cache_shape->n_pages > 0))
    return KDA_ERR_INVALID_ARG;
  return of(launch_cache_read(cache_args(cache, *cache_shape), block_table, table_pages,
                              cu_seqlens, starts, n_seqs, T, static_cast<__nv_bfloat16*>(out),
                              status, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_latent_decode_workspace_size(const kda_latent_decode_shape* shape,
                                        const kda_latent_cache* cache_shape) {
  if (check_decode(shape) != KDA_OK || check_cache(cache_shape) != KDA_OK) return 0;
  return align_up(decode_workspace(shape->L, shape->H), 256);
}

kda_status kda_latent_decode(const void* q, const void* cache, const int32_t* block_table,
                             const int32_t* seq_lens, const int64_t* draft_mask, void* out,
                             float* lse, const kda_latent_decode_shape* shape,
                             const kda_latent_cache* cache_shape, void* workspace,
                             size_t workspace_bytes, int32_t* status, kda_stream_t stream) {
  kda_status st = check_decode(shape);
  if (st == KDA_OK) st = check_cache(cache_shape);
  if (st != KDA_OK) return st;
  const kda_latent_decode_shape& s = *shape;
  if (misaligned(q) || misaligned(cache) || misaligned(block_table, 3) ||
      misaligned(seq_lens, 3) || misaligned(draft_mask, 7) || misaligned(out) ||
      misaligned(lse, 3) || misaligned(status, 3))
    return KDA_ERR_INVALID_ARG;
  if (q == nullptr || seq_lens == nullptr || out == nullptr ||
      (block_table == nullptr && s.table_pages > 0) ||
      (cache == nullptr && cache_shape->n_pages > 0))
    return KDA_ERR_INVALID_ARG;
  if (s.table_pages > (kMaxTokens - 256) / cache_shape->page_size) return KDA_ERR_UNSUPPORTED;
  if (workspace == nullptr || misaligned(workspace, 255) ||
      workspace_bytes < kda_latent_decode_workspace_size(shape, cache_shape))
    return KDA_ERR_INVALID_ARG;
  DecodeLatentArgs a{};
  a.c = cache_args(cache, *cache_shape);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.table = block_table;
  a.lens = seq_lens;
  a.mask = draft_mask;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.table_pages = s.table_pages;
  a.N = s.N; a.L = s.L; a.H = s.H;
  a.scale = s.scale > 0.f ? s.scale : 1.0f / sqrtf(static_cast<float>(DN + DP));
  a.ws = static_cast<unsigned char*>(workspace);
  a.status = status;
  return of(launch_latent_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_latent_status(kda_stream_t stream, int32_t* device_code) {
  static std::mutex one_at_a_time;
  std::lock_guard<std::mutex> lock(one_at_a_time);
  int32_t code = kda::kDevOk;
  for (auto take : {take_fwd_status, take_bwd_status, take_decode_status, take_cache_status}) {
    int32_t c = kda::kDevOk;
    if (take(reinterpret_cast<cudaStream_t>(stream), &c) != cudaSuccess) return KDA_ERR_CUDA;
    if (c != kda::kDevOk) code = c;
  }
  if (device_code != nullptr) *device_code = code;
  return code == kda::kDevOk ? KDA_OK : KDA_ERR_DEVICE;
}

}  // extern "C"
