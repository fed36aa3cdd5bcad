// kda_latent_fwd.cu -- expanded latent attention, forward.
//
//   s_ij = scale q_i . [k_nope_j | k_pe_j] (192),  p = softmax_j(s),  out_i = sum_j p_ij v_j (128)
//
// Bound by the tensor cores: 2 x 320 operations a (query, key, head) pair, against one
// exponential. A CTA takes 256 queries of one head as two tiles of 128 and walks the keys 128
// at a time; the two tiles alternate, so that one's products run while the other's softmax
// does. Tensor memory (all 512 columns) holds S and O of both tiles; P replaces its S in
// place, as bf16, and is read from there by the second product. K tiles are never formed: the
// shared k_pe is the third 64-channel column group of every head's keys.
//
// The softmax runs a query a thread, on a reference that follows the running maximum lazily:
// it is raised only when a score passes it by 16 in log2 units (p stays below 2^16; bf16 and
// the fp32 sums keep their relative precision there), and only then is O rescaled. So the
// exponentials need not wait for a tile's maximum. P goes over in two halves, the second
// product starting on the first.
//
// Shared memory: the two query tiles (96 KB) and a ring of eight 16 KB column groups
// [128 keys, 64 channels], five a key tile (k_nope 2, k_pe, v 2).
#include "kda_latent_tc.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int BM = 128, BN = 128;
constexpr uint32_t kAtom = BN * 128;     // a column group: 128 rows of 64 bf16
constexpr int kRing = 8, kPerTile = 5;   // column groups in the ring, of a key tile
constexpr float kRaise = 16.f;           // log2 units a score may pass its row's reference

struct Sm {
  static constexpr uint32_t Q = 0, RING = 6 * kAtom, BAR = RING + kRing * kAtom, TM = BAR + 256,
                            BAIL = TM + 4, BYTES = BAIL + 12;
};
static_assert(Sm::BYTES <= 232448, "shared memory");

struct Maps {
  CUtensorMap q, kn, kp, v;
};

__global__ void __launch_bounds__(384, 1)
    fwd_kernel(const __grid_constant__ Maps maps, const AttnArgs a, int q_blocks) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Sm::BAR);
  uint64_t *full = bar, *empty = bar + 8, *q_full = bar + 16, *s_full = bar + 18,
           *p_full = bar + 20, *o_full = bar + 22, *drain = bar + 24, *v_last = bar + 25, *v_fixed = bar + 26, *p_half = bar + 27;
  uint32_t* tmem = reinterpret_cast<uint32_t*>(sm + Sm::TM);
  volatile int* bail = reinterpret_cast<volatile int*>(sm + Sm::BAIL);
  const uint32_t sb = smem_u32(sm);

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(q_full + g, 1);
      mbar_init(s_full + g, 1);
      mbar_init(p_half + g, 128);
      mbar_init(p_full + g, 128);
      mbar_init(o_full + g, 1);
    }
    mbar_init(drain, 1);
    mbar_init(v_last, 1);
    mbar_init(v_fixed, 32);
    fence_mbar_init();
    *bail = 0;
  }
  if (warp == 2 && lane < 4)
    tma_prefetch_desc(lane == 0 ? &maps.q : lane == 1 ? &maps.kn : lane == 2 ? &maps.kp : &maps.v);
  griddep_launch_dependents();
  griddep_wait();  // so far nothing was read that a kernel before this one may have written

  int h, qb;  // of a head's blocks those with the most keys to see come first
  place_of(blockIdx.x, a.H, q_blocks, 8, h, qb);
  qb = q_blocks - 1 - qb;
  SeqRange r;
  if (!seq_range(a, blockIdx.y, r)) return;
  const int i0 = qb * 2 * BM;
  if (i0 >= r.lq) return;
  if (sb & 1023) {
    if (tid == 0) report(a.status, kDevWaitTimeout);
    return;
  }
  const int lag = r.lk - r.lq;  // causal: query i sees keys j <= i + lag
  // key tiles each query tile needs
  int nk[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int last = min(r.lq, i0 + (g + 1) * BM);  // one past the tile's last query
    const int end = i0 + g * BM >= r.lq ? 0 : a.causal ? max(0, last + lag) : r.lk;
    nk[g] = (min(end, r.lk) + BN - 1) / BN;
  }
  const int n = max(nk[0], nk[1]);

  // column group c of the keys (kPerTile a tile) into its place in the ring
  auto load_group = [&](int c) {
    const int j = c / kPerTile, i = c % kPerTile, s = c % kRing;
    const int row = static_cast<int>(r.k0) + j * BN;
    unsigned char* dst = sm + Sm::RING + s * kAtom;
    mbar_arrive_expect_tx(full + s, kAtom);
    if (i < 2) tma_load_3d(dst, &maps.kn, full + s, 64 * i, h, row);
    else if (i == 2) tma_load_2d(dst, &maps.kp, full + s, 0, row);
    else tma_load_3d(dst, &maps.v, full + s, 64 * (i - 3), h, row);
  };
  const int first = min(kRing, kPerTile * n);  // groups the ring holds without waiting
  if (tid == 0) {
    for (int g = 0; g < 2; ++g) {  // on their way while the CTA sets up
      if (nk[g] > 0) {
        mbar_arrive_expect_tx(q_full + g, 3 * kAtom);
        for (int i = 0; i < 3; ++i)
          tma_load_3d(sm + Sm::Q + (3 * g + i) * kAtom, &maps.q, q_full + g, 64 * i, h,
                      static_cast<int>(r.q0) + i0 + g * BM);
      }
      for (int c = 3 * g; c < (g ? first : min(first, 3)); ++c) load_group(c);  // keys, then the rest
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = *tmem;

  if (warp < 4) {
    reg_dec<72>();
    if (warp == 0) {
      // ---------------------------------------------------------------- loads
      if (elect_one()) {
        int c = first;
        for (; c < kPerTile * n; ++c) {
          wait_for(empty + c % kRing, (c / kRing - 1) & 1, bail);
          if (*bail) break;
          load_group(c);
        }
        for (int g = 0; g < 2; ++g)
          if (nk[g] > 0) mbar_wait(q_full + g, 0, kDrainCycles);
        for (int k = c > kRing ? c - kRing : 0; k < c; ++k)
          mbar_wait(full + k % kRing, k / kRing & 1, kDrainCycles);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------- products
      constexpr uint32_t iq = idesc_bf16(BM, BN, 0, 0), iv = idesc_bf16(BM, 128, 0, 1),
                         ih = idesc_bf16(BM, 64, 0, 1);
      const uint64_t q0 = sdesc_sw128(sb + Sm::Q, 16, 1024);
      auto ring = [&](int c) { return sb + Sm::RING + c % kRing * kAtom; };
      auto wait_group = [&](int c) { wait_for(full + c % kRing, c / kRing & 1, bail); };
      auto qk = [&](int g, int j, bool release) {
        if (j == 0) wait_for(q_full + g, 0, bail);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const int c = kPerTile * j + i;
          wait_group(c);
          tc_fence_after();
          const uint64_t qa = q0 + (3 * g + i) * (kAtom / 16), kb = sdesc_sw128(ring(c), 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(tb + g * BN, qa + 2 * k, kb + 2 * k, iq, i > 0 || k > 0);
          if (release) umma_commit(empty + c % kRing);
        }
        umma_commit(s_full + g);
      };
      auto pv = [&](int g, int j, bool release) {
        const int c = kPerTile * j + 3;
        wait_group(c);
        wait_group(c + 1);
        if (r.lk - j * BN < BN) {
          if (g == 0 || j >= nk[0]) mbar_arrive(v_last);
          wait_for(v_fixed, 0, bail);
        }
        const uint32_t o = tb + 256 + g * 128, p = tb + g * BN;
        const bool split = c % kRing == kRing - 1;  // the ring's end between v's column groups
        const uint64_t v0 = sdesc_sw128(ring(c), kAtom, 1024), v1 = sdesc_sw128(ring(c + 1), kAtom, 1024);
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // of the keys: P arrives in two parts
          wait_for((half ? p_full : p_half) + g, j & 1, bail);
          tc_fence_after();
          if (!split) {
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k)
              umma_bf16_tmem_a(o, p + 8 * k, v0 + 128 * k, iv, j > 0 || k > 0);
          } else {
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k) {
              umma_bf16_tmem_a(o, p + 8 * k, v0 + 128 * k, ih, j > 0 || k > 0);
              umma_bf16_tmem_a(o + 64, p + 8 * k, v1 + 128 * k, ih, j > 0 || k > 0);
            }
          }
        }
        if (release) {
          umma_commit(empty + c % kRing);
          umma_commit(empty + (c + 1) % kRing);
        }
        if (j + 1 == nk[g]) umma_commit(o_full + g);
      };
      if (elect_one()) {
        if (nk[0] > 0) qk(0, 0, nk[1] == 0);
        if (nk[1] > 0) qk(1, 0, true);
        for (int j = 0; j < n; ++j) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (j < nk[g]) pv(g, j, g == 1 || j >= nk[1]);
            if (j + 1 < nk[g]) qk(g, j + 1, g == 1 || j + 1 >= nk[1]);
          }
        }
        umma_commit(drain);
        mbar_wait(drain, 0, kDrainCycles);
      }
    } else if (warp == 2 && n > 0 && r.lk - (n - 1) * BN < BN) {
      // v's rows past the sequence may hold anything (0 x NaN is NaN): cleared
      const int c = kPerTile * (n - 1) + 3, valid = r.lk - (n - 1) * BN;
      wait_for(v_last, 0, bail);
      for (int e = lane; e < (BN - valid) * 16; e += 32)
        *reinterpret_cast<uint4*>(sm + Sm::RING + (c + (e >> 3 & 1)) % kRing * kAtom +
                                  sw128_chunk(valid + (e >> 4), e & 7, 0)) = make_uint4(0, 0, 0, 0);
      fence_async_smem();
      mbar_arrive(v_fixed);
    }
  } else {
    // -------------------------------------------------------- softmax, results
    reg_inc<216>();
    const int g = (warp - 4) / 4, w = warp % 4;
    const uint32_t lanes = tb + (static_cast<uint32_t>(w * 32) << 16);
    const uint32_t sc = lanes + g * BN, oc = lanes + 256 + g * 128;
    const int i = i0 + g * BM + w * 32 + lane;  // this thread's query
    const int kend = a.causal ? min(r.lk, max(0, i + 1 + lag)) : r.lk;
    const float sl = a.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl);
    float nm = INFINITY;  // minus the row's reference in log2 units; +inf before its first score
    float2 l2 = make_float2(0.f, 0.f);
    const int nt = nk[g];
    for (int j = 0; j < nt; ++j) {
      wait_for(s_full + g, j & 1, bail);
      tc_fence_after();
      uint32_t v[4][32];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(sc + 32 * q, v[q]);
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld_wait(v[q]);
      const int lim = kend - j * BN;  // keys of this tile the query sees
      if (__any_sync(0xffffffffu, lim < BN)) {
#pragma unroll
        for (int k = 0; k < BN; ++k)
          if (k >= lim) v[k / 32][k % 32] = 0xff800000u;
      }
      // y = log2 of p. The first half's exponentials are taken against the reference as it is
      // while the second half's maximum is found; both are looked at before P replaces S.
      float2 nm2 = make_float2(nm, nm);
      uint32_t p[32];
      float top = -INFINITY;
      float2 part = make_float2(0.f, 0.f);
      auto first_half = [&] {
        top = -INFINITY;
        part = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float2 y = fma2(make_float2(__uint_as_float(v[k / 16][2 * k % 32]),
                                            __uint_as_float(v[k / 16][2 * k % 32 + 1])), sl2, nm2);
          top = fmaxf(top, fmaxf(y.x, y.y));
          const float2 e = make_float2(ex2(y.x), ex2(y.y));
          part = add2(part, e);
          p[k] = pack2(e.x, e.y);
        }
      };
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        mx = fmaxf(mx, fmaxf(__uint_as_float(v[2][k]), __uint_as_float(v[3][k])));
      first_half();
      const bool up = fmaxf(top, fmaf(mx, sl, nm)) > kRaise;
      if (__any_sync(0xffffffffu, up || nm == INFINITY)) {
        // the running maximum becomes the reference of the rows that need it; O and the sum
        // are rescaled (S of this step comes after O of the last: O is at rest)
        tmem_ld32(sc, v[0]);
        tmem_ld32(sc + 32, v[1]);
        tmem_ld_wait(v[0]);
        tmem_ld_wait(v[1]);
#pragma unroll
        for (int k = 0; k < 64; ++k) {
          if (k >= lim) v[k / 32][k % 32] = 0xff800000u;
          mx = fmaxf(mx, __uint_as_float(v[k / 32][k % 32]));
        }
        const float n2 = up ? -sl * mx : nm;
        const float f = nm == INFINITY ? (up ? 0.f : 1.f) : ex2(n2 - nm);
        nm = n2;
        l2.x *= f;
        l2.y *= f;
        if (j > 0) {
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            uint32_t o[16];
            tmem_ld16(oc + 16 * q, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st16(oc + 16 * q, o);
          }
        }
        const float used = nm == INFINITY ? 0.f : nm;  // no score yet: masked (p = 0) or NaN
        nm2 = make_float2(used, used);
        first_half();
      }
      l2 = add2(l2, part);
      tmem_st32(sc, p);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_half + g);
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float2 y = fma2(make_float2(__uint_as_float(v[2 + k / 16][2 * k % 32]),
                                          __uint_as_float(v[2 + k / 16][2 * k % 32 + 1])), sl2, nm2);
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        l2 = add2(l2, e);
        p[k] = pack2(e.x, e.y);
      }
      tmem_st32(sc + 32, p);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_full + g);
    }
    const float l = l2.x + l2.y;
    if (nt > 0) wait_for_results(o_full + g, 0, bail);
    tc_fence_after();
    const float mul = l == 0.f ? 0.f : 1.f / l;
    const bool mine = i < r.lq;
    const int64_t row = (r.q0 + i) * a.H + h;
    if (mine && a.lse != nullptr)
      a.lse[row] = l == 0.f ? -INFINITY : (log2f(l) - nm) * kLn2;
    // through shared memory (the tile's queries are not needed any more): whole lines go out
    unsigned char* tile = sm + Sm::Q + 3 * g * kAtom;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      uint32_t o[32];
      if (nt > 0) {
        tmem_ld32(oc + 32 * q, o);
        tmem_ld_wait(o);
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = pack2(__uint_as_float(o[8 * k + 2 * e]) * mul,
                       __uint_as_float(o[8 * k + 2 * e + 1]) * mul);
        *reinterpret_cast<uint4*>(tile + sw128_chunk(w * 32 + lane, 4 * q + k, kAtom)) =
            make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
    __syncwarp();
    const int first = i0 + g * BM + w * 32;  // this warp's rows
    copy_rows<2>(tile, reinterpret_cast<unsigned char*>(a.out + ((r.q0 + first) * a.H + h) * DV),
                 static_cast<int64_t>(a.H) * DV * 2, w * 32, min(32, r.lq - first), 0, 1, lane);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *bail) report(a.status, kDevWaitTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

}  // namespace

cudaError_t launch_attn_fwd(const AttnArgs& a, cudaStream_t st) {
  // (first: it makes the device's context current in a thread that has none yet, as autograd's,
  // which the encoding of maps needs)
  cudaError_t e = cudaFuncSetAttribute(fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Sm::BYTES);
  if (e != cudaSuccess) return e;
  const int64_t tq = a.cu_q != nullptr ? a.Tq : a.Tq * a.n_seqs;
  const int64_t tk = a.cu_k != nullptr ? a.Tk : a.Tk * a.n_seqs;
  Maps m;
  memset(&m, 0, sizeof m);
  if (!make_head_map(&m.q, a.q, DQK, a.H, a.qh, tq, a.qt, BM) ||
      !make_head_map(&m.kn, a.kn, DN, a.H, a.kh, tk, a.kt, BN) ||
      !make_head_map(&m.v, a.v, DV, a.H, a.vh, tk, a.vt, BN))
    return cudaErrorInvalidValue;
  if (tk > 0) {
    const uint64_t dims[2] = {DP, static_cast<uint64_t>(tk)};
    const uint64_t strides[1] = {static_cast<uint64_t>(a.pt) * 2};
    const uint32_t box[2] = {64, BN};
    if (!make_tensor_map(&m.kp, a.kp, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const int64_t blocks = (a.max_q + 2 * BM - 1) / (2 * BM);
  if (blocks * a.H > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_early(fwd_kernel, dim3(static_cast<unsigned>(blocks * a.H), a.n_seqs), 384, Sm::BYTES,
                      st, m, a, static_cast<int>(blocks));
}

cudaError_t take_fwd_status(cudaStream_t st, int32_t* code) { return take_status(st, code); }

}  // namespace latent
}  // namespace kda
