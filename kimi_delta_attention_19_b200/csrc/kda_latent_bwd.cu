// kda_latent_bwd.cu -- expanded latent attention, backward.
//
//   p_ij = exp(s_ij - lse_i)   dP = dO V^T   D_i = dO_i . out_i   dS = p (dP - D)
//   dQ = scale dS K            dK = scale dS^T Q (k_pe: summed over heads)   dV = P^T dO
//
// Bound by the tensor cores. Scores and dP are formed twice, once a query tile (dQ) and once
// a key tile (dK, dV): 2 x 1280 operations a pair instead of 2 x 960 with dQ accumulated across
// key tiles, but every sum then stays in one CTA's tensor memory (192 columns of dQ, or
// 128 + 192 of dV and dK), without atomics, so the same inputs give the same bits. Both kinds
// of CTA are one launch, so that one kind fills the other's tail.
//
//   prepare   (lse log2 e, D) a (head, token), one array: the statistics of both kinds
//   dQ CTA    128 queries, keys 64 at a time: S, dP [q, keys]; dS as bf16 in tensor memory,
//             the A operand of dQ += dS K. Q and dO are A operands from there too, which
//             leaves shared memory to the keys: with two stages of 128 keys and Q, dO beside
//             them the CTA waited for keys half of its time (4300 clocks per 128 keys)
//   dK CTA    128 keys, queries 64 at a time (what tensor memory leaves): S^T, dP^T [keys, q];
//             P^T and dS^T the A operands of dV += P^T dO and dK += dS^T Q
//   k_pe      the heads' fp32 parts of dk_pe, summed in the heads' order
//
// dS enters its products as bf16, which brings its products the same error again as rounding the
// result does (1.66e-3 of the norm; together 2.35e-3, and what the rounding of out does through D on
// top). Tiles none of whose queries sees more than kFew keys add what dS lost, as a second bf16
// term: for dQ a tile of 128 queries, for dK a step of 64, so one query's term may be kept in one
// of the two and not in the other. Rows of few keys carry most of a gradient's squares, so of a
// sequence's first rows this pays the most. Relative errors of dq and dk_nope against 64 bits, in
// 1e-3 (causal, 4 heads; lq | lk: queries behind a prefix), and the time of a packed training step
// of 6 documents of 156 to 1432 tokens:
//   kFew                  32           128          256          384          512
//   4 of 245 tokens       2.48 2.45    2.03 2.01    1.81 1.79    1.81 1.79    1.81 1.79
//   3 of 425              2.42 2.40    2.09 2.07    1.94 1.92    1.81 1.80    1.78 1.76
//   1000                  2.41 2.36    2.17 2.14    2.06 2.03    1.99 1.96    1.92 1.89
//   4 of 64 | 320         2.49 2.45    2.49 2.45    2.49 2.45    1.76 1.74    1.76 1.74
//   125 | 425             2.38 2.36    2.38 2.36    2.38 2.36    2.38 2.03    1.74 1.71
//   300 | 600             2.42 2.38    2.42 2.38    2.42 2.38    2.42 2.23    2.12 1.93
//   packed step           264 us       264          269          270          275
// With 384, sequences of up to 2100 tokens that see themselves are below 2.1e-3 for 2.5 % of a packed
// step; behind a longer prefix (and without causality from 385 keys on) the single term's 2.4e-3 to
// 2.5e-3 stay.
//
// In both, S of the next step is issued as soon as this step's is in registers, dP likewise,
// so the products run beside the exponentials.
#include <algorithm>

#include "kda_latent_tc.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int BM = 128;                    // queries of a dQ CTA, keys of a dK CTA
constexpr int BQ = 64;                     // query step of a dK CTA, key step of a dQ CTA
constexpr uint32_t kAtom = BM * 128, kAtomQ = BQ * 128;
constexpr int kFew = 384;                  // most keys of a tile whose dS is kept in two terms
constexpr int kQStages = 3, kKStages = 4, kVStages = 3;
constexpr int kThreads = 384, kSoft = 256;

struct SmQ {  // dQ CTA
  static constexpr uint32_t Q = 0, DO = 3 * kAtom, K = 5 * kAtom, V = K + kKStages * 3 * kAtomQ,
                            END = V + kVStages * 2 * kAtomQ;
};
struct SmK {  // dK CTA
  static constexpr uint32_t K = 0, V = 3 * kAtom, ST = 5 * kAtom, STAGE = 5 * kAtomQ,
                            STAT = ST + kQStages * STAGE, END = STAT + 2 * BQ * 8;
};
constexpr uint32_t kBar = SmQ::END > SmK::END ? SmQ::END : SmK::END;
constexpr uint32_t kTm = kBar + 256, kBail = kTm + 4, kBytes = kBail + 12;
static_assert(kBytes <= 232448, "shared memory");

struct Maps {
  CUtensorMap q, qs, dout, douts, kn, kns, kp, kps, v, vs;  // s: boxes of BQ rows
};

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    s += __uint_as_float(u[e] << 16) * __uint_as_float(v[e] << 16) +
         __uint_as_float(u[e] & 0xffff0000u) * __uint_as_float(v[e] & 0xffff0000u);
  return s;
}

// (lse log2 e, D) of 32 tokens of a head a block; a row without keys gets +inf (p = 0) and 0 (its
// dO may hold anything). Half a warp a row (16 bytes a lane of dO and of out), all of a warp's
// loads at once.
__global__ void __launch_bounds__(256) prepare_kernel(AttnArgs a, int64_t tq) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, h = blockIdx.y;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 32;
  __shared__ float2 st[32];
  uint4 x[2], y[2];
  float l[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t t = t0 + warp * 4 + 2 * k + lane / 16, row = (t < tq ? t : tq - 1) * a.H + h;
    x[k] = ld16(a.dout + row * DV + 8 * (lane % 16));
    y[k] = ld16(a.o + row * DV + 8 * (lane % 16));
    l[k] = a.lse_in[row];
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float s = dot8(x[k], y[k]);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane % 16 == 0)
      st[warp * 4 + 2 * k + lane / 16] =
          l[k] == -INFINITY ? make_float2(INFINITY, 0.f) : make_float2(l[k] * kLog2e, s);
  }
  __syncthreads();
  if (threadIdx.x < 32 && t0 + threadIdx.x < tq)
    a.stat[h * tq + t0 + threadIdx.x] = st[threadIdx.x];
}

// D of the queries that see at most 32 keys, a warp a query: sum_j p_j (dO . v_j).
// The rounding of out, from which other rows' D comes, is a large part of the little that their
// dS holds (dq of sequences of 1 to 3 tokens was off by 5.5e-3, and is by 1.7e-3). In a launch of
// its own: found by prepare_kernel's warps these rows cost 40 us of a packed step, here 9 (a lane a key: 15).
__global__ void __launch_bounds__(256) few_kernel(AttnArgs a, int64_t tq) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, h = blockIdx.z;
  SeqRange r;
  if (!seq_range(a, blockIdx.y, r)) return;
  const int lag = r.lk - r.lq;  // causal: query i sees i + 1 + lag keys
  const int first = a.causal ? max(0, -lag) : 0;
  const int last = a.causal ? static_cast<int>(min(static_cast<int64_t>(r.lq), int64_t{32} - lag)) : r.lk <= 32 ? r.lq : 0;
  for (int64_t i = first + static_cast<int64_t>(blockIdx.x) * 8 + warp; i < last; i += 8 * gridDim.x) {
    const int see = a.causal ? static_cast<int>(i) + 1 + lag : r.lk;
    const int64_t t = r.q0 + i;
    float2* st = a.stat + h * tq + t;
    const int c = 8 * (lane % 8);  // eight lanes a key: whole lines
    const __nv_bfloat16 *q = a.q + t * a.qt + h * a.qh + c, *g = a.dout + (t * a.H + h) * DV + c;
    const uint4 q0 = ld16(q), q1 = ld16(q + 64), q2 = ld16(q + DN), g0 = ld16(g), g1 = ld16(g + 64);
    const float lse2 = st->x;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      float s = 0.f, dp = 0.f;
      if (k + lane / 8 < see) {
        const int64_t j = r.k0 + k + lane / 8;
        const __nv_bfloat16 *kn = a.kn + j * a.kt + h * a.kh + c, *v = a.v + j * a.vt + h * a.vh + c;
        s = dot8(q0, ld16(kn)) + dot8(q1, ld16(kn + 64)) + dot8(q2, ld16(a.kp + j * a.pt + c));
        dp = dot8(g0, ld16(v)) + dot8(g1, ld16(v + 64));
      }
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, off);
        dp += __shfl_xor_sync(0xffffffffu, dp, off);
      }
      if (k + lane / 8 < see) sum += dp * ex2(fmaf(s, a.scale * kLog2e, -lse2));
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (lane == 0) st->y = sum;
  }
}

// what the bf16 pair `hi` of (x, y) lost, as another pair
__device__ __forceinline__ uint32_t lost2(float x, float y, uint32_t hi) {
  return pack2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

__device__ __forceinline__ void zero_rows(unsigned char* tile, uint32_t atom, int atoms, int from,
                                          int rows, int lane) {
  const int per = atoms * 8;
  for (int e = lane; e < (rows - from) * per; e += 32)
    *reinterpret_cast<uint4*>(tile + sw128_chunk(from + e / per, e % per, atom)) =
        make_uint4(0, 0, 0, 0);
}

__global__ void __launch_bounds__(kThreads, 1)
    bwd_kernel(const __grid_constant__ Maps maps, const AttnArgs a, int64_t tq_all, int64_t tk_all,
               int k_blocks, int q_blocks) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + kBar);
  uint64_t *full = bar, *empty = bar + 4, *v_full = bar + 8, *v_empty = bar + 11,
           *res_full = bar + 14, *s_full = bar + 15, *dp_full = bar + 16, *s_read = bar + 17,
           *p_ready = bar + 18, *ds_ready = bar + 19, *p_free = bar + 20, *ds_free = bar + 21,
           *o_full = bar + 22, *drain = bar + 23, *last = bar + 24, *fixed = bar + 25,
           *a_ready = bar + 26, *first = bar + 27, *first_fixed = bar + 28;
  uint32_t* tmem = reinterpret_cast<uint32_t*>(sm + kTm);
  volatile int* bail = reinterpret_cast<volatile int*>(sm + kBail);
  const uint32_t sb = smem_u32(sm);

  // Key blocks first, those with the most queries ahead; then query blocks, likewise (the two
  // kinds in turn took 8 % longer). Groups of 16 heads: the 4K step 797 us, 815 with all 32.
  const int all_k = k_blocks * a.H;
  const bool is_k = blockIdx.x < all_k;
  int h, blk;
  if (is_k) place_of(blockIdx.x, a.H, k_blocks, 16, h, blk);
  else place_of(blockIdx.x - all_k, a.H, q_blocks, 16, h, blk);
  SeqRange r;
  if (!seq_range(a, blockIdx.y, r)) return;
  const int lag = r.lk - r.lq;  // causal: query i sees keys j <= i + lag
  const int b0 = (is_k ? blk : q_blocks - 1 - blk) * BM;  // first key or query
  if (b0 >= (is_k ? r.lk : r.lq)) return;
  if (sb & 1023) {
    if (tid == 0) report(a.status, kDevWaitTimeout);
    return;
  }
  // steps [j0, j1) of queries (dK CTA) or keys (dQ CTA)
  int j0 = 0, j1;
  if (is_k) {
    if (a.causal) j0 = max(0, b0 - lag) / BQ;
    j1 = max(j0, (r.lq + BQ - 1) / BQ);
  } else {
    const int last = min(r.lq, b0 + BM);
    j1 = (min(r.lk, a.causal ? max(0, last + lag) : r.lk) + BQ - 1) / BQ;
  }
  const int n = j1 - j0;

  if (warp == 2 && n > 0) {
    if (is_k && lane < 5)
      tma_prefetch_desc(lane == 0 ? &maps.kn : lane == 1 ? &maps.kp : lane == 2 ? &maps.v
                        : lane == 3 ? &maps.qs : &maps.douts);
    if (!is_k && lane < 5)
      tma_prefetch_desc(lane == 0 ? &maps.q : lane == 1 ? &maps.dout : lane == 2 ? &maps.kns
                        : lane == 3 ? &maps.kps : &maps.vs);
  }
  // step t's rows into their stage
  auto load_queries = [&](int t) {
    const int s = t % kQStages, row = static_cast<int>(r.q0) + (j0 + t) * BQ;
    unsigned char* st = sm + SmK::ST + s * SmK::STAGE;
    mbar_arrive_expect_tx(full + s, SmK::STAGE);
    for (int i = 0; i < 3; ++i) tma_load_3d(st + i * kAtomQ, &maps.qs, full + s, 64 * i, h, row);
    for (int i = 0; i < 2; ++i) tma_load_3d(st + (3 + i) * kAtomQ, &maps.douts, full + s, 64 * i, h, row);
  };
  auto load_keys = [&](int t) {
    const int s = t % kKStages, row = static_cast<int>(r.k0) + t * BQ;
    unsigned char* st = sm + SmQ::K + s * 3 * kAtomQ;
    mbar_arrive_expect_tx(full + s, 3 * kAtomQ);
    for (int i = 0; i < 2; ++i) tma_load_3d(st + i * kAtomQ, &maps.kns, full + s, 64 * i, h, row);
    tma_load_2d(st + 2 * kAtomQ, &maps.kps, full + s, 0, row);
  };
  auto load_values = [&](int t) {
    const int s = t % kVStages, row = static_cast<int>(r.k0) + t * BQ;
    mbar_arrive_expect_tx(v_full + s, 2 * kAtomQ);
    for (int i = 0; i < 2; ++i)
      tma_load_3d(sm + SmQ::V + (2 * s + i) * kAtomQ, &maps.vs, v_full + s, 64 * i, h, row);
  };
  if (tid == 0) {
    for (int i = 0; i < 14; ++i) mbar_init(bar + i, 1);  // stages, full and empty
    mbar_init(res_full, 1);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(s_read, kSoft);
    mbar_init(p_ready, kSoft);
    mbar_init(ds_ready, kSoft);
    mbar_init(p_free, 1);
    mbar_init(ds_free, 1);
    mbar_init(o_full, 1);
    mbar_init(a_ready, kSoft);
    mbar_init(drain, 1);
    mbar_init(last, 1);
    mbar_init(fixed, 32);
    mbar_init(first, 1);
    mbar_init(first_fixed, 32);
    fence_mbar_init();
    *bail = 0;
    if (n > 0) {  // the CTA's own rows and the first step's, on their way while it sets up
      mbar_arrive_expect_tx(res_full, 5 * kAtom);
      if (is_k) {
        const int row = static_cast<int>(r.k0) + b0;
        for (int i = 0; i < 2; ++i) tma_load_3d(sm + SmK::K + i * kAtom, &maps.kn, res_full, 64 * i, h, row);
        tma_load_2d(sm + SmK::K + 2 * kAtom, &maps.kp, res_full, 0, row);
        for (int i = 0; i < 2; ++i) tma_load_3d(sm + SmK::V + i * kAtom, &maps.v, res_full, 64 * i, h, row);
        load_queries(0);
      } else {
        const int row = static_cast<int>(r.q0) + b0;
        for (int i = 0; i < 3; ++i) tma_load_3d(sm + SmQ::Q + i * kAtom, &maps.q, res_full, 64 * i, h, row);
        for (int i = 0; i < 2; ++i) tma_load_3d(sm + SmQ::DO + i * kAtom, &maps.dout, res_full, 64 * i, h, row);
        load_keys(0);
        load_values(0);
      }
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
  const float sl = a.scale * kLog2e;
  const float2 sl2 = make_float2(sl, sl);

  if (is_k) {
    // =================================================================== dK, dV
    constexpr uint32_t S = 0, DP = 64, P = 128, DS = 160, DVC = 192, DK = 320;  // columns
    // rows of the first step that see no key: a sequence's first queries, when it has more than keys
    const int blind = a.causal ? max(0, -lag) - j0 * BQ : 0;
    auto sees_few = [&](int t) {
      return (a.causal ? min(r.lk, (j0 + t + 1) * BQ + lag) : r.lk) <= kFew;
    };
    if (warp == 0) {
      if (n > 0 && elect_one()) {
        int t = 1;
        for (; t < n; ++t) {
          if (t >= kQStages) wait_for(empty + t % kQStages, (t / kQStages - 1) & 1, bail);
          if (*bail) break;
          load_queries(t);
        }
        mbar_wait(res_full, 0, kDrainCycles);
        for (int k = t > kQStages ? t - kQStages : 0; k < t; ++k)
          mbar_wait(full + k % kQStages, k / kQStages & 1, kDrainCycles);
      }
    } else if (warp == 1 && n > 0) {
      constexpr uint32_t i64 = idesc_bf16(BM, BQ, 0, 0), iv = idesc_bf16(BM, 128, 0, 1),
                         ik = idesc_bf16(BM, 192, 0, 1);
      auto stage = [&](int t) { return sb + SmK::ST + t % kQStages * SmK::STAGE; };
      const uint64_t k0 = sdesc_sw128(sb + SmK::K, 16, 1024), v0 = sdesc_sw128(sb + SmK::V, 16, 1024);
      auto scores = [&](int t) {  // S^T = K Q^T
        wait_for(full + t % kQStages, t / kQStages & 1, bail);
        if (t == 0 && blind > 0) {
          mbar_arrive(first);
          wait_for(first_fixed, 0, bail);
        }
        if (r.lq - (j0 + t) * BQ < BQ) {
          mbar_arrive(last);
          wait_for(fixed, 0, bail);
        }
        tc_fence_after();
        const uint64_t qb = sdesc_sw128(stage(t), 16, 1024);
#pragma unroll
        for (int k = 0; k < 12; ++k)
          umma_bf16(tb + S, k0 + k / 4 * (kAtom / 16) + k % 4 * 2,
                    qb + k / 4 * (kAtomQ / 16) + k % 4 * 2, i64, k > 0);
        umma_commit(s_full);
      };
      auto dprobs = [&](int t) {  // dP^T = V dO^T
        const uint64_t gb = sdesc_sw128(stage(t) + 3 * kAtomQ, 16, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_bf16(tb + DP, v0 + k / 4 * (kAtom / 16) + k % 4 * 2,
                    gb + k / 4 * (kAtomQ / 16) + k % 4 * 2, i64, k > 0);
        umma_commit(dp_full);
      };
      if (elect_one()) {
        wait_for(res_full, 0, bail);
        scores(0);
        dprobs(0);
        for (int t = 0; t < n; ++t) {
          wait_for(s_read, t & 1, bail);
          if (t + 1 < n) scores(t + 1);
          wait_for(p_ready, t & 1, bail);
          tc_fence_after();
          const uint64_t gb = sdesc_sw128(stage(t) + 3 * kAtomQ, kAtomQ, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16_tmem_a(tb + DVC, tb + P + 8 * k, gb + 128 * k, iv, t > 0 || k > 0);
          umma_commit(p_free);
          wait_for(ds_ready, t & 1, bail);
          tc_fence_after();
          const bool few = sees_few(t);
          if (!few && t + 1 < n) dprobs(t + 1);
          const uint64_t qb = sdesc_sw128(stage(t), kAtomQ, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16_tmem_a(tb + DK, tb + DS + 8 * k, qb + 128 * k, ik, t > 0 || k > 0);
          if (few) {  // the second term is in dP's columns
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_tmem_a(tb + DK, tb + DP + 16 * (k & 2) + 8 * (k & 1), qb + 128 * k, ik, 1);
            if (t + 1 < n) dprobs(t + 1);
          }
          umma_commit(ds_free);
          umma_commit(empty + t % kQStages);
        }
        umma_commit(o_full);
        umma_commit(drain);
        mbar_wait(drain, 0, kDrainCycles);
      }
    } else if (warp == 2 && n > 0) {
      // queries that see no key and those past the sequence may hold anything (0 x NaN is NaN):
      // cleared
      if (blind > 0) {
        wait_for(first, 0, bail);
        zero_rows(sm + SmK::ST, kAtomQ, 5, 0, min(blind, BQ), lane);
        fence_async_smem();
        mbar_arrive(first_fixed);
      }
      if (r.lq - (j1 - 1) * BQ < BQ) {
        wait_for(last, 0, bail);
        zero_rows(sm + SmK::ST + (n - 1) % kQStages * SmK::STAGE, kAtomQ, 5, r.lq - (j1 - 1) * BQ, BQ, lane);
        fence_async_smem();
        mbar_arrive(fixed);
      }
    } else if (warp >= 4) {
      const int g = (warp - 4) / 4, w = warp % 4;
      const uint32_t lanes = tb + (static_cast<uint32_t>(w * 32) << 16);
      const int j = b0 + w * 32 + lane;  // this thread's key
      float2* stat = reinterpret_cast<float2*>(sm + SmK::STAT);
      const float2* st_g = a.stat + h * tq_all + r.q0;
      auto stat_of = [&](int t) {  // of query 32 g + lane of a step
        const int i = (j0 + t) * BQ + 32 * g + lane;
        return t < n && i < r.lq ? st_g[i] : make_float2(INFINITY, 0.f);
      };
      float2 next = w == 0 ? stat_of(0) : make_float2(0.f, 0.f);
      for (int t = 0; t < n; ++t) {
        float2* sd = stat + (t & 1) * BQ + 32 * g;
        if (w == 0) {
          sd[lane] = next;
          next = stat_of(t + 1);
        }
        group_sync(1 + g, 128);
        uint32_t v[32];
        wait_for(s_full, t & 1, bail);
        tc_fence_after();
        tmem_ld32(lanes + S + 32 * g, v);
        tmem_ld_wait(v);
        tc_fence_before();
        mbar_arrive(s_read);
        const float4* sd4 = reinterpret_cast<const float4*>(sd);
        float p[32];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float4 x = sd4[k / 2];
          p[k] = ex2(__uint_as_float(v[k]) * sl - x.x);
          p[k + 1] = ex2(__uint_as_float(v[k + 1]) * sl - x.z);
        }
        const int lim = j - lag - ((j0 + t) * BQ + 32 * g);  // queries below it do not see the key
        if (a.causal && __any_sync(0xffffffffu, lim > 0)) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (k < lim) p[k] = 0.f;
        }
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) pk[k] = pack2(p[2 * k], p[2 * k + 1]);
        if (t > 0) wait_for(p_free, (t - 1) & 1, bail);
        tmem_st16(lanes + P + 16 * g, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_ready);
        wait_for(dp_full, t & 1, bail);
        tc_fence_after();
        tmem_ld32(lanes + DP + 32 * g, v);
        tmem_ld_wait(v);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float4 x = sd4[k];
          p[2 * k] *= __uint_as_float(v[2 * k]) - x.y;
          p[2 * k + 1] *= __uint_as_float(v[2 * k + 1]) - x.w;
          pk[k] = pack2(p[2 * k], p[2 * k + 1]);
        }
        if (t > 0) wait_for(ds_free, (t - 1) & 1, bail);
        tmem_st16(lanes + DS + 16 * g, pk);
        if (sees_few(t)) {
#pragma unroll
          for (int k = 0; k < 16; ++k) pk[k] = lost2(p[2 * k], p[2 * k + 1], pk[k]);
          tmem_st16(lanes + DP + 32 * g, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_ready);
      }
      if (n > 0) wait_for_results(o_full, 0, bail);
      tc_fence_after();
      // dV: 64 columns a warpgroup; dK: 96 (the second one's last 64 are k_pe's, fp32). Through
      // shared memory, which nothing else needs any more: whole lines go out.
#pragma unroll 1
      for (int q = 0; q < 5; ++q) {
        uint32_t o[32];
        const bool is_v = q < 2;
        const int col = is_v ? 64 * g + 32 * q : 96 * g + 32 * (q - 2), rw = w * 32 + lane;
        if (n > 0) {
          tmem_ld32(lanes + (is_v ? DVC : DK) + col, o);
          tmem_ld_wait(o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        const float mul = is_v ? 1.f : a.scale;
        if (!is_v && col >= DN) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<float4*>(sm + SmK::ST + sw128_chunk(rw, (col - DN) / 4 + k, kAtom)) =
                make_float4(__uint_as_float(o[4 * k]) * mul, __uint_as_float(o[4 * k + 1]) * mul,
                            __uint_as_float(o[4 * k + 2]) * mul, __uint_as_float(o[4 * k + 3]) * mul);
          continue;
        }
        unsigned char* tile = sm + (is_v ? SmK::V : SmK::K);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = pack2(__uint_as_float(o[8 * k + 2 * e]) * mul, __uint_as_float(o[8 * k + 2 * e + 1]) * mul);
          *reinterpret_cast<uint4*>(tile + sw128_chunk(rw, col / 8 + k, kAtom)) = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      group_sync(3, kSoft);
      const int rows = min(BM, r.lk - b0);
      const int64_t tok = r.k0 + b0, at = (tok * a.H + h) * DN, step = static_cast<int64_t>(a.H) * DN * 2;
      copy_rows<2>(sm + SmK::V, reinterpret_cast<unsigned char*>(a.dv + at), step, 0, rows, warp - 4, 8, lane);
      copy_rows<2>(sm + SmK::K, reinterpret_cast<unsigned char*>(a.dkn + at), step, 0, rows, warp - 4, 8, lane);
      copy_rows<2>(sm + SmK::ST, reinterpret_cast<unsigned char*>(a.dpe_part + (h * tk_all + tok) * latent::DP),
                   latent::DP * 4, 0, rows, warp - 4, 8, lane);
    }
  } else {
    // ======================================================================= dQ
    constexpr uint32_t S = 0, DP = 64, DS = 128, QA = 160, GA = 256, DQ = 320;  // columns
    const bool few = (a.causal ? min(r.lk, b0 + BM + lag) : r.lk) <= kFew;
    if (warp == 0) {
      if (n > 0 && elect_one()) {
        int t = 1, tv = 1;
        for (; t < n; ++t) {
          if (t >= kKStages) wait_for(empty + t % kKStages, (t / kKStages - 1) & 1, bail);
          if (*bail) break;
          load_keys(t);
          if (t >= kVStages) wait_for(v_empty + t % kVStages, (t / kVStages - 1) & 1, bail);
          if (*bail) { ++t; break; }
          load_values(t);
          ++tv;
        }
        mbar_wait(res_full, 0, kDrainCycles);
        for (int k = t > kKStages ? t - kKStages : 0; k < t; ++k)
          mbar_wait(full + k % kKStages, k / kKStages & 1, kDrainCycles);
        for (int k = tv > kVStages ? tv - kVStages : 0; k < tv; ++k)
          mbar_wait(v_full + k % kVStages, k / kVStages & 1, kDrainCycles);
      }
    } else if (warp == 1 && n > 0) {
      constexpr uint32_t i64 = idesc_bf16(BM, BQ, 0, 0), iq = idesc_bf16(BM, 192, 0, 1);
      auto keys = [&](int t) { return sb + SmQ::K + t % kKStages * 3 * kAtomQ; };
      auto scores = [&](int t) {  // S = Q K^T
        wait_for(full + t % kKStages, t / kKStages & 1, bail);
        tc_fence_after();
        const uint64_t kb = sdesc_sw128(keys(t), 16, 1024);
#pragma unroll
        for (int k = 0; k < 12; ++k)
          umma_bf16_tmem_a(tb + S, tb + QA + 8 * k, kb + k / 4 * (kAtomQ / 16) + k % 4 * 2, i64, k > 0);
        umma_commit(s_full);
      };
      auto dprobs = [&](int t) {  // dP = dO V^T
        const int sv = t % kVStages;
        wait_for(v_full + sv, t / kVStages & 1, bail);
        tc_fence_after();
        const uint64_t vb = sdesc_sw128(sb + SmQ::V + 2 * sv * kAtomQ, 16, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_bf16_tmem_a(tb + DP, tb + GA + 8 * k, vb + k / 4 * (kAtomQ / 16) + k % 4 * 2, i64, k > 0);
        umma_commit(dp_full);
        umma_commit(v_empty + sv);
      };
      if (elect_one()) {
        wait_for(a_ready, 0, bail);
        scores(0);
        dprobs(0);
        for (int t = 0; t < n; ++t) {
          wait_for(s_read, t & 1, bail);
          if (t + 1 < n) scores(t + 1);
          wait_for(ds_ready, t & 1, bail);
          tc_fence_after();
          if (!few && t + 1 < n) dprobs(t + 1);
          if (r.lk - t * BQ < BQ) {
            mbar_arrive(last);
            wait_for(fixed, 0, bail);
          }
          const uint64_t kb = sdesc_sw128(keys(t), kAtomQ, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16_tmem_a(tb + DQ, tb + DS + 8 * k, kb + 128 * k, iq, t > 0 || k > 0);
          if (few) {  // the second term is in dP's columns
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_tmem_a(tb + DQ, tb + DP + 16 * (k & 2) + 8 * (k & 1), kb + 128 * k, iq, 1);
            if (t + 1 < n) dprobs(t + 1);
          }
          umma_commit(ds_free);
          umma_commit(empty + t % kKStages);
        }
        umma_commit(o_full);
        umma_commit(drain);
        mbar_wait(drain, 0, kDrainCycles);
      }
    } else if (warp == 2 && n > 0 && r.lk - (n - 1) * BQ < BQ) {
      // keys past the sequence may hold anything (0 x NaN is NaN): cleared once S is formed
      wait_for(last, 0, bail);
      zero_rows(sm + SmQ::K + (n - 1) % kKStages * 3 * kAtomQ, kAtomQ, 3, r.lk - (n - 1) * BQ, BQ, lane);
      fence_async_smem();
      mbar_arrive(fixed);
    } else if (warp >= 4) {
      const int g = (warp - 4) / 4, w = warp % 4;  // g: half of the keys of a step
      const uint32_t lanes = tb + (static_cast<uint32_t>(w * 32) << 16);
      const int i = b0 + w * 32 + lane;            // this thread's query
      const bool mine = i < r.lq;
      const float2 st = mine ? a.stat[h * tq_all + r.q0 + i] : make_float2(INFINITY, 0.f);
      const int kend = a.causal ? min(r.lk, max(0, i + 1 + lag)) : r.lk;
      const float2 nl2 = make_float2(-st.x, -st.x), nd2 = make_float2(-st.y, -st.y);
      if (n > 0) {  // Q (one warpgroup) and dO (the other) to tensor memory
        wait_for(res_full, 0, bail);
        const unsigned char* src = sm + (g ? SmQ::DO : SmQ::Q);
#pragma unroll 1
        for (int q = 0; q < (g ? 4 : 6); ++q) {  // 32 channels
          uint32_t x[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 y = *reinterpret_cast<const uint4*>(src + sw128_chunk(w * 32 + lane, 4 * q + k, kAtom));
            x[4 * k] = y.x;
            x[4 * k + 1] = y.y;
            x[4 * k + 2] = y.z;
            x[4 * k + 3] = y.w;
          }
          tmem_st16(lanes + (g ? GA : QA) + 16 * q, x);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(a_ready);
      }
      for (int t = 0; t < n; ++t) {
        wait_for(s_full, t & 1, bail);
        tc_fence_after();
        uint32_t v[32];
        tmem_ld32(lanes + S + 32 * g, v);
        tmem_ld_wait(v);
        tc_fence_before();
        mbar_arrive(s_read);
        float2 p[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 x = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sl2, nl2);
          p[k] = make_float2(ex2(x.x), ex2(x.y));
        }
        const int lim = kend - t * BQ - 32 * g;  // keys of this half the query sees
        const bool cut = __any_sync(0xffffffffu, lim < 32);
        wait_for(dp_full, t & 1, bail);
        tc_fence_after();
        tmem_ld32(lanes + DP + 32 * g, v);
        tmem_ld_wait(v);
        uint32_t ds[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          p[k] = mul2f(p[k], add2(make_float2(__uint_as_float(v[2 * k]),
                                              __uint_as_float(v[2 * k + 1])), nd2));
          ds[k] = pack2(p[k].x, p[k].y);
        }
        auto cut_off = [&] {  // keys the query does not see
          if (!cut) return;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (2 * k >= lim) ds[k] &= 0xffff0000u;
            if (2 * k + 1 >= lim) ds[k] &= 0x0000ffffu;
          }
        };
        cut_off();
        if (t > 0) wait_for(ds_free, (t - 1) & 1, bail);
        tmem_st16(lanes + DS + 16 * g, ds);
        if (few) {
#pragma unroll
          for (int k = 0; k < 16; ++k) ds[k] = lost2(p[k].x, p[k].y, ds[k]);
          cut_off();
          tmem_st16(lanes + DP + 32 * g, ds);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_ready);
      }
      if (n > 0) wait_for_results(o_full, 0, bail);
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < 6; ++q) {  // through shared memory: whole lines go out
        uint32_t o[16];
        if (n > 0) {
          tmem_ld16(lanes + DQ + 96 * g + 16 * q, o);
          tmem_ld_wait(o);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0;
        }
        uint32_t x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[k] = pack2(__uint_as_float(o[2 * k]) * a.scale, __uint_as_float(o[2 * k + 1]) * a.scale);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(sm + SmQ::Q + sw128_chunk(w * 32 + lane, 12 * g + 2 * q + k, kAtom)) =
              make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
      }
      group_sync(3, kSoft);
      copy_rows<3>(sm + SmQ::Q, reinterpret_cast<unsigned char*>(a.dq + ((r.q0 + b0) * a.H + h) * DQK),
                   static_cast<int64_t>(a.H) * DQK * 2, 0, min(BM, r.lq - b0), warp - 4, 8, lane);
    }
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

// dk_pe = the heads' parts, summed in the heads' order
__global__ void __launch_bounds__(256) dpe_kernel(AttnArgs a, int64_t tk_all) {
  SeqRange r;
  if (!seq_range(a, blockIdx.y, r)) return;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // four channels
  if (e >= static_cast<int64_t>(r.lk) * (DP / 4)) return;
  const int64_t at = r.k0 * (DP / 4) + e;
  const float4* part = reinterpret_cast<const float4*>(a.dpe_part);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int h = 0; h < a.H; ++h) {
    const float4 x = part[h * tk_all * (DP / 4) + at];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  reinterpret_cast<uint2*>(a.dkp)[at] = make_uint2(pack2(s.x, s.y), pack2(s.z, s.w));
}

int64_t blocks(int64_t n, int64_t per) { return (n + per - 1) / per; }

}  // namespace

cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t st) {
  // (first: it makes the device's context current in a thread that has none yet, as autograd's,
  // which the encoding of maps needs)
  cudaError_t e = cudaFuncSetAttribute(bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kBytes);
  if (e != cudaSuccess) return e;
  const int64_t tq = a.cu_q != nullptr ? a.Tq : a.Tq * a.n_seqs;
  const int64_t tk = a.cu_k != nullptr ? a.Tk : a.Tk * a.n_seqs;
  Maps m;
  memset(&m, 0, sizeof m);
  const int64_t ot = static_cast<int64_t>(a.H) * DV;
  if (!make_head_map(&m.q, a.q, DQK, a.H, a.qh, tq, a.qt, BM) ||
      !make_head_map(&m.qs, a.q, DQK, a.H, a.qh, tq, a.qt, BQ) ||
      !make_head_map(&m.dout, a.dout, DV, a.H, DV, tq, ot, BM) ||
      !make_head_map(&m.douts, a.dout, DV, a.H, DV, tq, ot, BQ) ||
      !make_head_map(&m.kn, a.kn, DN, a.H, a.kh, tk, a.kt, BM) ||
      !make_head_map(&m.kns, a.kn, DN, a.H, a.kh, tk, a.kt, BQ) ||
      !make_head_map(&m.v, a.v, DV, a.H, a.vh, tk, a.vt, BM) ||
      !make_head_map(&m.vs, a.v, DV, a.H, a.vh, tk, a.vt, BQ))
    return cudaErrorInvalidValue;
  if (tk > 0) {
    const uint64_t dims[2] = {DP, static_cast<uint64_t>(tk)};
    const uint64_t strides[1] = {static_cast<uint64_t>(a.pt) * 2};
    const uint32_t box[2] = {64, BM}, box_s[2] = {64, BQ};
    if (!make_tensor_map(&m.kp, a.kp, 2, dims, strides, box) ||
        !make_tensor_map(&m.kps, a.kp, 2, dims, strides, box_s))
      return cudaErrorInvalidValue;
  }
  if (tq > 0) {
    prepare_kernel<<<dim3(static_cast<unsigned>(blocks(tq, 32)), a.H), 256, 0, st>>>(a, tq);
    // Causal: at most 32 rows a sequence see so few keys, a warp each. Else all rows of a short
    // sequence do: enough blocks to fill the GPU (64 K queries of 32 keys, the whole backward: of
    // one head 1.49 ms, of 32 heads 5.1; with four blocks a sequence and head 6.97 and 7.7).
    const int64_t fill = blocks(16 * sm_count(), static_cast<int64_t>(a.n_seqs) * a.H);
    const int64_t few = a.causal ? 4 : std::min(std::max<int64_t>(fill, 4), blocks(a.max_q, 8));
    few_kernel<<<dim3(static_cast<unsigned>(few), a.n_seqs, a.H), 256, 0, st>>>(a, tq);
  }
  const int64_t kb = blocks(a.max_k, BM), qb = blocks(a.max_q, BM);
  if ((kb + qb) * a.H > 0x7fffffff) return cudaErrorInvalidValue;
  bwd_kernel<<<dim3(static_cast<unsigned>((kb + qb) * a.H), a.n_seqs), kThreads, kBytes, st>>>(
      m, a, tq, tk, static_cast<int>(kb), static_cast<int>(qb));
  if (a.max_k > 0)
    dpe_kernel<<<dim3(static_cast<unsigned>(blocks(a.max_k * (DP / 4), 256)), a.n_seqs), 256, 0,
                 st>>>(a, tk);
  return cudaGetLastError();
}

cudaError_t take_bwd_status(cudaStream_t st, int32_t* code) { return take_status(st, code); }

}  // namespace latent
}  // namespace kda
