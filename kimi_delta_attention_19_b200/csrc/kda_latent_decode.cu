// kda_latent_decode.cu -- absorbed latent attention over the paged cache.
//
//   s_j = scale q . x_j (576),  p = softmax_j(s),  o = sum_j p_j x_j[0:512]
//
// Bound by memory: a cached vector (1152 bytes, or 656 in 8 bits) is read once for all heads
// and used for 2 x (576 + 512) operations a head. 64 cached vectors at a time are a tile X
// [64 keys, 576], staged in shared memory once and used as the A operand of both products:
//   S^T [64 keys, rows]   = X Q^T        (K-major A),          rows = (query token, head)
//   O^T [512 ch, rows]   += X[:, :512]^T P^T  (MN-major A: the same bytes)
// so up to 64 rows cost one pass over X and short products do not waste the tensor core's
// 128 rows on 16 or 32 heads. A thread holds a key, the softmax statistics are per row (a
// column here) and uniform over the threads. They follow the running maximum lazily: a
// column's reference is raised only when a score passes it by 2^8 (one barrier with a vote a
// tile; p stays below 256, sums are fp32), which for real data is a tile or two a sequence;
// only then are O^T and the sums rescaled.
//
// Work: the (sequence, row block, tile) triples in order are cut into equal runs, one per SM,
// so ragged lengths balance and one long sequence fills the GPU; the at most two units a run
// does not cover whole leave fp32 partials, which a second kernel joins. Nothing is decided
// on the host: lengths may change under a captured graph.
//
// Warps: 0 loads (TMA boxes of a page's rows, 64 channels wide; two 74 KB stages, each in
// groups of channels that are loaded and released separately), 1 issues S^T, 2 O^T, 4-7 softmax and
// results (4-11 for 64 rows, 32 a warpgroup); with an 8-bit cache the warps behind them read
// the codes and write them as bf16 (exact) into the stage.
#include <cuda_fp16.h>

#include "kda_latent_tc.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int KT = 64;                    // keys of a tile
constexpr int kAtoms = DX / 64;           // 64-channel column groups of a tile
constexpr uint32_t kAtom = KT * 128;      // bytes of one
constexpr uint32_t kStage = kAtoms * kAtom;
constexpr int kGroups = 3;                // column groups of a tile: twice 256 channels, k_pe
constexpr int kMaxCtas = 160;             // of the workspace; the grid is at most this
constexpr float kRaise = 8.f;             // log2 units a score may pass its column's reference

template <int NC>
struct Sm {
  static constexpr uint32_t X = 0, Q = 2 * kStage, P = Q + kAtoms * NC * 128,
                            BAR = P + KT * 128, TM = BAR + 32 * 8, BAIL = TM + 4, BADT = BAIL + 4,
                            WORDS = BADT + 24, RED = WORDS + NC * 8, FAC = RED + 4 * NC * 4,
                            START = FAC + NC * 4, BYTES = START + 64;
};
static_assert(Sm<64>::BYTES <= 232448, "shared memory");
static_assert(Sm<64>::WORDS % 8 == 0 && Sm<64>::START % 8 == 0 && Sm<16>::START % 8 == 0, "");

struct Rec {               // per CTA, for the joining kernel
  int32_t cont, cont_lead, cont_last;  // unit its run begins inside of (-1: none), CTAs of it
  int32_t lead, lead_last;             // unit it leads into the next CTA (-1: none)
  int32_t pad[3];
};
struct Layout {
  size_t ml, part, total;
};
__host__ __device__ inline Layout ws_layout(int nc) {
  Layout l;
  l.ml = kMaxCtas * sizeof(Rec);
  l.part = l.ml + sizeof(float2) * kMaxCtas * 2 * nc;
  l.total = l.part + sizeof(float) * kMaxCtas * 2 * nc * DC;
  return l;
}

struct Args {
  DecodeLatentArgs d;
  int rb;                // row blocks of a sequence
  int R;                 // rows of a sequence, L * H
};
struct Maps {
  CUtensorMap x, q;
};

__device__ __forceinline__ bool len_ok(const DecodeLatentArgs& d, int64_t len) {
  return len >= 0 && len <= d.table_pages * d.c.page_size && (len == 0 || d.c.n_pages > 0);
}
__device__ __forceinline__ int tiles_of(const DecodeLatentArgs& d, int64_t len) {
  return len_ok(d, len) ? static_cast<int>((len + KT - 1) / KT) : 0;
}

// Walks a CTA's run: the segments (parts of units) it covers, in order.
struct Walk {
  int n, rb, tile;       // of the next segment
  int left;              // tiles of the run behind it
  int len, tiles, cnt;   // of the current segment: sequence length, unit tiles, segment tiles
  int sn, srb, st;       // current segment: sequence, row block, first tile
  __device__ bool next(const Args& a) {
    if (left <= 0) return false;
    for (;;) {
      len = a.d.lens[n];
      tiles = tiles_of(a.d, len);
      if (tiles > 0) break;
      ++n;               // the run's tiles end before N does
      rb = tile = 0;
    }
    sn = n;
    srb = rb;
    st = tile;
    cnt = min(tiles - tile, left);
    left -= cnt;
    tile = 0;
    if (++rb == a.rb) {
      rb = 0;
      ++n;
    }
    return true;
  }
};

// Sixteen e4m3 codes times 2^(be - 127) as bf16 pairs, exactly and with NaN: the conversion to
// fp16 holds every code, and an fp32 product has the range (2^-127 for be = 0 is a subnormal).
// Moving a code's bits into a bf16's place takes more integer instructions and a search for
// NaN codes: 0.263 ms against 0.244 for 256 sequences of up to 8 K.
__device__ __forceinline__ void values16(const uint4& code, uint32_t be, uint32_t (&v)[8]) {
  const uint32_t w[4] = {code.x, code.y, code.z, code.w};
  const float f = __uint_as_float(max(be << 23, 0x00400000u));
  const float2 ff = make_float2(f, f);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t h;
    const auto c = static_cast<unsigned short>(w[k / 2] >> (16 * (k & 1)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    __half2 hh;
    memcpy(&hh, &h, 4);
    const float2 x = mul2f(__half22float2(hh), ff);
    v[k] = pack2(x.x, x.y);
  }
}

// Loads of cached rows and block tables: ordinary (coherent) ones, as the kernel ahead may have
// been writing them when this one started, which the read-only path does not allow. Written so
// that the compiler may move them like that path's (plain accesses stay between the stores and
// barriers around them: 0.263 ms against 0.248 for 256 sequences of up to 8 K); none gets ahead of
// griddep_wait, as every address comes from lengths read behind it, and nothing here writes them.
__device__ __forceinline__ uint4 ld_row(const uint4* p) {
  uint4 r;
  asm("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ uint32_t ld_row(const uint32_t* p) {
  uint32_t r;
  asm("ld.global.u32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}
__device__ __forceinline__ int ld_row(const int32_t* p) {
  return static_cast<int>(ld_row(reinterpret_cast<const uint32_t*>(p)));
}

// Softmax warpgroups (up to 32 columns each), converting ones (8-bit caches), and registers a
// thread: of the first warpgroup, the softmax ones and the converting ones (8-bit caches).
template <int NC, bool F8>
struct Roles {
  static constexpr int kSoft = NC == 64 ? 2 : 1, kSets = F8 ? 2 : 0;
  static constexpr int kThreads = 128 + 128 * kSoft + 256 * kSets;
  static constexpr int kRegs = 512 / (kThreads / 128) / 8 * 8;  // at launch
  static constexpr int kR0 = NC == 64 ? 56 : 72, kRs = NC == 64 ? 96 : 120,
                       kRc = NC == 64 ? 64 : 72;
  static_assert(!F8 || (kR0 <= kRegs && kRs >= kRegs && kRc <= kRegs), "");
  static_assert(!F8 || kR0 + kRs * kSoft + kRc * 2 * kSets <= kRegs * (kThreads / 128), "");
};

template <int NC, bool F8>
__global__ void __launch_bounds__(Roles<NC, F8>::kThreads, 1)
    decode_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ __align__(1024) unsigned char sm[];
  using S = Sm<NC>;
  using R = Roles<NC, F8>;
  // Column groups are loaded and released together; few, as a wait or a commit costs an issuing
  // thread ~90 clocks.
  constexpr int kG = kGroups, kGA = 4;            // groups, 64-channel atoms of a latent one
  constexpr int NW = NC / R::kSoft, NH = NW / 2;  // rows of a softmax warpgroup, of a thread
  constexpr uint32_t kCols = NC == 64 ? 512 : NC == 32 ? 256 : 128;  // 4 NC of O^T, 2 NC of S^T
  constexpr int kThreads = R::kThreads;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + S::BAR);
  uint64_t *full = bar, *empty = bar + 6, *s_full = bar + 12, *p_full = bar + 14, *pv_done = bar + 15,
           *q_full = bar + 16, *q_empty = bar + 17, *o_free = bar + 18, *s_read = bar + 19,
           *drain = bar + 21;
  uint32_t* tmem = reinterpret_cast<uint32_t*>(sm + S::TM);
  volatile int* bail = reinterpret_cast<volatile int*>(sm + S::BAIL);
  volatile int* bad_tile = reinterpret_cast<volatile int*>(sm + S::BADT);
  uint64_t* words = reinterpret_cast<uint64_t*>(sm + S::WORDS);
  float* red = reinterpret_cast<float*>(sm + S::RED);
  float* fac = reinterpret_cast<float*>(sm + S::FAC);
  int64_t* start = reinterpret_cast<int64_t*>(sm + S::START);
  const uint32_t sb = smem_u32(sm);
  const DecodeLatentArgs& d = a.d;
  Rec* rec = reinterpret_cast<Rec*>(d.ws) + blockIdx.x;
  const Layout wl = ws_layout(NC);

  if (sb & 1023) {  // the operand tiles need it, and nothing else is in shared memory
    if (tid == 0) report(d.status, kDevWaitTimeout);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2 * kGroups; ++i) {
      mbar_init(full + i, F8 && i % kGroups < kG - 1 ? 8 : 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_full + 1, 1);
    mbar_init(p_full, 128 * R::kSoft);
    mbar_init(pv_done, 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_free, 128 * R::kSoft);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_read + i, 128 * R::kSoft);
      mbar_init(drain + i, 1);
    }
    fence_mbar_init();
    *bail = 0;
    bad_tile[0] = bad_tile[1] = 0;
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.x);
  }
  griddep_wait();  // so far nothing was read or written that a kernel before this one may touch
  if (tid == 0) rec->cont = rec->lead = -1;
  // (not before: a CTA of the kernel ahead may still need the columns, and would wait for this one
  // while this one waits for it)
  if (warp == 1) {
    tmem_alloc(tmem, kCols);
    tmem_relinquish();
  }
  // This CTA's run: tiles [t0, t1) of all sequences' tiles in order.
  const int per = (d.N + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int n = tid * per; n < min(d.N, (tid + 1) * per); ++n)
    mine += static_cast<int64_t>(tiles_of(d, d.lens[n])) * a.rb;
  int64_t pre = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, pre, off);
    if (lane >= off) pre += up;
  }
  int64_t* wsum = reinterpret_cast<int64_t*>(sm + S::P);  // not in use yet
  if (lane == 31) wsum[warp] = pre;
  __syncthreads();
  int64_t total = 0;
  pre -= mine;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) pre += wsum[w];
    total += wsum[w];
  }
  const int64_t G = total < gridDim.x ? total : gridDim.x;
  const int64_t c = blockIdx.x;
  const int64_t t0 = c < G ? c * total / G : 0, t1 = c < G ? (c + 1) * total / G : 0;
  if (t0 < t1 && pre <= t0 && t0 < pre + mine) {
    int64_t at = pre;
    for (int n = tid * per;; ++n) {
      const int tl = tiles_of(d, d.lens[n]);
      const int64_t u = static_cast<int64_t>(tl) * a.rb;
      if (t0 < at + u) {
        start[0] = n;
        start[1] = (t0 - at) / tl;
        start[2] = (t0 - at) % tl;
        break;
      }
      at += u;
    }
  }
  // sequences without a tile: empty (zeros) or refused (NaN), spread over the CTAs
  for (int n = blockIdx.x; n < d.N; n += gridDim.x) {
    const int64_t len = d.lens[n];
    if (tiles_of(d, len) > 0) continue;
    const bool bad = !len_ok(d, len);
    if (bad && tid == 0) report(d.status, kDevBadPage);
    const uint4 v = bad ? make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu)
                        : make_uint4(0, 0, 0, 0);
    uint4* o = reinterpret_cast<uint4*>(d.out + static_cast<int64_t>(n) * a.R * DC);
    for (int64_t i = tid; i < static_cast<int64_t>(a.R) * (DC / 8); i += kThreads) o[i] = v;
    if (d.lse != nullptr)
      for (int i = tid; i < a.R; i += kThreads)
        d.lse[static_cast<int64_t>(n) * a.R + i] = bad ? NAN : -INFINITY;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();  // the joining kernel waits for this one's end by itself
  const uint32_t tb = *tmem;
  Walk wk;
  wk.left = static_cast<int>(t1 - t0);
  wk.n = wk.left > 0 ? static_cast<int>(start[0]) : 0;
  wk.rb = wk.left > 0 ? static_cast<int>(start[1]) : 0;
  wk.tile = wk.left > 0 ? static_cast<int>(start[2]) : 0;
  const int n_tiles = wk.left;

  if (warp < 4) {
    if constexpr (F8) reg_dec<R::kR0>();
    if (warp == 0) {
      // ------------------------------------------------------------------ loads
      const int ps = d.c.page_size, pr = ps < KT ? ps : KT;  // rows of a box
      int t = 0, q_loads = 0, groups = 0;  // groups: column groups under way, in order
      bool stop = false;
      for (int seg = 0; wk.next(a); ++seg) {
        auto load_q = [&] {
          if (seg > 0) wait_for(q_empty, (seg - 1) & 1, bail);
          stop |= bailed(bail);
          if (stop) return;
          ++q_loads;
          if (lane == 0) mbar_arrive_expect_tx(q_full, kAtoms * NC * 128);
          __syncwarp();
          if (lane < kAtoms)
            tma_load_2d(sm + S::Q + lane * NC * 128, &maps.q, q_full, lane * 64,
                        wk.sn * a.R + wk.srb * NC);
        };
        if (seg == 0) load_q();
        for (int i = 0; i < wk.cnt; ++i, ++t) {
          const int s = t & 1;
          const int pos = (wk.st + i) * KT + lane * pr;
          int64_t page = 0;
          const bool there = lane < KT / pr && pos < wk.len;
          if (there) page = d.table[wk.sn * d.table_pages + pos / ps];
          const bool bad = page < 0 || page >= d.c.n_pages;
          if (bad) page = 0;
          const bool any_bad = __any_sync(0xffffffffu, bad);
          const int nb = __popc(__ballot_sync(0xffffffffu, there));
          const int row = static_cast<int>(page * ps + pos % ps);
          const int y = __shfl_sync(0xffffffffu, row, lane / kGA & 3);
#pragma unroll
          for (int g = F8 ? kG - 1 : 0; g < kG; ++g) {
            if (t >= 2) wait_for(empty + s * kGroups + g, (t / 2 - 1) & 1, bail);
            stop |= bailed(bail);
            if (stop) continue;
            ++groups;
            // (the stage's last tile has been looked at once its O^T is under way)
            if (!F8 && g == 0 && any_bad && lane == 0) bad_tile[s] = t + 1;
            uint64_t* f = full + s * kGroups + g;
            if (lane == 0) mbar_arrive_expect_tx(f, nb * pr * (g < kG - 1 ? kGA * 128 : 128));
            __syncwarp();
            const int atom = kGA * g + lane % kGA;
            if (lane < kGA * nb && atom < kAtoms)
              tma_load_2d(sm + S::X + s * kStage + atom * kAtom + lane / kGA * pr * 128, &maps.x, f,
                          F8 ? kPe8 / 2 : atom * 64, y);
          }
          if (seg > 0 && i == 0) load_q();
        }
      }
      if (q_loads > 0) mbar_wait(q_full, (q_loads - 1) & 1, kDrainCycles);
      constexpr int kPer = F8 ? 1 : kG;  // groups a tile
      for (int k = max(0, groups - 2 * kPer); k < groups; ++k)
        mbar_wait(full + (k / kPer & 1) * kGroups + (F8 ? kG - 1 : k % kPer), k / kPer / 2 & 1, kDrainCycles);
    } else if (warp == 1) {
      // --------------------------------------------------------- products: S^T
      // Two warps issue, so that O^T of a tile waits neither for the next tile to arrive nor for
      // its S^T to be issued (~30 clocks an instruction).
      constexpr uint32_t iq = idesc_bf16(64, NC, 0, 0);
      if (elect_one()) {
        int t = 0;
        for (int seg = 0; wk.next(a); ++seg) {
          wait_for(q_full, seg & 1, bail);
          for (int i = 0; i < wk.cnt; ++i, ++t) {
            const int s = t & 1;
            const uint32_t dst = tb + 4 * NC + s * NC;
            const uint64_t xa = sdesc_sw128(sb + S::X + s * kStage, 16, 1024);
            const uint64_t qb = sdesc_sw128(sb + S::Q, 16, 1024);
            if (t >= 2) wait_for(s_read + s, (t / 2 - 1) & 1, bail);
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              wait_for(full + s * kGroups + g, t / 2 & 1, bail);
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < (g < kG - 1 ? 4 * kGA : 4); ++k) {
                const int at = kGA * g + k / 4;  // atom
                umma_bf16(dst, xa + at * (kAtom / 16) + k % 4 * 2, qb + at * (NC * 8) + k % 4 * 2, iq,
                          g > 0 || k > 0);
              }
            }
            umma_commit(s_full + s);
            umma_commit(empty + s * kGroups + kG - 1);
            if (i + 1 == wk.cnt) umma_commit(q_empty);
          }
        }
        umma_commit(drain);
        mbar_wait(drain, 0, kDrainCycles);
      }
    } else if (warp == 2) {
      // --------------------------------------------------------- products: O^T
      constexpr uint32_t ip = idesc_bf16(128, NC, 1, 1);
      if (elect_one()) {
        int t = 0;
        for (int seg = 0; wk.next(a); ++seg) {
          for (int i = 0; i < wk.cnt; ++i, ++t) {
            const int s = t & 1;
            const uint64_t pb = sdesc_sw128(sb + S::P, 8192, 1024);
            const uint64_t xa = sdesc_sw128(sb + S::X + s * kStage, kAtom, 1024);
            wait_for(p_full, t & 1, bail);  // so S^T is formed, and the tile is there
            if (i == 0 && seg > 0) wait_for(o_free, (seg - 1) & 1, bail);
            tc_fence_after();
#pragma unroll
            for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_bf16(tb + mb * NC, xa + 2 * mb * (kAtom / 16) + 128 * k, pb + 128 * k, ip,
                          i > 0 || k > 0);
              if ((2 * mb + 2) % kGA == 0) umma_commit(empty + s * kGroups + 2 * mb / kGA);
            }
            umma_commit(pv_done);
          }
        }
        umma_commit(drain + 1);
        mbar_wait(drain + 1, 0, kDrainCycles);
      }
    }
  } else if (warp < 4 + 4 * R::kSoft) {
    if constexpr (F8) reg_inc<R::kRs>();
    // ---------------------------------------------------- softmax and results
    const int w = warp % 4, wg = (warp - 4) / 4, tw = tid % 128, c_lo = wg * NW;
    const uint32_t lanes = tb + (static_cast<uint32_t>(w * 32) << 16);
    const int half = lane >> 4, ch0 = c_lo + half * NH, kk = w * 16 + (lane & 15);
    const float sl = d.scale * kLog2e;
    int t = 0;
    bool first_seg = true;
    int64_t gt = t0;  // global index of the segment's first tile
    for (; wk.next(a); first_seg = false) {
      const int first = wk.len - d.L;  // position of the first query token
      if (tw < NW) {
        const int row = wk.srb * NC + c_lo + tw, i = row / d.H;
        words[c_lo + tw] = row >= a.R ? 0
                    : d.mask != nullptr
                        ? static_cast<uint64_t>(d.mask[static_cast<int64_t>(wk.sn) * d.L + i])
                        : (2ull << i) - 1;
      }
      group_sync(1 + wg, 128);
      // nm: minus a column's reference in log2 units, +inf before its first score
      float nm[NH], l[NH];
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        nm[i] = INFINITY;
        l[i] = 0.f;
      }
      bool bad = false;
      for (int i = 0; i < wk.cnt; ++i, ++t) {
        const int s = t & 1, valid = wk.len - (wk.st + i) * KT;
        wait_for(s_full + s, t / 2 & 1, bail);
        tc_fence_after();
        bad |= bad_tile[s] == t + 1;
        float x[NH];
        {
          // an M = 64 product's row r is in tensor-memory lane 32 (r / 16) + r % 16: the
          // upper half of a warp takes the upper half of the columns from the lower one
          const uint32_t sc = lanes + 4 * NC + s * NC + c_lo;
          uint32_t v[NW];
          if constexpr (NW == 32) tmem_ld32(sc, v);
          else tmem_ld16(sc, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int k = 0; k < NH; ++k) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, v[k + NH], 16);
            x[k] = __uint_as_float(half ? up : v[k]);
          }
        }
        tc_fence_before();
        mbar_arrive(s_read + s);
        const int kj = (wk.st + i) * KT + kk - first;  // among the query tokens
        if (kk >= valid) {
#pragma unroll
          for (int k = 0; k < NH; ++k) x[k] = -INFINITY;
        } else if (kj >= 0) {
#pragma unroll
          for (int k = 0; k < NH; ++k)
            if (!(words[ch0 + k] >> kj & 1)) x[k] = -INFINITY;
        }
        // y = log2 of p; a column without a reference gives +inf, a masked key there NaN,
        // which the maximum passes over
        float y[NH], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < NH; ++k) y[k] = fmaf(x[k], sl, nm[k]);
#pragma unroll
        for (int k = 0; k < NH; k += 2) top = fmaxf(top, fmaxf(y[k], y[k + 1]));
        if (group_any(1 + wg, 128, top > kRaise)) {
          // raise the columns' references to the running maximum, rescale sums and O^T
#pragma unroll
          for (int k = 0; k < NH; ++k) {
            float z = sl * x[k];
#pragma unroll
            for (int off = 8; off > 0; off >>= 1)
              z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, off));
            if ((lane & 15) == 0) red[w * NC + ch0 + k] = z;
          }
          group_sync(1 + wg, 128);
#pragma unroll
          for (int k = 0; k < NH; ++k) {
            const int cc = ch0 + k;
            const float z = fmaxf(fmaxf(red[cc], red[NC + cc]), fmaxf(red[2 * NC + cc], red[3 * NC + cc]));
            const float mn = -fmaxf(-nm[k], z);
            const float f = nm[k] == INFINITY ? 0.f : ex2(mn - nm[k]);
            l[k] *= f;
            nm[k] = mn;
            if (w == 0 && (lane & 15) == 0) fac[cc] = f;
          }
          group_sync(1 + wg, 128);
          if (i > 0) {
            wait_for(pv_done, (t - 1) & 1, bail);
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 4 * NW / 16; ++q) {
              const int c0 = c_lo + q * 16 % NW, at = q * 16 / NW * NC + c0;
              uint32_t v[16];
              tmem_ld16(lanes + at, v);
              tmem_ld_wait(v);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                v[k] = __float_as_uint(__uint_as_float(v[k]) * fac[c0 + k]);
              tmem_st16(lanes + at, v);
            }
            tmem_st_wait();
          }
#pragma unroll
          for (int k = 0; k < NH; ++k) y[k] = fmaf(x[k], sl, nm[k]);
        }
        // A column without a reference has seen masked keys (-inf) and NaN only: p of the score
        // itself. p enters the product as bf16 (half a step, 2^-9 of it); its sum is fp32.
        uint32_t p[NH / 2];
#pragma unroll
        for (int k = 0; k < NH; k += 2) {
          const float a0 = ex2(nm[k] == INFINITY ? x[k] : y[k]);
          const float a1 = ex2(nm[k + 1] == INFINITY ? x[k + 1] : y[k + 1]);
          l[k] += a0;
          l[k + 1] += a1;
          p[k / 2] = pack2(a0, a1);
        }
        if (t > 0) wait_for(pv_done, (t - 1) & 1, bail);  // P is free
#pragma unroll
        for (int q = 0; q < NH / 8; ++q)
          *reinterpret_cast<uint4*>(sm + S::P + sw128_chunk(kk, ch0 / 8 + q, 0)) =
              make_uint4(p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]);
        if (!F8 && valid < KT) {  // rows past the sequence may hold anything: 0 x NaN is NaN
          for (int e = tid - 128; e < (KT - valid) * 64; e += 128 * R::kSoft) {
            const int r = valid + (e >> 6), ck = e & 63;
            *reinterpret_cast<uint4*>(sm + S::X + s * kStage + sw128_chunk(r, ck, kAtom)) =
                make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(p_full);
      }
      // the segment's sums
      group_sync(1 + wg, 128);  // the last tile's factors are read
#pragma unroll
      for (int k = 0; k < NH; ++k) {
        float y = l[k];
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if ((lane & 15) == 0) {
          red[w * NC + ch0 + k] = y;
          if (w == 0) fac[ch0 + k] = -nm[k];
        }
      }
      group_sync(1 + wg, 128);
      const bool whole = wk.st == 0 && wk.cnt == wk.tiles;
      const int slot = wk.st > 0 ? 0 : 1;
      const int64_t part = (c * 2 + slot) * NC;
      const int64_t row0 = static_cast<int64_t>(wk.sn) * a.R + wk.srb * NC;
      const int rows = min(NC, a.R - wk.srb * NC);
      const int cw = c_lo + tw;  // a thread's column (tw < NW)
      float mul = 1.f;
      if (tw < NW) {
        const float ls = (red[cw] + red[NC + cw]) + (red[2 * NC + cw] + red[3 * NC + cw]);
        const float ms = fac[cw];
        if (whole) {
          mul = bad ? NAN : ls == 0.f ? 0.f : 1.f / ls;
          if (cw < rows && d.lse != nullptr)
            d.lse[row0 + cw] = bad ? NAN : ls == 0.f ? -INFINITY : (ms + log2f(ls)) * kLn2;
        } else {
          reinterpret_cast<float2*>(d.ws + wl.ml)[part + cw] = make_float2(ms, bad ? NAN : ls);
        }
      }
      group_sync(1 + wg, 128);
      if (tw < NW) fac[cw] = mul;
      if (tid == 128) {
        if (bad) report(d.status, kDevBadPage);
        const int64_t u0 = gt - wk.st, u1 = u0 + wk.tiles - 1;  // the unit's first, last tile
        const int unit = wk.sn * a.rb + wk.srb;
        const int last_cta = static_cast<int>(((u1 + 1) * G - 1) / total);
        if (wk.st > 0) {
          rec->cont_lead = static_cast<int>(((u0 + 1) * G - 1) / total);
          rec->cont_last = last_cta;
          rec->cont = unit;
        } else if (!whole) {
          rec->lead_last = last_cta;
          rec->lead = unit;
        }
      }
      group_sync(1 + wg, 128);
      wait_for_results(pv_done, (t - 1) & 1, bail);
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < 4 * NW / 16; ++q) {
        const int c0 = c_lo + q * 16 % NW, mb = q * 16 / NW, ch = mb * 128 + w * 32 + lane;
        uint32_t v[16];
        tmem_ld16(lanes + mb * NC + c0, v);
        tmem_ld_wait(v);
        if (whole) {
          // lane pairs trade values, so that each writes two adjacent channels of a row
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float f0 = __uint_as_float(v[k]) * fac[c0 + k];
            const float f1 = __uint_as_float(v[k + 1]) * fac[c0 + k + 1];
            const float o = __shfl_xor_sync(0xffffffffu, lane & 1 ? f0 : f1, 1);
            const int r = c0 + k + (lane & 1);
            const uint32_t pk = lane & 1 ? pack2(o, f1) : pack2(f0, o);
            if (r < rows)
              *reinterpret_cast<uint32_t*>(d.out + (row0 + r) * DC + (ch & ~1)) = pk;
          }
        } else {
          float* dst = reinterpret_cast<float*>(d.ws + wl.part) + (part + c0) * DC + ch;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (c0 + k < rows) dst[k * DC] = __uint_as_float(v[k]);
        }
      }
      tc_fence_before();
      mbar_arrive(o_free);
      gt += wk.cnt;
      group_sync(1 + wg, 128);  // fac, red and words are free
    }
  } else if (F8) {
    // ------------------------------------------- 8-bit rows, as bf16 into the stages
    reg_dec<R::kRc>();
    // Two sets of eight warps, one a column group (k_pe is copied as it is, by TMA). Four threads
    // a row; of 128 channels (a scale's) one takes the codes 16 q .. and 64 + 16 q .., so that 8
    // threads' stores touch all banks. The registers are refilled with the next tile's codes as
    // soon as they are converted; the block table is read a tile further ahead.
    const int i = tid - 128 - 128 * R::kSoft, set = i / 256, row = i % 256 / 4, qd = i % 4;
    Walk ahead = wk;
    int left = n_tiles, in_seg = 0;
    ahead.cnt = 0;
    const int shift = 31 - __clz(d.c.page_size);
    struct Row {
      int page, off;  // page -1: no row there, or (off >= 0) a page out of range
    };
    // The next tile's place of this thread's row. The page number is not looked at before the
    // tile after it is being converted, so its load is not waited for.
    auto fetch = [&]() -> Row {
      if (left == 0) return Row{-1, -1};
      --left;
      if (in_seg == ahead.cnt) {
        ahead.next(a);
        in_seg = 0;
      }
      const int pos = (ahead.st + in_seg++) * KT + row;
      if (pos >= ahead.len) return Row{-1, -1};
      return Row{ld_row(d.table + (ahead.sn * d.table_pages + (pos >> shift))),
                 pos & (d.c.page_size - 1)};
    };
    auto place = [&](const Row& r) -> const unsigned char* {
      if (r.page < 0 || r.page >= d.c.n_pages) return nullptr;
      return d.c.cache + ((static_cast<int64_t>(r.page) << shift) + r.off) * kRow8;
    };
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto ld = [&](const unsigned char* p, int off) {
      return p != nullptr ? ld_row(reinterpret_cast<const uint4*>(p + off)) : zero;
    };
    uint4 code[2][2];
    auto load = [&](const unsigned char* p, int k) {  // 128 channels of the set's 256
#pragma unroll
      for (int h = 0; h < 2; ++h) code[k][h] = ld(p, (2 * set + k) * 128 + h * 64 + qd * 16);
    };
    auto load_ex = [&](const unsigned char* p) {
      return p != nullptr ? ld_row(reinterpret_cast<const uint32_t*>(p + kExp8)) : 0u;
    };
    const Row r0 = fetch();
    const unsigned char* const p0 = place(r0);
    bool bad = p0 == nullptr && r0.off >= 0;
    Row nxt = fetch();
#pragma unroll
    for (int k = 0; k < 2; ++k) load(p0, k);
    uint32_t ex = load_ex(p0);
    const uint32_t sw = row & 7;
    unsigned char* const row_at = sm + S::X + (row >> 3) * 1024 + sw * 128;
    for (int t = 0; t < n_tiles; ++t) {
      const int s = t & 1;
      const unsigned char* const np = place(nxt);
      const bool nbad = np == nullptr && nxt.off >= 0;
      nxt = fetch();
      unsigned char* const dst = row_at + s * kStage;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int g = 2 * set + k;  // of 128 channels
        uint32_t v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) values16(code[k][h], ex >> (8 * g) & 0xffu, v[h]);
        load(np, k);
        if (k == 0) {
          if (t >= 2) wait_for(empty + s * kGroups + set, (t / 2 - 1) & 1, bail);
          if (bad) bad_tile[s] = t + 1;  // (the stage's last tile has been looked at)
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            *reinterpret_cast<uint4*>(dst + (2 * g + h) * kAtom + ((qd * 2 + j) ^ sw) * 16) =
                make_uint4(v[h][4 * j], v[h][4 * j + 1], v[h][4 * j + 2], v[h][4 * j + 3]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + s * kGroups + set);
      ex = load_ex(np);
      bad = nbad;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *bail) report(d.status, kDevWaitTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, kCols);
  }
}

// Joins the partials of the units that runs cut: sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c
// over the CTAs of a unit, in their order. Usually those are two: sixteen rows a block, the
// partials of its CTA and the next fetched before it is known whether they belong together (the
// kernel is a chain of memory latencies). Another unit is shared by the blocks of all of
// them: half a row is a warp's work; from 33 CTAs on a quarter row is a block's, its partials
// spread over the block's 16 warps and summed in the warps' order.
constexpr int kJoinRows = 16;

__device__ __forceinline__ void put_row(const Args& a, int64_t row, int ch, float4 acc, float M, float l) {
  const bool nan = l != l;  // poisons rows whose partials were not
  const float mul = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(a.d.out + row * DC + ch) =
      nan ? make_uint2(0x7fff7fffu, 0x7fff7fffu)
          : make_uint2(pack2(acc.x * mul, acc.y * mul), pack2(acc.z * mul, acc.w * mul));
  if (ch == 0 && a.d.lse != nullptr)
    a.d.lse[row] = nan ? l : l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

// a partial's weight against the joint reference, and what it adds to the sum
__device__ __forceinline__ float weight(float m, float M) { return m == -INFINITY ? 0.f : ex2(m - M); }
__device__ __forceinline__ float share(float f, float l) { return l != l ? l : f * l; }  // NaN: a bad page

template <int NC>
__global__ void __launch_bounds__(512, NC == 64 ? 2 : 1) join_kernel(const Args a) {
  const Layout wl = ws_layout(NC);
  const float2* ml = reinterpret_cast<const float2*>(a.d.ws + wl.ml);
  const float* part = reinterpret_cast<const float*>(a.d.ws + wl.part);
  __shared__ float4 acc_s[16][32];
  __shared__ float2 ml_s[16];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  griddep_launch_dependents();  // (a next call sets up meanwhile)
  griddep_wait();
  constexpr bool kPairs = NC <= 32;  // (of 64 rows the unneeded loads cost more: 111 us for 104)
  constexpr int kRows = kJoinRows / 4;  // of a thread
  float2 x[kRows][2];
  float4 o[kRows][2];
#pragma unroll
  for (int k = 0; kPairs && k < kRows; ++k)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int c = min(static_cast<int>(blockIdx.x) + p, kMaxCtas - 1);
      const int i = (c * 2 + 1 - p) * NC + blockIdx.y * kJoinRows + k * 4 + threadIdx.x / 128;
      x[k][p] = ml[i];
      o[k][p] = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(i) * DC + threadIdx.x % 128 * 4);
    }
  const Rec r = reinterpret_cast<const Rec*>(a.d.ws)[blockIdx.x];
  auto add = [](float4& acc, float f, const float4& v) {
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  };
  for (int pass = 0; pass < 2; ++pass) {
    const int unit = pass ? r.cont : r.lead;
    if (unit < 0) continue;
    const int c0 = pass ? r.cont_lead : blockIdx.x, np = (pass ? r.cont_last : r.lead_last) - c0 + 1;
    const int n = unit / a.rb, rb = unit % a.rb, rows = min(NC, a.R - rb * NC);
    const int64_t row0 = static_cast<int64_t>(n) * a.R + rb * NC;
    auto at = [&](int p, int row) { return ((c0 + p) * 2 + (p == 0 ? 1 : 0)) * NC + row; };
    if (kPairs && np == 2) {
      if (pass) continue;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int row = blockIdx.y * kJoinRows + k * 4 + threadIdx.x / 128;
        if (row >= rows) continue;
        const float M = fmaxf(x[k][0].x, x[k][1].x);
        const float f0 = weight(x[k][0].x, M), f1 = weight(x[k][1].x, M);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        add(acc, f0, o[k][0]);
        add(acc, f1, o[k][1]);
        put_row(a, row0 + row, threadIdx.x % 128 * 4, acc, M, share(f0, x[k][0].y) + share(f1, x[k][1].y));
      }
      continue;
    }
    const int b = (blockIdx.x - c0) * gridDim.y + blockIdx.y, blocks = np * gridDim.y;
    if (np <= 32) {
      for (int item = b * 16 + warp; item < rows * 2; item += blocks * 16) {
        const int row = item / 2, ch = item % 2 * 256 + lane * 4;
        const float2 y = lane < np ? ml[at(lane, row)] : make_float2(-INFINITY, 0.f);
        float M, f = 0.f, l = 0.f;
        float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
        constexpr int kAtOnce = 4;
        for (int p0 = 0; p0 < np; p0 += kAtOnce) {
          float4 v[kAtOnce][2];
#pragma unroll
          for (int p = 0; p < kAtOnce; ++p) {
            const float* src = part + static_cast<int64_t>(at(min(p0 + p, np - 1), row)) * DC + ch;
            v[p][0] = *reinterpret_cast<const float4*>(src);
            v[p][1] = *reinterpret_cast<const float4*>(src + 128);
          }
          if (p0 == 0) {  // weights and their sum, while the first are on their way
            M = y.x;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
            f = weight(y.x, M);
            l = share(f, y.y);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
          }
#pragma unroll
          for (int p = 0; p < kAtOnce; ++p) {
            const float fp = __shfl_sync(0xffffffffu, f, (p0 + p) & 31);
            if (p0 + p >= np) continue;
            add(acc[0], fp, v[p][0]);
            add(acc[1], fp, v[p][1]);
          }
        }
        put_row(a, row0 + row, ch, acc[0], M, l);
        put_row(a, row0 + row, ch + 128, acc[1], M, l);
      }
      continue;
    }
    for (int item = b; item < rows * 4; item += blocks) {
      const int row = item / 4, ch = item % 4 * 128 + lane * 4;
      float M = -INFINITY, l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = warp + 16 * lane; p < np; p += 16 * 32) M = fmaxf(M, ml[at(p, row)].x);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll 5
      for (int p = warp; p < np; p += 16) {
        const float2 y = ml[at(p, row)];
        const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(at(p, row)) * DC + ch);
        const float f = weight(y.x, M);
        l += share(f, y.y);
        add(acc, f, v);
      }
      acc_s[warp][lane] = acc;
      if (lane == 0) ml_s[warp] = make_float2(M, l);
      __syncthreads();
      if (warp == 0) {
        for (int g = 0; g < 16; ++g) M = fmaxf(M, ml_s[g].x);
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int g = 0; g < 16; ++g) {
          const float f = weight(ml_s[g].x, M);
          l += share(f, ml_s[g].y);
          add(acc, f, acc_s[g][lane]);
        }
        put_row(a, row0 + row, ch, acc, M, l);
      }
      __syncthreads();
    }
  }
}

// Rows of a block: the fewest of 16, 32, 64 that hold a sequence's rows, else 64 (more rows
// would not fit the query block beside two stages; 16 and 32 leave the tensor pipe half idle).
int block_rows(int L, int H) {
  const int64_t r = static_cast<int64_t>(L) * H;
  return r <= 16 ? 16 : r <= 32 ? 32 : 64;
}

template <int NC, bool F8>
cudaError_t launch(const DecodeLatentArgs& d, cudaStream_t st) {
  // (first: it makes the device's context current in a thread that has none yet, as autograd's,
  // which the encoding of maps needs)
  auto kern = decode_kernel<NC, F8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Sm<NC>::BYTES);
  if (e != cudaSuccess) return e;
  Args a{d, (d.L * d.H + NC - 1) / NC, d.L * d.H};
  Maps m;
  memset(&m, 0, sizeof m);
  const int64_t rows = d.c.n_pages * d.c.page_size;
  {
    const uint64_t dims[2] = {DX, static_cast<uint64_t>(d.N) * a.R}, strides[1] = {DX * 2};
    const uint32_t box[2] = {64, NC};
    if (!make_tensor_map(&m.q, d.q, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  if (rows > 0) {  // of an 8-bit cache: k_pe, copied as it is
    const uint64_t pitch = F8 ? kRow8 : DX * 2;
    const uint64_t dims[2] = {pitch / 2, static_cast<uint64_t>(rows)}, strides[1] = {pitch};
    const uint32_t box[2] = {64, static_cast<uint32_t>(d.c.page_size < KT ? d.c.page_size : KT)};
    if (!make_tensor_map(&m.x, d.c.cache, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const int sms = sm_count();
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  e = launch_early(kern, dim3(grid), Roles<NC, F8>::kThreads, Sm<NC>::BYTES, st, m, a);
  if (e != cudaSuccess) return e;
  return launch_early(join_kernel<NC>, dim3(grid, NC / kJoinRows), 512, 0, st, a);
}

}  // namespace

size_t decode_workspace(int L, int H) { return ws_layout(block_rows(L, H)).total; }

cudaError_t launch_latent_decode(const DecodeLatentArgs& d, cudaStream_t st) {
  const bool f8 = d.c.format == KDA_CACHE_E4M3;
  switch (block_rows(d.L, d.H)) {
    case 16: return f8 ? launch<16, true>(d, st) : launch<16, false>(d, st);
    case 32: return f8 ? launch<32, true>(d, st) : launch<32, false>(d, st);
    default: return f8 ? launch<64, true>(d, st) : launch<64, false>(d, st);
  }
}

cudaError_t take_decode_status(cudaStream_t st, int32_t* code) { return take_status(st, code); }

}  // namespace latent
}  // namespace kda
