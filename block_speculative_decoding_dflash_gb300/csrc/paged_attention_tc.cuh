// Attention over the paged cache on the tensor cores (bf16, head_dim <= 128).
//
// A CTA takes QT tiles of 128 packed query rows (row r of a tile: new row r / G,
// head r % G of the kv head's group) and walks the key tiles of 128 rows that
// any of them sees. S = Q K^T and O += P V are tcgen05 products with S, P and O
// in TMEM: a softmax thread owns one query row (one TMEM lane), so row maxima
// and sums need no exchange between threads, and P, in bf16, takes the place
// of the S it came from and is the A operand of P V where it lies.
//
// Warps: 4 per query tile for the softmax, then one that issues the TMA loads
// of K and V (a ring of stages, filled page by page), one that issues the MMAs,
// two that look after V. With two query tiles the MMAs of one run while the
// other's softmax does; with one, S has two buffers for the same purpose.
//
// The running maximum is raised, and O rescaled, only when a row's maximum
// grows by more than 8 (in log2 units): p stays below 2^8, which costs neither
// fp32 sums nor bf16 products any relative accuracy, and after the first tiles
// nearly no tile needs it.
//
// A tile of at most 32 (64) rows, a decode or verify block's, is held 4 (2) times
// in the tile's lanes (where a token's heads are 32 at most): each warp then takes
// a quarter (half) of the keys, its lanes' P is zero for the others', and the
// warps' outputs are joined at the end like those of splits. The softmax of a
// tile takes a quarter of the time, and all four warps have work, which pays for
// the second part of P (below).
//
// P as a product's operand is bf16. For those few rows, where K and V's bytes
// are the bound, it is two bf16 parts (16 bits of p, two products), the second
// in the half of S's columns that the first leaves free, or, of a sequence that
// a batch with prompts gives to the two-tile kernel, in the S of the tile that
// it does not have: what a batch holds beside a decode row does not change how
// exact the row is. For many rows, a prompt's, where the products are the bound, and a
// tree's that fill more than 64 of the tile's, where they share the time with the softmax,
// it is rounded: half a step, 2^-8 relative at most and independent from key to key,
// adds as much error to an output as the output's own rounding to bf16 does
// (measured against fp64: 0.0023 of the norm instead of 0.0017). The sum of p is
// taken before, in fp32.
//
// Rows that a query does not see get p = 0, but 0 times an infinite or NaN V is
// NaN. So in every tile that is not wholly seen by all its queries two warps
// look for such rows of V and zero them in shared memory, and the queries that
// do see them add p v themselves.
//
// 2048 rows over 32768 keys: 0.77 ms, 1.40 PFLOP/s; no pipe is full
// (tensor 58%, issue 36%, special functions 30%): what is left are the waves (256
// CTAs on 152 SMs) and each score's chain of dependent steps, a TMEM read, the
// maximum, a second read, the exponential and a write, which two query tiles take in
// turns. 48 sequences that decode one token, up to 12345 keys: 264 us, 5.1 TB/s; a
// block of 4 in a window of 2048: 14 us, of which the first loads' chain (ranges,
// length, page, rows) and the join are most. 24 trees of up to 64 rows and 12345
// keys: 182 us, 3.6 TB/s, two rounds of segments of 1.7 us a key tile and 16 us for
// both ends; a tree of 64 rows over 32768 keys 48 us, 10 of them the merge.
#pragma once

#include <cooperative_groups.h>
#include <math.h>

#include "mma_sync.cuh"
#include "paged_tc.cuh"

namespace dfl {

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxTiles = (1 << 20) / kPtKeys;
constexpr int kBitWords = kMaxTiles / 32 + 1;
constexpr float kLazy = 8.f;

template <int HDP, int QT>
struct TcShape {
  static constexpr int kHalves = HDP / 64;
  static constexpr int kTileB = kPtKeys * HDP * 2;      // a Q, K or V tile
  static constexpr int kHalfB = kPtKeys * 128;
  // K and V tiles take turns; an even number, so that a stage always holds the
  // same of the two and who waits for one kind only sees every phase of its
  // barriers. At most 8: see v_ok.
  static constexpr int kStages = HDP == 64 ? 8 : 4;
  static constexpr int kSoft = QT * 128;                // softmax threads
  static constexpr int kThreads = kSoft + 128;
  static constexpr int kQ = 0, kKV = QT * kTileB, kEnd = kKV + kStages * kTileB;
  static constexpr size_t kSmem = kEnd + 1024;
};

// EXTRA: a cap or a distance bias (their code would cost the others registers).
// MANY: with two query tiles, a batch of several sequences, some of few rows
// perhaps (their code costs a call of 300 rows over 2000 keys 1 us of 26).
// TREE: of the sequence's new rows a query sees itself and those it descends from.
template <int HDP, int QT, bool EXTRA, bool MANY, bool TREE>
__global__ void __launch_bounds__(QT * 128 + 128, 1)
paged_attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mq32,
                     const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const __grid_constant__ PagedAttnArgs a) {
  using C = TcShape<HDP, QT>;
  constexpr int NS = C::kStages;
  constexpr int kClusterLd = HDP + 4;                   // row stride of O in shared memory: rows a bank quad apart
  static_assert(QT * 128 * kClusterLd * 4 <= C::kEnd, "O over the Q, K and V tiles");
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t q_full, o_final, kv_full[NS], kv_empty[NS], v_ok[4], s_full[2], p_ready[2], o_done;
  __shared__ uint32_t tmem_holder;
  __shared__ float2 s_ml[QT * 128];                     // a row's maximum and sum, for the cluster
  __shared__ unsigned some[kBitWords], all[kBitWords];
  __shared__ unsigned bad[4][4];                        // of V tile i: [i & 3]
  __shared__ __align__(16) int kpos[QT * 4][kPtKeys];    // a warp's key positions, and
  __shared__ __align__(16) float kdist[EXTRA ? QT * 4 : 1][kPtKeys];   // their distances from wmin
  __shared__ __align__(16) int ktree[TREE ? QT * 4 : 1][kPtKeys];      // and the sizes of their subtrees

  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Segments come in one row of CTAs, all heads of one after the other: those that a
  // batch does not need are the last to start, when the others have their SMs.
  const bool segments = TREE && a.target > 0;
  const int h = segments ? blockIdx.x % c.nkv : blockIdx.y, bx = segments ? blockIdx.x / c.nkv : blockIdx.x, G = a.G;
  int z = blockIdx.z, splits = a.splits;
  const int tpt = kPtKeys / G;                          // new rows of a tile
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023) & ~1023u) - raw);
  constexpr int wLoad = QT * 4, wMma = QT * 4 + 1;

  if (threadIdx.x == wLoad * 32) {
    mbar_init(&q_full, 1);
    mbar_init(&o_final, 1);
    mbar_init(&o_done, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    // four: at most NS / 2 tiles of V are in the ring
    for (int i = 0; i < 4; ++i) mbar_init(&v_ok[i], 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 128);
    }
    fence_mbar_init();
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  // Query rows that no load fills are zeros, so that nothing depends on what was there:
  // those past a tile's tokens, and past a quarter's of a tile that is there 2 or 4 times.
  auto clear_q = [&](bool tile, bool quarters) {
    for (int e = threadIdx.x; e < QT * C::kHalves * kPtKeys; e += C::kThreads) {
      const int r = e & (kPtKeys - 1);
      if (!(tile && r >= tpt * G) && !(quarters && G <= 32 && (r & 31) >= 32 / G * G)) continue;
#pragma unroll
      for (int d = 0; d < 8; ++d) *reinterpret_cast<uint4*>(sm + C::kQ + (e >> 7) * C::kHalfB + r * 128 + d * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_shared();
  };
  // (a quarter's last rows are a whole tile's tokens where the group does not divide 32:
  // the load of Q overwrites these zeros, behind a barrier of the CTA)
  if (!segments) clear_q(true, QT == 1);
  pdl_wait();
  // every warp looks for the tile itself: no one waits for another's answer
  PagedTile t;
  if (segments) {                                        // z of the tile's `splits` segments is this CTA's
    const PagedSegment g = paged_find_segment(c, a.start, a.rows, 1, QT * tpt, kPtKeys, a.window, a.target, bx);
    t = g.t;
    z = g.z;
    splits = g.n;
  } else {
    t = paged_find_tile(a.start, c.n_seq, a.rows, 1, QT * tpt, bx);
  }
  if (segments && t.seq < 0) return;                     // one more than the batch needs
  // TMEM only once the kernel before has given its own back, and the next
  // kernel only once every CTA of this one has its share: neither can then
  // wait for columns that the other holds while it waits
  if (warp == wMma) {
    tmem_alloc(&tmem_holder, 512);
    pdl_launch_dependents();
  }
  int qmin = INT32_MAX, qmax = INT32_MIN, len = 0;
  PagedMask m{};
  if (t.seq >= 0) {
    len = paged_length(c, t.seq);
    m = paged_mask(a.causal, a.window, a.prefix, t.seq);
    const int r0 = t.tile * QT * tpt, r1 = min(t.count, r0 + QT * tpt);
    for (int i = r0 + lane; i < r1; i += 32) {
      const int p = a.q_pos[t.first + i];
      qmin = min(qmin, p);
      qmax = max(qmax, p);
    }
    qmin = __reduce_min_sync(0xffffffffu, qmin);
    qmax = __reduce_max_sync(0xffffffffu, qmax);
  }
  PagedShare sh = paged_range((len + kPtKeys - 1) / kPtKeys, a.window, z, splits);
  // One query tile without a window sees nearly every row there is: no
  // classification beforehand, the warps that need to know look at a tile's
  // positions, which they request a tile ahead.
  // (Not so for trees: with K and V streaming in, a load takes longer than a tile. 19
  // sequences of 64 rows over 8192 keys: 225 us looked at on the way, 146 us classified.)
  const bool direct = paged_direct(sh) || (QT == 1 && !TREE && !sh.by_share);
  const int row0 = t.tile * QT * tpt;                    // the CTA's first new row, within the sequence
  const int nt = (QT == 2 && row0 + tpt < t.count) ? 2 : 1;
  // With one query tile of at most 64 (32) rows, its rows are there 2 (4) times,
  // in quarters of 32 lanes, and a warp takes a half (a quarter) of the keys.
  const int t32 = 32 / G, n_tok = min(tpt, t.count - row0);
  const int rep = QT == 2 || n_tok > 2 * t32 ? 1 : (n_tok > t32 ? 2 : 4);
  // (a segment's Q may be loaded before the CTA's next barrier: only rows that this load leaves out)
  if (segments) clear_q(rep == 1, rep > 1);
  auto load_q = [&]() {
    if (rep == 1) {
      mbar_expect_tx(&q_full, nt * C::kHalves * tpt * G * 128);
      for (int i = 0; i < nt; ++i)
        for (int x = 0; x < C::kHalves; ++x)
          tma_load_3d(sm + C::kQ + i * C::kTileB + x * C::kHalfB, &mq, x * 64, h * G, t.first + row0 + i * tpt, &q_full);
    } else {
      mbar_expect_tx(&q_full, 4 * C::kHalves * t32 * G * 128);
      for (int i = 0; i < 4; ++i)
        for (int x = 0; x < C::kHalves; ++x)
          tma_load_3d(sm + C::kQ + x * C::kHalfB + i * 32 * 128, &mq32, x * 64, h * G, t.first + row0 + (i & (4 / rep - 1)) * t32, &q_full);
    }
  };
  const int box = min(1 << c.lg_rows, kPtKeys), boxes = kPtKeys / box;   // of a tile's loads, a lane to each
  auto row_of = [&](int rel) {
    const int slot = (sh.t0 + rel) * kPtKeys + lane * box;
    int y = (c.n_pages * c.nkv) << c.lg_rows;            // a row past the pool reads as zeros
    if (lane < boxes && slot < len) {
      const long long row = paged_row(c, t.seq, h, slot);
      if (row >= 0) y = (int)row;
      else if (c.status) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
    }
    return y;
  };
  auto load_kv = [&](int kv, int s, int y) {
    if (lane == 0) mbar_expect_tx(&kv_full[s], C::kTileB);
    __syncwarp();
    if (lane < boxes)
#pragma unroll
      for (int x = 0; x < C::kHalves; ++x)
        tma_load_2d(sm + C::kKV + s * C::kTileB + x * C::kHalfB + lane * box * 128, kv ? &mv : &mk, x * 64, y, &kv_full[s]);
  };
  // A segment's first tile is on its way while the tiles are classified; it is taken
  // whether it is seen or not.
  const bool early = segments && !direct && !sh.by_share && sh.t1 > sh.t0;
  if (early && warp == wLoad) {
    if (lane == 0) load_q();
    const int y = row_of(0);
    load_kv(0, 0, y);
    load_kv(1, 1, y);
    __syncwarp();
  }
  if (direct) {
    for (int i = threadIdx.x; i <= sh.take >> 5; i += C::kThreads) {
      const int left = sh.take - i * 32;
      some[i] = left >= 32 ? 0xffffffffu : (1u << left) - 1;
      all[i] = 0u;
    }
  } else {
    paged_classify<kPtKeys>(c, t.seq, h, len, m, qmin, qmax, sh.t0, sh.t1, some, all);
    if (early && threadIdx.x == 0) atomicOr(&some[0], 1u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  if (t.seq < 0) {
    __syncthreads();
    if (warp == wMma) tmem_dealloc(tmem, 512);
    return;
  }
  paged_take(sh, some, z, splits);
  const int N = sh.take;                                 // tiles this CTA works on
  PagedCursor cur(some, sh);
  bool ok = true;
  const bool parts = segments && splits > 1 && rep == 1; // a segment's partials, which leave by way of shared memory
  const bool joins = a.cluster || rep > 1 || parts;      // the output comes out of shared memory
  // Where the partial of (token in this CTA's tiles, head of the group) goes. Of segments
  // the merge hears where its sequence's start.
  const size_t part0 = segments ? ((size_t)bx * c.nkv + h) * (QT * kPtKeys) : (size_t)z * a.rows * a.nq;
  auto partial = [&](int token, int g) {
    return segments ? part0 + token * G + g : part0 + (size_t)(t.first + row0 + token) * a.nq + h * G + g;
  };
  if (segments && h == 0 && z == 0)
    for (int i = threadIdx.x; i < min(QT * tpt, t.count - row0); i += C::kThreads) a.segment[t.first + row0 + i] = make_int4(bx - t.tile * splits, splits, row0 + i, 0);
  // P in two parts, the second `low` columns on
  const bool two_parts = QT == 2 ? MANY && nt == 1 && n_tok <= 2 * t32 : rep > 1;
  constexpr int low = QT == 2 ? 128 : 64;

  // The page of a lane's four keys of a tile (-1: none) and their positions; a
  // page is requested two tiles ahead and positions one, so that neither load
  // waits for the other.
  auto page_of = [&](int rel) {
    const int slot = (sh.t0 + rel) * kPtKeys + lane * 4;
    return rel >= 0 && slot < len ? c.table[(size_t)t.seq * c.max_pages + (slot >> c.lg_rows)] : -1;
  };
  auto positions = [&](int rel, int page) {
    int4 p = make_int4(kPagedNoPos, kPagedNoPos, kPagedNoPos, kPagedNoPos);
    const int slot = (sh.t0 + rel) * kPtKeys + lane * 4;
    if (rel >= 0 && (unsigned)page < (unsigned)c.n_pages) {
      p = *reinterpret_cast<const int4*>(c.pos + ((((long long)page * c.nkv + h) << c.lg_rows) + (slot & ((1 << c.lg_rows) - 1))));
      if (slot + 1 >= len) p.y = kPagedNoPos;
      if (slot + 2 >= len) p.z = kPagedNoPos;
      if (slot + 3 >= len) p.w = kPagedNoPos;
    }
    return p;
  };
  struct Span { int lo, hi; bool whole; };
  auto span = [&](const int4& p) {
    const bool there = p.x != kPagedNoPos && p.y != kPagedNoPos && p.z != kPagedNoPos && p.w != kPagedNoPos;
    return Span{__reduce_min_sync(0xffffffffu, min(min(p.x, p.y), min(p.z, p.w))),
                __reduce_max_sync(0xffffffffu, max(max(p.x, p.y), max(p.z, p.w))), __all_sync(0xffffffffu, there) != 0};
  };
  // the first of the cached rows that are the tree, and whether a tile has some
  const int base = len - t.count;
  auto in_tree = [&](int rel) { return TREE && (sh.t0 + rel + 1) * kPtKeys > base; };
  auto classified = [&](int rel) { return !direct && !in_tree(rel) && ((all[rel >> 5] >> (rel & 31)) & 1u); };

  if (warp == wLoad) {
    // ---- loads: Q, then K and V of every tile, a box per page (or per 128 rows of one)
    if (N > 0 && lane == 0 && !early) load_q();
    int issued = 0;
    for (int i = 0; i < N && ok; ++i) {
      const int rel = cur.next();
      if (i == 0 && early) {
        issued = 2;
        continue;
      }
      const int y = row_of(rel);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int n = 2 * i + kv, s = n % NS;
        if (n >= NS) paged_wait(&kv_empty[s], (n / NS - 1) & 1, ok);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;                                    // the stage is not free: no further load
          break;
        }
        issued = n + 1;
        load_kv(kv, s, y);
      }
    }
    // no copy may be in flight when the CTA ends, whatever became of the others
    bool landed = true;
    if (N > 0) paged_wait(&q_full, 0, landed);
    for (int n = issued > NS ? issued - NS : 0; n < issued; ++n) paged_wait(&kv_full[n % NS], (n / NS) & 1, landed);
    ok = ok && landed;
  } else if (warp == wMma) {
    // ---- MMAs, all from one lane, so that they run in the order issued; the
    // warp stays together, so that descriptors live in uniform registers
    if (N > 0) {
      const bool leader = elect_one();
      const uint32_t sb = smem_u32(sm);
      const int ksteps = (c.hd + 15) >> 4;
      const uint32_t idesc_o = idesc_bf16(128, ksteps * 16) | kIdescBMnMajor;
      const uint64_t q_desc = smem_desc_sw128(sb + C::kQ), k_desc = smem_desc_sw128(sb + C::kKV);
      const uint64_t v_desc = smem_desc_sw128_mn(sb + C::kKV, C::kHalfB);
      // scores of query tile q against key tile i into buffer buf; the last
      // use of K frees its stage
      auto qk = [&](int q, int buf, int i, bool last) {
        const int s = (2 * i) % NS;
        if (leader) {
          tc_scores<C::kHalves>(tmem + buf * 128, q_desc + q * (C::kTileB >> 4), k_desc + s * (C::kTileB >> 4), ksteps);
          tc_commit(&s_full[buf]);
          if (last) tc_commit(&kv_empty[s]);
        }
        __syncwarp();
      };
      // the second part of P
      auto low_pv = [&](int buf, uint64_t v) {
#pragma unroll
        for (int k = 0; k < 8; ++k) tc_mma_bf16_ta(tmem + 256, tmem + buf * 128 + low + k * 8, v + k * (2048 >> 4), idesc_o, 1u);
      };
      auto pv = [&](int q, int buf, int i, bool last) {
        const int s = (2 * i + 1) % NS;
        if (leader) {
          const uint64_t v = v_desc + s * (C::kTileB >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k) tc_mma_bf16_ta(tmem + 256 + q * HDP, tmem + buf * 128 + k * 8, v + k * (2048 >> 4), idesc_o, 1u);
          if (QT == 1 && rep > 1) low_pv(buf, v);
          if (QT == 1) tc_commit(&o_done);
          if (last) tc_commit(&kv_empty[s]);
        }
        __syncwarp();
      };
      auto wait_k = [&](int i) { paged_wait(&kv_full[(2 * i) % NS], (2 * i / NS) & 1, ok); };
      auto wait_v = [&](int i) { paged_wait(&v_ok[i & 3], (i >> 2) & 1, ok); };
      paged_wait(&q_full, 0, ok);
      wait_k(0);
      qk(0, 0, 0, QT == 1 || nt == 1);
      if (QT == 2 && MANY && two_parts) {
        for (int i = 0; i < N; ++i) {
          wait_v(i);
          paged_wait(&p_ready[0], i & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc_fence_after();
          const int s = (2 * i + 1) % NS;
          pv(0, 0, i, false);
          if (i + 1 < N) {
            wait_k(i + 1);
            qk(0, 0, i + 1, true);
          }
          if (leader) {                                  // beside the next tile's softmax
            low_pv(0, v_desc + s * (C::kTileB >> 4));
            tc_commit(&o_done);
            tc_commit(&kv_empty[s]);
          }
          __syncwarp();
        }
      } else if (QT == 2) {
        if (nt == 2) qk(1, 1, 0, true);
        for (int i = 0; i < N; ++i) {
          const bool more = i + 1 < N;
          wait_v(i);
          paged_wait(&p_ready[0], i & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc_fence_after();
          pv(0, 0, i, nt == 1);
          if (more) {
            wait_k(i + 1);
            qk(0, 0, i + 1, nt == 1);
          }
          if (nt == 2) {
            paged_wait(&p_ready[1], i & 1, ok);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
            pv(1, 1, i, true);
            if (more) qk(1, 1, i + 1, true);
          }
        }
      } else {
        if (N > 1) {
          wait_k(1);
          qk(0, 1, 1, true);
        }
        for (int i = 0; i < N; ++i) {
          wait_v(i);
          paged_wait(&p_ready[i & 1], (i >> 1) & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc_fence_after();
          pv(0, i & 1, i, true);
          if (i + 2 < N) {
            wait_k(i + 2);
            qk(0, i & 1, i + 2, true);
          }
        }
      }
      if (leader) tc_commit(&o_final);
      __syncwarp();
      bool done = true;
      paged_wait(&o_final, 0, done);
      ok = ok && done;
    }
  } else if (warp > wMma) {
    // ---- V's non-finite rows, in tiles that some query sees only in part
    const int half = warp - wMma - 1;
    if (half == 0 && lane == 0 && h == 0 && z == 0 && t.tile == 0) {
      paged_report_length(c, t.seq, len);
      if (TREE && base < 0 && c.status) atomicOr(c.status, DFLASH_PAGED_BAD_ROWS);
    }
    const bool look = QT == 1 && direct;
    int rel = cur.next(), rel1 = cur.next(), page1 = -1;
    int4 pos4 = make_int4(0, 0, 0, 0);
    if (look) {
      const int page = page_of(rel);
      page1 = page_of(rel1);
      pos4 = positions(rel, page);
    }
    for (int i = 0; i < N; ++i) {
      const int n = 2 * i + 1, s = n % NS;
      bool full = classified(rel);
      if (look) {
        const Span k = span(pos4);
        full = k.whole && paged_class(m, qmin, qmax, k.lo, k.hi, true) == 2 && !in_tree(rel);
        pos4 = positions(rel1, page1);
      }
      rel = rel1;
      rel1 = cur.next();
      if (look) page1 = page_of(rel1);
      paged_wait(&kv_full[s], (n / NS) & 1, ok);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (!full) {
        uint8_t* v = sm + C::kKV + s * C::kTileB;
        for (int x = 0; x < 2; ++x) {
          const int r = half * 64 + x * 32 + lane;
          unsigned acc = 0;
#pragma unroll
          for (int y = 0; y < C::kHalves; ++y)
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              const uint4 u = *reinterpret_cast<const uint4*>(v + y * C::kHalfB + r * 128 + ((d ^ (r & 7)) << 4));
              // an exponent of all ones carries into the sign's place
              acc |= ((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
                     ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u);
            }
          const bool is_bad = (acc & 0x80008000u) != 0;
          const unsigned who = __ballot_sync(0xffffffffu, is_bad);
          if (lane == 0) bad[i & 3][half * 2 + x] = who;
          if (is_bad)
            for (int y = 0; y < C::kHalves; ++y)
              for (int d = 0; d < 8; ++d) *reinterpret_cast<uint4*>(v + y * C::kHalfB + r * 128 + (d << 4)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_shared();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&v_ok[i & 3]);
    }
  } else if (QT == 1 || (warp >> 2) < nt) {
    // ---- softmax: one query row to a thread
    const int q = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const int distinct = 4 / rep;                        // quarters of different rows
    const int lr = rep > 1 ? lane : r;
    const int tl = lr / G + (rep > 1 ? (quad & (distinct - 1)) * t32 : 0), g = lr % G, head = h * G + g;
    const int at_row = row0 + q * tpt + tl;
    const bool valid = (rep > 1 ? lane < t32 * G : tl < tpt) && at_row < t.count;
    const int n0 = rep > 1 ? quad / distinct * distinct : 0, n1 = rep > 1 ? n0 + distinct : 4;   // its chunks of 32 keys
    const int tok = t.first + (valid ? at_row : row0);
    const bool work = __any_sync(0xffffffffu, valid);
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_at = tmem + lanes + 256 + q * HDP;
    const int pq = a.q_pos[tok];
    const PagedSees sees = paged_sees_of(m, pq);
    const int wmin = __reduce_min_sync(0xffffffffu, valid ? pq : INT32_MAX), wmax = __reduce_max_sync(0xffffffffu, valid ? pq : INT32_MIN);
    const float slope2 = a.slopes ? a.slopes[valid ? head : h * G] * kLog2e : 0.f;
    const float scale2 = a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e;
    CapPoly cap = cap_poly(scale2, a.softcap * kLog2e);
    // (rows of the next sequence, which a load brings along, have no say in how
    // the warp's caps are computed)
    if (!valid) cap.limit = INFINITY;
    int* kp = kpos[warp];
    // A distance is the difference of two distances from the warp's first
    // query, converted once a key and not once a score (a conversion takes the
    // pipe of the exponentials); exact while the warp's queries are near each
    // other, otherwise taken from the integers.
    float* kd = kdist[EXTRA ? warp : 0];
    int* kt = ktree[TREE ? warp : 0];
    const bool near = (long long)wmax - wmin < (1 << 23);
    const float pqf = (float)(pq - wmin);
    float mx = -INFINITY, sum = 0.f;

    // positions of the tile's keys, four to a lane, loaded a tile ahead where
    // they will be needed
    int rel = cur.next(), rel1 = cur.next(), page1 = page_of(rel1);
    int4 pos4 = positions(rel, page_of(rel));
    auto advance = [&]() {
      rel = rel1;
      if (rel >= 0 && ((EXTRA && a.slopes) || !classified(rel))) pos4 = positions(rel, page1);
      rel1 = cur.next();
      page1 = page_of(rel1);
    };
    if (N > 0 && work) {
      const uint32_t zero[32] = {};
#pragma unroll
      for (int d = 0; d < HDP; d += 32) tmem_st32(o_at + d, zero);
      tmem_st_wait();
    }
    // The two-tile kernel's few rows have a loop of their own: their branch within
    // that of all others costs a prompt 3% (2048 rows over 32768 keys: 820 us, with
    // it 843 us; under a cap of 20: 1465 us, with it 1648 us).
#pragma unroll
    for (int few = 0; few < (QT == 2 && MANY ? 2 : 1); ++few) {
      const bool two = QT == 2 ? few == 1 : two_parts;
      if (two != two_parts) continue;
      for (int i = 0; i < N; ++i) {
        const int buf = QT == 2 ? q : (i & 1);
        const uint32_t s_at = tmem + lanes + buf * 128;
        paged_wait(&s_full[buf], QT == 2 ? (i & 1) : ((i >> 1) & 1), ok);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (!work) {                                       // rows of nobody: their P may be anything
          mbar_arrive(&p_ready[buf]);
          continue;
        }
        bool full = classified(rel);
        const int tile = sh.t0 + rel;
        // First pass over S: the row's maximum. What a mask or bias makes of a score
        // is put back in its place, so that the second pass is the same for all; S
        // is read twice because half as many registers then do. A cap alone keeps
        // the order of scores: the maximum's is enough here, and the second pass
        // caps the others.
        // (a tile that other warps see in part, or that was not classified, may be
        // wholly seen by this warp's rows)
        bool masked = !full;
        if (masked) {
          const Span k = span(pos4);
          masked = !k.whole || paged_class(m, wmin, wmax, k.lo, k.hi, true) != 2 || in_tree(rel);
          if (QT == 1 && direct) full = k.whole && paged_class(m, qmin, qmax, k.lo, k.hi, true) == 2 && !in_tree(rel);
        }
        const bool late = EXTRA && a.softcap > 0.f && !masked && !a.slopes;
        const bool change = masked || (EXTRA && a.slopes);
        if (masked || (EXTRA && a.slopes)) {
          __syncwarp();
          *reinterpret_cast<int4*>(kp + lane * 4) = pos4;
          if (EXTRA && a.slopes)
            *reinterpret_cast<float4*>(kd + lane * 4) =
                make_float4((float)(pos4.x - wmin), (float)(pos4.y - wmin), (float)(pos4.z - wmin), (float)(pos4.w - wmin));
          if (TREE) {
            const int node = tile * kPtKeys + lane * 4 - base;
            const int* ends = a.tree + t.first;
            *reinterpret_cast<int4*>(kt + lane * 4) = make_int4(paged_tree_size(ends, t.count, node), paged_tree_size(ends, t.count, node + 1),
                                                                paged_tree_size(ends, t.count, node + 2), paged_tree_size(ends, t.count, node + 3));
          }
          __syncwarp();
        }
        // the query's distance from the tile's first row, in rows
        const int from = at_row + base - tile * kPtKeys;
        auto visible = [&](int j, int pk, int size) { return paged_sees(sees, pk) && (!TREE || (unsigned)(from - j) < (unsigned)size); };
        float x[2][32], top = -INFINITY;
        auto rise = [&](const float* v) {
          float t2[2] = {v[0], v[1]};
#pragma unroll
          for (int j = 2; j < 32; j += 4) {
            t2[0] = j + 2 < 32 ? fmaxf(fmaxf(t2[0], v[j]), v[j + 2]) : fmaxf(t2[0], v[j]);
            t2[1] = j + 3 < 32 ? fmaxf(fmaxf(t2[1], v[j + 1]), v[j + 3]) : fmaxf(t2[1], v[j + 1]);
          }
          top = fmaxf(top, fmaxf(t2[0], t2[1]));
        };
        if (QT == 2 && !change) {
          tmem_ld32(s_at, x[0]);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            tmem_ld_wait32(x[n & 1]);
            if (n < 3) tmem_ld32(s_at + (n + 1) * 32, x[(n + 1) & 1]);
            rise(x[n & 1]);
          }
        } else if (!change) {
#pragma unroll 1
          for (int n = n0; n < n1; ++n) {
            tmem_ld32(s_at + n * 32, x[0]);
            tmem_ld_wait32(x[0]);
            rise(x[0]);
          }
        } else {
#pragma unroll 1
          for (int n = n0; n < n1; ++n) {
            float* v = x[0];
            uint32_t w[32];
            const int4* pk4 = reinterpret_cast<const int4*>(kp + n * 32);
            tmem_ld32(s_at + n * 32, v);
            tmem_ld_wait32(v);
            if (EXTRA && a.softcap > 0.f) {
              cap_tanh32(v, cap, masked, [&]() {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = visible(n * 32 + j, kp[n * 32 + j], TREE ? kt[n * 32 + j] : 0) ? v[j] : 0.f;
              });
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= scale2;
            }
            if (EXTRA && a.slopes && near) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 k = *reinterpret_cast<const float4*>(kd + n * 32 + j);
                v[j] = fmaf(-slope2, fabsf(pqf - k.x), v[j]);
                v[j + 1] = fmaf(-slope2, fabsf(pqf - k.y), v[j + 1]);
                v[j + 2] = fmaf(-slope2, fabsf(pqf - k.z), v[j + 2]);
                v[j + 3] = fmaf(-slope2, fabsf(pqf - k.w), v[j + 3]);
              }
            } else if (EXTRA && a.slopes) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = fmaf(-slope2, fabsf((float)(pq - kp[n * 32 + j])), v[j]);
            }
            if (masked) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const int4 k = pk4[j >> 2], e = TREE ? reinterpret_cast<const int4*>(kt + n * 32)[j >> 2] : make_int4(0, 0, 0, 0);
                v[j] = visible(n * 32 + j, k.x, e.x) ? v[j] : -INFINITY;
                v[j + 1] = visible(n * 32 + j + 1, k.y, e.y) ? v[j + 1] : -INFINITY;
                v[j + 2] = visible(n * 32 + j + 2, k.z, e.z) ? v[j + 2] : -INFINITY;
                v[j + 3] = visible(n * 32 + j + 3, k.w, e.w) ? v[j + 3] : -INFINITY;
              }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j]);
            tmem_st32(s_at + n * 32, w);
            rise(v);
          }
        }
        const float sc = change || late ? 1.f : scale2;
        top = EXTRA && late ? cap_tanh1(top, cap) : top * sc;
        if (change) tmem_st_wait();
        if (QT == 2 && two && i > 0) {
          // O and the second part of P are still in use by the last tile's product
          paged_wait(&o_done, (i - 1) & 1, ok);
          tc_fence_after();
        }
        // (rows of the next sequence, which a load brings along, have no say in it)
        if (!valid) top = -INFINITY;
        if (__any_sync(0xffffffffu, top > mx + kLazy)) {
          const float mn = fmaxf(mx, top);
          const float f = mn == -INFINITY ? 1.f : ex2(mx - mn);
          sum *= f;
          mx = mn;
          if (i > 0) {
            // O holds the tiles before this one: their P V is done (with two
            // query tiles because S of this tile was issued after it)
            if (QT == 1) {
              paged_wait(&o_done, (i - 1) & 1, ok);
              tc_fence_after();
            }
#pragma unroll
            for (int d = 0; d < HDP; d += 16) {
              float o[16];
              tmem_ld16(o_at + d, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= f;
              tmem_st16(o_at + d, o);
            }
            tmem_st_wait();
          }
        }
        const float base = mx == -INFINITY ? 0.f : mx;
        const uint64_t sc2 = pack2(sc, sc), nb2 = pack2(-base, -base);
        uint64_t add[2] = {0, 0};
        // two values' p, and the bf16 pair that they are stored as
        auto weigh = [&](const float* v, float& p0, float& p1) {
          unpack2(fma2(pack2(v[0], v[1]), sc2, nb2), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          return pack_bf16(p0, p1);
        };
        // what a stored pair leaves of them
        auto rest = [&](uint32_t hi, float p0, float p1) { return __uint_as_float(pack_bf16(p0 - bf_lo(hi), p1 - bf_hi(hi))); };
        if (QT == 2 && EXTRA && late) {
#pragma unroll 1
          for (int n = 0; n < 4; ++n) {
            float w[16], lo[16];
            tmem_ld32(s_at + n * 32, x[0]);
            tmem_ld_wait32(x[0]);
            cap_tanh32(x[0], cap, false, []() {});
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float p0, p1;
              const uint32_t hi = weigh(x[0] + j, p0, p1);
              w[j >> 1] = __uint_as_float(hi);
              if (two) lo[j >> 1] = rest(hi, p0, p1);
              add[(j >> 1) & 1] = add2(add[(j >> 1) & 1], pack2(p0, p1));
            }
            tmem_st16(s_at + n * 16, w);
            if (two) tmem_st16(s_at + low + n * 16, lo);
          }
        } else if (QT == 2) {
          tmem_ld32(s_at, x[0]);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            float* v = x[n & 1];
            tmem_ld_wait32(v);
            if (n < 3) tmem_ld32(s_at + (n + 1) * 32, x[(n + 1) & 1]);
            float w[16], lo[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float p0, p1;
              const uint32_t hi = weigh(v + j, p0, p1);
              w[j >> 1] = __uint_as_float(hi);
              if (two) lo[j >> 1] = rest(hi, p0, p1);
              add[(j >> 1) & 1] = add2(add[(j >> 1) & 1], pack2(p0, p1));
            }
            tmem_st16(s_at + n * 16, w);                   // columns whose scores have been read
            if (two) tmem_st16(s_at + low + n * 16, lo);
          }
        } else {
          // P's first part goes into columns 0 .. 63, its second into 64 .. 127; in
          // this order no chunk's parts fall on scores of the warp not yet read
          const bool down = rep == 2 && n0 == 2;
#pragma unroll 1
          for (int k = n0; k < n1; ++k) {
            const int n = down ? n0 + n1 - 1 - k : k;
            if (rep < 4) {
              tmem_ld32(s_at + n * 32, x[0]);
              tmem_ld_wait32(x[0]);
            }
            if (EXTRA && late) cap_tanh32(x[0], cap, false, []() {});
            float w[16], lo[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float p0, p1;
              const uint32_t hi = weigh(x[0] + j, p0, p1);
              add[(j >> 1) & 1] = add2(add[(j >> 1) & 1], pack2(p0, p1));
              w[j >> 1] = __uint_as_float(hi);
              lo[j >> 1] = rest(hi, p0, p1);
            }
            tmem_st16(s_at + n * 16, w);
            if (two) tmem_st16(s_at + low + n * 16, lo);
          }
          if (rep > 1) {
            // the other warps' keys have no weight in these lanes
            const float zero[16] = {};
#pragma unroll 1
            for (int n = 0; n < 4; ++n) {
              if (n >= n0 && n < n1) continue;
              tmem_st16(s_at + n * 16, zero);
              tmem_st16(s_at + low + n * 16, zero);
            }
          }
        }
        float a0, a1;
        unpack2(add2(add[0], add[1]), a0, a1);
        sum += a0 + a1;
        tmem_st_wait();
        if (!full) {
          const unsigned* who = bad[i & 3];
          paged_wait(&v_ok[i & 3], (i >> 2) & 1, ok);
          const unsigned any = who[0] | who[1] | who[2] | who[3];
          if (any && QT == 1 && i > 0) {
            paged_wait(&o_done, (i - 1) & 1, ok);
            tc_fence_after();
          }
          for (int w = 0; any && w < 4; ++w)
            for (unsigned b = who[w]; b; b &= b - 1) {
              const int j = w * 32 + __ffs(b) - 1, slot = tile * kPtKeys + j;
              if (slot >= len) continue;
              const uint32_t ph = tmem_ld1(s_at + (j >> 1)), pl = two ? tmem_ld1(s_at + low + (j >> 1)) : 0u;
              tmem_ld_wait();
              const float p = j & 1 ? bf_hi(ph) + bf_hi(pl) : bf_lo(ph) + bf_lo(pl);
              const long long row = paged_row(c, t.seq, h, slot);
              if (row < 0) continue;
              // one of this row's keys, and seen by it (its weight may have left fp32)
              const bool mine = w >= n0 && w < n1 && visible(j, c.pos[row], TREE && masked ? kt[j] : INT32_MAX);
              if (!__any_sync(0xffffffffu, mine)) continue;
              const bf16* vrow = static_cast<const bf16*>(c.v) + row * c.hd;
              for (int d = 0; d < HDP; d += 16) {
                float o[16];
                tmem_ld16(o_at + d, o);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const float v = d + x < c.hd ? to_f(vrow[d + x]) : 0.f;
                  if (mine) o[x] = fmaf(p, v, o[x]);
                }
                tmem_st16(o_at + d, o);
              }
              tmem_st_wait();
            }
        }
        tc_fence_before();
        mbar_arrive(&p_ready[buf]);
        advance();
      }
    }
    // ---- the row's output, or its split's partial (to shared memory for the
    // cluster, else to the workspace)
    if (N > 0) {
      paged_wait(&o_final, 0, ok);
      tc_fence_after();
    }
    const size_t at = (size_t)tok * a.nq + head;
    const bool none = sum == 0.f;                        // nothing seen (a NaN score makes the sum NaN)
    const float inv = none ? 0.f : 1.f / sum;
    if (joins) {
      // every copy into this memory has landed and been used by an MMA that is done
      fence_proxy_async_shared();
      s_ml[q * 128 + r] = make_float2(mx, valid ? sum : 0.f);
    }
    if (work) {
#pragma unroll
      for (int d = 0; d < HDP; d += 32) {
        float o[32];
        if (N > 0) {
          tmem_ld32(o_at + d, o);
          tmem_ld_wait32(o);
        }
        if (!valid) continue;
        if (joins || splits > 1) {
          float* po = joins ? reinterpret_cast<float*>(sm) + (q * 128 + r) * kClusterLd + d : a.part_o + partial(q * tpt + tl, g) * c.hd + d;
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            if (d + x < c.hd && !none) *reinterpret_cast<float4*>(po + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
        } else {
          bf16* out = static_cast<bf16*>(a.out) + at * c.hd + d;
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (!none) {
              uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
              for (int y = 0; y < 4; ++y) w[y] = pack_bf16(o[x + 2 * y] * inv, o[x + 2 * y + 1] * inv);
            }
            if (d + x < c.hd) *reinterpret_cast<uint4*>(out + x) = u;
          }
        }
      }
      if (TREE && parts) fence_proxy_async_shared();     // the row leaves as a bulk copy
      if (valid && !joins) {
        if (splits > 1) a.part_ml[partial(q * tpt + tl, g)] = make_float2(mx, sum);
        else if (a.lse) a.lse[at] = none ? -INFINITY : (mx + log2f(sum)) * kLn2;
      }
    }
  }
  if (parts) {
    // Row by row as bulk copies: a thread's own stores would be 16 bytes at a time, each in
    // a line of its own (a segment's end: 2 us, with them 8 us).
    __syncthreads();
    for (int R = threadIdx.x; R < nt * 128; R += C::kThreads) {
      const int tl = (R & 127) / G;
      if (tl >= tpt || row0 + (R >> 7) * tpt + tl >= t.count) continue;
      const size_t part = partial((R >> 7) * tpt + tl, (R & 127) % G);
      const float2 ml = s_ml[R];
      a.part_ml[part] = ml;
      if (ml.y != 0.f) bulk_store(a.part_o + part * c.hd, reinterpret_cast<const float*>(sm) + R * kClusterLd, c.hd * 4);
    }
    bulk_store_wait();
  } else if (joins) {
    // The parts of a row, `rep` in each CTA and the CTAs of the cluster where
    // those are the splits, are joined out of shared memory 4 dimensions at a
    // time: o = sum_x o_x exp2(m_x - M) / sum_x l_x exp2(m_x - M).
    cg::cluster_group cl = cg::this_cluster();
    if (a.cluster) cl.sync();
    else __syncthreads();
    const int ctas = a.cluster ? splits : 1, rows = nt * 128 / rep, quads = c.hd >> 2;
    for (int e = (a.cluster ? z : 0) * C::kThreads + (int)threadIdx.x; e < rows * quads; e += ctas * C::kThreads) {
      const int R = e / quads, d = (e - R * quads) * 4, lr = rep > 1 ? R & 31 : R & 127;
      const int tl = lr / G + (rep > 1 ? (R >> 5) * t32 : 0), at_row = row0 + (rep > 1 ? 0 : (R >> 7) * tpt) + tl;
      if ((rep > 1 ? lr >= t32 * G : tl >= tpt) || at_row >= t.count) continue;
      float M = -INFINITY, L = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int y = 0; y < rep; ++y) {
        const int at = R + y * rows;
        float2 ml[kMaxCluster];
        float4 o[kMaxCluster];
        float top = M;
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) {
          ml[x] = make_float2(-INFINITY, 0.f);
          if (x < ctas) {
            const float2* pm = &s_ml[at];
            const float* po = reinterpret_cast<const float*>(sm) + at * kClusterLd + d;
            ml[x] = *(a.cluster ? cl.map_shared_rank(pm, x) : pm);
            o[x] = *reinterpret_cast<const float4*>(a.cluster ? cl.map_shared_rank(po, x) : po);
          }
          top = fmaxf(top, ml[x].x);
        }
        const float base = top == -INFINITY ? 0.f : top, old = ex2(M - base);
        M = top;
        L *= old;
        v.x *= old; v.y *= old; v.z *= old; v.w *= old;
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) {
          if (ml[x].y == 0.f) continue;                  // it saw nothing: its o was not written
          const float f = ex2(ml[x].x - base);
          L = fmaf(ml[x].y, f, L);
          v.x = fmaf(o[x].x, f, v.x);
          v.y = fmaf(o[x].y, f, v.y);
          v.z = fmaf(o[x].z, f, v.z);
          v.w = fmaf(o[x].w, f, v.w);
        }
      }
      const size_t at = (size_t)(t.first + at_row) * a.nq + h * G + lr % G;
      if (splits > 1 && !a.cluster) {
        const size_t part = partial(at_row - row0, lr % G);
        *reinterpret_cast<float4*>(a.part_o + part * c.hd + d) = v;
        if (d == 0) a.part_ml[part] = make_float2(M, L);
        continue;
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + at * c.hd + d) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
      if (d == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
    if (a.cluster) cl.sync();                            // no CTA leaves while another reads it
  }
  if (!ok && c.status) atomicOr(c.status, DFLASH_PAGED_GAVE_UP);
  tc_fence_before();
  __syncthreads();
  if (warp == wMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HDP, int QT, bool TREE>
cudaError_t run(const PagedAttnArgs& a, long long tiles, cudaStream_t st) {
  CUtensorMap mq, mq32, mk, mv;
  if (!paged_map_rows(&mq, a.q, a, kPtKeys / a.G) || !paged_map_rows(&mq32, a.q, a, a.G <= 32 ? 32 / a.G : 1) || !paged_map_pages(&mk, a.c.k, a.c) || !paged_map_pages(&mv, a.c.v, a.c))
    return cudaErrorInvalidValue;
  using C = TcShape<HDP, QT>;
  const bool extra = a.softcap > 0.f || a.slopes;
  auto kernel = extra ? paged_attn_tc_kernel<HDP, QT, true, false, TREE> : paged_attn_tc_kernel<HDP, QT, false, false, TREE>;
  if (QT == 2 && a.c.n_seq > 1) kernel = extra ? paged_attn_tc_kernel<HDP, QT, true, QT == 2, TREE> : paged_attn_tc_kernel<HDP, QT, false, QT == 2, TREE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = a.target ? dim3((unsigned)(tiles * a.c.nkv)) : dim3((unsigned)tiles, a.c.nkv, a.splits);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = a.splits;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, mq, mq32, mk, mv, a);
}

}  // namespace

}  // namespace dfl
