// Key weights on the tensor cores (bf16, head_dim <= 128): for every cached row
// of a (sequence, kv head) the sum over the query rows of exp(t - lse).
//
// S^T = K Q^T: a CTA holds a tile of 128 keys as the A operand and passes the
// query rows by as B, 128 at a time. A key is a TMEM lane, so one thread owns it
// for the whole pass and adds up its row of S^T in registers: no exchange
// between threads, no atomics, and a fixed order. S has two buffers; the
// exponentials of one run while the next is computed, and a second CTA on the SM
// works while this one starts or ends. Many query rows (512 over 32768 keys: 154 us,
// 0.90 PFLOP/s) fill no pipe (issue 41%, special functions 38%, tensor 37%): what
// bounds them is a tile's chain of four dependent TMEM reads and their exponentials.
// Few are bound by a CTA's start and end (16 rows over 6000 keys: 7.5 us in a graph).
// (Two key tiles to a CTA, which would halve the passes over the query rows, and
// one CTA to an SM took 166 us instead of 154 us for 512 rows over 32768 keys.)
#include <math.h>

#include "paged_tc.cuh"

namespace dfl {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kChunk = 8192;               // query tiles classified at a time
constexpr int kBitWords = kChunk / 32 + 1;
constexpr int kNA = 4;                     // rows' lse, position and slope: ring stages

template <int HDP>
struct WtShape {
  static constexpr int kHalves = HDP / 64;
  static constexpr int kTileB = kPtKeys * HDP * 2;
  static constexpr int kHalfB = kPtKeys * 128;
  static constexpr int kStages = 2;
  static constexpr int kThreads = 256;
  static constexpr int kK = 0, kQ = kTileB, kEnd = kQ + kStages * kTileB;
  static constexpr size_t kSmem = kEnd + 1024;
};

// Of the query rows of a tile: minus lse and the slope, in log2 units, and the
// position (kPagedNoPos, seen by nobody, for what adds nothing).
// `base`: the first row's position, and the others' distances from it (see
// the attention kernel), `near` whether all are exact.
struct alignas(16) WtRows { float nlse2[kPtKeys]; float slope2[kPtKeys]; int pos[kPtKeys]; float dist[kPtKeys]; int base, near; };

// EXTRA: a cap or a distance bias.
template <int HDP, bool EXTRA>
__global__ void __launch_bounds__(256, 2)
paged_weight_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ PagedAttnArgs a) {
  using C = WtShape<HDP>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t k_full[2], k_empty[2], q_full[NS], q_empty[NS], rows_full[kNA], rows_empty[kNA], s_full[2], s_empty[2];
  __shared__ uint32_t tmem_holder;
  __shared__ int s_kmin, s_kmax;
  __shared__ unsigned some[kBitWords], all[kBitWords];
  __shared__ __align__(16) WtRows rows[kNA];

  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, seq = blockIdx.z, G = a.G, tpt = kPtKeys / G;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023) & ~1023u) - raw);
  constexpr int wMma = 4, wLoad = 5, wRows = 6;
  constexpr unsigned kTmemCols = 256;

  if (threadIdx.x == wLoad * 32) {
    for (int i = 0; i < 2; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
    for (int i = 0; i < NS; ++i) { mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1); }
    for (int i = 0; i < kNA; ++i) { mbar_init(&rows_full[i], 1); mbar_init(&rows_empty[i], 4); }
    for (int b = 0; b < 2; ++b) { mbar_init(&s_full[b], 1); mbar_init(&s_empty[b], 128); }
    fence_mbar_init();
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
  }
  // query rows of a tile past tpt * G are never loaded: zeros, so that their
  // scores are finite
  for (int e = threadIdx.x; e < NS * C::kHalves * (kPtKeys - tpt * G) * 8; e += C::kThreads) {
    const int left = kPtKeys - tpt * G, x = e / (left * 8), r = tpt * G + e / 8 % left;
    *reinterpret_cast<uint4*>(sm + C::kQ + x * C::kHalfB + r * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_shared();
  pdl_wait();
  // TMEM only once the kernel before has given its own back, and the next
  // kernel only once every CTA of this one has its share: neither can then
  // wait for columns that the other holds while it waits
  if (warp == wMma) {
    tmem_alloc(&tmem_holder, kTmemCols);
    pdl_launch_dependents();
  }
  const int len = paged_length(c, seq);
  const int2 ab = paged_new_rows(a.start, seq, a.rows);
  const int n_new = ab.y - ab.x, tiles = (n_new + tpt - 1) / tpt;
  const PagedMask m = paged_mask(a.causal, a.window, a.prefix, seq);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  bool ok = true;

  // lse, position and slope of the query rows of tile q, four to a lane
  struct RowData { float l[4], sl[4]; int p[4], base, near; bool whole; };
  auto row_data = [&](int q) {
    RowData d;
    bool whole = true;                     // every row has an lse
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = x * 32 + lane, tl = r / G, tok = q * tpt + tl, head = h * G + r - tl * G;
      const bool in = tl < tpt && tok < n_new;
      const float v = in ? a.lse[(size_t)(ab.x + tok) * a.nq + head] : -INFINITY;
      d.l[x] = v == -INFINITY ? -INFINITY : -v * kLog2e;
      d.p[x] = v == -INFINITY ? kPagedNoPos : a.q_pos[ab.x + tok];
      d.sl[x] = in && a.slopes ? a.slopes[head] * kLog2e : 0.f;
      whole = whole && (!in || v != -INFINITY);
    }
    d.whole = __all_sync(0xffffffffu, whole);
    d.base = 0;
    d.near = 1;
    if (EXTRA && a.slopes) {
      int lo = INT32_MAX, hi = INT32_MIN;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        lo = min(lo, d.p[x] == kPagedNoPos ? INT32_MAX : d.p[x]);
        hi = max(hi, d.p[x]);
      }
      d.base = __reduce_min_sync(0xffffffffu, lo);
      d.near = (long long)__reduce_max_sync(0xffffffffu, hi) - d.base < (1 << 23);
    }
    return d;
  };
  auto put_rows = [&](WtRows& to, const RowData& d) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = x * 32 + lane;
      to.nlse2[r] = d.l[x];
      to.pos[r] = d.p[x];
      to.slope2[r] = d.sl[x];
      if (EXTRA && a.slopes) to.dist[r] = (float)(d.p[x] - d.base);
    }
    if (EXTRA && lane == 0) {
      to.base = d.base;
      to.near = d.near;
    }
  };
  // adds the exponentials of 32 query rows (from row n * 32 of `rw`) to two sums
  const float scale2 = a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e;
  CapPoly cap = cap_poly(scale2, a.softcap * kLog2e);
  const float cap_limit = cap.limit;
  auto add_chunk = [&](float* v, const WtRows& rw, int n, const PagedSees& by, int pk, bool full, uint64_t* add) {
    float sc = scale2;
    if (EXTRA && a.softcap > 0.f) {
      cap_tanh32(v, cap, !full, [&]() {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = paged_sees(by, rw.pos[n * 32 + e]) ? v[e] : 0.f;
      });
      sc = 1.f;
    }
    if (EXTRA && a.slopes) {
      if (rw.near) {
        const float pkf = (float)(pk - rw.base);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 pq = *reinterpret_cast<const float4*>(rw.dist + n * 32 + e);
          const float4 sl = *reinterpret_cast<const float4*>(rw.slope2 + n * 32 + e);
          v[e] = fmaf(-sl.x, fabsf(pq.x - pkf), v[e] * sc);
          v[e + 1] = fmaf(-sl.y, fabsf(pq.y - pkf), v[e + 1] * sc);
          v[e + 2] = fmaf(-sl.z, fabsf(pq.z - pkf), v[e + 2] * sc);
          v[e + 3] = fmaf(-sl.w, fabsf(pq.w - pkf), v[e + 3] * sc);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = fmaf(-rw.slope2[n * 32 + e], fabsf((float)(rw.pos[n * 32 + e] - pk)), v[e] * sc);
      }
      sc = 1.f;
    }
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 l = *reinterpret_cast<const float4*>(rw.nlse2 + n * 32 + e);
      const int4 pq = *reinterpret_cast<const int4*>(rw.pos + n * 32 + e);
      const float p0 = ex2(fmaf(v[e], sc, l.x)), p1 = ex2(fmaf(v[e + 1], sc, l.y));
      const float p2 = ex2(fmaf(v[e + 2], sc, l.z)), p3 = ex2(fmaf(v[e + 3], sc, l.w));
      add[0] = add2(add[0], pack2(full || paged_sees(by, pq.x) ? p0 : 0.f, full || paged_sees(by, pq.y) ? p1 : 0.f));
      add[1] = add2(add[1], pack2(full || paged_sees(by, pq.z) ? p2 : 0.f, full || paged_sees(by, pq.w) ? p3 : 0.f));
    }
  };
  const int box = min(1 << c.lg_rows, kPtKeys), boxes = kPtKeys / box;   // K arrives a page (or 128 rows of one) at a time
  const int beyond = (c.n_pages * c.nkv) << c.lg_rows;                   // a row past the pool reads as zeros
  auto k_row = [&](int k0) {
    const int at = k0 + lane * box;
    const long long row = lane < boxes && at < len ? paged_row(c, seq, h, at) : -1;
    return row >= 0 ? (int)row : beyond;
  };
  auto load_k = [&](uint8_t* to, int y, uint64_t* bar) {
    if (lane == 0) mbar_expect_tx(bar, C::kTileB);
    __syncwarp();
    if (lane < boxes)
#pragma unroll
      for (int x = 0; x < C::kHalves; ++x) tma_load_2d(to + x * C::kHalfB + lane * box * 128, &mk, x * 64, y, bar);
  };
  auto load_q = [&](int q, int s) {
    mbar_expect_tx(&q_full[s], C::kHalves * tpt * G * 128);
    for (int x = 0; x < C::kHalves; ++x)
      tma_load_3d(sm + C::kQ + s * C::kTileB + x * C::kHalfB, &mq, x * 64, h * G, ab.x + q * tpt, &q_full[s]);
  };

  if (tiles == 1) {
    // One tile of query rows, a decode or verify block's: it stays, and the
    // CTA's key tiles pass by, two buffers of K (the second where the other
    // stage of Q would be) and of S ahead of the threads that own the keys.
    const int all_k = (len + kPtKeys - 1) / kPtKeys, x0 = blockIdx.x, dx = gridDim.x;
    const int nk = x0 < all_k ? (all_k - x0 + dx - 1) / dx : 0, chunks = (n_new * G + 31) >> 5;
    if (warp == wLoad) {
      if (nk > 0 && lane == 0) load_q(0, 0);
      int y = k_row(x0 * kPtKeys);
      int i = 0;
      for (; i < nk; ++i) {
        const int b = i & 1, next = k_row((x0 + (i + 1) * dx) * kPtKeys);
        if (i >= 2) paged_wait(&k_empty[b], ((i >> 1) - 1) & 1, ok);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        load_k(sm + (b ? C::kQ + C::kTileB : C::kK), y, &k_full[b]);
        y = next;
      }
      // no copy may be in flight when the CTA ends
      bool landed = true;
      if (nk > 0) paged_wait(&q_full[0], 0, landed);
      for (int j = i > 2 ? i - 2 : 0; j < i; ++j) paged_wait(&k_full[j & 1], (j >> 1) & 1, landed);
      ok = ok && landed;
    } else if (warp == wMma) {
      const bool leader = elect_one();
      const uint32_t sb = smem_u32(sm);
      const int ksteps = (c.hd + 15) >> 4;
      const uint64_t q_desc = smem_desc_sw128(sb + C::kQ), k_desc = smem_desc_sw128(sb + C::kK), k2_desc = smem_desc_sw128(sb + C::kQ + C::kTileB);
      if (nk > 0) paged_wait(&q_full[0], 0, ok);
      for (int i = 0; i < nk; ++i) {
        const int b = i & 1;
        paged_wait(&k_full[b], (i >> 1) & 1, ok);
        if (i >= 2) paged_wait(&s_empty[b], ((i >> 1) - 1) & 1, ok);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        if (leader) {
          tc_scores<C::kHalves>(tmem + b * 128, b ? k2_desc : k_desc, q_desc, ksteps);
          tc_commit(&s_full[b]);
          tc_commit(&k_empty[b]);
        }
        __syncwarp();
      }
    } else if (warp == wRows) {
      if (nk > 0) {
        put_rows(rows[0], row_data(0));
        __syncwarp();
        if (lane == 0) mbar_arrive(&rows_full[0]);
      }
    } else if (warp < wMma) {
      // the key's place, position and weight are requested a tile ahead
      auto place = [&](int i) {
        const int slot = (x0 + i * dx) * kPtKeys + (int)threadIdx.x;
        const long long row = slot < len ? paged_row(c, seq, h, slot) : -1;
        if (slot < len && row < 0 && c.status) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
        return row;
      };
      long long row = nk > 0 ? place(0) : -1;
      int pk = row >= 0 ? c.pos[row] : kPagedNoPos;
      float old = row >= 0 && a.weight_in ? a.weight_in[row] : 0.f;
      if (nk > 0) paged_wait(&rows_full[0], 0, ok);
      for (int i = 0; i < nk; ++i) {
        const int b = i & 1;
        const uint32_t s_at = tmem + (static_cast<uint32_t>(warp * 32) << 16) + b * 128;
        const long long next = i + 1 < nk ? place(i + 1) : -1;
        const PagedSees by = paged_seen_by(m, pk);
        paged_wait(&s_full[b], (i >> 1) & 1, ok);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        const int pk1 = next >= 0 ? c.pos[next] : kPagedNoPos;
        const float old1 = next >= 0 && a.weight_in ? a.weight_in[next] : 0.f;
        uint64_t add[2] = {0, 0};
#pragma unroll 1
        for (int n = 0; n < chunks; ++n) {
          float v[32];
          tmem_ld32(s_at + n * 32, v);
          tmem_ld_wait32(v);
          add_chunk(v, rows[0], n, by, pk, false, add);
        }
        tc_fence_before();
        mbar_arrive(&s_empty[b]);
        float a0, a1;
        unpack2(add2(add[0], add[1]), a0, a1);
        if (row >= 0) a.weight_out[row] = (a.weight_in ? a.decay * old : 0.f) + (a0 + a1);
        row = next;
        pk = pk1;
        old = old1;
      }
    }
    if (!ok && c.status) atomicOr(c.status, DFLASH_PAGED_GAVE_UP);
    if (threadIdx.x == 0 && h == 0 && blockIdx.x == 0) paged_report_length(c, seq, len);
    tc_fence_before();
    __syncthreads();
    if (warp == wMma) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    }
    return;
  }

  unsigned it = 0;                         // query tiles passed by, over the whole kernel
  unsigned kn = 0;                         // key tiles loaded

  for (int k0 = blockIdx.x * kPtKeys; k0 < len; k0 += gridDim.x * kPtKeys, ++kn) {
    if (threadIdx.x == 0) { s_kmin = INT32_MAX; s_kmax = INT32_MIN; }
    __syncthreads();
    const int slot = k0 + (int)threadIdx.x;
    long long my_row = -1;
    int pk = kPagedNoPos;
    if (warp < wMma) {
      if (slot < len) my_row = paged_row(c, seq, h, slot);
      if (my_row >= 0) pk = c.pos[my_row];
      if (slot < len && my_row < 0 && c.status) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
      if (tiles > kDirect) {
        const int lo = __reduce_min_sync(0xffffffffu, pk == kPagedNoPos ? INT32_MAX : pk);
        const int hi = __reduce_max_sync(0xffffffffu, pk);
        if (lane == 0) { atomicMin(&s_kmin, lo); atomicMax(&s_kmax, hi); }
      }
    } else if (warp == wLoad) {
      load_k(sm + C::kK, k_row(k0), &k_full[0]);
    }
    // few query tiles are not classified: that would cost more than a tile
    // too many
    const bool direct = tiles <= kDirect;
    if (!direct) __syncthreads();
    const int kmin = s_kmin, kmax = s_kmax;
    float w = 0.f;
    bool fresh = true;                      // K not yet waited for
    for (int c0 = 0; c0 < tiles; c0 += kChunk) {
      // which query tiles see any key here, and which see all of them
      const int cn = min(kChunk, tiles - c0);
      if (direct) {
        if (threadIdx.x == 0) { some[0] = (1u << cn) - 1; all[0] = 0u; }
      } else {
        __syncthreads();
        for (int i = threadIdx.x; i <= cn >> 5; i += C::kThreads) some[i] = all[i] = 0u;
        __syncthreads();
        for (int q = warp; q < cn; q += C::kThreads / 32) {
          int lo = INT32_MAX, hi = INT32_MIN;
          const int r0 = (c0 + q) * tpt, r1 = min(n_new, r0 + tpt);
          for (int i = r0 + lane; i < r1; i += 32) {
            const int p = a.q_pos[ab.x + i];
            lo = min(lo, p);
            hi = max(hi, p);
          }
          lo = __reduce_min_sync(0xffffffffu, lo);
          hi = __reduce_max_sync(0xffffffffu, hi);
          if (lane == 0) {
            const int k = paged_class(m, lo, hi, kmin, kmax, r1 - r0 == tpt);
            if (k >= 1) atomicOr(&some[q >> 5], 1u << (q & 31));
            if (k == 2) atomicOr(&all[q >> 5], 1u << (q & 31));
          }
        }
      }
      __syncthreads();
      PagedShare sh{0, cn, 0, 0, false};
      paged_take(sh, some, 0, 1);
      PagedCursor cur(some, sh);
      const int N = sh.take;
      if (warp == wLoad) {
        for (int i = 0; i < N; ++i) {
          const unsigned j = it + i;
          const int s = j % NS, q = c0 + cur.next();
          if (j >= NS) paged_wait(&q_empty[s], (j / NS - 1) & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          if (lane == 0) load_q(q, s);
          __syncwarp();
        }
      } else if (warp == wMma) {
        const bool leader = elect_one();
        const uint32_t sb = smem_u32(sm);
        const int ksteps = (c.hd + 15) >> 4;
        const uint64_t k_desc = smem_desc_sw128(sb + C::kK), q_desc = smem_desc_sw128(sb + C::kQ);
        if (fresh && N > 0) paged_wait(&k_full[0], kn & 1, ok);
        for (int i = 0; i < N; ++i) {
          const unsigned j = it + i;
          const int s = j % NS, b = j & 1;
          paged_wait(&q_full[s], (j / NS) & 1, ok);
          if (j >= 2) paged_wait(&s_empty[b], ((j >> 1) - 1) & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
            tc_scores<C::kHalves>(tmem + b * 128, k_desc, q_desc + s * (C::kTileB >> 4), ksteps);
            tc_commit(&s_full[b]);
            tc_commit(&q_empty[s]);
          }
          __syncwarp();
        }
      } else if (warp >= wRows) {
        // lse, position and slope of the rows of every other tile
        for (int i = 0; i < N; ++i) {
          const unsigned j = it + i;
          const int q = c0 + cur.next();
          if ((int)(j & 1) != warp - wRows) continue;
          RowData d = row_data(q);
          const int s = j % kNA;
          if (j >= kNA) paged_wait(&rows_empty[s], (j / kNA - 1) & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          put_rows(rows[s], d);
          // a row without an lse (padding, perhaps) adds nothing, but its score may
          // be NaN, which minus infinity does not hide: its tile is looked at row by
          // row (512 rows over 32768 keys: 155 us, without this 152 us)
          if (!d.whole && lane == 0) atomicAnd(&all[(q - c0) >> 5], ~(1u << ((q - c0) & 31)));
          __syncwarp();
          if (lane == 0) mbar_arrive(&rows_full[s]);
        }
      } else {
        const PagedSees by = paged_seen_by(m, pk);
        // a lane without a row holds scores of whatever its page has there, which
        // have no say in how the warp's caps are computed
        cap.limit = my_row >= 0 ? cap_limit : INFINITY;
        for (int i = 0; i < N; ++i) {
          const unsigned j = it + i;
          const int rel = cur.next(), b = j & 1, s = j % kNA;
          const uint32_t s_at = tmem + (static_cast<uint32_t>(warp * 32) << 16) + b * 128;
          paged_wait(&rows_full[s], (j / kNA) & 1, ok);
          const WtRows& rw = rows[s];
          const bool full = (all[rel >> 5] >> (rel & 31)) & 1u;
          paged_wait(&s_full[b], (j >> 1) & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc_fence_after();
          uint64_t add[2] = {0, 0};
          if (full && !EXTRA) {
            const uint64_t sc2 = pack2(scale2, scale2);
            float x[2][32];
            tmem_ld32(s_at, x[0]);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              float* v = x[n & 1];
              tmem_ld_wait32(v);
              if (n < 3) {
                tmem_ld32(s_at + (n + 1) * 32, x[(n + 1) & 1]);
              } else {
                tc_fence_before();
                mbar_arrive(&s_empty[b]);
              }
              const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(rw.nlse2 + n * 32);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const ulonglong2 l = nl[e >> 2];
                float p0, p1, p2, p3;
                unpack2(fma2(pack2(v[e], v[e + 1]), sc2, l.x), p0, p1);
                unpack2(fma2(pack2(v[e + 2], v[e + 3]), sc2, l.y), p2, p3);
                add[0] = add2(add[0], pack2(ex2(p0), ex2(p1)));
                add[1] = add2(add[1], pack2(ex2(p2), ex2(p3)));
              }
            }
          } else {
#pragma unroll 1
            for (int n = 0; n < 4; ++n) {
              float v[32];
              tmem_ld32(s_at + n * 32, v);
              tmem_ld_wait32(v);
              if (n == 3) {
                tc_fence_before();
                mbar_arrive(&s_empty[b]);
              }
              add_chunk(v, rw, n, by, pk, full, add);
            }
          }
          float a0, a1;
          unpack2(add2(add[0], add[1]), a0, a1);
          w += a0 + a1;
          __syncwarp();
          if (lane == 0) mbar_arrive(&rows_empty[s]);
        }
      }
      if (N > 0) fresh = false;
      it += N;
    }
    if (warp < wMma && my_row >= 0) a.weight_out[my_row] = (a.weight_in ? a.decay * a.weight_in[my_row] : 0.f) + w;
    // K has landed before its tile is loaded again or the CTA ends
    if (warp == wLoad) paged_wait(&k_full[0], kn & 1, ok);
    if (!ok && c.status) atomicOr(c.status, DFLASH_PAGED_GAVE_UP);
    if (__syncthreads_or(!ok)) { ok = false; break; }
  }
  // no copy of Q in flight either (what nobody took when a wait gave up)
  if (warp == wLoad && it > 0 && !ok) {
    for (int i = 0; i < NS; ++i) {
      bool landed = true;
      paged_wait(&q_full[i], 0, landed);
      paged_wait(&q_full[i], 1, landed);
    }
  }
  if (threadIdx.x == 0 && h == 0 && blockIdx.x == 0) paged_report_length(c, seq, len);
  tc_fence_before();
  __syncthreads();
  if (warp == wMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int HDP>
cudaError_t run(const PagedAttnArgs& a, long long tiles, cudaStream_t st) {
  CUtensorMap mq, mk;
  // without new rows there is nothing to map: K's map stands in, unread
  if (!paged_map_pages(&mk, a.c.k, a.c)) return cudaErrorInvalidValue;
  if (a.rows > 0) {
    if (!paged_map_rows(&mq, a.q, a, kPtKeys / a.G)) return cudaErrorInvalidValue;
  } else {
    mq = mk;
  }
  using C = WtShape<HDP>;
  auto kernel = a.softcap > 0.f || a.slopes ? paged_weight_tc_kernel<HDP, true> : paged_weight_tc_kernel<HDP, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)tiles, a.c.nkv, a.c.n_seq), dim3(C::kThreads), C::kSmem, st, mq, mk, a);
}

}  // namespace

cudaError_t launch_paged_weight_tc(const PagedAttnArgs& a, long long tiles, cudaStream_t st) {
  // Few query rows: CTAs, two to an SM, that pass several key tiles each, two
  // waves of them for sequences of different lengths (32 sequences of one row over
  // 12000 keys: 83 us, with a CTA to every key tile 292 us). (The kernel decides by each
  // sequence's own rows what it does; a grid for the other case only starts more
  // CTAs.)
  if ((long long)a.rows * a.G <= 128ll * a.c.n_seq) {
    const long long pairs = (long long)a.c.nkv * a.c.n_seq, most = (608 + pairs - 1) / pairs;
    if (tiles > most) tiles = most;
  }
  // a table far longer than its sequences need not start a CTA for every tile
  const long long limit = 65536 / ((long long)a.c.nkv * a.c.n_seq) + 1;
  if (tiles > limit) tiles = limit;
  return a.c.hd <= 64 ? run<64>(a, tiles, st) : run<128>(a, tiles, st);
}

}  // namespace dfl
