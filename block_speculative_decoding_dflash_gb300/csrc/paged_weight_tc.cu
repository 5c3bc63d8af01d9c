// Key weights on the tensor cores (bf16, head_dim <= 128): for every cached row
// of a (sequence, kv head) the sum over the query rows of exp(t - lse).
//
// S^T = K Q^T: a CTA holds a tile of 128 keys as the A operand and passes the
// query rows by as B, 128 at a time. A key is a TMEM lane, so one thread owns it
// for the whole pass and adds up its row of S^T in registers: no exchange
// between threads, no atomics, and a fixed order. S has two buffers; the
// exponentials of one run while the next is computed, and a second CTA on the SM
// works while this one starts or ends. Bounded by the exponentials, one ex2 to a
// score, against 2 head_dim flops on the tensor cores, for many query rows, and
// by a CTA's start and end for few.
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
  __shared__ uint64_t k_full, q_full[NS], q_empty[NS], rows_full[kNA], rows_empty[kNA], s_full[2], s_empty[2];
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
    mbar_init(&k_full, 1);
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
      // K, a box per page (or per 128 rows of one)
      const int box = min(1 << c.lg_rows, kPtKeys), boxes = kPtKeys / box;
      const int beyond = (c.n_pages * c.nkv) << c.lg_rows;
      if (lane == 0) mbar_expect_tx(&k_full, C::kTileB);
      __syncwarp();
      const int at = k0 + lane * box;
      int y = beyond;
      if (lane < boxes && at < len) {
        const long long row = paged_row(c, seq, h, at);
        if (row >= 0) y = (int)row;
      }
      if (lane < boxes)
#pragma unroll
        for (int x = 0; x < C::kHalves; ++x)
          tma_load_2d(sm + C::kK + x * C::kHalfB + lane * box * 128, &mk, x * 64, y, &k_full);
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
          if (lane == 0) {
            mbar_expect_tx(&q_full[s], C::kHalves * tpt * G * 128);
            for (int x = 0; x < C::kHalves; ++x)
              tma_load_3d(sm + C::kQ + s * C::kTileB + x * C::kHalfB, &mq, x * 64, h * G, ab.x + q * tpt, &q_full[s]);
          }
          __syncwarp();
        }
      } else if (warp == wMma) {
        const bool leader = elect_one();
        const uint32_t sb = smem_u32(sm);
        const int ksteps = (c.hd + 15) >> 4;
        const uint64_t k_desc = smem_desc_sw128(sb + C::kK), q_desc = smem_desc_sw128(sb + C::kQ);
        if (fresh && N > 0) paged_wait(&k_full, kn & 1, ok);
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
          float l[4], sl[4];
          int p[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = x * 32 + lane, tl = r / G, tok = q * tpt + tl, head = h * G + r - tl * G;
            const bool in = tl < tpt && tok < n_new;
            const float v = in ? a.lse[(size_t)(ab.x + tok) * a.nq + head] : -INFINITY;
            l[x] = v == -INFINITY ? -INFINITY : -v * kLog2e;
            p[x] = v == -INFINITY ? kPagedNoPos : a.q_pos[ab.x + tok];
            sl[x] = in && a.slopes ? a.slopes[head] * kLog2e : 0.f;
          }
          int base = 0, near = 1;
          if (EXTRA && a.slopes) {
            int lo = INT32_MAX, hi = INT32_MIN;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              lo = min(lo, p[x] == kPagedNoPos ? INT32_MAX : p[x]);
              hi = max(hi, p[x]);
            }
            base = __reduce_min_sync(0xffffffffu, lo);
            near = (long long)__reduce_max_sync(0xffffffffu, hi) - base < (1 << 23);
          }
          const int s = j % kNA;
          if (j >= kNA) paged_wait(&rows_empty[s], (j / kNA - 1) & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = x * 32 + lane;
            rows[s].nlse2[r] = l[x];
            rows[s].pos[r] = p[x];
            rows[s].slope2[r] = sl[x];
            if (EXTRA && a.slopes) rows[s].dist[r] = (float)(p[x] - base);
          }
          if (EXTRA && lane == 0) {
            rows[s].base = base;
            rows[s].near = near;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&rows_full[s]);
        }
      } else {
        const float scale2 = a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e;
        const CapPoly cap = cap_poly(scale2, a.softcap * kLog2e);
        const PagedSees by = paged_seen_by(m, pk);
        for (int i = 0; i < N; ++i) {
          const unsigned j = it + i;
          const int rel = cur.next(), b = j & 1, s = j % kNA;
          const bool full = (all[rel >> 5] >> (rel & 31)) & 1u;
          const uint32_t s_at = tmem + (static_cast<uint32_t>(warp * 32) << 16) + b * 128;
          paged_wait(&rows_full[s], (j / kNA) & 1, ok);
          paged_wait(&s_full[b], (j >> 1) & 1, ok);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc_fence_after();
          const WtRows& rw = rows[s];
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
              float sc = scale2;
              if (EXTRA && a.softcap > 0.f) {
                cap_tanh32(v, cap);
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
    if (warp == wLoad) paged_wait(&k_full, kn & 1, ok);
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
  return a.c.hd <= 64 ? run<64>(a, tiles, st) : run<128>(a, tiles, st);
}

}  // namespace dfl
