// How an attention call over the paged cache is divided; attention for bf16 heads
// of more than 128 dimensions, which the tensor-core kernel does not take; the
// merge of split partials; key weights for fp32 and for those heads.
//
// Per (query tile, kv head, split): an online softmax over key tiles. The
// scores are kept in log2 units, u = t * log2(e), so p = exp2(u - m).
#include <math.h>

#include "paged.cuh"
#include "paged_tf32.cuh"

namespace dfl {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBN = 64;                    // keys of a tile
constexpr int kMaxTiles = (1 << 20) / kBN; // of the longest table

// Score of a raw dot product in log2 units.
struct PagedScore { float scale2, cap2; };
__device__ __forceinline__ PagedScore paged_score_of(const PagedAttnArgs& a) {
  PagedScore s;
  s.scale2 = a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e;
  s.cap2 = a.softcap * kLog2e;
  return s;
}
__device__ __forceinline__ float paged_score(const PagedAttnArgs& a, const PagedScore& s, float dot, float slope2, int pq, int pk) {
  float u = dot * s.scale2;
  if (a.softcap > 0.f) u = s.cap2 * tanhf(u);
  if (slope2 != 0.f) u -= slope2 * fabsf((float)(pq - pk));
  return u;
}

// Rows of `n` values at src into shared rows of HDP + 4 floats, zero past hd
// and where src is NULL; 16-byte loads, `lanes` threads to a row.
template <typename T, int HDP>
__device__ __forceinline__ bool load_row(float* dst, const T* src, int hd, int lane, int lanes) {
  bool bad = false;
  for (int d = lane * 8; d < HDP; d += lanes * 8) {
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (src && d < hd) load8(src + d, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) bad |= !(fabsf(x[i]) <= 3.4028234663852886e38f);
    *reinterpret_cast<float4*>(dst + d) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(dst + d + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
  return bad;
}

// BM packed query rows (row r = token r / G, head r % G of the group) against
// kBN keys at a time. Thread (ty, tx) holds TM rows ty * TM .. and keys tx,
// tx + 16, .. of the scores, then dims tx * 4 + 64 j of the same rows' output:
// 16 lanes share a row, so row statistics are shuffles within half a warp.
// K and V tiles are read from HBM once per query tile; for few query rows
// that read bounds the kernel, for many the fp32 FMA rate.
template <int BM, int TM>
__global__ void __launch_bounds__(BM / TM * 16) paged_attn_simt_kernel(PagedAttnArgs a) {
  using T = bf16;
  constexpr int HDP = 256, NT = BM / TM * 16, LD = HDP + 4, NJ = HDP / 64;
  pdl_enter();
  extern __shared__ float smf[];
  float* sq = smf;                          // [BM][LD]
  float* sk = sq + BM * LD;                 // [kBN][LD]
  float* sv = sk + kBN * LD;                // [kBN][LD]
  float* sp = sv + kBN * LD;                // [BM][kBN + 4]
  int* spos = reinterpret_cast<int*>(sp + BM * (kBN + 4));     // [kBN]
  unsigned* some = reinterpret_cast<unsigned*>(spos + kBN);
  unsigned* all = some + kMaxTiles / 32 + 1;
  __shared__ PagedTile st;
  __shared__ int s_qmin, s_qmax;
  const PagedView& c = a.c;
  const int h = blockIdx.y, z = blockIdx.z, G = a.G;
  if (threadIdx.x < 32) {
    const PagedTile t = paged_find_tile(a.start, c.n_seq, a.rows, G, BM, blockIdx.x);
    int lo = INT32_MAX, hi = INT32_MIN;
    if (t.seq >= 0) {
      const int r0 = t.tile * BM, r1 = min(t.count * G, r0 + BM);
      for (int i = r0 / G + (int)threadIdx.x; i <= (r1 - 1) / G; i += 32) {
        const int p = a.q_pos[t.first + i];
        lo = min(lo, p);
        hi = max(hi, p);
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (threadIdx.x == 0) { st = t; s_qmin = lo; s_qmax = hi; }
  }
  __syncthreads();
  const PagedTile t = st;
  if (t.seq < 0) return;
  const int len = paged_length(c, t.seq);
  const PagedMask m = paged_mask(a.causal, a.window, a.prefix, t.seq);
  PagedShare sh = paged_range((len + kBN - 1) / kBN, a.window, z, a.splits);
  paged_classify<kBN>(c, t.seq, h, len, m, s_qmin, s_qmax, sh.t0, sh.t1, some, all);

  const int r0 = t.tile * BM, rows = min(BM, t.count * G - r0);
  for (int e = threadIdx.x; e < BM * 16; e += NT) {
    const int r = e >> 4;
    const T* src = r < rows ? static_cast<const T*>(a.q) + (size_t)(t.first + (r0 + r) / G) * a.q_stride +
                                  (size_t)(h * G + (r0 + r) % G) * c.hd : nullptr;
    load_row<T, HDP>(sq + r * LD, src, c.hd, e & 15, 16);
  }
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  int pq[TM];
  PagedSees sees[TM];
  float slope2[TM], mx[TM], sum[TM], o[TM][NJ * 4];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = r0 + min(ty * TM + i, rows - 1);
    pq[i] = a.q_pos[t.first + r / G];
    sees[i] = paged_sees_of(m, pq[i]);
    slope2[i] = a.slopes ? a.slopes[h * G + r % G] * kLog2e : 0.f;
    mx[i] = -INFINITY;
    sum[i] = 0.f;
#pragma unroll
    for (int d = 0; d < NJ * 4; ++d) o[i][d] = 0.f;
  }
  const PagedScore ps = paged_score_of(a);
  __syncthreads();
  paged_take(sh, some, z, a.splits);
  PagedCursor cur(some, sh);
  for (int rel = cur.next(); rel >= 0; rel = cur.next()) {
    const int k0 = (sh.t0 + rel) * kBN;
    const bool full = (all[rel >> 5] >> (rel & 31)) & 1u;
    bool bad = false;
    for (int e = threadIdx.x; e < kBN * 8; e += NT) {
      const int j = e >> 3, l8 = e & 7;
      const long long row = k0 + j < len ? paged_row(c, t.seq, h, k0 + j) : -1;
      load_row<T, HDP>(sk + j * LD, row >= 0 ? static_cast<const T*>(c.k) + row * c.hd : nullptr, c.hd, l8, 8);
      bad |= load_row<T, HDP>(sv + j * LD, row >= 0 ? static_cast<const T*>(c.v) + row * c.hd : nullptr, c.hd, l8, 8);
      if (l8 == 0) spos[j] = row >= 0 ? c.pos[row] : kPagedNoPos;
    }
    // a tile that some query sees only in part and whose V holds infinities or
    // NaN: the hidden rows must not be multiplied by their zero weight
    const bool careful = __syncthreads_or(bad && !full);
    float s[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < HDP; d += 4) {
      float4 q[TM], k[4];
#pragma unroll
      for (int i = 0; i < TM; ++i) q[i] = *reinterpret_cast<const float4*>(sq + (ty * TM + i) * LD + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LD + d);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(q[i].x, k[j].x, s[i][j]);
          s[i][j] = fmaf(q[i].y, k[j].y, s[i][j]);
          s[i][j] = fmaf(q[i].z, k[j].z, s[i][j]);
          s[i][j] = fmaf(q[i].w, k[j].w, s[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      unsigned seen = 0;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pk = spos[tx + 16 * j];
        const bool v = full || paged_sees(sees[i], pk);
        s[i][j] = v ? paged_score(a, ps, s[i][j], slope2[i], pq[i], pk) : -INFINITY;
        seen |= (unsigned)v << j;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(mx[i], top);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(mx[i] - base);
      float add = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - base);
        add += p;
        // a hidden row's weight is -0, a seen one's that underflowed +0
        sp[(ty * TM + i) * (kBN + 4) + tx + 16 * j] = (seen >> j) & 1u ? p : -0.f;
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) add += __shfl_xor_sync(0xffffffffu, add, x);
      sum[i] = sum[i] * f + add;
      mx[i] = mn;
#pragma unroll
      for (int d = 0; d < NJ * 4; ++d) o[i][d] *= f;
    }
    __syncwarp();
#pragma unroll 2
    for (int j = 0; j < kBN; j += 4) {
      float4 p[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (ty * TM + i) * (kBN + 4) + j);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
          const float4 v = *reinterpret_cast<const float4*>(sv + (j + jj) * LD + n * 64 + tx * 4);
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const float w = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
            if (careful && __float_as_uint(w) == 0x80000000u) continue;
            o[i][n * 4 + 0] = fmaf(w, v.x, o[i][n * 4 + 0]);
            o[i][n * 4 + 1] = fmaf(w, v.y, o[i][n * 4 + 1]);
            o[i][n * 4 + 2] = fmaf(w, v.z, o[i][n * 4 + 2]);
            o[i][n * 4 + 3] = fmaf(w, v.w, o[i][n * 4 + 3]);
          }
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = ty * TM + i;
    if (r >= rows) continue;
    const size_t at = (size_t)(t.first + (r0 + r) / G) * a.nq + h * G + (r0 + r) % G;
    if (a.splits > 1) {
      float* po = a.part_o + ((size_t)z * a.rows * a.nq + at) * c.hd;
#pragma unroll
      for (int n = 0; n < NJ; ++n)
        if (n * 64 + tx * 4 < c.hd)
          *reinterpret_cast<float4*>(po + n * 64 + tx * 4) = make_float4(o[i][n * 4], o[i][n * 4 + 1], o[i][n * 4 + 2], o[i][n * 4 + 3]);
      if (tx == 0) a.part_ml[(size_t)z * a.rows * a.nq + at] = make_float2(mx[i], sum[i]);
      continue;
    }
    const bool none = sum[i] == 0.f;           // nothing seen (a NaN score makes the sum NaN)
    const float inv = none ? 0.f : 1.f / sum[i];
    T* out = static_cast<T*>(a.out) + at * c.hd;
#pragma unroll
    for (int n = 0; n < NJ; ++n)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if (n * 64 + tx * 4 + d < c.hd) out[n * 64 + tx * 4 + d] = from_f<T>(none ? 0.f : o[i][n * 4 + d] * inv);
    if (tx == 0 && a.lse) a.lse[at] = none ? -INFINITY : (mx[i] + log2f(sum[i])) * kLn2;
  }
}

// Joins the splits of one (row, head), a warp to each: o = sum_z o_z
// exp2(m_z - M) / sum_z l_z exp2(m_z - M). Rows of no sequence are left alone.
template <typename T>
__global__ void __launch_bounds__(128) paged_attn_merge_kernel(PagedAttnArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31, hd = a.c.hd;
  const long long at = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int first = max(0, a.start[0]), last = min(a.rows, a.start[a.c.n_seq]);
  const long long n = (long long)a.rows * a.nq;
  if (at >= n || at / a.nq < first || at / a.nq >= last) return;
  float M = -INFINITY;
  for (int z = lane; z < a.splits; z += 32) M = fmaxf(M, a.part_ml[z * n + at].x);
  M = warp_max(M);
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int kU = 4;                      // splits requested together
  for (int z0 = 0; z0 < a.splits; z0 += kU) {
    float2 ml[kU];
    float4 x[kU][2];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const bool in = z0 + u < a.splits;
      ml[u] = in ? a.part_ml[(z0 + u) * n + at] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        x[u][j] = in && j * 128 + lane * 4 < hd ? *reinterpret_cast<const float4*>(a.part_o + ((z0 + u) * n + at) * hd + j * 128 + lane * 4)
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (ml[u].y == 0.f) continue;          // it saw nothing
      const float f = exp2f(ml[u].x - base);
      L += ml[u].y * f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[j * 4] = fmaf(f, x[u][j].x, acc[j * 4]);
        acc[j * 4 + 1] = fmaf(f, x[u][j].y, acc[j * 4 + 1]);
        acc[j * 4 + 2] = fmaf(f, x[u][j].z, acc[j * 4 + 2]);
        acc[j * 4 + 3] = fmaf(f, x[u][j].w, acc[j * 4 + 3]);
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  T* out = static_cast<T*>(a.out) + at * hd;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (j * 128 + lane * 4 + d < hd) out[j * 128 + lane * 4 + d] = from_f<T>(acc[j * 4 + d] * inv);
  if (lane == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// Key weights for fp32, and for bf16 heads of more than 128 dimensions: S^T = K Q^T
// on the tensor cores in tf32, fp32's factors in two parts (see paged_tf32.cuh;
// bf16 is a tf32 as it stands). A warp has 16 keys in registers, read once, and
// the CTA passes the sequence's query rows by in shared memory, kWRows at a time; a
// lane adds exp2(u - lse) over its columns for its two keys, the four lanes of a key
// are summed at the end: no atomics, and a fixed order. (On CUDA cores, 16
// sequences of up to 10 rows and 6000 keys, 8 heads, fp32: 220 us; so: 81 us.)
constexpr int kWRows = 64;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const bf16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y));
}

template <typename T, int HDP>
__global__ void __launch_bounds__(128, HDP > 128 ? 2 : 4) paged_weight_tf32_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr bool kParts = sizeof(T) == 4;
  constexpr int LD = HDP + 16, kSteps = HDP / 16;
  pdl_enter();
  extern __shared__ __align__(16) float sq[];     // [kWRows][LD]
  __shared__ int sqp[kWRows];
  __shared__ float snl[kWRows], sslope[kWRows];   // minus lse and the slope, in log2 units; -inf for what adds nothing
  const PagedView& c = a.c;
  const int h = blockIdx.y, s = blockIdx.z, G = a.G, hd = c.hd;
  const int2 ab = paged_new_rows(a.start, s, a.rows);
  const int len = paged_length(c, s), R = (ab.y - ab.x) * G;
  const PagedMask m = paged_mask(a.causal, a.window, a.prefix, s);
  const PagedScore ps = paged_score_of(a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, e4 = lane & 3;
  for (int k0 = blockIdx.x * kBN; k0 < len; k0 += gridDim.x * kBN) {
    // the lane's keys, g and g + 8 of the warp's
    long long row[2];
    int pk[2];
    PagedSees by[2];
    float w[2] = {0.f, 0.f};
    float4 k[kSteps][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int slot = k0 + warp * 16 + g + 8 * i;
      row[i] = slot < len ? paged_row(c, s, h, slot) : -1;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const T* src = static_cast<const T*>(c.k) + (row[i] >= 0 ? row[i] : 0) * hd;
      pk[i] = row[i] >= 0 ? c.pos[row[i]] : kPagedNoPos;
      by[i] = paged_seen_by(m, pk[i]);
#pragma unroll
      for (int t = 0; t < kSteps; ++t)
        k[t][i] = row[i] >= 0 && t * 16 + e4 * 4 < hd ? load4(src + t * 16 + e4 * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int q0 = 0; q0 < R; q0 += kWRows) {
      const int n = min(kWRows, R - q0), n16 = (n + 15) & ~15;
      __syncthreads();
      for (int e = threadIdx.x; e < n16 * (HDP / 4); e += 128) {
        const int r = e / (HDP / 4), d = e % (HDP / 4) * 4, rr = q0 + r;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n && d < hd) v = load4(static_cast<const T*>(a.q) + (size_t)(ab.x + rr / G) * a.q_stride + (size_t)(h * G + rr % G) * hd + d);
        *reinterpret_cast<float4*>(sq + r * LD + d) = v;
      }
      for (int r = threadIdx.x; r < n16; r += 128) {
        const bool in = r < n;
        const size_t tok = in ? ab.x + (q0 + r) / G : 0;
        const int head = in ? h * G + (q0 + r) % G : 0;
        const float l = in ? a.lse[tok * a.nq + head] : -INFINITY;
        sqp[r] = in ? a.q_pos[tok] : 0;
        snl[r] = l == -INFINITY ? -INFINITY : -l * kLog2e;
        sslope[r] = in && a.slopes ? a.slopes[head] * kLog2e : 0.f;
      }
      __syncthreads();
#pragma unroll 1
      for (int n0 = 0; n0 < n; n0 += 16) {
        // scores of keys g, g + 8 and rows n0 + 8 y + 2 e4, + 1
        float big[2][4], odd[2][4], low[2][4];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) big[y][x] = odd[y][x] = low[y][x] = 0.f;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
          uint32_t kh[2][4], kl[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float4 v = k[t][i];
            // (not to be taken out of the loop: the parts of all of K do not fit the registers)
            if (kParts) asm volatile("" : "+f"(v.x), "+f"(v.y), "+f"(v.z), "+f"(v.w));
            cut2(v.x, kh[i][0], kl[i][0]);
            cut2(v.y, kh[i][1], kl[i][1]);
            cut2(v.z, kh[i][2], kl[i][2]);
            cut2(v.w, kh[i][3], kl[i][3]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float4 q = *reinterpret_cast<const float4*>(sq + (n0 + y * 8 + g) * LD + t * 16 + e4 * 4);
            uint32_t qh[4], ql[4];
            round2(q.x, qh[0], ql[0]);
            round2(q.y, qh[1], ql[1]);
            round2(q.z, qh[2], ql[2]);
            round2(q.w, qh[3], ql[3]);
            float* to = t & 1 ? odd[y] : big[y];
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
              mma_tf32(to, kh[0][x], kh[1][x], kh[0][x + 1], kh[1][x + 1], qh[x], qh[x + 1]);
              if (kParts) {
                mma_tf32(low[y], kl[0][x], kl[1][x], kl[0][x + 1], kl[1][x + 1], qh[x], qh[x + 1]);
                mma_tf32(low[y], kh[0][x], kh[1][x], kh[0][x + 1], kh[1][x + 1], ql[x], ql[x + 1]);
              }
            }
          }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int i = x >> 1, r = n0 + y * 8 + e4 * 2 + (x & 1);
            const float nl = snl[r];
            const float u = paged_score(a, ps, big[y][x] + odd[y][x] + low[y][x], sslope[r], sqp[r], pk[i]);
            if (nl != -INFINITY && paged_sees(by[i], sqp[r])) w[i] += exp2f(u + nl);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
      w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
      if (e4 == 0 && row[i] >= 0) a.weight_out[row[i]] = (a.weight_in ? a.decay * a.weight_in[row[i]] : 0.f) + w[i];
    }
  }
}

template <int BM>
constexpr size_t simt_smem() {
  return ((size_t)(BM + 2 * kBN) * (256 + 4) + BM * (kBN + 4) + kBN) * 4 + 2 * (kMaxTiles / 32 + 1) * 4;
}

template <typename K>
cudaError_t big_smem(K* kernel, size_t bytes) {
  return bytes <= 48 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int BM, int TM>
cudaError_t run_simt(const PagedAttnArgs& a, dim3 grid, cudaStream_t st) {
  cudaError_t e = big_smem(paged_attn_simt_kernel<BM, TM>, simt_smem<BM>());
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_attn_simt_kernel<BM, TM>, grid, dim3(BM / TM * 16), simt_smem<BM>(), st, a);
}
template <typename T, int HDP>
cudaError_t run_weight(const PagedAttnArgs& a, dim3 grid, cudaStream_t st) {
  constexpr size_t smem = (size_t)kWRows * (HDP + 16) * 4;
  cudaError_t e = big_smem(paged_weight_tf32_kernel<T, HDP>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_weight_tf32_kernel<T, HDP>, grid, dim3(128), smem, st, a);
}

int expected_len(const PagedAttnArgs& a) {
  const int cap = a.c.max_pages << a.c.lg_rows;
  return a.max_len > 0 && a.max_len < cap ? a.max_len : cap;
}
// Tiles a batch of `units` query rows can have at most, `per` to a tile.
long long tile_bound(long long units, int per, const PagedAttnArgs& a) {
  return units / per + (a.c.n_seq < a.rows ? a.c.n_seq : a.rows);
}

}  // namespace

// kind 1 and 2: tensor cores (bf16, head_dim <= 128), that many tiles of 128
// packed query rows to a CTA; 16, 32, 64: CUDA cores, that many rows.
PagedPlan paged_attn_plan(int dtype, const PagedAttnArgs& a) {
  PagedPlan p{0, 1, 0, 0, 0};
  const long long len = expected_len(a), units = (long long)a.rows * a.G;
  long long fill, least;
  if (dtype && a.c.hd <= 128) {
    // two query tiles to a CTA where an average sequence fills more than one
    // (2048 rows over 32768 keys: 0.81 ms, with one 1.59 ms; 48 rows of decode: with
    // one 264 us, with two 298 us)
    const int per = 128 / a.G;
    p.kind = a.rows > (long long)per * a.c.n_seq ? 2 : 1;
    p.tiles = tile_bound(a.rows, p.kind * per, a);
    fill = 152;
    least = 512;
  } else {
    // the smallest tile that holds an average sequence's rows (100 rows of 4
    // sequences, 4 heads to a kv head: 670 us in tiles of 64, 2163 us of 16; one
    // row each of 8: 719 us and 710 us); fp32: 16 always
    p.kind = !dtype || units <= 16ll * a.c.n_seq ? 16 : 64;
    p.tiles = tile_bound(units, p.kind, a);
    fill = 608;
    least = 256;
  }
  // as many splits as fill the SMs, of at least `least` keys each (8 sequences of
  // fp32 blocks: 56 us, filling half as many 96 us, twice as many 64 us)
  const long long ctas = p.tiles * a.c.nkv, by_keys = (len + least - 1) / least;
  const long long n = ctas >= fill ? 1 : (fill / ctas < by_keys ? fill / ctas : by_keys);
  p.splits = n < 1 ? 1 : (int)n;
  if (p.kind <= 2 && ctas < fill && (p.splits <= 8 || len <= 8 * 1024)) {
    // Up to eight splits are a cluster that joins its partials in shared
    // memory: no second kernel and no workspace. A cluster is of CTAs of one
    // GPC (18 SMs or more), so what fits at once goes by its size; its splits may
    // be as short as a tile. (A block of 4 rows in a window of 2048: 14.0 us, with
    // the merge kernel 19.6 us. One row over 32768 keys of 8 heads: 76 us with eight
    // splits, 37 us with as many as fill the GPU and the merge kernel.)
    static const struct { int size, most; } kFit[5] = {{8, 16}, {6, 24}, {4, 32}, {3, 48}, {2, 72}};
    const long long key_tiles = (len + 127) / 128;
    p.splits = 1;
    for (const auto& f : kFit)
      if (p.splits == 1 && ctas <= f.most && f.size <= key_tiles) p.splits = f.size;
    p.cluster = p.splits > 1;
  } else if (p.kind == 1 && ctas >= fill && ctas < 4 * fill && len >= 4096) {
    // sequences of all lengths on a few waves of CTAs: halves even them out
    // (48 sequences of up to 12345 rows: 282 us to 264 us)
    p.splits = 2;
    p.cluster = 1;
  } else if (p.splits > 1) {
    p.bytes = (long long)p.splits * a.rows * a.nq * (a.c.hd + 2) * 4;
  }
  return p;
}

cudaError_t launch_paged_attention(int dtype, const PagedAttnArgs& a, const PagedPlan& p, cudaStream_t st) {
  const dim3 grid((unsigned)p.tiles, a.c.nkv, p.splits);
  cudaError_t e;
  if (p.kind <= 2) e = launch_paged_attention_tc(a, p.kind, p.tiles, st);
  else if (!dtype) e = launch_paged_attention_f32(a, p.tiles, st);
  else if (p.kind == 16) e = run_simt<16, 2>(a, grid, st);
  else e = run_simt<64, 4>(a, grid, st);
  if (e != cudaSuccess || p.splits <= 1 || p.cluster) return e;
  const dim3 mg((unsigned)(((long long)a.rows * a.nq + 3) / 4));
  return dtype ? launch_pdl(paged_attn_merge_kernel<bf16>, mg, dim3(128), 0, st, a)
               : launch_pdl(paged_attn_merge_kernel<float>, mg, dim3(128), 0, st, a);
}

cudaError_t launch_paged_key_weight(int dtype, const PagedAttnArgs& a, cudaStream_t st) {
  if (dtype && a.c.hd <= 128) return launch_paged_weight_tc(a, (expected_len(a) + 127) / 128, st);
  // at most so many CTAs that a table far longer than its sequences does not
  // start one for every tile
  long long x = (expected_len(a) + kBN - 1) / kBN;
  const long long limit = 65536 / ((long long)a.c.nkv * a.c.n_seq) + 1;
  if (x > limit) x = limit;
  const dim3 grid((unsigned)x, a.c.nkv, a.c.n_seq);
  if (dtype) return run_weight<bf16, 256>(a, grid, st);
  if (a.c.hd <= 64) return run_weight<float, 64>(a, grid, st);
  return a.c.hd <= 128 ? run_weight<float, 128>(a, grid, st) : run_weight<float, 256>(a, grid, st);
}

}  // namespace dfl
