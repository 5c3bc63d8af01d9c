// How an attention call over the paged cache is divided, the merge of split
// partials, and key weights for fp32 and for bf16 heads of more than 128
// dimensions. Scores are kept in log2 units, u = t * log2(e).
#include <math.h>

#include "paged.cuh"
#include "paged_tf32.cuh"

namespace dfl {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBN = 64;                    // keys of a key-weight tile

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
// sequences of up to 10 rows and 6000 keys, 16 and 8 heads, fp32: 220 us; so: 85 us.)
constexpr int kWRows = 64;

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
  if (threadIdx.x == 0 && h == 0 && blockIdx.x == 0) paged_report_length(c, s, len);
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
      if (slot < len && row[i] < 0 && c.status) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
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

template <typename K>
cudaError_t big_smem(K* kernel, size_t bytes) {
  return bytes <= 48 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
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

// kind 1 and 2: tcgen05 (bf16, head_dim <= 128), that many tiles of 128 packed
// query rows to a CTA; 16: mma.sync in tf32, that many rows.
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
    p.kind = 16;
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
  cudaError_t e;
  if (p.kind <= 2) e = launch_paged_attention_tc(a, p.kind, p.tiles, st);
  else e = launch_paged_attention_tf32(dtype, a, p.tiles, st);
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
