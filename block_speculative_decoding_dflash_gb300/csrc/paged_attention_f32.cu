// Attention over the paged cache in fp32 on CUDA cores.
//
// BM packed query rows (row r = token r / G, head r % G of the group) against
// 64 keys at a time. Thread (ty, tx) holds TM rows ty * TM .. and keys tx,
// tx + 16, .. of the scores, then dims tx * 4 + 64 j of the same rows' output:
// 16 lanes share a row, so row statistics are shuffles within half a warp. A
// 4 x 4 tile of scores takes 8 16-byte shared loads for 64 multiplications
// (two to an instruction), which keeps the FMA pipes, not shared memory, the
// bound. K and V have one buffer each: the next K arrives while P V runs, the
// next V while Q K^T does, and a second CTA on the SM fills the rest.
//
// Three bf16 or two tf32 parts of every factor on the tensor cores would give
// fp32's accuracy too, at 6 or 3 products; for the few rows of a decode or
// verify block that is no less time than this.
#include <math.h>

#include "mma_sync.cuh"
#include "paged_tc.cuh"

namespace dfl {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBN = 64;
constexpr int kMaxTiles = (1 << 20) / kBN;

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread's copies have landed.
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int BM, int HDP>
struct F32Shape {
  static constexpr int LD = HDP + 4;          // row stride: 16-byte loads of 8 rows touch all banks
  static constexpr int kQ = 0, kK = BM * LD, kV = kK + kBN * LD, kP = kV + kBN * LD, kPos = kP + BM * (kBN + 4), kRow = kPos + kBN, kEnd = kRow + 2 * kBN;
  static constexpr size_t kSmem = (size_t)kEnd * 4 + 2 * (kMaxTiles / 32 + 1) * 4;
};

template <int BM, int TM, int HDP>
__global__ void __launch_bounds__(BM / TM * 16, HDP > 128 || BM > 32 ? 1 : 2) paged_attn_f32_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = F32Shape<BM, HDP>;
  constexpr int NT = BM / TM * 16, LD = C::LD, NJ = HDP / 64;
  extern __shared__ __align__(16) float smf[];
  float *sq = smf + C::kQ, *sk = smf + C::kK, *sv = smf + C::kV, *sp = smf + C::kP;
  int* spos = reinterpret_cast<int*>(smf + C::kPos);
  int* srow = reinterpret_cast<int*>(smf + C::kRow);      // [2][kBN] places of a tile's rows, -1 for none
  unsigned* some = reinterpret_cast<unsigned*>(smf + C::kEnd);
  unsigned* all = some + kMaxTiles / 32 + 1;
  __shared__ PagedTile st;
  __shared__ int s_qmin, s_qmax;
  pdl_enter();
  const PagedView& c = a.c;
  const int h = blockIdx.y, z = blockIdx.z, G = a.G, hd = c.hd;
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
  const int r0 = t.tile * BM, n_rows = min(BM, t.count * G - r0);
  // rows of Q, zeros past hd and past the last
  constexpr int kChunks = HDP / 4;
  for (int e = threadIdx.x; e < BM * kChunks; e += NT) {
    const int r = e / kChunks, d = e % kChunks * 4;
    const bool in = r < n_rows && d < hd;
    const float* src = static_cast<const float*>(a.q);
    if (in) src += (size_t)(t.first + (r0 + r) / G) * a.q_stride + (size_t)(h * G + (r0 + r) % G) * hd + d;
    cp_async16(sq + r * LD + d, src, in);
  }
  cp_commit();
  paged_classify<kBN>(c, t.seq, h, len, m, s_qmin, s_qmax, sh.t0, sh.t1, some, all);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  int pq[TM];
  PagedSees sees[TM];
  float slope2[TM], mx[TM], sum[TM];
  uint64_t o[TM][NJ * 2];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = r0 + min(ty * TM + i, n_rows - 1);
    pq[i] = a.q_pos[t.first + r / G];
    sees[i] = paged_sees_of(m, pq[i]);
    slope2[i] = a.slopes ? a.slopes[h * G + r % G] * kLog2e : 0.f;
    mx[i] = -INFINITY;
    sum[i] = 0.f;
#pragma unroll
    for (int d = 0; d < NJ * 2; ++d) o[i][d] = 0;
  }
  // a score in log2 units: dot * scale2, or cap2 * tanh(dot * scale2)
  const float scale2 = a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e, cap2 = a.softcap * kLog2e;
  __syncthreads();
  paged_take(sh, some, z, a.splits);
  PagedCursor cur(some, sh);

  // thread e copies 16 bytes e % kChunks of rows e / kChunks, + NT / kChunks, ..
  static_assert(NT % kChunks == 0, "whole rows at a time");
  constexpr int kStep = NT / kChunks, kRows = kBN / kStep;
  const int lr = threadIdx.x / kChunks, ld = threadIdx.x % kChunks * 4;
  const bool cols = ld < hd;
  auto find = [&](int* rows, int tile) {
    if (threadIdx.x < kBN) {
      const int slot = tile * kBN + threadIdx.x;
      rows[threadIdx.x] = slot < len ? (int)paged_row(c, t.seq, h, slot) : -1;
    }
  };
  auto copy = [&](float* dst, const void* base, const int* rows) {
    const float* src = static_cast<const float*>(base) + ld;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int j = lr + i * kStep, row = rows[j];
      const bool in = row >= 0 && cols;
      cp_async16(dst + j * LD + ld, src + (in ? (long long)row * hd : 0ll), in);
    }
    cp_commit();
  };
  int rel = cur.next(), buf = 0;
  if (rel >= 0) find(srow, sh.t0 + rel);
  __syncthreads();
  if (rel >= 0) copy(sk, c.k, srow);
  for (; rel >= 0; buf ^= 1) {
    const bool full = (all[rel >> 5] >> (rel & 31)) & 1u;
    const int next = cur.next();
    const int* rows = srow + buf * kBN;
    copy(sv, c.v, rows);
    if (threadIdx.x < kBN && (!full || a.slopes)) {
      const int row = rows[threadIdx.x];
      spos[threadIdx.x] = row >= 0 ? c.pos[row] : kPagedNoPos;
    }
    if (next >= 0) find(srow + (buf ^ 1) * kBN, sh.t0 + next);
    cp_wait<1>();                            // K
    __syncthreads();
    uint64_t s2[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = 0;
#pragma unroll 8
    for (int d = 0; d < HDP; d += 4) {
      ulonglong2 q[TM], k[4];
#pragma unroll
      for (int i = 0; i < TM; ++i) q[i] = *reinterpret_cast<const ulonglong2*>(sq + (ty * TM + i) * LD + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 16 * j) * LD + d);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s2[i][j] = fma2(q[i].x, k[j].x, s2[i][j]);
          s2[i][j] = fma2(q[i].y, k[j].y, s2[i][j]);
        }
    }
    __syncthreads();                         // K is free
    if (next >= 0) copy(sk, c.k, srow + (buf ^ 1) * kBN);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      unsigned seen = 0;
      float s[4], top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x, y;
        unpack2(s2[i][j], x, y);
        float u = (x + y) * scale2;
        if (a.softcap > 0.f) u = cap2 * tanhf(u);
        bool v = true;
        if (!full || a.slopes) {
          const int pk = spos[tx + 16 * j];
          v = full || paged_sees(sees[i], pk);
          if (a.slopes) u -= slope2[i] * fabsf((float)(pq[i] - pk));
        }
        s[j] = v ? u : -INFINITY;
        seen |= (unsigned)v << j;
        top = fmaxf(top, s[j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(mx[i], top);
      const float base = mn == -INFINITY ? 0.f : mn;
      float add = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[j] - base);
        add += p;
        // a hidden row's weight is -0, a seen one's that underflowed +0
        sp[(ty * TM + i) * (kBN + 4) + tx + 16 * j] = (seen >> j) & 1u ? p : -0.f;
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) add += __shfl_xor_sync(0xffffffffu, add, x);
      if (mn != mx[i]) {
        const float f = exp2f(mx[i] - base);
        sum[i] *= f;
        mx[i] = mn;
        const uint64_t f2 = pack2(f, f);
#pragma unroll
        for (int d = 0; d < NJ * 2; ++d) o[i][d] = fma2(o[i][d], f2, 0);
      }
      sum[i] += add;
    }
    if (next >= 0) cp_wait<1>();             // V; the next K stays in flight
    else cp_wait<0>();
    __syncthreads();
    // infinite or NaN values of V in a tile that some query sees only in part:
    // its hidden rows must not be multiplied by their zero weight
    bool careful = false;
    if (!full) {
      bool bad = false;
      for (int e = threadIdx.x; e < kBN * kChunks; e += NT) {
        const float4 v = *reinterpret_cast<const float4*>(sv + e / kChunks * LD + e % kChunks * 4);
        bad = bad || !(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))) <= 3.4028234663852886e38f) || v.x != v.x || v.y != v.y ||
              v.z != v.z || v.w != v.w;
      }
      careful = __syncthreads_or(bad);
    }
    if (!careful) {
#pragma unroll 4
      for (int j = 0; j < kBN; j += 4) {
        float4 p[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (ty * TM + i) * (kBN + 4) + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          ulonglong2 v[NJ];
#pragma unroll
          for (int n = 0; n < NJ; ++n) v[n] = *reinterpret_cast<const ulonglong2*>(sv + (j + jj) * LD + n * 64 + tx * 4);
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const float w = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
            const uint64_t w2 = pack2(w, w);
#pragma unroll
            for (int n = 0; n < NJ; ++n) {
              o[i][n * 2] = fma2(w2, v[n].x, o[i][n * 2]);
              o[i][n * 2 + 1] = fma2(w2, v[n].y, o[i][n * 2 + 1]);
            }
          }
        }
      }
    } else {
      for (int j = 0; j < kBN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const float w = sp[(ty * TM + i) * (kBN + 4) + j];
          if (__float_as_uint(w) == 0x80000000u) continue;
          const uint64_t w2 = pack2(w, w);
#pragma unroll
          for (int n = 0; n < NJ; ++n) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sv + j * LD + n * 64 + tx * 4);
            o[i][n * 2] = fma2(w2, v.x, o[i][n * 2]);
            o[i][n * 2 + 1] = fma2(w2, v.y, o[i][n * 2 + 1]);
          }
        }
    }
    __syncthreads();                         // V, P and the positions are free
    rel = next;
  }
  cp_wait<0>();
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = ty * TM + i;
    if (r >= n_rows) continue;
    const size_t at = (size_t)(t.first + (r0 + r) / G) * a.nq + h * G + (r0 + r) % G;
    const bool none = sum[i] == 0.f;         // nothing seen (a NaN score makes the sum NaN)
    const bool split = a.splits > 1;
    const float inv = none ? 0.f : (split ? 1.f : 1.f / sum[i]);
    float* out = split ? a.part_o + ((size_t)z * a.rows * a.nq + at) * hd : static_cast<float*>(a.out) + at * hd;
#pragma unroll
    for (int n = 0; n < NJ; ++n) {
      float4 v;
      unpack2(o[i][n * 2], v.x, v.y);
      unpack2(o[i][n * 2 + 1], v.z, v.w);
      if (n * 64 + tx * 4 < hd)
        *reinterpret_cast<float4*>(out + n * 64 + tx * 4) =
            none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    }
    if (tx) continue;
    if (split) a.part_ml[(size_t)z * a.rows * a.nq + at] = make_float2(mx[i], sum[i]);
    else if (a.lse) a.lse[at] = none ? -INFINITY : (mx[i] + log2f(sum[i])) * kLn2;
  }
}

template <int BM, int TM, int HDP>
cudaError_t run(const PagedAttnArgs& a, dim3 grid, cudaStream_t st) {
  auto kernel = paged_attn_f32_kernel<BM, TM, HDP>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F32Shape<BM, HDP>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(BM / TM * 16), F32Shape<BM, HDP>::kSmem, st, a);
}
template <int BM, int TM>
cudaError_t run_hd(const PagedAttnArgs& a, dim3 grid, cudaStream_t st) {
  if (a.c.hd <= 64) return run<BM, TM, 64>(a, grid, st);
  if (a.c.hd <= 128) return run<BM, TM, 128>(a, grid, st);
  return run<BM, TM, 256>(a, grid, st);
}

}  // namespace

cudaError_t launch_paged_attention_f32(const PagedAttnArgs& a, int tile_rows, long long tiles, cudaStream_t st) {
  const dim3 grid((unsigned)tiles, a.c.nkv, a.splits);
  if (tile_rows == 16) return run_hd<16, 2>(a, grid, st);
  if (tile_rows == 32) return run_hd<32, 4>(a, grid, st);
  return run_hd<64, 4>(a, grid, st);
}

}  // namespace dfl
