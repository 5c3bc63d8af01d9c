// Append to the paged cache: per-head RMSNorm of q and k, rotation by one or
// several position axes, K and V into their pages.
//
// The angle of pair i at position p is p * theta^(-i / pairs). The host gives
// the frequency in turns as a fraction of 2^64, so p * freq mod 2^64 is the
// angle's fraction of a turn, exact to p * 2^-55 turns at any distance: no
// 64-bit floating point, whose rate on this GPU is far below fp32's, and no
// argument reduction.
#include <math.h>

#include "paged.cuh"

namespace dfl {

namespace {

constexpr int kWarps = 8;

// One CTA to a new row and a share of its heads: the row's (cos, sin) once
// into shared memory, then a warp to each head of q, k and v in turn.
// Bound by the bytes of the rows, read once and written once.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  __shared__ float2 cs[kPagedMaxPairs];
  __shared__ int s_seq;
  pdl_enter();
  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hd = c.hd, tok = blockIdx.x;
  if (warp == 0) {
    const PagedTile t = paged_find_tile(a.start, c.n_seq, a.rows, 1, 1, tok - max(0, a.start[0]));
    if (lane == 0) s_seq = (tok >= a.start[0] && t.seq >= 0 && t.first + t.tile == tok) ? t.seq : -1;
  }
  for (int i = threadIdx.x; i < a.pairs; i += blockDim.x) {
    const long long p = a.rope_pos[(size_t)a.axis[i] * a.rows + tok];
    const int half_turns = (int)(((unsigned long long)p * a.freq[i]) >> 32);   // of 2^31
    float s, co;
    sincospif((float)half_turns * 4.656612873077393e-10f, &s, &co);
    cs[i] = make_float2(co, s);
  }
  __syncthreads();
  const int seq = s_seq;
  if (seq < 0) return;
  const int2 ab = paged_new_rows(a.start, seq, a.rows);
  const int len = paged_length(c, seq), slot = len - (ab.y - tok);
  const bool cached = slot >= 0;
  if (threadIdx.x == 0 && blockIdx.y == 0 && c.status) {
    if (!cached || c.length[seq] != len) atomicOr(c.status, DFLASH_PAGED_BAD_ROWS);
    else if (paged_row(c, seq, 0, slot) < 0) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
  }
  const int heads = a.nq + 2 * c.nkv;
  for (int x = blockIdx.y * kWarps + warp; x < heads; x += gridDim.y * kWarps) {
    const int kind = x < a.nq ? 0 : (x < a.nq + c.nkv ? 1 : 2);
    const int h = kind == 0 ? x : (kind == 1 ? x - a.nq : x - a.nq - c.nkv);
    const T* src = kind == 0 ? static_cast<const T*>(a.q) + (long long)tok * a.q_stride + (size_t)h * hd
                 : kind == 1 ? static_cast<const T*>(a.k) + (long long)tok * a.k_stride + (size_t)h * hd
                             : static_cast<const T*>(a.v) + (long long)tok * a.v_stride + (size_t)h * hd;
    T* dst;
    if (kind == 0) {
      dst = static_cast<T*>(a.q_out) + ((size_t)tok * a.nq + h) * hd;
    } else {
      const long long row = cached ? paged_row(c, seq, h, slot) : -1;
      if (row < 0) continue;
      dst = static_cast<T*>(kind == 1 ? c.k : c.v) + row * hd;
      if (kind == 1 && lane == 0) {
        c.pos[row] = a.row_pos[tok];
        if (a.weight) a.weight[row] = 0.f;
      }
    }
    // up to 256 dims: 8 to a lane, in registers
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < 8; ++j) {
      const int d = lane + 32 * j;
      if (d < hd) v[j] = to_f(src[d]);
    }
    if (kind == 2) {
      for (int j = 0; j < 8; ++j)
        if (lane + 32 * j < hd) dst[lane + 32 * j] = from_f<T>(v[j]);
      continue;
    }
    const T* gain = static_cast<const T*>(kind == 0 ? a.q_norm : a.k_norm);
    if (gain) {
      float ss = 0.f;
      for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
      const float r = 1.0f / sqrtf(warp_sum(ss) / (float)hd + a.eps);
      for (int j = 0; j < 8; ++j)
        if (lane + 32 * j < hd) v[j] = v[j] * r * to_f(gain[lane + 32 * j]);
    }
    __shared__ float row[kWarps][256];
    for (int j = 0; j < 8; ++j) row[warp][lane + 32 * j] = v[j];
    __syncwarp();
    for (int i = lane; i < a.pairs; i += 32) {
      const int d0 = a.neox ? i : 2 * i, d1 = a.neox ? i + a.pairs : 2 * i + 1;
      const float x0 = row[warp][d0], x1 = row[warp][d1];
      row[warp][d0] = x0 * cs[i].x - x1 * cs[i].y;
      row[warp][d1] = x1 * cs[i].x + x0 * cs[i].y;
    }
    __syncwarp();
    for (int j = 0; j < 8; ++j)
      if (lane + 32 * j < hd) dst[lane + 32 * j] = from_f<T>(row[warp][lane + 32 * j]);
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_paged_append(int dtype, const PagedAppendArgs& a, cudaStream_t st) {
  const int heads = a.nq + 2 * a.c.nkv;
  int y = (heads + kWarps - 1) / kWarps;
  if ((long long)a.rows * y > 4096) y = (int)(4096 / a.rows > 1 ? 4096 / a.rows : 1);
  const dim3 grid(a.rows, y);
  return dtype ? launch_pdl(paged_append_kernel<bf16>, grid, dim3(kWarps * 32), 0, st, a)
               : launch_pdl(paged_append_kernel<float>, grid, dim3(kWarps * 32), 0, st, a);
}

}  // namespace dfl
