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

constexpr int kWarps = 4;

// (cos, sin) of pair i at the new row's position.
__device__ __forceinline__ float2 turn(const PagedAppendArgs& a, int i, int tok) {
  const long long p = a.rope_pos[(size_t)a.axis[i] * a.rows + tok];
  const int half_turns = (int)(((unsigned long long)p * a.freq[i]) >> 32);   // of 2^31
  float s, c;
  sincospif((float)half_turns * 4.656612873077393e-10f, &s, &c);
  return make_float2(c, s);
}

// Where a new row goes: its sequence and slot; called by one full warp.
struct NewRow { int seq, slot; };
__device__ __forceinline__ NewRow new_row(const PagedAppendArgs& a, int tok, bool report) {
  const PagedView& c = a.c;
  const int first = max(0, a.start[0]);
  if (tok < first) return NewRow{-1, 0};
  const PagedTile t = paged_find_tile(a.start, c.n_seq, a.rows, 1, 1, tok - first);
  if (t.seq < 0 || t.first + t.tile != tok) return NewRow{-1, 0};
  const int len = paged_length(c, t.seq), slot = len - (t.count - t.tile);
  if (report && c.status && (threadIdx.x & 31) == 0) {
    if (slot < 0 || c.length[t.seq] != len) atomicOr(c.status, DFLASH_PAGED_BAD_ROWS);
    else if (paged_row(c, t.seq, 0, slot) < 0) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
  }
  return NewRow{t.seq, slot};
}

// Head x of a new row, counted over q, then k, then v: where it is read and
// written, and what it is (0 q, 1 k, 2 v); dst NULL where it has no place.
template <typename T>
struct HeadPtr { const T* src; T* dst; int kind; };
template <typename T>
__device__ __forceinline__ HeadPtr<T> head_ptr(const PagedAppendArgs& a, const NewRow& r, int tok, int x, bool first_lane) {
  const PagedView& c = a.c;
  const int hd = c.hd;
  if (x < a.nq)
    return {static_cast<const T*>(a.q) + (long long)tok * a.q_stride + (size_t)x * hd, static_cast<T*>(a.q_out) + ((size_t)tok * a.nq + x) * hd, 0};
  const int kind = x < a.nq + c.nkv ? 1 : 2, h = x - a.nq - (kind == 2 ? c.nkv : 0);
  const long long row = r.slot >= 0 ? paged_row(c, r.seq, h, r.slot) : -1;
  const T* src = kind == 1 ? static_cast<const T*>(a.k) + (long long)tok * a.k_stride + (size_t)h * hd
                           : static_cast<const T*>(a.v) + (long long)tok * a.v_stride + (size_t)h * hd;
  if (row < 0) return {src, nullptr, kind};
  if (kind == 1 && first_lane) {
    c.pos[row] = a.row_pos[tok];
    if (a.weight) a.weight[row] = 0.f;
  }
  return {src, static_cast<T*>(kind == 1 ? c.k : c.v) + row * hd, kind};
}

__device__ __forceinline__ void store8(bf16* p, const float* v) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A warp takes `per_warp` heads of one new row. A head lies in hd / 8 lanes, 8
// dimensions to each (16-byte accesses), so 32 / (hd / 8) heads are worked on
// side by side; the lane keeps its dimensions' (cos, sin) in registers for
// all of them, and a rotated pair's other half is in the same
// lane (adjacent pairs) or one shuffle away. kU heads are requested before the
// first is used. Bound by the bytes of the rows, read once and written once.
// Needs pairs to fill whole lanes: a multiple of 8 (neox) or 4.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 5) paged_append_kernel(const __grid_constant__ PagedAppendArgs a, int per_warp, int splits) {
  constexpr int kU = 4;
  pdl_enter();
  const PagedView& c = a.c;
  const int lane = threadIdx.x & 31, hd = c.hd;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int tok = (int)(item / splits), part = (int)(item % splits);
  if (tok >= a.rows) return;
  const NewRow r = new_row(a, tok, part == 0);
  if (r.seq < 0) return;
  const int lpr = hd >> 3, side = 32 / lpr;               // lanes of a head, heads side by side
  const int sub = lane / lpr, l = lane - sub * lpr, d0 = l * 8;
  const bool in = sub < side;
  // this lane's rotation: own = v * cs + other * sn
  float cs[8], sn[8];
  int other = lane;                                       // lane that holds the pairs' other halves
  if (a.neox) {
    const int pl = a.pairs >> 3;                          // lanes of the first halves
    const bool lo = l < pl, hi = !lo && l < 2 * pl;
    other = lo ? lane + pl : (hi ? lane - pl : lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 t = in && (lo || hi) ? turn(a, (lo ? d0 : d0 - a.pairs) + j, tok) : make_float2(1.f, 0.f);
      cs[j] = t.x;
      sn[j] = lo ? -t.y : t.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 t = in && d0 < 2 * a.pairs ? turn(a, (d0 >> 1) + j, tok) : make_float2(1.f, 0.f);
      cs[2 * j] = cs[2 * j + 1] = t.x;
      sn[2 * j] = -t.y;
      sn[2 * j + 1] = t.y;
    }
  }
  const int heads = a.nq + 2 * c.nkv, x1 = min(heads, (part + 1) * per_warp);
  for (int x0 = part * per_warp; x0 < x1; x0 += side * kU) {
    HeadPtr<T> p[kU];
    float v[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int x = x0 + u * side + sub;
      p[u] = HeadPtr<T>{nullptr, nullptr, 2};
      if (in && x < x1) p[u] = head_ptr<T>(a, r, tok, x, l == 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
      if (p[u].dst) load8(p[u].src + d0, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const T* gain = static_cast<const T*>(p[u].kind == 0 ? a.q_norm : p[u].kind == 1 ? a.k_norm : nullptr);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[u][j], v[u][j], ss);
      // the sum over the head's lanes: every lane adds all of them in order of
      // a tree that needs no power of two
      float tot = ss;
      if ((lpr & (lpr - 1)) == 0) {
        for (int o = lpr >> 1; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
      } else {
        tot = 0.f;
        for (int o = 0; o < lpr; ++o) tot += __shfl_sync(0xffffffffu, ss, in ? sub * lpr + o : lane);
      }
      if (in && gain) {
        const float rs = 1.0f / sqrtf(tot / (float)hd + a.eps);
        float g[8];
        load8(gain + d0, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] *= rs * g[j];
      }
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = a.neox ? __shfl_sync(0xffffffffu, v[u][j], other) : v[u][j ^ 1];
      if (p[u].kind != 2)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] = fmaf(v[u][j], cs[j], w[j] * sn[j]);
      if (p[u].dst) store8(p[u].dst + d0, v[u]);
    }
  }
}

// Any number of pairs: a warp to a head, one value to a lane at a time, the
// rotation through shared memory.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) paged_append_any_kernel(const __grid_constant__ PagedAppendArgs a) {
  __shared__ float2 cs[kPagedMaxPairs];
  __shared__ float row[kWarps][256];
  __shared__ NewRow s_row;
  pdl_enter();
  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hd = c.hd, tok = blockIdx.x;
  if (warp == 0) {
    const NewRow r = new_row(a, tok, true);
    if (lane == 0) s_row = r;
  }
  for (int i = threadIdx.x; i < a.pairs; i += blockDim.x) cs[i] = turn(a, i, tok);
  __syncthreads();
  const NewRow r = s_row;
  if (r.seq < 0) return;
  for (int x = warp; x < a.nq + 2 * c.nkv; x += kWarps) {
    const HeadPtr<T> p = head_ptr<T>(a, r, tok, x, lane == 0);
    if (!p.dst) continue;
    float ss = 0.f;
    for (int d = lane; d < hd; d += 32) {
      const float v = to_f(p.src[d]);
      row[warp][d] = v;
      ss = fmaf(v, v, ss);
    }
    const T* gain = static_cast<const T*>(p.kind == 0 ? a.q_norm : p.kind == 1 ? a.k_norm : nullptr);
    if (gain) {
      const float rs = 1.0f / sqrtf(warp_sum(ss) / (float)hd + a.eps);
      for (int d = lane; d < hd; d += 32) row[warp][d] *= rs * to_f(gain[d]);
    }
    __syncwarp();
    if (p.kind != 2)
      for (int i = lane; i < a.pairs; i += 32) {
        const int d0 = a.neox ? i : 2 * i, d1 = a.neox ? i + a.pairs : 2 * i + 1;
        const float v0 = row[warp][d0], v1 = row[warp][d1];
        row[warp][d0] = v0 * cs[i].x - v1 * cs[i].y;
        row[warp][d1] = v1 * cs[i].x + v0 * cs[i].y;
      }
    __syncwarp();
    for (int d = lane; d < hd; d += 32) p.dst[d] = from_f<T>(row[warp][d]);
    __syncwarp();
  }
}

template <typename T>
cudaError_t run(const PagedAppendArgs& a, cudaStream_t st) {
  if (a.pairs % (a.neox ? 8 : 4)) return launch_pdl(paged_append_any_kernel<T>, dim3(a.rows), dim3(kWarps * 32), 0, st, a);
  // as many warps to a row as fill the GPU (32 warps on each of 152 SMs), each
  // with one round of heads at least: the rotation's sines are computed once a
  // warp
  const int heads = a.nq + 2 * a.c.nkv, side = 32 / (a.c.hd >> 3);
  int splits = (int)(4864 / (a.rows < 4864 ? a.rows : 4864));
  const int most = (heads + side - 1) / side;
  if (splits > most) splits = most;
  const int per_warp = (heads + splits - 1) / splits;
  splits = (heads + per_warp - 1) / per_warp;
  const long long warps = (long long)a.rows * splits;
  return launch_pdl(paged_append_kernel<T>, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, st, a, per_warp, splits);
}

}  // namespace

cudaError_t launch_paged_append(int dtype, const PagedAppendArgs& a, cudaStream_t st) {
  return dtype ? run<bf16>(a, st) : run<float>(a, st);
}

}  // namespace dfl
