// Append to the paged cache: per-head RMSNorm of q and k, rotation by one or
// several position axes, K and V into their pages.
//
// The angle of pair i at position p is p * theta^(-i / pairs). The host gives
// the frequency in turns as a fraction of 2^64, so p * freq mod 2^64 is the
// angle's fraction of a turn, exact to p * 2^-55 turns at any distance: no
// 64-bit floating point, whose rate on this GPU is far below fp32's, and no
// argument reduction. Of the fraction the upper 32 bits are kept and rounded to
// fp32's 24: 2^-25 of half a turn at most, 1e-7 in the angle, as much as a sine's
// own rounding (fp32 rows against fp64: 7.3e-8 of the norm, with angles in 64 bits
// 7.0e-8).
//
// Bound by the HBM for long prompts (16384 rows of 48 heads: 80 us, 5.0 TB/s), by
// the launch and one chain of loads for short ones (16 rows: 4.8 us in a graph).
#include <math.h>

#include "paged_tc.cuh"

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

// 8 values of a head as they lie in memory.
template <typename T>
struct Raw8 {
  static constexpr int kWords = sizeof(T) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
      w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
  __device__ __forceinline__ float at(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(w[i % kWords]);
    return i & 1 ? bf_hi(w[i >> 1]) : bf_lo(w[i >> 1]);
  }
};
__device__ __forceinline__ Raw8<bf16> round8(const float* v, bf16) {
  Raw8<bf16> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return r;
}
__device__ __forceinline__ Raw8<float> round8(const float* v, float) {
  Raw8<float> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
  return r;
}

// A warp takes heads [x0, x1) of one new row, counted over q, then k, then v.
// A head lies in hd / 8 lanes, 8 dimensions to each (16-byte accesses), so
// 32 / (hd / 8) heads are worked on side by side. With r the head's 1 / rms,
// a value becomes r (v A + w B): w the pair's other half, in the same lane
// (adjacent pairs) or one shuffle away, A and B the gains times cos and sin,
// which a lane holds for its dimensions. kU heads are requested before the first
// is used, and the next ones as soon as one is in its registers. PART: only a part
// of the dimensions is rotated; the other lanes take w = +0 and B = -0, which
// leaves v A as it is to the sign of a zero, whatever its neighbours hold (in
// every lane's code this costs 4096 rows of heads of 96 dimensions 1 us of 33).
// Bound by the bytes of the rows, read once and written once, for thousands of
// rows; by its chain of dependent loads for a few.
// Needs pairs to fill whole lanes: a multiple of 8 (NEOX) or 4. LPR: hd / 8
// where it is 8 or 16 (head_dim 64 and 128), else 0.
constexpr int kU = 2;
template <typename T, int LPR, bool NEOX, bool PART>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 6 : 5) paged_append_kernel(const __grid_constant__ PagedAppendArgs a, int per_warp, int splits) {
  pdl_enter();
  const PagedView& c = a.c;
  const int lane = threadIdx.x & 31, nq = a.nq, nkv = c.nkv;
  const int hd = LPR ? LPR * 8 : c.hd, lpr = hd >> 3, side = 32 / lpr;   // lanes of a head, heads side by side
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int tok = (int)(item / splits), part = (int)(item % splits);
  if (tok >= a.rows) return;
  const int x0 = part * per_warp, x1 = min(nq + 2 * nkv, x0 + per_warp);
  const int sub = lane / lpr, l = lane - sub * lpr, d0 = l * 8;
  const bool in = LPR || sub < side;
  const int step = side * hd;                             // elements between a lane's heads
  const T* qs = static_cast<const T*>(a.q) + (long long)tok * a.q_stride + (size_t)(x0 + sub) * hd + d0;
  Raw8<T> raw[kU];
  const int q_left = min(x1, nq) - x0;                    // q heads of this warp
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (in && u * side + sub < q_left) raw[u].load(qs + u * step);
  // the row's (cos, sin), two pairs or more to a lane, then this lane's
  __shared__ __align__(16) float2 table[kWarps][kPagedMaxPairs];
  float2* tab = table[threadIdx.x >> 5];
  for (int i = lane; i < a.pairs; i += 32) tab[i] = turn(a, i, tok);
  __syncwarp();
  int other = lane, od = d0, pair = -1;                   // where the pairs' other halves are; first pair of the lane
  bool second = false;                                    // the lane holds second halves
  if (NEOX) {
    const int pl = a.pairs >> 3;                          // lanes of the first halves
    second = l >= pl;
    if (l < 2 * pl) {
      other = second ? lane - pl : lane + pl;
      od = second ? d0 - a.pairs : d0 + a.pairs;
      pair = second ? od : d0;
    }
  } else if (d0 < 2 * a.pairs) {
    pair = d0 >> 1;
  }
  const uint32_t turns = !PART || pair >= 0 ? ~0u : 0u;   // keeps or clears the pairs' other halves
  Raw8<T> g_own, g_oth;                                   // the gains, requested before they are needed
  auto get_gain = [&](const void* g) {
    if (g && in) {
      g_own.load(static_cast<const T*>(g) + d0);
      if (NEOX) g_oth.load(static_cast<const T*>(g) + od);
    }
  };
  get_gain(q_left > 0 ? a.q_norm : a.k_norm);
  NewRow r{-1, -1};
  if (x1 > nq) {
    r = new_row(a, tok, x1 == nq + 2 * nkv);
    if (r.seq < 0) return;
  } else if (tok < a.start[0] || tok >= a.start[c.n_seq]) {
    return;
  }

  uint64_t A[4], B[4];
  bool norm;
  auto use_gain = [&](const void* g) {
    norm = g != nullptr;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float2 t0 = make_float2(1.f, 0.f), t1 = t0;
      if (in && pair >= 0) {
        t0 = tab[pair + (NEOX ? j : j >> 1)];
        t1 = NEOX ? tab[pair + j + 1] : t0;
      }
      float b0 = (NEOX ? second : false) ? t0.y : -t0.y, b1 = (NEOX ? second : true) ? t1.y : -t1.y;
      if (norm && in) {
        t0.x *= g_own.at(j);
        t1.x *= g_own.at(j + 1);
        b0 *= NEOX ? g_oth.at(j) : g_own.at(j + 1);
        b1 *= NEOX ? g_oth.at(j + 1) : g_own.at(j);
      }
      if (PART && pair < 0) b0 = b1 = -0.f;
      A[j >> 1] = pack2(t0.x, t1.x);
      B[j >> 1] = pack2(b0, b1);
    }
  };
  const float inv_hd = 1.f / (float)hd;
  // x turned; `next` is called as soon as x's registers are free
  auto turned = [&](Raw8<T>& x, auto next) {
    uint64_t v[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack2(x.at(2 * j), x.at(2 * j + 1));
    Raw8<T> y;
#pragma unroll
    for (int j = 0; j < Raw8<T>::kWords; ++j) y.w[j] = (NEOX ? __shfl_sync(0xffffffffu, x.w[j], other) : x.w[j]) & turns;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = NEOX ? pack2(y.at(2 * j), y.at(2 * j + 1)) : pack2(y.at(2 * j + 1), y.at(2 * j));
    next();
    float f = 1.f;
    if (norm) {
      uint64_t s2 = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = fma2(v[j], v[j], s2);
      float s0, s1;
      unpack2(s2, s0, s1);
      float tot = s0 + s1;
      if (LPR) {
#pragma unroll
        for (int o = LPR >> 1; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
      } else {
        const float own = tot;
        tot = 0.f;
        for (int o = 0; o < lpr; ++o) tot += __shfl_sync(0xffffffffu, own, in ? sub * lpr + o : lane);
      }
      f = rsqrtf(fmaf(tot, inv_hd, a.eps));
    }
    float z[8];
    const uint64_t f2 = pack2(f, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2(mul2(fma2(v[j], A[j], mul2(w[j], B[j])), f2), z[2 * j], z[2 * j + 1]);
    return round8(z, T());
  };

  if (q_left > 0) {
    use_gain(a.q_norm);
    T* qd = static_cast<T*>(a.q_out) + ((size_t)tok * nq + x0 + sub) * hd + d0;
    int left = in ? q_left - sub : 0;                     // heads from this lane's on
    for (int x = q_left; x > 0; x -= side * kU, left -= side * kU, qs += kU * step, qd += kU * step) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (u * side >= x) break;
        const Raw8<T> y = turned(raw[u], [&] {
          if ((kU + u) * side < left) raw[u].load(qs + (kU + u) * step);
        });
        if (u * side < left) y.store(qd + u * step);
      }
    }
  }
  // k and v: consecutive heads of a row lie page_rows rows apart
  for (int kind = 1; kind <= 2; ++kind) {
    const int base = nq + (kind - 1) * nkv, h0 = max(x0, base) - base, h1 = min(x1, base + nkv) - base;
    if (h0 >= h1) continue;
    const long long row0 = r.slot >= 0 ? paged_row(c, r.seq, 0, r.slot) : -1;
    if (row0 < 0) continue;
    if (kind == 1) {
      if (q_left > 0) get_gain(a.k_norm);
      use_gain(a.k_norm);
    }
    const T* src = (kind == 1 ? static_cast<const T*>(a.k) + (long long)tok * a.k_stride : static_cast<const T*>(a.v) + (long long)tok * a.v_stride) + d0;
    T* dst = static_cast<T*>(kind == 1 ? c.k : c.v) + row0 * hd + d0;
    const size_t apart = (size_t)hd << c.lg_rows;         // elements between heads in a page
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (in && h0 + u * side + sub < h1) raw[u].load(src + (h0 + u * side + sub) * hd);
    for (int h = h0; h < h1; h += side * kU) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (h + u * side >= h1) break;
        const int hh = h + u * side + sub;
        auto next = [&] {
          if (in && hh + kU * side < h1) raw[u].load(src + (hh + kU * side) * hd);
        };
        Raw8<T> y;
        if (kind == 1) {
          y = turned(raw[u], next);
        } else {
          y = raw[u];
          next();
        }
        if (in && hh < h1) {
          y.store(dst + hh * apart);
          if (kind == 1 && l == 0) {
            const long long row = row0 + ((long long)hh << c.lg_rows);
            c.pos[row] = a.row_pos[tok];
            if (a.weight) a.weight[row] = 0.f;
          }
        }
      }
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
    const int kind = x < a.nq ? 0 : (x < a.nq + c.nkv ? 1 : 2), h = kind == 0 ? x : x - a.nq - (kind - 1) * c.nkv;
    const long long at = kind > 0 && r.slot >= 0 ? paged_row(c, r.seq, h, r.slot) : -1;
    if (kind > 0 && at < 0) continue;
    const T* src = kind == 0   ? static_cast<const T*>(a.q) + (long long)tok * a.q_stride + (size_t)h * hd
                   : kind == 1 ? static_cast<const T*>(a.k) + (long long)tok * a.k_stride + (size_t)h * hd
                               : static_cast<const T*>(a.v) + (long long)tok * a.v_stride + (size_t)h * hd;
    T* dst = kind == 0 ? static_cast<T*>(a.q_out) + ((size_t)tok * a.nq + h) * hd : static_cast<T*>(kind == 1 ? c.k : c.v) + at * hd;
    if (kind == 1 && lane == 0) {
      c.pos[at] = a.row_pos[tok];
      if (a.weight) a.weight[at] = 0.f;
    }
    float ss = 0.f;
    for (int d = lane; d < hd; d += 32) {
      const float v = to_f(src[d]);
      row[warp][d] = v;
      ss = fmaf(v, v, ss);
    }
    const T* gain = static_cast<const T*>(kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr);
    if (gain) {
      const float rs = 1.0f / sqrtf(warp_sum(ss) / (float)hd + a.eps);
      for (int d = lane; d < hd; d += 32) row[warp][d] *= rs * to_f(gain[d]);
    }
    __syncwarp();
    if (kind != 2)
      for (int i = lane; i < a.pairs; i += 32) {
        const int d0 = a.neox ? i : 2 * i, d1 = a.neox ? i + a.pairs : 2 * i + 1;
        const float v0 = row[warp][d0], v1 = row[warp][d1];
        row[warp][d0] = v0 * cs[i].x - v1 * cs[i].y;
        row[warp][d1] = v1 * cs[i].x + v0 * cs[i].y;
      }
    __syncwarp();
    for (int d = lane; d < hd; d += 32) dst[d] = from_f<T>(row[warp][d]);
    __syncwarp();
  }
}

template <typename T, int LPR>
cudaError_t run_whole(const PagedAppendArgs& a, unsigned grid, int per_warp, int splits, cudaStream_t st) {
  auto kernel = a.neox ? paged_append_kernel<T, LPR, true, false> : paged_append_kernel<T, LPR, false, false>;
  if (2 * a.pairs < a.c.hd) kernel = a.neox ? paged_append_kernel<T, LPR, true, true> : paged_append_kernel<T, LPR, false, true>;
  return launch_pdl(kernel, dim3(grid), dim3(kWarps * 32), 0, st, a, per_warp, splits);
}

template <typename T>
cudaError_t run(const PagedAppendArgs& a, cudaStream_t st) {
  if (a.pairs % (a.neox ? 8 : 4)) return launch_pdl(paged_append_any_kernel<T>, dim3(a.rows), dim3(kWarps * 32), 0, st, a);
  // as many warps to a row as fill the GPU (16 warps on each of 152 SMs), each
  // with one round of heads at least: the rotation's sines are computed once a
  // warp (16 rows: 4.8 us, with one warp to a row 9.6 us; 16384 rows have one)
  const int heads = a.nq + 2 * a.c.nkv, side = 32 / (a.c.hd >> 3);
  int splits = 2432 / (a.rows < 2432 ? a.rows : 2432);
  const int most = (heads + side - 1) / side;
  if (splits > most) splits = most;
  const int per_warp = (heads + splits - 1) / splits;
  splits = (heads + per_warp - 1) / per_warp;
  const long long warps = (long long)a.rows * splits;
  const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
  if (a.c.hd == 128) return run_whole<T, 16>(a, grid, per_warp, splits, st);
  if (a.c.hd == 64) return run_whole<T, 8>(a, grid, per_warp, splits, st);
  return run_whole<T, 0>(a, grid, per_warp, splits, st);
}

}  // namespace

cudaError_t launch_paged_append(int dtype, const PagedAppendArgs& a, cudaStream_t st) {
  return dtype ? run<bf16>(a, st) : run<float>(a, st);
}

}  // namespace dfl
