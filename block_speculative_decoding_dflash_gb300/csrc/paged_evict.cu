// Eviction from the paged cache by weight.
//
// The kept rows are those of the `budget` largest keys, where a row's key is
// its weight in an unsigned order (larger weight, larger key; NaN 0; a
// protected row the key of +infinity) and equal keys prefer the lower row. A
// radix select finds the key of rank `budget` (8 bits at a time, from the
// top); a second pass over the rows ranks the holes below the budget and the
// kept rows beyond it; a second kernel moves the j-th of these into the j-th
// of those. Sources lie at or beyond row `budget` and destinations below it,
// so the moves are independent, and nothing that stays is touched.
#include <math.h>

#include "paged.cuh"

namespace dfl {

namespace {

constexpr int kSelThreads = 1024;

__device__ __forceinline__ unsigned weight_key(float w, bool keep) {
  if (keep) w = INFINITY;
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);            // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);      // -inf 0x007fffff, +inf 0xff800000
}

// Exclusive block-wide prefix sums of two counts; total in tot.
__device__ __forceinline__ int2 block_scan2(int2 v, int2* warps, int2* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) { x.x += a; x.y += b; }
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int2 w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, w.x, o), b = __shfl_up_sync(0xffffffffu, w.y, o);
      if (lane >= o) { w.x += a; w.y += b; }
    }
    warps[lane] = w;
  }
  __syncthreads();
  const int2 before = warp ? warps[warp - 1] : make_int2(0, 0);
  *tot = warps[31];
  __syncthreads();
  return make_int2(before.x + x.x - v.x, before.y + x.y - v.y);
}

// One CTA to a (sequence, kv head).
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(PagedEvictArgs a) {
  pdl_enter();
  const PagedView& c = a.c;
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  int* list = a.moves + ((size_t)s * c.nkv + h) * (1 + 2 * (size_t)a.max_moves);
  const int n = paged_length(c, s), b = a.budget;
  const long long guard = (long long)a.next_pos[s] - a.recent;
  __shared__ int hist[256];
  __shared__ int2 warps[32];
  __shared__ unsigned s_prefix;
  __shared__ int s_left;
  if (tid == 0 && h == 0 && c.status && c.length[s] != n) atomicOr(c.status, DFLASH_PAGED_BAD_ROWS);
  unsigned prefix = 0;                       // the key's known top bits
  int left = b;                              // rows still to take among those with that prefix
  if (n > b) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kSelThreads) {
        const long long row = paged_row(c, s, h, i);
        const unsigned k = row < 0 ? 0u : weight_key(a.weight[row], c.pos[row] >= guard);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255, take = left;
        while (d > 0 && hist[d] < take) take -= hist[d--];
        s_prefix = prefix | ((unsigned)d << shift);
        s_left = take;
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_left;
    }
  }
  // prefix is the key of rank b: greater keys stay, of the equal ones the
  // first `left`
  int equal = 0, holes = 0, late = 0;
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const long long row = i < n ? paged_row(c, s, h, i) : -1;
    const float w = row >= 0 ? a.weight[row] : 0.f;
    const int pos = row >= 0 ? c.pos[row] : 0;
    if (i < n && row < 0 && c.status) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
    bool kept = i < n;
    if (n > b) {
      const unsigned k = row < 0 ? 0u : weight_key(w, pos >= guard);
      int2 tot;
      const int2 e = block_scan2(make_int2(i < n && k == prefix, 0), warps, &tot);
      kept = i < n && (k > prefix || (k == prefix && equal + e.x < left));
      equal += tot.x;
      const int2 r = block_scan2(make_int2(i < n && i < b && !kept, kept && i >= b), warps, &tot);
      if (i < n && i < b && !kept && holes + r.x < a.max_moves) list[1 + holes + r.x] = i;
      if (kept && i >= b && late + r.y < a.max_moves) list[1 + a.max_moves + late + r.y] = i;
      holes += tot.x;
      late += tot.y;
    }
    if (kept && i < b && row >= 0) {
      if (a.weight_out != a.weight) a.weight_out[row] = w;
      if (a.pos_out != c.pos) a.pos_out[row] = pos;
    }
  }
  if (tid == 0) list[0] = holes < a.max_moves ? holes : a.max_moves;
}

// A warp to a move: 16-byte pieces of the K and V rows, position and weight.
template <int ES>
__global__ void __launch_bounds__(256) paged_move_kernel(PagedEvictArgs a) {
  pdl_enter();
  const PagedView& c = a.c;
  const int h = blockIdx.y, s = blockIdx.z, lane = threadIdx.x & 31;
  const int* list = a.moves + ((size_t)s * c.nkv + h) * (1 + 2 * (size_t)a.max_moves);
  const int count = list[0], bytes = c.hd * ES;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    const int n = paged_length(c, s);
    a.length_out[s] = n < a.budget ? n : a.budget;
  }
  for (int j = blockIdx.x * 8 + (threadIdx.x >> 5); j < count; j += gridDim.x * 8) {
    const long long to = paged_row(c, s, h, list[1 + j]), of = paged_row(c, s, h, list[1 + a.max_moves + j]);
    if (to < 0 || of < 0) continue;
    for (int i = lane * 16; i < 2 * bytes; i += 512) {
      char* base = static_cast<char*>(i < bytes ? c.k : c.v);
      const int o = i < bytes ? i : i - bytes;
      *reinterpret_cast<uint4*>(base + to * bytes + o) = *reinterpret_cast<const uint4*>(base + of * bytes + o);
    }
    if (lane == 0) {
      a.weight_out[to] = a.weight[of];
      a.pos_out[to] = c.pos[of];
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(int dtype, const PagedEvictArgs& a, cudaStream_t st) {
  cudaError_t e = launch_pdl(paged_select_kernel, dim3(a.c.nkv, a.c.n_seq), dim3(kSelThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  int x = (a.max_moves + 7) / 8;
  if (x > 256) x = 256;
  if (x < 1) x = 1;
  const dim3 grid(x, a.c.nkv, a.c.n_seq);
  return dtype ? launch_pdl(paged_move_kernel<2>, grid, dim3(256), 0, st, a)
               : launch_pdl(paged_move_kernel<4>, grid, dim3(256), 0, st, a);
}

}  // namespace dfl
