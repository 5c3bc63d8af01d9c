// Eviction from the paged cache by weight.
//
// The kept rows are those of the `budget` largest keys, where a row's key is
// its weight in an unsigned order (larger weight, larger key; NaN 0; a
// protected row the key of +infinity) and equal keys prefer the lower row. A
// radix select finds the key of rank `budget` (11, 11 and 10 bits, from the
// top); passes over the rows then rank the holes below the budget and the kept
// rows beyond it; a second kernel moves the j-th of these into the j-th of
// those. Sources lie at or beyond row `budget` and destinations below it, so
// the moves are independent, and nothing that stays is touched.
#include <cooperative_groups.h>
#include <math.h>

#include "paged.cuh"

namespace dfl {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = 32;
constexpr int kBins = 2048;
constexpr int kHeld = 40960;                 // keys a CTA holds in shared memory
constexpr int kMovesPerWarp = 8;

__device__ __forceinline__ unsigned weight_key(float w, bool keep) {
  if (keep) w = INFINITY;
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);            // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);      // -inf 0x007fffff, +inf 0xff800000
}

struct Shared {
  int hist[kBins];
  int2 warps[kWarps];
  int2 total;                                // of this CTA, for the others of its cluster
  int digit, left;
};

// Exclusive sums over the CTA's warps (lane 0's value of each) and, through
// the cluster, over the CTAs before this one; tot: the cluster's sums.
__device__ __forceinline__ int2 scan_warps(Shared& sh, cg::cluster_group& cl, int ranks, int2 v, int2* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sh.warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const int2 own = sh.warps[lane];
    int2 x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
      if (lane >= o) { x.x += a; x.y += b; }
    }
    sh.warps[lane] = make_int2(x.x - own.x, x.y - own.y);
    if (lane == 31) sh.total = x;
  }
  if (ranks > 1) cl.sync();
  else __syncthreads();
  int2 before = sh.warps[warp], all = make_int2(0, 0);
  for (int r = 0; r < ranks; ++r) {
    const int2 t = ranks > 1 ? *cl.map_shared_rank(&sh.total, r) : sh.total;
    if (r < (int)cl.block_rank()) { before.x += t.x; before.y += t.y; }
    all.x += t.x;
    all.y += t.y;
  }
  *tot = all;
  if (ranks > 1) cl.sync();
  else __syncthreads();
  return before;
}

// A cluster to a (sequence, kv head), a contiguous slice of its rows to a CTA.
// Keys are read once and held in shared memory where a slice fits (otherwise
// each pass reads them again, from L2). A warp takes contiguous rows, 32 at a
// time, so that ranks are ballots; the kept rows of each 32 are a word in
// shared memory after the first of the ranking passes. Bound by the latency of
// its dozen dependent steps for a few thousand rows, by one SM's read of the
// weights and positions beyond.
__global__ void __launch_bounds__(kThreads) paged_select_kernel(PagedEvictArgs a, int ranks) {
  extern __shared__ unsigned dyn[];          // [held] keys, then the masks of kept rows
  __shared__ Shared sh;
  pdl_enter();
  cg::cluster_group cl = cg::this_cluster();
  const PagedView& c = a.c;
  const int h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* list = a.moves + ((size_t)s * c.nkv + h) * (1 + 2 * (size_t)a.max_moves);
  const int n = paged_length(c, s), b = a.budget;
  const long long guard = (long long)a.next_pos[s] - a.recent;
  if (tid == 0 && h == 0 && blockIdx.x == 0 && c.status && c.length[s] != n) atomicOr(c.status, DFLASH_PAGED_BAD_ROWS);
  // a multiple of 1024, so that a warp's share is whole words
  const int per = (n + ranks * kThreads - 1) / (ranks * kThreads) * kThreads;
  const int i0 = min(n, (int)cl.block_rank() * per), i1 = min(n, i0 + per), m = i1 - i0;
  const bool held = per <= kHeld;
  unsigned* keys = dyn;
  unsigned* kept_bits = dyn + (held ? per : 0);
  const bool copies = a.weight_out != a.weight || a.pos_out != c.pos;
  // key of row i0 + i, from global memory (rows on no page count as NaN)
  auto fetch = [&](int i) -> unsigned {
    const long long row = paged_row(c, s, h, i0 + i);
    return row < 0 ? 0u : weight_key(a.weight[row], c.pos[row] >= guard);
  };
  auto key = [&](int i) -> unsigned { return held ? keys[i] : fetch(i); };

  unsigned prefix = 0;                       // the key of rank b: its known top bits
  int left = b;                              // rows still to take among those with that prefix
  if (n > b) {
    if (held) {
      // four rows to a thread: a page holds a multiple of 8
#pragma unroll 2
      for (int i = tid * 4; i < m; i += kThreads * 4) {
        const long long row = paged_row(c, s, h, i0 + i);
        uint4 k = make_uint4(0, 0, 0, 0);
        if (row >= 0) {
          const float4 w = *reinterpret_cast<const float4*>(a.weight + row);
          const int4 p = *reinterpret_cast<const int4*>(c.pos + row);
          k = make_uint4(weight_key(w.x, p.x >= guard), weight_key(w.y, p.y >= guard), weight_key(w.z, p.z >= guard), weight_key(w.w, p.w >= guard));
        } else if (c.status) {
          atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
        }
        *reinterpret_cast<uint4*>(keys + i) = k;
      }
    }
    const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int shift = shifts[d], top = shift + bits[d];
      for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < (m + 31) / 32 * 32; i += kThreads) {
        const unsigned k = i < m ? key(i) : 0u;
        const bool in = i < m && (top == 32 || (k >> top) == (prefix >> top));
        const unsigned dig = in ? (k >> shift) & ((1u << bits[d]) - 1) : 0xffffffffu;
        // equal weights are common (rows that nobody looked at): one add for a warp of them
        const unsigned one = __shfl_sync(0xffffffffu, dig, 0);
        if (__all_sync(0xffffffffu, dig == one)) {
          if (lane == 0 && in) atomicAdd(&sh.hist[dig], 32);
        } else if (in) {
          atomicAdd(&sh.hist[dig], 1);
        }
      }
      if (ranks > 1) cl.sync();
      else __syncthreads();
      // bins from the top, two to a thread: the bin in which the count reaches
      // `left`
      int v[2] = {0, 0};
      for (int r = 0; r < ranks; ++r) {
        const int* hist = ranks > 1 ? cl.map_shared_rank(sh.hist, r) : sh.hist;
        v[0] += hist[kBins - 1 - 2 * tid];
        v[1] += hist[kBins - 2 - 2 * tid];
      }
      int x = v[0] + v[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) sh.warps[warp].x = x;
      __syncthreads();
      if (warp == 0) {
        const int own = sh.warps[lane].x;
        int y = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int w = __shfl_up_sync(0xffffffffu, y, o);
          if (lane >= o) y += w;
        }
        sh.warps[lane].y = y - own;
      }
      __syncthreads();
      const int after = sh.warps[warp].y + x, before = after - v[0] - v[1];
      if (before < left && left <= after) {
        const bool first = left <= before + v[0];
        sh.digit = kBins - 1 - 2 * tid - (first ? 0 : 1);
        sh.left = left - before - (first ? 0 : v[0]);
      }
      if (ranks > 1) cl.sync();              // the others have read this CTA's bins
      else __syncthreads();
      prefix |= (unsigned)sh.digit << shift;
      left = sh.left;
    }
  }
  // `prefix` is now the key of rank b: greater keys stay, of the equal ones
  // the first `left`
  const int share = per / kWarps, w0 = warp * share, w1 = min(m, w0 + share);
  if (n > b) {
    int eq = 0;
    for (int i = w0; i < w1; i += 32) eq += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && key(i + lane) == prefix));
    int2 tot;
    eq = scan_warps(sh, cl, ranks, make_int2(eq, 0), &tot).x;
    int2 cnt = make_int2(0, 0);              // holes below row b, kept rows from it on
    for (int i = w0; i < w1; i += 32) {
      const unsigned k = i + lane < w1 ? key(i + lane) : 0u;
      const unsigned same = __ballot_sync(0xffffffffu, i + lane < w1 && k == prefix);
      const bool keep = i + lane < w1 && (k > prefix || (k == prefix && eq + __popc(same & ((1u << lane) - 1)) < left));
      eq += __popc(same);
      const unsigned stay = __ballot_sync(0xffffffffu, keep);
      const unsigned low = __ballot_sync(0xffffffffu, i + lane < w1 && i0 + i + lane < b);
      const unsigned there = __ballot_sync(0xffffffffu, i + lane < w1);
      cnt.x += __popc(low & ~stay);
      cnt.y += __popc(there & ~low & stay);
      if (lane == 0) kept_bits[i >> 5] = stay;
    }
    __syncwarp();
    int2 at = scan_warps(sh, cl, ranks, cnt, &tot);
    for (int i = w0; i < w1; i += 32) {
      const unsigned stay = kept_bits[i >> 5];
      const int row = i0 + i + lane;
      const bool there = i + lane < w1, keep = (stay >> lane) & 1u;
      const unsigned holes = __ballot_sync(0xffffffffu, there && row < b && !keep);
      const unsigned late = __ballot_sync(0xffffffffu, there && row >= b && keep);
      const unsigned below = (1u << lane) - 1;
      const int hj = at.x + __popc(holes & below), lj = at.y + __popc(late & below);
      if ((holes >> lane) & 1u) { if (hj < a.max_moves) list[1 + hj] = row; }
      if ((late >> lane) & 1u) { if (lj < a.max_moves) list[1 + a.max_moves + lj] = row; }
      at.x += __popc(holes);
      at.y += __popc(late);
    }
    if (tid == 0 && cl.block_rank() == 0) list[0] = min(tot.x, a.max_moves);
  } else if (tid == 0 && cl.block_rank() == 0) {
    list[0] = 0;
  }
  if (copies) {
    // position and weight of the rows that stay where they are
    for (int i = w0; i < w1; i += 32) {
      const int row = i0 + i + lane;
      const unsigned stay = n > b ? kept_bits[i >> 5] : 0xffffffffu;
      if (i + lane < w1 && row < b && ((stay >> lane) & 1u)) {
        const long long at = paged_row(c, s, h, row);
        if (at >= 0) {
          if (a.weight_out != a.weight) a.weight_out[at] = a.weight[at];
          if (a.pos_out != c.pos) a.pos_out[at] = c.pos[at];
        }
      }
    }
  }
}

// A warp to kMovesPerWarp moves: their places looked up side by side, their K
// and V rows requested together, 16 bytes to a lane. Bound by the bytes moved.
template <int ES>
__global__ void __launch_bounds__(256) paged_move_kernel(PagedEvictArgs a) {
  constexpr int kM = kMovesPerWarp;
  pdl_enter();
  const PagedView& c = a.c;
  const int h = blockIdx.y, s = blockIdx.z, lane = threadIdx.x & 31;
  const int* list = a.moves + ((size_t)s * c.nkv + h) * (1 + 2 * (size_t)a.max_moves);
  const int count = list[0], bytes = c.hd * ES;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    const int n = paged_length(c, s);
    a.length_out[s] = n < a.budget ? n : a.budget;
  }
  for (int j0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kM; j0 < count; j0 += gridDim.x * 8 * kM) {
    long long to = -1, of = -1;
    if (lane < kM && j0 + lane < count) {
      to = paged_row(c, s, h, list[1 + j0 + lane]);
      of = paged_row(c, s, h, list[1 + a.max_moves + j0 + lane]);
      if (of < 0) to = -1;
      if (to >= 0) {
        a.weight_out[to] = a.weight[of];
        a.pos_out[to] = c.pos[of];
      }
    }
    long long t[kM], f[kM];
#pragma unroll
    for (int u = 0; u < kM; ++u) {
      t[u] = __shfl_sync(0xffffffffu, to, u);
      f[u] = __shfl_sync(0xffffffffu, of, u);
    }
    for (int i = lane * 16; i < 2 * bytes; i += 512) {
      char* base = static_cast<char*>(i < bytes ? c.k : c.v);
      const int o = i < bytes ? i : i - bytes;
      uint4 x[kM];
#pragma unroll
      for (int u = 0; u < kM; ++u)
        if (t[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(base + f[u] * bytes + o);
#pragma unroll
      for (int u = 0; u < kM; ++u)
        if (t[u] >= 0) *reinterpret_cast<uint4*>(base + t[u] * bytes + o) = x[u];
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(int dtype, const PagedEvictArgs& a, cudaStream_t st) {
  const int cap = a.c.max_pages << a.c.lg_rows, pairs = a.c.nkv * a.c.n_seq;
  // CTAs to a (sequence, kv head): more where a CTA would have more than 4096
  // rows and SMs would be idle, and so that the masks fit
  int ranks = 1;
  while (ranks < 8 && (cap / ranks > 131072 || (cap / ranks > 4096 && (long long)pairs * ranks * 2 <= 304))) ranks *= 2;
  const int per = (cap + ranks * kThreads - 1) / (ranks * kThreads) * kThreads;
  const size_t smem = ((size_t)(per < kHeld ? per : kHeld) + per / 32) * 4;
  cudaError_t e = cudaFuncSetAttribute(paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kHeld + 131072 / 32) * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ranks, a.c.nkv, a.c.n_seq);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, paged_select_kernel, a, ranks);
  if (e != cudaSuccess) return e;
  int x = (a.max_moves + 8 * kMovesPerWarp - 1) / (8 * kMovesPerWarp);
  if (x > 512) x = 512;
  if (x < 1) x = 1;
  const dim3 grid(x, a.c.nkv, a.c.n_seq);
  return dtype ? launch_pdl(paged_move_kernel<2>, grid, dim3(256), 0, st, a)
               : launch_pdl(paged_move_kernel<4>, grid, dim3(256), 0, st, a);
}

}  // namespace dfl
