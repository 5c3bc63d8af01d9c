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

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kBinsEach = kBins / kThreads;
constexpr int kRanks = 8;                    // CTAs of a cluster, at most
constexpr int kHeld = 24576;                 // keys a CTA holds in shared memory
constexpr int kMostRows = (1 << 20) / kRanks;
constexpr int kMovesPerWarp = 8;

__device__ __forceinline__ unsigned weight_key(float w, bool keep) {
  if (keep) w = INFINITY;
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);            // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);      // -inf 0x007fffff, +inf 0xff800000
}

struct Shared {
  int hist[2][kBins];                        // in turns, so that a pass need not wait for the others' reads of the last
  int2 warps[kWarps];
  int2 total;                                // of this CTA, for the others of its cluster
  int digit, left, eq_before;
};

// Every CTA of the cluster (or, alone, every thread) has come here and sees
// what the others wrote to shared memory.
__device__ __forceinline__ void meet(cg::cluster_group& cl, int ranks) {
  if (ranks > 1) cl.sync();
  else __syncthreads();
}

// Exclusive sums over the CTA's warps of lane 0's values; total to all.
__device__ __forceinline__ int2 scan_warps(Shared& sh, int2 v, int2* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sh.warps[warp] = v;
  __syncthreads();
  int2 x = lane < kWarps ? sh.warps[lane] : make_int2(0, 0);
  const int2 own = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) { x.x += a; x.y += b; }
  }
  *tot = make_int2(__shfl_sync(0xffffffffu, x.x, 31), __shfl_sync(0xffffffffu, x.y, 31));
  x.x -= own.x;
  x.y -= own.y;
  return make_int2(__shfl_sync(0xffffffffu, x.x, warp), __shfl_sync(0xffffffffu, x.y, warp));
}

// A cluster to a (sequence, kv head), a contiguous slice of its rows to a CTA.
// Keys are read once and held in shared memory where a slice fits (otherwise
// each pass reads them again, from L2). A warp takes contiguous rows, 32 at a
// time, so that ranks are ballots; the kept rows of each 32 are a word in
// shared memory after the first of the ranking passes. Bound by the latency of
// its dozen dependent steps for a few thousand rows, by one SM's read of the
// weights and positions beyond.
__global__ void __launch_bounds__(kThreads, 2) paged_select_kernel(PagedEvictArgs a, int ranks) {
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
  // a multiple of kThreads, so that a warp's share is whole words
  const int per = (n + ranks * kThreads - 1) / (ranks * kThreads) * kThreads;
  const int i0 = min(n, (int)cl.block_rank() * per), i1 = min(n, i0 + per), m = i1 - i0;
  const bool held = per <= kHeld;
  unsigned* keys = dyn;
  unsigned* kept_bits = dyn + (held ? per : 0);
  // Position and weight of a remaining row go to the outputs as they are read;
  // a hole gets its new row's in the move, which comes after.
  const bool new_w = a.weight_out != a.weight, new_p = a.pos_out != c.pos;
  const int keep_n = min(n, b);
  auto copy4 = [&](long long row, int i, const float4& w, const int4& p) {
    if (i + 3 < keep_n) {
      if (new_w) *reinterpret_cast<float4*>(a.weight_out + row) = w;
      if (new_p) *reinterpret_cast<int4*>(a.pos_out + row) = p;
    } else {
      const float wv[4] = {w.x, w.y, w.z, w.w};
      const int pv[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < keep_n) {
          if (new_w) a.weight_out[row + j] = wv[j];
          if (new_p) a.pos_out[row + j] = pv[j];
        }
    }
  };
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
          copy4(row, i0 + i, w, p);
          k = make_uint4(weight_key(w.x, p.x >= guard), weight_key(w.y, p.y >= guard), weight_key(w.z, p.z >= guard), weight_key(w.w, p.w >= guard));
        } else if (c.status) {
          atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
        }
        *reinterpret_cast<uint4*>(keys + i) = k;
      }
    }
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0), top = d == 0 ? 32 : (d == 1 ? 21 : 10), mask = (1 << (top - shift)) - 1;
      int* hist = sh.hist[d & 1];
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < (m + 31) / 32 * 32; i += kThreads) {
        const unsigned k = i < m ? key(i) : 0u;
        const bool in = i < m && (d == 0 || (k >> top) == (prefix >> top));
        const unsigned dig = in ? (k >> shift) & mask : 0xffffffffu;
        // equal weights are common (rows that nobody looked at): one add for a warp of them
        const unsigned one = __shfl_sync(0xffffffffu, dig, 0);
        if (__all_sync(0xffffffffu, dig == one)) {
          if (lane == 0 && in) atomicAdd(&hist[dig], 32);
        } else if (in) {
          atomicAdd(&hist[dig], 1);
        }
      }
      meet(cl, ranks);
      // bins from the top, kBinsEach to a thread: the bin in which the count
      // reaches `left`
      int4 v = make_int4(0, 0, 0, 0);
      const int at = kBins - kBinsEach * (tid + 1);
      if (ranks > 1) {
        int4 p[kRanks];
#pragma unroll
        for (int r = 0; r < kRanks; ++r)
          p[r] = r < ranks ? *reinterpret_cast<const int4*>(cl.map_shared_rank(hist, r) + at) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kRanks; ++r) { v.x += p[r].x; v.y += p[r].y; v.z += p[r].z; v.w += p[r].w; }
      } else {
        v = *reinterpret_cast<const int4*>(hist + at);
      }
      const int cnt[4] = {v.w, v.z, v.y, v.x};
      const int mine = (v.x + v.y) + (v.z + v.w);
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      int2 tot;
      const int warp_total = __shfl_sync(0xffffffffu, x, 31);
      int before = scan_warps(sh, make_int2(warp_total, 0), &tot).x + x - mine;
      if (before < left && left <= before + mine) {
        int j = 0;
        while (left > before + cnt[j]) before += cnt[j++];
        sh.digit = at + kBinsEach - 1 - j;
        sh.left = left - before;
        if (d == 2) {
          // the last digit's bin counts the rows whose key is the one of rank b
          int eq = 0;
          for (int r = 0; r < (int)cl.block_rank(); ++r) eq += cl.map_shared_rank(hist, r)[sh.digit];
          sh.eq_before = eq;
        }
      }
      __syncthreads();
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
    eq = sh.eq_before + scan_warps(sh, make_int2(eq, 0), &tot).x;
    int2 cnt = make_int2(0, 0);              // holes below row b, kept rows from it on
    for (int i = w0; i < w1; i += 32) {
      const bool there = i + lane < w1;
      const unsigned k = there ? key(i + lane) : 0u;
      const unsigned same = __ballot_sync(0xffffffffu, there && k == prefix);
      const bool keep = there && (k > prefix || (k == prefix && eq + __popc(same & ((1u << lane) - 1)) < left));
      eq += __popc(same);
      const unsigned stay = __ballot_sync(0xffffffffu, keep);
      const unsigned low = __ballot_sync(0xffffffffu, there && i0 + i + lane < b);
      cnt.x += __popc(low & ~stay);
      cnt.y += __popc(~low & stay);
      if (lane == 0) kept_bits[i >> 5] = stay;
    }
    __syncthreads();                         // sh.warps is free again
    int2 at = scan_warps(sh, cnt, &tot);
    if (tid == 0) sh.total = tot;
    meet(cl, ranks);
    if (ranks > 1) {
      int2 p[kRanks];
#pragma unroll
      for (int r = 0; r < kRanks; ++r) p[r] = r < ranks ? *cl.map_shared_rank(&sh.total, r) : make_int2(0, 0);
      tot = make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < kRanks; ++r) {
        if (r < (int)cl.block_rank()) { at.x += p[r].x; at.y += p[r].y; }
        tot.x += p[r].x;
        tot.y += p[r].y;
      }
    }
    for (int i = w0; i < w1; i += 32) {
      const unsigned stay = kept_bits[i >> 5];
      const int row = i0 + i + lane;
      const bool there = i + lane < w1, keep = (stay >> lane) & 1u;
      const bool hole = there && row < b && !keep, late = there && row >= b && keep;
      const unsigned holes = __ballot_sync(0xffffffffu, hole), lates = __ballot_sync(0xffffffffu, late);
      const unsigned below = (1u << lane) - 1;
      if (hole || late) {
        // its place in the pool, so that the move need not look it up
        const int j = hole ? at.x + __popc(holes & below) : a.max_moves + at.y + __popc(lates & below);
        if (j < (hole ? a.max_moves : 2 * a.max_moves)) list[1 + j] = (int)paged_row(c, s, h, row);
      }
      at.x += __popc(holes);
      at.y += __popc(lates);
    }
    if (tid == 0 && cl.block_rank() == 0) list[0] = min(tot.x, a.max_moves);
  } else if (tid == 0 && cl.block_rank() == 0) {
    list[0] = 0;
  }
  if ((new_w || new_p) && !(n > b && held)) {
    for (int i = tid * 4; i < m && i0 + i < keep_n; i += kThreads * 4) {
      const long long row = paged_row(c, s, h, i0 + i);
      if (row >= 0) copy4(row, i0 + i, *reinterpret_cast<const float4*>(a.weight + row), *reinterpret_cast<const int4*>(c.pos + row));
    }
  }
  if (ranks > 1) cl.sync();                  // no CTA leaves while another reads its totals
}

// A warp to kMovesPerWarp moves: their K and V rows requested together, 16
// bytes to a lane. Bound by the bytes moved.
template <int ES>
__global__ void __launch_bounds__(256, 3) paged_move_kernel(PagedEvictArgs a) {
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
  const int stride = gridDim.x * 8 * kM;
  int j0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kM;
  int to = -1, of = -1;
  if (lane < kM && j0 + lane < count) {
    to = list[1 + j0 + lane];
    of = list[1 + a.max_moves + j0 + lane];
  }
  for (; j0 < count; j0 += stride) {
    if (of < 0) to = -1;                     // a row on no page
    const int my_to = to, my_of = of;
    to = of = -1;
    if (lane < kM && j0 + stride + lane < count) {
      to = list[1 + j0 + stride + lane];
      of = list[1 + a.max_moves + j0 + stride + lane];
    }
    int t[kM], f[kM];
#pragma unroll
    for (int u = 0; u < kM; ++u) {
      t[u] = __shfl_sync(0xffffffffu, my_to, u);
      f[u] = __shfl_sync(0xffffffffu, my_of, u);
    }
    for (int i = lane * 16; i < 2 * bytes; i += 512) {
      char* base = static_cast<char*>(i < bytes ? c.k : c.v);
      const int o = i < bytes ? i : i - bytes;
      uint4 x[kM];
#pragma unroll
      for (int u = 0; u < kM; ++u)
        if (t[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(base + (long long)f[u] * bytes + o);
#pragma unroll
      for (int u = 0; u < kM; ++u)
        if (t[u] >= 0) *reinterpret_cast<uint4*>(base + (long long)t[u] * bytes + o) = x[u];
    }
    if (my_to >= 0) {
      a.weight_out[my_to] = a.weight[my_of];
      a.pos_out[my_to] = c.pos[my_of];
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(int dtype, const PagedEvictArgs& a, cudaStream_t st) {
  const int cap = a.c.max_pages << a.c.lg_rows, pairs = a.c.nkv * a.c.n_seq;
  // CTAs to a (sequence, kv head): more where a CTA would have more than 4096
  // rows and SMs (two CTAs to each) would be idle, and so that the masks fit
  int ranks = 1;
  while (ranks < kRanks && (cap / ranks > kMostRows || (cap / ranks > 4096 && (long long)pairs * ranks * 2 <= 304))) ranks *= 2;
  const int per = (cap + ranks * kThreads - 1) / (ranks * kThreads) * kThreads;
  const size_t smem = ((size_t)(per < kHeld ? per : kHeld) + per / 32) * 4;
  cudaError_t e = cudaFuncSetAttribute(paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kHeld + kMostRows / 32) * 4);
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
  // CTAs for every move there may be, at most what 152 SMs hold twice over
  int x = (a.max_moves + 8 * kMovesPerWarp - 1) / (8 * kMovesPerWarp);
  const int most = (152 * 6 + pairs - 1) / pairs;
  if (x > most) x = most;
  if (x < 1) x = 1;
  const dim3 grid(x, a.c.nkv, a.c.n_seq);
  return dtype ? launch_pdl(paged_move_kernel<2>, grid, dim3(256), 0, st, a)
               : launch_pdl(paged_move_kernel<4>, grid, dim3(256), 0, st, a);
}

}  // namespace dfl
