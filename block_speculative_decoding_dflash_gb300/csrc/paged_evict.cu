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
//
// 2304 rows to 2048 in 8 heads: 10.9 us, the two kernels' dependent steps; 12
// sequences of up to 32768 rows to 16000: 76 us, of which the moves take 40 us (rows
// of 256 bytes, read and written at 4 TB/s).
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
  int digit, left, eq_before, all_stay;
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
// each pass reads them again, from L2). The ranking works on words of 32 rows,
// one to a thread. Bound by the latency of its dozen dependent steps for a few
// thousand rows, by one SM's passes over the keys beyond.
__global__ void __launch_bounds__(kThreads, 2) paged_select_kernel(PagedEvictArgs a, int ranks) {
  extern __shared__ __align__(16) unsigned dyn[];   // keys (where held), then four words to 32 rows
  __shared__ Shared sh;
  pdl_enter();
  cg::cluster_group cl = cg::this_cluster();
  const PagedView& c = a.c;
  const int h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* list = a.moves + ((size_t)s * c.nkv + h) * (1 + 2 * (size_t)a.max_moves);
  const int n = paged_length(c, s), b = a.budget;
  const long long guard = (long long)a.next_pos[s] - a.recent;
  if (tid == 0 && h == 0 && blockIdx.x == 0) paged_report_length(c, s, n);
  // a multiple of kThreads, so that a warp's share is whole words
  const int per = (n + ranks * kThreads - 1) / (ranks * kThreads) * kThreads;
  const int i0 = min(n, (int)cl.block_rank() * per), i1 = min(n, i0 + per), m = i1 - i0;
  const bool held = per <= kHeld;
  // a word of 32 rows: its kept rows, its rows of the bordering key, and the
  // number of holes and late rows before it
  unsigned* keys = dyn;
  unsigned* keep_bits = dyn + (held ? per : 0);
  unsigned* same_bits = keep_bits + per / 32;
  int2* offs = reinterpret_cast<int2*>(same_bits + per / 32);
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
  // keys of rows i .. i + 3 (i a multiple of 4); past the end 0, the lowest
  auto key4 = [&](int i, unsigned* k) {
    if (held) {
      const uint4 v = i < m ? *reinterpret_cast<const uint4*>(keys + i) : make_uint4(0, 0, 0, 0);
      k[0] = v.x; k[1] = v.y; k[2] = v.z; k[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = i + j < m ? fetch(i + j) : 0u;
    }
  };

  // (held keys report as they are read: a look at every row's page id costs the
  // others, whose passes are longer, 3% with 24 sequences of up to 32768 rows)
  if (c.status && !(n > b && held) && (n > b || new_w || new_p))
    for (int p = (i0 >> c.lg_rows) + tid; p << c.lg_rows < i1; p += kThreads)
      if ((unsigned)c.table[(size_t)s * c.max_pages + p] >= (unsigned)c.n_pages) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);

  unsigned prefix = 0;                       // the key of rank b: its known top bits
  int left = b;                              // rows still to take among those with that prefix
  if (n > b) {
    if (held) {
      // four rows to a thread (a page holds a multiple of 8), kU times at once
      constexpr int kU = 4;
      for (int b4 = tid * 4; b4 < m; b4 += kThreads * 4 * kU) {
        long long row[kU];
        float4 w[kU];
        int4 p[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = b4 + u * kThreads * 4;
          row[u] = i < m ? paged_row(c, s, h, i0 + i) : -1;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (row[u] >= 0) {
            w[u] = *reinterpret_cast<const float4*>(a.weight + row[u]);
            p[u] = *reinterpret_cast<const int4*>(c.pos + row[u]);
          }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = b4 + u * kThreads * 4;
          if (i >= m) break;
          uint4 k = make_uint4(0, 0, 0, 0);
          if (row[u] >= 0) {
            copy4(row[u], i0 + i, w[u], p[u]);
            k = make_uint4(weight_key(w[u].x, p[u].x >= guard), weight_key(w[u].y, p[u].y >= guard),
                           weight_key(w[u].z, p[u].z >= guard), weight_key(w[u].w, p[u].w >= guard));
          } else if (c.status) {
            atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
          }
          *reinterpret_cast<uint4*>(keys + i) = k;
        }
      }
    }
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0), top = d == 0 ? 32 : (d == 1 ? 21 : 10), mask = (1 << (top - shift)) - 1;
      int* hist = sh.hist[d & 1];
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid * 4; i - lane * 4 < m; i += kThreads * 4) {
        unsigned k[4], dig[4];
        key4(i, k);
        bool same = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = i + j < m && (d == 0 || (k[j] >> top) == (prefix >> top));
          dig[j] = in ? (k[j] >> shift) & mask : 0xffffffffu;
          same = same && dig[j] == dig[0];
        }
        // equal weights are common (rows that nobody looked at): one add for a warp of them
        const unsigned one = __shfl_sync(0xffffffffu, dig[0], 0);
        if (__all_sync(0xffffffffu, same && dig[0] == one)) {
          if (lane == 0 && one != 0xffffffffu) atomicAdd(&hist[one], 128);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (dig[j] != 0xffffffffu) atomicAdd(&hist[dig[j]], 1);
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
        sh.all_stay = left - before == cnt[j];
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
      if (d < 2 && sh.all_stay) {
        // every row with these top bits stays (weights seldom agree in 22 bits):
        // the border lies below them, and the digits left need no pass (2304
        // rows: 10.9 us, with all three passes 11.6 us). Not zero: with the lowest
        // digit n <= b rows would stay.
        prefix -= 1;
        left = 0;
        break;
      }
    }
  }
  // `prefix` is now the key of rank b: greater keys stay, of the equal ones
  // the first `left`
  if (n > b) {
    // a bit to a row: greater and equal keys, 128 rows to a warp at a time
    // (lane l's four rows are bits 4 (l mod 8) .. of word l / 8)
    const int words = (m + 31) >> 5;
    for (int i = tid * 4; i - lane * 4 < m; i += kThreads * 4) {
      unsigned k[4], gt = 0, eq = 0;
      key4(i, k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        gt |= (unsigned)(i + j < m && k[j] > prefix) << j;
        eq |= (unsigned)(i + j < m && k[j] == prefix) << j;
      }
      gt <<= 4 * (lane & 7);
      eq <<= 4 * (lane & 7);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        gt |= __shfl_xor_sync(0xffffffffu, gt, o);
        eq |= __shfl_xor_sync(0xffffffffu, eq, o);
      }
      if ((lane & 7) == 0 && i < m) {
        keep_bits[i >> 5] = gt;
        same_bits[i >> 5] = eq;
      }
    }
    __syncthreads();
    // words in order, one to a thread: which equal rows stay, and the number of
    // holes below row b and of kept rows from it on
    int eq_run = left ? sh.eq_before : 0;
    int2 run = make_int2(0, 0), tot;
    for (int x0 = 0; x0 < words; x0 += kThreads) {
      const int x = x0 + tid;
      const unsigned gt = x < words ? keep_bits[x] : 0u, eq = x < words ? same_bits[x] : 0u;
      int incl = __popc(eq);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      int before = eq_run + scan_warps(sh, make_int2(__shfl_sync(0xffffffffu, incl, 31), 0), &tot).x + incl - __popc(eq);
      eq_run += tot.x;
      unsigned take = eq;
      for (int over = before + __popc(eq) - left; over > 0 && take; --over) take &= ~(0x80000000u >> __clz(take));
      const unsigned stay = gt | take;
      const int r0 = i0 + x * 32;                        // rows below b: the low bits
      const unsigned there = x < words ? (m - x * 32 >= 32 ? 0xffffffffu : (1u << (m - x * 32)) - 1) : 0u;
      const unsigned low = b - r0 >= 32 ? 0xffffffffu : (b > r0 ? (1u << (b - r0)) - 1 : 0u);
      const int2 cnt = make_int2(__popc(there & low & ~stay), __popc(there & ~low & stay));
      int2 in = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, in.x, o), v = __shfl_up_sync(0xffffffffu, in.y, o);
        if (lane >= o) { in.x += u; in.y += v; }
      }
      __syncthreads();                                   // sh.warps is free again
      const int2 at = scan_warps(sh, make_int2(__shfl_sync(0xffffffffu, in.x, 31), __shfl_sync(0xffffffffu, in.y, 31)), &tot);
      if (x < words) {
        // a word has holes or late rows but for the one that row b - 1 lies in
        keep_bits[x] = stay;
        offs[x] = make_int2(run.x + at.x + in.x - cnt.x, run.y + at.y + in.y - cnt.y);
      }
      run.x += tot.x;
      run.y += tot.y;
      __syncthreads();
    }
    if (tid == 0) sh.total = run;
    meet(cl, ranks);
    int2 base = make_int2(0, 0), sum = run;
    if (ranks > 1) {
      int2 p[kRanks];
#pragma unroll
      for (int r = 0; r < kRanks; ++r) p[r] = r < ranks ? *cl.map_shared_rank(&sh.total, r) : make_int2(0, 0);
      sum = make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < kRanks; ++r) {
        if (r < (int)cl.block_rank()) { base.x += p[r].x; base.y += p[r].y; }
        sum.x += p[r].x;
        sum.y += p[r].y;
      }
    }
#pragma unroll 4
    for (int x = warp; x < words; x += kWarps) {
      const unsigned stay = keep_bits[x];
      const int2 at = offs[x];
      const int i = x * 32 + lane, row = i0 + i;
      const unsigned low = b - i0 - x * 32 >= 32 ? 0xffffffffu : (b > i0 + x * 32 ? (1u << (b - i0 - x * 32)) - 1 : 0u);
      const bool keep = (stay >> lane) & 1u, hole = i < m && row < b && !keep, late = i < m && row >= b && keep;
      if (hole || late) {
        // its place in the pool, so that the move need not look it up
        const unsigned below = (1u << lane) - 1;
        const int j = hole ? base.x + at.x + __popc(~stay & low & below) : base.y + at.y + __popc(stay & ~low & below);
        if (j < a.max_moves) list[1 + (hole ? 0 : a.max_moves) + j] = (int)paged_row(c, s, h, row);
      }
    }
    if (tid == 0 && cl.block_rank() == 0) list[0] = min(sum.x, a.max_moves);
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
  // rows and SMs (two CTAs to each) would be idle, and so that the masks fit (12
  // sequences of up to 32768 rows: 79 us, with one CTA to each 136 us, both with
  // all three passes)
  int ranks = 1;
  while (ranks < kRanks && (cap / ranks > kMostRows || (cap / ranks > 4096 && (long long)pairs * ranks * 2 <= 304))) ranks *= 2;
  const int per = (cap + ranks * kThreads - 1) / (ranks * kThreads) * kThreads;
  const size_t smem = ((size_t)(per < kHeld ? per : kHeld) + per / 8) * 4;
  cudaError_t e = cudaFuncSetAttribute(paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kHeld + kMostRows / 8) * 4);
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
  cfg.numAttrs = ranks > 1 ? 2 : 1;
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
