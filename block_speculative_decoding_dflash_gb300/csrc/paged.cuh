// Shared by the paged-cache kernels: their arguments, the page lookup, the
// search for a CTA's sequence and tile, the mask, and the classification of
// key tiles.
#pragma once

#include "common.cuh"
#include "dflash.h"
#include "kernels.h"
#include "launch.cuh"

namespace dfl {

constexpr int kPagedNoPos = INT32_MIN;     // position of a row that is not there

// Rows sequence s has: its length, cut to the table.
__device__ __forceinline__ int paged_length(const PagedView& c, int s) {
  const int n = c.length[s], cap = c.max_pages << c.lg_rows;
  return n < 0 ? 0 : (n > cap ? cap : n);
}
// Reports a length that was cut to `len`; one thread to a sequence.
__device__ __forceinline__ void paged_report_length(const PagedView& c, int s, int len) {
  if (c.status && c.length[s] != len) atomicOr(c.status, DFLASH_PAGED_BAD_ROWS);
}
// New rows [first, last) of sequence s, cut to [0, rows].
__device__ __forceinline__ int2 paged_new_rows(const int* start, int s, int rows) {
  int a = start[s], b = start[s + 1];
  a = a < 0 ? 0 : (a > rows ? rows : a);
  b = b < a ? a : (b > rows ? rows : b);
  return make_int2(a, b);
}
// Row index (in units of rows of head_dim) of slot `slot` of sequence s and
// kv head h, or -1 where its page id is outside the pool. slot < capacity.
__device__ __forceinline__ long long paged_row(const PagedView& c, int s, int h, int slot) {
  const int page = c.table[(size_t)s * c.max_pages + (slot >> c.lg_rows)];
  if ((unsigned)page >= (unsigned)c.n_pages) return -1;
  return (((long long)page * c.nkv + h) << c.lg_rows) + (slot & ((1 << c.lg_rows) - 1));
}

// The sequence and the tile within it of tile number `t` of the batch, with
// `per` new rows (times G) to a tile; called by one full warp. seq = -1 past
// the last tile.
struct PagedTile { int seq, tile, first, count; };
__device__ __forceinline__ PagedTile paged_find_tile(const int* start, int n_seq, int rows, int G, int per, int t) {
  constexpr int kU = 4;                      // sequences of a lane requested together
  const int lane = threadIdx.x & 31;
  PagedTile r{-1, 0, 0, 0};
  for (int s0 = 0; s0 < n_seq; s0 += 32 * kU) {
    int2 ab[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int s = s0 + u * 32 + lane;
      ab[u] = s < n_seq ? make_int2(start[s], start[s + 1]) : make_int2(0, 0);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (s0 + u * 32 >= n_seq) break;
      const int a = min(max(ab[u].x, 0), rows), b = min(max(ab[u].y, a), rows);
      const int tiles = (int)(((long long)(b - a) * G + per - 1) / per);
      int incl = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, t < incl);
      if (hit) {
        const int l = __ffs(hit) - 1;
        r.seq = s0 + u * 32 + l;
        r.tile = t - __shfl_sync(0xffffffffu, incl - tiles, l);
        r.first = __shfl_sync(0xffffffffu, a, l);
        r.count = __shfl_sync(0xffffffffu, b - a, l);
        return r;
      }
      t -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  return r;
}

// The same where sequences are cut into segments of keys, for batches of trees, so
// that no sequence sets the time alone. `sms` CTAs of a head run at once; the segments
// are as short as fills them once, or as many times as the batch has query tiles for,
// or twice where that evens out sequences of different lengths. (A segment's start and
// end take as long as about 8 key tiles, joining them 4.) Number `t` of the segments:
// which sequence, which query tile, which of the tile's n ranges of keys. Up to 32
// sequences come in the order of their segments' lengths, longest first, which fills
// the SMs evenly.
constexpr int kPagedLeastTiles = 4;
struct PagedSegment { PagedTile t; int z, n; };
__device__ __forceinline__ PagedSegment paged_find_segment(const PagedView& c, const int* start, int rows, int G, int per, int keys,
                                                           int window, int sms, int t) {
  const int lane = threadIdx.x & 31;
  PagedSegment r{{-1, 0, 0, 0}, 0, 1};
  // of sequence s: its new rows, its query tiles and the key tiles that they may see (one
  // at least: rows of an empty sequence have a segment too, which writes that they saw nothing)
  int first = 0, count = 0, q_tiles = 0, k_tiles = 0;
  auto look = [&](int s) {
    first = count = q_tiles = k_tiles = 0;
    if (s >= c.n_seq) return;
    const int2 ab = paged_new_rows(start, s, rows);
    first = ab.x;
    count = ab.y - ab.x;
    q_tiles = (int)(((long long)count * G + per - 1) / per);
    k_tiles = max(1, (paged_length(c, s) + keys - 1) / keys);
    if (window > 0) k_tiles = min(k_tiles, (int)min(((long long)window + count) / keys + 2, 1ll << 20));
  };
  long long work = 0;
  int tiles = 0;
  for (int s0 = 0; s0 < c.n_seq; s0 += 32) {
    look(s0 + lane);
    work += (long long)q_tiles * k_tiles;
    tiles += q_tiles;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  int rounds = max(1, (tiles + sms - 1) / sms), length;
  if (c.n_seq <= 32) {
    const int longest = __reduce_max_sync(0xffffffffu, q_tiles ? k_tiles : 0);
    // the shortest segments of which there are at most `most`
    auto shortest = [&](int most) {
      if (c.n_seq == 1 && tiles > 0) {
        const int n = most / tiles;
        return max(kPagedLeastTiles, (longest + n - 1) / n);
      }
      int lo = max(kPagedLeastTiles, (int)(work / most)), hi = max(lo, longest);
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__reduce_add_sync(0xffffffffu, q_tiles * ((k_tiles + mid - 1) / mid)) <= most) hi = mid;
        else lo = mid + 1;
      }
      return lo;
    };
    length = shortest(rounds * sms);
    if (rounds == 1 && length + 8 + (length < longest ? 4 : 0) > (int)(work / sms) + (int)(work / sms) / 12 + 20) length = shortest(2 * sms);
  } else {
    // (the sum of the quotients rounded up is at most work / length + tiles)
    const int spare = (rounds + 1) * sms - tiles;
    length = max(kPagedLeastTiles, (int)((work + spare - 1) / spare));
  }
  for (int s0 = 0; s0 < c.n_seq; s0 += 32) {
    if (c.n_seq > 32) look(s0 + lane);
    int n = max(1, (k_tiles + length - 1) / length), mine = q_tiles * n, seq = s0 + lane;
    if (c.n_seq <= 32 && c.n_seq > 1) {
      const int each = q_tiles ? (k_tiles + n - 1) / n : -1;
      int rank = 0, from = 0;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const int other = __shfl_sync(0xffffffffu, each, i);
        rank += other > each || (other == each && i < lane);
      }
#pragma unroll 8
      for (int i = 0; i < 32; ++i) from = __shfl_sync(0xffffffffu, rank, i) == lane ? i : from;
      n = __shfl_sync(0xffffffffu, n, from);
      mine = __shfl_sync(0xffffffffu, mine, from);
      first = __shfl_sync(0xffffffffu, first, from);
      count = __shfl_sync(0xffffffffu, count, from);
      seq = from;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, t < incl);
    if (hit) {
      const int l = __ffs(hit) - 1;
      t -= __shfl_sync(0xffffffffu, incl - mine, l);
      r.n = __shfl_sync(0xffffffffu, n, l);
      r.z = t % r.n;
      r.t.seq = __shfl_sync(0xffffffffu, seq, l);
      r.t.tile = t / r.n;
      r.t.first = __shfl_sync(0xffffffffu, first, l);
      r.t.count = __shfl_sync(0xffffffffu, count, l);
      return r;
    }
    t -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}
// The mask of the header. What one query at pq sees is a range of positions
// and the prefix: two unsigned comparisons, both false for kPagedNoPos.
struct PagedMask { int causal, window, prefix; };
struct PagedSees { int lo; unsigned span, prefix; };
__device__ __forceinline__ PagedMask paged_mask(int causal, int window, const int* prefix, int seq) {
  const int p = prefix ? prefix[seq] : 0;
  return PagedMask{causal, window, p > 0 ? p : 0};
}
__device__ __forceinline__ PagedSees paged_sees_of(const PagedMask& m, int pq) {
  long long lo = INT32_MIN + 1, hi = m.causal ? pq : INT32_MAX;
  if (m.window > 0) {
    if ((long long)pq - m.window > lo) lo = (long long)pq - m.window;
    if (!m.causal && (long long)pq + m.window < hi) hi = (long long)pq + m.window;
  }
  // (pq = INT32_MIN with a causal mask: a range is never empty, so it gets one of
  // a negative position, which no row has)
  if (hi < lo) return PagedSees{INT32_MIN + 1, 0u, (unsigned)m.prefix};
  return PagedSees{(int)lo, (unsigned)(hi - lo), (unsigned)m.prefix};
}
__device__ __forceinline__ bool paged_sees(const PagedSees& s, int pk) {
  return (unsigned)pk - (unsigned)s.lo <= s.span || (unsigned)pk < s.prefix;
}
// The other way about: the positions of the queries that see a row at pk (none,
// and no query has a negative one, for a row that is not there).
__device__ __forceinline__ PagedSees paged_seen_by(const PagedMask& m, int pk) {
  if (pk == kPagedNoPos) return PagedSees{INT32_MIN + 1, 0u, 0u};
  long long lo = m.causal ? pk : INT32_MIN + 1, hi = INT32_MAX;
  if (m.window > 0) {
    if (!m.causal && (long long)pk - m.window > lo) lo = (long long)pk - m.window;
    if ((long long)pk + m.window < hi) hi = (long long)pk + m.window;
  }
  if ((unsigned)pk < (unsigned)m.prefix) { lo = INT32_MIN + 1; hi = INT32_MAX; }
  return PagedSees{(int)lo, (unsigned)(hi - lo), 0u};
}
// Queries at [qmin, qmax], rows at [kmin, kmax] (kmin > kmax: none are there):
// 0 no query sees any row, 2 every query sees every row (of a tile whose rows
// are all there), 1 otherwise. Never 0 or 2 wrongly; 1 may be more than needed.
__device__ __forceinline__ int paged_class(const PagedMask& m, int qmin, int qmax, int kmin, int kmax, bool whole) {
  if (kmin > kmax || qmin > qmax) return 0;
  const long long W = m.window > 0 ? m.window : (1ll << 40);
  const long long ahead = m.causal ? 0 : W;
  const bool some = kmin < m.prefix || (kmin <= qmax + ahead && kmax >= qmin - W);
  if (!some) return 0;
  const bool all = kmax < m.prefix || (kmax <= qmin + ahead && kmin >= qmax - W);
  return all && whole ? 2 : 1;
}

// Trees of drafted tokens: the new rows of a sequence, in depth-first order, are
// its last `count` cached rows. New row j is seen by the new rows i with 0 <= i - j
// < paged_tree_size(j): itself and its subtree, one unsigned comparison. `tree` starts
// at the sequence's first new row. An older row (node < 0) has a size that every
// difference is below.
__device__ __forceinline__ int paged_tree_size(const int* tree, int count, int node) {
  if (node < 0 || node >= count) return INT32_MAX;
  const int end = min(tree[node], count) - node;
  return end < 1 ? 1 : end;
}

// Classifies the key tiles [t0, t1) of `KEYS` rows of (s, h) against queries
// at [qmin, qmax]: bit t - t0 of `some` / `all` in shared memory (zeroed here)
// for classes >= 1 / 2. Called by every thread of the CTA, which synchronises
// afterwards. A lane takes 16 rows, so a warp 512 / KEYS tiles at a time, with
// its loads in flight together: without branches, what is not there reads row
// 0 of the pool. (Short code on purpose: it runs once a CTA, as fast as its
// instructions arrive.)
template <int KEYS>
__device__ __forceinline__ void paged_classify(const PagedView& c, int s, int h, int len, const PagedMask& m, int qmin, int qmax,
                                               int t0, int t1, unsigned* some, unsigned* all) {
  constexpr int kLanes = KEYS / 16, kTiles = 32 / kLanes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  for (int i = threadIdx.x; i <= (t1 - t0) >> 5; i += blockDim.x) some[i] = all[i] = 0u;
  __syncthreads();
#pragma unroll 1
  for (int b = t0 + warp * kTiles; b < t1; b += nw * kTiles) {
    const int tile = b + lane / kLanes, slot = tile * KEYS + (lane & (kLanes - 1)) * 16;
    const int end = tile < t1 ? len : 0;                  // rows from here on are not there
    int page[2];
    int4 p[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) page[u] = c.table[(size_t)s * c.max_pages + (slot + 8 * u < end ? (slot + 8 * u) >> c.lg_rows : 0)];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool on = (unsigned)page[u >> 1] < (unsigned)c.n_pages;
      const long long row = on ? (((long long)page[u >> 1] * c.nkv + h) << c.lg_rows) + ((slot + 4 * u) & ((1 << c.lg_rows) - 1)) : 0;
      p[u] = *reinterpret_cast<const int4*>(c.pos + row);
      if (!on) p[u] = make_int4(kPagedNoPos, kPagedNoPos, kPagedNoPos, kPagedNoPos);
      if (!on && slot + 4 * u < end && c.status) atomicOr(c.status, DFLASH_PAGED_BAD_PAGE);
    }
    int lo = INT32_MAX, hi = INT32_MIN;
    bool whole = slot + 16 <= end;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int v[4] = {p[u].x, p[u].y, p[u].z, p[u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool there = v[j] != kPagedNoPos && slot + 4 * u + j < end;
        whole = whole && there;
        lo = min(lo, there ? v[j] : INT32_MAX);
        hi = max(hi, there ? v[j] : INT32_MIN);
      }
    }
    int w = whole;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      w &= __shfl_xor_sync(0xffffffffu, w, o);
    }
    if ((lane & (kLanes - 1)) == 0 && tile < t1) {
      const int k = paged_class(m, qmin, qmax, lo, hi, w != 0);
      if (k >= 1) atomicOr(&some[(tile - t0) >> 5], 1u << ((tile - t0) & 31));
      if (k == 2) atomicOr(&all[(tile - t0) >> 5], 1u << ((tile - t0) & 31));
    }
  }
}

// The tiles that split z of n takes of the key tiles of a sequence: an equal
// range of them, which it classifies, or, with a window over more than
// kDirect n tiles, where most are seen by nobody, an equal share of those that
// are seen (skip .. skip + take - 1 in order), for which every split classifies
// all. A range of at most kDirect tiles is not classified: the two dependent
// loads and the meeting of the CTA would cost more than a tile too many (4 rows in
// a window of 2048: 13.9 us instead of 15.7 us).
constexpr int kDirect = 3;
struct PagedShare { int t0, t1, skip, take; bool by_share; };
__device__ __forceinline__ PagedShare paged_range(int tiles, int window, int z, int n) {
  if (window > 0 && tiles > kDirect * n) return PagedShare{0, tiles, 0, tiles, true};
  const int per = (tiles + n - 1) / n;
  const int a = min(tiles, z * per), b = min(tiles, a + per);
  return PagedShare{a, b, 0, b - a, false};
}
__device__ __forceinline__ bool paged_direct(const PagedShare& r) { return r.t1 - r.t0 <= kDirect; }
__device__ __forceinline__ void paged_take(PagedShare& r, const unsigned* some, int z, int n) {
  int seen = 0;
  for (int i = 0; i <= (r.t1 - r.t0) >> 5; ++i) seen += __popc(some[i]);
  r.skip = r.by_share ? (int)((long long)seen * z / n) : 0;
  r.take = r.by_share ? (int)((long long)seen * (z + 1) / n) - r.skip : seen;
}
// Walks the seen tiles of a share in ascending order.
struct PagedCursor {
  const unsigned* bits;
  int word, left;
  unsigned cur;
  __device__ __forceinline__ PagedCursor(const unsigned* some, const PagedShare& r) : bits(some), word(0), left(r.take) {
    int skip = r.skip;
    cur = left > 0 ? bits[0] : 0u;
    if (left > 0) {
      while (skip >= __popc(cur)) { skip -= __popc(cur); cur = bits[++word]; }
      while (skip-- > 0) cur &= cur - 1;
    }
  }
  // The next tile (relative to t0), or -1.
  __device__ __forceinline__ int next() {
    if (left <= 0) return -1;
    while (!cur) cur = bits[++word];
    const int b = __ffs(cur) - 1;
    cur &= cur - 1;
    --left;
    return word * 32 + b;
  }
};

}  // namespace dfl
