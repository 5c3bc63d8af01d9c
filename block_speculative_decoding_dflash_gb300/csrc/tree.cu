// Trees of drafted tokens: the walk that accepts one of their paths, and the move of
// the accepted rows to the front of the tree's rows in the paged caches.
#include "kernels.h"
#include "launch.cuh"
#include "paged.cuh"

namespace dfl {

namespace {

// One warp walks one tree. The children of a row follow it, each behind the subtree
// of the one before; the warp keeps the tree's rows in shared memory, where a step
// of the walk takes some tens of cycles and not a memory latency. Bound by the launch
// and three dependent loads (256 trees of up to 64 rows: 4.2 us in a graph).
constexpr int kAcceptWarps = 4, kAcceptHeld = 256;

__global__ void __launch_bounds__(kAcceptWarps * 32) tree_accept_kernel(const TreeAcceptArgs a) {
  __shared__ int held[kAcceptWarps][3][kAcceptHeld];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, s = blockIdx.x * kAcceptWarps + warp;
  pdl_enter();
  if (s >= a.n_seq) return;
  const int2 ab = paged_new_rows(a.start, s, a.rows);
  const int n = ab.y - ab.x, length = a.length ? a.length[s] : 0;
  for (int i = lane; i < min(n, kAcceptHeld); i += 32) {
    held[warp][0][i] = a.end[ab.x + i];
    held[warp][1][i] = a.draft[ab.x + i];
    held[warp][2][i] = a.sampled[ab.x + i];
  }
  __syncwarp();
  const int* const from[3] = {a.end + ab.x, a.draft + ab.x, a.sampled + ab.x};
  auto at = [&](int what, int i) { return i < kAcceptHeld ? held[warp][what][i] : from[what][i]; };
  int count = 0;
  for (int cur = n > 0 ? 0 : -1; cur >= 0 && count < a.width; ++count) {
    const int said = at(2, cur);
    if (said < 0) break;                     // the row had nothing to draw: the walk ends before it
    if (lane == 0) {
      a.tokens[(long long)s * a.width + count] = said;
      a.path[(long long)s * a.width + count] = cur;
    }
    const int end = min(at(0, cur), n);
    int child = cur + 1;
    while (child < end && at(1, child) != said) child = max(at(0, child), child + 1);
    cur = child < end ? child : -1;
  }
  for (int i = count + lane; i < a.width; i += 32) a.tokens[(long long)s * a.width + i] = a.path[(long long)s * a.width + i] = -1;
  if (lane == 0) {
    a.count[s] = count;
    if (a.length_out) a.length_out[s] = length - n + count;
  }
}

// Of a sequence and a cache: each thread owns one column, 16 bytes of K or V of one
// head, or one head's position or weight, and moves it row by row. Row i of the path
// goes to a place at or before its own, and later rows come from places behind it,
// so a thread that goes in order overwrites nothing that it still needs. Bound by its
// chain of loads, count, path, page, row (48 sequences and 24 layers: 7.3 us in a graph, 1.4
// TB/s), which is why eight rows are requested together.
constexpr int kCommitThreads = 512, kCommitRows = 64;         // at most; a CTA has kCommitRows threads at least

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const __grid_constant__ TreeCommitArgs a) {
  __shared__ long long from[kCommitRows], to[kCommitRows];   // rows of head 0, -1: not to be moved
  const int s = blockIdx.y, tid = threadIdx.x;
  const TreeCommitCache& c = a.cache[blockIdx.z];
  pdl_enter();
  int count = a.count[s];
  const int cap = a.max_pages << a.lg_rows, base = c.length[s] - count;
  bool bad_rows = count < 0 || count > a.width || (count > 0 && (base < 0 || base + count > cap)), bad_page = false;
  if (bad_rows) count = 0;
  const int* path = a.path + (long long)s * a.width;
  const int per_head = 2 * a.vecs + (c.weight ? 2 : 1), columns = a.nkv * per_head;
  const int e = blockIdx.x * blockDim.x + tid, head = e / per_head, x = e % per_head;
  for (int i0 = 0; i0 < count; i0 += kCommitRows) {
    __syncthreads();
    const int n = min(kCommitRows, count - i0);
    if (tid < n) {
      const int i = i0 + tid, p = path[i], before = i > 0 ? path[i - 1] : -1;
      long long f = -1, t = -1;
      if (p <= before || p < i || p >= cap - base) {
        bad_rows = true;
      } else if (p != i) {
        const int sf = base + p, st = base + i;
        const int pf = c.table[(long long)s * a.max_pages + (sf >> a.lg_rows)], pt = c.table[(long long)s * a.max_pages + (st >> a.lg_rows)];
        if ((unsigned)pf >= (unsigned)a.n_pages || (unsigned)pt >= (unsigned)a.n_pages) {
          bad_page = true;
        } else {
          f = (((long long)pf * a.nkv) << a.lg_rows) + (sf & ((1 << a.lg_rows) - 1));
          t = (((long long)pt * a.nkv) << a.lg_rows) + (st & ((1 << a.lg_rows) - 1));
        }
      }
      from[tid] = f;
      to[tid] = t;
    }
    __syncthreads();
    if (e >= columns) continue;
    const long long at_head = (long long)head << a.lg_rows;
    constexpr int kU = 8;                                    // rows requested together
    for (int j0 = 0; j0 < n; j0 += kU) {
      if (x < 2 * a.vecs) {
        uint4* p = static_cast<uint4*>(x < a.vecs ? c.k : c.v) + (x < a.vecs ? x : x - a.vecs);
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (j0 + u < n && from[j0 + u] >= 0) v[u] = p[(from[j0 + u] + at_head) * a.vecs];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (j0 + u < n && from[j0 + u] >= 0) p[(to[j0 + u] + at_head) * a.vecs] = v[u];
      } else {
        int* p = x == 2 * a.vecs ? c.pos : reinterpret_cast<int*>(c.weight);
        int v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (j0 + u < n && from[j0 + u] >= 0) v[u] = p[from[j0 + u] + at_head];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (j0 + u < n && from[j0 + u] >= 0) p[to[j0 + u] + at_head] = v[u];
      }
    }
  }
  if (blockIdx.x == 0 && c.status && (bad_rows || bad_page)) atomicOr(c.status, (bad_rows ? DFLASH_PAGED_BAD_ROWS : 0) | (bad_page ? DFLASH_PAGED_BAD_PAGE : 0));
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t st) {
  return launch_pdl(tree_accept_kernel, dim3((a.n_seq + kAcceptWarps - 1) / kAcceptWarps), dim3(kAcceptWarps * 32), 0, st, a);
}

cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t st) {
  // as few CTAs as there can be, and of as few warps (48 sequences of 272 columns in 24 layers by CTAs of 256: 8.8 us)
  const int columns = a.nkv * (2 * a.vecs + 2), ctas = (columns + kCommitThreads - 1) / kCommitThreads;
  const int threads = ((columns + ctas - 1) / ctas + 31) & ~31;
  return launch_pdl(tree_commit_kernel, dim3(ctas, a.n_seq, a.n_caches), dim3(threads < kCommitRows ? kCommitRows : threads), 0, st, a);
}

}  // namespace dfl
