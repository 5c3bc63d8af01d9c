// The paged attention kernel for trees of drafted tokens: instances of their own, so
// that calls without a tree keep their code.
#include "paged_attention_tc.cuh"

namespace dfl {

cudaError_t launch_paged_tree_attention_tc(const PagedAttnArgs& a, int q_tiles, long long tiles, cudaStream_t st) {
  if (a.c.hd <= 64) return q_tiles == 2 ? run<64, 2, true>(a, tiles, st) : run<64, 1, true>(a, tiles, st);
  return q_tiles == 2 ? run<128, 2, true>(a, tiles, st) : run<128, 1, true>(a, tiles, st);
}

}  // namespace dfl
