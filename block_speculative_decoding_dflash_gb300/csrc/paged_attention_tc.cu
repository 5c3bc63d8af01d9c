// The paged attention kernel of positions alone, and the maps of its operands.
#include "paged_attention_tc.cuh"

namespace dfl {

bool paged_map_pages(CUtensorMap* m, const void* base, const PagedView& c, int most) {
  const int rows = 1 << c.lg_rows;
  return tc_encode_map(m, base, c.hd, ((uint64_t)c.n_pages * c.nkv) << c.lg_rows, (uint64_t)c.hd * 2, 64,
                       rows < most ? rows : most);
}

bool paged_map_rows(CUtensorMap* m, const void* base, const PagedAttnArgs& a, int per) {
  const uint64_t dims[3] = {(uint64_t)a.c.hd, (uint64_t)a.nq, (uint64_t)a.rows};
  const uint64_t strides[2] = {(uint64_t)a.c.hd * 2, (uint64_t)a.q_stride * 2};
  const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)per};
  return tc_encode_map_3d(m, base, dims, strides, box);
}

cudaError_t launch_paged_attention_tc(const PagedAttnArgs& a, int q_tiles, long long tiles, cudaStream_t st) {
  if (a.c.hd <= 64) return q_tiles == 2 ? run<64, 2, false>(a, tiles, st) : run<64, 1, false>(a, tiles, st);
  return q_tiles == 2 ? run<128, 2, false>(a, tiles, st) : run<128, 1, false>(a, tiles, st);
}

}  // namespace dfl
