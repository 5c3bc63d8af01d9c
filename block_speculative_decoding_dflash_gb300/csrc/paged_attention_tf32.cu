// Attention over the paged cache in fp32, and in bf16 for heads of more than 128
// dimensions.
//
// The products run on the tensor cores in tf32 with every factor in two parts,
// x = hi + lo: x y = hi hi + hi lo + lo hi, whose missing lo lo is 2^-22 of x y, as
// much as lo's own rounding. Few query rows read K and V once, which the HBM
// bounds; on CUDA cores the same rows read them from shared memory many times
// over (8 sequences of up to 10 rows over up to 4099 keys, 8 heads: 84 us). A bf16
// value is a tf32 as it stands, so of bf16's factors only P has two parts.
//
// A CTA has 16 packed query rows (row r = token r / G, head r % G of the group)
// against 64 keys at a time. For the scores each of its 8 warps takes 8 of the
// keys; for P V an eighth of the dimensions. In both a lane's rows are the same,
// so the running maximum rescales the output where it lies. Which dimension (key)
// is which of an instruction's eight K elements is free as long as both operands
// agree, and so is the order of its columns: they are chosen so that a lane's
// elements are neighbours and shared loads are free of bank conflicts.
//
// A tensor core's sums are fp32 but not rounded to nearest: the large products of a
// tile are summed apart from the small ones, at most 16 of them in a chain, and
// tiles are joined by ordinary additions.
//
// K and V come by TMA, a box per page, 32 dimensions wide, into one buffer each:
// the next K arrives while P V runs, the next V while Q K^T does, and a second CTA
// on the SM fills the rest. (With cp.async, 16 to a thread and tile, half of a
// tile's time went into their instructions: 61 us.) Those blocks take 56 us, 2.3
// TB/s, 64 such sequences 384 us, 2.8 TB/s: nothing waits for memory any more; the
// time goes into taking values apart and into the products' latency (no pipe is
// full: issue 36%, tensor 31%, integer 31%; a warp waits for its own last step).
#include <math.h>

#include "paged_tc.cuh"
#include "paged_tf32.cuh"

namespace dfl {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBN = 64;
constexpr int kMaxTiles = (1 << 20) / kBN;

// W neighbours in one load.
template <int W>
struct Few {
  float v[W];
  __device__ __forceinline__ explicit Few(const float* p) {
    if constexpr (W == 4) *reinterpret_cast<float4*>(v) = load4(p);
    else if constexpr (W == 2) *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p);
    else v[0] = *p;
  }
  __device__ __forceinline__ explicit Few(const bf16* p) {
    static_assert(W == 4, "four bf16 to a load");
    *reinterpret_cast<float4*>(v) = load4(p);
  }
};
// Whether 16 bytes hold an infinity or NaN: an exponent of all ones carries into the sign's place.
template <typename T>
__device__ __forceinline__ bool not_finite(const uint4& u) {
  constexpr uint32_t kExp = sizeof(T) == 4 ? 0x7f800000u : 0x7f807f80u, kOne = sizeof(T) == 4 ? 0x00800000u : 0x00800080u;
  return ((((u.x & kExp) + kOne) | ((u.y & kExp) + kOne) | ((u.z & kExp) + kOne) | ((u.w & kExp) + kOne)) & (kOne << 8)) != 0;
}

constexpr int kBM = 16, kWarps = 8;

template <typename T, int HDP>
struct Tf32Shape {
  static constexpr int kCols = 128 / sizeof(T), kSub = HDP / kCols;   // K and V tiles lie in parts of 128 bytes a row, swizzled
  static constexpr int kTileB = kBN * HDP * sizeof(T), kSubB = kBN * 128;
  static constexpr int LDP = kBN + 8, LDQ = HDP + 16;
  static constexpr bool kQRegs = HDP <= 128;              // Q in registers, otherwise in shared memory
  static constexpr int kK = 0, kV = kTileB, kP = 2 * kTileB, kQ = kP + kBM * LDP * 4, kMax = kQ + (kQRegs ? 0 : kBM * LDQ * 4),
                       kRow = kMax + kWarps * kBM * 4, kBits = kRow + 2 * kBN * 4, kEnd = kBits + 2 * (kMaxTiles / 32 + 1) * 4;
  static constexpr size_t kSmem = kEnd + 1024;
};

template <typename T, int HDP>
__global__ void __launch_bounds__(kWarps * 32, HDP * sizeof(T) > 512 ? 1 : 2)
paged_attn_tf32_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const __grid_constant__ PagedAttnArgs a) {
  using C = Tf32Shape<T, HDP>;
  constexpr bool kParts = sizeof(T) == 4;
  constexpr int NT = kWarps * 32, LDP = C::LDP;
  constexpr int kSteps = HDP / 16;            // of 16 dimensions, two instructions each
  constexpr int W = HDP / 64;                 // a warp's tiles of 8 dimensions, all from one load
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t k_full, v_full;
  __shared__ PagedTile st;
  __shared__ int s_qmin, s_qmax;
  __shared__ unsigned s_bad[kBN / 32];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023) & ~1023u) - raw);
  float *sp = reinterpret_cast<float*>(sm + C::kP), *sq = reinterpret_cast<float*>(sm + C::kQ), *smax = reinterpret_cast<float*>(sm + C::kMax);
  int* srow = reinterpret_cast<int*>(sm + C::kRow);       // [2][kBN] places of a tile's rows, -1 for none
  unsigned* some = reinterpret_cast<unsigned*>(sm + C::kBits);
  unsigned* all = some + kMaxTiles / 32 + 1;
  if (threadIdx.x == 0) {
    mbar_init(&k_full, 1);
    mbar_init(&v_full, 1);
    fence_mbar_init();
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  pdl_enter();
  const PagedView& c = a.c;
  const int h = blockIdx.y, z = blockIdx.z, G = a.G, hd = c.hd;
  if (threadIdx.x < 32) {
    const PagedTile t = paged_find_tile(a.start, c.n_seq, a.rows, G, kBM, blockIdx.x);
    int lo = INT32_MAX, hi = INT32_MIN;
    if (t.seq >= 0) {
      const int r0 = t.tile * kBM, r1 = min(t.count * G, r0 + kBM);
      for (int i = r0 / G + (int)threadIdx.x; i <= (r1 - 1) / G; i += 32) {
        const int p = a.q_pos[t.first + i];
        lo = min(lo, p);
        hi = max(hi, p);
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (threadIdx.x == 0) { st = t; s_qmin = lo; s_qmax = hi; }
  }
  __syncthreads();
  const PagedTile t = st;
  if (t.seq < 0) return;
  const int len = paged_length(c, t.seq);
  if (threadIdx.x == 0 && h == 0 && z == 0 && t.tile == 0) paged_report_length(c, t.seq, len);
  const PagedMask m = paged_mask(a.causal, a.window, a.prefix, t.seq);
  PagedShare sh = paged_range((len + kBN - 1) / kBN, a.window, z, a.splits);
  const int r0 = t.tile * kBM, n_rows = min(kBM, t.count * G - r0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, e4 = lane & 3;
  // Q, zeros past hd and past the last row
  auto q_at = [&](int r, int d) {
    return r < n_rows && d < hd ? load4(static_cast<const T*>(a.q) + (size_t)(t.first + (r0 + r) / G) * a.q_stride + (size_t)(h * G + (r0 + r) % G) * hd + d)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 q[C::kQRegs ? kSteps : 1][2];
  if constexpr (C::kQRegs) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) q[s][i] = q_at(g + 8 * i, s * 16 + e4 * 4);
  } else {
    for (int e = threadIdx.x; e < kBM * HDP / 4; e += NT) *reinterpret_cast<float4*>(sq + e / (HDP / 4) * C::LDQ + e % (HDP / 4) * 4) = q_at(e / (HDP / 4), e % (HDP / 4) * 4);
  }
  paged_classify<kBN>(c, t.seq, h, len, m, s_qmin, s_qmax, sh.t0, sh.t1, some, all);
  // of the lane's two rows, g and g + 8
  int pq[2];
  PagedSees sees[2];
  float slope2[2], mx[2], sum[2], o[W][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + min(g + 8 * i, n_rows - 1);
    pq[i] = a.q_pos[t.first + r / G];
    sees[i] = paged_sees_of(m, pq[i]);
    slope2[i] = a.slopes ? a.slopes[h * G + r % G] * kLog2e : 0.f;
    mx[i] = -INFINITY;
    sum[i] = 0.f;
  }
#pragma unroll
  for (int n = 0; n < W; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
  // a score in log2 units: dot * scale2, or cap2 * tanh(dot * scale2)
  const float scale2 = a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e, cap2 = a.softcap * kLog2e;
  __syncthreads();
  paged_take(sh, some, z, a.splits);
  PagedCursor cur(some, sh);

  // A row's place: its page is requested a tile before it is needed.
  const int my_slot = threadIdx.x & (kBN - 1);
  auto page_of = [&](int rel) {
    const int slot = (sh.t0 + rel) * kBN + my_slot;
    return threadIdx.x < kBN && rel >= 0 && slot < len ? c.table[(size_t)t.seq * c.max_pages + (slot >> c.lg_rows)] : -1;
  };
  auto put_row = [&](int* rows, int rel, int page) {
    const int slot = (sh.t0 + rel) * kBN + my_slot;
    if (threadIdx.x < kBN)
      rows[my_slot] = (unsigned)page < (unsigned)c.n_pages ? ((page * c.nkv + h) << c.lg_rows) + (slot & ((1 << c.lg_rows) - 1)) : -1;
  };
  const int box = min(1 << c.lg_rows, kBN), boxes = kBN / box;
  const int beyond = (c.n_pages * c.nkv) << c.lg_rows;     // a row past the pool reads as zeros
  // warp 0: the boxes of a tile
  auto copy = [&](int off, const CUtensorMap* map, const int* rows, uint64_t* bar) {
    if (lane == 0) mbar_expect_tx(bar, C::kTileB);
    __syncwarp();
    if (lane >= boxes) return;
    const int row = rows[lane * box], y = row >= 0 ? row : beyond;
#pragma unroll
    for (int x = 0; x < C::kSub; ++x) tma_load_2d(sm + off + x * C::kSubB + lane * box * 128, map, x * 64, y, bar);
  };
  bool ok = true;
  unsigned phase = 0;
  int rel = cur.next(), next = cur.next(), buf = 0, page = page_of(next);
  if (rel >= 0) put_row(srow, rel, page_of(rel));
  __syncthreads();
  if (rel >= 0 && warp == 0) {
    copy(C::kK, &mk, srow, &k_full);
    copy(C::kV, &mv, srow, &v_full);
  }
  // where this lane's K and V elements lie: K's row 8 warp + perm(g) (column g of the
  // instruction is that key), V's rows 2 e4, + 1, + 8, + 9 of every 16
  const int k_row = warp * 8 + (g >> 1) + 4 * (g & 1);
  const uint8_t* k_at = sm + C::kK + k_row * 128;
  const uint8_t* v_at = sm + C::kV + warp * 8 * W / C::kCols * C::kSubB;
  const int v_byte = (warp * 8 * W + g * W) % C::kCols * (int)sizeof(T);
  for (; rel >= 0; buf ^= 1, phase ^= 1) {
    const bool full = (all[rel >> 5] >> (rel & 31)) & 1u;
    const int* rows = srow + buf * kBN;
    if (next >= 0) put_row(srow + (buf ^ 1) * kBN, next, page);
    const int after = cur.next();
    page = page_of(after);
    int pk[2] = {kPagedNoPos, kPagedNoPos};               // of keys 8 warp + e4, + 4
    if (!full || a.slopes)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = rows[warp * 8 + e4 + 4 * x];
        if (row >= 0) pk[x] = c.pos[row];
      }
    paged_wait(&k_full, phase, ok);
    // scores of rows g, g + 8 and keys 8 warp + e4, + 4
    float s4[4], odd[4], low[2][4];
#pragma unroll
    for (int x = 0; x < 4; ++x) s4[x] = odd[x] = low[0][x] = low[1][x] = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      uint32_t qh[2][4], ql[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4 v = C::kQRegs ? q[C::kQRegs ? s : 0][i] : *reinterpret_cast<const float4*>(sq + (g + 8 * i) * C::LDQ + s * 16 + e4 * 4);
        // (not to be taken out of the loop: the parts of all of Q do not fit the registers)
        asm volatile("" : "+f"(v.x), "+f"(v.y), "+f"(v.z), "+f"(v.w));
        round2(v.x, qh[i][0], ql[i][0]);
        round2(v.y, qh[i][1], ql[i][1]);
        round2(v.z, qh[i][2], ql[i][2]);
        round2(v.w, qh[i][3], ql[i][3]);
      }
      const int k_byte = (s * 16 + e4 * 4) % C::kCols * (int)sizeof(T);
      const float4 k = load4(reinterpret_cast<const T*>(k_at + s * 16 / C::kCols * C::kSubB + (((k_byte >> 4) ^ (k_row & 7)) << 4) + (k_byte & 15)));
      uint32_t kh[4], kl[4];
      cut2(k.x, kh[0], kl[0]);
      cut2(k.y, kh[1], kl[1]);
      cut2(k.z, kh[2], kl[2]);
      cut2(k.w, kh[3], kl[3]);
      float* big = s & 1 ? odd : s4;
#pragma unroll
      for (int x = 0; x < 4; x += 2) {
        mma_tf32(big, qh[0][x], qh[1][x], qh[0][x + 1], qh[1][x + 1], kh[x], kh[x + 1]);
        if (!kParts) continue;
        mma_tf32(low[0], qh[0][x], qh[1][x], qh[0][x + 1], qh[1][x + 1], kl[x], kl[x + 1]);
        mma_tf32(low[1], ql[0][x], ql[1][x], ql[0][x + 1], ql[1][x + 1], kh[x], kh[x + 1]);
      }
    }
    unsigned seen = 0;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = x >> 1;
      float u = (s4[x] + odd[x] + (low[0][x] + low[1][x])) * scale2;
      if (a.softcap > 0.f) u = cap2 * tanhf(u);
      if (a.slopes) u -= slope2[i] * fabsf((float)(pq[i] - pk[x & 1]));
      const bool v = full || paged_sees(sees[i], pk[x & 1]);
      s4[x] = v ? u : -INFINITY;
      seen |= (unsigned)v << x;
      top[i] = fmaxf(top[i], s4[x]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
      if (e4 == 0) smax[warp * kBM + g + 8 * i] = top[i];
    }
    __syncthreads();                         // maxima of all warps; K is free
    if (warp == 0 && next >= 0) copy(C::kK, &mk, srow + (buf ^ 1) * kBN, &k_full);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mn = mx[i];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mn = fmaxf(mn, smax[w * kBM + g + 8 * i]);
      const float base = mn == -INFINITY ? 0.f : mn;
      if (mn != mx[i]) {
        const float f = exp2f(mx[i] - base);
        sum[i] *= f;
        mx[i] = mn;
#pragma unroll
        for (int n = 0; n < W; ++n) {
          o[n][2 * i] *= f;
          o[n][2 * i + 1] *= f;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float p = exp2f(s4[2 * i + x] - base);
        sum[i] += p;
        // a hidden row's weight is -0, a seen one's that underflowed +0
        sp[(g + 8 * i) * LDP + warp * 8 + e4 + 4 * x] = (seen >> (2 * i + x)) & 1u ? p : -0.f;
      }
    }
    if (threadIdx.x < kBN / 32) s_bad[threadIdx.x] = 0u;
    paged_wait(&v_full, phase, ok);
    __syncthreads();
    // Infinite or NaN values of V in a tile that some query sees only in part:
    // its hidden rows must not be multiplied by their zero weight. Such rows are
    // made zeros, and added where they are seen.
    bool careful = false;
    if (!full) {
      unsigned bad = 0;
      constexpr int kEach = C::kTileB / 16 / NT;            // 16-byte pieces of a thread
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        bad |= (unsigned)not_finite<T>(*reinterpret_cast<const uint4*>(sm + C::kV + (i * NT + threadIdx.x) * 16)) << i;
      }
      careful = __syncthreads_or(bad != 0);
      if (careful) {
        for (int i = 0; i < kEach; ++i) {
          const int j = ((i * NT + (int)threadIdx.x) >> 3) & (kBN - 1);
          if ((bad >> i) & 1u) atomicOr(&s_bad[j >> 5], 1u << (j & 31));
        }
        __syncthreads();
        for (int i = 0; i < kEach; ++i) {
          const int e = i * NT + threadIdx.x, j = (e >> 3) & (kBN - 1);
          if ((s_bad[j >> 5] >> (j & 31)) & 1u) *reinterpret_cast<float4*>(sm + C::kV + e * 16) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        fence_proxy_async_shared();          // the next copy comes after these writes
        __syncthreads();
      }
    }
    // rows g, g + 8 and dimensions 8 W warp + W (2 e4 + x) + n
    float big[W][4], small[W][4];
#pragma unroll
    for (int n = 0; n < W; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) big[n][x] = small[n][x] = 0.f;
#pragma unroll
    for (int s = 0; s < kBN / 16; ++s) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int key = s * 16 + y * 8 + e4 * 2;           // and the next
        uint32_t ph[2][2], pl[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 p = *reinterpret_cast<const float2*>(sp + (g + 8 * i) * LDP + key);
          round2(p.x, ph[i][0], pl[i][0]);
          round2(p.y, ph[i][1], pl[i][1]);
        }
        const Few<W> v0(reinterpret_cast<const T*>(v_at + key * 128 + (((v_byte >> 4) ^ (key & 7)) << 4) + (v_byte & 15)));
        const Few<W> v1(reinterpret_cast<const T*>(v_at + (key + 1) * 128 + (((v_byte >> 4) ^ (key + 1 & 7)) << 4) + (v_byte & 15)));
#pragma unroll
        for (int n = 0; n < W; ++n) {
          uint32_t h0, l0, h1, l1;
          cut2(v0.v[n], h0, l0);
          cut2(v1.v[n], h1, l1);
          mma_tf32(big[n], ph[0][0], ph[1][0], ph[0][1], ph[1][1], h0, h1);
          if (kParts) mma_tf32(small[n], ph[0][0], ph[1][0], ph[0][1], ph[1][1], l0, l1);
          mma_tf32(small[n], pl[0][0], pl[1][0], pl[0][1], pl[1][1], h0, h1);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < W; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[n][x] += big[n][x] + small[n][x];
    if (careful) {
      for (int j = 0; j < kBN; ++j) {
        if (!((s_bad[j >> 5] >> (j & 31)) & 1u) || rows[j] < 0) continue;
        const T* v = static_cast<const T*>(c.v) + (long long)rows[j] * hd;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p = sp[(g + 8 * i) * LDP + j];
          if (__float_as_uint(p) == 0x80000000u) continue;
#pragma unroll
          for (int n = 0; n < W; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int d = (warp * 8 + 2 * e4 + x) * W + n;
              if (d < hd) o[n][2 * i + x] = fmaf(p, to_f(v[d]), o[n][2 * i + x]);
            }
        }
      }
    }
    const bool stop = __syncthreads_or(!ok);   // V and P are free
    if (warp == 0 && next >= 0 && !stop) copy(C::kV, &mv, srow + (buf ^ 1) * kBN, &v_full);
    if (stop) {
      // a wait gave up: the K on its way, and what V there was, land before the CTA ends
      ok = false;
      bool landed = true;
      paged_wait(&v_full, phase, landed);
      if (next >= 0) paged_wait(&k_full, phase ^ 1, landed);
      if (threadIdx.x == 0 && c.status) atomicOr(c.status, DFLASH_PAGED_GAVE_UP);
      break;
    }
    rel = next;
    next = after;
  }
  // the sums over the warps' keys
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    if (e4 == 0) smax[warp * kBM + g + 8 * i] = sum[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i;
    if (r >= n_rows) continue;
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += smax[w * kBM + r];
    const size_t at = (size_t)(t.first + (r0 + r) / G) * a.nq + h * G + (r0 + r) % G;
    const bool none = total == 0.f;          // nothing seen (a NaN score makes the sum NaN)
    const bool split = a.splits > 1;
    const float inv = none ? 0.f : (split ? 1.f : 1.f / total);
    float* part = a.part_o + ((size_t)z * a.rows * a.nq + at) * hd;
    T* out = static_cast<T*>(a.out) + at * hd;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int d = (warp * 8 + 2 * e4 + x) * W;
      if (d >= hd) continue;
#pragma unroll
      for (int n = 0; n < W; ++n) {
        const float v = none ? 0.f : o[n][2 * i + x] * inv;
        if (split) part[d + n] = v;
        else out[d + n] = from_f<T>(v);
      }
    }
    if (warp || e4) continue;
    if (split) a.part_ml[(size_t)z * a.rows * a.nq + at] = make_float2(mx[i], total);
    else if (a.lse) a.lse[at] = none ? -INFINITY : (mx[i] + log2f(total)) * kLn2;
  }
}

template <typename T, int HDP>
cudaError_t run(const PagedAttnArgs& a, long long tiles, cudaStream_t st) {
  // (fp32 rows are mapped as bf16 rows of twice the columns: the bytes are what counts)
  PagedView c = a.c;
  c.hd *= sizeof(T) / 2;
  CUtensorMap mk, mv;
  if (!paged_map_pages(&mk, c.k, c, kBN) || !paged_map_pages(&mv, c.v, c, kBN)) return cudaErrorInvalidValue;
  auto kernel = paged_attn_tf32_kernel<T, HDP>;
  constexpr size_t smem = Tf32Shape<T, HDP>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)tiles, a.c.nkv, a.splits), dim3(kWarps * 32), smem, st, mk, mv, a);
}

}  // namespace

cudaError_t launch_paged_attention_tf32(int dtype, const PagedAttnArgs& a, long long tiles, cudaStream_t st) {
  if (dtype) return run<bf16, 256>(a, tiles, st);
  if (a.c.hd <= 64) return run<float, 64>(a, tiles, st);
  return a.c.hd <= 128 ? run<float, 128>(a, tiles, st) : run<float, 256>(a, tiles, st);
}

}  // namespace dfl
