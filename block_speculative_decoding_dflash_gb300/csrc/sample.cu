// One token of each row of logits: temperature, top-k, top-p, min-p and a draw by a
// given uniform number.
//
// With M the row's largest logit a token's weight is w = 2^-((M - l) log2(e) / T).
// What the filters keep is a prefix of the tokens in descending order (ties: the
// lowest index first), so all of them together come down to one logit K and a
// number t: tokens above K are kept, of those equal to K the first t. Nothing is
// sorted: a histogram over M - l finds the bin in which the count (top-k) or the
// weight (top-p) is reached, histograms over the order of floats within that bin
// find K.
//
// Sums of weights decide which token is drawn, so they are exact: a weight is an
// integer, in units of 2^-44 of (nearly) the largest, a function of l, M and T alone;
// 64-bit sums of them are the same in any order and in every pass. A weight is right
// to about 2^-35: a prefix sum over a vocabulary then is off by some 2^-40 of the
// total, and a row's token is another than exact arithmetic's with a probability of
// 2^-22 or so even where all of 2^18 tokens weigh the same.
//
// A cluster of CTAs holds a row in its shared memory, each warp an unbroken stretch
// of the vocabulary; the logits are read from memory once. The CTAs exchange
// maxima, histograms and the warps' sums; each works out the outcome for itself, and
// the one that has the token writes it.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace dfl {

namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kNT = 512, kWarps = kNT / 32;
constexpr int kBins = kNT;
constexpr int kMaxCtas = 8;
constexpr int kSteps = 1024;               // of the exponential's table to a factor of 2
constexpr int kUnit = 44;                  // weights are integers of 2^-44

// 2^(-(i + 1) / 1024) as its first 24 bits and the rest. (A value of 1 would need a
// bit more; a factor common to all weights makes no difference.)
struct PowTable {
  float hi[kSteps], lo[kSteps];
  constexpr PowTable() : hi(), lo() {
    for (int i = 0; i < kSteps; ++i) {
      // Taylor's series at -(i + 1) / 1024 ln 2, in (-0.7, 0): below 2^-53 after 20 terms
      const double x = -(i + 1) / 1024.0 * 0.69314718055994530942;
      double sum = 1.0, term = 1.0;
      for (int k = 1; k <= 22; ++k) {
        term *= x / k;
        sum += term;
      }
      const long long whole = (long long)(sum * 16777216.0);
      hi[i] = (float)((double)whole / 16777216.0);
      lo[i] = (float)(sum - (double)whole / 16777216.0);
    }
    hi[kSteps - 1] = 0.5f;                 // (its 24 bits start at one half)
    lo[kSteps - 1] = 0.f;
  }
};
__device__ constexpr PowTable kPow{};

// The weight of a logit at distance M - l, for rows of one temperature.
struct Weigh {
  const float2* table;
  float top, chi, clo, far;                // log2(e) / T in two parts; the distance beyond which a weight is zero
  // The weight of a token within `far` as whole * 2^-shift units, before the shift drops bits.
  // EXACT: M - l is an fp32 number (of bf16 logits, whose distance is one wherever it counts).
  template <bool EXACT>
  __device__ __forceinline__ void parts(float l, u64& whole, int& shift) const {
    const float d = top - l, p = d * chi;
    float e = fmaf(d, clo, fmaf(d, chi, -p));
    if (!EXACT) {
      const float b = d - top;
      e = fmaf((top - (d - b)) + (-l - b), chi, e);
    }
    constexpr float kMagic = 12288.f;      // 1.5 * 2^13: sums are multiples of 2^-10
    const float t = p + kMagic;
    const int i = __float_as_int(t) & 0x3fffff;
    const float r = (p - (t - kMagic)) + e;               // p = i / 1024 + r, |r| <= 2^-11
    const float g = r * fmaf(r, fmaf(r, -0.0555041087f, 0.240226507f), -0.693147181f);   // 2^-r - 1
    const float2 w = table[i & (kSteps - 1)];
    const int c = __float2int_rn(fmaf(w.x, g, w.y) * 4398046511104.f);                   // the rest, in 2^-42
    const int a = (__float_as_int(w.x) & 0x7fffff) | 0x800000;                           // the first 24 bits, in 2^-24
    whole = (u64)(((long long)a << (kUnit - 24)) + ((long long)c << (kUnit - 42)));
    shift = i >> 10;
  }
  template <bool EXACT>
  __device__ __forceinline__ u64 of(float l) const {
    if (!(top - l <= far)) return 0ull;
    u64 whole;
    int shift;
    parts<EXACT>(l, whole, shift);
    return (whole >> shift) | 1ull;        // (what the shift drops is made up for by a set last bit, on average)
  }
};

// The order of floats as an unsigned number (-0 as 0).
template <typename T>
__device__ __forceinline__ unsigned key_of(float x) {
  const int u = __float_as_int(x + 0.f);
  return ((unsigned)u ^ ((unsigned)(u >> 31) | 0x80000000u)) >> (sizeof(T) == 2 ? 16 : 0);
}
template <typename T>
__device__ __forceinline__ float of_key(unsigned k) {
  if (sizeof(T) == 2) k = (k << 16) | (k & 0x8000u ? 0u : 0xffffu);
  return __int_as_float((int)(k & 0x80000000u ? k ^ 0x80000000u : ~k));
}

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  // NaN counts as -inf, +inf as the type's largest number.
  static __device__ __forceinline__ uint4 clean(uint4 u) {
    unsigned* w = reinterpret_cast<unsigned*>(&u);
    if constexpr (sizeof(T) == 2) {
      const unsigned any = ((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
                           ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u);
      if (any & 0x80008000u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int s = 0; s < 32; s += 16) {
            const unsigned x = (w[i] >> s) & 0xffffu;
            const unsigned y = x == 0x7f80u ? 0x7f7fu : (x & 0x7fffu) > 0x7f80u ? 0xff80u : x;
            w[i] ^= (x ^ y) << s;
          }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned x = w[i];
        w[i] = x == 0x7f800000u ? 0x7f7fffffu : (x & 0x7fffffffu) > 0x7f800000u ? 0xff800000u : x;
      }
    }
    return u;
  }
  static __device__ __forceinline__ float at(const uint4& u, int i) {
    const unsigned* w = reinterpret_cast<const unsigned*>(&u);
    if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    return __uint_as_float(w[i]);
  }
};

// A row as vectors of 16 bytes: vector j holds the elements j * N - lead + 0 .. N - 1,
// -inf where the row has none.
template <typename T>
struct Row {
  const T* base;
  int lead, vocab;
  __device__ __forceinline__ uint4 load(int j) const {
    constexpr int N = Vec<T>::N;
    const int v = j * N - lead;
    if (v >= 0 && v + N <= vocab) return Vec<T>::clean(__ldcs(reinterpret_cast<const uint4*>(base + v)));
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = v + i >= 0 && v + i < vocab ? base[v + i] : from_f<T>(-INFINITY);
    return Vec<T>::clean(u);
  }
};

struct Shared {
  unsigned lo[2][kBins], hi[2][kBins];     // histograms, which take turns
  float2 range;                            // of the CTA's logits
  u64 sum[kWarps];                         // of each warp's stretch: the weight above K,
  int equal[kWarps];                       // and how many are K
  unsigned kmin, kmax;
  u64 scan[kWarps];
  u64 found_before, total;
  int found;
};

// Inclusive sums over the CTA's threads.
__device__ __forceinline__ u64 scan_block(u64 x, u64* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = x;
  __syncthreads();
  u64 before = 0;
  for (int i = 0; i < warp; ++i) before += s[i];
  return x + before;
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kNT) sample_kernel(const SampleArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr bool kExact = sizeof(T) == 2;
  extern __shared__ __align__(16) uint4 held[];
  __shared__ Shared sh;
  __shared__ float2 table[kSteps];
  cg::cluster_group cl = cg::this_cluster();
  const int ctas = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r = blockIdx.x / ctas;
  for (int i = tid; i < kSteps; i += kNT) table[i] = make_float2(kPow.hi[i], kPow.lo[i]);
  sh.lo[0][tid] = sh.hi[0][tid] = sh.lo[1][tid] = sh.hi[1][tid] = 0u;
  pdl_enter();

  // ---- the row's stretch of this warp, and the largest and smallest logit
  Row<T> row;
  row.base = static_cast<const T*>(a.logits) + r * a.stride;
  row.lead = (int)((reinterpret_cast<uintptr_t>(row.base) & 15u) / sizeof(T));
  row.vocab = a.vocab;
  const int vectors = (row.lead + a.vocab + N - 1) / N, per = (vectors + ctas - 1) / ctas, each = (per + kWarps - 1) / kWarps;
  const int c0 = min(vectors, rank * per), c1 = min(vectors, c0 + per);
  const int v0 = min(c1, c0 + warp * each), v1 = min(c1, v0 + each);
  auto vector = [&](int j) { return STAGED ? held[j - c0] : row.load(j); };
  float hi = -INFINITY, lo = INFINITY;
#pragma unroll 4
  for (int j = v0 + lane; j < v1; j += 32) {
    const uint4 u = row.load(j);
    if (STAGED) held[j - c0] = u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float l = Vec<T>::at(u, i);
      hi = fmaxf(hi, l);
      lo = fminf(lo, l == -INFINITY ? INFINITY : l);
    }
  }
  hi = warp_max(hi);
  lo = -warp_max(-lo);
  if (lane == 0) sh.scan[warp] = ((u64)__float_as_uint(lo) << 32) | __float_as_uint(hi);
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < kWarps; ++i) {
      hi = fmaxf(hi, __uint_as_float((unsigned)sh.scan[i]));
      lo = fminf(lo, __uint_as_float((unsigned)(sh.scan[i] >> 32)));
    }
    sh.range = make_float2(hi, lo);
  }
  cl.sync();
  hi = -INFINITY;
  lo = INFINITY;
  for (int i = 0; i < ctas; ++i) {
    const float2 x = *cl.map_shared_rank(&sh.range, i);
    hi = fmaxf(hi, x.x);
    lo = fminf(lo, x.y);
  }
  if (hi == -INFINITY) {                   // nothing to choose from
    if (rank == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.prob) a.prob[r] = 0.f;
    }
    cl.sync();
    return;
  }

  // ---- the row's parameters
  const float temp = a.temperature ? a.temperature[r] : 1.f;
  const int top_k = a.top_k ? a.top_k[r] : 0;
  const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;
  const bool greedy = !(temp >= 5.4210109e-20f);          // 2^-64
  Weigh weigh;
  weigh.table = table;
  weigh.top = hi;
  {
    const double c = greedy ? 1.0 : 1.44269504088896340736 / (double)temp;
    weigh.chi = (float)c;
    weigh.clo = (float)(c - (double)weigh.chi);
    weigh.far = fminf((float)(kUnit / c), FLT_MAX);
  }
  int parity = 0;                          // the histogram in use
  float K = greedy ? hi : -INFINITY;       // kept: what is above K, and the first t of those equal to K
  u64 t = greedy ? 1 : 0;
  bool all = !greedy;                      // no cut so far

  // The histogram of all CTAs: this thread's bin, and the sum up to and with it.
  auto merged = [&](bool weights, u64& bin, u64& upto) {
    cl.sync();
    bin = 0;
    for (int i = 0; i < ctas; ++i) {
      bin += *cl.map_shared_rank(&sh.lo[parity][tid], i);
      if (weights) bin += (u64)*cl.map_shared_rank(&sh.hi[parity][tid], i) << 32;
    }
    upto = scan_block(bin, sh.scan);
    if (tid == kNT - 1) sh.total = upto;
    parity ^= 1;
    sh.lo[parity][tid] = sh.hi[parity][tid] = 0u;         // everyone has read it: they came to the last meeting since
    __syncthreads();
  };
  auto add = [&](bool weights, int bin, u64 w) {
    const unsigned old = atomicAdd(&sh.lo[parity][bin], (unsigned)w);
    if (weights) atomicAdd(&sh.hi[parity][bin], (unsigned)(w >> 32) + (old + (unsigned)w < old ? 1u : 0u));
  };
  // Cuts what is kept so far (above K, t of those equal to K) where the running
  // count (or weight) reaches `part` (a share of all of it, for weights).
  auto cut = [&](bool weights, double part) {
    const float K0 = K;
    const u64 t0 = t, wK = !all && weights ? weigh.of<kExact>(K0) : 1ull;
    const u64 tail = all ? 0ull : t0 * wK;                // what those equal to K count
    const float reach = fminf(weigh.far, hi - lo), scale = reach > 0.f ? (float)kBins / reach : 0.f;
    auto bin_of = [&](float l) { return min(kBins - 1, (int)((hi - l) * scale)); };
    auto in = [&](float l) { return l > K0 && hi - l <= weigh.far; };
#pragma unroll 1
    for (int j = v0 + lane; j < v1; j += 32) {
      const uint4 u = vector(j);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float l = Vec<T>::at(u, i);
        if (in(l)) add(weights, bin_of(l), weights ? weigh.of<kExact>(l) : 1ull);
      }
    }
    u64 bin, upto;
    merged(weights, bin, upto);
    const u64 total = sh.total + tail;
    u64 goal;                              // a token stays if what comes before it is below this
    if (weights) {
      const double g = ceil(part * (double)total);
      goal = g >= 18446744073709551615.0 ? ~0ull : g > 1.0 ? (u64)g : 1ull;
    } else {
      goal = (u64)part;
    }
    if (goal >= total) return;             // all of it
    if (goal > sh.total) {                 // reached among those equal to K
      const u64 n = (goal - sh.total + wK - 1) / wK;
      if (n < t0) t = n;
      return;
    }
    if (upto >= goal && upto - bin < goal) {
      sh.found = tid;
      sh.found_before = upto - bin;
    }
    if (tid == 0) { sh.kmin = 0xffffffffu; sh.kmax = 0u; }
    __syncthreads();
    const int where = sh.found;
    u64 before = sh.found_before;
    // the span of the bin in the order of floats
    unsigned kmin = 0xffffffffu, kmax = 0u;
#pragma unroll 1
    for (int j = v0 + lane; j < v1; j += 32) {
      const uint4 u = vector(j);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float l = Vec<T>::at(u, i);
        if (in(l) && bin_of(l) == where) {
          const unsigned k = key_of<T>(l);
          kmin = min(kmin, k);
          kmax = max(kmax, k);
        }
      }
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
      atomicMin(&sh.kmin, kmin);
      atomicMax(&sh.kmax, kmax);
    }
    cl.sync();
    for (int i = 0; i < ctas; ++i) {
      kmin = min(kmin, *cl.map_shared_rank(&sh.kmin, i));
      kmax = max(kmax, *cl.map_shared_rank(&sh.kmax, i));
    }
    while (kmin != kmax) {
      int shift = 0;
      while ((kmax - kmin) >> shift >= (unsigned)kBins) ++shift;
#pragma unroll 1
      for (int j = v0 + lane; j < v1; j += 32) {
        const uint4 u = vector(j);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float l = Vec<T>::at(u, i);
          const unsigned k = key_of<T>(l);
          if (k >= kmin && k <= kmax && in(l) && bin_of(l) == where) add(weights, (int)((kmax - k) >> shift), weights ? weigh.of<kExact>(l) : 1ull);
        }
      }
      merged(weights, bin, upto);
      if (before + upto >= goal && before + upto - bin < goal) {
        sh.found = tid;
        sh.found_before = before + upto - bin;
      }
      __syncthreads();
      before = sh.found_before;
      kmax -= (unsigned)sh.found << shift;
      const unsigned low = kmax - ((1u << shift) - 1u);
      kmin = max(kmin, low > kmax ? 0u : low);
      if (shift == 0) kmin = kmax;
      __syncthreads();
    }
    K = of_key<T>(kmax);
    t = weights ? (goal - before + weigh.of<kExact>(K) - 1) / weigh.of<kExact>(K) : goal - before;
    all = false;
  };
  if (!greedy && top_k > 0 && top_k < a.vocab) cut(false, (double)top_k);
  if (!greedy && top_p < 1.f) cut(true, (double)fmaxf(top_p, 0.f));
  if (!greedy && min_p > 0.f) {
    // l >= M + T ln(min_p): the smallest fp32 that is
    const double least = (double)hi + (double)temp * log((double)fminf(min_p, 1.f));
    const float f = __double2float_ru(least);
    if (f > K) {
      K = f;
      t = ~0ull;
      all = false;
    }
  }

  // ---- each warp's weight above K and number equal to K
  u64 sum = 0;
  int equal = 0;
#pragma unroll 1
  for (int j = v0 + lane; j < v1; j += 32) {
    const uint4 u = vector(j);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float l = Vec<T>::at(u, i);
      if (l > K) sum += weigh.of<kExact>(l);
      equal += l == K;
    }
  }
  u64 all_sum = sum;
#pragma unroll
  for (int o = 16; o; o >>= 1) all_sum += __shfl_xor_sync(0xffffffffu, all_sum, o);
  const int all_equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    sh.sum[warp] = all_sum;
    sh.equal[warp] = all_equal;
  }
  cl.sync();
  const u64 wK = all ? 0ull : weigh.of<kExact>(K);
  u64 mine = 0, eq = 0;
  if (tid < ctas * kWarps) {
    mine = *cl.map_shared_rank(&sh.sum[tid % kWarps], tid / kWarps);
    eq = (u64)*cl.map_shared_rank(&sh.equal[tid % kWarps], tid / kWarps);
  }
  const u64 eq_before = scan_block(eq, sh.scan) - eq;
  const u64 take = eq_before >= t ? 0 : min(eq, t - eq_before);
  mine += take * wK;
  const u64 upto = scan_block(mine, sh.scan);
  if (tid == kNT - 1) {
    sh.total = upto;
    sh.found = -1;
  }
  __syncthreads();
  const u64 total = sh.total;
  __syncthreads();
  // drawn: the first token at which the running sum exceeds u * total
  const double u01 = (double)a.uniform[r], x = u01 > 0.0 ? u01 * (double)total : 0.0;
  const u64 goal = x >= (double)total ? total - 1 : min((u64)x, total - 1);
  if (tid < ctas * kWarps && tid / kWarps == rank && goal < upto && goal >= upto - mine) {
    sh.found = tid % kWarps;               // the stretch that has it
    sh.found_before = upto - mine;
    sh.total = take;                       // how many of the stretch's equals are kept
  }
  cl.sync();                               // no CTA leaves while another reads it
  if (warp != sh.found) return;
  u64 left = goal - sh.found_before;
  int spare = (int)sh.total;
  for (int j0 = v0; j0 < v1; j0 += 32) {
    const int j = j0 + lane;
    uint4 u = make_uint4(0, 0, 0, 0);
    u64 s = 0;
    int n = 0;
    if (j < v1) {
      u = vector(j);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float l = Vec<T>::at(u, i);
        if (l > K) s += weigh.of<kExact>(l);
        n += l == K;
      }
    }
    int n_upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, n_upto, o);
      if (lane >= o) n_upto += y;
    }
    const int first = spare - (n_upto - n);               // equals that this lane may still keep
    s += (u64)max(0, min(n, first)) * wK;
    u64 s_upto = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, s_upto, o);
      if (lane >= o) s_upto += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, left < s_upto);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        u64 run = s_upto - s;
        int may = first;
        for (int i = 0; i < N; ++i) {
          const float l = Vec<T>::at(u, i);
          u64 w = 0;
          if (l > K) w = weigh.of<kExact>(l);
          else if (l == K && may-- > 0) w = wK;
          run += w;
          if (left < run) {
            a.token[r] = j * N - row.lead + i;
            if (a.prob) {
              u64 whole;
              int shift;
              weigh.parts<kExact>(l, whole, shift);
              a.prob[r] = (float)((double)whole * __longlong_as_double((long long)(1023 - shift) << 52) / (double)total);
            }
            break;
          }
        }
      }
      return;
    }
    left -= __shfl_sync(0xffffffffu, s_upto, 31);
    spare -= __shfl_sync(0xffffffffu, n_upto, 31);
  }
}

template <typename T>
cudaError_t run(const SampleArgs& a, cudaStream_t st) {
  // 16-byte vectors of a row, wherever it starts
  const long long vectors = ((long long)a.vocab * sizeof(T) + 15) / 16 + 1;
  int ctas = 1;
  while (ctas < kMaxCtas && vectors > 1024ll * ctas) ctas *= 2;
  const size_t bytes = (size_t)((vectors + ctas - 1) / ctas) * 16;
  const bool staged = bytes <= 200 * 1024;
  auto kernel = staged ? sample_kernel<T, true> : sample_kernel<T, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.rows * ctas));
  cfg.blockDim = dim3(kNT);
  cfg.dynamicSmemBytes = staged ? bytes : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_sample(int dtype, const SampleArgs& a, cudaStream_t st) { return dtype ? run<bf16>(a, st) : run<float>(a, st); }

}  // namespace dfl
