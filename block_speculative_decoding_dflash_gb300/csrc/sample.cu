// One token of each row of logits: temperature, top-k, top-p, min-p and a draw by a
// given uniform number.
//
// With M the row's largest logit a token's weight is w = 2^-((M - l) log2(e) / T).
// What the filters keep is a prefix of the tokens in descending order (ties: the
// lowest index first), so all of them together come down to one logit K and a
// number t: tokens above K are kept, of those equal to K the first t. The row is not
// sorted. There are three ways to K:
// * top_k of up to 256: a histogram of the threads' largest logits gives a distance
//   that holds top_k of them; the few tokens within it go to a list in the
//   cluster's first CTA, which sorts it, filters and draws (1 row of 202048: 10 us,
//   by histograms 32 us).
// * bf16 under top_p or a large top_k: a count of each bf16 number that is near enough to
//   M to weigh anything. A few thousand weights, times their counts, are the row's, a
//   running sum over them has K, and the CTA that has the draw is known from the counts
//   as well (16 rows of 202048 and top_p: 25 us, by histograms 47 us).
// * otherwise a histogram over M - l finds the bin in which the count (top_k) or the
//   weight (top_p) is reached, a list or histograms over the order of floats within
//   that bin find K (48 fp32 rows of 65537 and top_p: 33 us).
//
// Sums of weights decide which token is drawn, so they are exact: a weight is an
// integer, in units of 2^-44 of (nearly) the largest, a function of l, M and T alone;
// 64-bit sums of them are the same in any order and in every pass. A weight is right
// to about 2^-35: a prefix sum over a vocabulary then is off by some 2^-40 of the
// total, and a row's token is another than exact arithmetic's with a probability of
// 2^-22 or so even where all of 2^18 tokens weigh the same.
//
// A cluster of CTAs has a row, each warp an unbroken stretch of the vocabulary. They
// hold it in their shared memory where it fits; long rows of large batches do not, and
// are read again, from L2, in each pass. The CTAs exchange maxima, histograms and
// sums; each works out the outcome for itself, and the one that has the token writes it.
//
// 256 rows of 202048 in bf16 with mixed filters (four CTAs to a row, which hold none of
// it): 131 us, 0.8 TB/s, issue 42%. Without filters a weight's 35 instructions bound it;
// elsewhere a chain of short steps does, for which the instructions themselves often come
// too late, and every meeting of a cluster takes 0.9 us. Two CTAs of 64 registers and half of the SM's shared memory each work in the
// other's waits (one CTA of 1024 threads: 16 rows wait for a second round; three, with
// spills: 10 to 17% slower). More CTAs to a row do not find room at once (16 rows by 16:
// 41 us, by 8: 26 us).
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include <utility>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace dfl {

namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kNT = 512, kWarps = kNT / 32;
constexpr int kBins = 512;
constexpr int kMaxCtas = 8;
constexpr int kSteps = 1024;               // of the exponential's table to a factor of 2
constexpr int kUnit = 44;                  // weights are integers of 2^-44
constexpr int kBinShift = 7;               // bins of a factor of 2^(1/8): 353 of them

// 2^(-(i + 1) / 1024) as its first 24 bits and the rest, both times 2^42. (A value of
// 1 would need a bit more; a factor common to all weights makes no difference.)
constexpr double kScale = 4398046511104.0;
struct PowTable {
  float2 v[kSteps];
  constexpr PowTable() : v() {
    for (int i = 0; i < kSteps; ++i) {
      // Taylor's series at -(i + 1) / 1024 ln 2, in (-0.7, 0): below 2^-53 after 20 terms
      const double x = -(i + 1) / 1024.0 * 0.69314718055994530942;
      double sum = 1.0, term = 1.0;
      for (int k = 1; k <= 22; ++k) {
        term *= x / k;
        sum += term;
      }
      if (i == kSteps - 1) sum = 0.5;        // (its 24 bits start at one half)
      const double whole = (double)(long long)(sum * 16777216.0) / 16777216.0;
      v[i].x = (float)(whole * kScale);
      v[i].y = (float)((sum - whole) * kScale);
    }
  }
};
__device__ constexpr PowTable kPow{};

// The weight of a logit at distance M - l, for rows of one temperature. Written for the
// pipes: a sum or a product takes half as long as an operation on bits or a comparison.
// Every rounding is written out: a product that the compiler joins to a sum in one place
// and not in another would give a token two bins, or two weights.
struct Weigh {
  const float2* table;
  float top, chi, clo, least;              // log2(e) / T in two parts; the smallest logit whose weight is not zero
  __device__ __forceinline__ bool counts(float l) const { return l >= least; }
  // The distance in steps of 2^-10 to a factor of 2, rounded, of a logit that counts.
  __device__ __forceinline__ float distance(float d) const { return __fmul_rn(d, chi); }
  __device__ __forceinline__ float steps(float p) const { return __fadd_rn(p, 12288.f); }   // 1.5 * 2^13: sums are multiples of 2^-10
  static __device__ __forceinline__ int whole_steps(float t) { return __float_as_int(t) & 0x3fffff; }
  __device__ __forceinline__ int bin(float l) const { return whole_steps(steps(distance(top - l))) >> kBinShift; }
  // The weight of a token that counts as whole * 2^-(steps / 2^10) units, before the
  // shift drops bits; of others anything. No branches: a thread has several tokens' weights under way at once.
  __device__ __forceinline__ void parts(float l, u64& whole, int& i) const {
    const float d = top - l, p = distance(d);
    const float b = d - top;               // what d's rounding left: (M - (d - b)) + (-l - b)
    const float e = fmaf((top - (d - b)) + (-l - b), chi, fmaf(d, clo, fmaf(d, chi, -p)));
    const float t = steps(p);
    i = whole_steps(t);
    const float r = (p - (t - 12288.f)) + e;              // p = i / 1024 + r, |r| <= 2^-11
    const float g = __fmul_rn(r, fmaf(r, fmaf(r, -0.0555041087f, 0.240226507f), -0.693147181f));   // 2^-r - 1
    const float2 w = table[i & (kSteps - 1)];
    const int c = __float2int_rn(fmaf(w.x, g, w.y));                                     // the rest, in 2^-42
    // the first 24 bits are w.x's: its exponent is the same throughout
    constexpr u64 kBias = ((u64)(127 + 41) << 23) - (1u << 23);
    asm("{\n .reg .b64 t;\n mad.wide.u32 t, %1, %2, %3;\n mad.wide.s32 %0, %4, %5, t;\n}\n"
        : "=l"(whole) : "r"(__float_as_int(w.x)), "r"(1 << (kUnit - 24)), "l"((u64)0 - (kBias << (kUnit - 24))), "r"(c), "r"(1 << (kUnit - 42)));
  }
  // (what the shift drops is made up for by a set last bit, on average)
  __device__ __forceinline__ u64 of_counting(float l, int& i) const {
    u64 whole;
    parts(l, whole, i);
    return (whole >> (i >> 10)) | 1ull;
  }
  __device__ __forceinline__ u64 of(float l) const {
    int i;
    const u64 w = of_counting(l, i);
    return counts(l) ? w : 0ull;
  }
};

// floor(f * x), or the next whole number up, of an fp32 number f in (0, 1): all bits of
// the product, in integers. (Arithmetic in 64-bit floats has a few lanes to an SM.)
__device__ __forceinline__ u64 share(float f, u64 x, bool up) {
  const unsigned b = __float_as_uint(f), m = b >> 23 ? (b & 0x7fffffu) | 0x800000u : b;
  const int s = 150 - max(1, (int)(b >> 23));             // f = m 2^-s, 24 <= s <= 149
  const u64 lo = x * m, hi = __umul64hi(x, m);            // hi < 2^24
  const u64 whole = s < 64 ? (hi << (64 - s)) | (lo >> s) : s < 128 ? hi >> (s - 64) : 0ull;
  const bool rest = s < 64 ? (lo << (64 - s)) != 0 : (lo | (s < 128 ? hi & ((1ull << (s - 64)) - 1) : hi)) != 0;
  return whole + (up && rest ? 1ull : 0ull);
}
// The place of a uniform number in a sum.
__device__ __forceinline__ u64 drawn(float u, u64 total) { return u >= 1.f ? total - 1 : u > 0.f ? share(u, total, false) : 0ull; }

// The next smaller number.
__device__ __forceinline__ float least_below(float x) {
  const int u = __float_as_int(x);
  return x == 0.f ? __int_as_float((int)0x80000001u) : __int_as_float(u + (u < 0 ? 1 : -1));
}

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

// bf16 logits by a bin for each number: the order of the numbers 2^-9 and more from
// zero, zero, and the rest of either sign, which shares a bin (some ten thousand
// numbers that hardly a logit is). A place counts from zero up and down.
constexpr int kKeys = 4096;
constexpr int kNear = 0x3b00;              // 2^-9
__device__ __forceinline__ int place_of(int bits) {       // of the 16 bits, with their sign
  const int mag = bits & 0x7fff, z = max(mag - kNear + 2, min(mag, 1));
  return bits < 0 ? -z : z;
}
__device__ __forceinline__ int place_of(float l) { return place_of((int)__float_as_uint(l) >> 16); }
__device__ __forceinline__ bool shared_place(int place) { return place == 1 || place == -1; }
__device__ __forceinline__ float of_place(int place) {    // (0 for a shared one)
  const int z = place < 0 ? -place : place;
  return z < 2 ? 0.f : __int_as_float(((z - 2 + kNear) << 16) | (place < 0 ? (int)0x80000000u : 0));
}

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  // NaN counts as -inf, +inf as the type's largest number.
  static __device__ __forceinline__ bool odd(const uint4& u) {   // holds one of them, or -inf
    if constexpr (sizeof(T) == 2) {
      const unsigned any = ((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
                           ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u);
      return any & 0x80008000u;
    }
    return (((u.x & 0x7f800000u) + 0x00800000u) | ((u.y & 0x7f800000u) + 0x00800000u) |
            ((u.z & 0x7f800000u) + 0x00800000u) | ((u.w & 0x7f800000u) + 0x00800000u)) >> 31;
  }
  static __device__ __forceinline__ uint4 clean(uint4 u) {
    unsigned* w = reinterpret_cast<unsigned*>(&u);
    if constexpr (sizeof(T) == 2) {
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
  static __device__ __forceinline__ float largest(const uint4& u) {
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162 m[4];
      memcpy(m, &u, 16);
      const __nv_bfloat162 x = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
      return fmaxf(__low2float(x), __high2float(x));
    }
    return fmaxf(fmaxf(at(u, 0), at(u, 1)), fmaxf(at(u, 2), at(u, 3)));
  }
  static __device__ __forceinline__ float at(const uint4& u, int i) {
    const unsigned* w = reinterpret_cast<const unsigned*>(&u);
    if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    return __uint_as_float(w[i]);
  }
  // The same of an i that is not known when this is compiled.
  static __device__ __forceinline__ float some(const uint4& u, int i) {
    const int k = sizeof(T) == 2 ? i >> 1 : i;
    const unsigned w = k & 2 ? (k & 1 ? u.w : u.z) : (k & 1 ? u.y : u.x);
    return __uint_as_float(sizeof(T) == 4 ? w : i & 1 ? w & 0xffff0000u : w << 16);
  }
};

// A row as vectors of 16 bytes: vector j holds the elements j * N - lead + 0 .. N - 1,
// -inf where the row has none.
template <typename T>
struct Row {
  const T* base;
  int lead, vocab;
  __device__ __forceinline__ bool whole(int j) const {
    const int v = j * Vec<T>::N - lead;
    return v >= 0 && v + Vec<T>::N <= vocab;
  }
  __device__ __forceinline__ const uint4* at(int j) const { return reinterpret_cast<const uint4*>(base + (j * Vec<T>::N - lead)); }
  __device__ __forceinline__ uint4 raw(int j) const { return *at(j); }
  __device__ __noinline__ uint4 ragged(int j) const {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
    for (int i = 0; i < Vec<T>::N; ++i) {
      const int v = j * Vec<T>::N - lead + i;
      e[i] = v >= 0 && v < vocab ? base[v] : from_f<T>(-INFINITY);
    }
    return u;
  }
  __device__ __forceinline__ uint4 load(int j) const {
    const uint4 u = whole(j) ? raw(j) : ragged(j);
    return Vec<T>::odd(u) ? Vec<T>::clean(u) : u;
  }
};

// 16 bytes on their way to shared memory; all of a thread's are there.
__device__ __forceinline__ void copy_async(uint4* to, const uint4* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A list of tokens: one of a bin, or all that can still be drawn.
constexpr int kEach = 4, kList = kEach * kNT;
constexpr int kFew = kNT / 2, kNears = 1024;
struct Shared {
  unsigned lo[2][kBins], hi[2][kBins];     // histograms, which take turns
  union {
    u64 list[kList];                       // tokens as a number that sorts them (see entry)
    unsigned keys[kKeys + 32];             // bf16: how many of the CTA's logits each bin has, from the largest down, and a
                                           // place for each lane's others
  };
  unsigned near_lo[2], near_hi[2];         // the weight in the shared bins above and below zero
  // What every CTA says to every other, in the order of the CTAs:
  float tops[kMaxCtas];                    // the largest logit,
  int firsts[kMaxCtas];                    // and the first token that has it (of rows that take it)
  u64 slices[kMaxCtas];                    // its share of the bins: their weight
  unsigned slice_counts[kMaxCtas];
  u64 part_sums[kMaxCtas];                 // its part of the row: the weight above K,
  int part_equals[kMaxCtas];               // and how many are K
  u64 sums[kMaxCtas * kWarps];             // the same of each warp's stretch
  int equals[kMaxCtas * kWarps];
  int pick[2];                             // and the one that has it: the bin of the cut by top_k and by top_p (-1: none said
  u64 pick_t[2], above[2];                 // so), what of it stays, and the weight above it
  union {
    struct { u64 all[kNT], few[kFew]; } sort;
    float queue[kWarps][64];               // a warp's tokens above K on their way to a weight
    float nears[kNears];                   // logits of the shared bins on theirs
  };
  float chi, clo, far;                     // see Weigh; the distance beyond which a weight is zero
  double cut;                              // how far from the largest logit min_p reaches
  int near_listed;                         // may be more than kNears
  int listed;                              // may be more than kList: the list is cut
  unsigned kmin, kmax;
  u64 scan[kWarps];
  unsigned scan_n[kWarps];
  u64 found_before, total;
  int found;
};

// of a row, beside these and the table, by one CTA on an SM and by each of two
constexpr size_t kStaged = 180 * 1024, kStagedTwo = 70 * 1024;

// Inclusive sums over the CTA's threads.
__device__ __forceinline__ u64 scan_warp(u64 x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ u64 scan_block(u64 x, u64* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = scan_warp(x);
  __syncthreads();
  if (lane == 31) s[warp] = x;
  __syncthreads();
  u64 before = (lane & (kWarps - 1)) < warp ? s[lane & (kWarps - 1)] : 0ull;
#pragma unroll
  for (int o = kWarps / 2; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  return x + before;
}
// The same of a sum and a count.
__device__ __forceinline__ void scan_block(u64& x, unsigned& n, u64* s, unsigned* sn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    const unsigned m = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) { x += y; n += m; }
  }
  __syncthreads();
  if (lane == 31) { s[warp] = x; sn[warp] = n; }
  __syncthreads();
  u64 before = (lane & (kWarps - 1)) < warp ? s[lane & (kWarps - 1)] : 0ull;
  unsigned m = lane < warp ? sn[lane] : 0u;
#pragma unroll
  for (int o = kWarps / 2; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  x += before;
  n += __reduce_add_sync(0xffffffffu, m);
}
// Sorts one number of each of the first n threads, all different, ascending; the other threads' are ~0.
__device__ __forceinline__ u64 sort_block(u64 x, int n, u64* s, u64* few) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (n <= kFew) {                         // counts those before each, by several threads to one
    const int lg = n <= kFew / 4 ? 3 : n <= kFew / 2 ? 2 : 1, e = tid >> lg, step = 1 << lg;
    if (tid < n) s[tid] = x;
    __syncthreads();
    x = e < n ? s[e] : 0ull;
    int at = 0;
#pragma unroll 4
    for (int i = tid & (step - 1); i < n; i += step) at += s[i] < x;
    for (int o = 1; o < step; o <<= 1) at += __shfl_xor_sync(0xffffffffu, at, o);
    if (e < n && (tid & (step - 1)) == 0) few[at] = x;
    __syncthreads();
    return tid < n ? few[tid] : ~0ull;
  }
  int all = 2 * kFew;
  while (all < n) all <<= 1;
  for (int size = 2; size <= all; size <<= 1)
    for (int o = size >> 1; o; o >>= 1) {
      u64 y;
      if (o >= 32) {
        __syncthreads();
        s[tid] = x;
        __syncthreads();
        y = s[tid ^ o];
      } else {
        y = __shfl_xor_sync(0xffffffffu, x, o);
      }
      const bool up = (tid & size) == 0, first = (tid & o) == 0;
      if ((y < x) == (up == first)) x = y;
    }
  return x;
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kNT, 2) sample_kernel(const SampleArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr bool kBins16 = sizeof(T) == 2; // logits of 16 bits may have a bin for each number
  extern __shared__ __align__(16) uint4 held[];
  __shared__ Shared sh;
  __shared__ float2 table[kSteps];
  cg::cluster_group cl = cg::this_cluster();
  const int ctas = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r = blockIdx.x / ctas;
  // (as whole warps: one that has come apart stays so behind a barrier of threads, and takes twice as long)
  auto meet = [&]() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
  };
  for (int i = tid; i < kSteps; i += kNT) table[i] = kPow.v[i];
  sh.lo[0][tid] = sh.hi[0][tid] = sh.lo[1][tid] = sh.hi[1][tid] = 0u;
  if (tid == 0) {
    sh.listed = 0;
    sh.pick[0] = sh.pick[1] = -1;
  }
  auto clear_keys = [&]() {
    for (int i = tid; i < kKeys / 4; i += kNT) reinterpret_cast<uint4*>(sh.keys)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 2) sh.near_lo[tid] = sh.near_hi[tid] = 0u;
    if (tid == 0) sh.near_listed = 0;
  };
  if (kBins16) clear_keys();
  auto started = cl.barrier_arrive();      // (no CTA writes into another before that has done this)
  pdl_enter();

  // ---- the row's stretch of this warp, and the largest logit of the row and of each thread
  Row<T> row;
  row.base = static_cast<const T*>(a.logits) + r * a.stride;
  row.lead = (int)((reinterpret_cast<uintptr_t>(row.base) & 15u) / sizeof(T));
  row.vocab = a.vocab;
  // A lane loads and looks through every 32nd vector of its warp's stretch.
  const int vectors = (row.lead + a.vocab + N - 1) / N, per = (vectors + ctas - 1) / ctas, each = (per + kWarps - 1) / kWarps;
  const int c0 = min(vectors, rank * per), c1 = min(vectors, c0 + per);
  const int v0 = min(c1, c0 + warp * each), v1 = min(c1, v0 + each);
  auto vector = [&](int j) { return STAGED ? held[j - c0] : row.load(j); };
  const float temp = a.temperature ? a.temperature[r] : 1.f;
  const int top_k = a.top_k ? a.top_k[r] : 0;
  const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f, u01 = a.uniform[r];
  const bool greedy = !(temp >= 5.4210109e-20f);          // 2^-64
  float hi = -INFINITY;
  // (A loop over what is there already, as short as can be: unrolled with the loads in
  // registers the code comes in more slowly than the row.)
  if (STAGED) {
    for (int j = v0 + lane; j < v1; j += 32) {
      if (row.whole(j)) copy_async(&held[j - c0], row.at(j));
      else held[j - c0] = row.ragged(j);
    }
  }
  // (64-bit floats, while the row is on its way)
  if (tid == kNT - 1) {
    const double c = greedy ? 1.0 : 1.44269504088896340736 / (double)temp;
    sh.chi = (float)c;
    sh.clo = (float)(c - (double)sh.chi);
    sh.far = fminf((float)(kUnit / c), FLT_MAX);
    sh.cut = min_p > 0.f ? (double)temp * log((double)fminf(min_p, 1.f)) : 0.0;
  }
  if (STAGED) copies_done();
#pragma unroll 1
  for (int j = v0 + lane; j < v1; j += 32) {
    uint4 u = STAGED ? held[j - c0] : row.whole(j) ? row.raw(j) : row.ragged(j);
    if (Vec<T>::odd(u)) {
      u = Vec<T>::clean(u);
      if (STAGED) held[j - c0] = u;
    }
    hi = fmaxf(hi, Vec<T>::largest(u));
  }
  const float own = hi;                    // of the vectors that this thread looks through
  hi = warp_max(hi);
  if (lane == 0) sh.scan[warp] = __float_as_uint(hi);
  __syncthreads();
  hi = warp_max(lane < kWarps ? __uint_as_float((unsigned)sh.scan[lane]) : -INFINITY);   // the CTA's
  cl.barrier_wait(std::move(started));

  if (greedy) {                            // the first of the largest: the first CTA hears of all, which need not wait
    int first = INT32_MAX;
    if (own == hi && hi > -INFINITY)
      for (int j = v0 + lane; j < v1 && first == INT32_MAX; j += 32) {
        const uint4 u = vector(j);
        for (int i = N - 1; i >= 0; --i)
          if (Vec<T>::at(u, i) == hi) first = j * N - row.lead + i;
      }
    first = __reduce_min_sync(0xffffffffu, first);
    __syncthreads();
    if (lane == 0) sh.scan[warp] = (u64)first;
    __syncthreads();
    if (warp == 0) {
      first = __reduce_min_sync(0xffffffffu, lane < kWarps ? (int)sh.scan[lane] : INT32_MAX);
      if (lane == 0) {
        *cl.map_shared_rank(&sh.tops[rank], 0) = hi;
        *cl.map_shared_rank(&sh.firsts[rank], 0) = first;
      }
    }
    auto told = cl.barrier_arrive();
    if (rank) return;
    cl.barrier_wait(std::move(told));
    if (warp == 0) {
      const float top = lane < ctas ? sh.tops[lane] : -INFINITY, most = warp_max(top);
      first = __reduce_min_sync(0xffffffffu, lane < ctas && top == most ? sh.firsts[lane] : INT32_MAX);
      if (lane == 0) {
        a.token[r] = most > -INFINITY ? first : -1;
        if (a.prob) a.prob[r] = most > -INFINITY ? 1.f : 0.f;
      }
    }
    return;
  }

  if (warp == 0 && lane < ctas) *cl.map_shared_rank(&sh.tops[rank], lane) = hi;
  meet();
  hi = warp_max(lane < ctas ? sh.tops[lane] : -INFINITY);
  if (hi == -INFINITY) {                   // nothing to choose from
    if (rank == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.prob) a.prob[r] = 0.f;
    }
    return;
  }
  Weigh weigh;
  weigh.table = table;
  weigh.top = hi;
  weigh.chi = sh.chi;
  weigh.clo = sh.clo;
  // (of a vast temperature every logit whose distance is an fp32 number: FLT_MAX and half a step more)
  weigh.least = fmaxf(hi - sh.far - (sh.far == FLT_MAX ? 0x1p102f : 0.f), -FLT_MAX);
  auto put = [&](int token, float l, u64 total) {
    a.token[r] = token;
    if (!a.prob) return;
    u64 whole;
    int i;
    weigh.parts(l, whole, i);
    a.prob[r] = (float)((double)whole * __longlong_as_double((long long)(1023 - (i >> 10)) << 52) / (double)total);
  };

  int parity = 0;                          // the histogram in use
  // kept: what is above K, and the first t of those equal to K; at first what counts
  float K = least_below(weigh.least);
  u64 t = 0;
  bool all = true;                         // no cut so far

  // The histogram of all CTAs: this thread's bin, and the sum up to and with it.
  auto merged = [&](bool weights, u64& bin, u64& upto) {
    meet();
    bin = 0;
    static_assert(kBins == kNT, "a thread to each bin");
    unsigned lo[kMaxCtas], hi[kMaxCtas] = {};               // (all of them requested together)
#pragma unroll
    for (int i = 0; i < kMaxCtas; ++i) {
      const int c = min(i, ctas - 1);
      lo[i] = *cl.map_shared_rank(&sh.lo[parity][tid], c);
      if (weights) hi[i] = *cl.map_shared_rank(&sh.hi[parity][tid], c);
    }
#pragma unroll
    for (int i = 0; i < kMaxCtas; ++i) bin += i < ctas ? (u64)hi[i] << 32 | lo[i] : 0ull;
    upto = scan_block(bin, sh.scan);
    if (tid == kNT - 1) sh.total = upto;
    parity ^= 1;
    sh.lo[parity][tid] = sh.hi[parity][tid] = 0u;   // everyone has read it: they came to the last meeting since
    __syncthreads();
  };
  auto add = [&](bool weights, int bin, u64 w) {
    const unsigned old = atomicAdd(&sh.lo[parity][bin], (unsigned)w);
    if (weights) atomicAdd(&sh.hi[parity][bin], (unsigned)(w >> 32) + (old + (unsigned)w < old ? 1u : 0u));
  };
  // A token as a number: larger logits first, then lower ids.
  auto entry = [&](float l, int token) { return (u64)~key_of<T>(l) << 32 | (unsigned)token; };
  auto entry_logit = [&](u64 x) { return of_key<T>(sizeof(T) == 2 ? (unsigned)(~x >> 32) & 0xffffu : (unsigned)(~x >> 32)); };
  auto list = [&](float l, int token) {
    const int at = atomicAdd(&sh.listed, 1);
    if (at < kList) sh.list[at] = entry(l, token);
  };
  // The lists of all CTAs, kEach entries to a thread (~0: none): their number, or -1 where some do not fit.
  auto gathered = [&](u64 (&mine)[kEach]) {
    meet();
    const int some = lane < ctas ? *cl.map_shared_rank(&sh.listed, lane) : 0;
    int upto = some;
#pragma unroll
    for (int o = 1; o < kMaxCtas; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int n = __shfl_sync(0xffffffffu, upto, kMaxCtas - 1);
    const bool fit = __all_sync(0xffffffffu, some <= kList) && n <= kList;
    int from[kEach] = {}, before[kEach] = {};
#pragma unroll
    for (int i = 0; i < kMaxCtas - 1; ++i) {
      const int y = __shfl_sync(0xffffffffu, upto, i);
#pragma unroll
      for (int x = 0; x < kEach; ++x)
        if (tid + x * kNT >= y) { from[x] = i + 1; before[x] = y; }
    }
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      mine[x] = ~0ull;
      if (fit && tid + x * kNT < n) mine[x] = *cl.map_shared_rank(&sh.list[tid + x * kNT - before[x]], from[x]);
    }
    __syncthreads();                       // (what follows runs as whole warps)
    return fit ? n : -1;
  };

  // How many tokens of weight `one` reach a sum.
  auto reached = [](u64 sum, u64 one) { return (sum + one - 1) / one; };

  // ---- few tokens to choose from: top_k of them, by a list
  if (top_k > 0 && top_k <= kNT / 2) {
    // At least top_k threads have a token in the first bins that hold top_k of the
    // threads' largest: whatever is further away is not among the first top_k.
    if (weigh.counts(own)) atomicAdd(&sh.lo[parity][weigh.bin(own)], 1u);
    u64 bin, upto;
    merged(false, bin, upto);
    const u64 want = (u64)top_k;
    if (tid == kNT - 1 || upto >= want)
      if (upto - bin < want) sh.found = tid;
    __syncthreads();
    const int far = sh.found;              // (of all bins, where fewer threads have a token)
    bool room = true;
    if (weigh.counts(own) && weigh.bin(own) <= far)
      for (int j = v0 + lane; j < v1 && room; j += 32) {
        const uint4 u = vector(j);
        const float most = Vec<T>::largest(u);
        if (!weigh.counts(most) || weigh.bin(most) > far) continue;
        unsigned near = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float l = Vec<T>::at(u, i);
          near |= (unsigned)(weigh.counts(l) && weigh.bin(l) <= far) << i;
        }
        for (; near && room; near &= near - 1) {
          // into the first CTA's list
          const int i = __ffs(near) - 1, at = atomicAdd(cl.map_shared_rank(&sh.listed, 0), 1);
          room = at < kNT;                 // (else that list is of no use)
          if (room) *cl.map_shared_rank(&sh.list[at], 0) = entry(Vec<T>::some(u, i), j * N - row.lead + i);
        }
      }
    meet();
    const int n = __shfl_sync(0xffffffffu, lane == 0 ? *cl.map_shared_rank(&sh.listed, 0) : 0, 0);
    if (n <= kNT) {
      // the first CTA does the rest; the others are done once they have heard that it can
      auto heard = cl.barrier_arrive();
      if (rank) return;
      {
        u64 x = sort_block(tid < n ? sh.list[tid] : ~0ull, n, sh.sort.all, sh.sort.few);
        // in descending order of logits: top_k, top_p, min_p
        const float l = x == ~0ull ? -INFINITY : entry_logit(x);
        u64 w = tid < n && tid < top_k ? weigh.of(l) : 0ull;
        const u64 before = scan_block(w, sh.scan) - w;
        if (tid == kNT - 1) sh.total = before + w;
        __syncthreads();
        if (top_p < 1.f) {
          if (before > 0 && (!(top_p > 0.f) || before >= share(top_p, sh.total, true))) w = 0;
        }
        if (min_p > 0.f && l < __double2float_ru((double)hi + sh.cut)) w = 0;
        // the draw, in ascending order of ids
        x = w ? x << 32 | x >> 32 : ~0ull;
        const int kept = __syncthreads_count(w != 0);      // (the first ones)
        x = sort_block(x, kept, sh.sort.all, sh.sort.few);
        const float lt = entry_logit(x << 32 | x >> 32);
        w = x == ~0ull ? 0ull : weigh.of(lt);
        const u64 upto_t = scan_block(w, sh.scan);
        if (tid == kNT - 1) sh.total = upto_t;
        __syncthreads();
        const u64 total = sh.total, goal = drawn(u01, total);
        if (w && goal < upto_t && goal >= upto_t - w) put((int)(x >> 32), lt, total);
      }
      cl.barrier_wait(std::move(heard));
      return;
    }
    meet();                             // the lists are free again
    if (tid == 0) sh.listed = 0;
    if (kBins16) {
      clear_keys();
      __syncthreads();
    }
  }

  // Where the token is looked for at the end: the warps' stretches of the row, or of one CTA's part of it.
  const uint4* source = held;
  int first = v0, last = v1, origin = c0;
  u64 total = 0, goal = 0;
  bool placed = false;                     // total and goal are known

  // ---- bf16: a bin for each number. The row's weights are those of some thousand
  // numbers times their counts, a cut is found in one step, and what each CTA keeps
  // follows from its own counts: weights of single tokens are taken of one CTA's
  // part only, by all of them. Not without top_k and top_p, where nothing is looked for
  // but the draw, which costs one weight a token at most (256 rows of 202048 without filters
  // 155 us, by counting 162, under min_p 95 and 161; 16 rows 22 and 26, 14 and 26).
  if constexpr (kBins16) if (top_k > 0 || top_p < 1.f) {
    // (down to the smallest bf16 number that counts)
    const int low = __float_as_int(weigh.least), top = place_of(hi), bins = top - place_of((low + (low < 0 ? 0 : 0xffff)) >> 16) + 1;
    if (bins <= kKeys) {
      auto add_near = [&](float l) {
        const u64 w = weigh.of(l);
        const int side = l < 0.f;
        const unsigned old = atomicAdd(&sh.near_lo[side], (unsigned)w);
        atomicAdd(&sh.near_hi[side], (unsigned)(w >> 32) + (old + (unsigned)w < old ? 1u : 0u));
      };
      for (int j = v0 + lane; j < v1; j += 32) {
        const uint4 u = vector(j);
        const unsigned* words = reinterpret_cast<const unsigned*>(&u);
        unsigned near = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int bits = (int)(i & 1 ? words[i >> 1] : words[i >> 1] << 16) >> 16, place = place_of(bits);
          const int b = top - place;
          atomicAdd(&sh.keys[b < bins ? b : kKeys + lane], 1u);   // (with a branch to each logit a third slower)
          near |= (unsigned)shared_place(place) << i;
        }
        // Few are in a shared bin. Their weights wait until the end, where all warps take them together
        // (at once each would hold its warp up, and all others with it: 256 rows 130 us, so 127 us).
        for (; near; near &= near - 1) {
          const float l = Vec<T>::some(u, __ffs(near) - 1);
          if (top - place_of(l) >= bins) continue;
          const int at = atomicAdd(&sh.near_listed, 1);
          if (at < kNears) sh.nears[at] = l;
          else add_near(l);
        }
      }
      __syncthreads();
      for (int i = tid; i < min(sh.near_listed, kNears); i += kNT) add_near(sh.nears[i]);
      bool shared_cut = false;             // within a shared bin: not from counts
      {
        // this thread's bins
        const int some = (kKeys + ctas - 1) / ctas, share_of = (some + kNT - 1) / kNT, mine = rank * some + tid * share_of;
        const int n_mine = max(0, min(min(share_of, some - tid * share_of), kKeys - mine));
        meet();
        // a bin of all CTAs
        auto count_of = [&](int b) {
          unsigned n = 0, of[kMaxCtas];
#pragma unroll
          for (int i = 0; i < kMaxCtas; ++i) of[i] = *cl.map_shared_rank(&sh.keys[b], min(i, ctas - 1));
#pragma unroll
          for (int i = 0; i < kMaxCtas; ++i) n += i < ctas ? of[i] : 0u;
          return n;
        };
        // the shared bins' weights: of one CTA by each lane, all of a side by every lane of it
        u64 near = 0;
        if ((lane >> 1) < ctas)
          near = *cl.map_shared_rank(&sh.near_lo[lane & 1], lane >> 1) | (u64)*cl.map_shared_rank(&sh.near_hi[lane & 1], lane >> 1) << 32;
        __syncwarp();
#pragma unroll
        for (int o = 2; o < 2 * kMaxCtas; o <<= 1) near += __shfl_xor_sync(0xffffffffu, near, o);
        const u64 above_zero = __shfl_sync(0xffffffffu, near, 0), below_zero = __shfl_sync(0xffffffffu, near, 1);
        auto weight_of = [&](int b, unsigned n) {
          const int place = top - b;
          return shared_place(place) ? place > 0 ? above_zero : below_zero : n ? n * weigh.of(of_place(place)) : 0ull;
        };
        unsigned n = 0;
        u64 w = 0;
        for (int i = 0; i < n_mine; ++i) {
          const unsigned x = count_of(mine + i);
          n += x;
          w += weight_of(mine + i, x);
        }
        const u64 n_upto = top_k > 0 ? scan_block(n, sh.scan) : 0ull, w_upto = scan_block(w, sh.scan);
        if (tid == kNT - 1)
          for (int i = 0; i < ctas; ++i) {
            *cl.map_shared_rank(&sh.slices[rank], i) = w_upto;
            *cl.map_shared_rank(&sh.slice_counts[rank], i) = (unsigned)n_upto;
          }
        meet();
        // what the CTAs before this one have, and all of them
        u64 w_before = 0, w_all = 0;
        unsigned n_before = 0, n_all = 0;
        for (int i = 0; i < ctas; ++i) {
          const u64 x = sh.slices[i];
          const unsigned y = sh.slice_counts[i];
          if (i < rank) { w_before += x; n_before += y; }
          w_all += x;
          n_all += y;
        }
        // The bin where the running count (or weight) reaches `want`, found by the thread that has it.
        auto pick = [&](bool weights, u64 want) {
          const u64 upto = weights ? w_before + w_upto : n_before + n_upto, before = upto - (weights ? w : (u64)n);
          if (before < want && want <= upto) {
            u64 run = before, run_w = w_before + w_upto - w;
            for (int i = 0; i < n_mine; ++i) {
              const unsigned x = share_of > 1 ? count_of(mine + i) : n;
              const u64 wx = share_of > 1 ? weight_of(mine + i, x) : w, step = weights ? wx : (u64)x;
              if (run + step >= want) {
                const int place = top - (mine + i);
                const u64 stay = !weights ? want - run : shared_place(place) ? 0ull : reached(want - run, weigh.of(of_place(place)));
                for (int c = 0; c < ctas; ++c) {
                  *cl.map_shared_rank(&sh.pick[weights], c) = mine + i;
                  *cl.map_shared_rank(&sh.pick_t[weights], c) = stay;
                  *cl.map_shared_rank(&sh.above[weights], c) = run_w;
                }
                break;
              }
              run += step;
              run_w += wx;
            }
          }
          meet();
          const int b = sh.pick[weights], place = top - b;
          if (b < 0 || shared_place(place)) {
            shared_cut = true;
          } else {
            K = of_place(place);
            t = sh.pick_t[weights];
            w_all = sh.above[weights];              // above K
            all = false;
          }
        };
        if (top_k > 0 && (unsigned)top_k < n_all) pick(false, (u64)top_k);
        if (top_p < 1.f && !shared_cut) {
          const u64 one = all ? 0ull : weigh.of(K), want = top_p > 0.f ? max(share(top_p, w_all + t * one, true), 1ull) : 1ull;
          if (want > w_all && !all) {
            t = min(t, reached(want - w_all, one));         // among those equal to K
          } else if (want < w_all || !all) {
            pick(true, want);
          }
        }
      }
      if (min_p > 0.f && !shared_cut) {
        const float f = __double2float_ru((double)hi + sh.cut);
        if (f > K) {
          K = f;
          t = ~0ull;
          all = false;
        }
      }
      // (0 < |K| < 2^-9: a shared bin is kept in part)
      if (!shared_cut && (K == 0.f || fabsf(K) >= 0x1p-9f)) {
        // this CTA's weight above K, and how many are K
        __syncthreads();
        u64 sum = 0;
        const int upto_K = all ? bins : min(bins, top - place_of(K) + 1);
        for (int b = tid; b < upto_K; b += kNT) {
          const int place = top - b;
          const unsigned n = sh.keys[b];
          const float l = of_place(place);
          if (shared_place(place)) {
            if (place > 0 ? K <= 0.f : K < 0.f) sum += (u64)sh.near_lo[place < 0] | (u64)sh.near_hi[place < 0] << 32;
          } else if (n && l > K) {
            sum += n * weigh.of(l);
          }
        }
        const u64 upto = scan_block(sum, sh.scan);
        if (tid == kNT - 1) {
          const int b = top - place_of(K);
          const int eq = !all && b >= 0 && b < bins && of_place(top - b) == K ? (int)sh.keys[b] : 0;
          for (int i = 0; i < ctas; ++i) {
            *cl.map_shared_rank(&sh.part_sums[rank], i) = upto;
            *cl.map_shared_rank(&sh.part_equals[rank], i) = eq;
          }
        }
        meet();
        const u64 wK = all ? 0ull : weigh.of(K), part = lane < ctas ? sh.part_sums[lane] : 0ull,
                  eq = lane < ctas ? (u64)sh.part_equals[lane] : 0ull;
        const u64 eq_before = scan_warp(eq) - eq, take = eq_before >= t ? 0ull : min(eq, t - eq_before), w = part + take * wK, w_upto = scan_warp(w);
        total = __shfl_sync(0xffffffffu, w_upto, 31);
        goal = drawn(u01, total);
        const int who = __ffs(__ballot_sync(0xffffffffu, goal < w_upto)) - 1;
        goal -= __shfl_sync(0xffffffffu, w_upto - w, who);
        t = __shfl_sync(0xffffffffu, take, who);
        placed = true;
        // the CTA `who` has it: its part of the row, in stretches of all warps
        origin = min(vectors, who * per);
        const int end = min(vectors, origin + per), chunk = (per + ctas * kWarps - 1) / (ctas * kWarps);
        first = min(end, origin + (rank * kWarps + warp) * chunk);
        last = min(end, first + chunk);
        if (STAGED) source = cl.map_shared_rank(held, who);
      } else {
        K = least_below(weigh.least);
        t = 0;
        all = true;
        meet();
        if (tid == 0) sh.listed = 0;
        __syncthreads();
      }
    }
  }
  auto there = [&](int j) { return STAGED ? source[j - origin] : row.load(j); };

  // Cuts what is kept so far (above K, t of those equal to K) where the running
  // count (or weight) reaches `part` (a share of all of it, for weights).
  auto cut = [&](bool weights, float part) {
    const float K0 = K;
    const u64 t0 = t, wK = !all && weights ? weigh.of(K0) : 1ull;  // (a K that is a logit)
    const u64 tail = all ? 0ull : t0 * wK;                // what those equal to K count
    auto in = [&](float l) { return l > K0; };
    for (int j = v0 + lane; j < v1; j += 32) {
      const uint4 u = vector(j);
#pragma unroll 1
      for (int i0 = 0; i0 < N; i0 += 4) {
        const uint2 half = N == 8 && i0 ? make_uint2(u.z, u.w) : make_uint2(u.x, u.y);
        const uint4 four = N == 8 ? make_uint4(half.x, half.y, 0, 0) : u;
        u64 w[4];
        int at[4];
        unsigned old[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float l = Vec<T>::at(four, i);
          w[i] = 1;
          at[i] = 0;
          if (weights) {
            w[i] = weigh.of_counting(l, at[i]);
            at[i] >>= kBinShift;
          } else {
            at[i] = weigh.bin(l);
          }
          if (in(l)) old[i] = atomicAdd(&sh.lo[parity][at[i]], (unsigned)w[i]);
        }
        if (weights)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const unsigned up = (unsigned)(w[i] >> 32) + (old[i] + (unsigned)w[i] < old[i] ? 1u : 0u);
            if (in(Vec<T>::at(four, i)) && up) atomicAdd(&sh.hi[parity][at[i]], up);
          }
      }
    }
    u64 bin, upto;
    merged(weights, bin, upto);
    const u64 total = sh.total + tail;
    u64 goal;                              // a token stays if what comes before it is below this
    if (weights) {
      goal = part > 0.f ? max(share(part, total, true), 1ull) : 1ull;
    } else {
      goal = (u64)top_k;
    }
    if (goal >= total) return;             // all of it
    if (goal > sh.total) {                 // reached among those equal to K
      t = min(t0, reached(goal - sh.total, wK));
      return;
    }
    if (upto >= goal && upto - bin < goal) {
      sh.found = tid;
      sh.found_before = upto - bin;
    }
    if (tid == 0) {
      sh.kmin = 0xffffffffu;
      sh.kmax = 0u;
      sh.listed = 0;
    }
    __syncthreads();
    const int where = sh.found;
    u64 before = sh.found_before;
    // the bin's tokens, and their span in the order of floats
    unsigned kmin = 0xffffffffu, kmax = 0u;
    if (own > K0 && weigh.bin(own) <= where)
      for (int j = v0 + lane; j < v1; j += 32) {
        const uint4 u = vector(j);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float l = Vec<T>::at(u, i);
          if (in(l) && weigh.bin(l) == where) {
            const unsigned k = key_of<T>(l);
            kmin = min(kmin, k);
            kmax = max(kmax, k);
            list(l, 0);
          }
        }
      }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
      atomicMin(&sh.kmin, kmin);
      atomicMax(&sh.kmax, kmax);
    }
    u64 xs[kEach];
    const int n = gathered(xs);
    kmin = 0xffffffffu;
    kmax = 0u;
    if (lane < ctas) {
      kmin = *cl.map_shared_rank(&sh.kmin, lane);
      kmax = *cl.map_shared_rank(&sh.kmax, lane);
    }
    __syncwarp();
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    unsigned kx[kEach];
    u64 wx[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const float l = xs[i] == ~0ull ? -INFINITY : entry_logit(xs[i]);
      kx[i] = key_of<T>(l);
      wx[i] = weights ? weigh.of(l) : 1ull;
    }
    // (nine bits of a float at a time: four times end it, whatever the sums are)
    for (int pass = 0; pass < 4 && kmin != kmax; ++pass) {
      int shift = 0;
      while ((kmax - kmin) >> shift >= (unsigned)kBins) ++shift;
      if (n >= 0) {                        // every CTA has them all
#pragma unroll
        for (int i = 0; i < kEach; ++i)
          if (xs[i] != ~0ull && kx[i] >= kmin && kx[i] <= kmax) add(weights, (int)((kmax - kx[i]) >> shift), wx[i]);
        __syncthreads();
        bin = tid < kBins ? sh.lo[parity][tid] | (u64)sh.hi[parity][tid] << 32 : 0ull;
        upto = scan_block(bin, sh.scan);
        if (tid < kBins) sh.lo[parity][tid] = sh.hi[parity][tid] = 0u;
      } else {
        for (int j = v0 + lane; j < v1; j += 32) {
          const uint4 u = vector(j);
#pragma unroll 1
          for (int i = 0; i < N; ++i) {
            const float l = Vec<T>::at(u, i);
            const unsigned k = key_of<T>(l);
            if (k >= kmin && k <= kmax && in(l) && weigh.bin(l) == where) add(weights, (int)((kmax - k) >> shift), weights ? weigh.of(l) : 1ull);
          }
        }
        merged(weights, bin, upto);
      }
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
    const u64 w1 = weights ? weigh.of(K) : 1ull;
    t = reached(goal - before, w1);
    all = false;
    meet();                             // the lists and spans are free again
  };
  if (!placed && top_k > 0 && top_k < a.vocab) cut(false, 0.f);
  if (!placed && top_p < 1.f) cut(true, top_p);
  if (!placed && min_p > 0.f) {
    // l >= M + T ln(min_p): the smallest fp32 that is
    const float f = __double2float_ru((double)hi + sh.cut);
    if (f > K) {
      K = f;
      t = ~0ull;
      all = false;
    }
  }

  // ---- each warp's weight above K and number equal to K
  u64 sum = 0;
  int equal = 0;
  if (all || placed) {
    for (int j = first + lane; j < last; j += 32) {
      const uint4 u = there(j);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float l = Vec<T>::at(u, i);
        int steps;
        const u64 w = weigh.of_counting(l, steps);
        if (l > K) sum += w;
        if (!all) equal += l == K;
      }
    }
  } else {
    // few of them: those that are kept come together before they are weighed
    float* queue = sh.queue[warp];
    int queued = 0;
    auto weigh_queue = [&]() {
      __syncwarp();
      int steps;
      const u64 w = weigh.of_counting(queue[lane], steps);
      if (lane < queued) sum += w;
    };
    for (int j0 = first; j0 < last; j0 += 32) {
      const int j = j0 + lane;
      const uint4 u = j < last ? there(j) : make_uint4(0u, 0u, 0u, 0u);
      const float most = j < last ? Vec<T>::largest(u) : -INFINITY;
      if (!__any_sync(0xffffffffu, most >= K)) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float l = Vec<T>::at(u, i);
        const bool on = j < last && l > K;
        equal += j < last && l == K;
        const unsigned who = __ballot_sync(0xffffffffu, on);
        if (on) queue[queued + __popc(who & ((1u << lane) - 1u))] = l;
        queued += __popc(who);
        if (queued >= 32) {
          weigh_queue();
          queued -= 32;
          const float next = queue[32 + lane];
          __syncwarp();
          if (lane < queued) queue[lane] = next;
        }
      }
    }
    weigh_queue();
  }
  u64 all_sum = sum;
#pragma unroll
  for (int o = 16; o; o >>= 1) all_sum += __shfl_xor_sync(0xffffffffu, all_sum, o);
  const int all_equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane < ctas) {
    *cl.map_shared_rank(&sh.sums[rank * kWarps + warp], lane) = all_sum;
    *cl.map_shared_rank(&sh.equals[rank * kWarps + warp], lane) = all_equal;
  }
  meet();
  const u64 wK = all ? 0ull : weigh.of(K);
  u64 mine = 0;
  unsigned eq = 0;
  if (tid < ctas * kWarps) {
    mine = sh.sums[tid];
    eq = (unsigned)sh.equals[tid];
  }
  u64 upto = mine;
  unsigned eq_upto = eq;
  scan_block(upto, eq_upto, sh.scan, sh.scan_n);
  const u64 take = min((u64)eq_upto, t) - min((u64)(eq_upto - eq), t);   // of those equal to K, in order, the first t
  mine += take * wK;
  upto += min((u64)eq_upto, t) * wK;
  if (tid == kNT - 1) {
    sh.total = upto;
    sh.found = -1;
  }
  __syncthreads();
  if (!placed) {
    total = sh.total;
    goal = drawn(u01, total);
  }
  __syncthreads();
  if (tid < ctas * kWarps && tid / kWarps == rank && goal < upto && goal >= upto - mine) {
    sh.found = tid % kWarps;               // the stretch that has it
    sh.found_before = upto - mine;
    sh.total = take;                       // how many of the stretch's equals are kept
  }
  __syncthreads();
  const bool chosen_here = warp == sh.found;
  u64 left = goal - sh.found_before;
  int spare = (int)min(sh.total, (u64)INT32_MAX);
  for (int j0 = first; chosen_here && j0 < last; j0 += 32) {
    const int j = j0 + lane;
    const uint4 u = j < last ? there(j) : make_uint4(0u, 0u, 0u, 0u);
    u64 w[N], s = 0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float l = j < last ? Vec<T>::at(u, i) : -INFINITY;
      int steps;
      w[i] = weigh.of_counting(l, steps);
      if (!(l > K)) w[i] = 0ull;
      s += w[i];
      n += l == K;
    }
    int n_upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, n_upto, o);
      if (lane >= o) n_upto += y;
    }
    int may = spare - (n_upto - n);                       // equals that this lane may still keep
    s += (u64)max(0, min(n, may)) * wK;
    const u64 s_upto = scan_warp(s);
    const unsigned hit = __ballot_sync(0xffffffffu, left < s_upto);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        u64 before = s_upto - s;
        int at = -1;
        float chosen = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float l = Vec<T>::at(u, i);
          if (l == K && may-- > 0) w[i] = wK;
          before += w[i];
          if (at < 0 && left < before) {
            at = i;
            chosen = l;
          }
        }
        put(j * N - row.lead + at, chosen, total);
      }
      break;
    }
    left -= __shfl_sync(0xffffffffu, s_upto, 31);
    spare -= __shfl_sync(0xffffffffu, n_upto, 31);
  }
  if (placed) meet();                   // no CTA leaves while another reads it
}

template <typename T>
cudaError_t run(const SampleArgs& a, cudaStream_t st) {
  // 16-byte vectors of a row, wherever it starts
  const long long vectors = ((long long)a.vocab * sizeof(T) + 15) / 16 + 1;
  int ctas = 1;
  while (ctas < kMaxCtas && vectors > 512ll * ctas) ctas *= 2;
  auto part = [&]() { return (size_t)((vectors + ctas - 1) / ctas) * 16; };
  // Of more rows than run at once, fewer CTAs to a row: what a row takes besides looking
  // at its logits is the same for all of them. A cluster is of CTAs of one GPC, so what
  // runs at once goes by its size; the steps, 36 rows by 8, 52 by 5, 76 by 4 and 160 by 2,
  // are a few rows above that. Under top_p, by 1, 2, 4, 5 and 8 CTAs:
  //   40 fp32 rows of 65537: 93, 40, 36, 33 and 44 us; 64 rows: 94, 40, 37, 52 and 52;
  //   100 rows: 94, 69, 58, 62 and 76; 200 rows: 120, 111, 101, 115 and 145
  //   100 bf16 rows of 32000: 32, 33, 40, 48 and 57 us; 200 rows: 48, 52, 70, 89 and 107
  // At a step itself the next fewer are ahead (36 fp32 rows of 65537 by 8: 37 us, by
  // 5: 32; 76 rows by 4: 55 us, by 2: 40), and up to 45 rows by 6, which are none of the
  // choices, take 30 us.
  // But up to a hundred rows only where its part still fits beside another CTA's, and then
  // four at least: what is not held is read again in each pass (bf16 rows of 202048 by 8,
  // which hold them, and by 4: 48 rows under top_p 44 us both, without filters 40 and 43;
  // 100 rows 76 and 70, 66 and 72; 256 rows 178 and 164, 157 and 154, by 2 171 and 151, by 1
  // 226 and 162. By 5, which hold none either, 48 rows take 37 and 34.)
  static const struct { int most, fewer; } kFit[kMaxCtas + 1] = {{}, {}, {160, 1}, {}, {76, 2}, {52, 4}, {}, {}, {36, 5}};
  while (ctas > 1 && a.rows > kFit[ctas].most) {
    const int before = ctas;
    ctas = kFit[ctas].fewer;
    if (part() > kStagedTwo && (ctas < 4 || a.rows <= 100)) {
      ctas = before;
      break;
    }
  }
  const size_t bytes = part();
  const bool staged = bytes <= (a.rows * ctas <= 152 ? kStaged : kStagedTwo);
  auto kernel = staged ? sample_kernel<T, true> : sample_kernel<T, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kStaged);
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
