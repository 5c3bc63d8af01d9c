// Tensor-core pieces the paged kernels share: TMA maps of the pages and of the
// query rows, TMEM access 32 columns at a time, an MMA whose A operand lies in
// TMEM, and the fast exponential and cap.
#pragma once

#include "paged.cuh"
#include "ptx.cuh"

namespace dfl {

constexpr int kPtKeys = 128;               // keys (or query rows) of an operand tile

// A wait that stops waiting once any wait of the thread gave up.
__device__ __forceinline__ void paged_wait(uint64_t* bar, unsigned parity, bool& ok) {
  if (!ok) return;
  const uint32_t a = smem_u32(bar);
#pragma unroll 1
  for (unsigned i = 0; i < (1u << 20); ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(a), "r"(parity) : "memory");
    if (done) return;
  }
  ok = false;
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// 32 lanes x 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return r;
}
// Waits for the loads before it; v's values exist only afterwards.
__device__ __forceinline__ void tmem_ld_wait32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), 
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), 
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// S[tmem 128 x 128] = A B^T over `steps` (<= 4 HALVES) K steps of 16: both
// operands 128 K-major rows in tiles of 64 columns, given by the descriptors of
// their first bytes. Whatever one lane spends between two MMAs is time the
// tensor cores may wait, so a step adds a constant to a descriptor (its low
// bits count 16 bytes) and nothing else.
template <int HALVES>
__device__ __forceinline__ void tc_scores(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, int steps) {
  constexpr uint32_t idesc = idesc_bf16(128, 128);
#pragma unroll
  for (int k = 0; k < 4 * HALVES; ++k) {
    const uint64_t off = (k >> 2) * (kPtKeys * 128 >> 4) + (k & 3) * 2;
    if (k < steps) tc_mma_bf16(d_tmem, a_desc + off, b_desc + off, idesc, k ? 1u : 0u);
  }
}

// D[tmem] (+)= A[tmem] * B[smem desc], bf16 inputs, fp32 accumulators. A: row
// i in lane i, two consecutive K elements to a 32-bit column.
__device__ __forceinline__ void tc_mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A 128-byte-swizzled operand whose rows run along K (N contiguous): rows of
// 64 elements, 8-row atoms 1024 bytes apart along K, the next 64 elements of
// N `lead` bytes on.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kIdescBMnMajor = 1u << 16;   // instruction descriptor: B is N-contiguous

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction; operands are pairs of registers.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// cap2 * tanh(x / 2 / log2(e)) for x in log2 units of e^(2 z): 1 - 2 / (1 + e^2z),
// whose error is a few 2^-24 of cap2 everywhere (a hardware tanh has 2^-11).
__device__ __forceinline__ float cap_tanh(float x, float cap2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(x)));
  return fmaf(-2.f * cap2, r, cap2);
}

// v = cap2 * tanh(v * scale) for 32 values of every lane of a warp. For a value
// of at most half the cap, as most scores are, tanh(y) / y is a polynomial of
// degree 4 in y^2 (interpolated at the Chebyshev nodes of [0, 1/4]; within 2^-23
// of it in fp32), with scale and cap2 in its coefficients: six packed
// instructions to two values, where the exponential and the reciprocal would
// bound capped attention (512 rows' key weights over 32768 keys, cap 20: 335 us
// with it, 459 us without; 365 us since hidden scores have no say in the choice).
// Where some value of the warp is larger, all take the exponential, whose error of
// a few 2^-24 of the cap is nothing beside scores of half of it; under a cap so vast that it could be (cap2 > 1024) each value takes
// its own. (Each its own under every cap: 2048 rows over 32768 keys under a cap
// of 2 took 3.40 ms instead of 1.98 ms.) limit: the largest |v| for the
// polynomial, none where a power of the scale would leave fp32.
struct CapPoly { uint64_t c[5]; float scale, cap2, limit; };
__device__ __forceinline__ CapPoly cap_poly(float scale, float cap2) {
  const float c[5] = {1.0f, -0.3333306908607483f, 0.133247509598732f, -0.05298423767089844f, 0.017131345346570015f};
  CapPoly p;
  p.scale = scale;
  p.cap2 = cap2;
  p.limit = scale <= 1024.f ? 0.5f / scale : -1.f;
  float f = scale * cap2;
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    p.c[k] = pack2(c[k] * f, c[k] * f);
    f *= scale * scale;
  }
  return p;
}
// The same of one value.
__device__ __forceinline__ float cap_tanh1(float v, const CapPoly& p) {
  if (!(fabsf(v) <= p.limit)) return cap_tanh(v * (p.scale * 2.8853900817779268f), p.cap2);
  float r = 0.f, unused;
#pragma unroll
  for (int k = 4; k >= 0; --k) {
    float c;
    unpack2(p.c[k], c, unused);
    r = fmaf(r, v * v, c);
  }
  return r * v;
}
__device__ __forceinline__ bool cap_fits(const float* v, const CapPoly& p) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 32; j += 2) top = fmaxf(fmaxf(top, fabsf(v[j])), fabsf(v[j + 1]));
  return __all_sync(0xffffffffu, top <= p.limit);
}
// hide() makes zeros of the scores that are not seen: they must not decide how
// the others are computed. It is called only where they might.
template <typename F>
__device__ __forceinline__ void cap_tanh32(float* v, const CapPoly& p, bool some_hidden, F&& hide) {
  bool fits = cap_fits(v, p);
  if (!fits && some_hidden) {
    hide();
    fits = cap_fits(v, p);
  }
  auto poly = [&](float v0, float v1, float& r0, float& r1) {
    const uint64_t y = pack2(v0, v1), z = mul2(y, y);
    uint64_t r = p.c[4];
#pragma unroll
    for (int k = 3; k >= 0; --k) r = fma2(r, z, p.c[k]);
    unpack2(mul2(r, y), r0, r1);
  };
  if (fits) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) poly(v[j], v[j + 1], v[j], v[j + 1]);
  } else {
    const float twice = p.scale * 2.8853900817779268f;   // 2 log2(e)
    if (p.cap2 <= 1024.f) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = cap_tanh(v[j] * twice, p.cap2);
    } else {
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float r0, r1;
        poly(v[j], v[j + 1], r0, r1);
        v[j] = fabsf(v[j]) <= p.limit ? r0 : cap_tanh(v[j] * twice, p.cap2);
        v[j + 1] = fabsf(v[j + 1]) <= p.limit ? r1 : cap_tanh(v[j + 1] * twice, p.cap2);
      }
    }
  }
}

// Maps of K or V as rows of head_dim (boxes of 64 elements x up to `most` rows)
// and of the query rows as [rows][n_q_heads][head_dim] (boxes of 64 elements x
// G heads x per rows). Columns past head_dim and rows past the end read as 0.
bool paged_map_pages(CUtensorMap* m, const void* base, const PagedView& c, int most = kPtKeys);
bool paged_map_rows(CUtensorMap* m, const void* base, const PagedAttnArgs& a, int per);

}  // namespace dfl
