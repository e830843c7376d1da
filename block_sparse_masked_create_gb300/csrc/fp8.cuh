// e4m3 conversions and the block scale of the 8-bit paged cache.
#pragma once

#include <cuda_fp16.h>

#include "fa_internal.cuh"

namespace fa {

constexpr int kScaleTokens = FA_KV_SCALE_TOKENS;             // tokens that share a scale
constexpr float kScaleMin = 9.094947017729282e-13f;          // 2^-40
constexpr float kScaleMax = 1099511627776.0f;                // 2^40

// A scale read from memory. Outside [2^-40, 2^40], and NaN, it reads as the nearest bound (NaN: the lower one),
// so that the scale of a page that nobody wrote can reach no visible value.
__device__ __forceinline__ float clamp_scale(float s) { return fminf(fmaxf(s, kScaleMin), kScaleMax); }

// Smallest power of two s with amax <= 448 s, within the bounds above. 448 = 1.75 * 2^8, so with amax = m * 2^e the
// exponent is e - 8, or e - 7 where m > 1.75: exact, from the bits.
__device__ __forceinline__ float need_scale(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7FFFFFFFu;
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = min(max(e, -40), 40);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// four values -> four e4m3 (round to nearest even, saturating at 448; NaN stays NaN)
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// four e4m3 -> two pairs of fp16, exactly (e4m3's smallest subnormal is 2^-9)
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The key positions [begin, end) that some query row of batch row b may see, by the rule's terms: their causal and prefix bounds for
// the end, their windows for the begin. What pages hold before (they fell out of every window) and behind (slots after a
// sequence) is read as zero, and ids of pages with nothing in between are not looked at.
struct KeyRange {
  int begin, end;
};
__device__ __forceinline__ KeyRange key_range(const DevRule& R, int Bm, int b, int q_len, int kv_len) {
  const int64_t first = R.q_offset ? __ldg(R.q_offset + (Bm > 1 ? b : 0)) : 0, behind = first + q_len;
  int64_t begin = kv_len, end = 0;
  for (int t = 0; t < R.n_terms; ++t) {
    int64_t lo = 0, hi = kv_len;
    if (R.t[t].win != INT64_MAX) lo = max(lo, first - R.t[t].win + 1);
    if (R.t[t].causal) hi = min(hi, behind);
    if (R.t[t].pre != INT64_MAX) hi = min(hi, R.t[t].pre);
    begin = min(begin, lo);
    end = max(end, hi);
  }
  return KeyRange{(int)begin, (int)end};
}

// tanh(u) = 1 - 2 / (1 + e^2u), good to 2^-22 absolute: two special-function operations where tanh.approx takes one (and is
// off by 8e-6). Below kTanhSmall the difference would lose the small value's digits, and the Taylor series up to u^13 takes its
// place (its next term, 929569 / 638512875 u^15, is under 2^-23 of u there).
constexpr float kTanhSmall = 0.5f;
constexpr float kTanh3 = -1.f / 3.f, kTanh5 = 2.f / 15.f, kTanh7 = -17.f / 315.f, kTanh9 = 62.f / 2835.f,
                kTanh11 = -1382.f / 155925.f, kTanh13 = 21844.f / 6081075.f;

__device__ __forceinline__ float tanh_exact(float u) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(u * 2.885390081777927f /* 2 log2(e) */)));
  const float s = u * u;
  float p = fmaf(s, fmaf(s, kTanh13, kTanh11), kTanh9);
  p = fmaf(s, fmaf(s, fmaf(s, p, kTanh7), kTanh5), kTanh3);
  return fabsf(u) < kTanhSmall ? u * fmaf(s, p, 1.f) : fmaf(-2.f, r, 1.f);
}

// c * tanh(x / c)
__device__ __forceinline__ float softcap_exact(float x, float c, float inv_c) { return c * tanh_exact(x * inv_c); }

}  // namespace fa
