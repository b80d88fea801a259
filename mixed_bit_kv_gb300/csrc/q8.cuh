// Shared parts of the 8-bit paged cache (rdkv_q8_* in include/rdkv.h): the page layout, the codes and the
// host checks.
#pragma once

#include "paged.cuh"

namespace rdkv {
namespace q8 {

using namespace paged;

static_assert(RDKV_Q8_PAGE_TOKENS == kPage && RDKV_Q8_MAX_QUERIES == kMaxQueries && RDKV_Q8_COUNTER_BYTES == kCounterBytes, "as in the header");
constexpr int kLowExp = -24, kHighExp = 7;  // of a scale
constexpr float kMost = 57344.0f;           // 448 2^7

// What a kernel reads of the cache.
struct View : PageView {
  uint8_t* pages;
  float* scales;
};

inline View view_of(const rdkv_q8_cache* c) { return View{page_view(c), c->pages, c->scales}; }

// One (page, KV head): the codes of the keys, then the values', both in the order in which a lane of a product's
// operand takes them, so that its loads are 16 bytes and a warp's are 512 in a row.
//   Keys: lane (g, q) of a product has token g and, of every 64 channels, the 16 from 16 q on.
//   Values: it has of every run of 8 tokens the pair q and, of every 64 channels, the 8 from 8 g on, a pair's two codes side by side.
template <int D>
struct Layout {
  static constexpr int kHalf = kPage * D, kBytes = 2 * kHalf;
  static constexpr int kSides = D / 64;
  // byte of 8 channels 64 j + 8 c .. of token t
  static __device__ __forceinline__ int key_at(int t, int j, int c) { return t / 2 * 2 * D + j * 128 + (t & 1) * 64 + 8 * c; }
  // byte of the chunk of channels 64 j + 8 g .. of token pair p
  static __device__ __forceinline__ int value_at(int p, int j, int g) { return p / 4 * 8 * D + j * 512 + g * 64 + p % 4 * 16; }
};

// ---------------------------------------------------------------- scales
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ int exponent(float scale) { return (int)(__float_as_uint(scale) >> 23) - 127; }
// The scale's exponent for magnitudes up to top = m 2^k, 1 <= m < 2: 448 is 1.75 2^8.
__device__ __forceinline__ int exponent_for(float top) {
  const uint32_t w = __float_as_uint(fminf(top, kMost));
  return max(kLowExp, (int)(w >> 23) - 135 + ((w & 0x7fffffu) > 0x600000u ? 1 : 0));
}

// ---------------------------------------------------------------- codes
// Two codes in 16 bits, the first lowest; past +-448: +-448.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) { return codes2(a, b) | codes2(c, d) << 16; }
// What is no number has code 127, whatever its sign: it becomes 0.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  const uint32_t bad = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return w & ~((bad >> 7) * 255u);
}
// The halves of a word of codes as two fp16 numbers each, exactly.
__device__ __forceinline__ uint32_t halves_lo(uint32_t w) {
  uint32_t d;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t w) {
  uint32_t d;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(d) : "r"(w));
  return d;
}
// Four codes' values in units of their scale.
__device__ __forceinline__ void values4(uint32_t w, float (&x)[4]) {
  const float2 a = unpack2(halves_lo(w)), b = unpack2(halves_hi(w));
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
// The codes of a word in a scale 1 / f times as large.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float f) {
  float x[4];
  values4(w, x);
  return codes4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}

// ---------------------------------------------------------------- host checks
rdkv_status check_cache(const rdkv_q8_cache* c);
rdkv_status check_mass(const rdkv_q8_cache* c, const float* mass, int64_t mass_stride);

}  // namespace q8
}  // namespace rdkv
