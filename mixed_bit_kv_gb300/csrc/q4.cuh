// Shared parts of the 4-bit paged cache (rdkv_q4_* in include/rdkv.h): the page layout, the rows' types
// and the host checks.
#pragma once

#include <cfloat>

#include "paged.cuh"

namespace rdkv {
namespace q4 {

using namespace paged;

constexpr int kGroup = 32;             // channels that share a scale and a zero
constexpr float kHalfMax = 65504.0f;
static_assert(RDKV_Q4_PAGE_TOKENS == kPage && RDKV_Q4_MAX_QUERIES == kMaxQueries && RDKV_Q4_COUNTER_BYTES == kCounterBytes, "as in the header");

// Byte offsets inside one (page, KV head); the K half (codes, scales, zeros) comes first, so that each
// half is one bulk copy.
template <int D>
struct Layout {
  static constexpr int NG = D / kGroup;
  static constexpr int kCodes = kPage * D / 2, kMeta = kPage * NG * 2;
  static constexpr int kKCodes = 0, kKScales = kCodes, kKZeros = kCodes + kMeta;
  static constexpr int kHalf = kCodes + 2 * kMeta;  // bytes of the K half and of the V half: 40 D
  static constexpr int kVCodes = kHalf, kVScales = kHalf + kCodes, kVZeros = kHalf + kCodes + kMeta;
  static constexpr int kBytes = 2 * kHalf;
};

// What a kernel reads of the cache.
struct View : PageView {
  uint8_t* pages;
  __half* bounds;
};

inline View view_of(const rdkv_q4_cache* c) { return View{page_view(c), c->pages, reinterpret_cast<__half*>(c->bounds)}; }

// Four pairs of codes of a word: at bits 0 and 16 (2^-24), 4 and 20 (2^-20), and the same of the upper bytes.
struct Pairs {
  uint32_t a, b, c, d;
};
__device__ __forceinline__ Pairs code_pairs(uint32_t w) {
  const uint32_t u = w >> 8;
  return Pairs{w & 0x000f000fu, w & 0x00f000f0u, u & 0x000f000fu, u & 0x00f000f0u};
}

// two fp32 products and sums in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)), "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 add2f(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}

// ---------------------------------------------------------------- host checks
rdkv_status check_cache(const rdkv_q4_cache* c);
rdkv_status check_rows(const rdkv_q4_cache* c, int32_t dtype, const void* k, const void* v, int64_t rows, int64_t row_stride,
                       const int32_t* row_start, int32_t max_rows);
rdkv_status check_queries(const rdkv_q4_cache* c, int32_t h_q, int32_t n_q);
rdkv_status check_q(const rdkv_q4_cache* c, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q, int32_t n_q);

}  // namespace q4
}  // namespace rdkv
