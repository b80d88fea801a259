// Shared parts of the 4-bit paged cache (rdkv_q4_* in include/rdkv.h): the page layout, the rows' types
// and the host checks.
#pragma once

#include <cuda_bf16.h>

#include <cfloat>

#include "common.cuh"

namespace rdkv {
namespace q4 {

constexpr int kPage = RDKV_Q4_PAGE_TOKENS;
constexpr int kGroup = 32;             // channels that share a scale and a zero
constexpr float kHalfMax = 65504.0f;

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
struct View {
  int batch, h_kv, n_pages, page_stride;
  uint8_t* pages;
  __half* bounds;
  const int32_t* page_table;
  const int32_t* lens;
  int32_t* status;
};

inline View view_of(const rdkv_q4_cache* c) {
  return View{c->batch,  c->h_kv, c->n_pages, c->page_stride, c->pages, reinterpret_cast<__half*>(c->bounds), c->page_table, c->lens,
              c->status};
}

// Loads of what the kernel before may have written.  These kernels are set up while that one still runs
// (launch_after), so the read-only path, whose data must not change during the kernel, is not for them; and the
// volatile statements keep their place behind the wait.
__device__ __forceinline__ uint16_t fetch(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t fetch(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int32_t fetch(const int32_t* p) { return (int32_t)fetch(reinterpret_cast<const uint32_t*>(p)); }
__device__ __forceinline__ uint2 fetch(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 fetch(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Lets the next kernel on the stream be set up, and waits for the one before to end.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void raise(const View& v, int code) { atomicMax(v.status, code); }

// Reports a length that no sequence can have.
__device__ __forceinline__ void check_length(const View& v, int b) {
  const int len = fetch(v.lens + b);
  if (len < 0) raise(v, RDKV_ERR_INVALID_ARG);
  if ((int64_t)len > (int64_t)v.page_stride * kPage) raise(v, RDKV_ERR_CAPACITY);
}
// Tokens that sequence b holds, cut to what its page table can hold.
__device__ __forceinline__ int held_tokens(const View& v, int b) {
  const int n = fetch(v.lens + b);
  return max(0, (int)min((int64_t)n, (int64_t)v.page_stride * kPage));
}

// ---------------------------------------------------------------- rows of the model's types
// Two values in fp16, cut to its range.
__device__ __forceinline__ uint32_t cut_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <typename T>
struct Eight;  // eight consecutive channels
template <>
struct Eight<__half> {
  static __device__ __forceinline__ void load(const __half* p, float (&x)[8]) {
    const uint4 u = fetch(reinterpret_cast<const uint4*>(p));
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store(__half* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(cut_half2(x[0], x[1]), cut_half2(x[2], x[3]), cut_half2(x[4], x[5]), cut_half2(x[6], x[7]));
  }
};
template <>
struct Eight<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = fetch(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = u;
  }
};
template <>
struct Eight<float> {
  static __device__ __forceinline__ void load(const float* p, float (&x)[8]) {
    const uint4 a = fetch(reinterpret_cast<const uint4*>(p)), b = fetch(reinterpret_cast<const uint4*>(p) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// One value of a type that is named at run time.
__device__ __forceinline__ float load_q(const void* p, int64_t i, int dtype) {
  if (dtype == RDKV_F32) return static_cast<const float*>(p)[i];
  if (dtype == RDKV_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// ---------------------------------------------------------------- arithmetic
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
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four pairs of codes of a word: at bits 0 and 16 (2^-24), 4 and 20 (2^-20), and the same of the upper bytes.
struct Pairs {
  uint32_t a, b, c, d;
};
__device__ __forceinline__ Pairs code_pairs(uint32_t w) {
  const uint32_t u = w >> 8;
  return Pairs{w & 0x000f000fu, w & 0x00f000f0u, u & 0x000f000fu, u & 0x00f000f0u};
}

// ---------------------------------------------------------------- launches
// Launches a kernel that waits (griddepcontrol.wait) before it touches global memory, so that its blocks may
// be set up while the kernel before it on the stream ends.
template <class Kernel, class... Args>
inline cudaError_t launch_after(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- host checks
inline int size_of(int32_t dtype) { return dtype == RDKV_F32 ? 4 : 2; }
rdkv_status check_cache(const rdkv_q4_cache* c);
rdkv_status check_rows(const rdkv_q4_cache* c, int32_t dtype, const void* k, const void* v, int64_t rows, int64_t row_stride,
                       const int32_t* row_start, int32_t max_rows);
rdkv_status check_queries(const rdkv_q4_cache* c, int32_t h_q, int32_t n_q);
rdkv_status check_q(const rdkv_q4_cache* c, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q, int32_t n_q);

}  // namespace q4
}  // namespace rdkv
