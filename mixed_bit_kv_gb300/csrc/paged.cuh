// Shared parts of the paged caches (rdkv_q4_* and rdkv_q8_* in include/rdkv.h): which pages and rows a call
// touches, the rows' types, waits, products of 16-bit operands, launches and the host checks that both make.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace rdkv {
namespace paged {

constexpr int kPage = 64;              // tokens
constexpr int kMaxQueries = 64;        // query tokens of a sequence in a call
constexpr int kCounterBytes = 262144;  // of the workspaces that hold counters

// What a kernel reads of a cache, its pages' contents aside.
struct PageView {
  int batch, h_kv, n_pages, page_stride;
  const int32_t* page_table;
  const int32_t* lens;
  int32_t* status;
};
template <class Cache>
PageView page_view(const Cache* c) {
  return PageView{c->batch, c->h_kv, c->n_pages, c->page_stride, c->page_table, c->lens, c->status};
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

__device__ __forceinline__ void raise(const PageView& v, int code) { atomicMax(v.status, code); }

// Reports a length that no sequence can have.
__device__ __forceinline__ void check_length(const PageView& v, int b) {
  const int len = fetch(v.lens + b);
  if (len < 0) raise(v, RDKV_ERR_INVALID_ARG);
  if ((int64_t)len > (int64_t)v.page_stride * kPage) raise(v, RDKV_ERR_CAPACITY);
}
// Tokens that sequence b holds, cut to what its page table can hold.
__device__ __forceinline__ int held_tokens(const PageView& v, int b) {
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

// ---------------------------------------------------------------- rows and the pages they fall in
struct Rows {
  int64_t n, stride;     // rows of k and v, elements between them
  const int32_t* start;  // or NULL: max_rows rows a sequence
  const int32_t* first;  // reading: position of a sequence's first row (NULL: 0)
  int32_t max_rows;
  int runs;              // pages that max_rows consecutive positions can touch
};

// The part of sequence b's rows that lies in its run-th page.
struct Run {
  int64_t row;   // row of the first token
  int64_t page;  // physical page, -1: nothing to do
  int s0, s1;    // slots [s0, s1)
};

template <bool kWrite>
__device__ __forceinline__ Run find_run(const PageView& v, const Rows& r, int b, int run) {
  Run o{0, -1, 0, 0};
  const int len = fetch(v.lens + b);
  const int64_t cap = (int64_t)v.page_stride * kPage;
  int64_t r0, n;
  if (r.start) {
    r0 = fetch(r.start + b);
    n = (int64_t)fetch(r.start + b + 1) - r0;
  } else {
    r0 = (int64_t)b * r.max_rows;
    n = len != 0 || !kWrite ? r.max_rows : 0;
  }
  if (n == 0) return o;
  const int64_t first = kWrite ? (int64_t)len - n : r.first ? (int64_t)fetch(r.first + b) : 0;
  if (n < 0 || n > r.max_rows || r0 < 0 || r0 + n > r.n || first < 0 || len < 0) {
    if (threadIdx.x == 0) raise(v, RDKV_ERR_INVALID_ARG);
    return o;
  }
  int64_t end = first + n;
  if (!kWrite) end = min(end, (int64_t)len);
  if (end > cap) {
    if (threadIdx.x == 0) raise(v, RDKV_ERR_CAPACITY);
    end = cap;
  }
  const int64_t lp = first / kPage + run, t0 = lp * kPage;
  if (t0 >= end) return o;
  o.s0 = (int)(max(first, t0) - t0);
  o.s1 = (int)(min(end, t0 + kPage) - t0);
  o.row = r0 + (t0 + o.s0 - first);
  o.page = fetch(v.page_table + (int64_t)b * v.page_stride + lp);
  if (o.page < 0 || o.page >= v.n_pages) {
    if (threadIdx.x == 0) raise(v, RDKV_ERR_INVALID_ARG);
    o.page = -1;
  }
  return o;
}

// ---------------------------------------------------------------- arithmetic
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same product on a zero accumulator
__device__ __forceinline__ void mma16z(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// an 8 x 8 matrix of halves, a row in four lanes, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t w) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// the remainders of two values past their fp16 parts, times kUp
template <int kUp = 1>
__device__ __forceinline__ uint32_t rest2(float lo, float hi, uint32_t w) {
  const float2 f = unpack2(w);
  return pack2((lo - f.x) * kUp, (hi - f.y) * kUp);
}

// ---------------------------------------------------------------- waits and shares of the work
constexpr long long kWaitCycles = 4000000000LL;  // a bounded wait, about two seconds
constexpr long long kMinWaitCycles = 100000;     // shortest limit the self-test may ask for
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, long long limit) {
  if (try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!try_wait(bar, parity))
    if (clock64() - t0 > limit) return false;
  return true;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x / y for 0 <= x, 0 < y: 32 bits where they do (a 64-bit division takes some hundred instructions)
__device__ __forceinline__ int quotient(int64_t x, int y) {
  if ((x >> 32) == 0) return (int)((uint32_t)x / (uint32_t)y);
  return (int)(x / y);
}
// The first of n items that part i of `parts` equal ones takes.
__device__ __forceinline__ int share(int i, int n, int parts) { return quotient((int64_t)i * n, parts); }

// A row's sums by its sum of weights (0: zero).
__device__ __forceinline__ float4 scaled(float4 o, float l) {
  const float f = l != 0.0f ? 1.0f / l : 0.0f;
  return make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
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
inline rdkv_status check_dtype(int32_t dtype) {
  RDKV_REQUIRE(dtype == RDKV_F16 || dtype == RDKV_F32 || dtype == RDKV_BF16, RDKV_ERR_UNSUPPORTED, "dtype %d", dtype);
  return RDKV_OK;
}

// (the cache's own buffers aside)
template <class Cache>
rdkv_status check_pool(const Cache* c) {
  RDKV_REQUIRE(c != nullptr, RDKV_ERR_INVALID_ARG, "cache is NULL");
  RDKV_REQUIRE(c->batch >= 1 && c->h_kv >= 1 && c->n_pages >= 1 && c->page_stride >= 1, RDKV_ERR_INVALID_ARG,
               "cache sizes must be positive (batch=%d h_kv=%d n_pages=%d page_stride=%d)", c->batch, c->h_kv,
               c->n_pages, c->page_stride);
  RDKV_REQUIRE(c->head_dim == 64 || c->head_dim == 128, RDKV_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}",
               c->head_dim);
  RDKV_REQUIRE((int64_t)c->page_stride * kPage <= INT32_MAX, RDKV_ERR_UNSUPPORTED,
               "page_stride %d: more than 2^31 - 1 tokens a sequence", c->page_stride);
  RDKV_REQUIRE((int64_t)c->n_pages * c->h_kv <= INT32_MAX, RDKV_ERR_UNSUPPORTED, "more than 2^31 - 1 (page, KV head) pairs");
  RDKV_REQUIRE((int64_t)c->batch * c->h_kv <= 1 << 20, RDKV_ERR_UNSUPPORTED, "more than 2^20 (sequence, KV head) pairs");
  RDKV_REQUIRE(c->pages && c->page_table && c->lens && c->status, RDKV_ERR_INVALID_ARG, "NULL pointer in the cache");
  return RDKV_OK;
}

template <class Cache>
rdkv_status check_rows_of(const Cache* c, int32_t dtype, const void* k, const void* v, int64_t rows, int64_t row_stride,
                          const int32_t* row_start, int32_t max_rows) {
  const rdkv_status st = check_dtype(dtype);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(max_rows >= 0, RDKV_ERR_INVALID_ARG, "max_rows %d", max_rows);
  RDKV_REQUIRE(rows >= (row_start ? 0 : (int64_t)c->batch * max_rows), RDKV_ERR_INVALID_ARG, "%lld rows for %d sequences of %d",
               (long long)rows, c->batch, max_rows);
  RDKV_REQUIRE((k && v) || max_rows == 0, RDKV_ERR_INVALID_ARG, "NULL rows");
  RDKV_REQUIRE(((uintptr_t)k | (uintptr_t)v) % 16 == 0 && row_stride % (16 / size_of(dtype)) == 0, RDKV_ERR_INVALID_ARG,
               "rows must be 16-byte aligned (row_stride %lld)", (long long)row_stride);
  RDKV_REQUIRE(row_stride >= (int64_t)c->h_kv * c->head_dim, RDKV_ERR_INVALID_ARG, "row_stride %lld < h_kv * head_dim",
               (long long)row_stride);
  return RDKV_OK;
}

template <class Cache>
rdkv_status check_heads_of(const Cache* c, int32_t h_q, int32_t n_q) {
  RDKV_REQUIRE(h_q >= 1 && h_q % c->h_kv == 0, RDKV_ERR_INVALID_ARG, "h_q=%d is not a multiple of h_kv=%d", h_q, c->h_kv);
  RDKV_REQUIRE(h_q / c->h_kv <= 8, RDKV_ERR_UNSUPPORTED, "group size %d > 8", h_q / c->h_kv);
  RDKV_REQUIRE(n_q >= 1, RDKV_ERR_INVALID_ARG, "n_q %d", n_q);
  RDKV_REQUIRE(n_q <= kMaxQueries, RDKV_ERR_UNSUPPORTED, "n_q %d > %d", n_q, kMaxQueries);
  // a counter each in the workspaces; also a grid's second size
  RDKV_REQUIRE((int64_t)c->batch * n_q * c->h_kv <= kCounterBytes / 4 - 1, RDKV_ERR_UNSUPPORTED,
               "more than 65,535 (sequence, query token, KV head) triples");
  return RDKV_OK;
}

template <class Cache>
rdkv_status check_queries_of(const Cache* c, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q) {
  const rdkv_status st = check_dtype(dtype);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(q != nullptr, RDKV_ERR_INVALID_ARG, "NULL queries");
  RDKV_REQUIRE((uintptr_t)q % 16 == 0 && q_stride % (16 / size_of(dtype)) == 0, RDKV_ERR_INVALID_ARG,
               "queries must be 16-byte aligned (q_stride %lld)", (long long)q_stride);
  RDKV_REQUIRE(q_stride >= (int64_t)h_q * c->head_dim, RDKV_ERR_INVALID_ARG, "q_stride %lld < h_q * head_dim",
               (long long)q_stride);
  return RDKV_OK;
}

template <class Cache>
rdkv_status grid_of(const Cache* c, Rows* r, int64_t* blocks) {
  // max_rows positions from anywhere in a page, within what the table can hold
  r->runs = (int)std::min<int64_t>(ceil_div64((int64_t)r->max_rows + kPage - 1, kPage), c->page_stride);
  *blocks = (int64_t)c->batch * c->h_kv * r->runs;
  RDKV_REQUIRE(*blocks <= INT32_MAX, RDKV_ERR_UNSUPPORTED, "max_rows %d: too many (sequence, head, page) items", r->max_rows);
  return RDKV_OK;
}

}  // namespace paged
}  // namespace rdkv
