// The 4-bit paged cache: rows quantised as they are written (rdkv_q4_write) and read back
// (rdkv_q4_read), and the host checks that every rdkv_q4_* call makes.
#include "q4.cuh"
#include "stages.cuh"

namespace rdkv {
namespace q4 {

// ---------------------------------------------------------------- host checks
rdkv_status check_cache(const rdkv_q4_cache* c) {
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
  RDKV_REQUIRE(((uintptr_t)c->pages | (uintptr_t)c->bounds) % 16 == 0, RDKV_ERR_INVALID_ARG,
               "pages and bounds must be 16-byte aligned");
  return RDKV_OK;
}

static rdkv_status check_dtype(int32_t dtype) {
  RDKV_REQUIRE(dtype == RDKV_F16 || dtype == RDKV_F32 || dtype == RDKV_BF16, RDKV_ERR_UNSUPPORTED, "dtype %d", dtype);
  return RDKV_OK;
}

rdkv_status check_rows(const rdkv_q4_cache* c, int32_t dtype, const void* k, const void* v, int64_t row_stride,
                       int32_t max_rows) {
  rdkv_status st = check_cache(c);
  if (st != RDKV_OK) return st;
  st = check_dtype(dtype);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(max_rows >= 0, RDKV_ERR_INVALID_ARG, "max_rows %d", max_rows);
  RDKV_REQUIRE((k && v) || max_rows == 0, RDKV_ERR_INVALID_ARG, "NULL rows");
  RDKV_REQUIRE(((uintptr_t)k | (uintptr_t)v) % 16 == 0 && row_stride % (16 / size_of(dtype)) == 0, RDKV_ERR_INVALID_ARG,
               "rows must be 16-byte aligned (row_stride %lld)", (long long)row_stride);
  RDKV_REQUIRE(row_stride >= (int64_t)c->h_kv * c->head_dim, RDKV_ERR_INVALID_ARG, "row_stride %lld < h_kv * head_dim",
               (long long)row_stride);
  return RDKV_OK;
}

rdkv_status check_queries(const rdkv_q4_cache* c, int32_t h_q, int32_t n_q) {
  rdkv_status st = check_cache(c);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(h_q >= 1 && h_q % c->h_kv == 0, RDKV_ERR_INVALID_ARG, "h_q=%d is not a multiple of h_kv=%d", h_q, c->h_kv);
  RDKV_REQUIRE(h_q / c->h_kv <= 8, RDKV_ERR_UNSUPPORTED, "group size %d > 8", h_q / c->h_kv);
  RDKV_REQUIRE(n_q >= 1, RDKV_ERR_INVALID_ARG, "n_q %d", n_q);
  RDKV_REQUIRE(n_q <= RDKV_Q4_MAX_QUERIES, RDKV_ERR_UNSUPPORTED, "n_q %d > %d", n_q, RDKV_Q4_MAX_QUERIES);
  return RDKV_OK;
}

rdkv_status check_q(const rdkv_q4_cache* c, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q, int32_t n_q) {
  rdkv_status st = check_queries(c, h_q, n_q);
  if (st != RDKV_OK) return st;
  st = check_dtype(dtype);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(q != nullptr, RDKV_ERR_INVALID_ARG, "NULL queries");
  RDKV_REQUIRE((uintptr_t)q % 16 == 0 && q_stride % (16 / size_of(dtype)) == 0, RDKV_ERR_INVALID_ARG,
               "queries must be 16-byte aligned (q_stride %lld)", (long long)q_stride);
  RDKV_REQUIRE(q_stride >= (int64_t)h_q * c->head_dim, RDKV_ERR_INVALID_ARG, "q_stride %lld < h_q * head_dim",
               (long long)q_stride);
  return RDKV_OK;
}

// ---------------------------------------------------------------- rows and the pages they fall in
struct Rows {
  int64_t stride;
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
__device__ __forceinline__ Run find_run(const View& v, const Rows& r, int b, int run) {
  Run o{0, -1, 0, 0};
  const int len = __ldg(v.lens + b);
  const int64_t cap = (int64_t)v.page_stride * kPage;
  int64_t r0, n;
  if (r.start) {
    r0 = __ldg(r.start + b);
    n = (int64_t)__ldg(r.start + b + 1) - r0;
  } else {
    r0 = (int64_t)b * r.max_rows;
    n = len > 0 || !kWrite ? r.max_rows : 0;
  }
  if (n == 0) return o;
  const int64_t first = kWrite ? (int64_t)len - n : r.first ? (int64_t)__ldg(r.first + b) : 0;
  if (n < 0 || n > r.max_rows || r0 < 0 || first < 0 || len < 0) {
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
  o.page = __ldg(v.page_table + (int64_t)b * v.page_stride + lp);
  if (o.page < 0 || o.page >= v.n_pages) {
    if (threadIdx.x == 0) raise(v, RDKV_ERR_INVALID_ARG);
    o.page = -1;
  }
  return o;
}

constexpr int kThreads = 256;

// Codes of eight channels whose group of 32 is spread over four neighbouring lanes, with the group's
// scale and zero (the quantiser of the pack, on values cut to the fp16 range; a NaN takes no part in
// min and max and gets code 0).  xh: the values they stand for.
struct Codes {
  uint32_t c[8];
  QParams p;
};
__device__ __forceinline__ Codes quantise8(float (&x)[8], float (&xh)[8]) {
  float mn = INFINITY, mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = x[i] > kHalfMax ? kHalfMax : x[i] < -kHalfMax ? -kHalfMax : x[i];
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (mn > mx) mn = mx = 0.0f;
  Codes r;
  r.p = qparams(mn, mx, 4);
  const float rs = 1.0f / r.p.scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.c[i] = qcode_rcp(x[i], r.p.zero, r.p.scale, rs, 15.0f);
    xh[i] = fmaf(r.p.scale, (float)r.c[i], r.p.zero);
  }
  return r;
}

// One block per (sequence, KV head, page that its rows touch).  Eight channels a thread: one K code
// word, and the halves of two V code words.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) write_kernel(View v, Rows r, const T* __restrict__ k, const T* __restrict__ vv) {
  using L = Layout<D>;
  constexpr int kLanes = D / 8, kSlots = kThreads / kLanes, NG = L::NG;
  __shared__ __half lo_s[kSlots][D], hi_s[kSlots][D];
  const int run = blockIdx.x % r.runs, u = blockIdx.x / r.runs, h = u % v.h_kv, b = u / v.h_kv;
  const Run w = find_run<true>(v, r, b, run);
  if (w.page < 0) return;
  uint8_t* page = v.pages + ((int64_t)w.page * v.h_kv + h) * L::kBytes;
  const int l = threadIdx.x % kLanes, g0 = threadIdx.x / kLanes, grp = l / 4, q = l % 4;
  __half lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lo[i] = __float2half(INFINITY), hi[i] = __float2half(-INFINITY);
  for (int s0 = w.s0; s0 < w.s1; s0 += kSlots) {
    const int s = s0 + g0;
    const bool real = s < w.s1;
    const int64_t at = (w.row + (real ? s - w.s0 : 0)) * r.stride + (int64_t)h * D + 8 * l;
    float x[8], xh[8];
    Eight<T>::load(k + at, x);
    Codes c = quantise8(x, xh);
    if (real) {
      uint32_t word = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) word |= c.c[e] << bit_off(e, 4);
      reinterpret_cast<uint32_t*>(page + L::kKCodes)[(s * 4 + q) * NG + grp] = word;
      if (q == 0) {
        reinterpret_cast<uint16_t*>(page + L::kKScales)[(s / 2 * NG + grp) * 2 + s % 2] = c.p.scale_h;
        reinterpret_cast<uint16_t*>(page + L::kKZeros)[s * NG + grp] = c.p.zero_h;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half y = __float2half_rn(fminf(fmaxf(xh[i], -kHalfMax), kHalfMax));
        lo[i] = __hmin(lo[i], y), hi[i] = __hmax(hi[i], y);
      }
    }
    Eight<T>::load(vv + at, x);
    c = quantise8(x, xh);
    if (real) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t half = c.c[4 * j] | c.c[4 * j + 1] << 4 | c.c[4 * j + 2] << 8 | c.c[4 * j + 3] << 12;
        reinterpret_cast<uint16_t*>(page + L::kVCodes)[((s / 2 * 8 + 2 * q + j) * NG + grp) * 2 + s % 2] = (uint16_t)half;
      }
      if (q == 0) {
        const int m = (s / 2 * NG + grp) * 2 + s % 2;
        reinterpret_cast<uint16_t*>(page + L::kVScales)[m] = c.p.scale_h;
        reinterpret_cast<uint16_t*>(page + L::kVZeros)[m] = c.p.zero_h;
      }
    }
  }
  if (!v.bounds) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) lo_s[g0][8 * l + i] = lo[i], hi_s[g0][8 * l + i] = hi[i];
  __syncthreads();
  const int c = threadIdx.x % D, side = threadIdx.x / D;
  if (side >= 2) return;
  __half* out = v.bounds + (((int64_t)w.page * v.h_kv + h) * 2 + side) * D + c;
  __half m = side ? hi_s[0][c] : lo_s[0][c];
  for (int g = 1; g < kSlots; ++g) m = side ? __hmax(m, hi_s[g][c]) : __hmin(m, lo_s[g][c]);
  if (w.s0 > 0) m = side ? __hmax(m, *out) : __hmin(m, *out);
  *out = m;
}

// The same blocks the other way: eight channels a thread.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(View v, Rows r, T* __restrict__ k, T* __restrict__ vv) {
  using L = Layout<D>;
  constexpr int kLanes = D / 8, kSlots = kThreads / kLanes, NG = L::NG;
  const int run = blockIdx.x % r.runs, u = blockIdx.x / r.runs, h = u % v.h_kv, b = u / v.h_kv;
  const Run w = find_run<false>(v, r, b, run);
  if (w.page < 0) return;
  const uint8_t* page = v.pages + ((int64_t)w.page * v.h_kv + h) * L::kBytes;
  const int l = threadIdx.x % kLanes, grp = l / 4, q = l % 4;
  for (int s = w.s0 + threadIdx.x / kLanes; s < w.s1; s += kSlots) {
    const int64_t at = (w.row + s - w.s0) * r.stride + (int64_t)h * D + 8 * l;
    const int m = (s / 2 * NG + grp) * 2 + s % 2;
    float x[8];
    const uint32_t word = reinterpret_cast<const uint32_t*>(page + L::kKCodes)[(s * 4 + q) * NG + grp];
    float sc = __half2float(reinterpret_cast<const __half*>(page + L::kKScales)[m]);
    float z = __half2float(reinterpret_cast<const __half*>(page + L::kKZeros)[s * NG + grp]);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(sc, (float)((word >> bit_off(e, 4)) & 15u), z);
    Eight<T>::store(k + at, x);
    const uint16_t* codes = reinterpret_cast<const uint16_t*>(page + L::kVCodes);
    sc = __half2float(reinterpret_cast<const __half*>(page + L::kVScales)[m]);
    z = __half2float(reinterpret_cast<const __half*>(page + L::kVZeros)[m]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t half = codes[((s / 2 * 8 + 2 * q + j) * NG + grp) * 2 + s % 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * j + i] = fmaf(sc, (float)((half >> (4 * i)) & 15u), z);
    }
    Eight<T>::store(vv + at, x);
  }
}

static rdkv_status grid_of(const rdkv_q4_cache* c, Rows* r, int64_t* blocks) {
  // max_rows positions from anywhere in a page, within what the table can hold
  r->runs = (int)std::min<int64_t>(ceil_div64((int64_t)r->max_rows + kPage - 1, kPage), c->page_stride);
  *blocks = (int64_t)c->batch * c->h_kv * r->runs;
  RDKV_REQUIRE(*blocks <= INT32_MAX, RDKV_ERR_UNSUPPORTED, "max_rows %d: too many (sequence, head, page) items", r->max_rows);
  return RDKV_OK;
}

}  // namespace q4
}  // namespace rdkv

using namespace rdkv;
using namespace rdkv::q4;

extern "C" size_t rdkv_q4_page_bytes(int32_t head_dim) {
  return head_dim == 128 ? Layout<128>::kBytes : head_dim == 64 ? Layout<64>::kBytes : 0;
}

#define RDKV_Q4_ROWS_LAUNCH(kernel, ptr)                                                                         \
  switch (dtype * 256 + cache->head_dim) {                                                                       \
    case RDKV_F16 * 256 + 64: kernel<__half, 64><<<(unsigned)blocks, kThreads, 0, cs>>>(view, r, (ptr __half*)k, (ptr __half*)v); break;     \
    case RDKV_F16 * 256 + 128: kernel<__half, 128><<<(unsigned)blocks, kThreads, 0, cs>>>(view, r, (ptr __half*)k, (ptr __half*)v); break;   \
    case RDKV_F32 * 256 + 64: kernel<float, 64><<<(unsigned)blocks, kThreads, 0, cs>>>(view, r, (ptr float*)k, (ptr float*)v); break;        \
    case RDKV_F32 * 256 + 128: kernel<float, 128><<<(unsigned)blocks, kThreads, 0, cs>>>(view, r, (ptr float*)k, (ptr float*)v); break;      \
    case RDKV_BF16 * 256 + 64: kernel<__nv_bfloat16, 64><<<(unsigned)blocks, kThreads, 0, cs>>>(view, r, (ptr __nv_bfloat16*)k, (ptr __nv_bfloat16*)v); break; \
    default: kernel<__nv_bfloat16, 128><<<(unsigned)blocks, kThreads, 0, cs>>>(view, r, (ptr __nv_bfloat16*)k, (ptr __nv_bfloat16*)v);       \
  }

extern "C" rdkv_status rdkv_q4_write(const rdkv_q4_cache* cache, int32_t dtype, const void* k, const void* v,
                                     int64_t row_stride, const int32_t* row_start, int32_t max_rows, void* stream) {
  rdkv_status st = check_rows(cache, dtype, k, v, row_stride, max_rows);
  if (st != RDKV_OK) return st;
  if (max_rows == 0) return RDKV_OK;
  Rows r{row_stride, row_start, nullptr, max_rows, 0};
  int64_t blocks;
  st = grid_of(cache, &r, &blocks);
  if (st != RDKV_OK) return st;
  cudaStream_t cs = (cudaStream_t)stream;
  const View view = view_of(cache);
  RDKV_Q4_ROWS_LAUNCH(write_kernel, const)
  RDKV_CHECK_LAUNCH("4-bit cache write");
  return RDKV_OK;
}

extern "C" rdkv_status rdkv_q4_read(const rdkv_q4_cache* cache, int32_t dtype, void* k, void* v, int64_t row_stride,
                                    const int32_t* row_start, const int32_t* first, int32_t max_rows, void* stream) {
  rdkv_status st = check_rows(cache, dtype, k, v, row_stride, max_rows);
  if (st != RDKV_OK) return st;
  if (max_rows == 0) return RDKV_OK;
  Rows r{row_stride, row_start, first, max_rows, 0};
  int64_t blocks;
  st = grid_of(cache, &r, &blocks);
  if (st != RDKV_OK) return st;
  cudaStream_t cs = (cudaStream_t)stream;
  const View view = view_of(cache);
  RDKV_Q4_ROWS_LAUNCH(read_kernel, )
  RDKV_CHECK_LAUNCH("4-bit cache read");
  return RDKV_OK;
}

extern "C" rdkv_status rdkv_q4_status(const rdkv_q4_cache* cache, void* stream) {
  rdkv_status st = check_cache(cache);
  if (st != RDKV_OK) return st;
  cudaStream_t cs = (cudaStream_t)stream;
  int32_t code = 0;
  RDKV_TRY_CUDA(cudaMemcpyAsync(&code, cache->status, sizeof(code), cudaMemcpyDeviceToHost, cs), "status read");
  RDKV_TRY_CUDA(cudaStreamSynchronize(cs), "status read");
  if (code != 0) {
    RDKV_TRY_CUDA(cudaMemsetAsync(cache->status, 0, sizeof(code), cs), "status clear");
    set_error("the 4-bit cache's calls reported status %d on the device", code);
  }
  return (rdkv_status)code;
}
