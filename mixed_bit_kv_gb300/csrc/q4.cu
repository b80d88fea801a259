// The 4-bit paged cache: rows quantised as they are written (rdkv_q4_write) and read back
// (rdkv_q4_read), and the host checks that every rdkv_q4_* call makes.
#include <type_traits>

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

rdkv_status check_rows(const rdkv_q4_cache* c, int32_t dtype, const void* k, const void* v, int64_t rows, int64_t row_stride,
                       const int32_t* row_start, int32_t max_rows) {
  rdkv_status st = check_cache(c);
  if (st != RDKV_OK) return st;
  st = check_dtype(dtype);
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

rdkv_status check_queries(const rdkv_q4_cache* c, int32_t h_q, int32_t n_q) {
  rdkv_status st = check_cache(c);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(h_q >= 1 && h_q % c->h_kv == 0, RDKV_ERR_INVALID_ARG, "h_q=%d is not a multiple of h_kv=%d", h_q, c->h_kv);
  RDKV_REQUIRE(h_q / c->h_kv <= 8, RDKV_ERR_UNSUPPORTED, "group size %d > 8", h_q / c->h_kv);
  RDKV_REQUIRE(n_q >= 1, RDKV_ERR_INVALID_ARG, "n_q %d", n_q);
  RDKV_REQUIRE(n_q <= RDKV_Q4_MAX_QUERIES, RDKV_ERR_UNSUPPORTED, "n_q %d > %d", n_q, RDKV_Q4_MAX_QUERIES);
  // a counter each in the workspaces; also a grid's second size
  RDKV_REQUIRE((int64_t)c->batch * n_q * c->h_kv <= RDKV_Q4_COUNTER_BYTES / 4 - 1, RDKV_ERR_UNSUPPORTED,
               "more than 65,535 (sequence, query token, KV head) triples");
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
__device__ __forceinline__ Run find_run(const View& v, const Rows& r, int b, int run) {
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

__device__ __forceinline__ float2 wide2(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ float2 wide2(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ __half2 halves_of(__half a, __half b) { return __halves2half2(a, b); }
__device__ __forceinline__ __nv_bfloat162 halves_of(__nv_bfloat16 a, __nv_bfloat16 b) { return __halves2bfloat162(a, b); }

// Eight channels of one row as they lie in memory, in two runs of four that are `gap` channels apart.
template <typename T>
struct Raw {
  uint2 a, b;
};
template <>
struct Raw<float> {
  uint4 a, b;
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int gap) {
  using W = decltype(Raw<T>::a);
  return Raw<T>{fetch(reinterpret_cast<const W*>(p)), fetch(reinterpret_cast<const W*>(p + gap))};
}
__device__ __forceinline__ void widen(const Raw<__half>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&x)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}

// The smallest and the largest of eight values of four neighbouring lanes; a NaN takes no part (all NaN: not
// smallest <= largest).
__device__ __forceinline__ float2 extremes(const float (&x)[8]) {
  float mn = INFINITY, mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) mn = fminf(mn, x[i]), mx = fmaxf(mx, x[i]);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  return make_float2(mn, mx);
}
__device__ __forceinline__ float2 extremes_of(const Raw<float>& r, const float (&x)[8]) { return extremes(x); }
// 16-bit types: pairs at a time, the largest as the smallest of the negatives
template <typename T2>
__device__ __forceinline__ float2 extremes16(const uint32_t (&w)[4], T2 all) {
  auto as = [](uint32_t v) { return *reinterpret_cast<const T2*>(&v); };
  T2 mn = __hmin2(__hmin2(as(w[0]), as(w[1])), __hmin2(as(w[2]), as(w[3])));
  T2 mx = __hmax2(__hmax2(as(w[0]), as(w[1])), __hmax2(as(w[2]), as(w[3])));
  T2 both = halves_of(__hmin(mn.x, mn.y), __hneg(__hmax(mx.x, mx.y)));
  both = __hmin2(both, __shfl_xor_sync(0xffffffffu, both, 1));
  both = __hmin2(both, __shfl_xor_sync(0xffffffffu, both, 2));
  const float2 f = wide2(both);
  return make_float2(f.x, -f.y);
}
__device__ __forceinline__ float2 extremes_of(const Raw<__half>& r, const float (&)[8]) {
  return extremes16({r.a.x, r.a.y, r.b.x, r.b.y}, __half2());
}
__device__ __forceinline__ float2 extremes_of(const Raw<__nv_bfloat16>& r, const float (&)[8]) {
  return extremes16({r.a.x, r.a.y, r.b.x, r.b.y}, __nv_bfloat162());
}

// Codes (as whole floats) of eight channels whose group of 32 is spread over four neighbouring lanes, with
// the group's scale and zero (the quantiser of the pack, on values cut to the fp16 range; a NaN takes no
// part in min and max and gets code 0).
//   The fast way takes the quotients as products.  Range / 15 as range times fp32(1 / 15), within 2^-22 of the
// quotient: the fp16 scale is the same unless the product lies within 8 units of its last place of the middle
// of two fp16 values (or below fp16's normal range).  (x - zero) / scale as (x - zero) r, r within 2^-22 of
// 1 / scale: with every quotient of the group in (-0.49, 15.49), rounding gives the same code unless the
// product is within 2^-16 of a half-integer (the product and the quotient differ by less than 2^-18).  What fails a test, and groups that hold a NaN or values past
// fp16's range, goes the exact way.
struct Codes {
  float c[8];
  QParams p;
};
__device__ __noinline__ Codes quantise8_exact(float mn, float mx, float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                              float x7) {
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
  if (!(mn <= mx)) mn = mx = 0.0f;  // nothing but NaN
  mn = fminf(fmaxf(mn, -kHalfMax), kHalfMax), mx = fminf(fmaxf(mx, -kHalfMax), kHalfMax);
  Codes r;
  r.p = qparams(mn, mx, 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = x[i] > kHalfMax ? kHalfMax : x[i] < -kHalfMax ? -kHalfMax : x[i];
    const float t = __fdiv_rn(y - r.p.zero, r.p.scale);
    r.c[i] = r.p.scale == 0.0f ? 0.0f : fminf(fmaxf(rintf(t), 0.0f), 15.0f);  // a NaN: 0
  }
  return r;
}
__device__ __noinline__ float rounded_quotient(float d, float scale) { return fminf(fmaxf(rintf(__fdiv_rn(d, scale)), 0.0f), 15.0f); }
template <typename T>
__device__ __forceinline__ Codes quantise8(const Raw<T>& raw) {
  float x[8];
  widen(raw, x);
  float2 ex = extremes_of(raw, x);
  Codes r;
  r.p.zero_h = half_bits(ex.x);
  r.p.zero = __half2float(__ushort_as_half(r.p.zero_h));
  const float step = (ex.y - ex.x) * 0.066666670143604279f;
  r.p.scale_h = half_bits(step);
  r.p.scale = __half2float(__ushort_as_half(r.p.scale_h));
  const uint32_t below = (__float_as_uint(step) - 0xff8u) & 0x1fffu;  // 0 .. 16 next to the middle of two fp16 values
  float rs;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(r.p.scale));
  constexpr float kRound = 12582912.0f;  // 1.5 2^23: its last place is 1
  const float2 zero = make_float2(-r.p.zero, -r.p.zero), rs2 = make_float2(rs, rs), up = make_float2(kRound, kRound),
               down = make_float2(-kRound, -kRound);
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 d = add2f(make_float2(x[i], x[i + 1]), zero);
    const float2 c = add2f(fma2(d, rs2, up), down);
    const float2 e = fma2(d, rs2, make_float2(-c.x, -c.y));
    r.c[i] = c.x, r.c[i + 1] = c.y;
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(far) : "f"(fabsf(e.x)), "f"(fabsf(e.y)));
  }
  // (the comparisons are false for NaN and infinities)
  bool fine = (step >= 6.1035156e-5f) & (step < 8000.0f) & (below > 16u);
  if constexpr (!std::is_same<T, __half>::value) {  // fp16 rows: zero is the smallest value itself, none is too large
    fine &= ((ex.x - r.p.zero) * rs > -0.49f) & ((ex.y - r.p.zero) * rs < 15.49f) & (ex.x >= -kHalfMax) & (ex.y <= kHalfMax);
  }
  fine &= far == far;  // a NaN among the values
  if (!fine) {
    r = quantise8_exact(ex.x, ex.y, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
  } else if (far > 0.5f - 0.0000152587890625f) {
    // next to a half-integer: the quotient itself (fp16 rows meet exact ones in one of some ten warps)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = x[i] - r.p.zero;
      if (fabsf(fmaf(d, rs, -r.c[i])) > 0.5f - 0.0000152587890625f) r.c[i] = rounded_quotient(d, r.p.scale);
    }
  }
  return r;
}
// Four codes in 16 bits, the first lowest.
__device__ __forceinline__ uint32_t nibbles(float a, float b, float c, float d) {
  return __float_as_uint(fmaf(d, 4096.0f, fmaf(c, 256.0f, fmaf(b, 16.0f, a))) + 8388608.0f);  // the low 16 bits
}
__device__ __forceinline__ uint32_t low_halves(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x5410); }
// One block per (sequence, page that its rows touch, KV head), heads fastest: neighbouring blocks read
// neighbouring memory.  A thread has eight channels of a token pair: of K eight in a row (a code word of each
// token), of V the runs 4 q and 4 q + 16 (two words that hold both tokens), so that a warp's stores fill whole
// sectors.  Every load of a thread's kSteps pairs is under way before the first is used.  kThreads, kSteps:
// as few as the call's rows need (a decode step has one token a sequence: 3.8 us for 32 sequences of 8 heads
// with 32 threads a block, 9.8 with 256).
//   Bound: 47 us for 32,768 rows of 8 heads at D = 128 in fp16 (134 MB read, 42 MB written: 3.7 TB/s).  A warp runs
// 1,180 instructions for both halves of its eight rows; the issue slots are 71 % used, the ALU 52 %, DRAM 46 %, and
// warps wait for their rows as often as for one another (22 of 64 warps fit at 80 registers).  As one division a value it took 94 us; with the
// tests as short-circuit conditions 76; with an exact way for the whole group on a near half 54.
template <typename T, int D, int kThreads, int kSteps>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 1) write_kernel(View v, Rows r, const T* k, const T* vv) {
  using L = Layout<D>;
  constexpr int kLanes = D / 8, kPairs = kThreads / kLanes, kWarps = kThreads / 32, NG = L::NG;
  __shared__ __half2 lo_s[kWarps][D / 2], hi_s[kWarps][D / 2];
  after_previous();
  const int h = blockIdx.x % v.h_kv, u = blockIdx.x / v.h_kv, run = u % r.runs, b = u / r.runs;
  const Run w = find_run<true>(v, r, b, run);
  if (w.page < 0) return;
  uint8_t* page = v.pages + ((int64_t)w.page * v.h_kv + h) * L::kBytes;
  const int l = threadIdx.x % kLanes, grp = l / 4, q = l % 4, first = w.s0 / 2 + threadIdx.x / kLanes;
  __half2 lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) lo[i] = __float2half2_rn(INFINITY), hi[i] = __float2half2_rn(-INFINITY);
  Raw<T> kr[kSteps][2], vr[kSteps][2];
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // a token outside the run: the run's nearest, whose codes go nowhere
      const int s = min(max(2 * (first + i * kPairs) + j, w.s0), w.s1 - 1);
      const int64_t at = (w.row + s - w.s0) * r.stride + (int64_t)h * D + 32 * grp;
      kr[i][j] = load_raw(k + at + 8 * q, 4);
      vr[i][j] = load_raw(vv + at + 4 * q, 16);
    }
  auto pairs = [&](auto full) {
    constexpr bool kFull = decltype(full)::value;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int pair = first + i * kPairs, m = pair * NG + grp;
      const bool in[2] = {kFull || (2 * pair >= w.s0 && 2 * pair < w.s1), kFull || (2 * pair + 1 >= w.s0 && 2 * pair + 1 < w.s1)};
      if (!kFull && !__any_sync(0xffffffffu, in[0] || in[1])) continue;
      uint32_t word[2][2];
      QParams pp[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Codes c = quantise8(kr[i][j]);
        pp[j] = c.p;
        if (in[j]) {
          reinterpret_cast<uint32_t*>(page + L::kKCodes)[((2 * pair + j) * 4 + q) * NG + grp] =
              low_halves(nibbles(c.c[0], c.c[2], c.c[4], c.c[6]), nibbles(c.c[1], c.c[3], c.c[5], c.c[7]));
          if (q == 0) reinterpret_cast<uint16_t*>(page + L::kKZeros)[(2 * pair + j) * NG + grp] = c.p.zero_h;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = fma2(make_float2(c.p.scale, c.p.scale), make_float2(c.c[2 * e], c.c[2 * e + 1]), make_float2(c.p.zero, c.p.zero));
            const uint32_t zw = cut_half2(y.x, y.y);
          const __half2 z = *reinterpret_cast<const __half2*>(&zw);
            lo[e] = __hmin2(lo[e], z), hi[e] = __hmax2(hi[e], z);
          }
        }
      }
      auto store_pair = [&](int at, int index, uint32_t even, uint32_t odd) {
        if (in[0] && in[1]) reinterpret_cast<uint32_t*>(page + at)[index] = low_halves(even, odd);
        else if (in[0]) reinterpret_cast<uint16_t*>(page + at)[2 * index] = (uint16_t)even;
        else if (in[1]) reinterpret_cast<uint16_t*>(page + at)[2 * index + 1] = (uint16_t)odd;
      };
      if (q == 0) store_pair(L::kKScales, m, pp[0].scale_h, pp[1].scale_h);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Codes c = quantise8(vr[i][j]);
        pp[j] = c.p;
        word[j][0] = nibbles(c.c[0], c.c[1], c.c[2], c.c[3]), word[j][1] = nibbles(c.c[4], c.c[5], c.c[6], c.c[7]);
      }
      store_pair(L::kVCodes, (pair * 8 + q) * NG + grp, word[0][0], word[1][0]);
      store_pair(L::kVCodes, (pair * 8 + q + 4) * NG + grp, word[0][1], word[1][1]);
      if (q == 0) {
        store_pair(L::kVScales, m, pp[0].scale_h, pp[1].scale_h);
        store_pair(L::kVZeros, m, pp[0].zero_h, pp[1].zero_h);
      }
    }
  };
  if (w.s0 == 0 && w.s1 == kPage) pairs(std::true_type());
  else pairs(std::false_type());
  if (!v.bounds) return;
  // the page's bounds: the pairs of a warp, the block's warps, and what the page held before
#pragma unroll
  for (int d = kLanes; d < 32; d <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = __hmin2(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], d));
      hi[e] = __hmax2(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], d));
    }
  if (threadIdx.x % 32 < kLanes) {
#pragma unroll
    for (int e = 0; e < 4; ++e) lo_s[threadIdx.x / 32][4 * l + e] = lo[e], hi_s[threadIdx.x / 32][4 * l + e] = hi[e];
  }
  __syncthreads();
  __half2* out = reinterpret_cast<__half2*>(v.bounds + ((int64_t)w.page * v.h_kv + h) * 2 * D);
#pragma unroll
  for (int c = threadIdx.x; c < D; c += kThreads) {
    const int side = c / (D / 2), e = c % (D / 2);
    __half2 m = side ? hi_s[0][e] : lo_s[0][e];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) m = side ? __hmax2(m, hi_s[i][e]) : __hmin2(m, lo_s[i][e]);
    if (w.s0 > 0) m = side ? __hmax2(m, out[c]) : __hmin2(m, out[c]);
    out[c] = m;
  }
}

// The values of a code word's four pairs (codes at bits 0 and 16, 4 and 20, 8 and 24, 12 and 28): a code at bit
// p < 8 of a half word is the fp16 subnormal code 2^(p - 24), exactly, and so is its product with a scale.
// scale: of the low and the high halves, times 2^24.
__device__ __forceinline__ void word_values(uint32_t w, float2 scale, float2 zero, float2 (&x)[4]) {
  const float2 less = make_float2(scale.x * 0.0625f, scale.y * 0.0625f);
  const Pairs c = code_pairs(w);
  const uint32_t p[4] = {c.a, c.b, c.c, c.d};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = fma2(__half22float2(*reinterpret_cast<const __half2*>(&p[i])), i & 1 ? less : scale, zero);
}
__device__ __forceinline__ float half_of(uint32_t w, int i) { return __half2float(__ushort_as_half((uint16_t)(w >> (16 * i)))); }

// The same blocks the other way: eight channels in a row of a token pair a thread.  Bound: 190 us for eight 32K
// caches of 8 heads in fp16 (235 MB read, 866 MB written: 5.8 TB/s, 85 % of the measured copy); 200 us with
// integer conversions, whose shifts and clamps filled the ALU.
template <typename T, int D, int kThreads, int kSteps>
__global__ void __launch_bounds__(kThreads) read_kernel(View v, Rows r, T* k, T* vv) {
  using L = Layout<D>;
  constexpr int kLanes = D / 8, kPairs = kThreads / kLanes, NG = L::NG;
  after_previous();
  const int h = blockIdx.x % v.h_kv, u = blockIdx.x / v.h_kv, run = u % r.runs, b = u / r.runs;
  const Run w = find_run<false>(v, r, b, run);
  if (w.page < 0) return;
  const uint8_t* page = v.pages + ((int64_t)w.page * v.h_kv + h) * L::kBytes;
  const int l = threadIdx.x % kLanes, grp = l / 4, q = l % 4, first = w.s0 / 2 + threadIdx.x / kLanes;
  auto word = [&](int at, int index) { return fetch(reinterpret_cast<const uint32_t*>(page + at) + index); };
  uint32_t kc[kSteps][2], vc[kSteps][2], ks[kSteps], vs[kSteps], vz[kSteps];
  uint16_t kz[kSteps][2];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int pair = min(first + i * kPairs, kPage / 2 - 1), m = pair * NG + grp;  // past the run: not used
    ks[i] = word(L::kKScales, m), vs[i] = word(L::kVScales, m), vz[i] = word(L::kVZeros, m);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      kc[i][j] = word(L::kKCodes, ((2 * pair + j) * 4 + q) * NG + grp);
      vc[i][j] = word(L::kVCodes, (pair * 8 + 2 * q + j) * NG + grp);
      kz[i][j] = fetch(reinterpret_cast<const uint16_t*>(page + L::kKZeros) + (2 * pair + j) * NG + grp);
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    constexpr float kUnit = 16777216.0f;
    float2 v0[4], v1[4];  // channels 8 l .. + 3 and + 4 .. 7 of both tokens
    const float2 vscale = make_float2(half_of(vs[i], 0) * kUnit, half_of(vs[i], 1) * kUnit), vzero = make_float2(half_of(vz[i], 0), half_of(vz[i], 1));
    word_values(vc[i][0], vscale, vzero, v0);
    word_values(vc[i][1], vscale, vzero, v1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int s = 2 * (first + i * kPairs) + j;
      if (s < w.s0 || s >= w.s1) continue;
      const int64_t at = (w.row + s - w.s0) * r.stride + (int64_t)h * D + 8 * l;
      const float sc = half_of(ks[i], j) * kUnit, z = half_of(kz[i][j], 0);
      float2 x[4];
      word_values(kc[i][j], make_float2(sc, sc), make_float2(z, z), x);
      Eight<T>::store(k + at, {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y});
      if (j == 0) Eight<T>::store(vv + at, {v0[0].x, v0[1].x, v0[2].x, v0[3].x, v1[0].x, v1[1].x, v1[2].x, v1[3].x});
      else Eight<T>::store(vv + at, {v0[0].y, v0[1].y, v0[2].y, v0[3].y, v1[0].y, v1[1].y, v1[2].y, v1[3].y});
    }
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

namespace {
// Threads and steps that cover the token pairs n rows can touch in a page.
template <typename T, int D, int kThreads, int kSteps>
constexpr bool covers(int n) {
  return std::min(kPage / 2, n / 2 + 1) <= kThreads / (D / 8) * kSteps;
}
template <typename T, int D>
cudaError_t launch_write(unsigned blocks, const View& view, const Rows& r, const void* k, const void* v, cudaStream_t cs) {
  const T *kt = static_cast<const T*>(k), *vt = static_cast<const T*>(v);
  if (covers<T, D, 32, 1>(r.max_rows)) return launch_after(write_kernel<T, D, 32, 1>, dim3(blocks), 32, 0, cs, view, r, kt, vt);
  if (covers<T, D, 128, 1>(r.max_rows)) return launch_after(write_kernel<T, D, 128, 1>, dim3(blocks), 128, 0, cs, view, r, kt, vt);
  return launch_after(write_kernel<T, D, 256, D / 64>, dim3(blocks), 256, 0, cs, view, r, kt, vt);
}
template <typename T, int D>
cudaError_t launch_read(unsigned blocks, const View& view, const Rows& r, void* k, void* v, cudaStream_t cs) {
  T *kt = static_cast<T*>(k), *vt = static_cast<T*>(v);
  if (covers<T, D, 32, 1>(r.max_rows)) return launch_after(read_kernel<T, D, 32, 1>, dim3(blocks), 32, 0, cs, view, r, kt, vt);
  return launch_after(read_kernel<T, D, 256, D / 64>, dim3(blocks), 256, 0, cs, view, r, kt, vt);
}
}  // namespace

extern "C" rdkv_status rdkv_q4_write(const rdkv_q4_cache* cache, int32_t dtype, const void* k, const void* v,
                                     int64_t rows, int64_t row_stride, const int32_t* row_start, int32_t max_rows, void* stream) {
  rdkv_status st = check_rows(cache, dtype, k, v, rows, row_stride, row_start, max_rows);
  if (st != RDKV_OK) return st;
  if (max_rows == 0) return RDKV_OK;
  Rows r{rows, row_stride, row_start, nullptr, max_rows, 0};
  int64_t blocks;
  st = grid_of(cache, &r, &blocks);
  if (st != RDKV_OK) return st;
  cudaStream_t cs = (cudaStream_t)stream;
  const View view = view_of(cache);
  const bool wide = cache->head_dim == 128;
  cudaError_t e;
  if (dtype == RDKV_F16) e = (wide ? launch_write<__half, 128> : launch_write<__half, 64>)((unsigned)blocks, view, r, k, v, cs);
  else if (dtype == RDKV_F32) e = (wide ? launch_write<float, 128> : launch_write<float, 64>)((unsigned)blocks, view, r, k, v, cs);
  else e = (wide ? launch_write<__nv_bfloat16, 128> : launch_write<__nv_bfloat16, 64>)((unsigned)blocks, view, r, k, v, cs);
  RDKV_TRY_CUDA(e, "4-bit cache write");
  count_launch();
  return RDKV_OK;
}

extern "C" rdkv_status rdkv_q4_read(const rdkv_q4_cache* cache, int32_t dtype, void* k, void* v, int64_t rows,
                                    int64_t row_stride, const int32_t* row_start, const int32_t* first, int32_t max_rows, void* stream) {
  rdkv_status st = check_rows(cache, dtype, k, v, rows, row_stride, row_start, max_rows);
  if (st != RDKV_OK) return st;
  if (max_rows == 0) return RDKV_OK;
  Rows r{rows, row_stride, row_start, first, max_rows, 0};
  int64_t blocks;
  st = grid_of(cache, &r, &blocks);
  if (st != RDKV_OK) return st;
  cudaStream_t cs = (cudaStream_t)stream;
  const View view = view_of(cache);
  const bool wide = cache->head_dim == 128;
  cudaError_t e;
  if (dtype == RDKV_F16) e = (wide ? launch_read<__half, 128> : launch_read<__half, 64>)((unsigned)blocks, view, r, k, v, cs);
  else if (dtype == RDKV_F32) e = (wide ? launch_read<float, 128> : launch_read<float, 64>)((unsigned)blocks, view, r, k, v, cs);
  else e = (wide ? launch_read<__nv_bfloat16, 128> : launch_read<__nv_bfloat16, 64>)((unsigned)blocks, view, r, k, v, cs);
  RDKV_TRY_CUDA(e, "4-bit cache read");
  count_launch();
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
