// The 8-bit paged cache: rows quantised as they are written (rdkv_q8_write) and read back (rdkv_q8_read), and the
// host checks that every rdkv_q8_* call makes.
#include <type_traits>

#include "q8.cuh"

namespace rdkv {
namespace q8 {

// ---------------------------------------------------------------- host checks
rdkv_status check_cache(const rdkv_q8_cache* c) {
  const rdkv_status st = check_pool(c);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(c->scales, RDKV_ERR_INVALID_ARG, "NULL pointer in the cache");
  RDKV_REQUIRE((uintptr_t)c->pages % 16 == 0 && (uintptr_t)c->scales % 8 == 0, RDKV_ERR_INVALID_ARG,
               "pages must be 16-byte aligned, scales 8-byte aligned");
  return RDKV_OK;
}

rdkv_status check_mass(const rdkv_q8_cache* c, const float* mass, int64_t mass_stride) {
  RDKV_REQUIRE((uintptr_t)mass % 8 == 0 && mass_stride % 2 == 0, RDKV_ERR_INVALID_ARG, "mass must be 8-byte aligned (mass_stride %lld)",
               (long long)mass_stride);
  RDKV_REQUIRE(mass_stride >= (int64_t)c->page_stride * kPage, RDKV_ERR_INVALID_ARG, "mass_stride %lld < 64 * page_stride",
               (long long)mass_stride);
  return RDKV_OK;
}

// ---------------------------------------------------------------- rows
// Eight channels of one row as they lie in memory.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = fetch(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ void widen(const Raw<__half>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(w[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&x)[8]) {
  const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}
// The largest magnitude of eight channels and top (as the bits of a number that is no less than 0); kNan: a NaN, if there is one,
// else it takes no part.
template <bool kNan>
__device__ __forceinline__ float larger(float a, float b) {
  float d;
  if constexpr (kNan) asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  else d = fmaxf(a, b);
  return d;
}
template <bool kNan>
__device__ __forceinline__ __half2 larger(__half2 a, __half2 b) {
  return kNan ? __hmax2_nan(a, b) : __hmax2(a, b);
}
template <bool kNan>
__device__ __forceinline__ __nv_bfloat162 larger(__nv_bfloat162 a, __nv_bfloat162 b) {
  return kNan ? __hmax2_nan(a, b) : __hmax2(a, b);
}
template <bool kNan>
__device__ __forceinline__ float largest(const Raw<float>& r, float top) {
  float x[8];
  widen(r, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) top = larger<kNan>(top, fabsf(x[i]));
  return top;
}
template <bool kNan, class T2>
__device__ __forceinline__ float largest16(const uint4& w, float top) {
  auto as = [](uint32_t v) { return __habs2(*reinterpret_cast<const T2*>(&v)); };
  const T2 m = larger<kNan>(larger<kNan>(as(w.x), as(w.y)), larger<kNan>(as(w.z), as(w.w)));
  return larger<kNan>(top, larger<kNan>((float)m.x, (float)m.y));
}
template <bool kNan>
__device__ __forceinline__ float largest(const Raw<__half>& r, float top) {
  return largest16<kNan, __half2>(r.w[0], top);
}
template <bool kNan>
__device__ __forceinline__ float largest(const Raw<__nv_bfloat16>& r, float top) {
  return largest16<kNan, __nv_bfloat162>(r.w[0], top);
}

// Eight channels' codes, and those of a token pair side by side, in the scale 2^e.  nan: there may be NaN among them, which become 0.
__device__ __forceinline__ uint32_t clean(uint32_t w, bool nan) { return nan ? without_nan(w) : w; }
template <typename T>
struct Coder {
  float f;
  bool nan;
  __device__ __forceinline__ Coder(int e, bool nan) : f(two_to(-e)), nan(nan) {}
  __device__ __forceinline__ uint2 eight(const Raw<T>& r) const {
    float x[8];
    widen(r, x);
    return make_uint2(clean(codes4(x[0] * f, x[1] * f, x[2] * f, x[3] * f), nan), clean(codes4(x[4] * f, x[5] * f, x[6] * f, x[7] * f), nan));
  }
  __device__ __forceinline__ uint4 pairs(const Raw<T>& a, const Raw<T>& b) const {
    float x[8], y[8];
    widen(a, x);
    widen(b, y);
    uint32_t c[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) c[m] = clean(codes4(x[2 * m] * f, y[2 * m] * f, x[2 * m + 1] * f, y[2 * m + 1] * f), nan);
    return make_uint4(c[0], c[1], c[2], c[3]);
  }
};
// fp16 rows stay fp16: times 2^-e, two at a time, is exact down to 2^-14 and within 2^-25 below, where every code's middle to the next
// (2^-10 and up) is far.  2^-e past 2^15, of the smallest scales, in two factors.
template <>
struct Coder<__half> {
  __half2 f, more;
  bool twice, nan;
  __device__ __forceinline__ Coder(int e, bool nan)
      : f(__float2half2_rn(two_to(min(-e, 15)))), more(__float2half2_rn(two_to(max(-e - 15, 0)))), twice(e < -15), nan(nan) {}
  __device__ __forceinline__ uint32_t two(uint32_t w) const {
    __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&w), f);
    if (twice) x = __hmul2(x, more);
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
    return d;
  }
  __device__ __forceinline__ uint32_t four(uint32_t a, uint32_t b) const { return clean(two(a) | two(b) << 16, nan); }
  __device__ __forceinline__ uint2 eight(const Raw<__half>& r) const { return make_uint2(four(r.w[0].x, r.w[0].y), four(r.w[0].z, r.w[0].w)); }
  __device__ __forceinline__ uint4 pairs(const Raw<__half>& a, const Raw<__half>& b) const {
    auto both = [&](uint32_t x, uint32_t y) { return four(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632)); };
    return make_uint4(both(a.w[0].x, b.w[0].x), both(a.w[0].y, b.w[0].y), both(a.w[0].z, b.w[0].z), both(a.w[0].w, b.w[0].w));
  }
};

constexpr int kWriteBlocks = 4;  // of 256 threads an SM, 16-bit rows
// One block per (sequence, page that its rows touch, KV head), heads fastest.  A thread takes eight channels of a
// token of the keys (8 bytes of codes) and eight channels of a token pair of the values (16 bytes), both in the
// order of the page, so that a warp stores 256 and 512 bytes in a row; of the rows it then loads whole 128-byte
// lines.  All rows are held in registers between their largest magnitude, which the block has to know first, and
// their codes.  Where the page was begun before and the new rows raise a scale, the block takes the earlier codes
// in it too (one append in some dozens).
//   Bound: 34 us for 32,768 rows of 8 heads at D = 128 in fp16 (134 MB read, 67 MB written: 5.9 TB/s, 87 % of the measured copy);
// 2.8 us for one row of 32 sequences.  With rows widened to fp32, a test for NaN of every code and two blocks an SM 45 us: the
// ALU was half used and the registers held too little under way.  The other types still are widened: 35.6 us in bf16 (the same bytes; 76
// bytes a thread are spilled at four blocks an SM), 53.7 in fp32 (336 MB: 6.2 TB/s, two blocks an SM).
template <typename T, int D, int kThreads, int kKeys, int kValues>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? (sizeof(T) == 2 ? kWriteBlocks : 2) : 1) write_kernel(View v, Rows r, const T* k, const T* vv) {
  using L = Layout<D>;
  constexpr int kS = L::kSides, kWarps = kThreads / 32;
  __shared__ uint32_t top_s[2][kWarps];
  after_previous();
  const int h = blockIdx.x % v.h_kv, u = blockIdx.x / v.h_kv, run = u % r.runs, b = u / r.runs;
  const Run w = find_run<true>(v, r, b, run);
  if (w.page < 0) return;
  const int64_t at = (int64_t)w.page * v.h_kv + h;
  uint8_t* page = v.pages + at * L::kBytes;
  const int tid = threadIdx.x, lane = tid % 32;
  const uint2 was = fetch(reinterpret_cast<const uint2*>(v.scales + at * 2));
  // this thread's units, in the order of the page; a token outside the run: the run's nearest
  auto key_unit = [&](int i, int& t, int& j, int& c) {
    const int n = tid + i * kThreads;
    c = n % 8, j = n / 16 % kS, t = w.s0 / 2 * 2 + n / (16 * kS) * 2 + n / 8 % 2;
  };
  auto value_unit = [&](int i, int& p, int& j, int& g) {
    const int n = tid + i * kThreads;
    p = w.s0 / 8 * 4 + n / (32 * kS) * 4 + n % 4, j = n / 32 % kS, g = n % 32 / 4;
  };
  auto row_at = [&](int t) { return (w.row + min(max(t, w.s0), w.s1 - 1) - w.s0) * r.stride + (int64_t)h * D; };
  Raw<T> kr[kKeys], vr[kValues][2];
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    int t, j, c;
    key_unit(i, t, j, c);
    kr[i] = load_raw(k + row_at(t) + 64 * j + 8 * c);
  }
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    int p, j, g;
    value_unit(i, p, j, g);
    vr[i][0] = load_raw(vv + row_at(2 * p) + 64 * j + 8 * g);
    vr[i][1] = load_raw(vv + row_at(2 * p + 1) + 64 * j + 8 * g);
  }
  // the largest magnitudes (a token taken twice counts as once), first as if there were no NaN: the bits of one are larger than any
  // number's
  uint32_t all[2];
  auto find = [&](auto nan) {
    constexpr bool kNan = decltype(nan)::value;
    float top[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kKeys; ++i) top[0] = largest<kNan>(kr[i], top[0]);
#pragma unroll
    for (int i = 0; i < kValues; ++i) top[1] = largest<kNan>(vr[i][1], largest<kNan>(vr[i][0], top[1]));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(top[s]));
      if (lane == 0) top_s[s][tid / 32] = m;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      all[s] = top_s[s][0];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) all[s] = max(all[s], top_s[s][i]);
    }
  };
  find(std::true_type());
  const bool nan = max(all[0], all[1]) > 0x7f800000u;
  if (nan) {
    __syncthreads();
    find(std::false_type());
  }
  int e[2], old[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    e[s] = exponent_for(__uint_as_float(all[s]));
    old[s] = min(max(exponent(__uint_as_float(s ? was.y : was.x)), kLowExp), kHighExp);
    if (w.s0 > 0) e[s] = max(e[s], old[s]);
  }
  if (tid == 0) *reinterpret_cast<float2*>(v.scales + at * 2) = make_float2(two_to(e[0]), two_to(e[1]));
  const float again = two_to(old[1] - e[1]);
  const Coder<T> key_codes(e[0], nan), value_codes(e[1], nan);
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    int t, j, c;
    key_unit(i, t, j, c);
    if (t < w.s0 || t >= w.s1) continue;
    *reinterpret_cast<uint2*>(page + L::key_at(t, j, c)) = key_codes.eight(kr[i]);
  }
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    int p, j, g;
    value_unit(i, p, j, g);
    const bool in0 = 2 * p >= w.s0 && 2 * p < w.s1, in1 = 2 * p + 1 >= w.s0 && 2 * p + 1 < w.s1;
    if (!in0 && !in1) continue;
    uint4* to = reinterpret_cast<uint4*>(page + L::kHalf + L::value_at(p, j, g));
    uint4 c = value_codes.pairs(vr[i][0], vr[i][1]);
    if (!(in0 && in1)) {  // the pair's other token: an earlier one, or one that holds nothing yet
      uint4 o = fetch(to);
      const uint32_t mine = in0 ? 0x00ff00ffu : 0xff00ff00u;
      if (in1 && e[1] != old[1]) o = make_uint4(rescaled(o.x, again), rescaled(o.y, again), rescaled(o.z, again), rescaled(o.w, again));
      c = make_uint4((c.x & mine) | (o.x & ~mine), (c.y & mine) | (o.y & ~mine), (c.z & mine) | (o.z & ~mine), (c.w & mine) | (o.w & ~mine));
    }
    *to = c;
  }
  // the earlier rows in the new scale
  if (w.s0 > 0 && e[0] != old[0]) {
    const float f = two_to(old[0] - e[0]);
    for (int n = tid; n < w.s0 * (D / 8); n += kThreads) {
      uint2* to = reinterpret_cast<uint2*>(page + L::key_at(n / (D / 8), n / 8 % kS, n % 8));
      const uint2 c = fetch(to);
      *to = make_uint2(rescaled(c.x, f), rescaled(c.y, f));
    }
  }
  if (w.s0 > 1 && e[1] != old[1]) {
    for (int n = tid; n < w.s0 / 2 * (D / 8); n += kThreads) {
      uint4* to = reinterpret_cast<uint4*>(page + L::kHalf + L::value_at(n / (D / 8), n / 8 % kS, n % 8));
      const uint4 c = fetch(to);
      *to = make_uint4(rescaled(c.x, again), rescaled(c.y, again), rescaled(c.z, again), rescaled(c.w, again));
    }
  }
}

// The same units the other way.  Bound: HBM, 32 us for those rows back in fp16 or bf16 (6.3 TB/s, 92 % of the measured copy), 67.5 in fp32
// (336 MB: 5.0 TB/s; the reason was not looked for).
template <typename T, int D, int kThreads, int kKeys, int kValues>
__global__ void __launch_bounds__(kThreads) read_kernel(View v, Rows r, T* k, T* vv) {
  using L = Layout<D>;
  constexpr int kS = L::kSides;
  after_previous();
  const int h = blockIdx.x % v.h_kv, u = blockIdx.x / v.h_kv, run = u % r.runs, b = u / r.runs;
  const Run w = find_run<false>(v, r, b, run);
  if (w.page < 0) return;
  const int64_t at = (int64_t)w.page * v.h_kv + h;
  const uint8_t* page = v.pages + at * L::kBytes;
  const int tid = threadIdx.x;
  const uint2 sc = fetch(reinterpret_cast<const uint2*>(v.scales + at * 2));
  uint2 kc[kKeys];
  uint4 vc[kValues];
  // (units past the run's last page token: the page's last, not used)
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int n = tid + i * kThreads, t = w.s0 / 2 * 2 + n / (16 * kS) * 2 + n / 8 % 2;
    kc[i] = fetch(reinterpret_cast<const uint2*>(page + L::key_at(min(t, kPage - 1), n / 16 % kS, n % 8)));
  }
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    const int n = tid + i * kThreads, p = w.s0 / 8 * 4 + n / (32 * kS) * 4 + n % 4;
    vc[i] = fetch(reinterpret_cast<const uint4*>(page + L::kHalf + L::value_at(min(p, kPage / 2 - 1), n / 32 % kS, n % 32 / 4)));
  }
  const float ks = __uint_as_float(sc.x), vs = __uint_as_float(sc.y);
  auto out_at = [&](int t) { return (w.row + t - w.s0) * r.stride + (int64_t)h * D; };
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int n = tid + i * kThreads, t = w.s0 / 2 * 2 + n / (16 * kS) * 2 + n / 8 % 2;
    if (t < w.s0 || t >= w.s1) continue;
    float x[4], y[4];
    values4(kc[i].x, x);
    values4(kc[i].y, y);
    Eight<T>::store(k + out_at(t) + 64 * (n / 16 % kS) + 8 * (n % 8),
                    {x[0] * ks, x[1] * ks, x[2] * ks, x[3] * ks, y[0] * ks, y[1] * ks, y[2] * ks, y[3] * ks});
  }
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    const int n = tid + i * kThreads, p = w.s0 / 8 * 4 + n / (32 * kS) * 4 + n % 4, ch = 64 * (n / 32 % kS) + 8 * (n % 32 / 4);
    const uint32_t c[4] = {vc[i].x, vc[i].y, vc[i].z, vc[i].w};
    float x[2][8];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float y[4];
      values4(c[m], y);
      x[0][2 * m] = y[0] * vs, x[1][2 * m] = y[1] * vs, x[0][2 * m + 1] = y[2] * vs, x[1][2 * m + 1] = y[3] * vs;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (2 * p + s >= w.s0 && 2 * p + s < w.s1) Eight<T>::store(vv + out_at(2 * p + s) + ch, x[s]);
  }
}

// Threads and units a thread that cover what n rows can touch of a page: n / 2 + 1 token pairs of keys, (n + 6) / 8 + 1
// runs of eight tokens of values.
template <int D, int kThreads, int kKeys, int kValues>
constexpr bool covers(int n) {
  return std::min(kPage / 2, n / 2 + 1) * (16 * D / 64) <= kThreads * kKeys &&
         std::min(kPage / 8, (n + 6) / 8 + 1) * (32 * D / 64) <= kThreads * kValues;
}
template <typename T, int D>
cudaError_t launch_write(unsigned blocks, const View& view, const Rows& r, const void* k, const void* v, cudaStream_t cs) {
  const T *kt = static_cast<const T*>(k), *vt = static_cast<const T*>(v);
  constexpr int S = D / 64;
  static_assert(covers<D, 256, 2 * S, S>(kPage), "a whole page");
  if (covers<D, 32, 1, S>(r.max_rows)) return launch_after(write_kernel<T, D, 32, 1, S>, dim3(blocks), 32, 0, cs, view, r, kt, vt);
  if (covers<D, 128, S, 1>(r.max_rows)) return launch_after(write_kernel<T, D, 128, S, 1>, dim3(blocks), 128, 0, cs, view, r, kt, vt);
  return launch_after(write_kernel<T, D, 256, 2 * S, S>, dim3(blocks), 256, 0, cs, view, r, kt, vt);
}
template <typename T, int D>
cudaError_t launch_read(unsigned blocks, const View& view, const Rows& r, void* k, void* v, cudaStream_t cs) {
  T *kt = static_cast<T*>(k), *vt = static_cast<T*>(v);
  constexpr int S = D / 64;
  if (covers<D, 128, S, 1>(r.max_rows)) return launch_after(read_kernel<T, D, 128, S, 1>, dim3(blocks), 128, 0, cs, view, r, kt, vt);
  return launch_after(read_kernel<T, D, 256, 2 * S, S>, dim3(blocks), 256, 0, cs, view, r, kt, vt);
}

}  // namespace q8
}  // namespace rdkv

using namespace rdkv;
using namespace rdkv::q8;

extern "C" size_t rdkv_q8_page_bytes(int32_t head_dim) {
  return head_dim == 128 ? Layout<128>::kBytes : head_dim == 64 ? Layout<64>::kBytes : 0;
}

extern "C" rdkv_status rdkv_q8_write(const rdkv_q8_cache* cache, int32_t dtype, const void* k, const void* v,
                                     int64_t rows, int64_t row_stride, const int32_t* row_start, int32_t max_rows, void* stream) {
  rdkv_status st = check_cache(cache);
  if (st == RDKV_OK) st = check_rows_of(cache, dtype, k, v, rows, row_stride, row_start, max_rows);
  if (st != RDKV_OK || max_rows == 0) return st;
  Rows r{rows, row_stride, row_start, nullptr, max_rows, 0};
  int64_t blocks;
  st = grid_of(cache, &r, &blocks);
  if (st != RDKV_OK) return st;
  const bool wide = cache->head_dim == 128;
  auto launch = dtype == RDKV_F16   ? (wide ? launch_write<__half, 128> : launch_write<__half, 64>)
                : dtype == RDKV_F32 ? (wide ? launch_write<float, 128> : launch_write<float, 64>)
                                    : (wide ? launch_write<__nv_bfloat16, 128> : launch_write<__nv_bfloat16, 64>);
  RDKV_TRY_CUDA(launch((unsigned)blocks, q8::view_of(cache), r, k, v, (cudaStream_t)stream), "8-bit cache write");
  count_launch();
  return RDKV_OK;
}

extern "C" rdkv_status rdkv_q8_read(const rdkv_q8_cache* cache, int32_t dtype, void* k, void* v, int64_t rows,
                                    int64_t row_stride, const int32_t* row_start, const int32_t* first, int32_t max_rows, void* stream) {
  rdkv_status st = check_cache(cache);
  if (st == RDKV_OK) st = check_rows_of(cache, dtype, k, v, rows, row_stride, row_start, max_rows);
  if (st != RDKV_OK || max_rows == 0) return st;
  Rows r{rows, row_stride, row_start, first, max_rows, 0};
  int64_t blocks;
  st = grid_of(cache, &r, &blocks);
  if (st != RDKV_OK) return st;
  const bool wide = cache->head_dim == 128;
  auto launch = dtype == RDKV_F16   ? (wide ? launch_read<__half, 128> : launch_read<__half, 64>)
                : dtype == RDKV_F32 ? (wide ? launch_read<float, 128> : launch_read<float, 64>)
                                    : (wide ? launch_read<__nv_bfloat16, 128> : launch_read<__nv_bfloat16, 64>);
  RDKV_TRY_CUDA(launch((unsigned)blocks, q8::view_of(cache), r, k, v, (cudaStream_t)stream), "8-bit cache read");
  count_launch();
  return RDKV_OK;
}

extern "C" rdkv_status rdkv_q8_status(const rdkv_q8_cache* cache, void* stream) {
  rdkv_status st = check_cache(cache);
  if (st != RDKV_OK) return st;
  cudaStream_t cs = (cudaStream_t)stream;
  int32_t code = 0;
  RDKV_TRY_CUDA(cudaMemcpyAsync(&code, cache->status, sizeof(code), cudaMemcpyDeviceToHost, cs), "status read");
  RDKV_TRY_CUDA(cudaStreamSynchronize(cs), "status read");
  if (code != 0) {
    RDKV_TRY_CUDA(cudaMemsetAsync(cache->status, 0, sizeof(code), cs), "status clear");
    set_error("the 8-bit cache's calls reported status %d on the device", code);
  }
  return (rdkv_status)code;
}
