// Page selection of the 4-bit paged cache (rdkv_q4_select).
//
//   score(page) = max over the G query heads of sum_c max(q_c lo_c, q_c hi_c)
//               = max over heads of (max(q, 0) . hi + min(q, 0) . lo)
//
// The blocks of a row (sequence, query token, KV head) take the sums as tensor-core products (pages on M, the
// group's heads on N, the 2 D bounds on K), each within eps of the exact sum.  The row's last block to finish
// then finds an interval around the n-th best score, takes what lies above it by more than the error, and
// sums only the pages within the error again, to twice fp32's precision, so that the order next to the
// border is the exact one.  A few of them are ranked in pairs; many (equal scores put a whole row there) by the digits
// of (sum, page), so that the time goes with their number: 0.13 ms for 2,048 equal pages, 0.93 for 16,384.
//   Bound: latency.  13.0 us for 64 of 2,048 pages of 8 heads (8.4 MB of bounds): 3 us to the scores, 1 for the
// ticket, 1 to read the scores again, the rest the block's own turns.  As two launches 13.9; four ends of an
// interval a turn instead of 2,048 parts 14.4.
#include "q4.cuh"

namespace rdkv {
namespace q4 {

struct SelectArgs {
  View c;
  const void* q;
  int32_t* sel;
  float* score;  // [rows][page_stride]
  float* error;  // [rows][tiles]: bound of a tile's scores' errors
  int32_t* list;  // [rows][page_stride]: pages near the border
  uint32_t* mask;  // [rows][words]: kept pages, for rows that do not fit in shared memory
  float2* value;  // [rows][page_stride]: their sums, high and low part
  int32_t* tickets;  // [rows] blocks that have written their scores
  int64_t q_stride;
  int dtype, n_q, G, keep, first, last, tiles, words;
};

constexpr int kTilePages = 16;
constexpr int kWarps = 8, kThreads = 32 * kWarps;

// Pages of row (b, t) that hold a key its query token sees.
__device__ __forceinline__ int pages_seen(const SelectArgs& a, int b, int t) {
  const int seen = held_tokens(a.c, b) - a.n_q + t + 1;
  return seen > 0 ? ceil_div(seen, kPage) : 0;
}

__device__ __forceinline__ uint32_t half2_of(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&m);
}

__device__ __forceinline__ void load_eight(const void* q, int64_t at, int dtype, float (&x)[8]) {
  if (dtype == RDKV_F16) Eight<__half>::load(static_cast<const __half*>(q) + at, x);
  else if (dtype == RDKV_BF16) Eight<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(q) + at, x);
  else Eight<float>::load(static_cast<const float*>(q) + at, x);
}

// This warp's tiles of 16 pages (tile, tile + step, ..): every bound is read once, 16 bytes a lane and load, a
// tile's loads all in flight together.  Returns the power of two by which the row's queries are taken: 1, or what keeps
// the sums of very large or small ones inside fp32's range.  A head that holds a NaN or an infinity takes no part.
template <int D>
__device__ __forceinline__ float score_tiles(const SelectArgs& a, int row, int b, int t, int h, int P, int tile, int step) {
  constexpr int NC = D / 32;
  const int lane = threadIdx.x % 32, g = lane / 4, qd = lane % 4, bt = row / a.c.h_kv, n_tiles = ceil_div(P, kTilePages);
  // B: head g of the group, its channels 32 i + 8 qd .. + 7, positive and negative parts and magnitudes
  uint32_t pos[NC][4], neg[NC][4], mag[NC][4];
  float back, unit;
  {
    float x[NC][8], top = 0.0f, odd = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
    if (g < a.G) {
      const int64_t at = (int64_t)bt * a.q_stride + ((int64_t)h * a.G + g) * D + 8 * qd;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        load_eight(a.q, at + 32 * i, a.dtype, x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i][e])), odd = fmaf(x[i][e], 0.0f, odd);  // NaN where one is not finite
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    odd += __shfl_xor_sync(0xffffffffu, odd, 1);
    odd += __shfl_xor_sync(0xffffffffu, odd, 2);
    float most = odd == 0.0f ? top : 0.0f;
    for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    unit = most >= 1.8446744e19f ? 5.4210109e-20f : most > 0.0f && most < 1e-12f ? 1.8446744e19f : 1.0f;  // 2^64
    top *= unit;
    // the head times 2^s, its largest value in [1, 2)
    // (times `unit` inside fp32's range)
    const int s = top > 0.0f ? max(-100, min(unit > 1.0f ? 60 : 100, 127 - (int)(__float_as_uint(top) >> 23))) : 0;
    const float up = __uint_as_float((uint32_t)(s + 127) << 23) * unit;
    back = odd == 0.0f ? __uint_as_float((uint32_t)(127 - s) << 23) : NAN;  // (maxima drop it)
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y0 = x[i][2 * j] * up, y1 = x[i][2 * j + 1] * up;
        pos[i][j] = half2_of(fmaxf(y0, 0.0f), fmaxf(y1, 0.0f));
        neg[i][j] = half2_of(fminf(y0, 0.0f), fminf(y1, 0.0f));
        // 2^-12 more: 2^-13 of the product then covers what fp16's subnormals drop (at most 2^-25 a channel)
        mag[i][j] = half2_of(fabsf(y0) + 0.000244140625f, fabsf(y1) + 0.000244140625f);
      }
  }
  // The products' error against the exact sum, relative to the sum of the magnitudes: at most 16 sums of 17
  // terms, each cut 2^-22 below the largest: below 2^-13.8; the queries' own rounding is none for fp16
  // and bf16, and 2^-11 for fp32.
  const float rel = a.dtype == RDKV_F32 ? 0.0006103515625f + 0.0001220703125f : 0.0001220703125f;
  const float back0 = __shfl_sync(0xffffffffu, back, 8 * qd), back1 = __shfl_sync(0xffffffffu, back, 8 * qd + 4);
  for (; tile < n_tiles; tile += step) {
    uint4 lo[2][NC], hi[2][NC];
    bool bad[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int p = min(tile * kTilePages + 8 * r + g, P - 1);
      const int phys = fetch(a.c.page_table + (int64_t)b * a.c.page_stride + p);
      bad[r] = phys < 0 || phys >= a.c.n_pages;
      if (bad[r] && qd == 0) raise(a.c, RDKV_ERR_INVALID_ARG);
      const uint4* e = reinterpret_cast<const uint4*>(a.c.bounds + ((int64_t)(bad[r] ? 0 : phys) * a.c.h_kv + h) * 2 * D) + qd;
#pragma unroll
      for (int i = 0; i < NC; ++i) lo[r][i] = fetch(e + 4 * i), hi[r][i] = fetch(e + D / 8 + 4 * i);
    }
    float s[4] = {}, m[4] = {};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t l0[4] = {lo[0][i].x, lo[0][i].y, lo[0][i].z, lo[0][i].w}, l1[4] = {lo[1][i].x, lo[1][i].y, lo[1][i].z, lo[1][i].w};
      const uint32_t h0[4] = {hi[0][i].x, hi[0][i].y, hi[0][i].z, hi[0][i].w}, h1[4] = {hi[1][i].x, hi[1][i].y, hi[1][i].z, hi[1][i].w};
      uint32_t b0[4], b1[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b0[j] = max2(l0[j] & 0x7fff7fffu, h0[j] & 0x7fff7fffu);
        b1[j] = max2(l1[j] & 0x7fff7fffu, h1[j] & 0x7fff7fffu);
      }
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        mma16(s, h0[j], h1[j], h0[j + 1], h1[j + 1], pos[i][j], pos[i][j + 1]);
        mma16(s, l0[j], l1[j], l0[j + 1], l1[j + 1], neg[i][j], neg[i][j + 1]);
        mma16(m, b0[j], b1[j], b0[j + 1], b1[j + 1], mag[i][j], mag[i][j + 1]);
      }
    }
    // rows g, g + 8 are pages, columns 2 qd, 2 qd + 1 heads
    float err = 0.0f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int p = tile * kTilePages + 8 * r + g;
      // (pages that are kept anyway, and those without a place, say nothing about the error of the others)
      const bool counts = !bad[r] && p >= a.first && p < P - a.last;
      float x = -INFINITY;
      if (2 * qd < a.G) x = s[2 * r] * back0, err = fmaxf(err, counts ? m[2 * r] * back0 : 0.0f);
      if (2 * qd + 1 < a.G) x = fmaxf(x, s[2 * r + 1] * back1), err = fmaxf(err, counts ? m[2 * r + 1] * back1 : 0.0f);
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      if (qd == 0 && p < P)
        a.score[(int64_t)row * a.c.page_stride + p] = bad[r] || !(x > -FLT_MAX) ? -FLT_MAX : fminf(x, FLT_MAX);
    }
    for (int d = 16; d; d >>= 1) err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, d));
    if (lane == 0) a.error[(int64_t)row * a.tiles + tile] = err * rel;
  }
  return unit;
}

// Sums of a high and a low part (about twice fp32's precision).
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return make_float2(s, (a - (s - t)) + (b - t));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  const float2 s = two_sum(a.x, b.x);
  const float lo = s.y + (a.y + b.y), hi = s.x + lo;
  return make_float2(hi, lo - (hi - s.x));
}
__device__ __forceinline__ float2 add_product(float2 sum, float x, float y) {
  const float p = x * y;
  return add2(sum, make_float2(p, fmaf(x, y, -p)));
}
__device__ __forceinline__ bool above(float2 a, float2 b) { return a.x > b.x || (a.x == b.x && a.y > b.y); }

constexpr int kShared = 8192;  // scores that are kept in shared memory (longer rows are read through L2)
constexpr int kPer = 8, kBins = kPer * kThreads;  // parts an interval is cut into, eight a thread
constexpr int kFew = 32;                          // pages near the border whose sums are taken a head a warp

// Sum of v over the threads before this one, and over all of them (two barriers).
__device__ __forceinline__ int2 block_scan(int v, int* part) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int in = v;
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, in, d);
    if (lane >= d) in += x;
  }
  if (lane == 31) part[warp] = in;
  __syncthreads();
  int before = in - v, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? part[w] : 0;
    all += part[w];
  }
  __syncthreads();
  return make_int2(before, all);
}

// The part that holds the want-th of what bin_s counts, from its first part on, behind `above` others (all threads
// take part; the counts are cleared).
struct Border {
  int part, before, in;  // the part, what lies above it and in it
};
__device__ __forceinline__ Border find_border(int* bin_s, int* part, Border* found_s, int want, int above) {
  int4* mine_s = reinterpret_cast<int4*>(bin_s) + 2 * threadIdx.x;
  __syncthreads();
  const int4 x = mine_s[0], y = mine_s[1];
  mine_s[0] = mine_s[1] = make_int4(0, 0, 0, 0);
  const int n[kPer] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  const int mine = ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
  int before = above + block_scan(mine, part).x;
  if (before < want && before + mine >= want) {
    int j = 0;
#pragma unroll
    for (int i = 0; i < kPer - 1; ++i)
      if (j == i && before + n[i] < want) before += n[i], j = i + 1;
    int in = n[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) in = j == i ? n[i] : in;
    *found_s = Border{kPer * (int)threadIdx.x + j, before, in};
  }
  __syncthreads();
  return *found_s;
}

// Order of pages near the border as a number of three words: the sum's high part, its low part, and the page (the
// lower the larger).
struct Key {
  uint32_t w[3];
};
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 is 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ Key key_of(float2 sum, int page) {  // (infinite sums have no low part)
  return Key{{ordered(sum.x), ordered(sum.y == sum.y ? sum.y : 0.0f), 0xffffffffu - (uint32_t)page}};
}
__device__ __forceinline__ bool at_least(const Key& a, const Key& b) {
  return a.w[0] != b.w[0] ? a.w[0] > b.w[0] : a.w[1] != b.w[1] ? a.w[1] > b.w[1] : a.w[2] >= b.w[2];
}

template <int D>
__global__ void __launch_bounds__(kThreads) select_kernel(SelectArgs a) {
  extern __shared__ float score_s[];
  __shared__ float part_f[kWarps][3];
  __shared__ __align__(16) int bin_s[kBins];
  __shared__ int part[kWarps], list_s[kFew];
  __shared__ uint32_t mask_s[kShared / 32];
  __shared__ float2 value_s[kFew][8];
  __shared__ int list_n, sure_n, last_s;
  __shared__ Border found_s;
  after_previous();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int row = blockIdx.y, h = row % a.c.h_kv, bt = row / a.c.h_kv, t = bt % a.n_q, b = bt / a.n_q;
  const int P = pages_seen(a, b, t);
  if (blockIdx.x == 0 && t == 0 && h == 0 && tid == 0) check_length(a.c, b);
  int32_t* sel = a.sel + (int64_t)row * a.keep;
  if (P <= a.keep) {
    if (blockIdx.x == 0)
      for (int i = tid; i < a.keep; i += kThreads) sel[i] = i < P ? i : -1;
    return;
  }
  const int blocks = min((int)gridDim.x, ceil_div(ceil_div(P, kTilePages), kWarps));
  if ((int)blockIdx.x >= blocks) return;
  const float unit = score_tiles<D>(a, row, b, t, h, P, blockIdx.x * kWarps + warp, blocks * kWarps);
  __syncthreads();
  if (tid == 0) {
    int before;
    asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(before) : "l"(a.tickets + row) : "memory");
    last_s = before == blocks - 1;
    if (last_s) a.tickets[row] = 0;
    list_n = 0, sure_n = 0;
  }
  __syncthreads();
  if (!last_s) return;
  float* score = a.score + (int64_t)row * a.c.page_stride;
  const int lo_p = a.first, hi_p = P - a.last, want = a.keep - a.first - a.last;  // of hi_p - lo_p > want pages
  int4* mine_s = reinterpret_cast<int4*>(bin_s) + 2 * tid;  // this thread's parts
  mine_s[0] = mine_s[1] = make_int4(0, 0, 0, 0);
  float top = -INFINITY, low = INFINITY, eps = 0.0f;
  int scored = 0;  // pages with a score: others (no place, or nothing but NaN) hold -FLT_MAX and come behind them
  const bool here = P <= kShared;
  for (int p = tid; p < P; p += kThreads) {
    const float s = __ldcg(score + p);
    if (here) score_s[p] = s;
    if (p >= lo_p && p < hi_p && s > -FLT_MAX) top = fmaxf(top, s), low = fminf(low, s), ++scored;
  }
  for (int i = tid; i < ceil_div(P, kTilePages); i += kThreads) eps = fmaxf(eps, __ldcg(a.error + (int64_t)row * a.tiles + i));
  for (int d = 16; d; d >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
    eps = fmaxf(eps, __shfl_xor_sync(0xffffffffu, eps, d));
  }
  scored = __reduce_add_sync(0xffffffffu, scored);
  if (lane == 0) part_f[warp][0] = top, part_f[warp][1] = low, part_f[warp][2] = eps, part[warp] = scored;
  __syncthreads();
  scored = 0;
  for (int w = 0; w < kWarps; ++w)
    top = fmaxf(top, part_f[w][0]), low = fminf(low, part_f[w][1]), eps = fmaxf(eps, part_f[w][2]), scored += part[w];
  if (!(eps <= FLT_MAX)) eps = FLT_MAX;
  if (here) score = score_s;
  float lo = low, hi = top;
  if (scored < want) lo = hi = -FLT_MAX;  // the border lies behind all scores
  if (want > 0) {
    // [lo, hi] holds the want-th best score: its part of 2048, counted from the top, then that one's part, until
    // the interval is narrower than the error or holds few (an interval widened by the rounding of its ends
    // still holds it)
    int above_n = 0;  // scores above the interval
#pragma unroll 1
    for (int turn = 0; turn < 8 && hi - lo > eps; ++turn) {
      const float from = lo, width = hi - lo, per = (float)kBins / width;
      if (!(width < FLT_MAX)) break;
#pragma unroll 4
      for (int p = lo_p + tid; p < hi_p; p += kThreads) {
        const float s = score[p];
        if (s >= from && s <= hi) atomicAdd(bin_s + kBins - 1 - min(kBins - 1, (int)((s - from) * per)), 1);
      }
      const Border at = find_border(bin_s, part, &found_s, want, above_n);  // thread 0 has the top parts
      const int j = kBins - 1 - at.part;
      const float slack = 4.0f * FLT_EPSILON * fmaxf(fabsf(from), fabsf(hi)) + 4.0f * FLT_EPSILON * width;
      const float l = from + width * ((float)j / kBins) - slack, u = from + width * ((float)(j + 1) / kBins) + slack;
      const float was = hi - lo;
      lo = fmaxf(lo, l), hi = fminf(hi, u);
      if (at.in <= 4 || !(hi - lo < 0.5f * was)) break;
      int over = 0;
#pragma unroll 4
      for (int p = lo_p + tid; p < hi_p; p += kThreads) over += score[p] > hi;
      above_n = block_scan(over, part).y;
    }
  }
  // in: above the interval by more than twice the error, or one of the first or last; near: within it
  const float sure = hi + 2.0f * eps, out = lo - 2.0f * eps;
  uint32_t* mask = here ? mask_s : a.mask + (int64_t)row * a.words;
  int32_t* list = a.list + (int64_t)row * a.c.page_stride;
  const int words = ceil_div(P, 32);
  {
    int in_n = 0;
#pragma unroll 4
    for (int w = warp; w < words; w += kWarps) {
      const int p = 32 * w + lane;
      const bool mid = p >= lo_p && p < hi_p;
      const float s = mid ? score[p] : -INFINITY;
      const bool in = mid && want > 0 && s > sure, near = mid && want > 0 && !in && s >= out;
      const uint32_t kept = __ballot_sync(0xffffffffu, p < P && (in || !mid)), mids = __ballot_sync(0xffffffffu, in);
      if (lane == 0) mask[w] = kept;
      in_n += __popc(mids);
      if (near) {
        const int i = atomicAdd(&list_n, 1);
        list[i] = p;
        if (i < kFew) list_s[i] = p;
      }
    }
    if (lane == 0 && in_n) atomicAdd(&sure_n, in_n);
  }
  __syncthreads();
  const int need = want - sure_n, near = list_n;
  auto keep_page = [&](int p) { atomicOr(mask + p / 32, 1u << p % 32); };
  if (near <= need) {
    for (int i = tid; i < near; i += kThreads) keep_page(list[i]);
  } else if (need > 0) {
    // their sums again: a head of a page a warp, or (many) a page eight lanes
    float2* value = a.value + (int64_t)row * a.c.page_stride;
    const bool few = near <= kFew;
    if (few) {
#pragma unroll 1
      for (int task = warp; task < near * a.G; task += kWarps) {
        const int i = task / a.G, g = task - i * a.G;
        const int phys = fetch(a.c.page_table + (int64_t)b * a.c.page_stride + list_s[i]);
        float2 best = make_float2(-INFINITY, 0.0f);
        if (phys >= 0 && phys < a.c.n_pages) {
          const __half* e = a.c.bounds + ((int64_t)phys * a.c.h_kv + h) * 2 * D;
          float2 sum = make_float2(0.0f, 0.0f);
          float x[D / 32], l[D / 32], u[D / 32];
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            x[c] = unit * load_q(a.q, (int64_t)bt * a.q_stride + ((int64_t)h * a.G + g) * D + 32 * c + lane, a.dtype);
            l[c] = __half2float(e[32 * c + lane]), u[c] = __half2float(e[D + 32 * c + lane]);
          }
#pragma unroll
          for (int c = 0; c < D / 32; ++c) sum = add_product(sum, x[c], x[c] > 0.0f ? u[c] : l[c]);
#pragma unroll 1
          for (int d = 16; d; d >>= 1)
            sum = add2(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, d), __shfl_xor_sync(0xffffffffu, sum.y, d)));
          if (above(sum, best)) best = sum;
        }
        if (lane == 0) value_s[i][g] = best;
      }
    } else {
#pragma unroll 1
      for (int i0 = 4 * warp; i0 < near; i0 += 4 * kWarps) {
        const int i = i0 + lane / 8;
        const int phys = i < near ? fetch(a.c.page_table + (int64_t)b * a.c.page_stride + list[i]) : -1;
        const bool ok = phys >= 0 && phys < a.c.n_pages;
        const uint4* e = reinterpret_cast<const uint4*>(a.c.bounds + ((int64_t)(ok ? phys : 0) * a.c.h_kv + h) * 2 * D) + lane % 8;
        uint4 l[D / 64], u[D / 64];  // this lane's channels 64 c + 8 (lane % 8) .. + 7
#pragma unroll
        for (int c = 0; c < D / 64; ++c) l[c] = fetch(e + 8 * c), u[c] = fetch(e + D / 8 + 8 * c);
        float2 best = make_float2(-INFINITY, 0.0f);
#pragma unroll 1
        for (int g = 0; g < a.G; ++g) {
          const int64_t at = (int64_t)bt * a.q_stride + ((int64_t)h * a.G + g) * D + 8 * (lane % 8);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            float x[8];
            load_eight(a.q, at + 64 * c, a.dtype, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= unit;
            const uint32_t lw[4] = {l[c].x, l[c].y, l[c].z, l[c].w}, uw[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 lo2 = __half22float2(*reinterpret_cast<const __half2*>(&lw[j])), hi2 = __half22float2(*reinterpret_cast<const __half2*>(&uw[j]));
              sum = add_product(sum, x[2 * j], x[2 * j] > 0.0f ? hi2.x : lo2.x);
              sum = add_product(sum, x[2 * j + 1], x[2 * j + 1] > 0.0f ? hi2.y : lo2.y);
            }
          }
#pragma unroll
          for (int d = 4; d; d >>= 1)
            sum = add2(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, d), __shfl_xor_sync(0xffffffffu, sum.y, d)));
          if (ok && above(sum, best)) best = sum;
        }
        if (lane % 8 == 0 && i < near) value[i] = best;
      }
    }
    __syncthreads();
    if (few) {
      if (warp == 0 && lane < near) {
        float2 best = value_s[lane][0];
        for (int g = 1; g < a.G; ++g)
          if (above(value_s[lane][g], best)) best = value_s[lane][g];
        value_s[lane][0] = best;
      }
      __syncthreads();
    }
    if (few) {
      if (tid < near) {
        const float2 v = value_s[tid][0];
        const int p = list_s[tid];
        int before = 0;
        for (int j = 0; j < near; ++j) {
          const float2 o = value_s[j][0];
          before += above(o, v) || (!above(v, o) && list_s[j] < p);
        }
        if (before < need) keep_page(p);
      }
    } else {
      // the need-th best: the digits of its key one after another, until all that share them are wanted
      Key edge{{0, 0, 0}};
      int taken = 0;
#pragma unroll 1
      for (int d = 0; d < 9; ++d) {
        const int w = d / 3, low = d % 3 == 0 ? 21 : d % 3 == 1 ? 10 : 0;  // the digit: bits low .. top - 1 of word w
        const int top = d % 3 == 0 ? 32 : d % 3 == 1 ? 21 : 10;
        int run = -1, n = 0;  // counts of equal digits are added as one (equal scores would queue for one address)
#pragma unroll 1
        for (int i = tid; i < near; i += kThreads) {
          const Key k = key_of(value[i], list[i]);
          const uint32_t word = w == 0 ? k.w[0] : w == 1 ? k.w[1] : k.w[2], at = w == 0 ? edge.w[0] : w == 1 ? edge.w[1] : edge.w[2];
          if ((w > 0 && k.w[0] != edge.w[0]) || (w > 1 && k.w[1] != edge.w[1]) || ((uint64_t)(word ^ at) >> top) != 0) continue;
          const int digit = kBins - 1 - (int)((word >> low) & (kBins - 1) & ((1u << (top - low)) - 1u));
          if (digit != run) {
            if (n) atomicAdd(bin_s + run, n);
            run = digit, n = 0;
          }
          ++n;
        }
        if (n) atomicAdd(bin_s + run, n);
        const Border at = find_border(bin_s, part, &found_s, need, taken);
        const uint32_t digit = (uint32_t)(kBins - 1 - at.part) << low;
        if (w == 0) edge.w[0] |= digit;
        else if (w == 1) edge.w[1] |= digit;
        else edge.w[2] |= digit;
        taken = at.before;
        if (taken + at.in == need) break;
      }
      for (int i = tid; i < near; i += kThreads)
        if (at_least(key_of(value[i], list[i]), edge)) keep_page(list[i]);
    }
  }
  __syncthreads();
  // the kept pages in order: a run of words a lane
  if (warp == 0) {
    const int per = ceil_div(words, 32), w0 = min(words, lane * per), w1 = min(words, w0 + per);
    int n = 0;
    auto word = [&](int w) { return here ? mask[w] : __ldcg(mask + w); };  // (atomics have changed it in L2)
    for (int w = w0; w < w1; ++w) n += __popc(word(w));
    int at = n;
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, at, d);
      if (lane >= d) at += x;
    }
    at -= n;
    for (int w = w0; w < w1; ++w)
      for (uint32_t m = word(w); m && at < a.keep; m &= m - 1) sel[at++] = 32 * w + __ffs(m) - 1;
  }
}

}  // namespace q4
}  // namespace rdkv

using namespace rdkv;
using namespace rdkv::q4;

namespace {
struct SelectGeometry {
  int64_t rows;
  int tiles;
  size_t value_at, error_at, list_at, score_at, mask_at, bytes;
};
SelectGeometry select_geometry(const rdkv_q4_cache* c, int n_q) {
  SelectGeometry o;
  o.rows = (int64_t)c->batch * n_q * c->h_kv;
  o.tiles = ceil_div(c->page_stride, kTilePages);
  const int64_t pages = o.rows * c->page_stride;
  o.value_at = RDKV_Q4_COUNTER_BYTES;  // after the tickets, whose place is the same for every shape
  o.error_at = o.value_at + (size_t)align_up(8 * pages, 256);
  o.list_at = o.error_at + (size_t)align_up(4 * o.rows * o.tiles, 256);
  o.score_at = o.list_at + (size_t)align_up(4 * pages, 256);
  o.mask_at = o.score_at + (size_t)align_up(4 * pages, 256);
  o.bytes = o.mask_at + (size_t)align_up(4 * o.rows * ceil_div(c->page_stride, 32), 256);
  return o;
}
}  // namespace

extern "C" size_t rdkv_q4_select_workspace_bytes(const rdkv_q4_cache* cache, int32_t h_q, int32_t n_q) {
  return check_queries(cache, h_q, n_q) == RDKV_OK ? select_geometry(cache, n_q).bytes : 0;
}

extern "C" rdkv_status rdkv_q4_select(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride,
                                      int32_t h_q, int32_t n_q, int32_t n_keep, int32_t n_first, int32_t n_last, int32_t* sel,
                                      void* ws, size_t ws_bytes, void* stream) {
  rdkv_status st = check_q(cache, dtype, q, q_stride, h_q, n_q);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(cache->bounds && sel, RDKV_ERR_INVALID_ARG, "NULL bounds or selection");
  RDKV_REQUIRE(n_keep >= 1 && n_first >= 0 && n_last >= 0 && (int64_t)n_first + n_last <= n_keep, RDKV_ERR_INVALID_ARG,
               "n_keep=%d n_first=%d n_last=%d", n_keep, n_first, n_last);
  const SelectGeometry geo = select_geometry(cache, n_q);
  RDKV_REQUIRE(ws && (uintptr_t)ws % 16 == 0 && ws_bytes >= geo.bytes, RDKV_ERR_WORKSPACE,
               "selection workspace too small (%zu < %zu) or unaligned", ws_bytes, geo.bytes);
  char* w = static_cast<char*>(ws);
  const SelectArgs a{view_of(cache), q, sel,
                     reinterpret_cast<float*>(w + geo.score_at),
                     reinterpret_cast<float*>(w + geo.error_at), reinterpret_cast<int32_t*>(w + geo.list_at),
                     reinterpret_cast<uint32_t*>(w + geo.mask_at),
                     reinterpret_cast<float2*>(w + geo.value_at), reinterpret_cast<int32_t*>(w), q_stride, dtype, n_q, h_q / cache->h_kv, n_keep, n_first, n_last,
                     geo.tiles, ceil_div(cache->page_stride, 32)};
  cudaStream_t cs = (cudaStream_t)stream;
  // a tile a warp, as far as about four blocks an SM go; warps take further tiles in turn
  const int64_t most = std::max<int64_t>(1, 4LL * num_sms() / geo.rows);
  const dim3 grid((unsigned)std::min<int64_t>(ceil_div(geo.tiles, kWarps), most), (unsigned)geo.rows);
  const size_t smem = 4 * (size_t)std::min(cache->page_stride, kShared);
  RDKV_TRY_CUDA(launch_after(cache->head_dim == 128 ? select_kernel<128> : select_kernel<64>, grid, kThreads, smem, cs, a),
                "4-bit cache page selection");
  count_launch();
  return RDKV_OK;
}
