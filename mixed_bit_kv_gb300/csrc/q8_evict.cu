// Eviction from the 8-bit paged cache by accumulated weight (rdkv_q8_evict).
//
// Choice.  Of a (sequence, KV head) with more than n_keep tokens the n_keep - n_first - n_last largest weights
// between the first and the last are found by their digits: a weight's bits, turned into a number of the same order, eight
// bits a pass from the top, each pass counting the candidates by digit.  The row is spread over a cluster of blocks;
// their counts meet through distributed shared memory, so that one launch does all passes without a trip
// through global memory between them.  Counts lie in 32 columns, a lane its own, so that lanes that meet the same digit
// (most do: weights share few exponents) do not wait for one another.  Of the weights equal to the last one kept, the
// lowest positions are.
//
// Move.  A kept row goes to a place at or below its own.  The pages of a row are taken in ascending order, each by one
// block (a ticket says which: blocks that wait do so for lower tickets, which have started): it reads its
// 64 rows from wherever they are, raises its page's flag, waits for the flags of the lower pages that have rows of theirs in
// this page, and writes.  So every row is read once and written once, in place, without a copy of the cache.
#include <atomic>

#include "q8.cuh"

namespace rdkv {
namespace q8 {

struct EvictArgs {
  View c;
  float* mass;
  int64_t mass_stride;
  int n_keep, n_first, n_last;
  int32_t* kept;
  int32_t* ranks;   // [batch * h_kv][page_stride + 1]: rows kept before each page
  int32_t* flags;   // [batch * h_kv][page_stride]: 1: the page's rows have been read
  int2* todo;       // [batch * h_kv * page_stride] (sequence * h_kv + head, page): the pages to move, ascending in a row
  int32_t* ticket;  // [1] pages taken
};

constexpr int kPickThreads = 512;
constexpr int kMoveThreads = 256;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// A word of another block's shared memory.
__device__ __forceinline__ uint32_t remote(const uint32_t* p, uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// A number that orders weights as their values do; a NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_of(uint32_t w) {
  if ((w & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if ((w & 0x7fffffffu) == 0u) w = 0u;
  return w & 0x80000000u ? ~w : w | 0x80000000u;
}

// Pages that sequence b holds.
__device__ __forceinline__ int pages_of(const PageView& v, int b) { return ceil_div(held_tokens(v, b), kPage); }

// A cluster a (sequence, KV head); a warp has a run of the row's pages, a lane two positions of each.
__global__ void __launch_bounds__(kPickThreads, 1) pick_kernel(EvictArgs a) {
  constexpr int kWarps = kPickThreads / 32;
  __shared__ uint32_t count_s[256 * 32];  // by digit and lane
  __shared__ uint32_t block_s[256];       // this block's counts
  __shared__ uint32_t sum_s[256 / 32], digit_s, above_s, within_s;
  __shared__ uint2 warp_s[kWarps];        // a warp's rows kept for sure, and its candidates equal to the border
  __shared__ uint32_t total_s[2];
  after_previous();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int row = blockIdx.x / size, H = a.c.h_kv, b = row / H, h = row - b * H;
  const int len = held_tokens(a.c, b), pages = ceil_div(len, kPage), stride = a.c.page_stride;
  const float* mass = a.mass + (int64_t)row * a.mass_stride;
  int32_t* kept = a.kept + (int64_t)row * a.n_keep;
  int32_t* ranks = a.ranks + (int64_t)row * (stride + 1);
  if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;
  if (h == 0 && rank == 0 && tid == 0) check_length(a.c, b);
  const int part = rank * kWarps + warp, parts = size * kWarps;
  const int p0 = share(part, pages, parts), p1 = share(part + 1, pages, parts);
  // where this row's pages are listed
  int64_t base = 0;
  for (int i = tid; i < b; i += kPickThreads) base += pages_of(a.c, i);
  for (int d = 16; d; d >>= 1) base += __shfl_xor_sync(0xffffffffu, base, d);
  // a page outside the pool: the row stays
  bool bad = false;
  for (int p = tid; p < pages; p += kPickThreads) {
    const int at = fetch(a.c.page_table + (int64_t)b * stride + p);
    bad |= at < 0 || at >= a.c.n_pages;
  }
  if (tid < 256) block_s[tid] = 0;
  if (tid == 0) total_s[0] = total_s[1] = 0;
  bad = __syncthreads_or(bad);
  // (the lists' starts: over the warps)
  if (lane == 0 && base) atomicAdd(&block_s[warp], (uint32_t)base);
  __syncthreads();
  base = 0;
  for (int i = 0; i < kWarps; ++i) base += block_s[i];
  base = base * H + (int64_t)h * pages;
  __syncthreads();
  int2* todo = a.todo + base;
  const int part_of_all = rank * kPickThreads + tid, all = size * kPickThreads;
  const bool stays = bad || len <= a.n_keep;  // (the same in the whole cluster)
  if (stays) {
    if (bad && part_of_all == 0) raise(a.c, RDKV_ERR_INVALID_ARG);
    for (int i = part_of_all; i < a.n_keep; i += all) kept[i] = !bad && i < len ? i : -1;
    for (int p = part_of_all; p < pages; p += all) todo[p] = make_int2(-1, 0);
    return;
  }
  for (int p = part_of_all; p < pages; p += all) a.flags[(int64_t)row * stride + p] = 0;

  // ---- the border: the need-th largest of the weights between the first and the last
  const int lo = a.n_first, hi = len - a.n_last;
  uint32_t need = a.n_keep - a.n_first - a.n_last, border = 0, mask = 0;
  bool some = need > 0;
#pragma unroll 1
  for (int shift = 24; some && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256 * 32; i += kPickThreads) count_s[i] = 0;
    __syncthreads();
    constexpr int kAhead = 4;
#pragma unroll 1
    for (int p = p0; p < p1; p += kAhead) {
      uint2 w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        w[i] = p + i < p1 ? fetch(reinterpret_cast<const uint2*>(mass + (int64_t)(p + i) * kPage + 2 * lane)) : make_uint2(0, 0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int t = (p + i) * kPage + 2 * lane;
        const uint32_t x = order_of(w[i].x), y = order_of(w[i].y);
        if (p + i < p1 && t >= lo && t < hi && (x & mask) == border) atomicAdd(&count_s[(x >> shift & 255) * 32 + lane], 1u);
        if (p + i < p1 && t + 1 >= lo && t + 1 < hi && (y & mask) == border) atomicAdd(&count_s[(y >> shift & 255) * 32 + lane], 1u);
      }
    }
    __syncthreads();
    // a digit's count: its 32 columns, each thread from another one on (no bank conflicts)
    for (int d = tid; d < 256; d += kPickThreads) {
      uint32_t n = 0;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) n += count_s[d * 32 + (i + tid) % 32];
      block_s[d] = n;
    }
    cluster_sync();
    uint32_t n = 0;
    if (tid < 256)  // digit 255 - tid: from the largest down
      for (uint32_t r = 0; r < size; ++r) n += size > 1 ? remote(&block_s[255 - tid], r) : block_s[255 - tid];
    uint32_t in = n;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += x;
    }
    if (tid < 256 && lane == 31) sum_s[warp] = in;
    __syncthreads();
    if (tid < 256) {
      for (int i = 0; i < warp; ++i) in += sum_s[i];
      if (in >= need && in - n < need) digit_s = 255 - tid, above_s = in - n, within_s = n;
    }
    cluster_sync();  // (also: every block has read the counts)
    need -= above_s;
    border |= digit_s << shift;
    mask |= 0xffu << shift;
    if (within_s == need) break;  // all of them: no further digit decides
  }
  // kept are: the first, the last, what is above the border and, of what lies on it (under the mask), `need`
  // ---- how many of each before this warp's pages
  auto classes = [&](int p, bool (&sure)[2], bool (&tie)[2]) {
    const uint2 w = fetch(reinterpret_cast<const uint2*>(mass + (int64_t)p * kPage + 2 * lane));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = p * kPage + 2 * lane + i;
      const uint32_t x = order_of(i ? w.y : w.x) & mask;
      const bool open = t >= lo && t < hi;
      sure[i] = t < len && (!open || (some && x > border));
      tie[i] = open && some && x == border;
    }
  };
  uint32_t n_sure = 0, n_tie = 0;
#pragma unroll 4
  for (int p = p0; p < p1; ++p) {
    bool sure[2], tie[2];
    classes(p, sure, tie);
    n_sure += sure[0] + sure[1], n_tie += tie[0] + tie[1];
  }
  n_sure = __reduce_add_sync(0xffffffffu, n_sure), n_tie = __reduce_add_sync(0xffffffffu, n_tie);
  if (lane == 0) {
    warp_s[warp] = make_uint2(n_sure, n_tie);
    atomicAdd(&total_s[0], n_sure), atomicAdd(&total_s[1], n_tie);
  }
  cluster_sync();
  uint32_t sure0 = 0, tie0 = 0;
  for (uint32_t r = 0; r < rank; ++r) sure0 += remote(&total_s[0], r), tie0 += remote(&total_s[1], r);
  for (int i = 0; i < warp; ++i) sure0 += warp_s[i].x, tie0 += warp_s[i].y;
  cluster_sync();  // a block's shared memory outlives the others' reads
  // ---- their places
  uint32_t at = sure0 + min(tie0, need);
#pragma unroll 2
  for (int p = p0; p < p1; ++p) {
    bool sure[2], tie[2];
    classes(p, sure, tie);
    const uint32_t before = (1u << lane) - 1u;
    const uint32_t t0 = __ballot_sync(0xffffffffu, tie[0]), t1 = __ballot_sync(0xffffffffu, tie[1]);
    const uint32_t mine = tie0 + __popc(t0 & before) + __popc(t1 & before);
    const bool k0 = sure[0] || (tie[0] && mine < need), k1 = sure[1] || (tie[1] && mine + tie[0] < need);
    const uint32_t b0 = __ballot_sync(0xffffffffu, k0), b1 = __ballot_sync(0xffffffffu, k1);
    const uint32_t to = at + __popc(b0 & before) + __popc(b1 & before);
    const int t = p * kPage + 2 * lane;
    if (k0) kept[to] = t;
    if (k1) kept[to + k0] = t + 1;
    const uint32_t next = at + __popc(b0) + __popc(b1);
    if (lane == 0) {
      ranks[p] = at;
      if (p == pages - 1) ranks[pages] = next;
      // nothing to do where every row stays
      todo[p] = at == (uint32_t)p * kPage && next == (uint32_t)min(len, (p + 1) * kPage) ? make_int2(-1, 0) : make_int2(row, p);
    }
    at = next, tie0 += __popc(t0) + __popc(t1);
  }
}

// Loads past L1, in the order in which they stand: before the flag that says that they are done.
__device__ __forceinline__ uint32_t fetch_l2(const float* p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 fetch_l2(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 fetch_l2(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
// The largest magnitude of four codes in a scale f, and top.
__device__ __forceinline__ float largest(uint32_t w, float f, float top) {
  float x[4];
  values4(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(x[i]) * f);
  return top;
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(EvictArgs a) {
  using L = Layout<D>;
  constexpr int kS = L::kSides, kKeys = kPage * D / 8 / kMoveThreads, kValues = kPage * D / 16 / kMoveThreads;
  __shared__ int64_t from_s[kPage];   // a row's (page, head), -1: no row
  __shared__ int slot_s[kPage];
  __shared__ float2 scale_s[kPage];   // its scales
  __shared__ uint32_t top_s[2][kMoveThreads / 32];
  __shared__ int ticket_s, total_s;
  const int tid = threadIdx.x, H = a.c.h_kv, stride = a.c.page_stride;
  after_previous();
  int total = 0;  // (the host has made sure that all rows' pages fit)
  for (int i = tid; i < a.c.batch; i += kMoveThreads) total += pages_of(a.c, i) * H;
  if (tid == 0) total_s = 0;
  __syncthreads();
  if (total) atomicAdd(&total_s, total);
  __syncthreads();
  total = total_s;
#pragma unroll 1
  for (;;) {
    if (tid == 0) ticket_s = atomicAdd(a.ticket, 1);
    __syncthreads();
    const int ticket = ticket_s;
    if (ticket >= total) return;
    const int2 what = *reinterpret_cast<const int2*>(a.todo + ticket);
    if (what.x < 0) {
      __syncthreads();  // (before the next ticket)
      continue;
    }
    const int row = what.x, p = what.y, b = row / H, h = row - b * H;
    const int len = held_tokens(a.c, b);
    const int32_t* kept = a.kept + (int64_t)row * a.n_keep;
    const int32_t* ranks = a.ranks + (int64_t)row * (stride + 1);
    const int32_t* table = a.c.page_table + (int64_t)b * stride;
    float* mass = a.mass + (int64_t)row * a.mass_stride;
    const int n = max(0, min(kPage, a.n_keep - p * kPage));  // rows that come here
    float m = 0.0f;
    if (tid < kPage) {
      int64_t from = -1;
      if (tid < n) {
        const int t = kept[p * kPage + tid];
        from = (int64_t)table[t / kPage] * H + h;
        slot_s[tid] = t % kPage;
        const uint2 sc = fetch_l2(reinterpret_cast<const uint2*>(a.c.scales + from * 2));
        scale_s[tid] = make_float2(__uint_as_float(sc.x), __uint_as_float(sc.y));
        m = __uint_as_float(fetch_l2(mass + t));
      }
      from_s[tid] = from;
    }
    __syncthreads();
    // the rows' codes: eight channels of a token of the keys, of a token pair of the values
    uint2 kc[kKeys];
    uint4 vc[kValues][2];
    float top[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int u = tid + i * kMoveThreads, t = u / (16 * kS) * 2 + u / 8 % 2;
      kc[i] = t < n ? fetch_l2(reinterpret_cast<const uint2*>(a.c.pages + from_s[t] * L::kBytes + L::key_at(slot_s[t], u / 16 % kS, u % 8)))
                    : make_uint2(0, 0);
    }
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int u = tid + i * kMoveThreads, t = (u / (32 * kS) * 4 + u % 4) * 2, j = u / 32 % kS, g = u % 32 / 4;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        vc[i][s] = t + s < n ? fetch_l2(reinterpret_cast<const uint4*>(a.c.pages + from_s[t + s] * L::kBytes + L::kHalf +
                                                                     L::value_at(slot_s[t + s] / 2, j, g)))
                             : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int u = tid + i * kMoveThreads, t = u / (16 * kS) * 2 + u / 8 % 2;
      const float f = t < n ? scale_s[t].x : 0.0f;
      top[0] = largest(kc[i].x, f, largest(kc[i].y, f, top[0]));
    }
    uint2 vb[kValues][2];  // a token's eight codes
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int u = tid + i * kMoveThreads, t = (u / (32 * kS) * 4 + u % 4) * 2;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool real = t + s < n;
        const uint32_t pick = real && (slot_s[t + s] & 1) ? 0x7531u : 0x6420u;
        const uint4 w = vc[i][s];
        vb[i][s] = make_uint2(__byte_perm(w.x, w.y, pick), __byte_perm(w.z, w.w, pick));
        const float f = real ? scale_s[t + s].y : 0.0f;
        top[1] = largest(vb[i][s].x, f, largest(vb[i][s].y, f, top[1]));
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(top[s]));
      if (tid % 32 == 0) top_s[s][tid / 32] = w;
    }
    __syncthreads();  // every row has been read
    if (tid == 0) {
      asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(a.flags + (int64_t)row * stride + p), "r"(1) : "memory");
    }
    // lower pages that have rows of theirs here
    bool ok = true;
    const int first = ranks[p] / kPage, last = min(p - 1, (ranks[p + 1] - 1) / kPage);
    for (int l = first + tid; l <= last; l += kMoveThreads) {
      const int32_t* f = a.flags + (int64_t)row * stride + l;
      int seen;
      const long long t0 = clock64();
      do {
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(f) : "memory");
      } while (!seen && clock64() - t0 < kWaitCycles);
      ok &= seen != 0;
    }
    if (!__syncthreads_and(ok)) {
      if (tid == 0) raise(a.c, RDKV_ERR_TIMEOUT);
      return;
    }
    if (tid < kPage && p * kPage + tid < len) mass[p * kPage + tid] = m;
    if (n > 0) {  // (what is left of the last page: zero)
      uint32_t w[2] = {top_s[0][0], top_s[1][0]};
#pragma unroll
      for (int i = 1; i < kMoveThreads / 32; ++i) w[0] = max(w[0], top_s[0][i]), w[1] = max(w[1], top_s[1][i]);
      const int ke = exponent_for(__uint_as_float(w[0])), ve = exponent_for(__uint_as_float(w[1]));
      const int64_t to = (int64_t)table[p] * H + h;
      uint8_t* page = a.c.pages + to * L::kBytes;
      if (tid == 0) *reinterpret_cast<float2*>(a.c.scales + to * 2) = make_float2(two_to(ke), two_to(ve));
      const float kf = two_to(-ke), vf = two_to(-ve);
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const int u = tid + i * kMoveThreads, t = u / (16 * kS) * 2 + u / 8 % 2;
        const float f = t < n ? scale_s[t].x * kf : 1.0f;
        if (f != 1.0f) kc[i] = make_uint2(rescaled(kc[i].x, f), rescaled(kc[i].y, f));
        *reinterpret_cast<uint2*>(page + L::key_at(t, u / 16 % kS, u % 8)) = kc[i];
      }
#pragma unroll
      for (int i = 0; i < kValues; ++i) {
        const int u = tid + i * kMoveThreads, q = u / (32 * kS) * 4 + u % 4, t = 2 * q;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const float f = t + s < n ? scale_s[t + s].y * vf : 1.0f;
          if (f != 1.0f) vb[i][s] = make_uint2(rescaled(vb[i][s].x, f), rescaled(vb[i][s].y, f));
        }
        *reinterpret_cast<uint4*>(page + L::kHalf + L::value_at(q, u / 32 % kS, u % 32 / 4)) =
            make_uint4(__byte_perm(vb[i][0].x, vb[i][1].x, 0x5140), __byte_perm(vb[i][0].x, vb[i][1].x, 0x7362),
                       __byte_perm(vb[i][0].y, vb[i][1].y, 0x5140), __byte_perm(vb[i][0].y, vb[i][1].y, 0x7362));
      }
    }
    __syncthreads();  // (before the next ticket and its rows)
  }
}

struct EvictLayout {
  size_t ranks_at, flags_at, todo_at, bytes;
};
static EvictLayout evict_layout(const rdkv_q8_cache* c) {
  const int64_t rows = (int64_t)c->batch * c->h_kv;
  EvictLayout o;
  o.ranks_at = 256;
  o.flags_at = o.ranks_at + (size_t)align_up(4 * rows * (c->page_stride + 1), 256);
  o.todo_at = o.flags_at + (size_t)align_up(4 * rows * c->page_stride, 256);
  o.bytes = o.todo_at + (size_t)align_up(8 * rows * c->page_stride, 256);
  return o;
}

}  // namespace q8
}  // namespace rdkv

using namespace rdkv;
using namespace rdkv::q8;

extern "C" size_t rdkv_q8_evict_workspace_bytes(const rdkv_q8_cache* cache) {
  if (check_cache(cache) != RDKV_OK) return 0;
  return evict_layout(cache).bytes;
}

extern "C" rdkv_status rdkv_q8_evict(const rdkv_q8_cache* cache, float* mass, int64_t mass_stride, int32_t n_keep, int32_t n_first,
                                     int32_t n_last, int32_t* kept, void* ws, size_t ws_bytes, void* stream) {
  rdkv_status st = check_cache(cache);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(mass && kept, RDKV_ERR_INVALID_ARG, "NULL mass or kept");
  st = check_mass(cache, mass, mass_stride);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE((uintptr_t)kept % 4 == 0, RDKV_ERR_INVALID_ARG, "kept must be 4-byte aligned");
  RDKV_REQUIRE(n_keep >= 1 && n_first >= 0 && n_last >= 0 && (int64_t)n_first + n_last <= n_keep, RDKV_ERR_INVALID_ARG,
               "n_keep %d, n_first %d, n_last %d", n_keep, n_first, n_last);
  RDKV_REQUIRE((int64_t)cache->batch * cache->h_kv * cache->page_stride <= INT32_MAX, RDKV_ERR_UNSUPPORTED,
               "more than 2^31 - 1 (sequence, KV head, page) items");
  const EvictLayout lay = evict_layout(cache);
  RDKV_REQUIRE(ws && (uintptr_t)ws % 16 == 0 && ws_bytes >= lay.bytes, RDKV_ERR_WORKSPACE, "eviction workspace too small (%zu < %zu) or unaligned",
               ws_bytes, lay.bytes);
  char* w = static_cast<char*>(ws);
  const EvictArgs a{q8::view_of(cache), mass, mass_stride, n_keep, n_first, n_last, kept, reinterpret_cast<int32_t*>(w + lay.ranks_at),
                    reinterpret_cast<int32_t*>(w + lay.flags_at), reinterpret_cast<int2*>(w + lay.todo_at), reinterpret_cast<int32_t*>(w)};
  cudaStream_t cs = (cudaStream_t)stream;
  const int rows = cache->batch * cache->h_kv;
  // blocks of a row: 16 warps each; a warp takes four pages at least, and eight blocks are the most a cluster holds everywhere
  int size = 1;
  while (size < 8 && size * 64 < cache->page_stride) size *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * size), cfg.blockDim = dim3(kPickThreads), cfg.stream = cs;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 2;
  RDKV_TRY_CUDA(cudaLaunchKernelEx(&cfg, pick_kernel, a), "8-bit cache eviction");
  count_launch();
  const int64_t pages = (int64_t)rows * cache->page_stride;
  const unsigned grid = (unsigned)std::min<int64_t>(pages, (int64_t)num_sms() * 6);
  auto move = cache->head_dim == 128 ? move_kernel<128> : move_kernel<64>;
  RDKV_TRY_CUDA(launch_after(move, dim3(grid), kMoveThreads, 0, cs, a), "8-bit cache eviction");
  count_launch();
  return RDKV_OK;
}
