// Eviction from the 8-bit paged cache by accumulated weight (rdkv_q8_evict).
//
// Choice.  Of a (sequence, KV head) with more than n_keep tokens the n_keep - n_first - n_last largest weights
// between the first and the last are found by their digits: a weight's bits, turned into a number of the same order, eight
// bits a pass from the top, each pass counting the candidates by digit.  The row is spread over a cluster of blocks, which
// hold its weights in shared memory; their counts meet through distributed shared memory, so that one launch does all
// passes without a trip through global memory.  Counts lie in 32 columns, a lane its own, so that lanes that meet the
// same digit (most do: weights share few exponents) do not wait for one another.  Of the weights equal to the last one
// kept, the lowest positions are.
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
  int2* from;       // [batch * h_kv][n_keep]: the (page, head) that a kept row lies in, and its slot and scales (how_of)
  int32_t* flags;   // [batch * h_kv][page_stride]: 1: the page's rows have been read
  int2* waits;      // [batch * h_kv][page_stride]: the first and last lower page that has rows of a page
  int2* todo;       // [count] the pages to fill, (sequence, head) and page, ascending in a row
  int32_t* count;   // pages to fill, pages taken, blocks done: zero between the calls
  int withhold;           // 0, or (the self-test) pages with (index + KV head) % withhold == 0 do not raise their flags
  long long wait_cycles;  // limit of a wait for a flag
};

constexpr int kStay = -2;  // in a page's place: it stays
constexpr int kPickThreads = 512;
constexpr int kMoveThreads = 128, kMoveBlocks = 8;  // an SM
// Blocks of a row's cluster at most.  (131,072 tokens of 8 heads to a quarter, in a build that took 85 us: with 16, which have to be asked
// for, 95, as of eight such clusters one waits for another.  In one that took 80: with 16 and two blocks an SM, so that none waits, 1 more;
// with eight blocks of 1,024 threads 1 more, and rows of 3,000 tokens 2.5 more.)
constexpr int kMaxBlocks = 8;
// Pages of the table a warp has before the row takes twice as many blocks.  A middle between few rows, which more blocks serve sooner, and
// many, which fill the SMs by themselves (16,384 tokens, hardly a row moved: with 4, 8 and 16 pages a warp 8 rows take 15.0, 17.4 and
// 20.4 us, 128 rows 48.2, 31.3 and 20.6).
constexpr int kSplit = 8;
constexpr int kHold = 16;  // pages of a warp whose weights shared memory holds; those of longer rows are loaded again

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
// All blocks of a cluster (of one: the block alone).
__device__ __forceinline__ void cluster_sync(uint32_t size) {
  if (size == 1) __syncthreads();
  else asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
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

// A row's slot and its page's scales' exponents, in a word.
__device__ __forceinline__ int how_of(int slot, uint2 scales) {
  auto e = [](uint32_t s) { return min(max(exponent(__uint_as_float(s)), kLowExp), kHighExp) - kLowExp; };
  return slot | e(scales.x) << 8 | e(scales.y) << 16;
}
__device__ __forceinline__ int slot_of(int how) { return how & 63; }
__device__ __forceinline__ float key_scale(int how) { return two_to((how >> 8 & 31) + kLowExp); }
__device__ __forceinline__ float value_scale(int how) { return two_to((how >> 16 & 31) + kLowExp); }
// The two words of a page's weights that are this lane's; past the row: not used.
__device__ __forceinline__ uint2 weights_of(const float* mass, int p, int lane) {
  return fetch(reinterpret_cast<const uint2*>(mass + (int64_t)p * kPage + 2 * lane));
}

// A cluster a (sequence, KV head); a warp has a run of the row's pages, a lane two positions of each.
//   Bound: a chain of passes, each a count, a sum over lanes and blocks and a scan, some 1.2 us (0.5 of them counting at three
// pages a warp), 3 at sixteen pages a warp, where the issue slots are half used.  8 us for 32 rows of 3,000 tokens, 11 for 128 rows of 4,160, 26 for 8
// rows of 131,072 (8 blocks each).  Blocks and shared memory are those of the table: where sequences are much shorter than it the
// rows pay for clusters that they do not need (16 x 4,160 tokens, all pages moving, in tables of 131,072: 149 us, in their own 75).
// (Short loops: the code is fetched anew by every launch.  With the weights in registers and every loop unrolled, 30 KB of it, the
// choice took 16 us for 32 rows of 3,000 tokens under the profiler.)
__global__ void __launch_bounds__(kPickThreads, 1) pick_kernel(EvictArgs a, int hold) {
  constexpr int kWarps = kPickThreads / 32;
  __shared__ uint32_t count_s[256 * 32];  // by digit and lane
  __shared__ uint32_t block_s[256];       // this block's counts
  __shared__ uint32_t sum_s[256 / 32], digit_s, above_s, within_s;
  __shared__ uint2 warp_s[kWarps];        // a warp's rows kept for sure, and its candidates equal to the border
  __shared__ uint32_t total_s[2], first_s, base_s;
  extern __shared__ uint2 held_s[];       // [warps][hold][32]
  after_previous();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int row = blockIdx.x / size, H = a.c.h_kv, b = row / H, h = row - b * H;
  const int len = held_tokens(a.c, b), pages = ceil_div(len, kPage), stride = a.c.page_stride;
  float* mass = a.mass + (int64_t)row * a.mass_stride;
  const int32_t* table = a.c.page_table + (int64_t)b * stride;
  int32_t* kept = a.kept + (int64_t)row * a.n_keep;
  const int part = rank * kWarps + warp, parts = size * kWarps;
  const int p0 = share(part, pages, parts), p1 = share(part + 1, pages, parts);
  uint2* held = held_s + (int64_t)warp * hold * 32 + lane;
  if (len > a.n_keep) {
#pragma unroll 4
    for (int p = p0; p < min(p1, p0 + hold); ++p)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(held + (p - p0) * 32)), "l"(mass + (int64_t)p * kPage + 2 * lane) : "memory");
  }
  // a page's two weights as numbers of their order
  auto orders = [&](int p) {
    if (p - p0 < hold) return held[(p - p0) * 32];
    const uint2 w = weights_of(mass, p, lane);
    return make_uint2(order_of(w.x), order_of(w.y));
  };
  if (h == 0 && rank == 0 && tid == 0) check_length(a.c, b);
  // a page outside the pool: the row stays
  bool bad = false;
  for (int p = tid; p < pages; p += kPickThreads) {
    const int at = fetch(table + p);
    bad |= at < 0 || at >= a.c.n_pages;
  }
  if (tid == 0) total_s[0] = total_s[1] = 0, first_s = 0x7fffffffu;
  for (int i = tid; i < 256 * 32; i += kPickThreads) count_s[i] = 0;
  bad = __syncthreads_or(bad);
  const int part_of_all = rank * kPickThreads + tid, all = size * kPickThreads;
  if (bad || len <= a.n_keep) {  // (the same in the whole cluster)
    if (bad && part_of_all == 0) raise(a.c, RDKV_ERR_INVALID_ARG);
    for (int64_t i = part_of_all; i < a.n_keep; i += all) kept[i] = !bad && i < len ? (int)i : -1;
    asm volatile("cp.async.wait_all;" ::: "memory");  // (the weights of a row that would have been brought down)
    return;
  }
  const int filled = ceil_div(a.n_keep, kPage);
  for (int p = part_of_all; p < filled; p += all) a.flags[(int64_t)row * stride + p] = 0;
  asm volatile("cp.async.wait_all;" ::: "memory");  // (each thread reads what it asked for)
#pragma unroll 2
  for (int p = p0; p < min(p1, p0 + hold); ++p) {
    const uint2 w = held[(p - p0) * 32];
    held[(p - p0) * 32] = make_uint2(order_of(w.x), order_of(w.y));
  }

  // ---- the border: the need-th largest of the weights between the first and the last
  const int lo = a.n_first;
  const uint32_t range = len - a.n_last - a.n_first;  // positions that may go, from lo on
  uint32_t need = a.n_keep - a.n_first - a.n_last, border = 0, mask = 0;
  const bool some = need > 0;
#pragma unroll 1
  for (int shift = 24; some && shift >= 0; shift -= 8) {
#pragma unroll 2
    for (int p = p0; p < p1; ++p) {
      const uint2 w = orders(p);
      const uint32_t t = (uint32_t)(p * kPage + 2 * lane - lo);
      if (t < range && (w.x & mask) == border) atomicAdd(&count_s[(w.x >> shift & 255) * 32 + lane], 1u);
      if (t + 1 < range && (w.y & mask) == border) atomicAdd(&count_s[(w.y >> shift & 255) * 32 + lane], 1u);
    }
    __syncthreads();
    // a digit's count: its 32 columns, each thread from another one on (no bank conflicts); cleared for the next pass
    if (tid < 256) {
      uint32_t n = 0;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        uint32_t* at = &count_s[tid * 32 + (i + tid) % 32];
        n += *at;
        *at = 0;
      }
      block_s[tid] = n;
    }
    cluster_sync(size);
    uint32_t n = 0;
    if (tid < 256) {  // digit 255 - tid: from the largest down
      if (size == 1) {
        n = block_s[255 - tid];
      } else {
        uint32_t c[kMaxBlocks];
#pragma unroll
        for (int r = 0; r < kMaxBlocks; ++r) c[r] = r < size ? remote(&block_s[255 - tid], r) : 0;
#pragma unroll
        for (int r = 0; r < kMaxBlocks; ++r) n += c[r];
      }
    }
    uint32_t in = n;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += x;
    }
    if (tid < 256 && lane == 31) sum_s[warp] = in;
    __syncthreads();
    if (tid < 256) {
#pragma unroll
      for (int i = 0; i < 8; ++i) in += i < warp ? sum_s[i] : 0;
      if (in >= need && in - n < need) digit_s = 255 - tid, above_s = in - n, within_s = n;
    }
    cluster_sync(size);  // (also: every block has read the counts)
    need -= above_s;
    border |= digit_s << shift;
    mask |= 0xffu << shift;
    if (within_s == need) break;  // all of them: no further digit decides
  }
  // kept are: the first, the last, what is above the border and, of what lies on it (under the mask), `need`
  // ---- how many of each before this warp's pages
  auto classes = [&](int p, bool (&sure)[2], bool (&tie)[2]) {
    const uint2 w = orders(p);
    const int t = p * kPage + 2 * lane;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = (i ? w.y : w.x) & mask;
      const bool open = (uint32_t)(t + i - lo) < range;
      tie[i] = open && some && x == border;
      sure[i] = open ? some && x > border : t + i < len;
    }
  };
  uint32_t n_sure = 0, n_tie = 0, first = 0x7fffffffu;  // first: page of a row that may go
#pragma unroll 2
  for (int p = p0; p < p1; ++p) {
    bool sure[2], tie[2];
    classes(p, sure, tie);
    n_sure += sure[0] + sure[1], n_tie += tie[0] + tie[1];
    if (!(sure[0] && sure[1])) first = min(first, (uint32_t)p);
  }
  first = __reduce_min_sync(0xffffffffu, first);
  n_sure = __reduce_add_sync(0xffffffffu, n_sure), n_tie = __reduce_add_sync(0xffffffffu, n_tie);
  if (lane == 0) {
    warp_s[warp] = make_uint2(n_sure, n_tie);
    atomicAdd(&total_s[0], n_sure), atomicAdd(&total_s[1], n_tie);
    atomicMin(&first_s, first);
  }
  cluster_sync(size);
  uint32_t sure0 = 0, tie0 = 0;
  {
    uint32_t c[kMaxBlocks], d[kMaxBlocks], f[kMaxBlocks];
#pragma unroll
    for (int r = 0; r < kMaxBlocks; ++r) {
      c[r] = r < rank ? remote(&total_s[0], r) : 0, d[r] = r < rank ? remote(&total_s[1], r) : 0;
      f[r] = size > 1 && r < size ? remote(&first_s, r) : 0x7fffffffu;
    }
    first = size > 1 ? f[0] : first_s;
#pragma unroll
    for (int r = 0; r < kMaxBlocks; ++r) sure0 += c[r], tie0 += d[r], first = min(first, f[r]);
  }
#pragma unroll
  for (int i = 0; i < kWarps; ++i) sure0 += i < warp ? warp_s[i].x : 0, tie0 += i < warp ? warp_s[i].y : 0;
  // (every row of a page before `first` stays where it is; some go, so there is one.  Behind it those of a page may still, where
  // weights are equal to the border.)
  if (rank == 0 && tid == 0) base_s = atomicAdd(a.count, max(0, filled - (int)first));
  // ---- their places
  int2 *from = a.from + (int64_t)row * a.n_keep, *waits = a.waits + (int64_t)row * stride;
  uint32_t at = sure0 + min(tie0, need);
  int at_lane = 0, how_lane = 0;  // where the warp's pages lie and their scales, 32 at a time, a lane a page
#pragma unroll 1
  for (int p = p0; p < p1; ++p) {
    if ((p - p0) % 32 == 0 && p + lane < p1) {
      at_lane = fetch(table + p + lane) * H + h;
      how_lane = how_of(0, fetch(reinterpret_cast<const uint2*>(a.c.scales + (int64_t)at_lane * 2)));
    }
    const int lies = __shfl_sync(0xffffffffu, at_lane, (p - p0) % 32);
    bool sure[2], tie[2];
    classes(p, sure, tie);
    const uint32_t below = (1u << lane) - 1u;
    bool k0 = sure[0], k1 = sure[1];
    if (__any_sync(0xffffffffu, tie[0] || tie[1])) {  // (of equal weights the lower positions)
      const uint32_t t0 = __ballot_sync(0xffffffffu, tie[0]), t1 = __ballot_sync(0xffffffffu, tie[1]);
      const uint32_t mine = tie0 + __popc(t0 & below) + __popc(t1 & below);
      k0 |= tie[0] && mine < need, k1 |= tie[1] && mine + tie[0] < need;
      tie0 += __popc(t0) + __popc(t1);
    }
    const uint32_t b0 = __ballot_sync(0xffffffffu, k0), b1 = __ballot_sync(0xffffffffu, k1);
    const uint32_t to = at + __popc(b0 & below) + __popc(b1 & below);
    const int t = p * kPage + 2 * lane, how = __shfl_sync(0xffffffffu, how_lane, (p - p0) % 32) + 2 * lane;
    if (k0) kept[to] = t, from[to] = make_int2(lies, how);
    if (k1) kept[to + k0] = t + 1, from[to + k0] = make_int2(lies, how + 1);
    // a weight that goes and that no row's will take the place of (of the rows that stay the move sees to)
    if ((p + 1) * kPage > a.n_keep) {
      if (!k0 && t >= a.n_keep && t < len) mass[t] = 0.0f;
      if (!k1 && t + 1 >= a.n_keep && t + 1 < len) mass[t + 1] = 0.0f;
    }
    const uint32_t next = at + __popc(b0) + __popc(b1);
    if (lane == 0 && p < filled)
      waits[p] = at == (uint32_t)p * kPage && next == (uint32_t)(p + 1) * kPage
                     ? make_int2(kStay, 0)  // nothing to do where every row stays
                     : make_int2((int)(at / kPage), next > at ? min(p - 1, (int)((next - 1) / kPage)) : -1);
    at = next;
  }
  // ---- the pages to fill
  cluster_sync(size);
  const uint32_t base = size == 1 ? base_s : remote(&base_s, 0);
  for (int p = max(p0, (int)first) + lane; p < min(p1, filled); p += 32)
    a.todo[base + p - first] = make_int2(fetch(reinterpret_cast<const int32_t*>(waits + p)) == kStay ? kStay : row, p);
  cluster_sync(size);  // a block's shared memory outlives the others' reads
}

// The largest magnitude of four codes in a scale f, and top.
__device__ __forceinline__ float largest(uint32_t w, float f, float top) {
  float x[4];
  values4(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(x[i]) * f);
  return top;
}
__device__ __forceinline__ void copy16(void* to, const uint8_t* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// Bound: 131,072 tokens of 8 heads down to a quarter, some 49 us: 185 MB read, 62 written, 5.0 TB/s.  The four pairs of a run of eight
// tokens alternate every 16 bytes of the values (q8.cuh), so a kept row brings its pair's and, by sectors, the run's other pairs' along:
// 2.8 times the rows' bytes.
//   A block takes a page in some 8 us, of which it waits for memory most, so what counts is how much is under way: the rows are
// gathered into shared memory (24 KB a page at D = 128, the values' pairs with a half that is not used), eight pages an SM.  With
// the codes in registers (four pages an SM) 131,072 tokens of 8 heads brought down to a quarter took 75 us to move, now some 49.
template <int D>
__global__ void __launch_bounds__(kMoveThreads, kMoveBlocks) move_kernel(EvictArgs a) {
  using L = Layout<D>;
  constexpr int kS = L::kSides, kWarps = kMoveThreads / 32, kChunks = kPage * D / 16;  // of 16 bytes, in a page's half
  __shared__ __align__(16) uint8_t keys_s[L::kHalf];
  __shared__ __align__(16) uint8_t values_s[2][L::kHalf];  // the chunks that a pair's first and second token lie in
  __shared__ int2 from[kPage];                             // a row's (page, head) and how it lies there
  __shared__ uint32_t top_s[2][kWarps], weight_s[kPage];
  __shared__ int2 next_s;
  const int tid = threadIdx.x, H = a.c.h_kv, stride = a.c.page_stride;
  after_previous();
  const int total = fetch(a.count);
  constexpr int kNone = -1;
  auto todo = [&](int ticket) { return ticket < total ? a.todo[ticket] : make_int2(kNone, 0); };
  // this thread's row of a page: where it lies, and its position
  auto look_up = [&](const int2& page, int2& lies, int& t) {
    if (page.x >= 0 && tid < min(kPage, a.n_keep - page.y * kPage)) {
      const int64_t at = (int64_t)page.x * a.n_keep + page.y * kPage + tid;
      lies = a.from[at], t = a.kept[at];
    }
  };
  if (tid == 0) next_s = todo(atomicAdd(a.count + 1, 1));
  __syncthreads();
  int2 what = next_s, lies = make_int2(0, 0);
  int t = 0;
  look_up(what, lies, t);
  const bool one = total <= (int)gridDim.x;  // a page a block at most
  bool ok = true;
#pragma unroll 1
  while (what.x != kNone) {
    const int row = what.x, p = what.y, n = row == kStay ? 0 : min(kPage, a.n_keep - p * kPage);  // rows that come here
    if (tid < n) from[tid] = lies;  // (behind a barrier since the page before was written)
    __syncthreads();
    if (row == kStay) {
      if (one) break;
      if (tid == 0) next_s = todo(atomicAdd(a.count + 1, 1));
      __syncthreads();
      what = next_s;
      look_up(what, lies, t);
      continue;
    }
    float* mass = a.mass + (int64_t)row * a.mass_stride;
    int32_t* flags = a.flags + (int64_t)row * stride;
#pragma unroll 4
    for (int u = tid; u < kChunks; u += kMoveThreads) {  // 16 channels of a token
      const int t = u / (D / 16), j = u % (D / 16) / 4, c = u % 4 * 2;
      const int2 f = from[t];
      if (t < n) copy16(keys_s + L::key_at(t, j, c), a.c.pages + (int64_t)f.x * L::kBytes + L::key_at(slot_of(f.y), j, c));
    }
#pragma unroll 4
    for (int u = tid; u < kChunks; u += kMoveThreads) {  // eight channels of a token pair
      const int q = u / (32 * kS) * 4 + u % 4, j = u / 32 % kS, g = u % 32 / 4;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int2 f = from[2 * q + s];
        if (2 * q + s < n)
          copy16(values_s[s] + 16 * u, a.c.pages + (int64_t)f.x * L::kBytes + L::kHalf + L::value_at(slot_of(f.y) / 2, j, g));
      }
    }
    uint32_t m = 0;
    if (tid < n) m = fetch(reinterpret_cast<const uint32_t*>(mass + t));
    const int to = fetch(a.c.page_table + (int64_t)(row / H) * stride + p) * H + row % H;
    const int2 wait = a.waits[(int64_t)row * stride + p];
    // of the lower pages that have rows of theirs here, two at most (a page's rows go to at most 64 places in a row), a thread each: have
    // they been read?  (acquire: what this block writes behind it comes after the reads that the flag tells of)
    auto read = [&](int l) {
      int seen;
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(flags + l) : "memory");
      return seen != 0;
    };
    bool seen = wait.x + tid > wait.y || read(wait.x + tid);
    if (tid < n) {
      weight_s[tid] = m;
      if (t >= a.n_keep) mass[t] = 0.0f;  // (this row's alone)
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // every row and weight has been read
    // (release: with the barrier before it the reads of all threads come before the flag.  With relaxed accesses, here and where
    // blocks that are done are counted, which leave the order to the hardware, 16 x 4,160 tokens take 39.6 us where they now take
    // 41.1, 131,072 to a quarter 77 for 79, small ragged rows 19.8 for 16.8)
    const bool withheld = a.withhold && (p + row % H) % a.withhold == 0;
    if (tid == 0 && !withheld) asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(flags + p), "r"(1) : "memory");
    float top[2] = {0.0f, 0.0f};
#pragma unroll 2
    for (int u = tid; u < kChunks; u += kMoveThreads) {
      const int t = u / (2 * D / 16) * 2 + u / 4 % 2;  // (in the order of the page)
      if (t >= n) continue;
      const uint4 c = reinterpret_cast<const uint4*>(keys_s)[u];
      const float f = key_scale(from[t].y);
      top[0] = largest(c.x, f, largest(c.y, f, largest(c.z, f, largest(c.w, f, top[0]))));
    }
    // a token's eight codes of its chunk
    auto codes_of = [&](int u, int s, int how) {
      const uint32_t pick = how & 1 ? 0x7531u : 0x6420u;
      const uint4 w = reinterpret_cast<const uint4*>(values_s[s])[u];
      return make_uint2(__byte_perm(w.x, w.y, pick), __byte_perm(w.z, w.w, pick));
    };
#pragma unroll 2
    for (int u = tid; u < kChunks; u += kMoveThreads) {
      const int t = (u / (32 * kS) * 4 + u % 4) * 2;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (t + s >= n) continue;
        const int how = from[t + s].y;
        const uint2 c = codes_of(u, s, how);
        const float f = value_scale(how);
        top[1] = largest(c.x, f, largest(c.y, f, top[1]));
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(top[s]));
      if (tid % 32 == 0) top_s[s][tid / 32] = w;
    }
    if (!seen) {
      const long long t0 = clock64();
      while (!(seen = read(wait.x + tid)) && clock64() - t0 < a.wait_cycles) {
      }
    }
    ok = __syncthreads_and(seen);
    if (!ok) break;
    // The next ticket, not before: a page that is taken and not yet read holds up the pages above it.  (With the ticket taken
    // while this page's rows were on their way 52.5 us where it now takes 40.7 for 16 x 4,160 tokens.)
    int ticket = 0;
    if (tid == 0 && !one) ticket = atomicAdd(a.count + 1, 1);
    if (tid < n) mass[p * kPage + tid] = __uint_as_float(weight_s[tid]);
    uint32_t w[2] = {top_s[0][0], top_s[1][0]};
#pragma unroll
    for (int i = 1; i < kWarps; ++i) w[0] = max(w[0], top_s[0][i]), w[1] = max(w[1], top_s[1][i]);
    const int ke = exponent_for(__uint_as_float(w[0])), ve = exponent_for(__uint_as_float(w[1]));
    uint8_t* page = a.c.pages + (int64_t)to * L::kBytes;
    if (tid == 0) *reinterpret_cast<float2*>(a.c.scales + (int64_t)to * 2) = make_float2(two_to(ke), two_to(ve));
    const float kf = two_to(-ke), vf = two_to(-ve);
    // (what is left of the last page: zero)
#pragma unroll 2
    for (int u = tid; u < kChunks; u += kMoveThreads) {
      const int t = u / (2 * D / 16) * 2 + u / 4 % 2;
      uint4 c = t < n ? reinterpret_cast<const uint4*>(keys_s)[u] : make_uint4(0, 0, 0, 0);
      const float f = t < n ? key_scale(from[t].y) * kf : 1.0f;
      if (f != 1.0f) c = make_uint4(rescaled(c.x, f), rescaled(c.y, f), rescaled(c.z, f), rescaled(c.w, f));
      reinterpret_cast<uint4*>(page)[u] = c;
    }
#pragma unroll 2
    for (int u = tid; u < kChunks; u += kMoveThreads) {
      const int t = (u / (32 * kS) * 4 + u % 4) * 2;
      uint2 c[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int how = from[t + s].y;
        c[s] = t + s < n ? codes_of(u, s, how) : make_uint2(0, 0);
        const float f = t + s < n ? value_scale(how) * vf : 1.0f;
        if (f != 1.0f) c[s] = make_uint2(rescaled(c[s].x, f), rescaled(c[s].y, f));
      }
      reinterpret_cast<uint4*>(page + L::kHalf)[u] =
          make_uint4(__byte_perm(c[0].x, c[1].x, 0x5140), __byte_perm(c[0].x, c[1].x, 0x7362), __byte_perm(c[0].y, c[1].y, 0x5140),
                     __byte_perm(c[0].y, c[1].y, 0x7362));
    }
    if (one) break;
    if (tid == 0) next_s = todo(ticket);
    __syncthreads();
    what = next_s;
    look_up(what, lies, t);
  }
  // the last block to end leaves the counters as it found them
  __syncthreads();
  if (tid == 0) {
    if (!ok) raise(a.c, RDKV_ERR_TIMEOUT);
    // (acquire and release: the counters are cleared behind what every other block has read of them and added to them)
    int done;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(done) : "l"(a.count + 2) : "memory");
    if (done == (int)gridDim.x - 1) a.count[0] = a.count[1] = a.count[2] = 0;
  }
}

struct EvictLayout {
  size_t flags_at, waits_at, todo_at, from_at, bytes;
};
static EvictLayout evict_layout(const rdkv_q8_cache* c) {
  const int64_t pages = (int64_t)c->batch * c->h_kv * c->page_stride;
  EvictLayout o;
  o.flags_at = kCounterBytes;
  o.waits_at = o.flags_at + (size_t)align_up(4 * pages, 256);
  o.todo_at = o.waits_at + (size_t)align_up(8 * pages, 256);
  o.from_at = o.todo_at + (size_t)align_up(8 * pages, 256);
  // (rows are kept only of sequences that hold more: n_keep is then below what a table holds)
  o.bytes = o.from_at + (size_t)align_up(8 * pages * kPage, 256);
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

// withhold > 0: the self-test
static rdkv_status evict_impl(const rdkv_q8_cache* cache, float* mass, int64_t mass_stride, int32_t n_keep, int32_t n_first, int32_t n_last,
                              int32_t* kept, void* ws, size_t ws_bytes, void* stream, int withhold, long long wait_cycles) {
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
  const EvictArgs a{q8::view_of(cache), mass, mass_stride, n_keep, n_first, n_last, kept, reinterpret_cast<int2*>(w + lay.from_at),
                    reinterpret_cast<int32_t*>(w + lay.flags_at), reinterpret_cast<int2*>(w + lay.waits_at), reinterpret_cast<int2*>(w + lay.todo_at),
                    reinterpret_cast<int32_t*>(w), withhold, wait_cycles};
  cudaStream_t cs = (cudaStream_t)stream;
  const int rows = cache->batch * cache->h_kv;
  // blocks of a row: a warp has kSplit pages before the row takes another block
  constexpr int kWarps = kPickThreads / 32;
  int size = 1;
  while (size < kMaxBlocks && size * kWarps * kSplit < cache->page_stride) size *= 2;
  const int hold = std::min(kHold, ceil_div(cache->page_stride, size * kWarps));
  static std::atomic<uint64_t> ready{0};  // once a device (of the first 64; the others pay for the call every time)
  int dev = 0;
  RDKV_TRY_CUDA(cudaGetDevice(&dev), "8-bit cache eviction");
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    RDKV_TRY_CUDA(cudaFuncSetAttribute(pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * kHold * 256), "8-bit cache eviction");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * size), cfg.blockDim = dim3(kPickThreads), cfg.stream = cs, cfg.dynamicSmemBytes = kWarps * hold * 256;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 2;
  RDKV_TRY_CUDA(cudaLaunchKernelEx(&cfg, pick_kernel, a, hold), "8-bit cache eviction");
  count_launch();
  const int64_t pages = (int64_t)rows * std::min<int64_t>(cache->page_stride, ceil_div64(n_keep, kPage));
  const unsigned grid = (unsigned)std::min<int64_t>(pages, (int64_t)num_sms() * kMoveBlocks);
  auto move = cache->head_dim == 128 ? move_kernel<128> : move_kernel<64>;
  RDKV_TRY_CUDA(launch_after(move, dim3(grid), kMoveThreads, 0, cs, a), "8-bit cache eviction");
  count_launch();
  return RDKV_OK;
}

extern "C" rdkv_status rdkv_q8_evict(const rdkv_q8_cache* cache, float* mass, int64_t mass_stride, int32_t n_keep, int32_t n_first,
                                     int32_t n_last, int32_t* kept, void* ws, size_t ws_bytes, void* stream) {
  return evict_impl(cache, mass, mass_stride, n_keep, n_first, n_last, kept, ws, ws_bytes, stream, 0, kWaitCycles);
}

extern "C" rdkv_status rdkv_q8_evict_timeout_selftest(const rdkv_q8_cache* cache, float* mass, int64_t mass_stride, int32_t n_keep,
                                                      int32_t n_first, int32_t n_last, int32_t* kept, void* ws, size_t ws_bytes,
                                                      int32_t withhold, int64_t wait_cycles, void* stream) {
  RDKV_REQUIRE(withhold >= 1, RDKV_ERR_INVALID_ARG, "withhold %d must be positive", withhold);
  RDKV_REQUIRE(wait_cycles > 0, RDKV_ERR_INVALID_ARG, "wait_cycles %lld must be positive", (long long)wait_cycles);
  return evict_impl(cache, mass, mass_stride, n_keep, n_first, n_last, kept, ws, ws_bytes, stream, withhold,
                    std::min(kWaitCycles, std::max(kMinWaitCycles, (long long)wait_cycles)));
}
