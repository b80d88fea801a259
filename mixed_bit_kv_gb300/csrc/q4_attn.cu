// Attention over the 4-bit paged cache (rdkv_q4_attn).
//
//   logits  s_t = (q . k^_t) / sqrt(D),  k^ = zero + scale code per group of 32 channels, so
//           q . k^_t = sum_grp scale_t,grp (sum_c q_c code_t,c) + sum_grp zero_t,grp (sum_c q_c)
//   out     = sum_t p_t v^_t / sum_t p_t,  p_t = 2^(s_t log2 e - ref), the values by the same split
//
// Work.  A unit is (sequence, chunk of query tokens, KV head): up to 8 NT query rows, NT = 1 or 2, that
// share the unit's keys; an item is one page (64 tokens) of a unit.  The items of all units, one after
// another, are dealt evenly to the warps of the grid (one block of eight warps an SM): each warp takes a run
// of items and works alone, copying pages into its own ring of two with bulk copies, so that no barrier
// stands between the pages.  Units that end inside a warp's run are written by it; the pieces of the others
// are joined per block in shared memory and, where a unit spans blocks, by the last of its blocks through
// the workspace, always in the same order: the result does not depend on who comes first.
//
// Products: mma.sync, channels on M and queries on N for the values; for the logits tokens on M and queries on N
// where the unit has up to eight rows and 16-bit outputs, else queries on M (rows 8 .. 15 a second eight, or
// the first's low parts) and tokens on N.  A code at bit p < 8 of a half word is the fp16 subnormal code 2^(p - 24),
// so one AND makes two codes of the keys an operand register; the units are undone in fp32.  Each group's logits
// accumulate on their own and take the token's scale in fp32; the zeros' part is one more product, of the queries'
// group sums (fp16 high part and remainder).  The values are taken as zero + 8 scale and scale (code - 8): what
// fp16 and the tensor core (it cuts, it does not round) lose is then lost of a small sum, not of the
// difference of two large ones.  For fp32 outputs (PREC) the keys are split the same way, the middles' part
// is summed in fp32, and weight times scale keeps a remainder.
//
// Roundings.  Logits, maxima, weights' sums and outputs' sums are fp32 in every variant.  The operands of the tensor
// cores are fp16:
//   16-bit outputs  fp16 and bf16 queries as they are (a row times a power of two); a weight, once more weight times
//           scale, and the middle zero + 8 scale, 2^-11 of each: together less than the outputs' own rounding (fp16 outputs
//           are 2.1e-4 off when fp32 sums are rounded once, 2.1e-4 .. 2.4e-4 here).  Carrying them in two parts is the fp32
//           variant: 111 us for 64 at 262,144 tokens.
//   fp32 outputs  queries in two parts (22 bits of 24), weight times scale in two parts (22 bits), the middles and the
//           weights themselves in fp32: 4.4e-7 off at 513 tokens, where plain fp32 sums are 5.2e-7 off.
// A weight has those bits while its part of an operand is a normal fp16 number: 16-bit outputs down to 2^-25 of the
// largest weight where the values' scales are below 1/4, to 2^-9 at the largest scale there is (values of 65504).
//
// Bound.  160 bytes a token and KV head at D = 128: 79 % of the measured copy bandwidth at 262,144 tokens (62.8
// us for 335 MB).  A scheduler has two warps, whose products wait for one another: a page of up to eight rows takes
// 72 products (104 with the queries on M and half of its rows empty: 68.5 us).  About 1,150 instructions a page,
// a third of them to unpack codes.  Start (lengths, page table, queries, first page: each a trip to memory) and
// joins take about 10 us of every call.  Two row sets: 136 products a page, 1,600 instructions, 255 registers; the
// tensor pipe is 26 % busy and the issue slots 37 %: the latency of two warps a scheduler again, not the products' rate.
//   Measured and not kept (us at 262,144 tokens, against 68.5 .. 69): 11 or 12 warps of 168 registers 74 .. 79, 16
// of 128 74; 16 or 32 tokens under way at once 79 and 72; pages copied with the 128-byte swizzle of a tensor map,
// which takes away the values' four-fold bank conflicts (96 of 270 shared-memory cycles a page), 75 against 73; the
// same through 21 copies a page into shifted quarters, 91; the values' codes as subnormals too, less eight times the
// weights' sum by one more product a group: 128 instructions a page fewer, 16 products more, 70.4.
#include <atomic>

#include "q4.cuh"

namespace rdkv {
namespace q4 {

struct AttnArgs {
  View c;
  const void* q;
  void* out;
  float* lse;
  const int32_t* sel;
  float* heads;      // [grid * NW] partials: pieces of units that end inside a warp's run
  float* parts;      // [grid * 2] partials: a block's part of a unit that began before it, of one that goes on
  int32_t* tickets;  // [units] blocks that have written their part
  int64_t q_stride;
  int dtype, out_dtype, n_q, G, n_sel, chunk, n_chunks;  // chunk: query tokens of a unit
  int withhold;           // 0, or (the self-test) pages with (index + KV head) % withhold == 0 are waited for, not copied
  long long wait_cycles;  // limit of a wait for a page
};

constexpr int kMinItems = 4;                     // of a block (1 to 8: within 3 % of one another on the smallest calls)
constexpr int kInfo = 32;                        // items whose places a warp knows ahead

__device__ __forceinline__ void mma8z(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.0f));
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 d = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
constexpr int kRest = 4096;  // of the weights' remainders: a fp16 part of up to 2^9 leaves up to 2^-3
template <int NG>
__device__ __forceinline__ void lds_groups(const uint8_t* p, uint32_t (&w)[NG]) {
  if constexpr (NG == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}
// The same codes less eight, exactly: 1024 + code (and 1024 + 16 code) are the fp16 values of the code bits
// under the exponent of 1024.
__device__ __forceinline__ uint32_t minus(uint32_t w, uint32_t one) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&one));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(bits));
  return d;
}
// Two values of at most 2^15 (or, a sixteenth, 2^11) rounded to multiples of 16 (of 1) or of twice or four times that:
// half of the value added to 24,576 and taken off again.
__device__ __forceinline__ uint32_t whole16(uint32_t w, bool sixteenth) {
  const __half2 v = *reinterpret_cast<const __half2*>(&w), k = __float2half2_rn(24576.0f);
  const __half2 h = __hsub2(__hfma2(v, __float2half2_rn(sixteenth ? 8.0f : 0.5f), k), k);
  const __half2 d = __hmul2(h, __float2half2_rn(sixteenth ? 0.125f : 2.0f));
  return *reinterpret_cast<const uint32_t*>(&d);
}
// k1024: the exponent's bits, in a register that the compiler takes for a variable, so that mask and bits are
// one instruction (it can hold one constant only).
__device__ __forceinline__ Pairs centred_pairs(uint32_t w, uint32_t k1024) {
  const uint32_t u = w >> 8;
  constexpr uint32_t k1032 = 0x64086408u, k1152 = 0x64806480u;
  return Pairs{minus(and_or(w, 0x000f000fu, k1024), k1032), minus(and_or(w, 0x00f000f0u, k1024), k1152),
               minus(and_or(u, 0x000f000fu, k1024), k1032), minus(and_or(u, 0x00f000f0u, k1024), k1152)};
}

// A piece of a unit: ROWS x D sums and each row's reference (base 2) and sum of weights.
template <int D, int NT>
struct Partial {
  static constexpr int kRows = 8 * NT, kFloats = kRows * (D + 2);
};

// Items of (sequence, chunk) bc in each of its KV heads, and the keys that its last query token sees.
__device__ __forceinline__ int seen_by(const AttnArgs& a, int b, int chunk) {
  return held_tokens(a.c, b) - a.n_q + min((chunk + 1) * a.chunk, a.n_q);
}
__device__ __forceinline__ int items_of(const AttnArgs& a, int bc) {
  const int seen = seen_by(a, bc / a.n_chunks, bc % a.n_chunks);
  return seen <= 0 ? 0 : a.sel ? a.n_sel : ceil_div(seen, kPage);
}

// What a unit's index stands for.
struct Unit {
  int b, t0, h, rows;  // sequence, first query token, KV head, query rows
};
__device__ __forceinline__ Unit unit_at(const AttnArgs& a, int unit) {
  const int bc = unit / a.c.h_kv, b = bc / a.n_chunks, t0 = (bc - b * a.n_chunks) * a.chunk;
  return Unit{b, t0, unit - bc * a.c.h_kv, min(a.chunk, a.n_q - t0) * a.G};
}
// Output row (and place in lse) of a unit's query row.
__device__ __forceinline__ int64_t row_at(const AttnArgs& a, const Unit& u, int row) {
  const int t = row / a.G;
  return (((int64_t)u.b * a.n_q + u.t0 + t) * a.c.h_kv + u.h) * a.G + (row - t * a.G);
}
__device__ __forceinline__ void put4(const AttnArgs& a, int64_t at, float4 o) {
  if (a.out_dtype == RDKV_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = o;
  } else {
    uint2 w;
    if (a.out_dtype == RDKV_F16) {
      // a mean is no larger than the values (65504 at most), but the weights it is taken with are rounded
      w = make_uint2(cut_half2(o.x, o.y), cut_half2(o.z, o.w));
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(o.x, o.y), y = __floats2bfloat162_rn(o.z, o.w);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = w;
  }
}
// (a NaN sum, of a query that holds one, is not a sum of nothing)
__device__ __forceinline__ void put_lse(const AttnArgs& a, int64_t row, float m, float l) {
  if (a.lse) a.lse[row] = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// One warp's running state over the pages of one unit.
template <int D, int NT, bool PREC>
struct Warp {
  static constexpr int NG = D / kGroup;
  using L = Layout<D>;
  // Eight rows in 16 bits: tokens on M, queries on N for the logits too, with no rows for low parts: half as
  // many products, whose weights one transposition a tile turns into the values' operand.
  static constexpr bool kCols = NT == 1 && !PREC;
  // The query rows whose statistics a lane keeps: g (+ 8), or its columns 2 qd and 2 qd + 1.
  static constexpr int kStats = kCols ? 2 : NT;
  static __device__ __forceinline__ int stat_row(int n, int g, int qd) { return kCols ? 2 * qd + n : g + 8 * n; }

  uint32_t q[kCols ? 1 : 2][NG][4];  // operand registers: rows g, and rows g + 8 (the chunk's second half, or the low parts of the first)
  uint32_t qz[2];                    // operand registers of the zeros' product
  float qs[NG];                      // (PREC) the same sums in fp32
  float scale[kStats];               // 2^(14 - s): a row's logits are held times 2^(s - 14)
  float ref[kStats], l[kStats];      // the running maximum (base 2) and this lane's share of the sum
  float o[NT][NG][2][4];
  float oz[NT][PREC ? NG : 2];  // the zeros' part: by row g < NG = group and columns, or (PREC) this lane's row's, by group
  int off;                      // weights are held times 2^off
  // Tokens whose products are under way together: as many as the registers hold (72B-shaped layer: 64 in 62.5
  // us, 32 in 68.3; with two row sets 32 in 51.9 us on the drafted tokens, 64 spill: 63.9)
  static constexpr int kTurn = NT == 1 && !PREC ? 64 : 32;
  static constexpr int kMaxOff = PREC ? 23 : 11;

  // This lane's channels of the unit's query rows, as they lie in memory (rows past the last: zero).  Kept
  // apart from begin() so that copies can be issued while they are under way.
  struct Rows {
    uint4 w[NT][NG][2];
  };
  __device__ __forceinline__ static void queries(const AttnArgs& a, const Unit& un, int g, int qd, Rows& r) {
    const int size = a.dtype == RDKV_F32 ? 4 : 2;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = g + 8 * n, t = row / a.G;
      const bool real = row < un.rows;
      const int64_t at = ((int64_t)un.b * a.n_q + un.t0 + t) * a.q_stride + ((int64_t)un.h * a.G + row - t * a.G) * D + 8 * qd;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) + (real ? at * size : 0));
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        r.w[n][i][0] = real ? fetch(src + 2 * i * size) : make_uint4(0, 0, 0, 0);
        if (PREC) r.w[n][i][1] = real && size == 4 ? fetch(src + 2 * i * size + 1) : make_uint4(0, 0, 0, 0);
      }
    }
  }
  // (fp32 queries have fp32 outputs, so only PREC reads them)
  __device__ __forceinline__ static void widen(int dtype, const uint4 (&w)[2], float (&x)[8]) {
    const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    if (PREC && dtype == RDKV_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = dtype == RDKV_F16 ? unpack2(v[e]) : make_float2(__uint_as_float(v[e] << 16), __uint_as_float(v[e] & 0xffff0000u));
        x[2 * e] = f.x, x[2 * e + 1] = f.y;
      }
    }
  }

  __device__ __forceinline__ void begin(int dtype, const Rows& rows, int qd) {
    constexpr float kK = 1.4426950408889634f / (D == 128 ? 11.313708498984761f : 8.0f);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[NG][8], top = 0.0f;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        widen(dtype, rows.w[n][i], x[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i][e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the row times 2^s, its largest value in [2^14, 2^15): what fp16 drops is 2^-25 against that.  Down to s =
      // -113 and its inverse 2^127, so that every finite row has its place.
      const int e2 = (int)(__float_as_uint(top) >> 23) - 127;
      const int s = top > 0.0f ? max(-113, min(111, 14 - e2)) : 0;
      const float up = __uint_as_float((uint32_t)(s + 127) << 23);
      const float down = __uint_as_float((uint32_t)(14 - s + 127) << 23);
      if constexpr (kCols) {
#pragma unroll
        for (int j = 0; j < 2; ++j) scale[j] = __shfl_sync(0xffffffffu, down, 8 * qd + 4 * j);
      } else {
        scale[n] = down;
      }
      float sum[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        sum[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= up, sum[i] += x[i][e];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // pairs 1 and 3 meet codes that stand for sixteen times as much
          const float f = j & 1 ? 0.0625f : 1.0f, y0 = x[i][2 * j] * f, y1 = x[i][2 * j + 1] * f;
          q[n][i][j] = pack2(y0, y1);
          if constexpr (PREC) q[1][i][j] = rest2(y0, y1, q[0][i][j]);
        }
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        sum[i] *= kK / 16384.0f;
      }
      if constexpr (PREC) {
#pragma unroll
        for (int i = 0; i < NG; ++i) qs[i] = sum[i];
      }
      // k slots 0 .. NG - 1: the sums' fp16 parts, the next NG: the remainders
      uint32_t hi[NG / 2], lo[NG / 2];
#pragma unroll
      for (int i = 0; i < NG / 2; ++i) {
        hi[i] = pack2(sum[2 * i], sum[2 * i + 1]);
        lo[i] = rest2(sum[2 * i], sum[2 * i + 1], hi[i]);
      }
      if constexpr (NT == 1) qz[1] = 0u;
      if constexpr (NG == 4) qz[n] = qd == 0 ? hi[0] : qd == 1 ? hi[1] : qd == 2 ? lo[0] : lo[1];
      else qz[n] = qd == 0 ? hi[0] : qd == 1 ? lo[0] : 0u;
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) o[n][i][j / 4][j % 4] = 0.0f;
#pragma unroll
      for (int j = 0; j < (PREC ? NG : 2); ++j) oz[n][j] = 0.0f;
    }
#pragma unroll
    for (int n = 0; n < kStats; ++n) ref[n] = -INFINITY, l[n] = 0.0f;
    off = kMaxOff;
  }

  // Row sums and weighted sums times f, each lane's row's own (of its columns: f and g).
  __device__ __forceinline__ void rescale(int n, float f, float g, int qd) {
    l[n] *= f;
    if constexpr (kCols) l[1] *= g;
    // columns 2 qd and 2 qd + 1 of the sums are rows that lanes 8 qd and 8 qd + 4 keep
    const float f0 = kCols ? f : __shfl_sync(0xffffffffu, f, 8 * qd), f1 = kCols ? g : __shfl_sync(0xffffffffu, f, 8 * qd + 4);
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        o[n][i][m][0] *= f0, o[n][i][m][1] *= f1, o[n][i][m][2] *= f0, o[n][i][m][3] *= f1;
    if constexpr (PREC) {
#pragma unroll
      for (int i = 0; i < NG; ++i) oz[n][i] *= f;
    } else {
      oz[n][0] *= f0, oz[n][1] *= f1;
    }
  }

  // (kCols) The tensor core cuts its sums some 2^-23 below their largest product: 1e-5 of a logit of fp16 queries.  Long
  // rows average that away; one of a single page may not, so its queries are taken in two parts: multiples of 16 (their
  // largest value is 2^15), whose products and sums with codes are all whole, and what that leaves.  This takes the
  // second part's logits (base 2, times 2^(s - 14), in the order of page()) to r and leaves the first in q.  (lse of
  // one or two tokens: 4e-7 off instead of 1.4e-6.  With two row sets its code costs 5 % on drafted tokens.)
  __device__ __forceinline__ void split(const uint8_t* k, float2* r, int g, int qd) {
    constexpr float kK = 16777216.0f / 16384.0f * 1.4426950408889634f / (D == 128 ? 11.313708498984761f : 8.0f);
    auto left = [&](int i, int j) { return minus(q[0][i][j], whole16(q[0][i][j], j & 1)); };
#pragma unroll 1
    for (int t = 0; t < kPage / 8; ++t) {  // eight tokens, on the upper half of M
      uint32_t w[NG], sw[NG];
      lds_groups<NG>(k + L::kKCodes + ((8 * t + g) * 4 + qd) * NG * 4, w);
      lds_groups<NG>(k + L::kKScales + (8 * t + g) / 2 * NG * 4, sw);
      float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const Pairs p = code_pairs(w[i]);
        const float2 f = unpack2(sw[i]);
        float c[4];
        mma16z(c, p.a, 0u, p.b, 0u, left(i, 0), left(i, 1));
        mma16(c, p.c, 0u, p.d, 0u, left(i, 2), left(i, 3));
        s.x = fmaf(g & 1 ? f.y : f.x, c[0], s.x), s.y = fmaf(g & 1 ? f.y : f.x, c[1], s.y);
      }
      r[t * 32 + 4 * g + qd] = make_float2(s.x * kK, s.y * kK);
    }
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) q[0][i][j] = whole16(q[0][i][j], j & 1);
  }

  // One page.  cut (the same in all lanes): its last tokens may hold nothing (live of them do; what the others
  // hold is arbitrary bits, which logits and values must not meet) or be hidden from some rows (row n of this
  // lane sees low[n] of the page's tokens), or it is (only) the unit's one page.  One body for all pages: it runs once or a few times a call, and the
  // time to fetch a second one shows.
  __device__ __forceinline__ void page(uint8_t* k, const float2* r, int g, int qd, bool cut, bool only, int live, const int (&low)[kStats]) {
    if (cut) {
      const int lane = 4 * g + qd;
      if (2 * lane + 1 >= live) {  // the values' scales and zeros of tokens that hold nothing: zero
        const uint32_t keep = 2 * lane < live ? 0xffffu : 0u;
        uint32_t* w = reinterpret_cast<uint32_t*>(k + L::kVScales) + lane * NG;
#pragma unroll
        for (int i = 0; i < NG; ++i) w[i] &= keep, w[i + L::kMeta / 4] &= keep;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy into the stage
      __syncwarp();
    }
    constexpr float kUnit = PREC ? 1.0f : 16777216.0f;  // of the codes in the products
    constexpr float kK = kUnit / 16384.0f * 1.4426950408889634f / (D == 128 ? 11.313708498984761f : 8.0f);
    uint32_t k1024;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));
    {  // The weights' exponent follows the largest value scale met, so that weight times scale stays in
       // fp16's range: with the weight at most 2^(4 + off) and the scale below 2^(e + 1), the product is
       // below 2^13, and off <= 11 keeps the weight itself in range.  (PREC: weights at most 2^off, products
       // below 2^9.)
      const int lane = 4 * g + qd;
      uint32_t sw[NG], top = 0;
      lds_groups<NG>(k + L::kVScales + lane * NG * 4, sw);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        top = __vmaxu2(top, sw[i]);
      }
      top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
      const int now = min(off, 23 - (int)(top >> 10));
      if (now < off) {
        const float f = __uint_as_float((uint32_t)(now - off + 127) << 23);
#pragma unroll
        for (int n = 0; n < NT; ++n) rescale(n, f, f, qd);
        off = now;
      }
    }
#pragma unroll 1
    for (int t32 = 0; t32 < kPage; t32 += kTurn) {
      // logits (base 2, times 2^(s - 14)): of tokens t32 + 8 t + 2 qd + {0, 1}, or (kCols) of token t32 + 8 t + g
      // and both columns
      float2 u[NT][kTurn / 8];
      if constexpr (kCols) {
#pragma unroll
        for (int t = 0; t < kTurn / 8; t += 2) {
          const int tok = t32 + 8 * t + g;
          uint32_t w0[NG], w1[NG], s0[NG], s1[NG];
          lds_groups<NG>(k + L::kKCodes + (tok * 4 + qd) * NG * 4, w0);
          lds_groups<NG>(k + L::kKCodes + ((tok + 8) * 4 + qd) * NG * 4, w1);
          lds_groups<NG>(k + L::kKScales + tok / 2 * NG * 4, s0);
          lds_groups<NG>(k + L::kKScales + (tok / 2 + 4) * NG * 4, s1);
          const uint32_t* zw = reinterpret_cast<const uint32_t*>(k + L::kKZeros) + tok * (NG / 2) + (NG == 4 ? qd & 1 : 0);
          float z[4];
          mma8z(z, zw[0], zw[8 * (NG / 2)], qz[0]);
          float2 a0 = make_float2(0.0f, 0.0f), a1 = a0;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const Pairs x = code_pairs(w0[i]), y = code_pairs(w1[i]);
            float c[4];
            mma16z(c, x.a, y.a, x.b, y.b, q[0][i][0], q[0][i][1]);
            mma16(c, x.c, y.c, x.d, y.d, q[0][i][2], q[0][i][3]);
            const float2 f = unpack2(__byte_perm(s0[i], s1[i], g & 1 ? 0x7632 : 0x5410));  // tokens tok and tok + 8
            a0.x = fmaf(f.x, c[0], a0.x), a0.y = fmaf(f.x, c[1], a0.y);
            a1.x = fmaf(f.y, c[2], a1.x), a1.y = fmaf(f.y, c[3], a1.y);
          }
          u[0][t] = fma2(a0, make_float2(kK, kK), make_float2(z[0], z[1]));
          u[0][t + 1] = fma2(a1, make_float2(kK, kK), make_float2(z[2], z[3]));
        }
      }
#pragma unroll
      for (int t = 0; !kCols && t < kTurn / 8; ++t) {
        const int tok = t32 + 8 * t;
        uint32_t w[NG], sw[NG];
        lds_groups<NG>(k + L::kKCodes + ((tok + g) * 4 + qd) * NG * 4, w);
        lds_groups<NG>(k + L::kKScales + (tok / 2 + qd) * NG * 4, sw);
        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (PREC) {  // the keys' middles (zero + 8 scale), in fp32
          uint32_t zw[NG];
          lds_groups<NG>(k + L::kKZeros + (tok + 2 * qd) * NG * 2, zw);
#pragma unroll
          for (int i = 0; i < NG; ++i) {  // words 0 .. NG / 2 - 1: the even token's groups in pairs, then the odd one's
            const float2 f = unpack2(sw[i]), e = unpack2(zw[i / 2]), o = unpack2(zw[NG / 2 + i / 2]);
            z[0] = fmaf(fmaf(8.0f, f.x, i & 1 ? e.y : e.x), qs[i], z[0]);
            z[1] = fmaf(fmaf(8.0f, f.y, i & 1 ? o.y : o.x), qs[i], z[1]);
          }
        } else {
          mma8z(z, qz[0], qz[1], reinterpret_cast<const uint32_t*>(k + L::kKZeros)[(tok + g) * (NG / 2) + (NG == 4 ? qd & 1 : 0)]);
        }
        float2 s[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const Pairs p = PREC ? centred_pairs(w[i], k1024) : code_pairs(w[i]);
          constexpr int k1 = kCols ? 0 : 1;
          float c[4];
          mma16z(c, q[0][i][0], q[k1][i][0], q[0][i][1], q[k1][i][1], p.a, p.b);
          mma16(c, q[0][i][2], q[k1][i][2], q[0][i][3], q[k1][i][3], p.c, p.d);
          const float2 f = unpack2(sw[i]);
          if constexpr (PREC) c[0] += c[2], c[1] += c[3];
          s[0] = fma2(f, make_float2(c[0], c[1]), s[0]);
          if constexpr (NT == 2) s[1] = fma2(f, make_float2(c[2], c[3]), s[1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          u[n][t] = fma2(s[n], make_float2(kK, kK), make_float2(z[2 * n], z[2 * n + 1]));
        }
      }
      if (cut) {
        if constexpr (kCols) {
          if (only) {
#pragma unroll
            for (int t = 0; t < kTurn / 8; ++t) u[0][t] = add2f(u[0][t], r[(t32 / 8 + t) * 32 + 4 * g + qd]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int t = 0; t < kTurn / 8; ++t) {
            const int tok = t32 + 8 * t + (kCols ? g : 2 * qd);
            if (tok >= low[n]) u[n][t].x = -INFINITY;
            if (tok + (kCols ? 0 : 1) >= low[kCols ? kStats - 1 : n]) u[n][t].y = -INFINITY;
          }
      }
      // a row's reference rises when a logit passes it by more than 4, so that weights stay at most 2^4
      // (PREC: whenever one passes it)
      if constexpr (kCols) {
        float m0 = u[0][0].x, m1 = u[0][0].y;
#pragma unroll
        for (int t = 1; t < kTurn / 8; ++t) m0 = fmaxf(m0, u[0][t].x), m1 = fmaxf(m1, u[0][t].y);
        m0 *= scale[0], m1 *= scale[kStats - 1];
        if (__any_sync(0xffffffffu, m0 > ref[0] + 4.0f || m1 > ref[kStats - 1] + 4.0f)) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
          }
          m0 = fmaxf(m0, ref[0]), m1 = fmaxf(m1, ref[kStats - 1]);
          const float f0 = ref[0] == -INFINITY ? 0.0f : ex2(ref[0] - m0);
          const float f1 = ref[kStats - 1] == -INFINITY ? 0.0f : ex2(ref[kStats - 1] - m1);
          ref[0] = m0, ref[kStats - 1] = m1;
          rescale(0, f0, f1, qd);
        }
      }
#pragma unroll
      for (int n = 0; !kCols && n < NT; ++n) {
        float m = fmaxf(u[n][0].x, u[n][0].y);
#pragma unroll
        for (int t = 1; t < kTurn / 8; ++t) m = fmaxf(m, fmaxf(u[n][t].x, u[n][t].y));
        m *= scale[n];
        if (__any_sync(0xffffffffu, m > ref[n] + (PREC ? 0.0f : 4.0f))) {
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          m = fmaxf(m, ref[n]);
          const float f = ref[n] == -INFINITY ? 0.0f : ex2(ref[n] - m);
          ref[n] = m;
          rescale(n, f, f, qd);
        }
      }
      // the weights, in fp16 too, in the order of the values' products: 16 tokens a step
      uint32_t hi[NT][kTurn / 16][2], s0[kTurn / 16][NG], s1[kTurn / 16][NG], w0[kTurn / 16][NG], w1[kTurn / 16][NG];
      float p[NT][kTurn / 16][4], cz[NT][4];
#pragma unroll
      for (int t = 0; t < kTurn / 16; ++t) {
        const int p0 = t32 / 2 + 8 * t + qd, p1 = p0 + 4;  // this lane's token pairs
        lds_groups<NG>(k + L::kVCodes + (p0 * 8 + g) * NG * 4, w0[t]);
        lds_groups<NG>(k + L::kVCodes + (p1 * 8 + g) * NG * 4, w1[t]);
        lds_groups<NG>(k + L::kVScales + p0 * NG * 4, s0[t]);
        lds_groups<NG>(k + L::kVScales + p1 * NG * 4, s1[t]);
        if constexpr (kCols) {
          const float2 r = make_float2((float)off - (ref[0] == -INFINITY ? 0.0f : ref[0]),
                                       (float)off - (ref[kStats - 1] == -INFINITY ? 0.0f : ref[kStats - 1]));
          const float2 up = make_float2(scale[0], scale[kStats - 1]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const float2 y = fma2(u[0][2 * t + m], up, r), x = make_float2(ex2(y.x), ex2(y.y));
            l[0] += x.x, l[kStats - 1] += x.y;
            hi[0][t][m] = transposed(pack2(x.x, x.y));
          }
        }
#pragma unroll
        for (int n = 0; !kCols && n < NT; ++n) {
          const float r = (float)off - (ref[n] == -INFINITY ? 0.0f : ref[n]);
          const float2 y0 = fma2(u[n][2 * t], make_float2(scale[n], scale[n]), make_float2(r, r));
          const float2 y1 = fma2(u[n][2 * t + 1], make_float2(scale[n], scale[n]), make_float2(r, r));
          float(&x)[4] = p[n][t];
          x[0] = ex2(y0.x), x[1] = ex2(y0.y), x[2] = ex2(y1.x), x[3] = ex2(y1.y);
          l[n] += (x[0] + x[1]) + (x[2] + x[3]);
        }
        if constexpr (PREC) {  // the values' middles (zero + 8 scale), in fp32
          uint32_t z0[NG], z1[NG];
          lds_groups<NG>(k + L::kVZeros + p0 * NG * 4, z0);
          lds_groups<NG>(k + L::kVZeros + p1 * NG * 4, z1);
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const float2 a0 = unpack2(z0[i]), a1 = unpack2(z1[i]), f0 = unpack2(s0[t][i]), f1 = unpack2(s1[t][i]);
            const float(&x)[4] = p[0][t];
            oz[0][i] += (x[0] * fmaf(8.0f, f0.x, a0.x) + x[1] * fmaf(8.0f, f0.y, a0.y)) +
                        (x[2] * fmaf(8.0f, f1.x, a1.x) + x[3] * fmaf(8.0f, f1.y, a1.y));
          }
        } else {  // the same as one product of the middles in fp16 (rows g >= NG of its operand are not used)
          const uint32_t *zs = reinterpret_cast<const uint32_t*>(k + L::kVZeros) + g % NG, *ss = zs - L::kMeta / 4;
          const uint32_t z0 = hfma2(ss[p0 * NG], 0x48004800u, zs[p0 * NG]);
          const uint32_t z1 = hfma2(ss[p1 * NG], 0x48004800u, zs[p1 * NG]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float(&x)[4] = p[n][t];
            if constexpr (!kCols) hi[n][t][0] = pack2(x[0], x[1]), hi[n][t][1] = pack2(x[2], x[3]);
            if (t == 0) mma16z(cz[n], z0, 0u, z1, 0u, hi[n][t][0], hi[n][t][1]);
            else mma16(cz[n], z0, 0u, z1, 0u, hi[n][t][0], hi[n][t][1]);
          }
        }
      }
      // The tensor core cuts what it adds to an accumulator: its accumulators start at zero every turn, and the
      // sums over the turns are rounded fp32 additions.  PREC: weight times scale (below 2^9) as its fp16 part and,
      // in accumulators of their own and times 2^12, the remainders: 22 bits of every product down to 2^-15, so that
      // a group of small values, or many keys of small weight, keep theirs beside the largest.
      if constexpr (!PREC) {
#pragma unroll
        for (int n = 0; n < NT; ++n) oz[n][0] += cz[n][0], oz[n][1] += cz[n][1];
      }
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        float c[NT][2][4], rest[PREC ? 2 : 1][4];
#pragma unroll
        for (int t = 0; t < kTurn / 16; ++t) {
          const Pairs x = centred_pairs(w0[t][i], k1024), y = centred_pairs(w1[t][i], k1024);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint32_t b0, b1;
            if constexpr (PREC) {
              const float2 f0 = unpack2(s0[t][i]), f1 = unpack2(s1[t][i]);
              const float e0 = p[n][t][0] * f0.x, e1 = p[n][t][1] * f0.y, e2 = p[n][t][2] * f1.x, e3 = p[n][t][3] * f1.y;
              b0 = pack2(e0, e1), b1 = pack2(e2, e3);
              const uint32_t c0 = rest2<kRest>(e0, e1, b0), c1 = rest2<kRest>(e2, e3, b1);
              if (t == 0) {
                mma16z(rest[0], x.a, x.b, y.a, y.b, c0, c1);
                mma16z(rest[1], x.c, x.d, y.c, y.d, c0, c1);
              } else {
                mma16(rest[0], x.a, x.b, y.a, y.b, c0, c1);
                mma16(rest[1], x.c, x.d, y.c, y.d, c0, c1);
              }
            } else {
              b0 = hmul2(hi[n][t][0], s0[t][i]), b1 = hmul2(hi[n][t][1], s1[t][i]);
            }
            if (t == 0) {
              mma16z(c[n][0], x.a, x.b, y.a, y.b, b0, b1);
              mma16z(c[n][1], x.c, x.d, y.c, y.d, b0, b1);
            } else {
              mma16(c[n][0], x.a, x.b, y.a, y.b, b0, b1);
              mma16(c[n][1], x.c, x.d, y.c, y.d, b0, b1);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              float2 sum = make_float2(c[n][m][j], c[n][m][j + 1]);
              if constexpr (PREC) sum = fma2(make_float2(rest[m][j], rest[m][j + 1]), make_float2(1.0f / kRest, 1.0f / kRest), sum);
              const float2 y = add2f(make_float2(o[n][i][m][j], o[n][i][m][j + 1]), sum);
              o[n][i][m][j] = y.x, o[n][i][m][j + 1] = y.y;
            }
      }
    }
  }

  // The unit's sums: put(row, first channel, four sums) for every row and channel of this lane, then
  // stat(row, reference, sum) once a row.  All without 2^off: a reference less off and the log of a sum times
  // 2^off would both be rounded near 23, and their sum, the log-sum-exp of a few keys, by 1e-6.
  template <class Put, class Stat>
  __device__ __forceinline__ void finish(int g, int qd, Put put, Stat stat) {
    const float a = __uint_as_float((uint32_t)(127 - off) << 23), b = 0.0625f * a;  // (b: of the codes' units)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float sum = l[n] * a, l0, l1;
      if constexpr (kCols) {
        l0 = l[0] * a, l1 = l[1] * a;
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l0 += __shfl_xor_sync(0xffffffffu, l0, d), l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      } else {
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        // the sums' columns are rows of lanes 8 qd and 8 qd + 4
        l0 = __shfl_sync(0xffffffffu, sum, 8 * qd), l1 = __shfl_sync(0xffffffffu, sum, 8 * qd + 4);
      }
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        float z0, z1;
        if constexpr (PREC) {
          float z = oz[n][i];
          z += __shfl_xor_sync(0xffffffffu, z, 1);
          z += __shfl_xor_sync(0xffffffffu, z, 2);
          z0 = __shfl_sync(0xffffffffu, z, 8 * qd), z1 = __shfl_sync(0xffffffffu, z, 8 * qd + 4);
        } else {
          z0 = __shfl_sync(0xffffffffu, oz[n][0], 4 * i + qd), z1 = __shfl_sync(0xffffffffu, oz[n][1], 4 * i + qd);
        }
        const float(&c)[2][4] = o[n][i];
        z0 *= a, z1 *= a;
        put(8 * n + 2 * qd, 32 * i + 4 * g, l0,
            make_float4(fmaf(c[0][0], a, z0), fmaf(c[0][2], b, z0), fmaf(c[1][0], a, z0), fmaf(c[1][2], b, z0)));
        put(8 * n + 2 * qd + 1, 32 * i + 4 * g, l1,
            make_float4(fmaf(c[0][1], a, z1), fmaf(c[0][3], b, z1), fmaf(c[1][1], a, z1), fmaf(c[1][3], b, z1)));
      }
      if constexpr (kCols) {
        if (g == 0) stat(2 * qd, ref[0], l0), stat(2 * qd + 1, ref[1], l1);
      } else {
        if (qd == 0) stat(8 * n + g, ref[n], sum);
      }
    }
  }
};

// What a block knows of a piece it joins.
struct Piece {
  int base, unit, items;  // the unit's first item, the unit, its items
};

template <int D, int NT, bool PREC, int NW, int NS>
struct Smem {
  static constexpr int kRing = NS * Layout<D>::kBytes;
  static_assert(Partial<D, NT>::kFloats * 4 <= kRing, "a warp's piece goes into its ring");
  static_assert(2 * NW <= 32, "a lane a piece");
  static constexpr size_t kBars = (size_t)NW * kRing, kInfoAt = kBars + 16 * ((NW * NS + 1) / 2), kRestAt = kInfoAt + 16 * NW * kInfo;
  static constexpr int kRestLogits = Warp<D, NT, PREC>::kCols ? kPage / 8 * 32 : 0;  // logits of a warp's page
  static constexpr size_t kBytes = kRestAt + 8 * (size_t)NW * kRestLogits;
};

// ---------------------------------------------------------------- joins
// Joins pieces of one query row: a lane's four channels of the sums and, in every lane, the row's reference
// and sum.  n pieces, m_of(i), l_of(i) their statistics, y_of(i) this lane's channels: the loads of J
// pieces are under way together.  Eight of a block's own (drafted tokens: 49.0 us; 51.1 with 16, 56.8 with 32, whose
// code takes longer to fetch), 16 of other blocks' (32,777 tokens: 18.9 us; 19.3 with eight).
template <int J, class M, class L, class Y>
__device__ __forceinline__ void join_row(int n, int lane, M m_of, L l_of, Y y_of, float4& o, float& top, float& sum) {
  o = make_float4(0, 0, 0, 0);
  top = -INFINITY, sum = 0.0f;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += J) {
    const bool mine = lane < J && i0 + lane < n;
    const float m = mine ? m_of(i0 + lane) : -INFINITY, l = mine ? l_of(i0 + lane) : 0.0f;
    float4 y[J];
#pragma unroll
    for (int i = 0; i < J; ++i) y[i] = i0 + i < n ? y_of(i0 + i) : make_float4(0, 0, 0, 0);
    float now = m;
    for (int d = J / 2; d; d >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
    now = fmaxf(top, __shfl_sync(0xffffffffu, now, 0));
    const float back = top == -INFINITY ? 0.0f : ex2(top - now), f = m == -INFINITY ? 0.0f : ex2(m - now);
    top = now;
    o = make_float4(o.x * back, o.y * back, o.z * back, o.w * back);
    float part = f * l;
    for (int d = J / 2; d; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
    sum = fmaf(sum, back, __shfl_sync(0xffffffffu, part, 0));
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const float w = __shfl_sync(0xffffffffu, f, i);
      o.x = fmaf(w, y[i].x, o.x), o.y = fmaf(w, y[i].y, o.y), o.z = fmaf(w, y[i].z, o.z), o.w = fmaf(w, y[i].w, o.w);
    }
  }
}

template <int D, int NT, bool PREC, int NW, int NS>
__global__ void __launch_bounds__(32 * NW, 1) attn_kernel(AttnArgs a) {
  using L = Layout<D>;
  using P = Partial<D, NT>;
  using S = Smem<D, NT, PREC, NW, NS>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Piece piece_s[2 * NW];
  __shared__ uint32_t valid_s, start_s, end_s;
  __shared__ int total_s;
  __shared__ int last_s[2], first_s[2];
  __shared__ uint8_t member_s[2 * NW];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, qd = lane % 4, H = a.c.h_kv;
  uint8_t* ring = smem + (size_t)warp * S::kRing;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars) + warp * NS;
  float2* rest = reinterpret_cast<float2*>(smem + S::kRestAt) + warp * S::kRestLogits;
  int4* info = reinterpret_cast<int4*>(smem + S::kInfoAt) + warp * kInfo;
  const int BC = a.c.batch * a.n_chunks;
  if (tid == 0) total_s = 0, valid_s = start_s = end_s = 0;
  if (lane < NS) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(bars + lane)) : "memory");
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  after_previous();

  // ---- the items of all units, and where this warp's run of them begins
  if (blockIdx.x == 0)
    for (int i = tid; i < a.c.batch; i += 32 * NW) check_length(a.c, i);
  const int c0 = lane < BC ? items_of(a, lane) : 0;  // of the first 32 (sequence, chunk) pairs
  int total;  // the host has made sure that all units' items fit
  if (BC <= 32) {
    total = __reduce_add_sync(0xffffffffu, c0);
    __syncthreads();
  } else {
    int n = 0;
    __syncthreads();
    for (int i = tid; i < BC; i += 32 * NW) n += items_of(a, i);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n) atomicAdd(&total_s, n);
    __syncthreads();
    total = total_s;
  }
  total *= H;
  // units without a key: nothing else writes their rows
  for (int bc = blockIdx.x; bc < BC; bc += gridDim.x) {
    if (items_of(a, bc) > 0) continue;
    for (int h = 0; h < H; ++h) {
      const Unit un = unit_at(a, bc * H + h);
      for (int i = tid; i < un.rows * (D / 4); i += 32 * NW)
        put4(a, row_at(a, un, i / (D / 4)) * D + i % (D / 4) * 4, make_float4(0, 0, 0, 0));
      if (tid < un.rows) put_lse(a, row_at(a, un, tid), 0.0f, 0.0f);
    }
  }
  // a block for every kMinItems items: few items stay in few blocks
  const int nb = min((int)gridDim.x, ceil_div(total, kMinItems));
  if ((int)blockIdx.x >= nb) return;
  const int nw = nb * NW, me = blockIdx.x * NW + warp;
  const int w0 = share(me, total, nw), w1 = share(me + 1, total, nw), n_items = w1 - w0;
  int bc = 0, h = 0, p = 0, cnt = 0;  // the next item to look up
  if (BC == 1) {
    cnt = __shfl_sync(0xffffffffu, c0, 0);
    h = w0 / cnt, p = w0 - h * cnt;
  } else {
    int before = 0;
    for (int i0 = 0; i0 < BC && n_items > 0; i0 += 32) {
      const int c = i0 == 0 ? c0 : i0 + lane < BC ? items_of(a, i0 + lane) : 0;
      int in = c * H;
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + in > w0);
      if (past) {
        const int l = __ffs(past) - 1;
        cnt = __shfl_sync(0xffffffffu, c, l);
        const int rem = w0 - before - (__shfl_sync(0xffffffffu, in, l) - cnt * H);
        bc = i0 + l, h = rem / cnt, p = rem - h * cnt;
        break;
      }
      before += __shfl_sync(0xffffffffu, in, 31);
    }
  }
  // The next n items' places, one a lane: (physical page, head) (-1: nothing to copy, -2: a copy withheld),
  // logical page, unit, and whether the item is its unit's first (1) or last (2).
  int known = 0;
  auto look_up = [&](int n) {
    const int i = known + lane;
    int4 e = make_int4(-1, 0, 0, 0);
    int b1 = bc, h1 = h, p1 = p + lane, c1 = cnt;
    if (lane < n && i < n_items) {
      while (p1 >= c1) {
        p1 -= c1;
        if (++h1 == H) {
          h1 = 0;
          do c1 = items_of(a, ++b1);
          while (c1 == 0);
        }
      }
      const int unit = b1 * H + h1, b = b1 / a.n_chunks;
      int lp = p1;
      if (a.sel) {
        lp = fetch(a.sel + (int64_t)unit * a.n_sel + p1);
        if (lp < 0 || (int64_t)lp * kPage >= seen_by(a, b, b1 % a.n_chunks)) lp = -1;
      }
      if (lp >= 0) {
        e.x = fetch(a.c.page_table + (int64_t)b * a.c.page_stride + lp);
        if (e.x < 0 || e.x >= a.c.n_pages) {
          raise(a.c, RDKV_ERR_INVALID_ARG);
          e.x = -1;
        } else {
          e.x = a.withhold && (lp + h1) % a.withhold == 0 ? -2 : e.x * H + h1;
        }
      }
      e.y = lp, e.z = unit, e.w = (p1 == 0 ? 1 : 0) | (p1 == c1 - 1 ? 2 : 0);
      info[i % kInfo] = e;
    }
    // from the last lane's item the next begins one further; only items that exist are passed on
    const int from = min(n, n_items - known) - 1;
    if (from >= 0) {
      bc = __shfl_sync(0xffffffffu, b1, from), h = __shfl_sync(0xffffffffu, h1, from);
      p = __shfl_sync(0xffffffffu, p1, from) + 1, cnt = __shfl_sync(0xffffffffu, c1, from);
      known += from + 1;
    }
    __syncwarp();
  };
  // Copies item i's page into stage i % NS.
  auto issue = [&](int i) {
    if (i >= known) look_up(kInfo / 2);
    if (lane == 0) {
      const int4 e = info[i % kInfo];
      const uint32_t bar = smem_u32(bars + i % NS);
      if (e.x < 0) {
        if (e.x == -1) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
        else asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], 16;" ::"r"(bar) : "memory");
      } else {
        const uint8_t* src = a.c.pages + (int64_t)e.x * L::kBytes;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(L::kBytes) : "memory");
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(ring + i % NS * L::kBytes)),
                     "l"(src), "r"(L::kBytes), "r"(bar)
                     : "memory");
      }
    }
    __syncwarp();
  };

  // Enters the piece of a unit that this warp has written up to item i.
  auto leave_piece = [&](int i, int unit, bool began, bool ends) {
    const int at = 2 * warp + (ends ? 0 : 1), items = items_of(a, unit / H);
    // the unit's first item: this one is its last, or the lookup stands one past the run's last item
    piece_s[at] = Piece{ends ? w0 + i - (items - 1) : w1 - p, unit, items};
    atomicOr(&valid_s, 1u << at);
    if (began) atomicOr(&start_s, 1u << at);
    if (ends) atomicOr(&end_s, 1u << at);
  };

  // ---- the run
  Warp<D, NT, PREC> w;
  bool in_unit = false, began = false, ok = true;
  bool only = false;  // the unit's one page is here, its queries split
  int held = 0;  // tokens of the unit's sequence
  using W = Warp<D, NT, PREC>;
  int low[W::kStats];  // keys that this lane's rows see
  Unit un{0, 0, 0, 0};
  int i = 0;
  if (n_items > 0) {
    look_up(kInfo);
    // the first queries are asked for before the pages, behind which they would wait
    typename Warp<D, NT, PREC>::Rows x;
    un = unit_at(a, info[0].z);
    w.queries(a, un, g, qd, x);
#pragma unroll 1
    for (int j = 0; j < min(NS, n_items); ++j) issue(j);
    w.begin(a.dtype, x, qd);
    in_unit = true;
  }
#pragma unroll 1
  for (; i < n_items; ++i) {
    const int4 e = info[i % kInfo];
    if (!in_unit) {
      typename Warp<D, NT, PREC>::Rows x;
      un = unit_at(a, e.z);
      w.queries(a, un, g, qd, x);
      w.begin(a.dtype, x, qd);
    }
    if (!in_unit || i == 0) {
      in_unit = true, began = e.w & 1;
      held = held_tokens(a.c, un.b);
#pragma unroll
      for (int n = 0; n < W::kStats; ++n) low[n] = held - a.n_q + min(un.t0 + W::stat_row(n, g, qd) / a.G, a.n_q - 1) + 1;
      if constexpr (W::kCols) {  // (in the page's branch below: 2.5 % more at 262,144 tokens)
        // a page that has not landed by now is taken with whole queries, if it lands in the wait below
        only = (e.w & 3) == 3 && e.x >= 0 && __all_sync(0xffffffffu, wait_for(bars + i % NS, (i / NS) & 1, a.wait_cycles));
        if (only) w.split(ring + i % NS * L::kBytes, rest, g, qd);
      }
    }
    if (!__all_sync(0xffffffffu, wait_for(bars + i % NS, (i / NS) & 1, a.wait_cycles))) {  // the warp goes on, or stops, as one
      ok = false;
      break;
    }
    if (e.x >= 0) {
      int see[W::kStats];
      bool cut = false;
#pragma unroll
      for (int n = 0; n < W::kStats; ++n) see[n] = low[n] - e.y * kPage, cut |= see[n] < kPage;
      w.page(ring + i % NS * L::kBytes, rest, g, qd, only || __any_sync(0xffffffffu, cut), only, held - e.y * kPage, see);
    }
    __syncwarp();
    if (i + NS < n_items) issue(i + NS);
    if ((e.w & 2) || i == n_items - 1) {  // the unit, or the run, ends
      const bool ends = e.w & 2;
      // a unit that ends here without having begun lies first in the run: copies are under way, its piece
      // goes to global memory
      float* dst = ends ? a.heads + (int64_t)me * P::kFloats : reinterpret_cast<float*>(ring);
      if (began && ends) {
        w.finish(
            g, qd,
            [&](int row, int ch, float l, float4 o) {
              if (row < un.rows) put4(a, row_at(a, un, row) * D + ch, scaled(o, l));
            },
            [&](int row, float m, float l) {
              if (row < un.rows) put_lse(a, row_at(a, un, row), m, l);
            });
      } else {
        w.finish(
            g, qd, [&](int row, int ch, float, float4 o) { *reinterpret_cast<float4*>(dst + row * D + ch) = o; },
            [&](int row, float m, float l) { dst[P::kRows * D + row] = m, dst[P::kRows * (D + 1) + row] = l; });
        if (lane == 0) leave_piece(i, e.z, began, ends);
      }
      in_unit = false;
    }
  }
  if (!ok) {
    // A wait ran out: report it and let the copies under way land (again with a limit; a withheld one is none).  The
    // units of the rest of the run get pieces that hold nothing, so that their blocks' tickets come out even and the
    // workspace serves the next call.
    if (lane == 0) raise(a.c, RDKV_ERR_TIMEOUT);
#pragma unroll 1
    for (int j = i; j < min(i + NS, n_items); ++j)
      if (info[j % kInfo].x != -2) wait_for(bars + j % NS, (j / NS) & 1, kWaitCycles);
    __syncwarp();
#pragma unroll 1
    for (; i < n_items; ++i) {
      if (i >= known) look_up(kInfo / 2);
      const int4 e = info[i % kInfo];
      if (!in_unit) in_unit = true, began = e.w & 1;
      if (!(e.w & 2) && i < n_items - 1) continue;
      const bool ends = e.w & 2;
      if (began && ends) {
        un = unit_at(a, e.z);
        for (int x = lane; x < un.rows * (D / 4); x += 32)
          put4(a, row_at(a, un, x / (D / 4)) * D + x % (D / 4) * 4, make_float4(0, 0, 0, 0));
        if (lane < un.rows) put_lse(a, row_at(a, un, lane), 0.0f, 0.0f);
      } else {
        float* dst = ends ? a.heads + (int64_t)me * P::kFloats : reinterpret_cast<float*>(ring);
        for (int x = lane; x < P::kFloats; x += 32) dst[x] = x / P::kRows == D ? -INFINITY : 0.0f;
        if (lane == 0) leave_piece(i, e.z, began, ends);
      }
      in_unit = false;
    }
  }
  __syncthreads();

  // ---- joining the block's pieces: runs of pieces of one unit, a run begins at a piece that holds its
  // unit's first item, or at the block's first piece; a query row of a run a warp
  const uint32_t valid = valid_s, ends = end_s, begins = start_s;
  const uint32_t starts = begins | (valid & (0u - valid));
  if (tid < 2 * NW && (valid >> tid & 1)) member_s[__popc(valid & ((1u << tid) - 1u))] = (uint8_t)tid;
  __syncthreads();
  int open[2] = {-1, -1};  // pieces of runs that are a part of their unit: one that began before the block, one that goes on
  auto block_of = [&](int64_t item) { return quotient((item + 1) * nb - 1, total); };
  int task = 0;
  for (uint32_t left = starts; left; left &= left - 1) {
    const int s = __ffs(left) - 1;
    const uint32_t rest = left & (left - 1), members = valid & ~((1u << s) - 1u) & (rest ? (rest & (0u - rest)) - 1u : 0xffffffffu);
    const bool whole = (begins >> s & 1) && (ends & members);
    const Piece pc = piece_s[s];
    const int slot = begins >> s & 1, n = __popc(members), first = __popc(valid & ((1u << s) - 1u));
    const Unit ru = unit_at(a, pc.unit);
    float* part = a.parts + ((int64_t)blockIdx.x * 2 + slot) * P::kFloats;
    auto src = [&](int j) -> const float* {
      const int e = member_s[first + j];
      return e & 1 ? reinterpret_cast<const float*>(smem + (size_t)(e / 2) * S::kRing)
                   : a.heads + ((int64_t)blockIdx.x * NW + e / 2) * P::kFloats;
    };
    for (int row = 0; row < ru.rows; ++row) {
      if (task++ % NW != warp) continue;
      float4 o;
      float m, l;
      const int ch = 4 * lane % D;
      join_row<8>(
          n, lane, [&](int j) { return src(j)[P::kRows * D + row]; }, [&](int j) { return src(j)[P::kRows * (D + 1) + row]; },
          [&](int j) { return *reinterpret_cast<const float4*>(src(j) + row * D + ch); }, o, m, l);
      if (whole) {
        const int64_t at = row_at(a, ru, row);
        if (4 * lane < D) put4(a, at * D + ch, scaled(o, l));
        if (lane == 0) put_lse(a, at, m, l);
      } else {
        if (4 * lane < D) *reinterpret_cast<float4*>(part + row * D + ch) = o;
        if (lane == 0) part[P::kRows * D + row] = m, part[P::kRows * (D + 1) + row] = l;
      }
    }
    if (!whole) open[slot] = s;
  }
  // ---- joining the blocks' parts: the last block of a unit to arrive does it
  if (open[0] < 0 && open[1] < 0) return;
  __syncthreads();
  if (tid < 2 && open[tid] >= 0) {
    const Piece pc = piece_s[open[tid]];
    const int first = block_of(pc.base), n = block_of(pc.base + pc.items - 1) - first + 1;
    int32_t* t = a.tickets + pc.unit;
    int before;
    asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(before) : "l"(t) : "memory");
    const bool last = before == n - 1;
    if (last) *t = 0;
    last_s[tid] = last ? n : 0;
    first_s[tid] = first;
  }
  __syncthreads();
#pragma unroll 1
  for (int slot = 0; slot < 2; ++slot) {
    const int e = slot ? open[1] : open[0];
    if (e < 0 || last_s[slot] == 0) continue;
    const int unit = piece_s[e].unit, n = last_s[slot], first = first_s[slot];
    const Unit ru = unit_at(a, unit);
    for (int row = warp; row < ru.rows; row += NW) {
      // the unit's first block wrote it as the unit that goes on, the others as the one that began before
      auto part = [&](int j) { return a.parts + ((int64_t)(first + j) * 2 + (j == 0 ? 1 : 0)) * P::kFloats; };
      float4 o;
      float m, l;
      const int ch = 4 * lane % D;
      join_row<16>(
          n, lane, [&](int j) { return __ldcg(part(j) + P::kRows * D + row); },
          [&](int j) { return __ldcg(part(j) + P::kRows * (D + 1) + row); },
          [&](int j) { return __ldcg(reinterpret_cast<const float4*>(part(j) + row * D + ch)); }, o, m, l);
      const int64_t at = row_at(a, ru, row);
      if (4 * lane < D) put4(a, at * D + ch, scaled(o, l));
      if (lane == 0) put_lse(a, at, m, l);
    }
  }
}

// ---------------------------------------------------------------- launch
// The workspace has the same places for every shape, so that calls of any shape may follow one another: the
// tickets, then pieces of the largest variant.
constexpr int kMaxWarps = 8;

struct Geometry {
  int chunk, n_chunks, nt, grid;
  size_t heads_at, parts_at, bytes;
};

static Geometry geometry(const rdkv_q4_cache* c, int h_q, int n_q, bool prec, bool own_pages) {
  Geometry o;
  const int G = h_q / c->h_kv;
  // Query tokens that share one pass over the keys: as many as fit in 16 rows (8 for fp32 outputs, whose
  // other 8 rows hold the queries' low parts); one when every query token has its own pages
  o.chunk = own_pages ? 1 : std::min(n_q, std::max(1, (prec ? 8 : 16) / G));
  o.n_chunks = ceil_div(n_q, o.chunk);
  o.nt = o.chunk * G > 8 ? 2 : 1;
  o.grid = num_sms();
  const int64_t part = 4LL * Partial<128, 2>::kFloats;
  o.heads_at = RDKV_Q4_COUNTER_BYTES;
  o.parts_at = o.heads_at + (size_t)align_up((int64_t)o.grid * kMaxWarps * part, 256);
  o.bytes = o.parts_at + (size_t)align_up(2LL * o.grid * part, 256);
  return o;
}

template <int D, int NT, bool PREC, int NW, int NS>
static rdkv_status launch(const AttnArgs& a, int grid, cudaStream_t cs) {
  using S = Smem<D, NT, PREC, NW, NS>;
  static_assert(NW <= kMaxWarps, "the workspace counts with kMaxWarps");
  auto kernel = attn_kernel<D, NT, PREC, NW, NS>;
  // once a device (of the first 64; the others pay for the call every time)
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  RDKV_TRY_CUDA(cudaGetDevice(&dev), "4-bit cache attention");
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    RDKV_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes), "4-bit cache attention");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  RDKV_TRY_CUDA(launch_after(kernel, dim3(grid), 32 * NW, S::kBytes, cs, a), "4-bit cache attention");
  count_launch();
  return RDKV_OK;
}

}  // namespace q4
}  // namespace rdkv

using namespace rdkv;
using namespace rdkv::q4;

extern "C" size_t rdkv_q4_attn_workspace_bytes(const rdkv_q4_cache* cache, int32_t h_q, int32_t n_q) {
  if (check_queries(cache, h_q, n_q) != RDKV_OK) return 0;
  return geometry(cache, h_q, n_q, false, false).bytes;
}

// withhold > 0: the self-test
static rdkv_status attn_impl(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q, int32_t n_q,
                             const int32_t* sel, int32_t n_sel, void* out, int32_t out_dtype, float* lse, void* ws, size_t ws_bytes,
                             void* stream, int withhold, long long wait_cycles) {
  rdkv_status st = check_q(cache, dtype, q, q_stride, h_q, n_q);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(out != nullptr, RDKV_ERR_INVALID_ARG, "NULL output");
  RDKV_REQUIRE((uintptr_t)out % 16 == 0, RDKV_ERR_INVALID_ARG, "out must be 16-byte aligned");
  RDKV_REQUIRE(out_dtype == dtype || out_dtype == RDKV_F32, RDKV_ERR_UNSUPPORTED, "out_dtype %d for dtype %d", out_dtype, dtype);
  RDKV_REQUIRE(!sel || n_sel >= 1, RDKV_ERR_INVALID_ARG, "n_sel %d", n_sel);
  RDKV_REQUIRE((int64_t)cache->batch * cache->h_kv * n_q * (sel ? n_sel : cache->page_stride) <= INT32_MAX, RDKV_ERR_UNSUPPORTED,
               "more than 2^31 - 1 (sequence, query token, KV head, page) items");
  const bool prec = out_dtype == RDKV_F32;
  const Geometry geo = geometry(cache, h_q, n_q, prec, sel != nullptr);
  RDKV_REQUIRE(ws && (uintptr_t)ws % 16 == 0 && ws_bytes >= geo.bytes, RDKV_ERR_WORKSPACE,
               "attention workspace too small (%zu < %zu) or unaligned", ws_bytes, geo.bytes);
  char* w = static_cast<char*>(ws);
  const AttnArgs a{view_of(cache), q, out, lse, sel, reinterpret_cast<float*>(w + geo.heads_at),
                   reinterpret_cast<float*>(w + geo.parts_at), reinterpret_cast<int32_t*>(w), q_stride, dtype, out_dtype, n_q, h_q / cache->h_kv, n_sel,
                   geo.chunk, geo.n_chunks, withhold, wait_cycles};
  cudaStream_t cs = (cudaStream_t)stream;
  if (cache->head_dim == 128) {
    if (prec) return launch<128, 1, true, 8, 2>(a, geo.grid, cs);
    if (geo.nt == 2) return launch<128, 2, false, 8, 2>(a, geo.grid, cs);
    return launch<128, 1, false, 8, 2>(a, geo.grid, cs);
  }
  if (prec) return launch<64, 1, true, 8, 4>(a, geo.grid, cs);
  if (geo.nt == 2) return launch<64, 2, false, 8, 4>(a, geo.grid, cs);
  return launch<64, 1, false, 8, 4>(a, geo.grid, cs);
}

extern "C" rdkv_status rdkv_q4_attn(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q,
                                    int32_t n_q, const int32_t* sel, int32_t n_sel, void* out, int32_t out_dtype, float* lse,
                                    void* ws, size_t ws_bytes, void* stream) {
  return attn_impl(cache, dtype, q, q_stride, h_q, n_q, sel, n_sel, out, out_dtype, lse, ws, ws_bytes, stream, 0, kWaitCycles);
}

extern "C" rdkv_status rdkv_q4_timeout_selftest(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride,
                                                int32_t h_q, int32_t n_q, const int32_t* sel, int32_t n_sel, void* out,
                                                int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, int32_t withhold,
                                                int64_t wait_cycles, void* stream) {
  RDKV_REQUIRE(withhold >= 1, RDKV_ERR_INVALID_ARG, "withhold %d must be positive", withhold);
  RDKV_REQUIRE(wait_cycles > 0, RDKV_ERR_INVALID_ARG, "wait_cycles %lld must be positive", (long long)wait_cycles);
  return attn_impl(cache, dtype, q, q_stride, h_q, n_q, sel, n_sel, out, out_dtype, lse, ws, ws_bytes, stream, withhold,
                   std::min(kWaitCycles, std::max(kMinWaitCycles, (long long)wait_cycles)));
}
