// Attention over the 8-bit paged cache (rdkv_q8_attn), and the weights that its keys receive.
//
//   logits  s_t = (q . code_t) scale_k / sqrt(D), scale_k = 2^e of the key's page
//   out     = sum_t p_t 2^f code'_t / sum_t p_t, p_t = exp(s_t - ref), 2^f the scale of the value's page
//   mass_t += sum over query rows of exp(s_t - lse)
//
// Work.  A unit is (sequence, chunk of query tokens, KV head): up to 8 NT query rows, NT = 1 or 2, that share the
// unit's keys; an item is one page (64 tokens) of a unit.  The items of all units, one after another, are dealt evenly
// to the warps of the grid (one block an SM); each warp takes a run of items and works alone on pages in a ring of its
// own, whose stages are halves of a page: while the keys are multiplied the values arrive, and the next page's keys
// follow as soon as the logits stand.  Units that end inside a warp's run are written by it; the pieces of the others
// are joined per block in shared memory and, where a unit spans blocks, by the last of its blocks through the
// workspace, always in the same order: the result does not depend on who comes first.
//
// Products: mma.sync with fp16 operands.  A code is an fp16 number exactly, one conversion a pair, so the operands'
// only roundings are the queries' and the weights'.  Up to eight query rows (NT = 1): tokens on M and queries on N for
// the logits, channels on M and queries on N for the values; a movmatrix a tile of eight tokens turns weights into the
// values' operand.  More rows (NT = 2): queries on M for both, and the weights' registers are the values' operand as
// they are.  The page's order (q8.cuh) gives every operand in 16-byte loads without bank conflicts.
//
// Scales.  The keys' scale, 1 / sqrt(D), log2 e and the row's power of two are one factor of the page.  The values' scale
// 2^f joins the exponent: what is held is 2^(s + f - ref), ref the running maximum of s + f, so that weights are rounded
// relative to what they contribute, not to the largest probability, and a page of small values costs no bits of
// one of large values.  The sum of weights takes 2^-f back, once a page.  (ref is held as its two parts, whose sum
// would lose f beside a logit of 2^24.)
//
// Roundings.  Logits, maxima, sums of weights and outputs' sums are fp32.  The tensor core cuts what it adds to an
// accumulator (it does not round), so its accumulators start at zero for every page and the pages' sums are fp32 additions.
//   16-bit outputs  queries as they are (a row times a power of two); weights rounded to fp16: 2^-12 of each.
//   fp32 outputs    (PREC) queries and weights in two fp16 parts, 22 bits.
//
// Bound.  256 bytes a token and KV head at D = 128: 262,144 tokens of 8 heads (537 MB) in 86 us, 92 % of the measured copy
// bandwidth, fp32 outputs as fast; eight sequences of 16,384 to 32,768 tokens (382 MB) in 65, 86 %.  A page of up to eight rows takes 64
// products and some 550 instructions; issue slots are 26 % used, the tensor pipe 14 %.  Above the bytes stand some 3 us until
// the first page is asked for, 4 us of joins, and that SMs do not get equal shares of the bandwidth: at 262,144 tokens 40 of
// 152 take 9 % longer than the others for as many pages, always the same ones.  A dealing by who comes first would even that
// out, but then the sums' order, and so their last bits, would change from call to call.  16 rows (four drafted tokens of 4 heads: 47 us, the
// bytes 29) lose more to their own instructions, chains of which two warps a scheduler hide little: by clocks read in the loop, which
// slow it, a page takes a warp 3.7 us, of which it waits for bytes 0.7 (8 rows: 2.3, of which 0.9), and a change of unit 3 (1.3).
// A warp's 16 rows by 128 channels of sums fill the 255 registers (56 bytes spilled at D = 128), so eight warps fit; a page shared by two
// warps, half of the channels each, has not been built.  More query tokens than fit in 16 rows (fp32 outputs: 8) read the cache once for
// every such chunk: 16 x up to 8,191 tokens of 4 heads a group take 68 us for 8 query tokens, 122 for 16 and 429 for 64 (fp32 outputs 126, 240
// and 910; the bytes 30, the operations 7, 14 and 55).
//   Measured and not kept (us at 262,144 tokens, 16-bit and fp32 outputs; against 90.8 and 89.5): warps x half
// pages 12 x 2 92.4 and 117, 10 x 2 89.7 and 100, 8 x 3 89.7 and 90.6 (batched 68.8 and 70.9, here 67.9 and 68.1), 6 x 4 91.7 and 98.5, 5 x 5
// 93.5 and 117, 4 x 6 91.1 and 107; the joins in a second launch, by a row a block or a row a group of warps: 104 and 96 against 94; the
// next unit's queries asked for while the last page is multiplied, into registers (64 x 2,000 tokens: 55.6 against 55.0) or into L1
// (55.8); items of 32 tokens instead of 64, in copies half as large, 101 against 87, and for 16 rows 51.6 against 51.2; the code that
// begins a unit once instead of twice, its first pages asked for inside: 16 rows 0.9 less, others up to 0.4 more.
#include <atomic>

#include "q8.cuh"

namespace rdkv {
namespace q8 {

struct AttnArgs {
  View c;
  const void* q;
  void* out;
  float* lse;
  float* logits;     // or NULL; [units][page_stride][rows][64]: base 2
  float2* stats;     // (with logits) each query row's reference (base 2) and sum of weights
  float* heads;      // [grid * NW] partials: pieces of units that end inside a warp's run
  float* parts;      // [grid * 2] partials: a block's part of a unit that began before it, of one that goes on
  int32_t* tickets;  // [units] blocks that have written their part
  int64_t q_stride;
  int dtype, out_dtype, n_q, G, chunk, n_chunks;  // chunk: query tokens of a unit
  int rows;               // of a unit at most
  int withhold;           // 0, or (the self-test) pages with (index + KV head) % withhold == 0 are waited for, not copied
  long long wait_cycles;  // limit of a wait for a page
};

constexpr int kMinItems = 1;  // of a block (513 tokens of one head: 7.9 us; with 4 8.3, with 14 8.7; of eight heads 9.4, 10.9 and 13.7)
constexpr int kInfo = 16;     // items whose places a warp knows ahead

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
  return seen <= 0 ? 0 : ceil_div(seen, kPage);
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
      w = make_uint2(cut_half2(o.x, o.y), cut_half2(o.z, o.w));
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(o.x, o.y), y = __floats2bfloat162_rn(o.z, o.w);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = w;
  }
}
// The row's log-sum-exp, of a reference and a sum that may be some 2^30 (the reference is the logit of the key that
// contributes most, not the largest): the sum's exponent goes to the reference first, so that no two large parts that cancel are rounded.  (a NaN sum, of a query that holds one, is not a sum of nothing)
__device__ __forceinline__ void put_lse(const AttnArgs& a, int64_t row, float m, float l) {
  if (a.lse) {
    const int e = (int)(__float_as_uint(l) >> 23 & 255u) - 127;
    a.lse[row] = l != 0.0f ? ((m + (float)e) + log2f(l * two_to(-e))) * 0.6931471805599453f : -INFINITY;
  }
  if (a.stats) a.stats[row] = make_float2(m, l);
}

// A unit's rows, by one warp, where no key is seen.
template <int D>
__device__ __noinline__ void write_nothing(const AttnArgs& a, Unit un, int lane) {
  for (int i = lane; i < un.rows * (D / 4); i += 32) put4(a, row_at(a, un, i / (D / 4)) * D + i % (D / 4) * 4, make_float4(0, 0, 0, 0));
  if (lane < un.rows) put_lse(a, row_at(a, un, lane), 0.0f, 0.0f);
}

// One warp's running state over the pages of one unit.
template <int D, int NT, bool PREC>
struct Warp {
  static_assert(NT == 1 || !PREC, "two parts take eight rows");
  using L = Layout<D>;
  static constexpr int kS = L::kSides;
  static constexpr bool kCols = NT == 1;  // queries on N
  // The query rows whose statistics a lane keeps: its columns 2 qd and 2 qd + 1, or g and g + 8.
  static __device__ __forceinline__ int stat_row(int n, int g, int qd) { return kCols ? 2 * qd + n : g + 8 * n; }
  // Weights are held times 2^kOff: at most 2^15 (they pass the reference by 2^4 at most; PREC: not at all), and normal fp16
  // numbers down to 2^-25 of the largest contribution (PREC: 2^-28).
  static constexpr int kOff = PREC ? 14 : 11;
  static constexpr int kRest = 2048;  // of the weights' remainders
  static constexpr float kFar = 262144.0f;

  uint32_t q[kS][4][2 * NT];            // operand registers by 64 channels and 16 of them
  uint32_t qlow[PREC ? kS : 1][4][2];   // (PREC) the remainders
  float scale[2];                       // base-2 logits of sums of codes, the keys' scale aside
  float ref[2], rf[2], l[2];            // the running maximum as a logit (base 2) and its values' exponent; this lane's share of the sum
  // kCols: [64 channels][pair m][channel 2 m, + 1 of this lane's 8 x columns]; else [64 channels][channel c of 8][rows x columns]
  float o[kS][kCols ? 4 : 8][4];

  // This lane's channels of the unit's query rows, as they lie in memory (rows past the last: zero): of every 64
  // channels the 16 from 16 qd on.  Kept apart from begin() so that copies can be issued while they are under way.
  struct Rows {
    uint4 w[NT][kS][PREC ? 4 : 2];
  };
  __device__ __forceinline__ static void queries(const AttnArgs& a, const Unit& un, int g, int qd, Rows& r) {
    const bool wide = PREC && a.dtype == RDKV_F32;
    const int size = wide ? 4 : 2;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = g + 8 * n, t = row / a.G;
      const bool real = row < un.rows;
      const int64_t at = ((int64_t)un.b * a.n_q + un.t0 + t) * a.q_stride + ((int64_t)un.h * a.G + row - t * a.G) * D + 16 * qd;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) + (real ? at * size : 0));
#pragma unroll
      for (int j = 0; j < kS; ++j)
#pragma unroll
        for (int i = 0; i < (PREC ? 4 : 2); ++i)
          r.w[n][j][i] = real && (i < 2 || wide) ? fetch(src + 4 * j * size + i) : make_uint4(0, 0, 0, 0);
    }
  }
  // (fp32 queries have fp32 outputs, so only PREC reads them)
  __device__ __forceinline__ static void widen(int dtype, const Rows& r, int n, int j, float (&x)[16]) {
    if constexpr (PREC) {
      if (dtype == RDKV_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = r.w[n][j][i];
          x[4 * i] = __uint_as_float(w.x), x[4 * i + 1] = __uint_as_float(w.y), x[4 * i + 2] = __uint_as_float(w.z),
                x[4 * i + 3] = __uint_as_float(w.w);
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {r.w[n][j][i].x, r.w[n][j][i].y, r.w[n][j][i].z, r.w[n][j][i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = dtype == RDKV_F16 ? unpack2(w[e]) : make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
        x[8 * i + 2 * e] = f.x, x[8 * i + 2 * e + 1] = f.y;
      }
    }
  }

  __device__ __forceinline__ void begin(int dtype, const Rows& rows, int qd) {
    constexpr float kK = 1.4426950408889634f / (D == 128 ? 11.313708498984761f : 8.0f);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < kS; ++j) {
        float x[16];
        widen(dtype, rows, n, j, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the row times 2^s, its largest value in [2^14, 2^15): what fp16 drops is 2^-25 against that.  Down to s =
      // -113, so that every finite row has its place, and up to 97, so that the factor stays a normal number.
      const int e2 = (int)(__float_as_uint(top) >> 23) - 127;
      const int s = top > 0.0f ? max(-113, min(97, 14 - e2)) : 0;
      const float up = two_to(s), down = two_to(-s) * kK;
      if constexpr (kCols) {
#pragma unroll
        for (int j = 0; j < 2; ++j) scale[j] = __shfl_sync(0xffffffffu, down, 8 * qd + 4 * j);
      } else {
        scale[n] = down;
      }
#pragma unroll
      for (int j = 0; j < kS; ++j) {
        float x[16];
        widen(dtype, rows, n, j, x);
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float y0 = x[4 * w + 2 * i] * up, y1 = x[4 * w + 2 * i + 1] * up;
            q[j][w][kCols ? i : 2 * i + n] = pack2(y0, y1);
            if constexpr (PREC) qlow[j][w][i] = rest2(y0, y1, q[j][w][i]);
          }
      }
    }
#pragma unroll
    for (int j = 0; j < kS; ++j)
#pragma unroll
      for (int m = 0; m < (kCols ? 4 : 8); ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][m][i] = 0.0f;
#pragma unroll
    for (int n = 0; n < 2; ++n) ref[n] = -INFINITY, rf[n] = l[n] = 0.0f;
  }

  // Sums of a lane's two rows (or columns) times f0 and f1.
  __device__ __forceinline__ void rescale(float f0, float f1) {
    l[0] *= f0, l[1] *= f1;
#pragma unroll
    for (int j = 0; j < kS; ++j)
#pragma unroll
      for (int m = 0; m < (kCols ? 4 : 8); ++m) {
        if constexpr (kCols) o[j][m][0] *= f0, o[j][m][1] *= f1, o[j][m][2] *= f0, o[j][m][3] *= f1;
        else o[j][m][0] *= f0, o[j][m][1] *= f0, o[j][m][2] *= f1, o[j][m][3] *= f1;
      }
  }

  // Sums of queries and codes.  kCols: tokens 16 i + g (elements 0, 1) and + 8 (2, 3), columns 2 qd and + 1; else rows
  // g (0, 1) and g + 8 (2, 3), tokens 8 i + 2 qd and + 1.
  static constexpr int kTiles = kCols ? kPage / 16 : kPage / 8;
  struct Logits {
    float c[kTiles][4];
  };
  __device__ __forceinline__ void logits(const uint8_t* k, int g, int qd, Logits& s) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint8_t* at = k + L::key_at((kCols ? 16 : 8) * i + g, 0, 2 * qd);
      float low[4];
#pragma unroll
      for (int j = 0; j < kS; ++j) {
        const uint4 x4 = *reinterpret_cast<const uint4*>(at + 128 * j);
        const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
        if constexpr (kCols) {
          const uint4 y4 = *reinterpret_cast<const uint4*>(at + 8 * D + 128 * j);
          const uint32_t y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = halves_lo(x[w]), a1 = halves_lo(y[w]), a2 = halves_hi(x[w]), a3 = halves_hi(y[w]);
            if (j == 0 && w == 0) mma16z(s.c[i], a0, a1, a2, a3, q[j][w][0], q[j][w][1]);
            else mma16(s.c[i], a0, a1, a2, a3, q[j][w][0], q[j][w][1]);
            if constexpr (PREC) {
              if (j == 0 && w == 0) mma16z(low, a0, a1, a2, a3, qlow[j][w][0], qlow[j][w][1]);
              else mma16(low, a0, a1, a2, a3, qlow[j][w][0], qlow[j][w][1]);
            }
          }
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t b0 = halves_lo(x[w]), b1 = halves_hi(x[w]);
            if (j == 0 && w == 0) mma16z(s.c[i], q[j][w][0], q[j][w][1], q[j][w][2], q[j][w][3], b0, b1);
            else mma16(s.c[i], q[j][w][0], q[j][w][1], q[j][w][2], q[j][w][3], b0, b1);
          }
        }
      }
      if constexpr (PREC) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s.c[i][e] += low[e];
      }
    }
  }
  // Element e of tile i: its token, and which of the lane's two rows it belongs to.
  static __device__ __forceinline__ int token_of(int i, int e, int g, int qd) {
    return kCols ? 16 * i + g + (e & 2) * 4 : 8 * i + 2 * qd + (e & 1);
  }
  static constexpr __device__ __forceinline__ int row_of(int e) { return kCols ? e & 1 : e >> 1; }

  // The weights of a page, as the values' operand (PREC: and what that drops, times kRest).
  struct Weights {
    uint32_t hi[kPage / 16][kCols ? 2 : 4], low[PREC ? kPage / 16 : 1][2];
  };
  // cut (the same in all lanes): some tokens of the page are hidden from some rows: row n sees see[n] of them.
  __device__ __forceinline__ void weigh(Logits& s, float2 page, int g, int qd, bool cut, const int (&see)[2], float* store, int rows,
                                        Weights& p) {
    const float f = (float)exponent(page.y);
    float sc[2] = {scale[0] * page.x, scale[1] * page.x};
    if (cut) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (token_of(i, e, g, qd) >= see[row_of(e)]) s.c[i][e] = -INFINITY;
    }
    if (store) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        if constexpr (kCols) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (2 * qd + (e & 1) < rows) store[(2 * qd + (e & 1)) * kPage + token_of(i, e, g, qd)] = __fmul_rn(s.c[i][e], sc[e & 1]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            if (g + 4 * e < rows)
              *reinterpret_cast<float2*>(store + (g + 4 * e) * kPage + token_of(i, e, g, qd)) =
                  make_float2(__fmul_rn(s.c[i][e], sc[e >> 1]), __fmul_rn(s.c[i][e + 1], sc[e >> 1]));
        }
      }
    }
    // a row's reference rises when one of its logits with the values' scale passes it by more than 4 (PREC: at all)
    float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) m[row_of(e)] = fmaxf(m[row_of(e)], s.c[i][e]);
    m[0] = __fmul_rn(m[0], sc[0]), m[1] = __fmul_rn(m[1], sc[1]);
    constexpr float kPast = PREC ? 0.0f : 4.0f;
    // (nothing seen yet: infinity; nothing seen in this page either: a NaN, which passes nothing)
    if (__any_sync(0xffffffffu, (m[0] - ref[0]) + (f - rf[0]) > kPast || (m[1] - ref[1]) + (f - rf[1]) > kPast)) {
      float back[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int d = kCols ? 4 : 1; d < (kCols ? 32 : 4); d *= 2) m[n] = fmaxf(m[n], __shfl_xor_sync(0xffffffffu, m[n], d));
        const float past = (m[n] - ref[n]) + (f - rf[n]);
        back[n] = 1.0f;
        if (past > 0.0f) back[n] = ex2(-past), ref[n] = m[n], rf[n] = f;
      }
      rescale(back[0], back[1]);
    }
    const float r[2] = {ref[0] == -INFINITY ? 0.0f : ref[0], ref[1] == -INFINITY ? 0.0f : ref[1]};
    const float off[2] = {(float)kOff + f - rf[0], (float)kOff + f - rf[1]};
    float up[2] = {off[0] - r[0], off[1] - r[1]};
    if (__any_sync(0xffffffffu, fmaxf(fabsf(r[0]), fabsf(r[1])) > kFar)) {
      // logits so large that the roundings of product and sum, up to 2^-24 of them, would show in the exponent: their difference
      // from the reference, which is exact
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.c[i][e] = __fadd_rn(__fmul_rn(s.c[i][e], sc[row_of(e)]), -r[row_of(e)]) + off[row_of(e)];
      sc[0] = sc[1] = 1.0f, up[0] = up[1] = 0.0f;
    }
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = ex2(fmaf(s.c[i][e], sc[row_of(e)], up[row_of(e)]));
        sum[row_of(e)] += x[e];
      }
      const uint32_t w0 = pack2(x[0], x[1]), w1 = pack2(x[2], x[3]);
      if constexpr (kCols) {
        p.hi[i][0] = transposed(w0), p.hi[i][1] = transposed(w1);
        if constexpr (PREC) {
          p.low[i][0] = transposed(rest2<kRest>(x[0], x[1], w0)), p.low[i][1] = transposed(rest2<kRest>(x[2], x[3], w1));
        }
      } else {
        p.hi[i / 2][i % 2 * 2] = w0, p.hi[i / 2][i % 2 * 2 + 1] = w1;
      }
    }
    const float less = two_to(-exponent(page.y));
    l[0] = fmaf(sum[0], less, l[0]), l[1] = fmaf(sum[1], less, l[1]);
  }

  // Adds the weighted values of a page.
  __device__ __forceinline__ void values(const uint8_t* v, int g, int qd, const Weights& p) {
    const uint8_t* at = v + g * 64 + qd * 16;
#pragma unroll
    for (int j = 0; j < kS; ++j) {
      if constexpr (kCols) {
        float c[4][4], low[PREC ? 4 : 1][4];
#pragma unroll
        for (int t = 0; t < kPage / 16; ++t) {
          const uint4 x4 = *reinterpret_cast<const uint4*>(at + 512 * j + 2 * t * 8 * D);
          const uint4 y4 = *reinterpret_cast<const uint4*>(at + 512 * j + (2 * t + 1) * 8 * D);
          const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t a0 = halves_lo(x[m]), a1 = halves_hi(x[m]), a2 = halves_lo(y[m]), a3 = halves_hi(y[m]);
            if (t == 0) mma16z(c[m], a0, a1, a2, a3, p.hi[t][0], p.hi[t][1]);
            else mma16(c[m], a0, a1, a2, a3, p.hi[t][0], p.hi[t][1]);
            if constexpr (PREC) {
              if (t == 0) mma16z(low[m], a0, a1, a2, a3, p.low[t][0], p.low[t][1]);
              else mma16(low[m], a0, a1, a2, a3, p.low[t][0], p.low[t][1]);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (PREC) c[m][e] = fmaf(low[m][e], 1.0f / kRest, c[m][e]);
            o[j][m][e] += c[m][e];
          }
      } else {
        float c[8][4];
#pragma unroll
        for (int t = 0; t < kPage / 16; ++t) {
          const uint4 x4 = *reinterpret_cast<const uint4*>(at + 512 * j + 2 * t * 8 * D);
          const uint4 y4 = *reinterpret_cast<const uint4*>(at + 512 * j + (2 * t + 1) * 8 * D);
          const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const uint32_t b0 = m & 1 ? halves_hi(x[m / 2]) : halves_lo(x[m / 2]), b1 = m & 1 ? halves_hi(y[m / 2]) : halves_lo(y[m / 2]);
            if (t == 0) mma16z(c[m], p.hi[t][0], p.hi[t][1], p.hi[t][2], p.hi[t][3], b0, b1);
            else mma16(c[m], p.hi[t][0], p.hi[t][1], p.hi[t][2], p.hi[t][3], b0, b1);
          }
        }
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][m][e] += c[m][e];
      }
    }
  }

  // Clears the codes of tokens live .. 63 of a page's values, which may be any bits, NaN among them.
  static __device__ __forceinline__ void clear(uint8_t* v, int live, int lane) {
    for (int n = live / 8 * (D / 2) + lane; n < kPage / 8 * (D / 2); n += 32) {
      const int t = n / (D / 2) * 8 + n % 4 * 2;
      if (t + 1 < live) continue;
      uint4* w = reinterpret_cast<uint4*>(v) + n;
      if (t >= live) {
        *w = make_uint4(0, 0, 0, 0);
      } else {
        const uint4 x = *w;
        *w = make_uint4(x.x & 0x00ff00ffu, x.y & 0x00ff00ffu, x.z & 0x00ff00ffu, x.w & 0x00ff00ffu);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy into the stage
    __syncwarp();
  }

  // The unit's sums: put(row, first channel, four sums) for every row and channel of this lane, then
  // stat(row, reference, sum) once a row.
  template <class Put, class Stat>
  __device__ __forceinline__ void finish(int g, int qd, Put put, Stat stat) {
    float a[2], s[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      a[n] = two_to((int)rf[n] - kOff);
      s[n] = l[n] * a[n];
#pragma unroll
      for (int d = kCols ? 4 : 1; d < (kCols ? 32 : 4); d *= 2) s[n] += __shfl_xor_sync(0xffffffffu, s[n], d);
    }
#pragma unroll
    for (int j = 0; j < kS; ++j)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int row = stat_row(n, g, qd);
        if constexpr (kCols) {
#pragma unroll
          for (int m = 0; m < 4; m += 2)
            put(row, 64 * j + 8 * g + 2 * m, s[n],
                make_float4(o[j][m][n] * a[n], o[j][m][2 + n] * a[n], o[j][m + 1][n] * a[n], o[j][m + 1][2 + n] * a[n]));
        } else {
#pragma unroll
          for (int m = 0; m < 16; m += 4)
            put(row, 64 * j + 16 * qd + m, s[n],
                make_float4(o[j][m % 8][2 * n + m / 8] * a[n], o[j][m % 8 + 1][2 * n + m / 8] * a[n], o[j][m % 8 + 2][2 * n + m / 8] * a[n],
                            o[j][m % 8 + 3][2 * n + m / 8] * a[n]));
        }
      }
    if (kCols ? g == 0 : qd == 0) {
#pragma unroll
      for (int n = 0; n < 2; ++n) stat(stat_row(n, g, qd), ref[n], s[n]);
    }
  }
};

// Eight sums of a row.
struct Sums {
  float4 x, y;
};
__device__ __forceinline__ Sums no_sums() { return Sums{make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)}; }
__device__ __forceinline__ void add(float4& o, float f, float4 y) {
  o.x = fmaf(f, y.x, o.x), o.y = fmaf(f, y.y, o.y), o.z = fmaf(f, y.z, o.z), o.w = fmaf(f, y.w, o.w);
}
// Adds a piece (its reference m, sum of weights l and eight of its sums y) to those of a row, whose reference is top.  (A piece
// without a reference may hold NaN, and keeps it.)
__device__ __forceinline__ void add_piece(Sums& o, float& sum, float top, float m, float l, const Sums& y) {
  const float f = m == -INFINITY ? 0.0f : ex2(m - top);
  sum = fmaf(f, l, sum);
  add(o.x, f, y.x), add(o.y, f, y.y);
}

// What a block knows of a piece it joins.
struct Piece {
  int base, unit, items;  // the unit's first item, the unit, its items
};

template <int D, int NT, int NW, int NS>
struct Smem {
  static constexpr int kRing = NS * Layout<D>::kHalf;
  static_assert(Partial<D, NT>::kFloats * 4 <= kRing, "a warp's piece goes into its ring");
  static_assert(2 * NW <= 32, "a lane a piece");
  // A piece of a unit that ends inside a warp's run, while copies into the ring are under way: beside the ring where there is
  // room for every warp's; else for the first kSlots that come, and of the others in global memory, from where a warp fetches
  // its own behind its other piece when its copies have ended.  (Long units leave a block one or two; with all of them in global
  // memory four drafted tokens of 16 sequences took 48.6 us, now 46.6.)
  static constexpr int kPiece = Partial<D, NT>::kFloats * 4;
  static constexpr int kSlots = NT == 1 ? NW : 3;
  static_assert(kSlots == NW || 2 * kPiece <= kRing, "both pieces in the ring");
  static constexpr size_t kBars = (size_t)NW * kRing, kInfoAt = kBars + 16 * ((NW * NS + 1) / 2), kScalesAt = kInfoAt + 16 * NW * kInfo,
                          kHeads = kScalesAt + 8 * NW * kInfo, kBytes = kHeads + (size_t)kSlots * kPiece;
  static_assert(kBytes <= 226 * 1024, "with the block's own variables at most 227 KB");
};

template <int D, int NT, bool PREC, int NW, int NS>
__global__ void __launch_bounds__(32 * NW, 1) attn_kernel(AttnArgs a) {
  using L = Layout<D>;
  using P = Partial<D, NT>;
  using S = Smem<D, NT, NW, NS>;
  using W = Warp<D, NT, PREC>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Piece piece_s[2 * NW];
  __shared__ uint32_t valid_s, start_s, end_s;
  __shared__ int total_s;
  __shared__ int last_s[2], first_s[2], at_s[2 * NW], slots_s;  // at_s: where a piece lies; slots_s: slots taken
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, qd = lane % 4, H = a.c.h_kv;
  uint8_t* ring = smem + (size_t)warp * S::kRing;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars) + warp * NS;
  int4* info = reinterpret_cast<int4*>(smem + S::kInfoAt) + warp * kInfo;
  float2* scales = reinterpret_cast<float2*>(smem + S::kScalesAt) + warp * kInfo;
  const int BC = a.c.batch * a.n_chunks;
  if (tid == 0) total_s = 0, slots_s = 0, valid_s = start_s = end_s = 0;
  if (lane < NS) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(bars + lane)) : "memory");
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  after_previous();

  // ---- the items of all units, and where this warp's run of them begins
  if (blockIdx.x == 0)
    for (int i = tid; i < a.c.batch; i += 32 * NW) check_length(a.c, i);
  const int c0 = lane < BC ? items_of(a, lane) : 0;  // of the first 32 (sequence, chunk) pairs
  int total;  // the host has made sure that all units' items fit
  bool empty;  // some unit has no key
  if (BC <= 32) {
    total = __reduce_add_sync(0xffffffffu, c0);
    empty = __any_sync(0xffffffffu, lane < BC && c0 == 0);
    __syncthreads();
  } else {
    int n = 0;
    bool none = false;
    __syncthreads();
    for (int i = tid; i < BC; i += 32 * NW) {
      const int c = items_of(a, i);
      n += c, none |= c == 0;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n) atomicAdd(&total_s, n);
    empty = __syncthreads_or(none);
    total = total_s;
  }
  total *= H;
  // a block for every kMinItems items: few items stay in few blocks
  const int nb = min((int)gridDim.x, ceil_div(total, kMinItems));
  const bool idle = (int)blockIdx.x >= nb;
  const int nw = nb * NW, me = blockIdx.x * NW + warp;
  const int w0 = idle ? 0 : share(me, total, nw), w1 = idle ? 0 : share(me + 1, total, nw), n_items = w1 - w0;
  int bc = 0, h = 0, p = 0, cnt = 0;  // the next item to look up
  if (BC == 1) {
    cnt = __shfl_sync(0xffffffffu, c0, 0);
    if (!idle) h = w0 / cnt, p = w0 - h * cnt;  // (an empty sequence: 0)
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
  // logical page, unit, and whether the item is its unit's first (1) or last (2).  Their scales are asked for and
  // waited for when they are needed.
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
      const int b = b1 / a.n_chunks;
      e.x = fetch(a.c.page_table + (int64_t)b * a.c.page_stride + p1);
      if (e.x < 0 || e.x >= a.c.n_pages) {
        raise(a.c, RDKV_ERR_INVALID_ARG);
        e.x = -1;
      } else {
        const int at = e.x * H + h1;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(scales + i % kInfo)), "l"(a.c.scales + (int64_t)at * 2)
                     : "memory");
        e.x = a.withhold && (p1 + h1) % a.withhold == 0 ? -2 : at;
      }
      e.y = p1, e.z = b1 * H + h1, e.w = (p1 == 0 ? 1 : 0) | (p1 == c1 - 1 ? 2 : 0);
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
  // With logits to keep, pages leave the L2 first: the launch that follows reads the logits, and each page is read once (or, by
  // several chunks of queries, at about the same time).
  uint64_t policy;
  if (a.logits) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
  // Copies half x of the run (the keys of item x / 2, or its values) into the stage that it falls in.
  auto issue = [&](int x, int stage) {
    const int i = x / 2;
    if (lane == 0) {
      const int4 e = info[i % kInfo];
      const uint32_t bar = smem_u32(bars + stage);
      if (e.x < 0) {
        if (e.x == -1) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
        else asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], 16;" ::"r"(bar) : "memory");
      } else {
        const uint8_t* src = a.c.pages + (int64_t)e.x * L::kBytes + (x & 1) * L::kHalf;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(L::kHalf) : "memory");
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                         smem_u32(ring + stage * L::kHalf)),
                     "l"(src), "r"(L::kHalf), "r"(bar), "l"(policy)
                     : "memory");
      }
    }
    __syncwarp();
  };

  bool away = false;  // this warp's such piece lies in global memory
  // Where the piece of a unit goes, one that ends inside the run or one that does not.
  auto piece_at = [&](bool ends) {
    int at = warp * S::kRing;
    if (ends) {
      int slot = warp;
      if constexpr (S::kSlots < NW) {
        if (lane == 0) slot = atomicAdd(&slots_s, 1);
        slot = __shfl_sync(0xffffffffu, slot, 0);
      }
      away = slot >= S::kSlots;
      at = away ? at + S::kPiece : (int)S::kHeads + slot * S::kPiece;
    }
    if (lane == 0) at_s[2 * warp + (ends ? 0 : 1)] = at;
    return ends && away ? a.heads + (int64_t)me * P::kFloats : reinterpret_cast<float*>(smem + at);
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
  W w;
  bool in_unit = false, began = false, ok = true;
  int held = 0;  // tokens of the unit's sequence
  int low[2];    // keys that this lane's rows see
  Unit un{0, 0, 0, 0};
  int i = 0, stage = 0, turn = 0;  // the next half's stage and the parity that its landing has
  auto next_stage = [&] {
    if (++stage == NS) stage = 0, turn ^= 1;
  };
  if (n_items > 0) {
    look_up(kInfo);
    // the first queries are asked for before the pages, behind which they would wait
    typename W::Rows x;
    un = unit_at(a, info[0].z);
    w.queries(a, un, g, qd, x);
#pragma unroll 1
    for (int j = 0; j < min(NS, 2 * n_items); ++j) issue(j, j);
    w.begin(a.dtype, x, qd);
    in_unit = true;
  }
  if (empty) {  // units without a key: nothing else writes their rows
#pragma unroll 1
    for (int u = warp * gridDim.x + blockIdx.x; u < BC * H; u += NW * gridDim.x)
      if (items_of(a, u / H) == 0) write_nothing<D>(a, unit_at(a, u), lane);
  }
  if (idle) return;
#pragma unroll 1
  for (; i < n_items; ++i) {
    // (once a turn and not where a copy is issued, twice in this loop: less code to fetch, 0.2 us of calls of a few pages)
    constexpr int kReach = (1 + NS) / 2;  // the items that this turn issues are not further ahead
    static_assert(kReach + kInfo / 2 < kInfo, "places that are still read");
    if (known <= i + kReach && known < n_items) look_up(kInfo / 2);
    const int4 e = info[i % kInfo];
    if (!in_unit) {
      typename W::Rows x;
      un = unit_at(a, e.z);
      w.queries(a, un, g, qd, x);
      w.begin(a.dtype, x, qd);
    }
    if (!in_unit || i == 0) {
      in_unit = true, began = e.w & 1;
      held = held_tokens(a.c, un.b);
#pragma unroll
      for (int n = 0; n < 2; ++n) low[n] = held - a.n_q + min(un.t0 + W::stat_row(n, g, qd) / a.G, a.n_q - 1) + 1;
    }
    if (!__all_sync(0xffffffffu, wait_for(bars + stage, turn, a.wait_cycles))) {  // the warp goes on, or stops, as one
      ok = false;
      break;
    }
    typename W::Logits s;
    if (e.x >= 0) w.logits(ring + stage * L::kHalf, g, qd, s);
    __syncwarp();
    if (2 * i + NS < 2 * n_items) issue(2 * i + NS, stage);
    next_stage();
    typename W::Weights pw;
    bool cut = false;
    if (e.x >= 0) {
      int see[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) see[n] = low[n] - e.y * kPage, cut |= see[n] < kPage;
      cut = __any_sync(0xffffffffu, cut);
      asm volatile("cp.async.wait_all;" ::: "memory");  // the scales
      __syncwarp();
      const float2 sc = scales[i % kInfo];
      float* store = a.logits ? a.logits + ((int64_t)e.z * a.c.page_stride + e.y) * a.rows * kPage : nullptr;
      w.weigh(s, sc, g, qd, cut, see, store, un.rows, pw);
    }
    if (!__all_sync(0xffffffffu, wait_for(bars + stage, turn, a.wait_cycles))) {
      ok = false;
      break;
    }
    if (e.x >= 0) {
      uint8_t* v = ring + stage * L::kHalf;
      const int live = held - e.y * kPage;
      if (live < kPage) W::clear(v, live, lane);
      w.values(v, g, qd, pw);
    }
    __syncwarp();
    if (2 * i + 1 + NS < 2 * n_items) issue(2 * i + 1 + NS, stage);
    next_stage();
    if ((e.w & 2) || i == n_items - 1) {  // the unit, or the run, ends
      const bool ends = e.w & 2;
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
        // a unit that ends here without having begun lies first in the run: copies are under way
        float* dst = piece_at(ends);
        w.finish(
            g, qd, [&](int row, int ch, float, float4 o) { *reinterpret_cast<float4*>(dst + row * D + ch) = o; },
            [&](int row, float m, float l) { dst[P::kRows * D + row] = m, dst[P::kRows * (D + 1) + row] = l; });
        if (lane == 0) leave_piece(i, e.z, began, ends);
      }
      in_unit = false;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!ok) {
    // A wait ran out: report it and let the copies under way land (again with a limit; a withheld one is none).  The
    // units of the rest of the run get pieces that hold nothing, so that their blocks' tickets come out even and the
    // workspace serves the next call.
    if (lane == 0) raise(a.c, RDKV_ERR_TIMEOUT);
    // the half that was waited for lies at `stage`: the keys of item i, or its values
    const int x0 = 2 * i + ((2 * i) % NS == stage ? 0 : 1);
#pragma unroll 1
    for (int x = x0; x < min(x0 + NS, 2 * n_items); ++x) {
      if (x / 2 < known && info[x / 2 % kInfo].x != -2) wait_for(bars + stage, turn, kWaitCycles);
      next_stage();
    }
    __syncwarp();
#pragma unroll 1
    for (; i < n_items; ++i) {
      if (i >= known) look_up(kInfo / 2);
      const int4 e = info[i % kInfo];
      if (!in_unit) in_unit = true, began = e.w & 1;
      if (!(e.w & 2) && i < n_items - 1) continue;
      const bool ends = e.w & 2;
      if (began && ends) {
        write_nothing<D>(a, unit_at(a, e.z), lane);
      } else {
        float* dst = piece_at(ends);
        for (int x = lane; x < P::kFloats; x += 32) dst[x] = x / P::kRows == D ? -INFINITY : 0.0f;
        if (lane == 0) leave_piece(i, e.z, began, ends);
      }
      in_unit = false;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  if (S::kSlots < NW && away) {
    __syncwarp();
    const float* head = a.heads + (int64_t)me * P::kFloats;
#pragma unroll 8
    for (int x = lane; x < P::kFloats / 4; x += 32) reinterpret_cast<float4*>(ring + S::kPiece)[x] = reinterpret_cast<const float4*>(head)[x];
  }
  __syncthreads();

  // ---- joining the block's pieces: runs of pieces of one unit, a run begins at a piece that holds its
  // unit's first item, or at the block's first piece.  (Short loops: the code is fetched once a call, and what unrolling
  // saves is less than the fetch of more of it.  A thread takes eight channels of a row, here and below, so that 8 or 16 rows take
  // one turn: with four channels and two turns 87.9 us where it now takes 86.2 for 262,144 tokens of 8 rows, 51.3 for 48.8 with 16 rows; a
  // few pages of 4 rows 9.9 for 10.2.)
  const uint32_t valid = valid_s, ends = end_s, begins = start_s;
  const uint32_t starts = begins | (valid & (0u - valid));
  int open0 = -1, open1 = -1;  // pieces of runs that are a part of their unit: one that began before the block, one that goes on
#pragma unroll 1
  for (uint32_t left = starts; left; left &= left - 1) {
    const int s = __ffs(left) - 1;
    const uint32_t rest = left & (left - 1), members = valid & ~((1u << s) - 1u) & (rest ? (rest & (0u - rest)) - 1u : 0xffffffffu);
    const int slot = begins >> s & 1;
    const bool whole = slot && (ends & members);
    const Unit ru = unit_at(a, piece_s[s].unit);
    float* part = a.parts + ((int64_t)blockIdx.x * 2 + slot) * P::kFloats;
#pragma unroll 1
    for (int i = tid; i < ru.rows * (D / 8); i += 32 * NW) {
      const int row = i / (D / 8), ch = i % (D / 8) * 8;
      auto src = [&](uint32_t m) -> const float* {
        return reinterpret_cast<const float*>(smem + at_s[__ffs(m) - 1]);
      };
      float m = -INFINITY, l = 0.0f;
#pragma unroll 1
      for (uint32_t x = members; x; x &= x - 1) m = fmaxf(m, src(x)[P::kRows * D + row]);
      Sums o = no_sums();
#pragma unroll 2
      for (uint32_t x = members; x; x &= x - 1) {
        const float* y = src(x);
        add_piece(o, l, m, y[P::kRows * D + row], y[P::kRows * (D + 1) + row], *reinterpret_cast<const Sums*>(y + row * D + ch));
      }
      if (whole) {
        const int64_t at = row_at(a, ru, row);
        put4(a, at * D + ch, scaled(o.x, l));
        put4(a, at * D + ch + 4, scaled(o.y, l));
        if (ch == 0) put_lse(a, at, m, l);
      } else {
        *reinterpret_cast<Sums*>(part + row * D + ch) = o;
        if (ch == 0) part[P::kRows * D + row] = m, part[P::kRows * (D + 1) + row] = l;
      }
    }
    if (!whole) (slot ? open1 : open0) = s;
  }
  // ---- joining the blocks' parts: the last block of a unit to arrive does it
  if (open0 < 0 && open1 < 0) return;
  __syncthreads();
  auto block_of = [&](int64_t item) { return quotient((item + 1) * nb - 1, total); };
  if (tid < 2) {
    const int e = tid ? open1 : open0;
    int n = 0;
    if (e >= 0) {
      const Piece pc = piece_s[e];
      const int first = block_of(pc.base);
      n = block_of(pc.base + pc.items - 1) - first + 1;
      int32_t* t = a.tickets + pc.unit;
      int before;
      asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(before) : "l"(t) : "memory");
      if (before == n - 1) *t = 0;
      else n = 0;
      first_s[tid] = first;
    }
    last_s[tid] = n;
  }
  __syncthreads();
#pragma unroll 1
  for (int slot = 0; slot < 2; ++slot) {
    const int n = last_s[slot];
    if (n == 0) continue;
    const Unit ru = unit_at(a, piece_s[slot ? open1 : open0].unit);
    // the unit's first block wrote it as the unit that goes on, the others as the one that began before
    const float* parts = a.parts + (int64_t)first_s[slot] * 2 * P::kFloats;
#pragma unroll 1
    for (int i = tid; i < ru.rows * (D / 8); i += 32 * NW) {
      const int row = i / (D / 8), ch = i % (D / 8) * 8;
      constexpr int kAhead = 10;  // parts whose loads are under way together
      Sums o = no_sums();
      float top = -INFINITY, sum = 0.0f;
#pragma unroll 1
      for (int j0 = 0; j0 < n; j0 += kAhead) {
        float m[kAhead], l[kAhead];
        Sums y[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const float* part = parts + (int64_t)(2 * (j0 + j) + (j0 + j == 0 ? 1 : 0)) * P::kFloats;
          const bool real = j0 + j < n;
          m[j] = real ? __ldcg(part + P::kRows * D + row) : -INFINITY;
          l[j] = real ? __ldcg(part + P::kRows * (D + 1) + row) : 0.0f;
          y[j].x = real ? __ldcg(reinterpret_cast<const float4*>(part + row * D + ch)) : make_float4(0, 0, 0, 0);
          y[j].y = real ? __ldcg(reinterpret_cast<const float4*>(part + row * D + ch) + 1) : make_float4(0, 0, 0, 0);
        }
        float now = top;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) now = fmaxf(now, m[j]);
        const Sums was = o;
        const float had = sum, ref = top;
        o = no_sums(), sum = 0.0f, top = now;
        add_piece(o, sum, now, ref, had, was);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) add_piece(o, sum, now, m[j], l[j], y[j]);
      }
      const int64_t at = row_at(a, ru, row);
      put4(a, at * D + ch, scaled(o.x, sum));
      put4(a, at * D + ch + 4, scaled(o.y, sum));
      if (ch == 0) put_lse(a, at, top, sum);
    }
  }
}

// ---------------------------------------------------------------- the keys' weights
// mass_t += sum over the query rows that see t of 2^(logit - reference) / sum, chunk after chunk and row after row.
// A thread four positions of a (sequence, KV head); the loads of eight rows under way together, the first with the rows'
// statistics, the weights so far and the page table.
//   Bound: the logits.  With the stores of the launch before it 29 us beside the attention's 86 at 262,144 tokens of 64 heads
// (67 MB of logits, 17 MB of weights), 7.4 beside 40 for sixteen sequences of 8,192 of 32 heads.  The grid is the table's: blocks behind
// a sequence's end fetch its length and return (16 x 4,160 tokens: 4.6 beside 31 in their own
// tables, 34 in tables of 131,072).  With the logits by key
// instead of by row, and pages that pushed them out of the L2, 44 and 17; with two keys a thread 30.5 and 9.
constexpr int kMassThreads = 128, kMassKeys = 4 * kMassThreads;
constexpr int kMassRows = kMaxQueries * 8;
__global__ void __launch_bounds__(kMassThreads) mass_kernel(AttnArgs a, float* mass, int64_t mass_stride) {
  __shared__ float2 stat_s[kMassRows];
  after_previous();
  const int H = a.c.h_kv, rows = a.n_q * a.G, tid = threadIdx.x;
  const int tiles = ceil_div(a.c.page_stride, kMassKeys / kPage), bh = blockIdx.x / tiles, b = bh / H, h = bh - b * H;
  const int t = (int)(blockIdx.x % tiles) * kMassKeys + 4 * tid, held = held_tokens(a.c, b);
  if (t - 4 * tid >= held) return;
  const bool real = t < held;
  float* to = mass + ((int64_t)b * H + h) * mass_stride + t;
  // (a wait that ran out: the logits are not all there; a page outside the pool: nothing was attended there)
  const int page = real ? fetch(a.c.page_table + (int64_t)b * a.c.page_stride + t / kPage) : -1, status = fetch(a.c.status);
  const uint2 had0 = real ? fetch(reinterpret_cast<const uint2*>(to)) : make_uint2(0, 0);
  const uint2 had1 = real ? fetch(reinterpret_cast<const uint2*>(to + 2)) : make_uint2(0, 0);
  constexpr int kAhead = 8;
  uint4 w[kAhead];
  auto load = [&](int c, int r0, int m, int seen) {
    const float* u = a.logits + (((((int64_t)b * a.n_chunks + c) * H + h) * a.c.page_stride + t / kPage) * a.rows + r0) * kPage + t % kPage;
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      constexpr uint32_t kHidden = 0xff800000u;  // (a page's logits are all there as soon as one of its keys is seen)
      w[r] = t < seen && r0 + r < m ? fetch(reinterpret_cast<const uint4*>(u + r * kPage)) : make_uint4(kHidden, kHidden, kHidden, kHidden);
    }
  };
  auto rows_of = [&](int c) { return min(a.chunk, a.n_q - c * a.chunk) * a.G; };
  load(0, 0, rows_of(0), seen_by(a, b, 0));
  for (int i = tid; i < rows; i += kMassThreads) {
    const int q = i / a.G;
    const uint2 x = fetch(reinterpret_cast<const uint2*>(a.stats + (((int64_t)b * a.n_q + q) * H + h) * a.G + i - q * a.G));
    const float l = __uint_as_float(x.y);
    stat_s[i] = make_float2(__uint_as_float(x.x), l > 0.0f && l < INFINITY ? 1.0f / l : 0.0f);
  }
  __syncthreads();
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = 0; c < a.n_chunks; ++c) {
    const int m = rows_of(c), seen = seen_by(a, b, c);
    const float2* st = stat_s + c * a.chunk * a.G;
#pragma unroll 1
    for (int r0 = 0; r0 < m; r0 += kAhead) {
      if (c || r0) load(c, r0, m, seen);
#pragma unroll
      for (int r = 0; r < kAhead; ++r) {
        const float2 s = r0 + r < m ? st[r0 + r] : make_float2(0.0f, 0.0f);
        if (s.y > 0.0f) {
          const uint32_t x[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[k] = fmaf(ex2(__uint_as_float(x[k]) - s.x), s.y, sum[k]);
        }
      }
    }
  }
  if (page < 0 || page >= a.c.n_pages || status == RDKV_ERR_TIMEOUT) return;
  const uint32_t had[4] = {had0.x, had0.y, had1.x, had1.y};
#pragma unroll
  for (int k = 0; k < 4; ++k) sum[k] += __uint_as_float(had[k]);
  if (t + 3 < held) {
    reinterpret_cast<float2*>(to)[0] = make_float2(sum[0], sum[1]), reinterpret_cast<float2*>(to)[1] = make_float2(sum[2], sum[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (t + k < held) to[k] = sum[k];
  }
}

// ---------------------------------------------------------------- launch
// The workspace has the same places for every shape, so that calls of any shape may follow one another: the
// tickets, then pieces of the largest variant; last, for calls with mass, the rows' statistics and the logits.
constexpr int kMaxWarps = 8;

struct Geometry {
  int chunk, n_chunks, nt, grid, rows;
  size_t heads_at, parts_at, stats_at, logits_at, bytes;
};

static Geometry geometry(const rdkv_q8_cache* c, int h_q, int n_q, bool prec, bool with_mass) {
  Geometry o;
  const int G = h_q / c->h_kv;
  // Query tokens that share one pass over the keys: as many as fit in 16 rows (8 for fp32 outputs, whose
  // registers hold two parts of queries and weights)
  o.chunk = std::min(n_q, std::max(1, (prec ? 8 : 16) / G));
  o.n_chunks = ceil_div(n_q, o.chunk);
  o.rows = o.chunk * G;
  o.nt = o.rows > 8 ? 2 : 1;
  o.grid = num_sms();
  const int64_t part = 4LL * Partial<128, 2>::kFloats;
  o.heads_at = kCounterBytes;
  o.parts_at = o.heads_at + (size_t)align_up((int64_t)o.grid * kMaxWarps * part, 256);
  o.stats_at = o.parts_at + (size_t)align_up(2LL * o.grid * part, 256);
  o.logits_at = o.stats_at + (with_mass ? (size_t)align_up(8LL * c->batch * n_q * h_q, 256) : 0);
  o.bytes = o.logits_at + (with_mass ? 4ull * c->batch * c->h_kv * o.n_chunks * o.rows * c->page_stride * kPage : 0);
  return o;
}

template <int D, int NT, bool PREC, int NW, int NS>
static rdkv_status launch(const AttnArgs& a, int grid, cudaStream_t cs) {
  using S = Smem<D, NT, NW, NS>;
  static_assert(NW <= kMaxWarps, "the workspace counts with kMaxWarps");
  auto kernel = attn_kernel<D, NT, PREC, NW, NS>;
  // once a device (of the first 64; the others pay for the call every time)
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  RDKV_TRY_CUDA(cudaGetDevice(&dev), "8-bit cache attention");
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    RDKV_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes), "8-bit cache attention");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  RDKV_TRY_CUDA(launch_after(kernel, dim3(grid), 32 * NW, S::kBytes, cs, a), "8-bit cache attention");
  count_launch();
  return RDKV_OK;
}

}  // namespace q8
}  // namespace rdkv

using namespace rdkv;
using namespace rdkv::q8;

extern "C" size_t rdkv_q8_attn_workspace_bytes(const rdkv_q8_cache* cache, int32_t h_q, int32_t n_q, int32_t with_mass) {
  if (check_cache(cache) != RDKV_OK || check_heads_of(cache, h_q, n_q) != RDKV_OK) return 0;
  // (of 16-bit and of fp32 outputs)
  return std::max(geometry(cache, h_q, n_q, false, with_mass != 0).bytes, geometry(cache, h_q, n_q, true, with_mass != 0).bytes);
}

// withhold > 0: the self-test
static rdkv_status attn_impl(const rdkv_q8_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q, int32_t n_q,
                             float* mass, int64_t mass_stride, void* out, int32_t out_dtype, float* lse, void* ws, size_t ws_bytes,
                             void* stream, int withhold, long long wait_cycles) {
  rdkv_status st = check_cache(cache);
  if (st == RDKV_OK) st = check_heads_of(cache, h_q, n_q);
  if (st == RDKV_OK) st = check_queries_of(cache, dtype, q, q_stride, h_q);
  if (st == RDKV_OK && mass) st = check_mass(cache, mass, mass_stride);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(out != nullptr, RDKV_ERR_INVALID_ARG, "NULL output");
  RDKV_REQUIRE((uintptr_t)out % 16 == 0, RDKV_ERR_INVALID_ARG, "out must be 16-byte aligned");
  RDKV_REQUIRE(out_dtype == dtype || out_dtype == RDKV_F32, RDKV_ERR_UNSUPPORTED, "out_dtype %d for dtype %d", out_dtype, dtype);
  RDKV_REQUIRE((int64_t)cache->batch * cache->h_kv * n_q * cache->page_stride <= INT32_MAX, RDKV_ERR_UNSUPPORTED,
               "more than 2^31 - 1 (sequence, query token, KV head, page) items");
  const bool prec = out_dtype == RDKV_F32;
  const Geometry geo = geometry(cache, h_q, n_q, prec, mass != nullptr);
  RDKV_REQUIRE(ws && (uintptr_t)ws % 16 == 0 && ws_bytes >= geo.bytes, RDKV_ERR_WORKSPACE,
               "attention workspace too small (%zu < %zu) or unaligned", ws_bytes, geo.bytes);
  char* w = static_cast<char*>(ws);
  const AttnArgs a{q8::view_of(cache), q, out, lse, mass ? reinterpret_cast<float*>(w + geo.logits_at) : nullptr,
                   mass ? reinterpret_cast<float2*>(w + geo.stats_at) : nullptr, reinterpret_cast<float*>(w + geo.heads_at),
                   reinterpret_cast<float*>(w + geo.parts_at), reinterpret_cast<int32_t*>(w), q_stride, dtype, out_dtype, n_q,
                   h_q / cache->h_kv, geo.chunk, geo.n_chunks, geo.rows, withhold, wait_cycles};
  cudaStream_t cs = (cudaStream_t)stream;
  const bool wide = cache->head_dim == 128;
  if (prec) st = (wide ? launch<128, 1, true, 7, 3> : launch<64, 1, true, 7, 6>)(a, geo.grid, cs);
  else if (geo.nt == 2) st = (wide ? launch<128, 2, false, 8, 3> : launch<64, 2, false, 8, 6>)(a, geo.grid, cs);
  else st = (wide ? launch<128, 1, false, 7, 3> : launch<64, 1, false, 7, 6>)(a, geo.grid, cs);
  if (st != RDKV_OK || !mass) return st;
  const int64_t tiles = (int64_t)ceil_div(cache->page_stride, kMassKeys / kPage) * cache->batch * cache->h_kv;  // (no more than items)
  RDKV_TRY_CUDA(launch_after(mass_kernel, dim3((unsigned)tiles), kMassThreads, 0, cs, a, mass, mass_stride),
                "8-bit cache weights");
  count_launch();
  return RDKV_OK;
}

extern "C" rdkv_status rdkv_q8_attn(const rdkv_q8_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q,
                                    int32_t n_q, float* mass, int64_t mass_stride, void* out, int32_t out_dtype, float* lse, void* ws,
                                    size_t ws_bytes, void* stream) {
  return attn_impl(cache, dtype, q, q_stride, h_q, n_q, mass, mass_stride, out, out_dtype, lse, ws, ws_bytes, stream, 0, kWaitCycles);
}

extern "C" rdkv_status rdkv_q8_timeout_selftest(const rdkv_q8_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q,
                                                int32_t n_q, void* out, int32_t out_dtype, float* lse, void* ws, size_t ws_bytes,
                                                int32_t withhold, int64_t wait_cycles, void* stream) {
  RDKV_REQUIRE(withhold >= 1, RDKV_ERR_INVALID_ARG, "withhold %d must be positive", withhold);
  RDKV_REQUIRE(wait_cycles > 0, RDKV_ERR_INVALID_ARG, "wait_cycles %lld must be positive", (long long)wait_cycles);
  return attn_impl(cache, dtype, q, q_stride, h_q, n_q, nullptr, 0, out, out_dtype, lse, ws, ws_bytes, stream, withhold,
                   std::min(kWaitCycles, std::max(kMinWaitCycles, (long long)wait_cycles)));
}
