// Attention over the 4-bit paged cache (rdkv_q4_attn).
#include "q4.cuh"

namespace rdkv {
namespace q4 {

struct AttnArgs {
  View c;
  const void* q;
  void* out;
  float* lse;
  const int32_t* sel;
  int64_t q_stride;
  int dtype, out_dtype, n_q, G, n_sel;
};

// One block per (sequence, query token, KV head): page after page, the logits of the group's heads by
// a dot product a (token, head), then the running softmax and the values, a channel a thread.
template <int D>
__global__ void __launch_bounds__(128) attn_kernel(AttnArgs a) {
  using L = Layout<D>;
  constexpr int NG = L::NG;
  __shared__ float q_s[8][D], p_s[8][kPage], k_s[kPage][D + 1], m_s[8], l_s[8], f_s[8];
  const int h = blockIdx.x % a.c.h_kv, bt = blockIdx.x / a.c.h_kv, t = bt % a.n_q, b = bt / a.n_q, tid = threadIdx.x;
  const int held = held_tokens(a.c, b), seen = held - a.n_q + t + 1;
  const int64_t qrow = ((int64_t)b * a.n_q + t) * a.q_stride + (int64_t)h * a.G * D;
  for (int i = tid; i < a.G * D; i += 128) q_s[i / D][i % D] = load_q(a.q, qrow + i, a.dtype);
  if (tid < 8) m_s[tid] = -INFINITY, l_s[tid] = 0.0f;
  float o[8] = {};
  const int n_pages = seen > 0 ? ceil_div(seen, kPage) : 0, n = a.sel ? a.n_sel : n_pages;
  const int32_t* sel = a.sel ? a.sel + ((int64_t)bt * a.c.h_kv + h) * a.n_sel : nullptr;
  for (int i = 0; i < n; ++i) {
    const int lp = sel ? sel[i] : i;
    if (lp < 0 || lp >= n_pages) continue;
    const int phys = a.c.page_table[(int64_t)b * a.c.page_stride + lp];
    if (phys < 0 || phys >= a.c.n_pages) {
      if (tid == 0) raise(a.c, RDKV_ERR_INVALID_ARG);
      continue;
    }
    const uint8_t* page = a.c.pages + ((int64_t)phys * a.c.h_kv + h) * L::kBytes;
    const int live = min(kPage, seen - lp * kPage);
    __syncthreads();
    for (int j = tid; j < kPage * D; j += 128) {
      const int s = j / D, c = j % D, grp = c / 32, e = c % 8, q = c % 32 / 8;
      const uint32_t w = reinterpret_cast<const uint32_t*>(page + L::kKCodes)[(s * 4 + q) * NG + grp];
      const uint32_t code = (w >> (16 * (e & 1) + 4 * (e >> 1))) & 15u;
      k_s[s][c] = fmaf(__half2float(reinterpret_cast<const __half*>(page + L::kKScales)[(s / 2 * NG + grp) * 2 + s % 2]),
                       (float)code, __half2float(reinterpret_cast<const __half*>(page + L::kKZeros)[s * NG + grp]));
    }
    __syncthreads();
    for (int j = tid; j < a.G * kPage; j += 128) {
      const int g = j / kPage, s = j % kPage;
      float x = 0.0f;
      for (int c = 0; c < D; ++c) x = fmaf(q_s[g][c], k_s[s][c], x);
      p_s[g][s] = s < live ? x * rsqrtf((float)D) : -INFINITY;
    }
    __syncthreads();
    if (tid < a.G) {
      float m = m_s[tid];
      for (int s = 0; s < live; ++s) m = fmaxf(m, p_s[tid][s]);
      const float f = expf(m_s[tid] - m);
      float l = l_s[tid] * f;
      for (int s = 0; s < kPage; ++s) {
        const float p = s < live ? expf(p_s[tid][s] - m) : 0.0f;
        p_s[tid][s] = p;
        l += p;
      }
      m_s[tid] = m, l_s[tid] = l, f_s[tid] = f;
    }
    __syncthreads();
    if (tid < D) {
      const int c = tid, grp = c / 32, g8 = c % 32 / 4, j4 = c % 4;
      for (int g = 0; g < a.G; ++g) o[g] *= f_s[g];
      for (int s = 0; s < live; ++s) {
        const int m = (s / 2 * NG + grp) * 2 + s % 2;
        const uint32_t w = reinterpret_cast<const uint16_t*>(page + L::kVCodes)[((s / 2 * 8 + g8) * NG + grp) * 2 + s % 2];
        const float x = fmaf(__half2float(reinterpret_cast<const __half*>(page + L::kVScales)[m]), (float)((w >> (4 * j4)) & 15u),
                             __half2float(reinterpret_cast<const __half*>(page + L::kVZeros)[m]));
        for (int g = 0; g < a.G; ++g) o[g] = fmaf(p_s[g][s], x, o[g]);
      }
    }
  }
  __syncthreads();
  const int64_t row = (int64_t)bt * a.c.h_kv * a.G + (int64_t)h * a.G;
  if (tid < D)
    for (int g = 0; g < a.G; ++g) store_as(a.out, (row + g) * D + tid, a.out_dtype, l_s[g] > 0.0f ? o[g] / l_s[g] : 0.0f);
  if (a.lse && tid < a.G) a.lse[row + tid] = l_s[tid] > 0.0f ? m_s[tid] + logf(l_s[tid]) : -INFINITY;
}

}  // namespace q4
}  // namespace rdkv

using namespace rdkv;
using namespace rdkv::q4;

extern "C" size_t rdkv_q4_attn_workspace_bytes(const rdkv_q4_cache* cache, int32_t h_q, int32_t n_q) {
  return check_queries(cache, h_q, n_q) == RDKV_OK ? 256 : 0;
}

extern "C" rdkv_status rdkv_q4_attn(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q,
                                    int32_t n_q, const int32_t* sel, int32_t n_sel, void* out, int32_t out_dtype, float* lse,
                                    void* ws, size_t ws_bytes, void* stream) {
  rdkv_status st = check_q(cache, dtype, q, q_stride, h_q, n_q);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(out != nullptr, RDKV_ERR_INVALID_ARG, "NULL output");
  RDKV_REQUIRE((uintptr_t)out % 16 == 0, RDKV_ERR_INVALID_ARG, "out must be 16-byte aligned");
  RDKV_REQUIRE(out_dtype == dtype || out_dtype == RDKV_F32, RDKV_ERR_UNSUPPORTED, "out_dtype %d for dtype %d", out_dtype, dtype);
  RDKV_REQUIRE(!sel || n_sel >= 1, RDKV_ERR_INVALID_ARG, "n_sel %d", n_sel);
  const size_t need = rdkv_q4_attn_workspace_bytes(cache, h_q, n_q);
  RDKV_REQUIRE(ws && (uintptr_t)ws % 16 == 0 && ws_bytes >= need, RDKV_ERR_WORKSPACE, "attention workspace too small (%zu < %zu) or unaligned",
               ws_bytes, need);
  AttnArgs a{view_of(cache), q, out, lse, sel, q_stride, dtype, out_dtype, n_q, h_q / cache->h_kv, n_sel};
  const unsigned blocks = (unsigned)((int64_t)cache->batch * n_q * cache->h_kv);
  if (cache->head_dim == 64) attn_kernel<64><<<blocks, 128, 0, (cudaStream_t)stream>>>(a);
  else attn_kernel<128><<<blocks, 128, 0, (cudaStream_t)stream>>>(a);
  RDKV_CHECK_LAUNCH("4-bit cache attention");
  return RDKV_OK;
}
